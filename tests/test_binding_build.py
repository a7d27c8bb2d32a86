"""The native form of the binding: what it may be used with, and the build without it (no GPU)."""

from __future__ import annotations

import os
import types

import pytest


@pytest.fixture(scope="module")
def L():
    from w8a8_rotated_int8_token_b200 import _lib, build

    build.build()
    return _lib.load()


def test_library_and_binding_carry_the_hash_of_one_header(L):
    import hashlib

    from w8a8_rotated_int8_token_b200 import _lib, build

    with open(os.path.join(build.ROOT, "include", "convrot.h"), "rb") as f:
        want = hashlib.sha256(f.read()).hexdigest()[:16]
    assert L.convrot_header() == want.encode() and _lib.binding().header == want


@pytest.mark.parametrize("other", [dict(header="0123456789abcdef"), dict(header=""), dict(torch_version="1.0")])
def test_a_binding_of_another_build_is_not_used(L, monkeypatch, other):
    """Struct layouts of another header, or of another torch: the Python form serves, nothing is bound."""
    import w8a8_rotated_int8_token_b200 as cr

    real = cr._lib.binding()
    bound = []
    fake = types.SimpleNamespace(header=real.header, torch_version=real.torch_version, bind=lambda *a: bound.append(a))
    monkeypatch.setattr(cr, "_binding", fake)
    assert cr._lib.binding() is fake and len(bound) == 1
    for name, value in other.items():
        setattr(fake, name, value)
    assert cr._lib.binding() is None and len(bound) == 1
    delattr(fake, next(iter(other)))  # one that does not say
    assert cr._lib.binding() is None and len(bound) == 1


def test_the_file_names_its_python():
    import sysconfig

    from w8a8_rotated_int8_token_b200 import build

    assert "cpython" in sysconfig.get_config_var("EXT_SUFFIX")
    assert build.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """build() into a folder of its own, with compilers that write what they are asked for, or fail."""
    from w8a8_rotated_int8_token_b200 import build

    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libconvrot.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_binding.so"))

    def compiler(name, variable, works):
        path = tmp_path / name
        path.write_text("#!/bin/sh\n" + ('while [ "$1" != -o ]; do shift; done; echo made > "$2"\n' if works else
                                         "echo no such header >&2; exit 1\n"))
        path.chmod(0o755)
        monkeypatch.setenv(variable, str(path))

    compiler("nvcc", "NVCC", True)
    compiler("g++", "CXX", True)
    return build, compiler


def test_build_makes_both(tools, recwarn):
    build, _ = tools
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BINDING_PATH) and not recwarn.list


def test_build_without_torch_makes_the_library(tools, monkeypatch):
    import sys

    build, _ = tools
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)


def test_a_binding_that_does_not_compile_is_a_warning(tools):
    build, compiler = tools
    with open(build.BINDING_PATH, "w") as f:
        f.write("of older sources")
    compiler("g++", "CXX", False)
    with pytest.warns(UserWarning, match="Python form of the binding(.|\n)*no such header"):
        assert build.build(force=True) == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)


def test_a_compiler_that_is_not_there_is_a_warning_for_the_binding(tools, monkeypatch):
    build, _ = tools
    monkeypatch.setenv("CXX", "/nowhere/g++")
    with pytest.warns(UserWarning, match="Python form of the binding"):
        assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)


def test_a_library_that_does_not_compile_is_an_error(tools):
    build, compiler = tools
    compiler("nvcc", "NVCC", False)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert not os.path.exists(build.LIB_PATH)


@pytest.mark.gpu
def test_an_error_behind_a_launch_is_not_answered_by_a_second_one():
    """A library that launches and then reports a CUDA error (one left by an earlier call will do): the call is not
    repeated in Python, which would turn heads in place twice."""
    import ctypes

    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_rotated_int8_token_b200 as cr

    heads = torch.randn(5, 2, 128, device="cuda").bfloat16()
    pos = torch.arange(5, dtype=torch.int32, device="cuda").view(1, 5)
    freq, axis = cr.convrot_rope_tables([64])
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    cache = cr.ConvRotCache(1, 2, 16)
    pages, lengths = torch.zeros(5, 1, dtype=torch.int32, device="cuda"), torch.ones(5, dtype=torch.int32, device="cuda")
    native = cr._lib.binding()
    assert native is not None
    real = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        cr.lib().convrot_rope, cr.lib().convrot_cache_append, cr.lib().convrot_cache_read,
        cr.lib().convrot_cache_attention_ex, cr.lib().convrot_cache_attention_workspace_bytes)]
    calls = [(lambda: cr.convrot_rope(heads, pos, freq, axis, Y=heads), "convrot_rope"),
             (lambda: cache.append(heads, heads, slots), "convrot_cache_append"),
             (lambda: cache.read(slots), "convrot_cache_read"),
             (lambda: cache.attention(heads, pages, lengths), "convrot_cache_attention")]
    for call, _ in calls:
        call()  # the native form is bound
    was = [t.clone() for t in (heads, *cache.cells)]
    seen = []
    three = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)
    four = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p)
    fails = three(lambda *a: seen.append(0) or 4), four(lambda *a: seen.append(0) or 4)
    at = [ctypes.cast(f, ctypes.c_void_p).value for f in fails]
    try:
        native.bind(at[0], at[0], at[0], at[1], real[4])
        for call, name in calls:
            with pytest.raises(cr.ConvRotError, match=name) as e:
                call()
            assert e.value.status == 4 and len(seen) == 1
            seen.clear()
    finally:
        native.bind(*real)
    assert all(torch.equal(a, b) for a, b in zip(was, (heads, *cache.cells)))
