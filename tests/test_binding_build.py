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
