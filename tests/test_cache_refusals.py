"""What the rope and cache entry points refuse, on the host (no GPU: nothing is launched)."""

from __future__ import annotations

import pytest

FAKE = 0x10000  # aligned and never dereferenced: every call fails validation or has nothing to do


@pytest.fixture(scope="module")
def L():
    from w8a8_rotated_int8_token_b200 import _lib, build

    build.build()
    return _lib.load()


def _caller(fn, layout, names, values):
    """A call of `fn` with a struct of the named fields, some of them other than `values`; its status."""
    names = names.split()
    assert len(names) == len(values)

    def call(**over):
        assert set(over) <= set(names)
        return fn(layout.pack(*[over.get(n, v) for n, v in zip(names, values)]), None)

    return call


CELLS = "kc vc ks vs pages H page D "
CELLS_OK = [FAKE, FAKE, FAKE, FAKE, 8, 2, 64, 128]


def test_structs_are_laid_out_as_the_compiler_does(tmp_path):
    import os
    import subprocess

    from w8a8_rotated_int8_token_b200 import _lib, build

    ends = {"convrot_rope_args": ("inverse", _lib.ROPE_ARGS), "convrot_cache_args": ("dtype", _lib.CACHE_ARGS),
            "convrot_cache_attention_args": ("dtype", _lib.CACHE_ATTENTION_ARGS)}
    mids = {"convrot_rope_args": ("axes", "@5P5q6q"), "convrot_cache_args": ("T", "@4P4q4P"),
            "convrot_cache_attention_args": ("ws_bytes", "@4P4q7P")}
    import struct

    lines = [f'printf("%zu %zu\\n", offsetof({t}, {ends[t][0]}), offsetof({t}, {mids[t][0]}));' for t in ends]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "convrot.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [[int(v) for v in ln.split()] for ln in subprocess.run([str(exe)], capture_output=True, text=True,
                                                                 check=True).stdout.splitlines()]
    assert got == [[ends[t][1].size - 4, struct.calcsize(mids[t][1])] for t in ends]


def test_no_arguments(L):
    for fn in (L.convrot_rope, L.convrot_cache_append, L.convrot_cache_read, L.convrot_cache_attention):
        assert fn(None, None) == 1


def test_rope(L):
    from w8a8_rotated_int8_token_b200 import _lib

    call = _caller(L.convrot_rope, _lib.ROPE_ARGS, "X Y pos freq axis B S H D R xb xs xh yb ys yh axes pa pb ps dtype "
                   "pos_dtype inter inverse",
                   [FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 2, 128, 128, 0, 256, 128, 0, 256, 128, 3, 4, 0, 1, 0, 0, 0, 0])
    assert call(dtype=2) == 2 and call(pos_dtype=2) == 2
    assert call(R=127) == 1 and call(R=130) == 1 and call(R=-2) == 1
    assert call(H=0) == 1 and call(D=0, R=0) == 1 and call(B=-1) == 1 and call(S=-1) == 1 and call(axes=0) == 1
    assert call(D=514) == 2 and call(H=65536) == 2 and call(B=1 << 20, S=1 << 12) == 2 and call(axes=1 << 31) == 2
    for name in ("X", "Y", "pos", "freq", "axis"):
        assert call(**{name: 0}) == 1, name
    assert call(X=FAKE + 1) == 1 and call(pos=FAKE + 2) == 1 and call(freq=FAKE + 4) == 1 and call(axis=FAKE + 2) == 1
    assert call(S=0, X=0, Y=0, pos=0) == 0 and call(B=0) == 0
    assert call(S=0, R=127) == 1


def test_append_and_read(L):
    from w8a8_rotated_int8_token_b200 import _lib

    for fn in (L.convrot_cache_append, L.convrot_cache_read):
        call = _caller(fn, _lib.CACHE_ARGS, CELLS + "K V slots status T kt kh vt vh dtype",
                       [*CELLS_OK, FAKE, FAKE, FAKE, 0, 4, 256, 128, 256, 128, 0])
        assert call(dtype=3) == 2 and call(D=64) == 2
        assert call(page=8) == 2 and call(page=48) == 2 and call(page=2048) == 2 and call(page=0) == 1
        assert call(pages=0) == 1 and call(H=0) == 1 and call(T=-1) == 1
        assert call(H=1025) == 2 and call(pages=1 << 25) == 2 and call(T=1 << 29) == 2
        assert call(kt=4) == 1 and call(vh=12) == 1
        for name in ("K", "V", "slots", "kc", "vc", "ks", "vs"):
            assert call(**{name: 0}) == 1, name
        assert call(K=FAKE + 8) == 1 and call(slots=FAKE + 2) == 1 and call(kc=FAKE + 8) == 1 and call(vs=FAKE + 8) == 1
        assert call(status=FAKE + 2) == 1
        assert call(T=0, K=0, V=0, slots=0) == 0 and call(T=0, D=64) == 2


def test_attention(L):
    from w8a8_rotated_int8_token_b200 import _lib

    call = _caller(L.convrot_cache_attention, _lib.CACHE_ATTENTION_ARGS,
                   CELLS + "Q O table lengths starts tree ws ws_bytes T Hq B cols stride qt qh ot oh scale dtype",
                   [*CELLS_OK, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 1 << 30, 4, 8, 4, 3, 3, 1024, 128, 1024, 128, 0.1, 0])
    assert call(dtype=2) == 2 and call(D=64) == 2
    assert call(Hq=7) == 1 and call(H=0) == 1 and call(Hq=0) == 1 and call(pages=0) == 1 and call(cols=-1) == 1
    assert call(stride=-1) == 1 and call(page=24) == 2 and call(page=4096) == 2 and call(page=0) == 1
    assert call(T=5) == 1  # one token per sequence without starts
    assert call(T=5, starts=FAKE, B=(1 << 24) + 1) == 2 and call(T=(1 << 20) + 1, starts=FAKE) == 2
    assert call(pages=1 << 24) == 2 and call(cols=1 << 28) == 2 and call(Hq=2 * 1025) == 2
    assert call(scale=0.0) == 1 and call(scale=-1.0) == 1 and call(scale=float("inf")) == 1
    assert call(scale=float("nan")) == 1
    assert call(qt=1020) == 1 and call(oh=4) == 1
    for name in ("Q", "O", "kc", "vc", "ks", "vs", "lengths", "table"):
        assert call(**{name: 0}) == 1, name
    assert call(Q=FAKE + 8) == 1 and call(lengths=FAKE + 2) == 1 and call(starts=FAKE + 1) == 1
    assert call(tree=FAKE + 4) == 1
    assert call(ws=0) == 3 and call(ws=FAKE + 16) == 3 and call(ws_bytes=4096) == 3
    assert call(T=0, B=0, Q=0, O=0, ws=0) == 0 and call(T=0, starts=FAKE, Q=0, O=0, ws=0) == 0
    assert call(T=0, B=0, Hq=7) == 1


def test_attention_workspace(L):
    size = L.convrot_cache_attention_workspace_bytes
    assert size(0, 0, 8, 2, 128) == 256
    assert size(4, 4, 8, 2, 64) == 0 and size(4, 4, 7, 2, 128) == 0 and size(-1, 4, 8, 2, 128) == 0
    # a row of sums per piece's two ends: 640 pieces, tiles of 8 or 16 rows
    assert size(4, 4, 8, 2, 128) >= 2 * 640 * 8 * 128 * 4
    assert size(64, 4, 8, 2, 128) >= 2 * 640 * 16 * 128 * 4


def test_binding_refuses_before_the_library():
    import torch

    import w8a8_rotated_int8_token_b200 as cr

    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    cells = (torch.zeros(2, 2, 16, 128, dtype=torch.int8),) * 2 + (torch.zeros(2, 2, 16),) * 2
    for call in (lambda: cr.convrot_rope(x, i[None], *cr.convrot_rope_tables([64], device="cpu")),
                 lambda: cr.convrot_cache_append(x, x, i, *cells),
                 lambda: cr.convrot_cache_read(i, *cells),
                 lambda: cr.convrot_cache_attention(x, *cells, i[:, None], i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        cr.convrot_rope(x.float(), i[None], None, None)
    with pytest.raises(ValueError):
        cr.convrot_rope_tables([4, -1], device="cpu")


def test_rope_tables():
    import numpy as np
    import torch

    import w8a8_rotated_int8_token_b200 as cr

    freq, axis = cr.convrot_rope_tables([1, 2, 0, 1], theta=100.0, device="cpu")
    assert axis.dtype == torch.int32 and axis.tolist() == [0, 1, 1, 3]
    np.testing.assert_allclose(freq.numpy(), [1.0, 1.0, 0.1, 1.0], rtol=1e-15)
    freq, _ = cr.convrot_rope_tables([1, 2, 0, 1], theta=16.0, shared=True, device="cpu")
    np.testing.assert_allclose(freq.numpy(), [1.0, 0.5, 0.25, 0.125], rtol=1e-15)


def test_cache_slots():
    import torch

    import w8a8_rotated_int8_token_b200 as cr

    cache = cr.ConvRotCache(4, 1, 16, device="cpu")
    pages = torch.tensor([[3, 1], [2, -1]], dtype=torch.int32)
    seq = torch.tensor([0, 0, 1, 1, 0, 2, -1, 0])
    pos = torch.tensor([0, 17, 15, 16, 32, 0, 0, -1])
    assert cache.slots(pages, seq, pos).tolist() == [48, 17, 47, -1, -1, -1, -1, -1]
    assert cache.slots(pages[:, :0], seq, pos).tolist() == [-1] * 8


def test_native_binding_leaves_other_calls_to_python(L):
    """Built, of this torch, bound to the library; what it does not take it hands back without a launch."""
    import torch

    from w8a8_rotated_int8_token_b200 import _lib

    b = _lib.binding()
    assert b is not None
    x = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    i32, f64 = torch.zeros((3, 4), dtype=torch.int32), torch.zeros((4,), dtype=torch.float64)
    c, s = torch.zeros((1, 2, 16, 128), dtype=torch.int8), torch.zeros((1, 2, 16))
    assert b.rope(x, i32, f64, i32[0], False, False, None) is None
    assert b.append(x[0], x[0], i32[0], c, c, s, s, None) is None
    assert b.read(i32[0], c, c, s, s, 0, None, None, None) is None
    assert b.attention(x[0], c, c, s, s, i32, i32[0], None, None, None, None, None) is None
    for fn, n in ((b.rope, 7), (b.append, 8), (b.read, 9), (b.attention, 12)):
        assert fn(*[None] * n) is None and fn(*[0] * n) is None and fn() is None
    with pytest.raises(TypeError):
        b.bind(1)


def test_attention_with_a_status_and_a_limit(L):
    from w8a8_rotated_int8_token_b200 import _lib

    args = _lib.CACHE_ATTENTION_ARGS.pack(*CELLS_OK, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 1 << 30, 0, 8, 0, 3, 3, 1024, 128,
                                          1024, 128, 0.1, 0)  # no tokens: nothing is launched
    assert L.convrot_cache_attention_ex(args, None, 0, None) == 0
    assert L.convrot_cache_attention_ex(args, FAKE, 1000, None) == 0
    assert L.convrot_cache_attention_ex(args, FAKE + 2, 0, None) == 1
    assert L.convrot_cache_attention_ex(args, None, -1, None) == 1
    assert L.convrot_cache_attention_ex(None, None, 0, None) == 1


def test_binding_without_its_status_argument_is_left_to_python(L):
    from w8a8_rotated_int8_token_b200 import _lib

    b = _lib.binding()
    assert b.attention(*[None] * 12) is None and b.attention(*[None] * 13) is None


def test_a_softmax_scale_that_overflows_in_base_2(L):
    """Times log2(e) it is infinite, and an all-zero query's equal logits 0 * inf."""
    from w8a8_rotated_int8_token_b200 import _lib

    def status(scale):  # no tokens: what is fine returns 0
        args = _lib.CACHE_ATTENTION_ARGS.pack(*CELLS_OK, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 1 << 30, 0, 8, 0, 3, 3, 1024,
                                              128, 1024, 128, scale, 0)
        return L.convrot_cache_attention(args, None)

    assert status(2.3e38) == 0 and status(2.4e38) == 1 and status(2.9e38) == 1


def test_queries_of_no_sequence_need_a_workspace(L):
    """Their call clears its status word, as every call with tokens writes it."""
    from w8a8_rotated_int8_token_b200 import _lib

    for ws, size in ((0, 1 << 20), (FAKE + 16, 1 << 20), (FAKE, 255)):
        args = _lib.CACHE_ATTENTION_ARGS.pack(*CELLS_OK, FAKE, FAKE, FAKE, FAKE, FAKE, 0, ws, size, 4, 8, 0, 3, 3, 1024, 128,
                                              1024, 128, 0.1, 0)
        assert L.convrot_cache_attention(args, None) == 3


def test_cache_slots_of_pages_past_the_cache():
    """They stay past it, where the append reports them, also where 32 bits would bring them back to its first slots."""
    import torch

    import w8a8_rotated_int8_token_b200 as cr

    cache = cr.ConvRotCache(4, 1, 64, device="cpu")
    pages = torch.tensor([[4, 1 << 26, (1 << 26) + 1, 2**31 - 1, -2**31, 3]], dtype=torch.int32)
    at = torch.arange(6) * 64 + 5
    got = cache.slots(pages, torch.zeros(6, dtype=torch.int64), at)
    assert got.dtype == torch.int32
    assert got.tolist() == [4 * 64 + 5, 2**31 - 1, 2**31 - 1, 2**31 - 1, -1, 3 * 64 + 5]


def test_workspace_of_each_tile_height(L):
    """Parts of 640 pieces of 8 or 16 rows, of 160 pieces of 128."""
    size = L.convrot_cache_attention_workspace_bytes
    part = lambda pieces, rows: 2 * pieces * rows * 128 * 4  # noqa: E731
    few, some, many = size(4, 4, 8, 2, 128), size(32, 4, 8, 2, 128), size(33, 4, 8, 2, 128)
    assert part(640, 8) <= few < part(640, 16) <= some < part(160, 128) <= many < 2 * part(160, 128)
