"""convrot_cache_append and convrot_cache_read on a B200: the cells to the bits of
convrot_quant_act, what they stand for against the oracle.

A value read back is (sum of signed codes, exact) * (scale / sqrt(128)): three
float32 roundings and the output's half step.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle
from parity import OUT_ABS, OUT_REL, check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cr():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_rotated_int8_token_b200 as cr

    cr.lib()
    return cr


def _dtype(kind):
    import torch

    return torch.bfloat16 if kind == "bf16" else torch.float16


def _heads(T, H, kind, seed, pad=0):
    """K and V [T, H, 128] as parts of a projection's rows; a zero vector and an outlier channel among them."""
    import torch

    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn(T, pad + 2 * H, 128, generator=g, device="cuda")
    rows[..., 9] *= 40.0
    if T > 2:
        rows[1, pad] = 0.0
        rows[2] *= 1e-3
    rows = rows.to(_dtype(kind))
    return rows[:, pad:pad + H], rows[:, pad + H:]


def _cell(cache, slots):
    """(k codes, v codes, k scale, v scale) of slots, token by token."""
    page = cache.page_size
    s = slots.long()
    return [t[s // page, :, s % page] for t in cache.cells]


@pytest.mark.parametrize("kind,T,H,page,pad", [("bf16", 1, 1, 16, 0), ("f16", 16, 8, 16, 32), ("bf16", 333, 3, 32, 5),
                                               ("f16", 1027, 2, 1024, 0), ("bf16", 129, 5, 64, 1)])
def test_append_then_read(cr, kind, T, H, page, pad):
    import torch

    K, V = _heads(T, H, kind, T, pad)
    cache = cr.ConvRotCache(2 * (T // page + 1), H, page)
    for t in cache.cells:
        t.fill_(77)
    capacity = cache.k_codes.shape[0] * page
    g = torch.Generator("cuda").manual_seed(T)
    slots = torch.randperm(capacity, generator=g, device="cuda")[:T].to(torch.int32)
    skipped = torch.arange(T, device="cuda") % 7 == 3
    slots[skipped] = -1 - torch.arange(T, device="cuda", dtype=torch.int32)[skipped]
    kept = ~skipped
    cache.append(K, V, slots)
    cells = _cell(cache, slots[kept])
    for X, codes, scale in ((K, cells[0], cells[2]), (V, cells[1], cells[3])):
        X = X[kept].reshape(-1, 128)
        want_codes, want_scale = cr.convrot_quant_act_ex(X, 128)
        assert torch.equal(codes.reshape(-1, 128), want_codes)
        assert torch.equal(scale.reshape(-1), want_scale)
        turned = oracle.rotate(X.double().cpu().numpy(), 128)
        check_codes(codes.reshape(-1, 128).cpu().numpy(), scale.reshape(-1).cpu().numpy(), turned,
                    *oracle.quantize_per_token(turned))
    # every other cell is as it was
    for t in cache.cells:
        flat = t.transpose(1, 2).reshape(capacity, -1).clone()
        flat[slots[kept].long()] = 77
        assert bool((flat == 77).all())
    for out in ("bf16", "f16"):
        k, v = cache.read(slots, _dtype(out))
        for x, codes, scale in ((k, cells[0], cells[2]), (v, cells[1], cells[3])):
            ref = oracle.cache_value(codes.cpu().numpy(), scale.cpu().numpy())
            got = x[kept].double().cpu().numpy()
            # where the signed codes cancel to 0 the kernel gives 0 and the oracle its own rounding: sums of 128
            # products, each off by 2^-53 of up to 128 * 127 s / sqrt(128), with a step for the matrix's rounding
            own = 2 * 128 * 2.0**-53 * 128 * 127 / np.sqrt(128.0) * scale.cpu().numpy().astype(np.float64)[..., None]
            assert np.all(np.abs(got - ref) <= (OUT_REL[out] + 2.0**-22) * np.abs(ref) + OUT_ABS[out] + own)
            assert not bool(x[skipped].any())
    cache.check()


def test_read_strided_repeated_and_head_major(cr):
    import torch

    K, V = _heads(50, 4, "bf16", 1)
    cache = cr.ConvRotCache(4, 4, 16)
    slots = torch.arange(50, dtype=torch.int32, device="cuda")
    cache.append(K, V, slots)
    again = torch.tensor([3, 3, 49, -1, 0, 3], dtype=torch.int32, device="cuda")
    k, v = cache.read(again)
    all_k, all_v = cache.read(slots)
    assert torch.equal(k[[0, 1, 5]], all_k[[3, 3, 3]]) and torch.equal(v[2], all_v[49]) and not bool(k[3].any())
    heads = torch.full((2, 4, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")  # room for two more tokens
    cache.read(again, K=heads[0, :, :6].transpose(0, 1), V=heads[1, :, :6].transpose(0, 1))
    assert torch.equal(heads[0, :, :6].transpose(0, 1), k) and torch.equal(heads[1, :, :6].transpose(0, 1), v)
    assert bool((heads[:, :, 6:] == 5.0).all())


def test_slots_past_the_cache_are_skipped_and_reported(cr):
    import torch

    K, V = _heads(6, 2, "f16", 2)
    cache = cr.ConvRotCache(2, 2, 16)
    slots = torch.tensor([0, 32, 5, 2**31 - 1, -2**31, 31], dtype=torch.int32, device="cuda")
    cr.convrot_cache_append(K, V, slots, *cache.cells)  # without a status word
    fine = torch.tensor([0, 5, 31], device="cuda")
    k, v = cr.convrot_cache_read(slots, *cache.cells, dtype=torch.float16)
    assert not bool(k[[1, 3, 4]].any()) and not bool(v[[1, 3, 4]].any()) and bool(k[[0, 2, 5]].any())
    used = torch.zeros(32, dtype=torch.bool, device="cuda")
    used[fine] = True
    assert not bool(cache.k_scale.transpose(1, 2).reshape(32, 2)[~used].any())
    cache.check()
    cache.append(K, V, slots)
    with pytest.raises(cr.ConvRotError) as e:
        cache.check()
    assert e.value.status == 1
    cache.status.zero_()
    cache.read(slots)
    with pytest.raises(cr.ConvRotError):
        cache.check()


def test_no_tokens(cr):
    import torch

    cache = cr.ConvRotCache(1, 2, 16)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    cache.append(x, x, none)
    assert cache.read(none)[0].shape == (0, 2, 128)


def test_bad_arguments_are_refused(cr):
    import torch

    K, V = _heads(8, 2, "bf16", 3)
    cache = cr.ConvRotCache(2, 2, 16)
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    for bad in (dict(K=K[:7]), dict(K=K.half()), dict(K=K.float()), dict(V=V[:, :1]), dict(slots=slots.long()),
                dict(slots=slots[:7]), dict(slots=slots.cpu()), dict(K=K[..., ::2])):
        args = dict(K=K, V=V, slots=slots) | bad
        with pytest.raises((ValueError, TypeError)):
            cache.append(**args)
    with pytest.raises(ValueError):
        cr.convrot_cache_append(K, V, slots, cache.k_codes[:1], *cache.cells[1:])
    with pytest.raises(ValueError):
        cr.convrot_cache_append(K, V, slots, *cache.cells[:2], cache.k_scale.transpose(0, 1), cache.v_scale)
    with pytest.raises(cr.ConvRotError) as e:  # pages of 24 tokens
        cr.ConvRotCache(2, 2, 24).append(K, V, slots)
    assert e.value.status == 2
    with pytest.raises(cr.ConvRotError) as e:  # vectors off 16 bytes
        wide = torch.zeros(8, 2, 136, dtype=K.dtype, device="cuda")
        cache.append(wide[..., 4:132], V, slots)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        cache.read(slots, K=K[:, :1].expand(8, 2, 128))


def test_captured_and_on_another_stream(cr):
    import torch

    K, V = _heads(40, 4, "bf16", 4)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    cache = cr.ConvRotCache(4, 4, 16)
    cache.append(K, V, slots)
    want = cache.read(slots)
    side = torch.cuda.Stream()
    other = cr.ConvRotCache(4, 4, 16)
    side.wait_stream(torch.cuda.current_stream())
    other.append(K, V, slots, stream=side)
    got = other.read(slots, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    k, v = K.clone(), V.clone()
    out = [torch.empty_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.append(k, v, slots)
        other.read(slots, K=out[0], V=out[1])
    k.copy_(V)
    v.copy_(K)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[1]) and torch.equal(out[1], want[0])
    del graph


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_read_any_codes(cr, kind):
    """Cells filled by hand: each sign pattern of the transform, the largest sums, -128 among the codes."""
    import torch

    cache = cr.ConvRotCache(20, 1, 16)
    g = torch.Generator("cuda").manual_seed(11)
    for codes, scale in (cache.cells[::2], cache.cells[1::2]):
        codes.copy_(torch.randint(-128, 128, codes.shape, generator=g, device="cuda"))
        scale.copy_(torch.rand(scale.shape, generator=g, device="cuda") * 0.01)
    flat = cache.k_codes.view(320, 128)
    i = torch.arange(128)
    for c in range(128):  # row c: the signs of channel c, the sum 127 * 128 in one place
        flat[c] = torch.tensor([127 if bin(c & int(j)).count("1") % 2 == 0 else -127 for j in i], dtype=torch.int8)
    flat[128:256] = 0
    flat[128 + i, i] = 1  # one code at each channel
    flat[256] = -128
    slots = torch.arange(320, dtype=torch.int32, device="cuda")
    k, v = cache.read(slots, _dtype(kind))
    for x, codes, scale in ((k, cache.k_codes, cache.k_scale), (v, cache.v_codes, cache.v_scale)):
        codes, scale = codes.view(320, 1, 128).cpu().numpy(), scale.view(320, 1).cpu().numpy()
        ref = oracle.cache_value(codes, scale)
        own = 2 * 128 * 2.0**-53 * 128 * 128 / np.sqrt(128.0) * scale.astype(np.float64)[..., None]  # the oracle's, as above
        assert np.all(np.abs(x.double().cpu().numpy() - ref) <= (OUT_REL[kind] + 2.0**-22) * np.abs(ref) + OUT_ABS[kind] + own)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_read_with_a_last_warp_partly_without_tokens(cr, kind):
    """Every count of vectors in the last warp (eight fill it), some of them without a cell: the bits of a read in
    which each warp is full, and nothing behind the last token written."""
    import torch

    K, V = _heads(32, 1, kind, 5)
    cache = cr.ConvRotCache(2, 1, 16)
    slots = torch.randperm(32, device="cuda").to(torch.int32)
    cache.append(K, V, slots)
    full = cache.read(slots, _dtype(kind))
    for T in range(1, 18):
        some = slots[:T].clone()
        some[T // 2] = -1
        room = torch.full((2, 32, 1, 128), 3.0, dtype=_dtype(kind), device="cuda")
        got = cache.read(some, K=room[0, :T], V=room[1, :T])
        for x, want, rest in zip(got, full, room):
            want = want[:T].clone()
            want[T // 2] = 0.0
            assert torch.equal(x, want) and bool((rest[T:] == 3.0).all())


@pytest.mark.parametrize("native", [True, False])
def test_autograd_learns_of_outputs_written(cr, monkeypatch, native):
    """An operation that keeps a tensor for its gradient learns that a read or an attention has overwritten it."""
    import torch

    if not native:
        for name in ("read", "attention"):
            monkeypatch.setattr(cr._T, name, lambda *a: None)
    K, V = _heads(4, 2, "bf16", 6)
    cache = cr.ConvRotCache(1, 2, 16)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    cache.append(K, V, slots)
    pages = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([4], dtype=torch.int32, device="cuda")

    def write(at):
        room = [torch.ones(4, 2, 128, dtype=K.dtype, device="cuda") for _ in range(3)]
        w = torch.ones(4, 2, 128, dtype=K.dtype, device="cuda", requires_grad=True)
        out = (w * room[at]).sum()
        if at < 2:
            cache.read(slots, K=room[0], V=room[1])
        else:
            cache.attention(K[:1], pages, lengths, O=room[2][:1])
        return out

    for at in range(3):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            write(at).backward()


def test_vectors_that_the_kernels_cannot_take_are_named(cr):
    import torch

    K, V = _heads(4, 2, "bf16", 6)
    cache = cr.ConvRotCache(1, 2, 16)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    pages = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    lengths = torch.ones(4, dtype=torch.int32, device="cuda")
    wide = torch.zeros(4, 2, 136, dtype=K.dtype, device="cuda")
    odd = torch.zeros(4, 2, 132, dtype=K.dtype, device="cuda")[..., :128]  # strides of 132
    for bad in (wide[..., 4:132], odd):
        for call, name in ((lambda: cache.append(bad, V, slots), "K"), (lambda: cache.append(K, bad, slots), "V"),
                           (lambda: cache.read(slots, K=bad), "K"), (lambda: cache.read(slots, V=bad), "V"),
                           (lambda: cache.attention(bad, pages, lengths), "Q"),
                           (lambda: cache.attention(K, pages, lengths, O=bad), "O")):
            with pytest.raises(cr.ConvRotError, match=f": {name} must start on 16 bytes") as e:
                call()
            assert e.value.status == 1
    with pytest.raises(cr.ConvRotError) as e:
        cache.attention(K, pages, lengths, softmax_scale=-1.0)
    assert "16 bytes" not in str(e.value)
