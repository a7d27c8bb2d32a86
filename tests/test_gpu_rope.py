"""convrot_rope against the oracle's complex products, on a B200.

Tolerance of an element, from the pair (a, b) it is made of: the output's half
step, and float32 errors relative to |a| + |b|: 2 pi 2^-26 of the reduced angle,
2 units of 2^-24 in the sine or cosine, 2 in the product and sum: 3.4e-7, taken
as 5e-7.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle
from parity import OUT_ABS, OUT_REL

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


def _check(cr, X, pos, freq, axis, kind, interleaved, inverse, Y):
    """Y against the oracle; X [B, S, H, D], pos [axes, S] or [axes, B, S] on the GPU."""
    x = X.double().cpu().numpy()
    p = pos.double().cpu().numpy()
    if p.ndim == 2:
        p = np.repeat(p[:, None], x.shape[0], 1)
    ax = axis.cpu().numpy()
    ref = oracle.rope(x, p, freq.cpu().numpy(), ax, interleaved, inverse)
    size = np.zeros_like(x)
    half = len(ax)
    for i in range(half):
        if 0 <= ax[i] < len(p):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    y = Y.double().cpu().numpy()
    bound = OUT_REL[kind] * np.abs(ref) + 5e-7 * size + OUT_ABS[kind]
    bound[..., 2 * half:] = 0.0
    assert np.all(np.abs(y - ref) <= bound), np.max(np.abs(y - ref) / np.maximum(bound, 1e-300))


def _inputs(B, S, H, D, kind, seed, pad=0, far=100000):
    import torch

    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn(B, S, (H + pad) * D, generator=g, device="cuda").to(_dtype(kind))
    pos = torch.randint(0, far, (3, B, S), generator=g, device="cuda", dtype=torch.int32)
    return rows[..., :H * D].view(B, S, H, D), pos


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("kind,B,S,H,D,sections", [
    ("bf16", 16, 1, 40, 128, (16, 24, 24)), ("f16", 1, 1, 1, 128, (64, 0, 0)), ("bf16", 2, 77, 3, 64, (8, 12, 12)),
    ("f16", 1, 1500, 3, 128, (8, 28, 28)), ("bf16", 1, 130, 33, 128, (0, 16, 16)), ("f16", 1, 9, 5, 256, (32, 48, 48)),
    ("bf16", 1, 1100, 1, 256, (128, 0, 0)), ("f16", 1, 50, 7, 96, (16, 16, 16)), ("bf16", 1, 12, 2, 512, (256, 0, 0)),
    # the slower kernel: odd numbers of pairs and channels
    ("bf16", 2, 5, 3, 80, (4, 8, 8)), ("f16", 1, 7, 2, 7, (1, 1, 1)), ("bf16", 1, 3, 2, 36, (6, 6, 6)),
    ("f16", 1, 300, 70, 6, (3, 0, 0))])
def test_rope(cr, kind, B, S, H, D, sections, interleaved, inverse):
    X, pos = _inputs(B, S, H, D, kind, S + D, pad=2)
    freq, axis = cr.convrot_rope_tables(sections)
    Y = cr.convrot_rope(X, pos, freq, axis, interleaved, inverse)
    assert Y.is_contiguous() and Y.shape == X.shape
    _check(cr, X, pos, freq, axis, kind, interleaved, inverse, Y)


def test_no_pairs_copies(cr):
    import torch

    X, pos = _inputs(1, 5, 3, 128, "bf16", 1)
    freq, axis = cr.convrot_rope_tables([0])
    assert torch.equal(cr.convrot_rope(X, pos[:1], freq, axis), X)


def test_empty(cr):
    freq, axis = cr.convrot_rope_tables([32])
    for shape in ((2, 0, 3, 64), (0, 4, 3, 64)):
        X, pos = _inputs(*shape, "f16", 1)
        assert cr.convrot_rope(X, pos[:1], freq, axis).shape == shape


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_head_major_and_shared_positions(cr, interleaved):
    import torch

    X, pos = _inputs(2, 40, 6, 128, "bf16", 3, pad=1)
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    shared = pos[:, 0]
    Y = cr.convrot_rope(X, shared, freq, axis, interleaved)
    _check(cr, X, shared, freq, axis, "bf16", interleaved, False, Y)
    heads = torch.empty(2, 6, 40, 128, dtype=X.dtype, device="cuda")
    cr.convrot_rope(X, shared, freq, axis, interleaved, Y=heads.transpose(1, 2))
    assert torch.equal(heads.transpose(1, 2), Y)
    # three dimensions, positions with a stride
    wide = torch.zeros(3, 80, dtype=torch.int32, device="cuda")
    wide[:, ::2] = shared
    assert torch.equal(cr.convrot_rope(X[1], wide[:, ::2], freq, axis, interleaved), Y[1])
    # the rest of a row stays as it was
    base = torch.cat([X.reshape(2, 40, -1), torch.full((2, 40, 128), 7.0, device="cuda", dtype=X.dtype)], -1)
    view = base[..., :6 * 128].view(2, 40, 6, 128)
    cr.convrot_rope(view, shared, freq, axis, interleaved, Y=view)
    assert torch.equal(view, Y) and bool((base[..., 6 * 128:] == 7.0).all())


def test_unaligned_views_take_the_slower_kernel(cr):
    import torch

    X, pos = _inputs(1, 33, 4, 129, "f16", 4)
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    for view in (X[..., 1:], X[..., :128]):
        _check(cr, view, pos, freq, axis, "f16", False, False, cr.convrot_rope(view, pos, freq, axis))
    flat = torch.empty(33 * 4 * 128 + 1, dtype=X.dtype, device="cuda")
    Y = flat[1:].view(1, 33, 4, 128)
    cr.convrot_rope(X[..., 1:], pos, freq, axis, Y=Y)
    _check(cr, X[..., 1:], pos, freq, axis, "f16", False, False, Y)


def test_far_and_fractional_positions(cr):
    import torch

    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    X, _ = _inputs(1, 64, 2, 128, "f16", 5)
    far = torch.randint(-2**31, 2**31 - 1, (3, 64), device="cuda", dtype=torch.int32)
    _check(cr, X, far, freq, axis, "f16", False, False, cr.convrot_rope(X, far, freq, axis))
    part = (torch.rand(3, 64, device="cuda") - 0.5) * 3000.0
    _check(cr, X, part, freq, axis, "f16", False, False, cr.convrot_rope(X, part, freq, axis))


def test_pairs_of_no_axis_are_not_turned(cr):
    import torch

    X, pos = _inputs(1, 20, 2, 128, "bf16", 6)
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    axis[3], axis[40] = -1, 3
    Y = cr.convrot_rope(X, pos, freq, axis)
    _check(cr, X, pos, freq, axis, "bf16", False, False, Y)
    assert torch.equal(Y[..., 3], X[..., 3]) and torch.equal(Y[..., 104], X[..., 104])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(cr, interleaved):
    """<G, rope(D)> = <rope inverse(G), D> for every direction D: with one-hot D both sides are single
    elements, each within its half step of the exact product (bound as above, twice)."""
    X, pos = _inputs(1, 6, 1, 64, "f16", 7)
    freq, axis = cr.convrot_rope_tables([8, 12, 12])
    import torch

    eye = torch.eye(64, dtype=X.dtype, device="cuda").view(1, 64, 1, 64).repeat(1, 6, 1, 1)  # six tokens x 64 directions
    where = pos.repeat_interleave(64, dim=2)
    J = cr.convrot_rope(eye.view(1, 384, 1, 64), where, freq, axis, interleaved).view(6, 64, 64).double()
    G = X.view(6, 64)
    by_parts = torch.einsum("tde,te->td", J, G.double())
    grad = cr.convrot_rope(X, pos, freq, axis, interleaved, inverse=True).view(6, 64).double()
    assert bool(((grad - by_parts).abs() <= 2 * 2.0**-11 * (G.double().abs().amax() * 2) + 1e-6).all())


def test_bad_outputs_are_refused(cr):
    import torch

    X, pos = _inputs(1, 4, 2, 64, "bf16", 8)
    freq, axis = cr.convrot_rope_tables([8, 12, 12])
    for Y in (X[:, :1].expand(1, 4, 2, 64), X.half(), X[:, :3], X.cpu()):
        with pytest.raises((ValueError, TypeError)):
            cr.convrot_rope(X, pos, freq, axis, Y=Y)
    with pytest.raises(ValueError):
        cr.convrot_rope(X, pos[:, :, :3], freq, axis)
    with pytest.raises(TypeError):
        cr.convrot_rope(X, pos.long(), freq, axis)
    with pytest.raises(TypeError):
        cr.convrot_rope(X, pos, freq.float(), axis)
    with pytest.raises(ValueError):
        cr.convrot_rope(X, pos, freq.cpu(), axis.cpu())
    with pytest.raises(ValueError):
        cr.convrot_rope(X, pos, *cr.convrot_rope_tables([33]))


def test_captured_and_on_another_stream(cr):
    import torch

    X, pos = _inputs(1, 200, 8, 128, "bf16", 9)
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    Y = cr.convrot_rope(X, pos, freq, axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z = cr.convrot_rope(X, pos, freq, axis, stream=side)
    W = cr.convrot_rope(X, pos, freq, axis, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(Z, Y) and torch.equal(W, Y)
    held, out = X.clone(), torch.empty_like(X)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_rope(held, pos, freq, axis, Y=out)
    held.copy_(X.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, Y.flip(2))
    del graph


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_pairs_of_no_axis_are_copied_whatever_they_hold(cr, kind, interleaved, shift):
    """To the bit: an infinity beside a number, NaN, and zeros of either sign; the other pairs are turned as ever.
    Off 16 bytes (shift) the scalar kernel does the same."""
    import torch

    X, pos = _inputs(1, 20, 9, 136, kind, 10)
    X = X[..., 4 * shift:][..., :128]
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    want = cr.convrot_rope(X, pos, freq, axis, interleaved)
    off = torch.tensor([0, 3, 17, 40, 41, 63], device="cuda")
    axis[off] = torch.tensor([-1, 3, -2**31, 2**31 - 1, 4, -1], dtype=torch.int32, device="cuda")
    first = 2 * off if interleaved else off
    second = 2 * off + 1 if interleaved else off + 64
    odd = torch.tensor([float("inf"), -0.0, float("nan"), 0.0, -float("inf"), 1.0], dtype=X.dtype, device="cuda")
    X[..., first] = odd
    X[..., second] = odd.flip(0) * -1.0
    Y = cr.convrot_rope(X, pos, freq, axis, interleaved)
    both = torch.cat([first, second])
    assert torch.equal(Y[..., both].view(torch.int16), X[..., both].view(torch.int16))
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[both] = False
    assert torch.equal(Y[..., rest], want[..., rest])


@pytest.mark.parametrize("kind,interleaved,D,R", [("bf16", False, 128, 128), ("f16", True, 128, 64), ("f16", False, 36, 30)])
def test_autograd_records_it(cr, kind, interleaved, D, R):
    """The gradient is the inverse's, of any gradient of the output: also a strided or broadcast one, of heads turned in
    place, of heads written into a buffer of another order, and of the gradient itself."""
    import torch

    X, pos = _inputs(2, 9, 3, D, kind, 11, pad=1)
    sizes = [R // 2 - 2 * (R // 6), R // 6, R // 6]
    freq, axis = cr.convrot_rope_tables(sizes)
    G = torch.randn_like(X, memory_format=torch.contiguous_format)
    x = X.detach().clone().requires_grad_()
    y = cr.convrot_rope(x, pos, freq, axis, interleaved)
    assert torch.equal(y.detach(), cr.convrot_rope(X, pos, freq, axis, interleaved))
    y.backward(G)
    _check(cr, G, pos, freq, axis, kind, interleaved, True, x.grad)
    want = x.grad.clone()

    def gradient(make, g=G):
        x = X.detach().clone().requires_grad_()
        return torch.autograd.grad(make(x), x, g)[0]

    def in_place(x):
        z = x * 1
        assert cr.convrot_rope(z, pos, freq, axis, interleaved, Y=z) is z
        return z

    def head_major(x):
        room = torch.empty(2, 3, 9, D, dtype=X.dtype, device="cuda")
        cr.convrot_rope(x, pos, freq, axis, interleaved, Y=room.transpose(1, 2))
        return room.transpose(1, 2)

    def three(x):
        return torch.stack([cr.convrot_rope(x[b], pos[:, b], freq, axis, interleaved) for b in range(2)])

    side = torch.cuda.Stream()

    def elsewhere(x):
        side.wait_stream(torch.cuda.current_stream())
        out = cr.convrot_rope(x, pos, freq, axis, interleaved, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        return out

    def part_of_a_row(x):  # in place in a view, beside what stays
        rows = torch.cat([x, x * 0], 2)
        part = rows[:, :, :3]
        cr.convrot_rope(part, pos, freq, axis, interleaved, Y=part)
        return rows[:, :, :3]

    for make in (in_place, head_major, three, elsewhere, part_of_a_row):
        assert torch.equal(gradient(make), want), make
    turned = lambda x: cr.convrot_rope(x, pos, freq, axis, interleaved)  # noqa: E731
    strided = G.transpose(1, 3).contiguous().transpose(1, 3)
    assert strided.stride(-1) != 1 and torch.equal(gradient(turned, strided), want)
    ones = gradient(lambda x: turned(x).sum(), None)
    assert torch.equal(ones, cr.convrot_rope(torch.ones_like(X), pos, freq, axis, interleaved, inverse=True))
    # what is overwritten has no gradient, what stands beside it keeps its own
    x, w = X.detach().clone().requires_grad_(), torch.randn(2, 9, 4, D, device="cuda").to(X.dtype).requires_grad_()
    rows = w * 1
    cr.convrot_rope(x, pos, freq, axis, interleaved, Y=rows[:, :, 1:])
    dx, dw = torch.autograd.grad(rows[:, :, 1:], (x, w), G, retain_graph=True)
    assert torch.equal(dx, want) and not bool(dw.any())
    dw = torch.autograd.grad(rows.sum(), w)[0]
    assert bool((dw[:, :, 0] == 1).all()) and not bool(dw[:, :, 1:].any())
    # through the inverse, and the gradient's own gradient
    back = lambda x: cr.convrot_rope(x, pos, freq, axis, interleaved, inverse=True)  # noqa: E731
    assert torch.equal(gradient(back), cr.convrot_rope(G, pos, freq, axis, interleaved))
    x, g = X.detach().clone().requires_grad_(), G.clone().requires_grad_()
    dx = torch.autograd.grad(turned(x), x, g, create_graph=True)[0]
    assert torch.equal(torch.autograd.grad(dx, g, G)[0], cr.convrot_rope(G, pos, freq, axis, interleaved))


def test_autograd_against_elementary_operations(cr):
    """In float64, of the same pairs: the kernel's gradient is within its rounding."""
    import torch

    X, pos = _inputs(1, 7, 2, 64, "f16", 12)
    freq, axis = cr.convrot_rope_tables([8, 12, 12])
    G = torch.randn_like(X, memory_format=torch.contiguous_format)
    x = X.detach().clone().requires_grad_()
    cr.convrot_rope(x, pos, freq, axis).backward(G)
    z = X.detach().double().requires_grad_()
    angle = (pos.double()[axis.long()].permute(1, 2, 0) * freq)[:, :, None, :]
    a, b = z[..., :32], z[..., 32:]
    torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).backward(G.double())
    pair = G.double().abs().view(1, 7, 2, 2, 32).sum(-2, keepdim=True).expand(1, 7, 2, 2, 32).reshape(1, 7, 2, 64)
    bound = OUT_REL["f16"] * z.grad.abs() + 5e-7 * pair + OUT_ABS["f16"]
    assert bool(((x.grad.double() - z.grad).abs() <= bound).all())


@pytest.mark.parametrize("native", [True, False])
def test_autograd_learns_of_writes_and_is_told_what_cannot_be(cr, monkeypatch, native):
    import torch

    if not native:
        monkeypatch.setattr(cr._T, "rope", lambda *a: None)
    X, pos = _inputs(1, 5, 2, 64, "bf16", 13)
    X = X.contiguous()
    freq, axis = cr.convrot_rope_tables([32])
    x = X.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="leaf"):
        cr.convrot_rope(x, pos, freq, axis, Y=x)
    with pytest.raises(RuntimeError, match="leaf"):
        part = x[:, 1:]
        cr.convrot_rope(part, pos[..., 1:], freq, axis, Y=part)
    assert torch.equal(x.detach(), X)
    for given in (dict(positions=pos.float().requires_grad_()), dict(freq=freq.clone().requires_grad_())):
        with pytest.raises(ValueError, match="detach"):
            cr.convrot_rope(**(dict(X=X, positions=pos, freq=freq, axis=axis) | given))
        with torch.no_grad():
            assert not cr.convrot_rope(**(dict(X=X, positions=pos, freq=freq, axis=axis) | given)).requires_grad
    with torch.no_grad():
        assert not cr.convrot_rope(x, pos, freq, axis).requires_grad
        cr.convrot_rope(x, pos, freq, axis, Y=x)
    with torch.inference_mode():
        z = X.clone()
        cr.convrot_rope(z, pos, freq, axis, Y=z)
    cr.convrot_rope(X, pos, freq, axis, Y=z)  # a tensor without versions
    # an operation that keeps its input learns that it has been overwritten
    x = X.clone().requires_grad_()
    z = x * 2
    out = (z * z).sum()
    with torch.no_grad():
        cr.convrot_rope(z, pos, freq, axis, Y=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()
