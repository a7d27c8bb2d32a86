"""convrot_cache_attention against the oracle on the same cells, on a B200.

Tolerance of an output row, in the 2-norm, which the final rotation keeps. Before
the rotation a channel is sum_k w_k s_k c_k with weights w of the softmax. Its
error is at most
    A eps + 2^-24 max_k(w_k s_k) sum_k |c_k|,   A = sum_k w_k s_k |c_k|,
    eps = 2^-11 (weight to fp16) + 2 e (exponent, above and below the line)
          + (L/16 + 64) 2^-22 (float32 sums: a term per 16 keys in the matrix
          instruction, the joins),
    e = ln 2 * 6 * 2^-24 max|t| (logits in base 2, six roundings) + 2^-22 (exp2) + f,
the second term for weights below fp16's normal range (2^-25 of the largest, the
largest kept above 1). f covers query codes that round the other way: where the
oracle's quotient lies within 1e-3 of a tie, a step of that code moves logit k by
s_q s_k |c_k| softmax_scale. The output's half step comes on top, and 8 float32
roundings of the rotation.
"""

from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
from parity import OUT_ABS, OUT_REL

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def cr():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_rotated_int8_token_b200 as cr

    cr.lib()
    return cr


class Setup:
    """Sequences with (keys, new tokens) each over a cache whose unused cells hold NaN scales and any codes."""

    def __init__(self, cr, seqs, hq, hkv, page, kind="bf16", seed=0, tree=None, spare=3):
        import torch

        self.cr, self.seqs, self.hq, self.hkv, self.page, self.kind = cr, seqs, hq, hkv, page, kind
        rng = np.random.default_rng(seed)
        need = [-(-k // page) for k, _ in seqs]
        order = rng.permutation(sum(need) + spare)
        self.pages = np.full((len(seqs), max(need + [0]) + 1), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = order[at:at + n]
            at += n
        shape = (len(order), hkv, page)
        self.codes = [rng.integers(-127, 128, (*shape, 128)).astype(np.int8) for _ in range(2)]
        self.scales = [np.full(shape, np.nan, np.float32) for _ in range(2)]
        for b, (keys, _) in enumerate(seqs):
            for s in self.scales:
                for j in range(0, keys, page):
                    n = min(page, keys - j)
                    s[self.pages[b, j // page], :, :n] = rng.uniform(0.005, 0.03, (hkv, n))
        self.starts = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        self.tree = tree
        self.T = int(self.starts[-1])
        self.dtype = torch.bfloat16 if kind == "bf16" else torch.float16
        q = torch.from_numpy(rng.standard_normal((self.T, hq, 128)) * 3.0).to(self.dtype)
        self.q = q.double().numpy()
        self.Q = q.cuda()

    def cells(self):
        import torch

        return [torch.from_numpy(x).cuda() for x in (*self.codes, *self.scales)]

    def args(self, starts=True):
        import torch

        a = [torch.from_numpy(self.pages).cuda(),
             torch.tensor([k for k, _ in self.seqs], dtype=torch.int32, device="cuda"),
             torch.from_numpy(self.starts).cuda() if starts else None]
        if self.tree is not None:
            a.append(torch.from_numpy(np.asarray(self.tree, np.uint64).view(np.int64)).cuda())
        return a

    def run(self, starts=True, status=0, **more):
        import torch

        need = self.cr.convrot_cache_attention_workspace_bytes(self.T, len(self.seqs), self.hq, self.hkv)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
        O = self.cr.convrot_cache_attention(self.Q, *self.cells(), *self.args(starts), ws=ws, **more)
        assert self.cr.convrot_read_device_status(ws) == status
        return O

    def dense(self, b, which, keep=None):
        """(codes [Hkv, keys, 128], scales [Hkv, keys]) of sequence b."""
        keys = self.seqs[b][0]
        at = self.pages[b, np.arange(keys) // self.page]
        off = np.arange(keys) % self.page
        return self.codes[which][at, :, off].transpose(1, 0, 2), self.scales[which][at, :, off].T

    def check(self, O, scale=SCALE, see=None, sequences=None):
        """Every row of O against the oracle; `see` replaces the visibility of sequences."""
        o = O.double().cpu().numpy()
        assert np.all(np.isfinite(o))
        group = self.hq // self.hkv
        for b in range(len(self.seqs)) if sequences is None else sequences:
            keys, news = self.seqs[b]
            rows = slice(self.starts[b], self.starts[b + 1])
            tree = None if self.tree is None else self.tree[rows]
            on = oracle.seen(keys, news, tree) if see is None else see[b]
            (kc, ks), (vc, vs) = self.dense(b, 0), self.dense(b, 1)
            some = on.any(0)  # cells nothing sees may hold anything
            ks, vs = np.where(some, ks, 1.0), np.where(some, vs, 0.0)
            ref, w, qc, sq = oracle.cache_attention(self.q[rows], kc, ks, vc, vs, on, scale)
            turned = oracle.rotate(self.q[rows], 128)
            quot = turned / np.where(sq > 0, sq, 1.0)[..., None].astype(np.float64)
            tie = np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 1e-3
            for h in range(self.hq):
                c, s = np.abs(vc[h // group].astype(np.float64)), vs[h // group].astype(np.float64)
                kk = np.abs(kc[h // group].astype(np.float64)) * ks[h // group].astype(np.float64)[:, None]
                logits = np.abs(qc[:, h].astype(np.float64) @ (kc[h // group] * ks[h // group][:, None]).T) \
                    * sq[:, h, None] * scale if keys else np.zeros((news, 0))
                for i in range(news):
                    got, want = o[self.starts[b] + i, h], ref[i, h]
                    if not on[i].any():
                        assert not got.any()
                        continue
                    ws = w[i, h] * s
                    e = math.log(2) * 6 * 2.0**-24 * (logits[i].max() * math.log2(math.e)) + 2.0**-22
                    if tie[i, h].any():
                        f = float((kk[on[i]] * tie[i, h]).sum(1).max()) * float(sq[i, h]) * scale
                        e += f * math.exp(f)
                    eps = 2.0**-11 + 2 * e + (keys / 16 + 64) * 2.0**-22
                    # Keys without a value may hold all of a row's sum, and the others' weights be far below it: an
                    # exponential below float32's 2^-126 may be lost, and where a row's sum is held below 2^101 a
                    # weight rounded to fp16's 2^-25 is off by 2^-125 of the sum and less.
                    off = eps * (ws @ c) + 2.0**-24 * ws.max() * c[on[i]].sum(0)
                    off = off + (2.0**-126 * s[on[i]] + 2.0**-125) @ c[on[i]]
                    u = OUT_REL[self.kind]
                    slack = np.linalg.norm(off) * (1 + u) + 8 * 2.0**-24 * np.linalg.norm(ws @ c)
                    bound = u * np.linalg.norm(want) + slack + OUT_ABS[self.kind] * math.sqrt(128)
                    assert np.linalg.norm(got - want) <= bound, (b, i, h, np.linalg.norm(got - want) / bound)
                    assert np.all(np.abs(got - want) <= u * np.abs(want) + slack + OUT_ABS[self.kind]), (b, i, h)
        return o


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,hq,hkv,page", [
    ([1], 1, 1, 16), ([16], 4, 1, 16), ([17], 8, 2, 16), ([64], 5, 5, 32), ([65], 3, 1, 32), ([1000], 8, 2, 64),
    ([5, 0, 130, 63], 6, 2, 16), ([300, 1, 64, 200, 128], 16, 1, 128), ([90, 257], 20, 1, 256), ([700], 64, 2, 1024),
    ([0, 0], 4, 4, 16), ([31] * 9, 2, 2, 16)])
def test_single_tokens(cr, kind, lengths, hq, hkv, page):
    s = Setup(cr, [(n, 1) for n in lengths], hq, hkv, page, kind, seed=sum(lengths) + hq)
    O = s.run(starts=False)
    s.check(O)
    import torch

    assert torch.equal(s.run(), O)  # with starts, bit by bit the same


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("seqs,hq,hkv,page", [
    ([(70, 70), (200, 3), (5, 5), (40, 0), (0, 0), (33, 1)], 4, 2, 32), ([(129, 17)], 7, 1, 16), ([(64, 64)], 1, 1, 64),
    ([(3, 7), (0, 2), (500, 2)], 2, 1, 16), ([(400, 100)], 8, 8, 16), ([(1, 1), (66, 2)], 32, 2, 128)])
def test_causal_chunks(cr, kind, seqs, hq, hkv, page):
    s = Setup(cr, seqs, hq, hkv, page, kind, seed=len(seqs) + hq)
    s.check(s.run())


def _tree(rng, news):
    """Masks of random trees; now and then a token that sees nothing of the draft, not even itself."""
    out = []
    for n in news:
        masks = []
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            masks.append((masks[parent] if parent >= 0 else 0) | 1 << i)
        if n > 3:
            masks[2] = 0
        out += masks
    return np.array(out, np.uint64)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("seqs,hq,hkv,page", [([(64, 64)], 4, 1, 16), ([(300, 12), (1, 1), (77, 33), (9, 9)], 8, 2, 32),
                                              ([(2000, 64)], 2, 2, 64), ([(5, 9), (0, 4)], 3, 1, 16),
                                              ([(90, 2), (40, 5), (130, 3)], 2, 1, 128)])
def test_trees(cr, kind, seqs, hq, hkv, page):
    rng = np.random.default_rng(hq)
    s = Setup(cr, seqs, hq, hkv, page, kind, seed=hq, tree=_tree(rng, [n for _, n in seqs]))
    s.check(s.run())


def test_causal_equals_a_line_of_drafts(cr):
    import torch

    seqs = [(100, 20), (64, 64), (3, 3)]
    line = np.array([(1 << (i + 1)) - 1 for _, n in seqs for i in range(n)], np.uint64)
    a, b = Setup(cr, seqs, 4, 2, 16), Setup(cr, seqs, 4, 2, 16, tree=line)
    assert torch.equal(a.run(), b.run())


def test_drafts_past_the_64th_are_not_seen(cr):
    full = np.full(70, 2**64 - 1, np.uint64)
    s = Setup(cr, [(100, 70)], 2, 1, 16, tree=full)
    see = np.ones((70, 100), bool)
    see[:, 94:] = False  # 30 keys of context, then 64 drafts
    s.check(s.run(status=1), see=[see])


@pytest.mark.parametrize("hq,hkv,keys", [(4, 1, 20000), (40, 1, 9000), (16, 8, 6001)])
def test_one_long_sequence_is_cut_among_all_ctas(cr, hq, hkv, keys):
    s = Setup(cr, [(keys, 1)], hq, hkv, 64, "f16", seed=keys)
    s.check(s.run(starts=False))


def test_many_sequences(cr):
    rng = np.random.default_rng(5)
    seqs = [(int(n), 1) for n in rng.integers(0, 200, 400)]
    s = Setup(cr, seqs, 4, 2, 16, seed=5)
    O = s.run(starts=False)
    s.check(O, sequences=range(0, 400, 7))


def test_maximum_that_keeps_rising(cr):
    s = Setup(cr, [(900, 2)], 4, 1, 64, "f16", seed=6)
    for b, j in [(0, j) for j in range(900)]:
        s.scales[0][s.pages[b, j // 64], :, j % 64] = 0.001 * 1.01 ** j
    s.check(s.run())


def test_value_scales_of_any_range(cr):
    """Value scales over 24 powers of ten, in either order along the keys, and values that are all zero."""
    for order in (1, -1):
        s = Setup(cr, [(600, 1), (50, 1)], 4, 2, 16, "bf16", seed=7)
        for j in range(600):
            s.scales[1][s.pages[0, j // 16], :, j % 16] = 10.0 ** (order * (j - 300) / 25.0)
        for j in range(50):
            s.scales[1][s.pages[1, j // 16], :, j % 16] = 0.0
        o = s.check(s.run(starts=False))
        assert not o[1].any()


def test_unseen_cells_may_hold_anything(cr):
    """Infinities and NaN in drafted cells that no mask names, and in those behind the last key."""
    seqs = [(40, 6)]
    tree = np.array([1, 3, 1, 9, 17, 33], np.uint64)  # nothing sees draft 2
    s = Setup(cr, seqs, 4, 2, 16, seed=8, tree=tree)
    j = 40 - 6 + 2
    s.scales[0][s.pages[0, j // 16], :, j % 16] = np.inf
    s.scales[1][s.pages[0, j // 16], :, j % 16] = np.nan
    s.check(s.run())


def test_zero_keys_and_queries(cr):
    s = Setup(cr, [(100, 1)], 2, 1, 16, seed=9)
    s.Q.zero_()
    s.q[:] = 0.0
    s.check(s.run())  # equal weights
    s = Setup(cr, [(100, 1)], 2, 1, 16, seed=9)
    s.scales[0][np.isfinite(s.scales[0])] = 0.0
    s.check(s.run())


def test_softmax_scale(cr):
    s = Setup(cr, [(200, 3)], 4, 2, 32, seed=10)
    s.check(s.run(softmax_scale=0.5), scale=0.5)
    s.check(s.run(softmax_scale=1e-6), scale=1e-6)


def test_strided_queries_and_outputs_and_rows_left_alone(cr):
    import torch

    s = Setup(cr, [(100, 2), (30, 1)], 6, 2, 16, seed=11)
    want = s.run()
    rows = torch.full((5, 10, 128), 9.0, dtype=s.dtype, device="cuda")
    rows[:3, :6] = s.Q
    out = torch.full((7, 5, 128), 3.0, dtype=s.dtype, device="cuda")  # head-major, two tokens behind the last
    cr.convrot_cache_attention(rows[:, :6], *s.cells(), *s.args(), O=out[:6].transpose(0, 1))
    assert torch.equal(out[:6, :3].transpose(0, 1), want)
    assert bool((out[:6, 3:] == 3.0).all()) and bool((out[6] == 3.0).all())


def test_shared_table_row_and_wide_table(cr):
    import torch

    s = Setup(cr, [(50, 1)], 4, 2, 16, seed=12)
    pages, lengths, _ = s.args()
    two = torch.cat([s.Q, s.Q])
    O = cr.convrot_cache_attention(two, *s.cells(), pages.expand(2, -1), lengths.repeat(2))
    assert torch.equal(O[0], O[1]) and torch.equal(O[:1], s.run())


def test_bad_pages_hide_their_keys(cr):
    for page in (16, 64):
        s = Setup(cr, [(200, 1), (40, 1)], 4, 2, page, seed=13)
        see = [np.ones((1, 200), bool), np.ones((1, 40), bool)]
        good = s.pages.copy()
        for column, bad in ((0, -1), (2, len(s.codes[0]))):
            s.pages[0, column] = bad
            see[0][0, column * page:(column + 1) * page] = False
        O = s.run(starts=False, status=1)
        s.pages = good
        s.check(O, see=see)


def test_bad_lengths_and_starts_are_bounded(cr):
    import torch

    s = Setup(cr, [(32, 1), (20, 1), (16, 1)], 2, 1, 16, seed=14)
    pages, lengths, starts = s.args()
    pages[:, 2:] = 0  # a table of valid pages
    ws = torch.empty(cr.convrot_cache_attention_workspace_bytes(3, 3, 2, 1), dtype=torch.uint8, device="cuda")
    cells = [c.nan_to_num(0.5) if c.is_floating_point() else c for c in s.cells()]
    want = cr.convrot_cache_attention(s.Q, *cells, pages, lengths, starts, ws=ws)
    wrong = lengths.clone()
    wrong[0] = -5
    O = cr.convrot_cache_attention(s.Q, *cells, pages, wrong, starts, ws=ws)
    assert cr.convrot_read_device_status(ws) == 1
    assert not bool(O[0].any()) and torch.equal(O[1:], want[1:])
    wrong[0] = 2**31 - 1
    full = lengths.clone()
    full[0] = pages.shape[1] * 16
    O = cr.convrot_cache_attention(s.Q, *cells, pages, wrong, starts, ws=ws)
    assert cr.convrot_read_device_status(ws) == 1
    assert torch.equal(O, cr.convrot_cache_attention(s.Q, *cells, pages, full, starts, ws=ws))
    assert cr.convrot_read_device_status(ws) == 0
    for bad in ([0, 1, 2, 2**31 - 1], [-9, 1, 2, 3], [0, 5, 2, 3], [3, 2, 1, 0]):
        cr.convrot_cache_attention(s.Q, *cells, pages, lengths, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws=ws)
        assert cr.convrot_read_device_status(ws) == 1
    assert torch.equal(cr.convrot_cache_attention(s.Q, *cells, pages, lengths, starts, ws=ws), want)


def test_no_table(cr):
    import torch

    s = Setup(cr, [(0, 1), (0, 1)], 2, 1, 16, seed=15)
    _, lengths, _ = s.args()
    O = cr.convrot_cache_attention(s.Q, *s.cells(), torch.empty(2, 0, dtype=torch.int32, device="cuda"), lengths)
    assert not bool(O.any())


def test_refusals(cr):
    import torch

    s = Setup(cr, [(40, 1), (20, 1)], 4, 2, 16, seed=16)
    pages, lengths, starts = s.args()
    cells = s.cells()

    def call(Q=s.Q, pages=pages, lengths=lengths, **more):
        return cr.convrot_cache_attention(Q, *cells, pages, lengths, **more)

    for bad in (dict(Q=s.Q[:1]), dict(Q=s.Q[:, :3]), dict(Q=s.Q.float()), dict(pages=pages.long()),
                dict(pages=pages[:1]), dict(pages=pages.cpu()), dict(lengths=lengths.long()), dict(lengths=lengths[:1]),
                dict(starts=starts[:2]), dict(starts=starts.long()), dict(tree=torch.zeros(2, device="cuda")),
                dict(tree=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(O=s.Q[:, :1].expand(2, 4, 128)),
                dict(O=s.Q.float()), dict(pages=pages.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for bad, status in ((dict(softmax_scale=0.0), 1), (dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda")), 3)):
        with pytest.raises(cr.ConvRotError) as e:
            call(**bad)
        assert e.value.status == status


def test_the_same_every_time_and_on_another_stream(cr):
    import torch

    s = Setup(cr, [(5000, 2), (300, 1), (64, 5)], 8, 2, 64, seed=17)
    cells, args = s.cells(), s.args()
    want = cr.convrot_cache_attention(s.Q, *cells, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [cr.convrot_cache_attention(s.Q, *cells, *args, stream=st) for _ in range(5) for st in (None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_two_graphs_share_a_workspace_and_follow_the_lengths(cr):
    import torch

    s = Setup(cr, [(900, 1), (700, 1)], 4, 2, 16, seed=18)
    pages, lengths, _ = s.args()
    cells = s.cells()
    ws = torch.empty(cr.convrot_cache_attention_workspace_bytes(2, 2, 4, 2), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(s.Q) for _ in range(2)], []
    other = s.Q.flip(0).contiguous()
    for q, o in ((s.Q, outs[0]), (other, outs[1])):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cr.convrot_cache_attention(q, *cells, pages, lengths, O=o, ws=ws)
        graphs.append(graph)
    for now in ((900, 700), (1, 650), (0, 64), (513, 700)):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], cr.convrot_cache_attention(s.Q, *cells, pages, lengths))
        assert torch.equal(outs[1], cr.convrot_cache_attention(other, *cells, pages, lengths))
    s.seqs = [(513, 1), (700, 1)]
    s.check(outs[0])
    graphs.clear()


# ---- more than 32 rows a sequence and key head on average: tiles of 128 rows


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("seqs,hq,hkv,page", [
    ([(1, 1)], 80, 1, 16), ([(127, 1)], 128, 1, 16), ([(128, 1), (129, 1)], 200, 2, 32), ([(1000, 1)], 90, 1, 1024),
    ([(0, 1), (300, 1), (0, 2)], 100, 1, 64), ([(256, 256)], 2, 2, 16), ([(300, 130), (90, 90), (5, 9)], 3, 3, 16),
    ([(3000, 33)], 12, 3, 64), ([(20000, 1)], 96, 1, 256), ([(385, 2)] * 7, 130, 2, 128)])
def test_tall_tiles(cr, kind, seqs, hq, hkv, page):
    s = Setup(cr, seqs, hq, hkv, page, kind, seed=len(seqs) + hq)
    s.check(s.run())


@pytest.mark.parametrize("seqs,hq,hkv,page", [([(64, 64)], 8, 4, 16), ([(191, 64), (192, 64), (193, 64)], 6, 3, 32),
                                              ([(1500, 50), (70, 64)], 4, 2, 128), ([(2600, 64)], 8, 2, 64),
                                              ([(90, 64), (0, 40)], 4, 2, 16)])
def test_tall_trees(cr, seqs, hq, hkv, page):
    tree = _tree(np.random.default_rng(hq), [n for _, n in seqs])
    s = Setup(cr, seqs, hq, hkv, page, "f16", seed=hq, tree=tree)
    s.check(s.run())


def test_tall_tiles_at_their_limits(cr):
    """The cases above that strain the references, with 80 query heads to a key head."""
    s = Setup(cr, [(900, 1)], 80, 1, 64, "f16", seed=6)
    for j in range(900):
        s.scales[0][s.pages[0, j // 64], :, j % 64] = 0.001 * 1.01 ** j
    s.check(s.run())
    for order in (1, -1):
        s = Setup(cr, [(600, 1), (50, 1), (700, 1)], 80, 1, 16, "bf16", seed=7)
        for j in range(600):
            s.scales[1][s.pages[0, j // 16], :, j % 16] = 10.0 ** (order * (j - 300) / 25.0)
        for j in range(50):
            s.scales[1][s.pages[1, j // 16], :, j % 16] = 0.0
        for j in range(700):  # nothing to weigh for four tiles
            if j < 520:
                s.scales[1][s.pages[2, j // 16], :, j % 16] = 0.0
        o = s.check(s.run())
        assert not o[1].any()
    tree = np.array([1, 3, 1, 9, 17, 33], np.uint64)  # nothing sees draft 2
    s = Setup(cr, [(130, 6)], 80, 2, 16, seed=8, tree=tree)
    j = 130 - 6 + 2
    s.scales[0][s.pages[0, j // 16], :, j % 16] = np.inf
    s.scales[1][s.pages[0, j // 16], :, j % 16] = np.nan
    s.check(s.run())
    s = Setup(cr, [(500, 1)], 80, 1, 16, seed=9)
    s.Q.zero_()
    s.q[:] = 0.0
    s.check(s.run())


def test_tall_tiles_with_bad_pages_bounds_and_rows_left_alone(cr):
    import torch

    s = Setup(cr, [(400, 1), (40, 1)], 80, 1, 64, seed=13)
    see = [np.ones((1, 400), bool), np.ones((1, 40), bool)]
    good = s.pages.copy()
    for column, bad in ((0, -1), (4, len(s.codes[0]))):
        s.pages[0, column] = bad
        see[0][0, column * 64:(column + 1) * 64] = False
    O = s.run(status=1)
    s.pages = good
    s.check(O, see=see)
    out = torch.full((4, 80, 128), 3.0, dtype=s.dtype, device="cuda")
    cr.convrot_cache_attention(torch.cat([s.Q, s.Q]), *s.cells(), *s.args(), O=out)
    s.check(out[:2])
    assert bool((out[2:] == 3.0).all())


def test_tall_tiles_the_same_every_time_and_in_a_graph(cr):
    import torch

    s = Setup(cr, [(5000, 2), (300, 1), (64, 5)], 64, 2, 64, "f16", seed=17)
    cells, args = s.cells(), s.args()
    want = cr.convrot_cache_attention(s.Q, *cells, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [cr.convrot_cache_attention(s.Q, *cells, *args, stream=st) for _ in range(5) for st in (None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(s.Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_cache_attention(s.Q, *cells, *args, O=out)
    for keys in (5000, 130, 0):
        args[1][0] = keys
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cr.convrot_cache_attention(s.Q, *cells, *args))
    del graph


def test_a_decoder_step_by_step(cr):
    """Projection, positions, cache and attention as a decoder runs them: a prompt, single tokens, then a tree of
    drafts, against the oracle on the cells the cache ends up with, and the cells against the tokens' own keys."""
    import torch

    torch.manual_seed(0)
    hq, hkv, width, page, B = 4, 2, 256, 16, 2
    layer = cr.ConvRotLinear(torch.randn((hq + 2 * hkv) * 128, width, device="cuda").mul_(0.1).bfloat16())
    freq, axis = cr.convrot_rope_tables([16, 24, 24], shared=True)
    cache = cr.ConvRotCache(12, hkv, page)
    pages = torch.randperm(12, device="cuda").view(B, 6).to(torch.int32)
    length = [0, 0]

    def step(news, tree=None):
        T = sum(news)
        seq = torch.tensor([b for b in range(B) for _ in range(news[b])], device="cuda")
        at = torch.tensor([length[b] + i for b in range(B) for i in range(news[b])], device="cuda")
        rows = layer(torch.randn(T, width, device="cuda").bfloat16()).view(T, hq + 2 * hkv, 128)
        pos = torch.stack([at, at // 3, at % 3]).to(torch.int32)
        heads = cr.convrot_rope(rows[:, :hq + hkv], pos, freq, axis)
        slots = cache.slots(pages, seq, at)
        cache.append(heads[:, hq:], rows[:, hq + hkv:], slots)
        for b in range(B):
            length[b] += news[b]
        lengths = torch.tensor(length, dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, news[0], T], dtype=torch.int32, device="cuda")
        O = cache.attention(heads[:, :hq], pages, lengths, starts, tree)
        # the cells hold this step's keys and values
        kc, vc, ks, vs = [t[slots.long() // page, :, slots.long() % page].cpu().numpy() for t in cache.cells]
        for X, c, f in ((heads[:, hq:], kc, ks), (rows[:, hq + hkv:], vc, vs)):
            ref_c, ref_f = oracle.cache_write(X.double().cpu().numpy())
            assert np.abs(c.astype(int) - ref_c).max() <= 1 and np.allclose(f, ref_f, rtol=1e-6)
        s = Setup.__new__(Setup)
        s.hq, s.hkv, s.page, s.kind = hq, hkv, page, "bf16"
        s.seqs, s.pages = list(zip(length, news)), pages.cpu().numpy()
        s.codes = [t.cpu().numpy() for t in (cache.k_codes, cache.v_codes)]
        s.scales = [t.cpu().numpy() for t in (cache.k_scale, cache.v_scale)]
        s.starts, s.tree = starts.cpu().numpy(), None if tree is None else tree.cpu().numpy().view(np.uint64)
        s.q = heads[:, :hq].double().cpu().numpy()
        s.check(O)

    step([37, 5])
    for _ in range(3):
        step([1, 1])
    step([4, 2], torch.tensor([1, 3, 5, 13, 1, 2], dtype=torch.int64, device="cuda"))
    cache.check()


def test_a_prompt_through_the_dense_attention(cr):
    """Positions written head by head feed the dense INT8 attention, and keys read back from the cache stand for
    the same cells: the attention over the cache agrees with the dense one on the values read back."""
    import torch

    torch.manual_seed(1)
    S, heads = 200, 3
    x = torch.randn(3, S, heads, 128, device="cuda").bfloat16()
    freq, axis = cr.convrot_rope_tables([16, 24, 24])
    pos = torch.stack([torch.zeros(S), torch.arange(S) // 20, torch.arange(S) % 20]).to(torch.int32).cuda()
    q, k = (torch.empty(heads, S, 128, dtype=x.dtype, device="cuda") for _ in range(2))
    cr.convrot_rope(x[0], pos, freq, axis, True, Y=q.transpose(0, 1))
    cr.convrot_rope(x[1], pos, freq, axis, True, Y=k.transpose(0, 1))
    cache = cr.ConvRotCache(13, heads, 16)
    slots = torch.randperm(13 * 16, device="cuda")[:S].to(torch.int32)
    cache.append(k.transpose(0, 1), x[2], slots)
    kb, vb = (torch.empty(heads, S, 128, dtype=x.dtype, device="cuda") for _ in range(2))
    cache.read(slots, K=kb.transpose(0, 1), V=vb.transpose(0, 1))
    ref = oracle.attention_int8(*(t.double().cpu().numpy() for t in (q, k, vb)))
    # the last token over the cache, its keys gathered through one page per token place
    dense = cr.convrot_attention_int8(q, k, vb).double().cpu().numpy()
    assert np.linalg.norm(dense - ref) <= 3e-3 * np.linalg.norm(ref)
    # the order of keys does not matter to a token that sees them all
    flat = torch.full((1, 13), -1, dtype=torch.int32, device="cuda")
    tight = cr.ConvRotCache(13, heads, 16)
    tight.append(k.transpose(0, 1), x[2], torch.arange(S, dtype=torch.int32, device="cuda"))
    flat[0] = torch.arange(13)
    O = tight.attention(q[:, -1:].transpose(0, 1).contiguous(), flat, torch.tensor([S], dtype=torch.int32, device="cuda"))
    last = O[0].double().cpu().numpy()
    assert np.linalg.norm(last - ref[:, -1]) <= 1e-2 * np.linalg.norm(ref[:, -1])


def test_native_and_python_binding_agree(cr, monkeypatch):
    """The native form takes a decoding step's calls, strided views, outputs and fp16 too, and gives what
    the Python form gives, bit for bit; both refuse the same."""
    import torch

    g = torch.Generator("cuda").manual_seed(5)

    def rnd(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def step(dtype, given):
        rows = rnd(6, 16, 128, dtype=dtype)
        q, k, v = rows[:, :8], rows[:, 8:12], rows[:, 12:]
        cache = cr.ConvRotCache(8, 4, 16)
        freq, axis = cr.convrot_rope_tables([16, 24, 24])
        where = torch.arange(18, device="cuda", dtype=torch.int32).view(3, 6)
        table = torch.arange(6, device="cuda", dtype=torch.int32).view(3, 2)
        lengths = torch.tensor([20, 7, 0], device="cuda", dtype=torch.int32)
        starts = torch.tensor([0, 2, 6, 6], device="cuda", dtype=torch.int32)
        tree = torch.tensor([1, 3, 1, 3, 5, 9], device="cuda", dtype=torch.int64)
        slots = torch.tensor([18, 19, 35, 36, 37, 38], device="cuda", dtype=torch.int32)
        room = [torch.empty(6, 12, 128, dtype=dtype, device="cuda")[:, 1:9] if given else None for _ in range(4)]

        def calls():
            out = [cr.convrot_rope(q, where, freq, axis, interleaved=given, inverse=given, Y=room[0])]
            out.append(cr.convrot_rope(q[None], where[:, None], freq, axis))
            cache.append(k, v, slots)
            out += cache.read(slots, dtype=dtype, K=room[1][:, :4] if given else None,
                              V=room[2][:, :4] if given else None)
            scale = 0.3 if given else None
            room_ws = cr.convrot_cache_attention_workspace_bytes(6, 3, 8, 4)
            ws = torch.empty(room_ws, dtype=torch.uint8, device="cuda") if given else None
            out.append(cache.attention(q, table, lengths, starts, tree=tree, softmax_scale=scale, O=room[3], ws=ws))
            out.append(cache.attention(q[:3], table, lengths))
            return [t.clone() for t in out] + [t.clone() for t in cache.cells]

        return calls, q, cache

    T = cr._T
    for dtype in (torch.bfloat16, torch.float16):
        for given in (False, True):
            calls, q, cache = step(dtype, given)
            took = []

            def count(fn):
                def run(*a):
                    done = fn(*a)
                    took.append(done is not None)
                    return done
                return run

            with monkeypatch.context() as m:
                for name in ("rope", "append", "read", "attention"):
                    m.setattr(T, name, count(getattr(T, name)))
                native = calls()
            assert took == [True] * 6
            with monkeypatch.context() as m:
                for name in ("rope", "append", "read", "attention"):
                    m.setattr(T, name, lambda *a: None)
                plain = calls()
            assert all(torch.equal(a.view(torch.int8), b.view(torch.int8)) for a, b in zip(native, plain))

    table = torch.zeros(6, 1, device="cuda", dtype=torch.int32)
    lengths = torch.ones(6, device="cuda", dtype=torch.int32)
    for bad in (dict(O=q.float()), dict(O=q[:, :1].expand(6, 8, 128)), dict(ws=lengths[::2]),
                dict(tree=lengths), dict(starts=lengths), dict(softmax_scale=float("nan"))):
        with pytest.raises((TypeError, ValueError, cr.ConvRotError)):
            cache.attention(q, table, lengths, **bad)
    with pytest.raises(cr.ConvRotError):
        cache.attention(q, table, lengths, ws=lengths[:0])
    with pytest.raises(TypeError):
        cache.read(lengths, dtype=torch.float32)
    with pytest.raises(ValueError):
        cache.read(lengths, dtype=torch.bfloat16, K=torch.empty(6, 4, 128, dtype=torch.float16, device="cuda"))


def test_first_calls_may_be_captured():
    """In a fresh process nothing has been launched or looked up before the capture."""
    import subprocess
    import sys

    code = """
import torch
import w8a8_rotated_int8_token_b200 as cr
g = torch.Generator("cuda").manual_seed(3)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
cache = cr.ConvRotCache(16, 2, 16)
freq, axis = cr.convrot_rope_tables([32, 32])
q, k, v = rnd(100, 8, 128), rnd(100, 2, 128), rnd(100, 2, 128)
pos = torch.arange(200, device="cuda", dtype=torch.int32).view(2, 100)
slots = torch.arange(100, device="cuda", dtype=torch.int32)
pages = torch.arange(16, device="cuda", dtype=torch.int32)[None]
lengths = torch.tensor([100], device="cuda", dtype=torch.int32)
starts = torch.tensor([0, 100], device="cuda", dtype=torch.int32)
def step():
    y = cr.convrot_rope(q, pos, freq, axis)
    cache.append(cr.convrot_rope(k, pos, freq, axis), v, slots)
    wide = cache.attention(y, pages, lengths, starts)            # many rows
    few = cache.attention(y[99:], pages, lengths)                # one token
    return wide, few, *cache.read(slots)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
for t in cache.cells:
    t.zero_()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert all(bool(t.isfinite().all()) and bool(t.any()) for t in got)
torch.cuda.synchronize()
del graph
print("captured")
"""
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_mean_rows_decide_the_tile(cr):
    """Either side of the rule that picks 16 or 128 rows, and sequences far from the mean."""
    for news in (2, 3, 7, 8, 9, 16):  # 4 heads a key head: 8, 12, 28, 32, 36, 64 rows each
        s = Setup(cr, [(40 + news, news), (333, news), (news, news)], 8, 2, 32, seed=news)
        s.check(s.run())
    s = Setup(cr, [(200, 40), (77, 1), (50, 0), (129, 4)], 8, 2, 16, "f16", seed=9)
    s.check(s.run())


@pytest.mark.parametrize("hq,hkv", [(4, 2), (80, 2)])
@pytest.mark.parametrize("value", [np.inf, 3e38, 1e30])
def test_unseen_values_of_any_size(cr, hq, hkv, value):
    """A draft that no mask names, with a value scale that would dwarf the others, beside them in one tile and
    in a tile of its own kind behind them; seen by some rows only, it counts for those alone."""
    tree = np.array([1, 3, 1, 9, 17, 33], np.uint64)  # nothing sees draft 2
    for keys in (100, 131):
        s = Setup(cr, [(keys, 6)], hq, hkv, 16, seed=8, tree=tree)
        j = keys - 6 + 2
        s.scales[0][s.pages[0, j // 16], :, j % 16] = np.nan
        s.scales[1][s.pages[0, j // 16], :, j % 16] = value
        s.check(s.run())
    if value == 1e30:
        tree[2] = 4 | 1
        s = Setup(cr, [(100, 6)], hq, hkv, 16, seed=8, tree=tree)
        j = 100 - 6 + 2
        s.scales[1][s.pages[0, j // 16], :, j % 16] = value
        s.check(s.run())


@pytest.mark.parametrize("hq,hkv", [(4, 1), (80, 1)])
def test_values_of_zero_before_others(cr, hq, hkv):
    """Keys with large logits and values of zero, then small logits far below them, then large ones again: a
    row's sum is kept through all of it. Many sequences, so that a CTA meets the whole of one."""
    s = Setup(cr, [(768, 1)] * 160, hq, hkv, 64, seed=10)
    for b in range(160):
        for j in range(0, 768, 64):
            page = s.pages[b, j // 64]
            s.scales[0][page] *= 1e-6 if 256 <= j < 512 else 30.0
            if j < 256:
                s.scales[1][page] = 0.0
    s.check(s.run(), sequences=range(0, 160, 16))


def test_tall_tiles_with_pages_missing_here_and_there(cr):
    """Tiles of 128 keys in which some of the eight boxes of 16 keys have no page, others no key."""
    rng = np.random.default_rng(3)
    s = Setup(cr, [(2900, 1), (75, 1)], 80, 1, 16, seed=19)
    see = [np.ones((1, n), bool) for n, _ in s.seqs]
    good = s.pages.copy()
    for b, (keys, _) in enumerate(s.seqs):
        for column in np.flatnonzero(rng.random(-(-keys // 16)) < 0.4):
            s.pages[b, column] = -1
            see[b][0, column * 16:(column + 1) * 16] = False
    O = s.run(status=1)
    s.pages = good
    s.check(O, see=see)


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("hq", [4, 160])
def test_a_cache_learns_what_its_attention_met(cr, monkeypatch, native, hq):
    """Without a workspace of the caller's the status is not lost: it is kept in the cache's own word."""
    import torch

    if not native:
        monkeypatch.setattr(cr._T, "attention", lambda *a: None)
    s = Setup(cr, [(40, 1), (20, 1)], hq, 2, 16, seed=20)
    cache = cr.ConvRotCache(len(s.codes[0]), 2, 16)
    for t, x in zip(cache.cells, s.cells()):
        t.copy_(x)
    pages, lengths, starts = s.args()
    O = cache.attention(s.Q, pages, lengths, starts)
    cache.check()
    s.check(O)
    for bad in (dict(lengths=torch.tensor([40, -1], dtype=torch.int32, device="cuda")),
                dict(pages=torch.full_like(pages, -1)), dict(starts=starts + 1)):
        cache.attention(s.Q, **({"pages": pages, "lengths": lengths, "starts": starts} | bad))
        cache.attention(s.Q, pages, lengths, starts)  # a good call does not clear it
        with pytest.raises(cr.ConvRotError) as e:
            cache.check()
        assert e.value.status == 1
        cache.status.zero_()
    own = torch.zeros(1, dtype=torch.int32, device="cuda")
    cr.convrot_cache_attention(s.Q, *cache.cells, pages, -lengths, starts, status=own)
    assert own.item() == 1 and cache.status.item() == 0
    with pytest.raises(TypeError):
        cr.convrot_cache_attention(s.Q, *cache.cells, pages, lengths, starts, status=own.float())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_a_wait_that_runs_out_makes_rows_nan_and_is_reported(cr, kind):
    """A limit of a nanosecond on the waits of the 128-row kernel, some of which take longer: each row is what it is
    with time, or NaN, and the status says so; the next call is as if nothing had been."""
    import torch

    s = Setup(cr, [(20000, 1), (0, 1)] + [(300, 1)] * 198, 40, 1, 64, kind, seed=21)
    cells, (pages, lengths, starts) = s.cells(), s.args()
    need = cr.convrot_cache_attention_workspace_bytes(200, 200, 40, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = cr.convrot_cache_attention(s.Q, *cells, pages, lengths, starts, ws=ws)
    told = torch.zeros(1, dtype=torch.int32, device="cuda")
    O = torch.full_like(want, 7.0)
    args = cr._lib.CACHE_ATTENTION_ARGS.pack(
        *(t.data_ptr() for t in cells), *cells[0].shape, s.Q.data_ptr(), O.data_ptr(), pages.data_ptr(),
        lengths.data_ptr(), starts.data_ptr(), 0, ws.data_ptr(), need, 200, 40, 200, pages.shape[1], pages.stride(0),
        *s.Q.stride()[:2], *O.stride()[:2], SCALE, cr.DTYPE_F16 if kind == "f16" else cr.DTYPE_BF16)
    stream = torch.cuda.current_stream().cuda_stream
    assert cr.lib().convrot_cache_attention_ex(args, told.data_ptr(), 1, stream) == 0
    assert cr.convrot_read_device_status(ws) == 5 and told.item() == 5
    lost = O.isnan().all(-1)
    assert bool(lost.any()) and not bool(lost[1].any())
    assert torch.equal(O[~lost], want[~lost])
    told.zero_()
    assert cr.lib().convrot_cache_attention_ex(args, told.data_ptr(), 0, stream) == 0
    assert cr.convrot_read_device_status(ws) == 0 and told.item() == 0 and torch.equal(O, want)


@pytest.mark.parametrize("hq", [4, 80])
def test_logits_of_any_size(cr, hq):
    """Equal keys, so that every key weighs the same however far below (or above) zero its logit lies."""
    keys = [1, 70, 300]
    s = Setup(cr, [(n, 1) for n in keys], hq, 1, 16, seed=23)
    for b, n in enumerate(keys):
        s.codes[0][s.pages[b, :-(-n // 16)]] = s.codes[0][s.pages[b, 0], :, :1]
        s.scales[0][s.pages[b, :-(-n // 16)]] = np.float32(1e30)
    o = s.run().double().cpu().numpy()
    for b, n in enumerate(keys):
        (kc, ks), (vc, vs) = s.dense(b, 0), s.dense(b, 1)
        qc, _ = oracle.quantize_heads(s.q[b], 128)
        sums = qc.astype(np.int64) @ kc[0, 0].astype(np.int64)
        assert (sums < 0).any() and (sums > 0).any() and not (sums == 0).any()
        held = oracle.cache_value(vc[0], vs[0])
        # a weight is 1 / n to fp16's half step, times the value's size; the rest as in the header
        size = (vs[0][:, None].astype(np.float64) * np.abs(vc[0].astype(np.float64))).sum(0) / n
        slack = (2.0**-11 + (n / 16 + 64) * 2.0**-22) * np.linalg.norm(size) * (1 + OUT_REL["bf16"])
        want = held.mean(0)
        assert np.all(np.abs(o[b] - want) <= OUT_REL["bf16"] * np.abs(want) + slack + OUT_ABS["bf16"])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [4, 80])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_no_number_gives_none(cr, kind, hq, odd):
    """Its own row alone: no code stands for such a vector, so its weights are not those of any other query."""
    import torch

    s = Setup(cr, [(200, 1), (130, 1), (0, 1)] + [(1, 1)] * 9, hq, 1, 16, kind, seed=22)
    want = s.run()
    s.Q[2, 0, 0] = odd  # sees no key: zeros
    lost = torch.zeros(12, hq, dtype=torch.bool, device="cuda")
    for t, h, c in ((0, 1, 77), (1, hq - 1, 5), *((3 + i, i % 4, 14 * i) for i in range(9))):
        s.Q[t, h, c] = odd
        lost[t, h] = True
    O = s.run()
    assert bool(O[lost].isnan().all()) and torch.equal(O[~lost], want[~lost])


@pytest.mark.parametrize("hq", [4, 10, 80])
@pytest.mark.parametrize("value", [1e30, 1e33, 1e35])
def test_seen_values_of_any_size_under_rising_logits(cr, hq, value):
    """Value scales near the end of float32 while a row's maximum rises from key to key, by little and by much."""
    for rise in (1.01, 1.3):
        s = Setup(cr, [(500, 1), (33, 1)], hq, 1, 16, seed=24)
        for b, (n, _) in enumerate(s.seqs):
            for j in range(n):
                s.scales[0][s.pages[b, j // 16], :, j % 16] = min(0.001 * rise ** j, 0.03)
                s.scales[1][s.pages[b, j // 16], :, j % 16] *= value / 0.03
        s.check(s.run())
    s = Setup(cr, [(20000, 1)], hq, 1, 64, seed=25)  # cut among all CTAs, equal values
    s.scales[1][np.isfinite(s.scales[1])] = value
    s.check(s.run())


def test_queries_of_no_sequence(cr):
    import torch

    s = Setup(cr, [(40, 1)], 4, 2, 16, seed=26)
    pages, lengths, starts = s.args()
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    O = torch.full_like(s.Q, 3.0)
    cr.convrot_cache_attention(s.Q, *s.cells(), pages[:0], lengths[:0], starts[:1], O=O, ws=ws)
    assert cr.convrot_read_device_status(ws) == 0 and bool((O == 3.0).all())
    assert bool((ws[4:] == 255).all())


@pytest.mark.parametrize("hq,hkv,keys,page", [(8, 2, 700, 64), (12, 1, 333, 16), (80, 1, 1000, 16), (130, 1, 129, 32),
                                              (96, 2, 64, 16), (70, 1, 65, 16)])
def test_fp16_outputs_keep_the_weights_bits(cr, hq, hkv, keys, page):
    """On every tile height a weight is held in two fp16 numbers, to 2^-22 of it or 2^-25 of the row's largest: what is
    left is the output's half step and the float32 terms of the header."""
    s = Setup(cr, [(keys, 1), (keys // 2 + 1, 1)], hq, hkv, page, "f16", seed=keys)
    o = s.run().double().cpu().numpy()
    u = OUT_REL["f16"]
    for b, (n, _) in enumerate(s.seqs):
        (kc, ks), (vc, vs) = s.dense(b, 0), s.dense(b, 1)
        q = s.q[b:b + 1]
        ref, w, qc, sq = oracle.cache_attention(q, kc, ks, vc, vs, np.ones((1, n), bool), SCALE)
        quot = oracle.rotate(q, 128) / sq[..., None].astype(np.float64)
        tie = (np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 1e-3)[0]
        some = 0
        for h in range(hq):
            g = h // (hq // hkv)
            if tie[h].any():  # a code may round the other way: the looser bound of check() covers those rows
                continue
            some += 1
            c, f = np.abs(vc[g].astype(np.float64)), vs[g].astype(np.float64)
            top = np.abs((qc[0, h].astype(np.float64) @ kc[g].T) * ks[g]).max() * float(sq[0, h]) * SCALE
            e = math.log(2) * 6 * 2.0**-24 * top * math.log2(math.e) + 2.0**-22
            ws = w[0, h] * f
            off = (2.0**-22 + 2 * e + (n / 16 + 64) * 2.0**-22) * (ws @ c) + 2.0**-25 * ws.max() * c.sum(0)
            slack = np.linalg.norm(off) * (1 + u) + 8 * 2.0**-24 * np.linalg.norm(ws @ c)
            want, got = ref[0, h], o[b, h]
            assert np.all(np.abs(got - want) <= u * np.abs(want) + slack + OUT_ABS["f16"]), (b, h)
        assert some >= hq // 4


@pytest.mark.parametrize("hq", [4, 12, 80])
def test_strained_references_with_fp16_outputs(cr, hq):
    """What strains the references above, where the weights' second product and, on tiles of 128 rows, the steps of 64
    keys take part: value scales over many powers of ten in either order, keys without a value before others (also
    whole steps of them), logits that rise by steps, a draft that no mask names and drafts that few see."""
    for order in (1, -1):
        s = Setup(cr, [(600, 1), (50, 1), (700, 1)], hq, 1, 16, "f16", seed=7)
        for j in range(600):
            s.scales[1][s.pages[0, j // 16], :, j % 16] = 10.0 ** (order * (j - 300) / 30.0 - 9.0)
        for j in range(50):
            s.scales[1][s.pages[1, j // 16], :, j % 16] = 0.0
        for j in range(700):
            if j < 520 and j // 64 % 3 != 1:
                s.scales[1][s.pages[2, j // 16], :, j % 16] = 0.0
            s.scales[0][s.pages[2, j // 16], :, j % 16] *= 1.0 + 0.5 * (j // 64)
        o = s.check(s.run())
        assert not o[1].any()
    tree = np.array([1, 3, 1, 9, 17, 33], np.uint64)  # nothing sees draft 2
    for keys in (64, 68, 130):  # the drafts before, across and behind the border of two steps
        s = Setup(cr, [(keys, 6)], hq, 1, 16, "f16", seed=8, tree=tree)
        j = keys - 6 + 2
        s.scales[0][s.pages[0, j // 16], :, j % 16] = np.nan
        s.scales[1][s.pages[0, j // 16], :, j % 16] = np.inf
        s.check(s.run())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [4, 12, 80])
def test_a_heavy_value_beside_sums_without_values(cr, kind, hq):
    """Most of a row's sum lies in keys with next to no value, its mean in one key with a large one: the unit of a
    row's weights differs by 2^120 and more between tiles, pipelines and pieces, and no sum is lost on the way."""
    heavy, next_to_none = (1e15, 1e-28) if kind == "bf16" else (40.0, 1e-35)
    for keys in (136, 300, 5000):
        for at in (5, 100, 131, keys - 2):
            s = Setup(cr, [(keys, 1)], hq, 1, 16, kind, seed=27)
            s.scales[0][np.isfinite(s.scales[0])] = 0.002  # logits near one another
            s.scales[1][np.isfinite(s.scales[1])] = next_to_none
            s.scales[1][s.pages[0, at // 16], :, at % 16] = heavy
            s.check(s.run())


@pytest.mark.parametrize("hq", [4, 12, 80])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 1e12, 1e30])
def test_far_logits_pick_their_largest(cr, hq, size):
    """Key scales so large, and so far apart, that one key holds a row's whole weight: its value is the row."""
    s = Setup(cr, [(300, 1), (20, 2), (131, 1)], hq, 1, 16, "bf16", seed=28)
    rng = np.random.default_rng(4)
    held = np.isfinite(s.scales[0])
    s.scales[0][held] = (size * 10.0 ** rng.uniform(-3, 1, held.sum())).astype(np.float32)
    o = s.run().double().cpu().numpy()
    assert np.all(np.isfinite(o))
    u, sure = OUT_REL["bf16"], 0
    for b, (n, news) in enumerate(s.seqs):
        (kc, ks), (vc, vs) = s.dense(b, 0), s.dense(b, 1)
        for i in range(news):
            row = s.starts[b] + i
            qc, sq = oracle.quantize_heads(s.q[row], 128)
            seen = n - news + i + 1
            logits = (qc.astype(np.float64) @ kc[0, :seen].T.astype(np.float64)) * ks[0, :seen] * sq[:, None] * SCALE
            for h in range(hq):
                order = np.argsort(logits[h])
                first, second = logits[h, order[-1]], logits[h, order[-2]]
                # what codes that round the other way move, and the float32 roundings of both logits
                sway = 3 * float(sq[h]) * SCALE * 127 * float(ks[0, order[-2:]].max())
                if first - second <= 2 * sway + 12 * 2.0**-24 * abs(first) + 60:
                    continue
                sure += 1
                at = order[-1]
                want = oracle.cache_value(vc[0, at], vs[0, at])
                off = np.linalg.norm(vc[0, at] * float(vs[0, at])) * (2.0**-11 + 2.0**-18)
                assert np.all(np.abs(o[row, h] - want) <= u * np.abs(want) + off), (b, i, h)
    assert sure >= 2


@pytest.mark.parametrize("hq", [4, 12, 80])
def test_far_logits_with_values_of_any_size(cr, hq):
    """Equal keys with logits of any magnitude, values over 40 powers of ten, in any order: every weight is 1 / n."""
    rng = np.random.default_rng(6)
    for size in (1e6, 1e8, 1e9, 1e12, 1e25):
        for order in ("rising", "falling", "any", "zeros first"):
            keys = [300, 140, 40]
            s = Setup(cr, [(n, 1) for n in keys], hq, 1, 16, seed=29)
            for b, n in enumerate(keys):
                at = s.pages[b, :-(-n // 16)]
                s.codes[0][at] = s.codes[0][s.pages[b, 0], :, :1]
                s.scales[0][at] = np.float32(size)
                power = rng.uniform(-20, 20, n)
                power = {"rising": np.sort(power), "falling": -np.sort(-power)}.get(order, power)
                for j in range(n):
                    s.scales[1][s.pages[b, j // 16], :, j % 16] = 0.0 if order == "zeros first" and j < n - 9 \
                        else 10.0 ** power[j]
            o = s.run().double().cpu().numpy()
            assert np.all(np.isfinite(o))
            for b, n in enumerate(keys):
                _, (vc, vs) = s.dense(b, 0), s.dense(b, 1)
                want = oracle.cache_value(vc[0], vs[0]).mean(0)
                size_ = (vs[0][:, None].astype(np.float64) * np.abs(vc[0].astype(np.float64))).sum(0) / n
                slack = (2.0**-11 + (n / 16 + 64) * 2.0**-22) * np.linalg.norm(size_) * (1 + OUT_REL["bf16"])
                assert np.all(np.abs(o[b] - want) <= OUT_REL["bf16"] * np.abs(want) + slack + OUT_ABS["bf16"]), (size, order, b)
