"""Cases of the operators around the INT8 attention: rotary positions with several axes, the rotated
int8 key/value cache (written and read back) and attention over that cache.

``run`` computes an operator in elementary torch operations, or (``own``) with the framework's kernels.
A head vector has 128 channels in the cache; its rotation is the normalised Walsh-Hadamard matrix of
order 128, and its int8 codes have one scale per token and head, as in the ConvRot linear layer.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DIM = 128  # head dimension of the cache
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # One decoding step of a text encoder with 16 sequences: the 32 query and 8 key heads of the fused
        # projection's rows, positions of time, height and width on one ladder of frequencies.
        {"name": "rope_step_16", "op": "rope", "batch": 16, "tokens": 1, "heads": 40, "dim": 128, "rotary": 128,
         "first": 16, "second": 24, "shared": True, "interleaved": False, "inverse": False, "head_major": False,
         "type": "bf16"},
        # The attention workload's tokens: a 64 x 64 image behind 128 text tokens, 32 heads, written head by head
        # as the dense INT8 attention reads them; a ladder of frequencies per axis, neighbouring channels paired.
        {"name": "rope_image_4224", "op": "rope", "batch": 1, "tokens": 4224, "heads": 32, "dim": 128, "rotary": 128,
         "first": 8, "second": 28, "shared": False, "interleaved": True, "inverse": False, "head_major": True,
         "type": "bf16"},
        # The gradient of the rotary positions at the 2048 x 2048 image's token count, in fp16.
        {"name": "rope_grad_16896", "op": "rope", "batch": 1, "tokens": 16896, "heads": 32, "dim": 128,
         "rotary": 128, "first": 16, "second": 24, "shared": False, "interleaved": False, "inverse": True,
         "head_major": False, "type": "f16"},
        # The same decoding step's 16 new tokens go into the cache and are read back.
        {"name": "append_step_16", "op": "append", "tokens": 16, "heads": 8, "page": 16, "padding": 0,
         "capacity": 4096, "type": "bf16"},
        # Prompts of 8191 tokens in all, with the padding of their batch, go into the cache and are read back
        # for the dense attention over the prompt.
        {"name": "append_prompts_8191", "op": "append", "tokens": 8191, "heads": 8, "page": 64, "padding": 130,
         "capacity": 32768, "type": "f16"},
        # A short shared prefix is read back.
        {"name": "read_prefix_333", "op": "read", "tokens": 333, "heads": 8, "page": 32, "padding": 3,
         "capacity": 8192, "type": "f16"},
        # Long prompts are read back for the dense attention.
        {"name": "read_prompts_32768", "op": "read", "tokens": 32768, "heads": 8, "page": 128, "padding": 0,
         "capacity": 65536, "type": "bf16"},
        # One new token of one sequence behind the attention workload's 4224 tokens.
        {"name": "attend_one_4224", "op": "attend", "batch": 1, "length": 4224, "low": 1.0, "idle": 0, "nodes": 0,
         "heads": 32, "kv_heads": 8, "page": 64, "type": "bf16"},
        # One new token of each of 16 sequences of very different lengths, two places of the batch unused.
        {"name": "attend_16_ragged", "op": "attend", "batch": 16, "length": 8191, "low": 0.01, "idle": 2, "nodes": 0,
         "heads": 32, "kv_heads": 8, "page": 16, "type": "bf16"},
        # A full batch of long sequences, one new token each.
        {"name": "attend_64_long", "op": "attend", "batch": 64, "length": 16384, "low": 0.25, "idle": 0, "nodes": 0,
         "heads": 32, "kv_heads": 8, "page": 128, "type": "bf16"},
        # Trees of up to 32 drafted tokens for 8 sequences.
        {"name": "tree_8x32", "op": "attend", "batch": 8, "length": 4096, "low": 0.3, "idle": 0, "nodes": 32,
         "heads": 32, "kv_heads": 8, "page": 64, "type": "bf16"},
        # A tree of 64 drafted tokens behind a long context, 8 query heads to a key head, in fp16.
        {"name": "tree_64_deep", "op": "attend", "batch": 1, "length": 32768, "low": 1.0, "idle": 0, "nodes": 64,
         "heads": 16, "kv_heads": 2, "page": 256, "type": "f16"},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng: random.Random):
    op = rng.choice(("rope", "append", "read", "attend", "attend"))
    kind = rng.choice(("bf16", "f16"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "rope":
        tokens, heads, dim = _log(rng, 1, 16896), _log(rng, 1, 48), rng.choice((64, 128, 128, 256))
        tokens = min(tokens, 16896 * 32 * 128 // (heads * dim))
        batch = rng.choice((1, 1, 2, 3)) if tokens <= 4096 else 1
        batch = min(batch, max(1, 16896 * 32 * 128 // (tokens * heads * dim)))
        rotary = rng.choice((dim, dim, dim // 2))
        first = rng.randint(0, rotary // 4)
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary,
                "first": first, "second": rng.randint(0, rotary // 2 - first), "shared": rng.random() < 0.5,
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5, "head_major": rng.random() < 0.5,
                "type": kind}
    if op in ("append", "read"):
        tokens = _log(rng, 1, 8191 if op == "append" else 32768)
        heads = rng.choice((1, 2, 3, 4, 8))
        return {"op": op, "tokens": tokens, "heads": heads, "page": page, "padding": rng.randint(0, tokens // 8),
                "capacity": -(-2 * tokens // page) * page, "type": kind}
    batch = _log(rng, 1, 64)
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16))
    nodes = rng.choice((0, 0, _log(rng, 2, 64)))
    length = _log(rng, 1, 16384)
    # no more multiply-adds than the deep tree and no more cache than the full batch
    rows = max(1, nodes) * kv_heads * group
    length = max(1, min(length, 64 * 16 * 32768 // (batch * rows), 64 * 8 * 16384 // (batch * kv_heads)))
    return {"op": op, "batch": batch, "length": length, "low": round(rng.uniform(0.02, 1.0), 3),
            "idle": rng.randint(0, batch // 4), "nodes": nodes, "heads": kv_heads * group, "kv_heads": kv_heads,
            "page": page, "type": kind}


# ------------------------------------------------------------------------------------------- inputs


def _spread(count, high, low):
    """`count` whole numbers in [low * high, high], the first of them `high`."""
    return [max(1, int(round(high * (1.0 - (1.0 - low) * ((b * 0.6180339887) % 1.0))))) for b in range(count)]


def _ragged(case):
    """(keys in the cache, new tokens) of each sequence; an idle place has no keys and one token."""
    batch, nodes = case["batch"], case["nodes"]
    news = _spread(batch, nodes, 0.25) if nodes else [1] * batch
    keys = [max(k, n) for k, n in zip(_spread(batch, case["length"], case["low"]), news)]
    idle = case["idle"]
    return keys[: batch - idle] + [0] * idle, news


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _vectors(shape, dtype, g):
    """Head vectors with a few channels that stand out, as keys have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 5] *= 12.0
    x[..., 77] *= 6.0
    return x.to(dtype)


def _codes(shape, g):
    """Codes of rotated vectors: near normal, the largest of a vector near 127."""
    c = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in c.view(-1, DIM).split(1 << 21):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 42.0).round_().clamp_(-127, 127))
    return c


def _hadamard():
    h = torch.ones(1, 1, device="cuda")
    while h.shape[0] < DIM:  # order doubles: 1, 2, 4, ... 128
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _cache(pages, heads, page, g, filled):
    shape = (pages, heads, page)
    if not filled:
        return {"k_codes": torch.zeros(*shape, DIM, dtype=torch.int8, device="cuda"),
                "v_codes": torch.zeros(*shape, DIM, dtype=torch.int8, device="cuda"),
                "k_scale": torch.zeros(shape, device="cuda"), "v_scale": torch.zeros(shape, device="cuda")}
    return {"k_codes": _codes((*shape, DIM), g), "v_codes": _codes((*shape, DIM), g),
            "k_scale": torch.rand(shape, generator=g, device="cuda") * 0.04 + 0.01,
            "v_scale": torch.rand(shape, generator=g, device="cuda") * 0.04 + 0.01}


def _rope_tables(case):
    """Frequency (radians a position, 64 bits) and axis of each pair of channels."""
    pairs = case["rotary"] // 2
    sizes = [case["first"], case["second"], pairs - case["first"] - case["second"]]
    axis = np.repeat(np.arange(3, dtype=np.int32), sizes)
    if case["shared"]:
        power = np.arange(pairs, dtype=np.float64) / max(1, pairs)
    else:
        power = np.concatenate([np.arange(n, dtype=np.float64) / max(1, n) for n in sizes])
    return torch.from_numpy(10000.0 ** -power).cuda(), torch.from_numpy(axis).cuda()


def _prepare_rope(case, g):
    batch, tokens, heads, dim = case["batch"], case["tokens"], case["heads"], case["dim"]
    rows = torch.randn(batch, tokens, (heads + 8) * dim, generator=g, device="cuda").to(TYPES[case["type"]])
    side = max(1, int(math.sqrt(max(1, tokens) / 4)))
    index = torch.arange(tokens, device="cuda")
    far = torch.randint(0, 100000, (3, batch, 1), generator=g, device="cuda")
    place = torch.stack([index // (side * side), index // side % side, index % side])
    freq, axis = _rope_tables(case)
    return {"x": rows[..., : heads * dim].view(batch, tokens, heads, dim), "freq": freq, "axis": axis,
            "positions": (place[:, None, :] + far).to(torch.int32)}


def _prepare_cells(case, g):
    tokens, heads, page = case["tokens"], case["heads"], case["page"]
    dtype = TYPES[case["type"]]
    slots = torch.randperm(case["capacity"], generator=g, device="cuda")[:tokens].to(torch.int32)
    unused = torch.randperm(tokens, generator=g, device="cuda")[: case["padding"]]
    slots[unused] = -1
    s = {"slots": slots, **_cache(case["capacity"] // page, heads, page, g, case["op"] == "read")}
    if case["op"] == "append":
        rows = _vectors((tokens, 6 * heads, DIM), dtype, g)  # the fused projection's rows: 4 query heads to a key head
        s["k"], s["v"] = rows[:, 4 * heads: 5 * heads], rows[:, 5 * heads:]
    return s


def _prepare_attend(case, seed, g):
    keys, news = _ragged(case)
    page = case["page"]
    need = [-(-k // page) for k in keys]
    total, wide = sum(need) + 1, max(1, max(need))
    order = torch.randperm(total, generator=g, device="cuda").cpu().numpy().astype(np.int32)
    pages = np.full((len(keys), wide), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at: at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    tokens = int(starts[-1])
    s = _cache(total, case["kv_heads"], page, g, True)
    s["q"] = torch.randn(tokens, case["heads"], DIM, generator=g, device="cuda").mul_(2.0).to(TYPES[case["type"]])
    s["pages"] = torch.from_numpy(pages).cuda()
    s["lengths"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    s["starts"] = s["tree"] = None
    if case["nodes"]:
        rng = np.random.default_rng(seed)
        tree = np.zeros(tokens, dtype=np.uint64)
        for b, n in enumerate(news):  # each drafted token follows one before it, or the context itself
            for i in range(n):
                parent = int(rng.integers(-1, i)) if i else -1
                line = tree[starts[b] + parent] if parent >= 0 else np.uint64(0)
                tree[starts[b] + i] = line | np.uint64(1 << i)
        s["starts"] = torch.from_numpy(starts).cuda()
        s["tree"] = torch.from_numpy(tree.view(np.int64)).cuda()
        s["most"] = max(news)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "rope":
        s = _prepare_rope(case, g)
    elif case["op"] == "attend":
        s = _prepare_attend(case, seed, g)
    else:
        s = _prepare_cells(case, g)
    if case["op"] != "rope":
        s["hadamard"] = _hadamard()
    s["case"] = case
    return s


# ------------------------------------------------------------------------------------ the operators


def _rotate(s, x):
    return torch.matmul(x, s["hadamard"]) * (1.0 / math.sqrt(DIM))


def _quantise(s, x):
    r = _rotate(s, x.float())
    scale = r.abs().amax(-1) / 127.0
    codes = torch.round(r / torch.where(scale > 0, scale, 1.0)[..., None]).clamp_(-127, 127)
    return codes, scale


def _rope(s):
    x, case = s["x"], s["case"]
    if own:
        import w8a8_rotated_int8_token_b200 as cr

        y = None
        if case["head_major"]:
            y = torch.empty(x.shape[0], x.shape[2], x.shape[1], x.shape[3], dtype=x.dtype, device=x.device)
        out = cr.convrot_rope(x, s["positions"], s["freq"], s["axis"], interleaved=case["interleaved"],
                              inverse=case["inverse"], Y=None if y is None else y.transpose(1, 2))
        return out if y is None else y
    angle = s["positions"].double()[s["axis"].long()].permute(1, 2, 0) * s["freq"]  # [batch, tokens, pairs]
    angle = (-angle if case["inverse"] else angle)[:, :, None, :]
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    r = case["rotary"]
    f = x.float()
    if case["interleaved"]:
        a, b = f[..., 0:r:2], f[..., 1:r:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = f[..., : r // 2], f[..., r // 2: r]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    y = torch.cat([y, f[..., r:]], -1).to(x.dtype)
    return y.transpose(1, 2).contiguous() if case["head_major"] else y


def _append(s):
    """Writes the new keys and values and reads them back as later tokens see them."""
    cells = (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if own:
        import w8a8_rotated_int8_token_b200 as cr

        cr.convrot_cache_append(s["k"], s["v"], s["slots"], *cells)
        return cr.convrot_cache_read(s["slots"], *cells, dtype=s["k"].dtype)
    page = s["k_codes"].shape[2]
    used = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][used].long()
    at, off = slots // page, slots % page
    for x, codes, scale in ((s["k"], cells[0], cells[2]), (s["v"], cells[1], cells[3])):
        c, f = _quantise(s, x[used])
        codes[at, :, off] = c.to(torch.int8)
        scale[at, :, off] = f
    return _read(s)


def _read(s):
    cells = (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    dtype = TYPES[s["case"]["type"]]
    if own:
        import w8a8_rotated_int8_token_b200 as cr

        return cr.convrot_cache_read(s["slots"], *cells, dtype=dtype)
    page = s["k_codes"].shape[2]
    slots = s["slots"].clamp_min(0).long()
    at, off = slots // page, slots % page
    there = (s["slots"] >= 0)[:, None, None]
    k = _rotate(s, cells[0][at, :, off].float() * cells[2][at, :, off][..., None])
    v = _rotate(s, cells[1][at, :, off].float() * cells[3][at, :, off][..., None])
    return torch.where(there, k, 0.0).to(dtype), torch.where(there, v, 0.0).to(dtype)


def _attend(s):
    q, case = s["q"], s["case"]
    if own:
        import w8a8_rotated_int8_token_b200 as cr

        return cr.convrot_cache_attention(q, s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["pages"],
                                          s["lengths"], starts=s["starts"], tree=s["tree"])
    device, batch, kv = q.device, s["lengths"].shape[0], case["kv_heads"]
    group = case["heads"] // kv
    starts = s["starts"] if s["starts"] is not None else torch.arange(batch + 1, device=device)
    most = s["most"] if s["starts"] is not None else 1
    new = starts.diff().long()
    step = torch.arange(most, device=device)
    token = (starts[:-1].long()[:, None] + step).clamp_max(q.shape[0] - 1)  # [batch, most]
    # the cache, padded: [batch, kv, keys, 128]
    ids = s["pages"].clamp_min(0).long()
    k = (s["k_codes"][ids].float() * s["k_scale"][ids][..., None]).transpose(1, 2).flatten(2, 3)
    v = (s["v_codes"][ids].float() * s["v_scale"][ids][..., None]).transpose(1, 2).flatten(2, 3)
    codes, scale = _quantise(s, q)
    rows = (codes * scale[..., None])[token].view(batch, most, kv, group, DIM).permute(0, 2, 1, 3, 4)
    logits = torch.matmul(rows.flatten(2, 3), k.transpose(2, 3)) * (1.0 / math.sqrt(DIM))
    logits = logits.view(batch, kv, most, group, -1)
    key = torch.arange(k.shape[2], device=device)
    context = s["lengths"].long() - new
    drafted = key - context[:, None]  # [batch, keys]
    if s["tree"] is not None:
        bits = (s["tree"][token][:, :, None] >> drafted.clamp(0, 63)[:, None, :]) & 1
        seen = (drafted[:, None, :] < 0) | (bits != 0)
    else:
        seen = drafted[:, None, :] <= step[:, None]
    seen = (seen & (key < s["lengths"][:, None])[:, None, :])[:, None, :, None, :]
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.flatten(2, 3), v).view(batch, kv, most, group, DIM)
    o = _rotate(s, o).permute(0, 2, 1, 3, 4).reshape(batch, most, case["heads"], DIM)
    there = step < new[:, None]
    return o[there].to(q.dtype)


def run(state):
    return {"rope": _rope, "append": _append, "read": _read, "attend": _attend}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["batch"] * case["tokens"]
        return {"bytes": 4.0 * n * case["heads"] * case["dim"] + 12.0 * n + 6.0 * case["rotary"],
                "flops": 3.0 * n * case["heads"] * case["rotary"]}
    if op in ("append", "read"):
        vectors = 2.0 * (case["tokens"] - case["padding"]) * case["heads"]
        cell, dense, both = DIM + 4.0, 2.0 * DIM, 2.0 * case["tokens"] * case["heads"] * 2.0 * DIM
        if op == "append":  # vectors in, cells out; cells in, vectors out
            return {"bytes": vectors * (dense + 2 * cell) + both + 4.0 * case["tokens"],
                    "flops": vectors * 2 * 7 * DIM}
        return {"bytes": vectors * cell + both + 4.0 * case["tokens"], "flops": vectors * 7 * DIM}
    keys, news = _ragged(case)
    return {"bytes": sum(keys) * case["kv_heads"] * 2.0 * (DIM + 4) + 4.0 * sum(news) * case["heads"] * DIM,
            "flops": 4.0 * DIM * case["heads"] * sum(k * n for k, n in zip(keys, news))}


# ------------------------------------------------------------------------ the definition in 64 bits


def _spin(x):
    """x R in 64 bits, by butterflies."""
    x = x.double()
    h = 1
    while h < DIM:
        x = x.reshape(*x.shape[:-1], DIM // (2 * h), 2, h)
        a, b = x[..., 0, :], x[..., 1, :]
        x = torch.stack([a + b, a - b], -2).flatten(-3)
        h *= 2
    return x / math.sqrt(DIM)


def _as_held(x):
    """The values that int8 codes of rotated vectors stand for, still rotated."""
    x = _spin(x)
    f = x.abs().amax(-1, keepdim=True) / 127
    return torch.where(f > 0, torch.round(x / f.clamp_min(1e-300)), 0.0) * f


def _exact_rope(s, case):
    x, r = s["x"].double(), case["rotary"]
    turn = torch.empty(*x.shape[:2], r // 2, dtype=torch.complex128, device=x.device)
    for i in range(r // 2):
        a = s["positions"][int(s["axis"][i])].double() * float(s["freq"][i])
        turn[..., i] = torch.complex(torch.cos(a), -torch.sin(a) if case["inverse"] else torch.sin(a))
    out = x.clone()
    for h in range(case["heads"]):
        u = x[:, :, h, :r]
        if case["interleaved"]:
            z = torch.view_as_complex(u.reshape(*u.shape[:2], r // 2, 2).contiguous()) * turn
            out[:, :, h, :r] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(u[..., : r // 2].contiguous(), u[..., r // 2:].contiguous()) * turn
            out[:, :, h, : r // 2], out[:, :, h, r // 2: r] = z.real, z.imag
    return out.permute(0, 2, 1, 3).contiguous() if case["head_major"] else out


def _exact_cells(s, case):
    slots = s["slots"].long()
    keep = (slots >= 0).double()[:, None, None]
    found = []
    for n in ("k", "v"):
        if case["op"] == "append":
            held = _as_held(s[n])
        else:
            flat = slots.clamp_min(0)
            heads = s[n + "_codes"].transpose(1, 2).reshape(-1, case["heads"], DIM)[flat].double()
            held = heads * s[n + "_scale"].transpose(1, 2).reshape(-1, case["heads"])[flat].double()[..., None]
        found.append(_spin(held) * keep)
    return tuple(found)


def _exact_attend(s, case):
    keys, news = _ragged(case)
    page, kv = case["page"], case["kv_heads"]
    group = case["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    tree = s["tree"].tolist() if s["tree"] is not None else None
    at = 0
    for length, n, table in zip(keys, news, s["pages"].tolist()):
        if length:
            ids = torch.tensor(table[: -(-length // page)], device="cuda")
            held = {}
            for x in ("k", "v"):
                c = s[x + "_codes"][ids].double() * s[x + "_scale"][ids].double()[..., None]
                held[x] = c.permute(1, 0, 2, 3).reshape(kv, -1, DIM)[:, :length]
            see = torch.ones(n, length, dtype=torch.bool)
            for i in range(n):
                for m in range(n):
                    if length - n + m >= 0:
                        see[i, length - n + m] = bool(tree[at + i] >> m & 1) if tree is not None else m <= i
            q = _as_held(s["q"][at: at + n]).view(n, kv, group, DIM)
            logits = torch.einsum("ihgd,hkd->higk", q, held["k"]) / math.sqrt(DIM)
            logits = logits.masked_fill(~see.cuda()[None, :, None, :], -math.inf)
            p = torch.softmax(logits, -1).nan_to_num(0.0)
            out[at: at + n] = _spin(torch.einsum("higk,hkd->ihgd", p, held["v"])).reshape(n, -1, DIM)
        at += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_cells, "read": _exact_cells, "attend": _exact_attend}[case["op"]](s, case)
