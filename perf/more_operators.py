"""Cases of speculation with a tree of drafted tokens over the paged cache: what each call
computes in plain torch, the library's own calls, the work one pass cannot do without, and the
results in 64 bits.

The operators (D = 64, 16-token blocks), each over both kinds of pools ("bf16", and "q8": e4m3
codes with one scale per (block, K/V head)):

  rope_append_at   rotate q and k by positions of their own, on one to four axes (a drafted
                   node's depth; an image's time, height and width), store k and v
  tree_attention   a sequence's last rows see every key before them, and of one another what a
                   bit mask says
  compact_tokens   the kept ones of a sequence's tokens move together, in place

A cached 8-bit value is code * scale.  The scale of a block and head is the smallest power of two
that brings the largest magnitude it has to hold to 448 or less; it grows while the block fills
(the codes held so far are then rescaled) and starts anew with the block's first token.
"""
import math
import random

import torch

own = False  # True: the library's kernels, False: the plain forms

HEAD_DIM = 64
PAIRS = HEAD_DIM // 2
BLOCK = 16
CODE_MAX = 448.0
MIN_EXP = -126
ROPE_BASE = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the drafted trees of a small batch on their way into the cache (latency)
        dict(name="rope_append_at trees 16 x 12", op="rope_append_at", pool="bf16", seqs=16, hkv=8, group=4, lo=100,
             hi=2000, new=12, new_hi=12, lengths=31, kind="tree", axes=1, cycled=False, interleaved=False, pad=0),
        # prompts with images: time, height and width in sections of the pairs
        dict(name="rope_append_at images 16k", op="rope_append_at", pool="bf16", seqs=20, hkv=8, group=4, lo=0, hi=700,
             new=300, new_hi=1300, lengths=32, kind="media", axes=3, cycled=False, interleaved=False, pad=0),
        # the same into the 8-bit pools, neighbouring dims paired, the axes taking turns
        dict(name="rope_append_at q8 images 12k", op="rope_append_at", pool="q8", seqs=20, hkv=8, group=4, lo=0, hi=700,
             new=200, new_hi=1000, lengths=33, kind="media", axes=3, cycled=True, interleaved=True, pad=0),
        # one short conversation with a small tree: the latency of one call
        dict(name="tree_attention one 300 x 12", op="tree_attention", pool="bf16", seqs=1, hkv=8, group=4, lo=300,
             hi=300, new=12, new_hi=12, lengths=34, kind="tree", pad=0),
        # a serving batch, trees of unlike size
        dict(name="tree_attention 32 ragged", op="tree_attention", pool="bf16", seqs=32, hkv=8, group=4, lo=100,
             hi=1500, new=8, new_hi=32, lengths=35, kind="tree", pad=0),
        # trees over very long contexts: the split over a long axis
        dict(name="tree_attention 4 x 131072 x 26", op="tree_attention", pool="bf16", seqs=4, hkv=8, group=4,
             lo=131072, hi=131072, new=26, new_hi=26, lengths=36, kind="tree", pad=0),
        # the latency of one call over the 8-bit pools
        dict(name="tree_attention q8 one 700 x 8", op="tree_attention", pool="q8", seqs=1, hkv=8, group=4, lo=700,
             hi=700, new=8, new_hi=8, lengths=37, kind="tree", pad=0),
        # a serving batch of mixed lengths, trees up to 64 nodes, rows of padding behind them
        dict(name="tree_attention q8 48 mixed", op="tree_attention", pool="q8", seqs=48, hkv=8, group=4, lo=1, hi=8192,
             new=4, new_hi=64, lengths=38, kind="forest", pad=7),
        # large trees over very long contexts
        dict(name="tree_attention q8 2 x 131072 x 60", op="tree_attention", pool="q8", seqs=2, hkv=8, group=4,
             lo=131072, hi=131072, new=60, new_hi=60, lengths=39, kind="tree", pad=0),
        # the accepted nodes of a verify step move behind the prefix (latency)
        dict(name="compact_tokens 32 x 5", op="compact_tokens", pool="bf16", seqs=32, hkv=8, lo=100, hi=2000, kept=1,
             kept_hi=5, span=26, lengths=40),
        # histories thinned out to half
        dict(name="compact_tokens 64 x 400", op="compact_tokens", pool="bf16", seqs=64, hkv=8, lo=0, hi=64, kept=300,
             kept_hi=500, span=1000, lengths=41),
        # the accepted nodes of many sequences in the 8-bit pools
        dict(name="compact_tokens q8 256 x 8", op="compact_tokens", pool="q8", seqs=256, hkv=8, lo=100, hi=500, kept=1,
             kept_hi=8, span=48, lengths=42),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append_at", "tree_attention", "tree_attention", "compact_tokens"])
    pool, hkv, tag = rng.choice(["bf16", "q8"]), rng.choice([1, 2, 3, 4, 8, 8]), rng.randrange(1 << 20)
    case = dict(op=op, pool=pool, hkv=hkv, lengths=tag)
    if op == "compact_tokens":
        seqs = _log_int(rng, 1, 300)
        top = min(_log_int(rng, 1, 1000), max(1, 25000 // seqs))
        case.update(seqs=seqs, lo=0, hi=_log_int(rng, 16, 2000), kept=rng.choice([0, 1, top]), kept_hi=top,
                    span=top + _log_int(rng, 1, 1000))
        return case
    case.update(group=rng.choice([1, 2, 4, 4]), pad=rng.choice([0, 0, 5]))
    if op == "rope_append_at":
        axes = rng.choice([1, 2, 3, 3, 4])
        seqs = _log_int(rng, 1, 200)
        top = _log_int(rng, 1, max(2, 14000 // seqs))
        case.update(seqs=seqs, lo=0, hi=_log_int(rng, 16, 1500), new=max(1, top // rng.choice([1, 4])), new_hi=top,
                    kind="tree" if top <= 100 else "media", axes=axes, cycled=rng.random() < 0.4,
                    interleaved=rng.random() < 0.5)
        return case
    seqs, nodes = _log_int(rng, 1, 64), _log_int(rng, 1, 200)
    top = min(_log_int(rng, 16, 131072), 4 * 131072 * 26 // (seqs * nodes), 300000 // seqs)
    case.update(seqs=seqs, lo=rng.choice([0, top // 50, top]), hi=top, new=max(1, nodes // rng.choice([1, 2, 5])),
                new_hi=nodes, kind=rng.choice(["chain", "tree", "forest", "mask"]))
    return case


def _lens(case):
    """(history, appended) tokens of every sequence: a function of the case alone."""
    r = random.Random(case["lengths"])
    lo, hi = case["lo"], case["hi"]
    if lo >= 1 and hi > 10 * lo:  # spread over the logarithm
        hist = [min(hi, max(lo, int(round(math.exp(r.gauss(0.5 * math.log(lo * hi) + 0.2 * math.log(hi / lo),
                                                            0.1 * math.log(hi / lo))))))) for _ in range(case["seqs"])]
    else:
        hist = [r.randint(lo, hi) for _ in range(case["seqs"])]
    if case["op"] == "compact_tokens":
        kept = [r.randint(case["kept"], case["kept_hi"]) for _ in range(case["seqs"])]
        return hist, [max(1, kept[0])] + kept[1:]
    return hist, [r.randint(case["new"], case["new_hi"]) for _ in range(case["seqs"])]


def _kept(case, seed):
    """Rising offsets of the kept tokens of every sequence, below the case's span."""
    r = random.Random(1000003 * case["lengths"] + seed)
    return [sorted(r.sample(range(case["span"]), n)) for n in _lens(case)[1]]


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- work
def work(case):
    hkv = case["hkv"]
    hist, new = _lens(case)
    size = 2 if case["pool"] == "bf16" else 1
    scales = 0 if case["pool"] == "bf16" else 8 * hkv  # of a block
    if case["op"] == "compact_tokens":
        # (of the tokens kept, those that stay where they are move in no pass, but they are few)
        n = sum(new)
        touched = sum(_blocks(h + k) - h // BLOCK for h, k in zip(hist, new) if k)
        return {"bytes": n * (2 * 2 * hkv * HEAD_DIM * size + 4) + 2 * touched * scales + 8 * case["seqs"], "flops": 0}
    hq = hkv * case["group"]
    t = sum(new)
    if case["op"] == "rope_append_at":
        touched = sum(_blocks(h + n) - h // BLOCK for h, n in zip(hist, new))
        b = t * (2 * hq * HEAD_DIM * 2 + 2 * hkv * HEAD_DIM * (2 + size) + HEAD_DIM * 4 + 4 * case["axes"])
        return {"bytes": b + touched * scales + 8 * case["seqs"], "flops": t * (hq + hkv) * HEAD_DIM * 3}
    ctx = [h + n for h, n in zip(hist, new)]
    b = sum(ctx) * hkv * 2 * HEAD_DIM * size + sum(_blocks(c) for c in ctx) * (4 + scales)
    b += 2 * t * hq * HEAD_DIM * 2 + t * 4 * -(-max(new) // 32)
    # (of the drafted keys, each row at least one)
    return {"bytes": b, "flops": 4 * HEAD_DIM * hq * sum(n * (h + 1) for h, n in zip(hist, new))}


# ---------------------------------------------------------------- inputs
def _power(e):
    """2^e as float32, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _needed_exp(amax):
    """Smallest e >= MIN_EXP with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _some_values(g, n, hkv, dev):
    """Keys or values of n tokens as a model makes them: a few strong channels, tokens of
    unlike size."""
    x = torch.randn(n, hkv, HEAD_DIM, generator=g, device=dev)
    x *= torch.exp(0.3 * torch.randn(n, 1, 1, generator=g, device=dev))
    chan = torch.exp(0.5 * torch.randn(1, hkv, HEAD_DIM, generator=g, device=dev))
    return (x * chan).to(torch.bfloat16)


def _pool(g, case, blocks, dev):
    """(pool, scales or None), every block full."""
    hkv = case["hkv"]
    x = _some_values(g, blocks * BLOCK, hkv, dev).view(blocks, BLOCK, hkv, HEAD_DIM).transpose(1, 2)
    if case["pool"] == "bf16":
        return x.contiguous(), None
    x = x.float()
    scale = _power(_needed_exp(x.abs().amax(dim=(2, 3))))
    return (x / scale[..., None, None]).contiguous().to(torch.float8_e4m3fn), scale


def _parents(r, kind, n):
    """The node each node of a tree hangs on (-1: on the prefix)."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "forest":
        return [-1 if r.random() < 0.3 else r.randint(-1, i - 1) for i in range(n)]
    return [-1 if i == 0 else r.randint(max(0, i - 6), i - 1) for i in range(n)]


def _seen(r, kind, n):
    """Row i's bits: which of the n drafted tokens it sees."""
    if kind == "mask":  # any bits; a few rows, as of unused nodes, see none
        return [0 if r.random() < 0.2 else r.getrandbits(n) for _ in range(n)]
    rows = []
    for i, p in enumerate(_parents(r, kind, n)):
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    return rows


def _positions(case, hist, new, seed):
    """[axes][tokens] of the appended tokens."""
    r = random.Random(1000003 * case["lengths"] + seed)
    out = [[] for _ in range(case["axes"])]
    for h, n in zip(hist, new):
        if case["kind"] == "tree":
            depth = []
            for p in _parents(r, "tree", n):
                depth.append(depth[p] + 1 if p >= 0 else 0)
            for row in out:
                row.extend(h + d for d in depth)
            continue
        width = r.randint(4, 12)  # of an image in patches; text and images of 60 tokens take turns
        for i in range(n):
            start, at = h + i // 60 * 60, i % 60
            place = [start, start + at // width, start + at % width, start + at // 2] if i // 60 % 2 else [h + i] * 4
            for row, p in zip(out, place):
                row.append(p)
    return out


def _pair_axes(case):
    """The axis of each of the 32 pairs: in turn, or in sections."""
    a = case["axes"]
    return [i % a for i in range(PAIRS)] if case["cycled"] else [min(i // (PAIRS // a // 4 * 4 or 1), a - 1) for i in range(PAIRS)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hkv = case["hkv"]
    hist, new = _lens(case)
    st = {"op": case["op"], "q8": case["pool"] == "q8", "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["op"] == "compact_tokens":
        kept = _kept(case, seed)
        ctx = [h + case["span"] for h in hist]
        st["kept"] = torch.tensor([k for ks in kept for k in ks], dtype=torch.int32).to(dev)
        st["max_kept"] = max(1, max(new))
        st["first"] = torch.tensor(hist, dtype=torch.int32).to(dev)
    else:
        ctx = [h + n for h, n in zip(hist, new)]
    st["starts"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    # tables: a shuffled pool dealt out in order
    per = [_blocks(c) for c in ctx]
    blocks = sum(per) + max(1, sum(per) // 10)
    base = torch.tensor([0] + per, dtype=torch.int64).cumsum(0).to(dev)
    perm = torch.randperm(blocks, generator=g, device=dev)
    col = torch.arange(max(per), device=dev)
    held = col[None, :] < (base[1:] - base[:-1])[:, None]
    at = (base[:-1, None] + col[None, :]).clamp(max=blocks - 1)
    st["bt"] = torch.where(held, perm[at], torch.full_like(at, -1)).to(torch.int32)
    st["ctx"] = torch.tensor(ctx, dtype=torch.int32).to(dev)
    st["kc"], st["ks"] = _pool(g, case, blocks, dev)
    st["vc"], st["vs"] = _pool(g, case, blocks, dev)
    if case["op"] == "compact_tokens":
        return st
    hq = hkv * case["group"]
    t = sum(new)
    st["tokens"], rows = t, t + case["pad"]  # rows of padding stay as they are
    if case["op"] == "rope_append_at":
        # the rows of one fused projection: [q | k | v] of every token
        qkv = torch.empty(rows, hq + 2 * hkv, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        for lo, n in ((0, hq), (hq, hkv), (hq + hkv, hkv)):
            qkv[:, lo:lo + n] = _some_values(g, rows, n, dev)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_out"] = torch.zeros(rows, hq, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        st["interleaved"], st["pair_axes"] = case["interleaved"], _pair_axes(case)
        p = torch.tensor(_positions(case, hist, new, seed), dtype=torch.int32)
        st["positions"] = torch.nn.functional.pad(p, (0, case["pad"])).to(dev).contiguous()
        # angles of far positions need 64 bits before the cosine
        pos = torch.arange(max(ctx) + 64, dtype=torch.float64, device=dev)
        inv = ROPE_BASE ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64, device=dev) / HEAD_DIM)
        ang = pos[:, None] * inv[None, :]
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        return st
    st["scale"], st["group"], st["max_new"] = HEAD_DIM ** -0.5, case["group"], max(new)
    st["q"] = (1.5 * torch.randn(rows, hq, HEAD_DIM, generator=g, device=dev)).to(torch.bfloat16)
    st["out"] = torch.zeros_like(st["q"])
    r = random.Random(1000003 * case["lengths"] + seed)
    words = -(-max(new) // 32)
    raw = b"".join(bits.to_bytes(4 * words, "little") for n in new for bits in _seen(r, case["kind"], n))
    raw += bytes(4 * words * case["pad"])
    st["mask"] = torch.frombuffer(bytearray(raw), dtype=torch.int32).view(rows, words).to(dev)
    # a serving program keeps one zeroed buffer, ample for its batches
    st["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"rope_append_at": _plain_rope_append_at, "tree_attention": _plain_tree_attention,
            "compact_tokens": _plain_compact_tokens}[st["op"]](st)


def _pools(st):
    return (st["kc"], st["vc"], st["ks"], st["vs"]) if st["q8"] else (st["kc"], st["vc"])


def _run_own(st):
    from paged_kv_cache_299_gb300 import binding as pa
    if st["op"] == "tree_attention":
        call = pa.pa_tree_attention_q8 if st["q8"] else pa.pa_tree_attention
        return call(st["out"], st["q"], st["mask"], st["starts"], st["max_new"], *_pools(st), st["bt"], st["ctx"],
                    st["scale"], workspace=st["workspace"], device_status=st["status"])
    if st["op"] == "rope_append_at":
        call = pa.pa_rope_append_at_q8 if st["q8"] else pa.pa_rope_append_at
        call(st["q"], st["k"], st["v"], st["cos_sin"], st["positions"], *_pools(st), st["bt"], st["ctx"],
             st["starts"], pair_axes=st["pair_axes"], q_out=st["q_out"], interleaved=st["interleaved"],
             device_status=st["status"])
        return st["q_out"], *_pools(st)
    call = pa.pa_compact_tokens_q8 if st["q8"] else pa.pa_compact_tokens
    call(st["kept"], st["starts"], st["first"], st["max_kept"], *_pools(st), st["bt"], device_status=st["status"])
    return _pools(st)


def _sequences(starts, n):
    """Sequence and place in it of n rows that follow one another."""
    t = torch.arange(n, device=starts.device)
    starts = starts.long()
    seq = torch.searchsorted(starts[1:], t, right=True)
    return seq, t - starts[seq]


def _plain_store_q8(x, codes, scales, block, off):
    """x [T, H, 64] float32 into codes [N, H, 16, 64] with scales [N, H]."""
    first = torch.full((codes.shape[0],), BLOCK, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, block, off, "amin")
    amax = torch.zeros(scales.shape, device=x.device)
    amax.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(dim=2), "amax")
    needed = _power(_needed_exp(amax))
    fresh, touched = (first == 0)[:, None], (first < BLOCK)[:, None]
    scale = torch.where(touched, torch.where(fresh, needed, torch.maximum(scales, needed)), scales)
    live = (torch.arange(BLOCK, device=x.device)[None] < first[:, None]) & touched  # tokens held before
    ratio = torch.where(live[:, None, :], (scales / scale)[..., None], torch.ones((), device=x.device))
    codes.copy_((codes.float() * ratio[..., None]).to(codes.dtype))
    codes.view(torch.uint8)[block, :, off] = (x / scale[block][..., None]).to(codes.dtype).view(torch.uint8)
    scales.copy_(scale)


def _plain_store(st, k, v, block, off):
    """float32 rows [T, H, 64] into the pools."""
    if st["q8"]:
        _plain_store_q8(k, st["kc"], st["ks"], block, off)
        _plain_store_q8(v, st["vc"], st["vs"], block, off)
    else:
        st["kc"][block, :, off] = k.to(torch.bfloat16)
        st["vc"][block, :, off] = v.to(torch.bfloat16)


def _plain_rope_append_at(st):
    n = st["tokens"]
    seq, i = _sequences(st["starts"], n)
    slot = (st["ctx"] - st["starts"].diff()).long()[seq] + i
    pair = torch.arange(PAIRS, device=slot.device)
    axis = torch.tensor(st["pair_axes"], device=slot.device)
    pos = st["positions"].long()[axis, :n].t()  # [T, 32]
    cos, sin = st["cos_sin"][pos, pair][:, None], st["cos_sin"][pos, pair + PAIRS][:, None]

    def turned(x):
        x = x[:n].float()
        a, b = (x[..., 0::2], x[..., 1::2]) if st["interleaved"] else (x[..., :PAIRS], x[..., PAIRS:])
        y = (a * cos - b * sin, b * cos + a * sin)
        return torch.stack(y, dim=-1).flatten(-2) if st["interleaved"] else torch.cat(y, dim=-1)

    st["q_out"][:n] = turned(st["q"])
    _plain_store(st, turned(st["k"]), st["v"][:n].float(), st["bt"].long()[seq, slot // BLOCK], slot % BLOCK)
    return st["q_out"], *_pools(st)


def _plain_gather(pool, scales, bt):
    """[S, Hkv, L, 64] float32 of every sequence, padded to the longest table."""
    at = bt.long().clamp(min=0)
    if scales is None:
        x = pool[at].float()
    else:
        x = pool.view(torch.uint8)[at].view(pool.dtype).float() * scales[at][..., None, None]  # [S, nb, H, 16, 64]
    s, nb, h = x.shape[:3]
    return x.transpose(1, 2).reshape(s, h, nb * BLOCK, HEAD_DIM)


def _plain_tree_attention(st):
    k, v = _plain_gather(st["kc"], st["ks"], st["bt"]), _plain_gather(st["vc"], st["vs"], st["bt"])
    s, hkv, length = k.shape[:3]
    group, rows, n = st["group"], st["max_new"], st["tokens"]
    seq, i = _sequences(st["starts"], n)
    count = st["starts"].diff().long()
    prefix = st["ctx"].long() - count
    q = torch.zeros(s, rows, hkv, group, HEAD_DIM, device=k.device)
    q[seq, i] = st["q"][:n].float().view(-1, hkv, group, HEAD_DIM)
    # what each row sees: all of the prefix, and of the drafted tokens its bits
    bits = (st["mask"][:n, :, None] >> torch.arange(32, dtype=torch.int32, device=k.device)) & 1
    drafted = torch.zeros(s, rows, rows, dtype=torch.bool, device=k.device)
    drafted[seq, i] = bits.flatten(1)[:, :rows] != 0
    key = torch.arange(length, device=k.device)[None] - prefix[:, None]  # [S, L] place among the drafted
    held = key < count[:, None]
    at = key.clamp(0, rows - 1)[:, None].expand(-1, rows, -1)
    seen = (drafted.gather(2, at) | (key < 0)[:, None]) & held[:, None]  # [S, R, L]
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device=v.device))
    q = q.permute(0, 2, 1, 3, 4).reshape(s, hkv, rows * group, HEAD_DIM)
    a = (q @ k.transpose(2, 3)) * st["scale"]
    a.masked_fill_(~seen.repeat_interleave(group, dim=1)[:, None], float("-inf"))
    top = a.amax(dim=3, keepdim=True)
    a = torch.exp(a - torch.where(top == -math.inf, torch.zeros((), device=a.device), top))
    o = (a @ v) / a.sum(dim=3, keepdim=True).clamp(min=1e-30)  # a row that sees nothing: 0
    o = o.view(s, hkv, rows, group, HEAD_DIM).permute(0, 2, 1, 3, 4)
    st["out"][:n] = o[seq, i].reshape(n, -1, HEAD_DIM)
    return st["out"]


def _plain_compact_tokens(st):
    seq, i = _sequences(st["starts"], st["kept"].shape[0])
    bt, first = st["bt"].long(), st["first"].long()[seq]
    src, dst = first + st["kept"].long(), first + i
    block, off = bt[seq, src // BLOCK], src % BLOCK
    rows = [st[n].view(torch.uint8 if st["q8"] else torch.bfloat16)[block, :, off].view(st[n].dtype).float()
            for n in ("kc", "vc")]
    if st["q8"]:
        rows = [x * st[n][block][..., None] for x, n in zip(rows, ("ks", "vs"))]
    _plain_store(st, *rows, bt[seq, dst // BLOCK], dst % BLOCK)
    return _pools(st)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree_attention":
        return _exact_tree(case, st, seed)
    hist, new = _lens(case)
    if case["op"] == "rope_append_at":
        q_out, n = st["q_out"].double(), sum(new)
        places = torch.tensor(_positions(case, hist, new, seed)).to(q_out.device)
        col = torch.arange(PAIRS, device=q_out.device)
        axis = torch.tensor(_pair_axes(case), device=q_out.device)
        table = st["cos_sin"].double()
        turn = torch.complex(table[places[axis], col[:, None]], table[places[axis], PAIRS + col[:, None]]).t()[:, None]

        def turned(x):
            x = x[:n].double()
            x = x.unflatten(-1, (PAIRS, 2)) if case["interleaved"] else x.unflatten(-1, (2, PAIRS)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(x.contiguous()) * turn)
            return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)

        q_out[:n] = turned(st["q"])
        pools = _exact_store(st, hist, new, (turned(st["k"]), st["v"][:n].double()))
        return (q_out, *pools)
    # the kept rows as they were, one sequence after the other
    tables, rows = st["bt"].tolist(), ([], [])
    for s, ks in enumerate(_kept(case, seed)):
        at = [hist[s] + k for k in ks]
        block = torch.tensor([tables[s][p // BLOCK] for p in at], dtype=torch.int64, device=st["kc"].device)
        off = torch.tensor([p % BLOCK for p in at], dtype=torch.int64, device=st["kc"].device)
        for out, pool, scale in zip(rows, ("kc", "vc"), ("ks", "vs")):
            x = st[pool].view(torch.uint8 if st["q8"] else torch.bfloat16)[block, :, off].view(st[pool].dtype).double()
            out.append(x * st[scale][block].double()[..., None] if st["q8"] else x)
    return _exact_store(st, hist, new, tuple(torch.cat(r) for r in rows))


def _exact_store(st, hist, new, rows):
    """The pools after the rows (float64, [T, H, 64], K and V) went to positions hist .. hist + new of
    their sequences; codes as real numbers, before their rounding."""
    pools = [st["kc"].double(), st["vc"].double()]
    scales = [st["ks"].double(), st["vs"].double()] if st["q8"] else None
    tables, at = st["bt"].tolist(), 0
    for s, (h, n) in enumerate(zip(hist, new)):
        for b in range(h // BLOCK, _blocks(h + n) if n else 0):
            lo, hi = max(h, b * BLOCK), min(h + n, (b + 1) * BLOCK)
            p, o = tables[s][b], lo % BLOCK
            for i, pool in enumerate(pools):
                x = rows[i][at + lo - h:at + hi - h].transpose(0, 1)  # [hkv, tokens, 64]
                if scales is None:
                    pool[p, :, o:o + hi - lo] = x
                    continue
                big = x.abs().amax(dim=(1, 2)).clamp(min=CODE_MAX * 2.0 ** MIN_EXP)
                need = torch.exp2(torch.ceil(torch.log2(big / CODE_MAX)))
                need = torch.where(big <= CODE_MAX * need / 2, need / 2, need)  # the logarithm rounds
                need = torch.where(big > CODE_MAX * need, 2 * need, need)
                grown = need if o == 0 else torch.maximum(need, scales[i][p])
                pool[p, :, :o] *= (scales[i][p] / grown)[:, None, None]
                pool[p, :, o:o + hi - lo] = x / grown[:, None, None]
                scales[i][p] = grown
        at += n
    return (*pools, *scales) if scales else tuple(pools)


def _exact_tree(case, st, seed):
    hist, new = _lens(case)
    hkv, group = case["hkv"], case["group"]
    r = random.Random(1000003 * case["lengths"] + seed)
    out, row = st["out"].double(), 0
    for s, (h, n) in enumerate(zip(hist, new)):
        length = h + n
        ids = st["bt"][s, :_blocks(length)].long()

        def cached(pool, scale):
            if st["q8"]:
                x = st[pool].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * st[scale][ids].double()[..., None, None]
            else:
                x = st[pool][ids].double()
            return x.permute(1, 0, 2, 3).reshape(hkv, -1, HEAD_DIM)[:, :length]

        k, v = cached("kc", "ks"), cached("vc", "vs")
        sees = torch.tensor([[bits >> j & 1 for j in range(n)] for bits in _seen(r, case["kind"], n)], device=k.device)
        step = max(1, 40_000_000 // (hkv * group * length))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = st["q"][row + r0:row + r1].double().view(r1 - r0, hkv, group, HEAD_DIM).permute(1, 0, 2, 3)
            a = (q.reshape(hkv, -1, HEAD_DIM) @ k.transpose(1, 2)).view(hkv, r1 - r0, group, length) * st["scale"]
            a[..., h:].masked_fill_((sees[r0:r1] == 0)[None, :, None], -math.inf)
            a = torch.softmax(a, dim=3).nan_to_num(0.0)  # (a row that sees nothing)
            o = (a.view(hkv, -1, length) @ v).view(hkv, r1 - r0, group, HEAD_DIM)
            out[row + r0:row + r1] = o.permute(1, 0, 2, 3).reshape(r1 - r0, -1, HEAD_DIM)
        row += n
    return out
