"""Cases of the 8-bit paged cache and of the appends that rotate keys on their way into a
paged cache: what each call computes in plain torch, the library's own calls, the work one
pass cannot do without, and the results in 64 bits.

The operators (D = 64, 16-token blocks):

  rope_append      rotate q and k by their positions, store k and v into the bf16 pools
  rope_append_q8   the same into pools of e4m3 codes with one scale per (block, K/V head)
  decode_q8        one query row per sequence over the 8-bit pools
  chunk_q8         causal chunks of query rows over the 8-bit pools
  copy_blocks_q8   copy-on-write copies of whole blocks, scales included

A cached value is code * scale.  The scale of a block and head is the smallest power of two
that brings the largest magnitude it has to hold to 448 or less; it grows while the block
fills (the codes held so far are then rescaled) and starts anew with the block's first token.
"""
import math
import random

import torch

own = False  # True: the library's kernels, False: the plain forms

HEAD_DIM = 64
BLOCK = 16
CODE_MAX = 448.0
MIN_EXP = -126
ROPE_BASE = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: rotate and store one token each (latency)
        dict(name="rope_append step 64", op="rope_append", seqs=64, hkv=8, group=4, lo=128, hi=2048,
             new=1, new_hi=1, lengths=11, interleaved=False),
        # a prefill step of ragged prompts over histories that end inside a block
        dict(name="rope_append prompts 16k", op="rope_append", seqs=24, hkv=8, group=4, lo=0, hi=500,
             new=250, new_hi=1100, lengths=12, interleaved=False),
        # a decode step of 256 sequences into the 8-bit pools: most blocks are half full
        dict(name="rope_append_q8 step 256", op="rope_append_q8", seqs=256, hkv=8, group=4, lo=1,
             hi=1500, new=1, new_hi=1, lengths=13, interleaved=False),
        # ragged prompts into the 8-bit pools, neighbouring dims paired
        dict(name="rope_append_q8 prompts 16k", op="rope_append_q8", seqs=24, hkv=8, group=4, lo=0,
             hi=500, new=250, new_hi=1100, lengths=14, interleaved=True),
        # a single short conversation: the latency of one call
        dict(name="decode_q8 one 300", op="decode_q8", seqs=1, hkv=8, group=4, lo=300, hi=300,
             lengths=15),
        # a serving batch of mixed lengths
        dict(name="decode_q8 256 mixed", op="decode_q8", seqs=256, hkv=8, group=4, lo=1, hi=8192,
             lengths=16),
        # four very long contexts: the split over a long axis
        dict(name="decode_q8 4 x 131072", op="decode_q8", seqs=4, hkv=8, group=4, lo=131072, hi=131072,
             lengths=17),
        # verification of a few drafted tokens: short chunks, memory-bound
        dict(name="chunk_q8 verify 32 x 5", op="chunk_q8", seqs=32, hkv=8, group=4, lo=100, hi=1500,
             new=5, new_hi=5, lengths=18),
        # the chunks of a continuous-batching step
        dict(name="chunk_q8 8 x 512", op="chunk_q8", seqs=8, hkv=8, group=4, lo=0, hi=2048, new=512,
             new_hi=512, lengths=19),
        # long prompts in large ragged chunks: bound by the matrix products
        dict(name="chunk_q8 3 x 4000", op="chunk_q8", seqs=3, hkv=8, group=4, lo=1000, hi=5000,
             new=3500, new_hi=4100, lengths=20),
        # a fork's few shared blocks
        dict(name="copy_blocks_q8 16", op="copy_blocks_q8", pairs=16, blocks=256, hkv=8),
        # many beams diverge at once
        dict(name="copy_blocks_q8 4096", op="copy_blocks_q8", pairs=4096, blocks=10000, hkv=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_append_q8", "decode_q8", "decode_q8", "chunk_q8", "chunk_q8",
                     "copy_blocks_q8"])
    hkv, group, tag = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([1, 2, 4, 4]), rng.randrange(1 << 20)
    if op == "copy_blocks_q8":
        pairs = _log_int(rng, 1, 4096)
        return dict(op=op, pairs=pairs, blocks=2 * pairs + rng.randrange(1, 1000), hkv=hkv)
    if op in ("rope_append", "rope_append_q8"):
        inter = rng.random() < 0.5
        if rng.random() < 0.5:  # decode steps
            return dict(op=op, seqs=_log_int(rng, 1, 512), hkv=hkv, group=group, lo=0,
                        hi=_log_int(rng, 16, 2000), new=1, new_hi=1, lengths=tag, interleaved=inter)
        seqs = _log_int(rng, 1, 32)
        top = _log_int(rng, 2, 16000 // seqs)
        return dict(op=op, seqs=seqs, hkv=hkv, group=group, lo=0, hi=_log_int(rng, 16, 600),
                    new=max(1, top // 4), new_hi=top, lengths=tag, interleaved=inter)
    if op == "decode_q8":
        seqs = _log_int(rng, 1, 300)
        top = min(_log_int(rng, 20, 131072), 300000 // seqs)
        return dict(op=op, seqs=seqs, hkv=hkv, group=group, lo=max(1, top // rng.choice([1, 4, 50])),
                    hi=top, lengths=tag)
    seqs = _log_int(rng, 1, 48)
    top = _log_int(rng, 2, 9000 // seqs)
    return dict(op=op, seqs=seqs, hkv=hkv, group=group, lo=0, hi=_log_int(rng, 16, 3000),
                new=max(1, top // 3), new_hi=top, lengths=tag)


def _lens(case):
    """(history, appended) tokens of every sequence: a function of the case alone."""
    r = random.Random(case["lengths"])
    lo, hi = case["lo"], case["hi"]
    if lo >= 1 and hi > 10 * lo:  # spread over the logarithm
        hist = [min(hi, max(lo, int(round(math.exp(r.gauss(0.5 * math.log(lo * hi) + 0.2 * math.log(hi / lo),
                                                            0.1 * math.log(hi / lo))))))) for _ in range(case["seqs"])]
    else:
        hist = [r.randint(lo, hi) for _ in range(case["seqs"])]
    new = [r.randint(case["new"], case["new_hi"]) for _ in range(case["seqs"])] if "new" in case else [0] * case["seqs"]
    return hist, new


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- work
def work(case):
    hkv = case["hkv"]
    if case["op"] == "copy_blocks_q8":
        per_block = hkv * (2 * BLOCK * HEAD_DIM + 8)
        return {"bytes": case["pairs"] * (2 * per_block + 16), "flops": 0}
    hq = hkv * case["group"]
    hist, new = _lens(case)
    if case["op"] in ("rope_append", "rope_append_q8"):
        t = sum(new)
        b = t * (2 * hq * HEAD_DIM * 2 + 2 * hkv * HEAD_DIM * 2 + HEAD_DIM * 4)  # q both ways, k, v, angles
        if case["op"] == "rope_append":
            b += t * 2 * hkv * HEAD_DIM * 2
        else:
            touched = sum(_blocks(h + n) - h // BLOCK for h, n in zip(hist, new))
            b += t * 2 * hkv * HEAD_DIM + touched * hkv * 8
        return {"bytes": b + 8 * case["seqs"], "flops": t * (hq + hkv) * HEAD_DIM * 3}
    ctx = [h + n for h, n in zip(hist, new)]
    rows = sum(new) if case["op"] == "chunk_q8" else case["seqs"]
    b = sum(ctx) * hkv * 2 * HEAD_DIM + sum(_blocks(c) for c in ctx) * (8 * hkv + 4)
    b += 2 * rows * hq * HEAD_DIM * 2
    if case["op"] == "chunk_q8":
        keys = sum(n * h + n * (n + 1) // 2 for h, n in zip(hist, new))
    else:
        keys = sum(ctx)
    return {"bytes": b, "flops": 4 * HEAD_DIM * hq * keys}


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


def _full_pool(g, blocks, hkv, dev):
    """(codes, scales) of a pool whose every block is full."""
    x = _some_values(g, blocks * BLOCK, hkv, dev).float().view(blocks, BLOCK, hkv, HEAD_DIM).transpose(1, 2)
    scale = _power(_needed_exp(x.abs().amax(dim=(2, 3))))
    return (x / scale[..., None, None]).contiguous().to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hkv = case["hkv"]
    st = {"op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["op"] == "copy_blocks_q8":
        st["kc"], st["ks"] = _full_pool(g, case["blocks"], hkv, dev)
        st["vc"], st["vs"] = _full_pool(g, case["blocks"], hkv, dev)
        perm = torch.randperm(case["blocks"], generator=g, device=dev)
        st["pairs"] = perm[: 2 * case["pairs"]].view(2, -1).t().contiguous()
        return st
    hq = hkv * case["group"]
    hist, new = _lens(case)
    ctx = [h + n for h, n in zip(hist, new)]
    per = [_blocks(c) for c in ctx]
    total = sum(per)
    blocks = total + max(1, total // 10)
    # tables: a shuffled pool dealt out in order
    width = max(per)
    base = torch.tensor([0] + per, dtype=torch.int64).cumsum(0).to(dev)
    perm = torch.randperm(blocks, generator=g, device=dev)
    col = torch.arange(width, device=dev)
    take = base[:-1, None] + col[None, :]
    held = col[None, :] < (base[1:] - base[:-1])[:, None]
    st["bt"] = torch.where(held, perm[take.clamp(max=blocks - 1)], torch.full_like(take, -1)).to(torch.int32)
    st["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    st["max_ctx"] = max(ctx)
    st["scale"] = HEAD_DIM ** -0.5
    st["group"] = case["group"]
    if case["op"] != "rope_append":
        st["kc"], st["ks"] = _full_pool(g, blocks, hkv, dev)
        st["vc"], st["vs"] = _full_pool(g, blocks, hkv, dev)
    if "new" in case:
        st["max_new"] = max(new)
        st["tokens"] = sum(new)
        one_each = case["new_hi"] == 1
        st["qsl"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
        st["starts"] = None if one_each and case["op"] != "chunk_q8" else st["qsl"]
    if case["op"] in ("rope_append", "rope_append_q8"):
        st["interleaved"] = case["interleaved"]
        t = st["tokens"]
        # the rows of one fused projection: [q | k | v] of every token
        qkv = torch.empty(t, hq + 2 * hkv, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        qkv[:, :hq] = _some_values(g, t, hq, dev)
        qkv[:, hq:hq + hkv] = _some_values(g, t, hkv, dev)
        qkv[:, hq + hkv:] = _some_values(g, t, hkv, dev)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_out"] = torch.empty(t, hq, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        # angles of far positions need 64 bits before the cosine
        pos = torch.arange(st["max_ctx"], dtype=torch.float64, device=dev)
        inv = ROPE_BASE ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64, device=dev) / HEAD_DIM)
        ang = pos[:, None] * inv[None, :]
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        if case["op"] == "rope_append":
            shape = (blocks, BLOCK, hkv, HEAD_DIM)
            st["kc"], st["vc"] = (_some_values(g, blocks * BLOCK, hkv, dev).view(shape).transpose(1, 2).contiguous()
                                  for _ in range(2))
        return st
    rows = st["tokens"] if case["op"] == "chunk_q8" else case["seqs"]
    st["q"] = (1.5 * torch.randn(rows, hq, HEAD_DIM, generator=g, device=dev)).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    if case["op"] == "decode_q8":  # a serving program keeps one zeroed buffer, ample for its batches
        st["workspace"] = torch.zeros(16 << 20, dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"rope_append": _plain_rope_append, "rope_append_q8": _plain_rope_append_q8,
            "decode_q8": _plain_decode_q8, "chunk_q8": _plain_chunk_q8,
            "copy_blocks_q8": _plain_copy_blocks_q8}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_299_gb300 import binding as pa
    op = st["op"]
    if op == "decode_q8":
        return pa.pa_decode_q8(st["out"], st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["bt"], st["ctx"],
                               st["scale"], st["max_ctx"], workspace=st["workspace"],
                               device_status=st["status"])
    if op == "chunk_q8":
        return pa.pa_prefill_chunk_q8(st["out"], st["q"], st["qsl"], st["max_new"], st["kc"], st["vc"], st["ks"],
                                      st["vs"], st["bt"], st["ctx"], st["scale"], device_status=st["status"])
    if op == "rope_append":
        pa.pa_rope_append(st["q"], st["k"], st["v"], st["cos_sin"], st["kc"], st["vc"], st["bt"], st["ctx"],
                          st["starts"], q_out=st["q_out"], interleaved=st["interleaved"],
                          device_status=st["status"])
        return st["q_out"], st["kc"], st["vc"]
    if op == "rope_append_q8":
        pa.pa_rope_append_q8(st["q"], st["k"], st["v"], st["cos_sin"], st["kc"], st["vc"], st["ks"], st["vs"],
                             st["bt"], st["ctx"], st["starts"], q_out=st["q_out"],
                             interleaved=st["interleaved"], device_status=st["status"])
        return st["q_out"], st["kc"], st["vc"], st["ks"], st["vs"]
    pa.pa_copy_blocks_q8(st["kc"], st["vc"], st["ks"], st["vs"], st["pairs"], device_status=st["status"])
    return st["kc"], st["vc"], st["ks"], st["vs"]


def _rotate(x, cos, sin, interleaved):
    """x [T, H, 64] float32, cos / sin [T, 32]."""
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., :HEAD_DIM // 2], x[..., HEAD_DIM // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _places(st):
    """Position, physical block and place in the block of every appended token."""
    t = torch.arange(st["tokens"], device=st["ctx"].device)
    qsl = st["qsl"].long()
    seq = torch.searchsorted(qsl[1:], t, right=True)
    pos = st["ctx"].long()[seq] - (qsl[seq + 1] - t)
    return pos, st["bt"].long()[seq, pos // BLOCK], pos % BLOCK


def _plain_rope_append(st):
    pos, block, off = _places(st)
    cos, sin = st["cos_sin"][pos].chunk(2, dim=1)
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, st["interleaved"]))
    st["kc"][block, :, off] = _rotate(st["k"].float(), cos, sin, st["interleaved"]).to(torch.bfloat16)
    st["vc"][block, :, off] = st["v"]
    return st["q_out"], st["kc"], st["vc"]


def _plain_store_q8(x, codes, scales, block, off):
    """x [T, H, 64] float32 into codes [N, H, 16, 64] with scales [N, H]."""
    first = torch.full((codes.shape[0],), BLOCK, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, block, off, "amin")
    amax = torch.zeros(scales.shape, device=x.device)
    amax.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(dim=2), "amax")
    needed = _power(_needed_exp(amax))
    kept = torch.maximum(scales, needed)
    fresh, touched = (first == 0)[:, None], (first < BLOCK)[:, None]
    scale = torch.where(touched, torch.where(fresh, needed, kept), scales)
    live = (torch.arange(BLOCK, device=x.device)[None] < first[:, None]) & touched  # tokens held before
    ratio = torch.where(live[:, None, :], (scales / scale)[..., None], torch.ones((), device=x.device))
    codes.copy_((codes.float() * ratio[..., None]).to(codes.dtype))
    codes.view(torch.uint8)[block, :, off] = (x / scale[block][..., None]).to(codes.dtype).view(torch.uint8)
    scales.copy_(scale)


def _plain_rope_append_q8(st):
    pos, block, off = _places(st)
    cos, sin = st["cos_sin"][pos].chunk(2, dim=1)
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, st["interleaved"]))
    _plain_store_q8(_rotate(st["k"].float(), cos, sin, st["interleaved"]), st["kc"], st["ks"], block, off)
    _plain_store_q8(st["v"].float(), st["vc"], st["vs"], block, off)
    return st["q_out"], st["kc"], st["vc"], st["ks"], st["vs"]


def _plain_gather(codes, scales, bt):
    """[S, Hkv, L, 64] float32 of every sequence, padded to the longest table."""
    at = bt.long().clamp(min=0)
    x = codes.view(torch.uint8)[at].view(codes.dtype).float() * scales[at][..., None, None]  # [S, nb, H, 16, 64]
    s, nb, h = x.shape[:3]
    return x.transpose(1, 2).reshape(s, h, nb * BLOCK, HEAD_DIM)


def _plain_attend(q, k, v, scale, seen):
    """q [S, Hkv, R, 64], k / v [S, Hkv, L, 64], seen [S, 1, R, L]."""
    a = (q @ k.transpose(2, 3)) * scale
    a = a.masked_fill(~seen, float("-inf"))
    a = torch.exp(a - a.amax(dim=3, keepdim=True))
    return (a @ v) / a.sum(dim=3, keepdim=True)


def _plain_decode_q8(st):
    k, v = _plain_gather(st["kc"], st["ks"], st["bt"]), _plain_gather(st["vc"], st["vs"], st["bt"])
    s, hkv, length = k.shape[:3]
    seen = torch.arange(length, device=k.device)[None, :] < st["ctx"][:, None]
    v = torch.where(seen[:, None, :, None], v, torch.zeros((), device=v.device))
    o = _plain_attend(st["q"].float().view(s, hkv, -1, HEAD_DIM), k, v, st["scale"], seen[:, None, None])
    st["out"].copy_(o.view(s, -1, HEAD_DIM))
    return st["out"]


def _plain_chunk_q8(st):
    k, v = _plain_gather(st["kc"], st["ks"], st["bt"]), _plain_gather(st["vc"], st["vs"], st["bt"])
    s, hkv, length = k.shape[:3]
    group, rows = st["group"], st["max_new"]
    t = torch.arange(st["tokens"], device=k.device)
    qsl = st["qsl"].long()
    seq = torch.searchsorted(qsl[1:], t, right=True)
    at = t - qsl[seq]
    q = torch.zeros(s, rows, hkv, group, HEAD_DIM, device=k.device)
    q[seq, at] = st["q"].float().view(-1, hkv, group, HEAD_DIM)
    pos = st["ctx"].long() - (qsl[1:] - qsl[:-1])
    pos = (pos[:, None] + torch.arange(rows, device=k.device)).clamp(max=length - 1)  # of every padded row
    key = torch.arange(length, device=k.device)
    held = key[None, :] < st["ctx"][:, None]
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device=v.device))
    seen = (key[None, None, :] <= pos[:, :, None]).repeat_interleave(group, dim=1)[:, None]
    q = q.permute(0, 2, 1, 3, 4).reshape(s, hkv, rows * group, HEAD_DIM)
    o = _plain_attend(q, k, v, st["scale"], seen).view(s, hkv, rows, group, HEAD_DIM)
    st["out"].copy_(o.permute(0, 2, 1, 3, 4)[seq, at].reshape(st["tokens"], -1, HEAD_DIM))
    return st["out"]


def _plain_copy_blocks_q8(st):
    src, dst = st["pairs"][:, 0], st["pairs"][:, 1]
    for name in ("kc", "vc"):
        raw = st[name].view(torch.uint8)
        raw[dst] = raw[src]
    for name in ("ks", "vs"):
        st[name][dst] = st[name][src]
    return st["kc"], st["vc"], st["ks"], st["vs"]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "copy_blocks_q8":
        out = [st[n].double() for n in ("kc", "vc", "ks", "vs")]
        for s, d in st["pairs"].tolist():
            for o, n in zip(out, ("kc", "vc", "ks", "vs")):
                o[d] = st[n][s].double()
        return tuple(out)
    if op in ("rope_append", "rope_append_q8"):
        return _exact_append(case, st)
    hist, new = _lens(case)
    hkv, group = case["hkv"], case["group"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    row = 0
    for s, (h, n) in enumerate(zip(hist, new)):
        length, n = h + n, max(n, 1)
        ids = st["bt"][s, :_blocks(length)].long()
        k = (st["kc"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * st["ks"][ids].double()[..., None, None])
        v = (st["vc"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * st["vs"][ids].double()[..., None, None])
        k = k.permute(1, 0, 2, 3).reshape(hkv, -1, HEAD_DIM)[:, :length]
        v = v.permute(1, 0, 2, 3).reshape(hkv, -1, HEAD_DIM)[:, :length]
        for r0 in range(0, n, 512):
            r1 = min(n, r0 + 512)
            keys = length - n + r1  # the last of these rows sees so many
            q = st["q"][row + r0:row + r1].double().view(r1 - r0, hkv, group, HEAD_DIM)
            a = torch.einsum("rhgd,hld->hrgl", q, k[:, :keys]) * st["scale"]
            late = torch.arange(keys, device=a.device)[None] > length - n + torch.arange(r0, r1, device=a.device)[:, None]
            a = torch.softmax(a.masked_fill(late[None, :, None, :], -math.inf), dim=3)
            out[row + r0:row + r1] = torch.einsum("hrgl,hld->rhgd", a, v[:, :keys]).reshape(r1 - r0, -1, HEAD_DIM)
        row += n
    return out


def _exact_append(case, st):
    """The rotated rows and the pools behind them; codes as real numbers, before their rounding."""
    hist, new = _lens(case)
    hkv = case["hkv"]
    table = st["cos_sin"].double()
    kc, vc = st["kc"].double(), st["vc"].double()
    scales = [st["ks"].double(), st["vs"].double()] if case["op"] == "rope_append_q8" else None
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(hist, new)]).to(table.device)
    half = HEAD_DIM // 2

    def turned(x):
        x = x.double()
        pairs = x.view(*x.shape[:-1], half, 2) if case["interleaved"] else x.view(*x.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_complex(pairs.contiguous())
        z = z * torch.complex(table[pos][:, :half], table[pos][:, half:])[:, None]
        y = torch.view_as_real(z)
        return (y if case["interleaved"] else y.transpose(-1, -2)).reshape(x.shape)

    q, rows = turned(st["q"]), (turned(st["k"]), st["v"].double())
    tables, at = st["bt"].tolist(), 0
    for s, (h, n) in enumerate(zip(hist, new)):
        for b in range(h // BLOCK, _blocks(h + n)):
            lo, hi = max(h, b * BLOCK), min(h + n, (b + 1) * BLOCK)
            p = tables[s][b]
            for i, pool in enumerate((kc, vc)):
                x = rows[i][at + lo - h:at + hi - h].transpose(0, 1)  # [hkv, tokens, 64]
                o = lo % BLOCK
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
    return (q, kc, vc) if scales is None else (q, kc, vc, *scales)
