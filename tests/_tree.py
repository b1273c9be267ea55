"""Drafted trees, their masks, and attention under them in 64 bits with the tests' tolerance."""
from __future__ import annotations

import random

import numpy as np
import torch

from _q8 import BF16_HALF_STEP, BLOCK, DIM, dequantise, quantise

KINDS = ("chain", "tree", "star", "mask")


def tree_bits(kind, n, rng):
    """One integer per row: bit j is set where the row sees drafted token j."""
    if kind == "mask":  # any bits, rows without one among them
        return [0 if rng.random() < 0.25 else rng.getrandbits(n) for _ in range(n)]
    rows = []
    for i in range(n):
        parent = {"chain": i - 1, "star": -1, "tree": rng.randint(max(-1, i - 5), i - 1)}[kind]
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    return rows


def batch_bits(kind, lens, seed):
    rng = random.Random(seed)
    return [tree_bits(kind, int(n), rng) for n in lens]


def mask_words(bits, lens, words=None, pad=0, junk=False):
    """int32 [rows + pad, words]; junk sets the bits that must not be looked at."""
    words = words or max(1, -(-max(int(n) for n in lens) // 32))
    raw = b""
    for rows, n in zip(bits, lens):
        for b in rows:
            if junk:
                b |= ((1 << 32 * words) - 1) ^ ((1 << int(n)) - 1)
            raw += b.to_bytes(4 * words, "little")
    raw += (b"\xff" if junk else b"\0") * (4 * words * pad)
    return torch.frombuffer(bytearray(raw), dtype=torch.int32).view(-1, words) if raw else torch.zeros(0, words, dtype=torch.int32)


def attend_tree(q, k64, v64, tables, context_lens, q_lens, bits, scale):
    """Rows in float64 and their tolerance.  q [rows, Hq, 64] bf16, k64 / v64 float64 pools [N, Hkv, 16,
    64] (on any device).  Keys that a row does not see are left out of its sums altogether.

    Tolerance: the output's own rounding (half a bf16 step of it); the weights' rounding to bf16,
    half a step of each, so the same share of sum w |v|; the scores' error in fp32, at most 64
    additions that may truncate (a whole step, 2^-23, each) of terms whose magnitudes sum to S =
    scale * sum |q k|, which moves every weight by twice that; and 2^-16 for exponentials, sums,
    the meeting of split rows and the final division."""
    rows, hq, _ = q.shape
    hkv = k64.shape[1]
    group = hq // hkv
    dev = k64.device
    out = torch.zeros(rows, hq, DIM, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    q = q.to(dev).double()
    row = 0
    for s, n in enumerate(int(x) for x in q_lens):
        length = int(context_lens[s])
        ids = torch.as_tensor(np.asarray(tables[s][: -(-length // BLOCK)]), dtype=torch.int64, device=dev)
        k, v = (p[ids].permute(1, 0, 2, 3).reshape(hkv, -1, DIM)[:, :length] for p in (k64, v64))
        prefix = length - n
        # rows that see the same drafted keys are one product
        for i, b in enumerate(bits[s]):
            seen = list(range(prefix)) + [prefix + j for j in range(n) if b >> j & 1]
            if seen:
                at = torch.tensor(seen, device=dev)
                kk, vv = k[:, at], v[:, at]
                qr = q[row + i].view(hkv, group, DIM)
                a = qr @ kk.transpose(1, 2) * scale
                size = ((qr.abs() @ kk.abs().transpose(1, 2)) * scale).amax(dim=2)
                p = torch.softmax(a, dim=2)
                o, big = p @ vv, p @ vv.abs()
                delta = 2 * 64 * 2.0 ** -23 * size
                out[row + i] = o.reshape(hq, DIM)
                tol[row + i] = (BF16_HALF_STEP * o.abs() + (BF16_HALF_STEP + delta[..., None] + 2.0 ** -16) * big).reshape(hq, DIM)
        row += n
    return out.cpu(), tol.cpu()


def random_pools(kind, num_blocks, hkv, seed, live=None, scales="powers", spread=0.5):
    """(tensors the call takes, float64 keys, float64 values).  Slots outside `live` ([N, 16] bool) hold
    poison: NaN, and NaN scales for blocks without a live slot."""
    g = torch.Generator().manual_seed(seed)
    pools, values, held = [], [], []
    for _ in range(2):
        x = torch.randn(num_blocks, hkv, 16, DIM, generator=g) * torch.exp(
            spread * torch.randn(num_blocks, hkv, 1, 1, generator=g))
        if kind == "bf16":
            x = x.to(torch.bfloat16)
            values.append(x.double())
            if live is not None:
                x = torch.where(live[:, None, :, None], x, torch.full_like(x, float("nan")))
            pools.append(x)
            continue
        codes, sc = quantise(x)
        if scales == "any":  # written by someone else: no powers of two
            sc = sc * (0.6 + torch.rand(sc.shape, generator=g))
        values.append(dequantise(codes, sc))
        if live is not None:
            raw = codes.view(torch.uint8).clone()
            raw[~live[:, None, :].expand(-1, hkv, -1)] = 0x7f
            codes = raw.view(torch.float8_e4m3fn)
            sc = torch.where(live.any(dim=1)[:, None], sc, torch.full_like(sc, float("nan")))
        pools.append(codes)
        held.append(sc)
    return pools + held, *values


def live_slots(num_blocks, tables, context_lens):
    live = torch.zeros(num_blocks, 16, dtype=torch.bool)
    for s, n in enumerate(int(c) for c in context_lens):
        for b in range(-(-n // 16)):
            live[int(tables[s, b]), :min(16, n - 16 * b)] = True
    return live


# Uneven batches, 4 query heads per K/V head: (pool, K/V heads, prefixes, nodes).  On 152 SMs neighbouring
# segments of more than ten pieces meet in one CTA, the first with its last piece (17, 25, ... in all) alone.
MEETING_BATCHES = {
    "bf16 one half": ("bf16", 8, [45519] * 2 + [326] * 18, [12] * 20),
    "bf16 two halves": ("bf16", 4, [45493] * 2 + [623] * 13, [40] * 15),
    "q8 short ones behind": ("q8", 4, [29294] * 2 + [363] * 14, [20] * 16),
    "q8 even": ("q8", 3, [131072] * 3, [40] * 3),
    "q8 more rows than a segment takes": ("q8", 4, [16217, 105684, 426], [101, 91, 107]),
}
