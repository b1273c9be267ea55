"""Plain 64-bit forms of the rotating appends and of attention over the 8-bit cache, and the
tolerances of the tests that use them.  Everything runs on the CPU, loop by loop."""
from __future__ import annotations

import numpy as np
import torch

BLOCK, DIM, CODE_MAX = 16, 64, 448.0
E4M3_HALF_STEP = 2.0 ** -4      # relative, normal codes
E4M3_SUB_HALF_STEP = 2.0 ** -10  # absolute, below the smallest normal code 2^-6
BF16_HALF_STEP = 2.0 ** -8
FP32_HALF_STEP = 2.0 ** -24


def angles(positions, base=500000.0):
    """float32 [positions, 64]: cosines, then sines, from 64-bit angles."""
    inv = base ** (-np.arange(0, DIM, 2) / DIM)
    a = np.arange(positions)[:, None] * inv[None]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1)).float()


def rotate(x, table_rows, interleaved):
    """x [T, H, 64], table_rows [T, 64], in float64."""
    x = x.to(torch.float64)
    c, s = table_rows[:, None, :32].to(torch.float64), table_rows[:, None, 32:].to(torch.float64)
    y = torch.empty_like(x)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        y[..., 0::2], y[..., 1::2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :32], x[..., 32:]
        y[..., :32], y[..., 32:] = a * c - b * s, b * c + a * s
    return y


def rotation_error(x, interleaved):
    """Bound of the fp32 rotation's error: two products and a sum, each off by half a step of
    a value of at most |a| + |b|."""
    x = x.to(torch.float64).abs()
    if interleaved:
        m = (x[..., 0::2] + x[..., 1::2]).repeat_interleave(2, dim=-1)
    else:
        m = (x[..., :32] + x[..., 32:]).repeat(1, 1, 2)
    return 3 * FP32_HALF_STEP * m


def needed_scale(amax: float) -> float:
    """2^e of the smallest e >= -126 with amax <= 448 * 2^e."""
    e = -126
    while CODE_MAX * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def tokens_of(w):
    """(sequence, position) of every appended token of a workload, in order."""
    return [(s, int(h) + i) for s, (h, n) in enumerate(zip(w.hist_lens, w.new_lens)) for i in range(int(n))]


def store_q8(x, codes, scales, w):
    """The append's definition: x float64 [T, H, 64] (values after rotation) into float64 codes
    [N, H, 16, 64] and scales [N, H], in place; new codes are left unrounded.  Returns the
    (block, place) of every token."""
    groups = {}
    for t, (s, p) in enumerate(tokens_of(w)):
        groups.setdefault((s, p // BLOCK), []).append((t, p % BLOCK))
    where = [None] * len(x)
    for (s, b), items in groups.items():
        phys = int(w.block_tables[s, b])
        ts, offs = [t for t, _ in items], [o for _, o in items]
        for h in range(x.shape[1]):
            v = x[ts, h].abs()
            v = v[torch.isfinite(v)]
            scale = needed_scale(float(v.max()) if v.numel() else 0.0)
            if offs[0] > 0:
                old = float(scales[phys, h])
                if scale > old:
                    was = codes[phys, h, :offs[0]] * (old / scale)
                    codes[phys, h, :offs[0]] = was.float().to(torch.float8_e4m3fn).double()
                else:
                    scale = old
            scales[phys, h] = scale
            codes[phys, h, offs] = x[ts, h] / scale
        for t, o in items:
            where[t] = (phys, o)
    return where


def quantise(x):
    """float [N, H, 16, 64] -> (e4m3 codes, float32 scales [N, H]) by the cache's rule."""
    amax = x.abs().amax(dim=(2, 3)).double()
    scales = torch.tensor([needed_scale(float(a)) for a in amax.flatten()], dtype=torch.float64).view(amax.shape)
    codes = (x.double() / scales[..., None, None]).float().to(torch.float8_e4m3fn)
    return codes, scales.float()


def dequantise(codes, scales):
    return codes.float().double() * scales.double()[..., None, None]


def gather(pool, table, length):
    """[H, length, 64] of one sequence from a [N, H, 16, 64] pool."""
    ids = torch.as_tensor(np.asarray(table[: -(-length // BLOCK)]), dtype=torch.int64)
    return pool[ids].permute(1, 0, 2, 3).reshape(pool.shape[1], -1, DIM)[:, :length]


def attend(q, kpool, vpool, tables, context_lens, scale, q_lens=None):
    """Causal attention rows in float64 and their tolerance.  kpool / vpool float64 pools of
    values; q [rows, Hq, 64]; q_lens: rows per sequence (None: one each).

    Tolerance: the output's own rounding (half a bf16 step of it); the weights' rounding to
    bf16 at worst, half a step of each, so the same share of sum w |v|; the scores' error in
    fp32, at most 64 additions that may truncate (a whole step, 2^-23, each) of terms whose
    magnitudes sum to S = scale * sum |q k|, which moves every weight by twice that; and 2^-16
    for exponentials, sums and the final division."""
    rows, hq, _ = q.shape
    hkv = kpool.shape[1]
    group = hq // hkv
    out = torch.zeros(rows, hq, DIM, dtype=torch.float64)
    tol = torch.zeros_like(out)
    q = q.double()
    row = 0
    for s, length in enumerate(int(c) for c in context_lens):
        n = 1 if q_lens is None else int(q_lens[s])
        k, v = gather(kpool, tables[s], length), gather(vpool, tables[s], length)
        for i in range(n):
            keys = length - n + i + 1
            if keys <= 0:
                row += 1
                continue
            qr = q[row].view(hkv, group, DIM)
            a = torch.einsum("hgd,hld->hgl", qr, k[:, :keys]) * scale
            size = (torch.einsum("hgd,hld->hgl", qr.abs(), k[:, :keys].abs()) * scale).amax(dim=2)
            p = torch.softmax(a, dim=2)
            o = torch.einsum("hgl,hld->hgd", p, v[:, :keys])
            big = torch.einsum("hgl,hld->hgd", p, v[:, :keys].abs())
            delta = 2 * 64 * 2.0 ** -23 * size
            out[row] = o.reshape(hq, DIM)
            tol[row] = (BF16_HALF_STEP * o.abs() + (BF16_HALF_STEP + delta[..., None] + 2.0 ** -16) * big).reshape(hq, DIM)
            row += 1
    return out, tol
