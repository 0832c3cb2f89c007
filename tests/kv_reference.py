"""Plain 64-bit (numpy) forms of the paged 8-bit cache operators: block assignment token by
token, the quantising append run by run, attention row by row.  Test infrastructure; shares no
code with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def decode(codes: torch.Tensor) -> np.ndarray:
    """Code values (before the scale)."""
    return codes.detach().cpu().float().numpy().astype(np.float64)


def scale_of(amax: float, dtype) -> float:
    e = -64
    while amax > QMAX[dtype] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_code_values(x: np.ndarray, dtype) -> np.ndarray:
    """Nearest code values, ties to even, saturated; NaN kept (e4m3) or 0 (int8)."""
    m = QMAX[dtype]
    y = np.clip(x, -m, m)
    if dtype == torch.int8:
        return np.rint(np.where(np.isnan(y), 0.0, y))
    a = np.abs(y)
    _, e = np.frexp(np.where(np.isfinite(a), a, 1.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(y / step) * step


def append(k, v, slots, values, scales, dtype):
    """values [n_blocks, Hkv, 2, bs, d] (code values) and scales, float64, updated in place."""
    n_blocks, _, _, bs, _ = values.shape
    slots = [int(s) for s in slots]
    valid = [0 <= s < n_blocks * bs for s in slots]
    a = 0
    while a < len(slots):
        if not valid[a]:
            a += 1
            continue
        b = a + 1
        while b < len(slots) and valid[b] and slots[b] == slots[b - 1] + 1 and slots[b] % bs:
            b += 1
        blk, off = divmod(slots[a], bs)
        for half, x in enumerate((k, v)):
            for h in range(x.shape[1]):
                rows = x[a:b, h]
                fin = np.abs(rows[np.isfinite(rows)])
                s = scale_of(float(fin.max()) if fin.size else 0.0, dtype)
                if off:
                    old = scales[blk, h, half]
                    s = max(s, old)
                    if s > old:
                        values[blk, h, half, :off] = to_code_values(values[blk, h, half, :off] * (old / s), dtype)
                values[blk, h, half, off:off + b - a] = to_code_values(rows / s, dtype)
                scales[blk, h, half] = s
        a = b


def assign(new, lens, table, ring, span, bs, n_slots):
    """Returns (slots, cu, lens, span); table and ring (lists of lists / list) updated in place."""
    n = len(ring)
    width = len(table[0])
    head, count = span
    taken, wanted, back, given = 0, 0, [], False
    slots, cu, out = [-1] * n_slots, [0], []
    front = [ring[(head + i) % n] for i in range(count)]
    for s, (a, ln) in enumerate(zip(new, lens)):
        ln = min(max(ln, 0), width * bs)
        have = -(-ln // bs)
        if a < 0:
            back += table[s][:have]
            cu.append(cu[-1])
            out.append(0)
            continue
        cu.append(cu[-1] + a)
        need = -(-(ln + a) // bs) - have
        fits = ln + a <= width * bs and cu[-1] <= n_slots
        if fits:
            wanted += need
        if not fits or (need and wanted > count):
            out.append(ln)
            continue
        for j in range(need):
            table[s][have + j] = front[taken]
            taken += 1
        for t in range(a):
            p = ln + t
            b = table[s][p // bs]
            if 0 <= b < n:
                slots[cu[-2] + t] = b * bs + p % bs
        out.append(ln + a)
    for i, b in enumerate(back):
        ring[(head + count + i) % n] = b
    return slots, cu, out, [(head + taken) % n, count - taken + len(back)]


def attention(q, values, scales, table, lens):
    """q [B, n_q, Hq, d], values/scales float64.  Returns (out, spread, reach, wmax): spread = sum_j w_j |v_j|,
    reach = max_j sum |q_e k_je| / sqrt(d), wmax = the largest weight times sum_j |v_j|: what
    the rounding errors of a row scale with."""
    B, nq, Hq, d = q.shape
    n_blocks, Hkv, _, bs, _ = values.shape
    out = np.zeros(q.shape)
    spread, reach, wmax = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape)
    for s in range(B):
        n = int(min(max(lens[s], 0), table.shape[1] * bs))
        pos = [p for p in range(n) if 0 <= table[s][p // bs] < n_blocks]
        if not pos:
            continue
        blk = np.array([table[s][p // bs] for p in pos])
        off = np.array(pos) % bs
        pos = np.array(pos)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            K = values[blk, g, 0, off] * scales[blk, g, 0][:, None]
            V = values[blk, g, 1, off] * scales[blk, g, 1][:, None]
            for i in range(nq):
                see = pos <= n - nq + i
                if not see.any():
                    continue
                Ki, Vi = K[see], V[see]
                x = Ki @ q[s, i, h] / math.sqrt(d)
                w = np.exp(x - x.max())
                w /= w.sum()
                out[s, i, h] = w @ Vi
                spread[s, i, h] = w @ np.abs(Vi)
                reach[s, i, h] = (np.abs(Ki) @ np.abs(q[s, i, h])).max() / math.sqrt(d)
                wmax[s, i, h] = w.max() * np.abs(Vi).sum(0)
    return out, spread, reach, wmax


def attention_tolerance(ref, dtype, d):
    """Bound of the kernel's error, from its roundings.  With u = 2^-24:
    - a score is a sum of d fp32 products of exact operands (fp32 queries: two fp16 terms that
      keep 22 bits), at most (d + 8) u reach off, and its log2 form is rounded a few times more
      relative to its size (8 u reach); a weight is then off by that, plus 2^-21 for the
      exponential, in its numerator and in the sum: twice;
    - a weight enters the second product in fp16, off by 2^-11 of itself (fp32: two terms, 2^-22), or by
      2^-25 absolutely, where the largest is at least 2^7 (2^-32 of it); its sum over tokens rounds
      by 2^-22 more at most here;
    - the output is rounded to its type, half a step."""
    out, spread, reach, wmax = ref
    fp32 = dtype == torch.float32
    u = 2.0 ** -24
    rel = 2 * ((d + 16) * u + (2.0 ** -22 if fp32 else 0.0)) * reach[..., None] + 2 * 2.0 ** -21 + 2.0 ** -20
    rel = rel + (2.0 ** -22 if fp32 else 2.0 ** -11)
    half = torch.finfo(dtype).eps / 2
    err = rel * spread + 2.0 ** -32 * wmax
    return err + half * (np.abs(out) + err) + 1e-30
