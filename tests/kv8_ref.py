"""Plain 64-bit forms of the paged 8-bit cache's operators, from their definitions, on the CPU.

A cache here is a dict of CPU tensors: codes uint8 [L, pages, 2, H, P, D], scales float32
[L, pages, 2, H, P / 16], table int32 [rows, W], lens int32 [rows], refs int32 [pages].
"""
import math

import numpy as np
import torch

TOP = 448.0
U_BF16, U_F16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half a step, relative


def e4m3_values():
    """Value of each of the 256 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[c] = math.nan if (c & 127) == 127 else (-x if c >= 128 else x)
    return torch.from_numpy(v)


VALUES = e4m3_values()
_POS = VALUES[:127]                     # ascending, 0 .. 448


def e4m3_code(x):
    """Code of the nearest value (float64 x), ties to the even code, saturating; NaN -> NaN."""
    a = x.abs().clamp(max=TOP)
    hi = torch.searchsorted(_POS, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = torch.where(torch.isnan(x), torch.full_like(pick, 127), pick)
    return (pick + torch.where(torch.signbit(x), 128, 0)).to(torch.uint8)


def scale_of(a):
    """The smallest power of two s >= 2^-126 with a <= 448 s."""
    a = float(a)
    if a == 0.0:
        return 2.0 ** -126
    e = math.frexp(a / TOP)[1] - 2
    while math.ldexp(TOP, e) < a:
        e += 1
    return math.ldexp(1.0, max(e, -126))


def values(cache, layer, row, n):
    """K and V of positions [0, n) of a row, float64 [2, n, H, D]; None where a page is missing."""
    codes, scales, table = cache["codes"][layer], cache["scales"][layer], cache["table"]
    P = codes.shape[3]
    out, there = [], []
    for p in range(n):
        page = int(table[row, p // P]) if p // P < table.shape[1] else -1
        ok = 0 <= page < codes.shape[0]
        there.append(ok)
        if ok:
            c, s = codes[page, :, :, p % P], scales[page, :, :, p % P // 16]
            out.append(VALUES[c.long()] * s.double()[..., None])
        else:
            out.append(torch.zeros(2, codes.shape[2], codes.shape[4], dtype=torch.float64))
    if not out:
        return torch.zeros(2, 0, codes.shape[2], codes.shape[4], dtype=torch.float64), torch.zeros(0, dtype=torch.bool)
    return torch.stack(out, 1), torch.tensor(there)


def append(cache, layer, k, v, cu, start):
    """In place; k, v [T, H, D] (any float type)."""
    codes, scales, table = cache["codes"][layer], cache["scales"][layer], cache["table"]
    P, W = codes.shape[3], table.shape[1]
    for b in range(len(start)):
        n, first = int(cu[b + 1]) - int(cu[b]), int(start[b])
        if n == 0:
            continue
        cache["lens"][b] = min(max(first + n, 0), W * P)
        if first < 0:
            continue
        for which, x in ((0, k), (1, v)):
            x = x[int(cu[b]):int(cu[b + 1])].double()
            for blk in range(first // 16, (first + n - 1) // 16 + 1):
                lo, hi = max(first, blk * 16), min(first + n, blk * 16 + 16)
                i = blk * 16 // P
                page = int(table[b, i]) if i < W else -1
                if not 0 <= page < codes.shape[0]:
                    continue
                slot = blk * 16 % P
                for h in range(codes.shape[2]):
                    part = x[lo - first:hi - first, h]
                    mag = torch.nan_to_num(part.abs(), nan=0.0, posinf=3.3895313892515355e38)
                    s = scale_of(mag.max())
                    if lo > blk * 16:
                        before = float(scales[page, which, h, slot // 16])
                        s = max(s, before)
                        if s > before:
                            kept = codes[page, which, h, slot:slot + lo - blk * 16]
                            kept.copy_(e4m3_code(VALUES[kept.long()] * (before / s)))
                    scales[page, which, h, slot // 16] = s
                    codes[page, which, h, slot + lo - blk * 16:slot + hi - blk * 16] = e4m3_code(part / s)


def attend(cache, layer, q, cu, kv_len, scale=None, split=False):
    """(out float64 [T, nq, D], bound [T, nq, D]): the value and how far a kernel may be from it.

    The kernel's roundings: the output to bf16 (half a step of it); each probability times its block's scale
    to f16, 2^-11 of it (or 2^-25 of 2^-15 of the largest, once below f16's normal range), which moves the
    weighted mean by at most 2^-11 of the weighted mean of |v|; fp32 scores, D products and sums of up to
    2^-23 of sum |q k| each (the accumulation of a tensor core may truncate), and the product with the scale and
    the log2 conversion, 4 roundings of the score, so the exponential is off by that absolute error and by
    2^-22 of its own; the sums of n terms and their rescalings, 2^-24 (n + 64) relative at most, in numerator
    and denominator.  split: q as two E4M3 values, each element off by up to 2^-18 of its row's largest, and the score
    by the sum of that times |k|."""
    T, nq, D = q.shape
    H = cache["codes"].shape[3]
    G = nq // H
    scale = D ** -0.5 if not scale else scale
    out = torch.zeros(T, nq, D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    cap = cache["table"].shape[1] * cache["codes"].shape[4]
    for b in range(len(kv_len)):
        lo, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        L = min(max(int(kv_len[b]), 0), cap)
        if n == 0:
            continue
        kv, there = values(cache, layer, b, L)
        pos = L - n + torch.arange(n)
        seen = (torch.arange(L)[None] <= pos[:, None]) & there[None]
        x = q[lo:lo + n].double().view(n, H, G, D)
        s = torch.einsum("nhgd,shd->hgns", x, kv[0]) * scale
        mag = torch.einsum("nhgd,shd->hgns", x.abs(), kv[0].abs()) * scale
        lost = torch.einsum("nhg,shd->hgns", x.abs().amax(-1), kv[0].abs()) * (scale * 2.0 ** -18 if split else 0.0)
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True) if L else torch.full(s.shape[:-1] + (1,), -math.inf, dtype=torch.float64)
        p = (s - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, torch.ones_like(total))
        o = torch.einsum("hgns,shd->nhgd", p, kv[1])
        off = (mag * D * 2.0 ** -23 + s.masked_fill(~seen, 0.0).abs() * 2.0 ** -22 + lost).masked_fill(~seen, 0.0)
        worst = off.amax(-1) if L else torch.zeros(s.shape[:-1], dtype=torch.float64)
        rel = U_F16 + 2 * (torch.expm1(worst) + 2.0 ** -22 + U_F32 * (L + 64))
        mean = torch.einsum("hgns,shd->nhgd", p, kv[1].abs()) * rel.permute(2, 0, 1)[..., None]
        vmax = kv[1][there].abs().amax() if bool(there.any()) else 0.0
        out[lo:lo + n] = o.reshape(n, nq, D)
        bound[lo:lo + n] = (o.abs() * U_BF16 * (1 + U_BF16) + mean * (1 + U_BF16) + L * 2.0 ** -39 * vmax + 1e-38).reshape(n, nq, D)
    return out, bound


def update(cache, parents, room):
    """(table, lens, refs, moves) or None when the pages do not suffice."""
    table, lens, pages = cache["table"], cache["lens"], cache["refs"].numel()
    P, (R, W) = cache["codes"].shape[4], table.shape
    parents = list(range(R)) if parents is None else [int(p) if 0 <= int(p) < R else -1 for p in parents]
    room = [0] * R if room is None else [max(0, int(r)) for r in room]
    new, new_lens, want, heirs = [], [], [], set()
    for b, p in enumerate(parents):
        row = [-1] * W
        n = 0
        if p >= 0:
            n = int(lens[p])
            if not 0 <= n <= W * P:
                n = 0
            old = [int(x) if 0 <= int(x) < pages else -1 for x in table[p]]
            keep = W if p not in heirs else n // P
            row[:keep] = old[:keep]
            ends = -(-(n + room[b]) // P)
            if ends > W:
                return None
            for i in range(ends):
                if row[i] < 0:
                    want.append((b, i, old[i] if old[i] >= 0 and i * P < n else -1))
            heirs.add(p)
        new.append(row)
        new_lens.append(n)
    used = {x for r in new for x in r if x >= 0}
    free = [p for p in range(pages) if p not in used]
    if len(want) > len(free):
        return None
    moves = []
    for (b, i, src), dst in zip(want, free):
        new[b][i] = dst
        if src >= 0:
            moves.append((src, dst))
    refs = [0] * pages
    for r in new:
        for x in r:
            if x >= 0:
                refs[x] += 1
    return torch.tensor(new, dtype=torch.int32), torch.tensor(new_lens, dtype=torch.int32), \
        torch.tensor(refs, dtype=torch.int32), moves


def compact(cache):
    refs = cache["refs"].tolist()
    used = [p for p, r in enumerate(refs) if r > 0]
    U = len(used)
    holes = [p for p in range(U) if refs[p] <= 0]
    moves = list(zip([p for p in used if p >= U], holes))
    to = {a: z for a, z in moves}
    new_refs = [max(r, 0) if p < U else 0 for p, r in enumerate(refs)]
    for a, z in moves:
        new_refs[z] = refs[a]
    table = [[to.get(int(x), int(x)) for x in r] for r in cache["table"]]
    return torch.tensor(table, dtype=torch.int32), cache["lens"].clone(), torch.tensor(new_refs, dtype=torch.int32), moves


def move(cache, moves):
    """The page copies of update / compact, in every layer."""
    codes, scales = cache["codes"].clone(), cache["scales"].clone()
    for a, z in moves:
        codes[:, z] = cache["codes"][:, a]
        scales[:, z] = cache["scales"][:, a]
    return codes, scales
