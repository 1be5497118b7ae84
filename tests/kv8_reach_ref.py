"""Plain 64-bit forms of attention through a window and of page updates with one, from their definitions, on the CPU."""
import math

import torch

import kv8_ref as R


def attend(cache, layer, q, cu, kv_len, window, sinks, scale=None, split=False):
    """(out, bound) as kv8_ref.attend, whose docstring has the bound's terms; a token at position p sees those of [0, p] from
    p - window + 1 on and those below sinks."""
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
        if n == 0 or L == 0:
            continue
        kv, there = R.values(cache, layer, b, L)
        j = torch.arange(L)[None]
        pos = (L - n + torch.arange(n))[:, None]
        seen = (j <= pos) & ((j > pos - window) | (j < sinks)) & there[None]
        some = seen.any(0)
        kv = torch.where(some[None, :, None, None], kv, torch.zeros((), dtype=torch.float64))   # the rest is not looked at
        x = q[lo:lo + n].double().view(n, H, G, D)
        s = (torch.einsum("nhgd,shd->hgns", x, kv[0]) * scale).masked_fill(~seen, -math.inf)
        mag = torch.einsum("nhgd,shd->hgns", x.abs(), kv[0].abs()) * scale
        lost = torch.einsum("nhg,shd->hgns", x.abs().amax(-1), kv[0].abs()) * (scale * 2.0 ** -18 if split else 0.0)
        top = s.amax(-1, keepdim=True)
        p = (s - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, torch.ones_like(total))
        o = torch.einsum("hgns,shd->nhgd", p, kv[1])
        off = (mag * D * 2.0 ** -23 + s.masked_fill(~seen, 0.0).abs() * 2.0 ** -22 + lost).masked_fill(~seen, 0.0)
        count = int(seen.sum(-1).max())
        rel = R.U_F16 + 2 * (torch.expm1(off.amax(-1)) + 2.0 ** -22 + R.U_F32 * (count + 64))
        mean = torch.einsum("hgns,shd->nhgd", p, kv[1].abs()) * rel.permute(2, 0, 1)[..., None]
        vmax = kv[1][some].abs().amax() if bool(some.any()) else 0.0
        out[lo:lo + n] = o.reshape(n, nq, D)
        bound[lo:lo + n] = (o.abs() * R.U_BF16 * (1 + R.U_BF16) + mean * (1 + R.U_BF16) + count * 2.0 ** -39 * vmax
                            + 1e-38).reshape(n, nq, D)
    return out, bound


def gone(n, P, window, sinks, i):
    """Whether page i of a row of n positions is behind the window of every later token, and holds no sink."""
    return i * P >= sinks and (i + 1) * P <= n - window + 1


def update(cache, parents, room, window, sinks):
    """(table, lens, refs, moves) or None when the pages do not suffice."""
    table, lens, pages = cache["table"], cache["lens"], cache["refs"].numel()
    P, (rows, W) = cache["codes"].shape[4], table.shape
    new, new_lens, want, heirs = [], [], [], set()
    for b, p in enumerate([int(p) for p in parents]):
        row, n = [-1] * W, 0
        if p >= 0:
            n = int(lens[p])
            old = [-1 if gone(n, P, window, sinks, i) else int(x) for i, x in enumerate(table[p])]
            keep = W if p not in heirs else n // P
            row[:keep] = old[:keep]
            ends = -(-(n + int(room[b])) // P)
            if ends > W:
                return None
            for i in range(ends):
                if row[i] < 0 and not gone(n, P, window, sinks, i):
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
