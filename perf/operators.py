"""Measured cases of the paged 8-bit key/value cache.

Operators:
  append   new K/V rows (bf16) of ragged sequences into the pages of an E4M3 cache, one fp32 scale for
           each block of 16 tokens, head, and K or V;
  attend   causal grouped-query attention of the new tokens over that cache: single tokens of an audio
           frame, whole prompts, and prompt chunks after cached positions;
  update   the page tables of the next step: rows forked, reordered or freed, pages taken for new tokens,
           shared part-filled pages copied in every layer;
  compact  the pages in use moved to the low end of the pool in every layer, tables rewritten.

``run`` computes them in elementary torch operations in fp32, or, where ``own`` is true, with the
library's calls.  Lengths, parents and page numbers come from the case alone (its "ragged" number), so
that ``work`` is exact; values come from the seed.
"""
import random

import numpy as np
import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_BLOCK = 16          # tokens that share a scale
_TOP = 448.0         # largest E4M3 value
_E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------- cases

def listed():
    full = {"q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64}
    tiny = {"q_heads": 4, "kv_heads": 2, "head_dim": 64, "page": 16}
    return [
        # one audio frame of 8 running streams: one token a row, most of them inside a part-filled block
        {"name": "append frame", "op": "append", "batch": 8, "new_lo": 1, "new_hi": 1, "kept_lo": 1024,
         "kept_hi": 2112, "ragged": 1, **full},
        # the keys and values of 8 long prompts
        {"name": "append prompts", "op": "append", "batch": 8, "new_lo": 1024, "new_hi": 2048, "kept_lo": 0,
         "kept_hi": 0, "ragged": 2, **full},
        # one frame of one short stream on the small model: latency alone
        {"name": "frame short", "op": "attend", "batch": 1, "new_lo": 1, "new_hi": 1, "kept_lo": 203,
         "kept_hi": 203, "ragged": 3, **tiny},
        # one frame of 8 streams after long prompts
        {"name": "frame long", "op": "attend", "batch": 8, "new_lo": 1, "new_hi": 1, "kept_lo": 1024,
         "kept_hi": 2112, "ragged": 4, **full},
        # a full server: 64 streams between their first and their eight-thousandth position
        {"name": "frame wide", "op": "attend", "batch": 64, "new_lo": 1, "new_hi": 1, "kept_lo": 15,
         "kept_hi": 8191, "ragged": 5, **full},
        # 32 short ragged prompts
        {"name": "prompts short", "op": "attend", "batch": 32, "new_lo": 16, "new_hi": 256, "kept_lo": 0,
         "kept_hi": 0, "ragged": 6, **full},
        # 8 long ragged prompts
        {"name": "prompts long", "op": "attend", "batch": 8, "new_lo": 1024, "new_hi": 2048, "kept_lo": 0,
         "kept_hi": 0, "ragged": 7, **full},
        # later chunks of very long prompts, 2 rows, odd sizes
        {"name": "prompts chunked", "op": "attend", "batch": 2, "new_lo": 500, "new_hi": 1021, "kept_lo": 9001,
         "kept_hi": 16001, "ragged": 8, **full},
        # one step of a server: most rows take a token, some end, some start as copies of others
        {"name": "update step", "op": "update", "layers": 36, "rows": 64, "held": 56, "len_lo": 1, "len_hi": 512,
         "fork": 1, "ended": 6, "room": 1, "spare": 80, "ragged": 9, "kv_heads": 8, "head_dim": 128, "page": 64},
        # 8 prompts of which each gets three more continuations
        {"name": "update fork", "op": "update", "layers": 36, "rows": 32, "held": 8, "len_lo": 1024, "len_hi": 2048,
         "fork": 4, "ended": 0, "room": 64, "spare": 80, "ragged": 10, "kv_heads": 8, "head_dim": 128, "page": 64},
        # a pool of the small model after a few streams have ended
        {"name": "compact small", "op": "compact", "layers": 2, "rows": 8, "len_lo": 1, "len_hi": 96, "pool": 96,
         "ragged": 11, "kv_heads": 2, "head_dim": 64, "page": 16},
        # a pool of the full-width model, about half of it in use
        {"name": "compact large", "op": "compact", "layers": 36, "rows": 16, "len_lo": 512, "len_hi": 1536,
         "pool": 512, "ragged": 12, "kv_heads": 8, "head_dim": 128, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "attend frame", "attend frame", "attend prompt", "attend prompt", "update", "compact"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op.split()[0], "ragged": rng.randrange(1 << 20), "kv_heads": kv, "head_dim": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 64, 128])}
    if case["op"] in ("append", "attend"):
        case["q_heads"] = kv * rng.choice([1, 2, 4, 8] if kv < 8 else [1, 2, 4])
    if op == "append":
        hi = _log_int(rng, 1, 2048)
        kept = rng.choice([0, _log_int(rng, 1, 4096)])
        case.update(batch=_log_int(rng, 1, 64) if hi < 256 else _log_int(rng, 1, 8), new_lo=rng.randint(1, hi), new_hi=hi,
                    kept_lo=rng.randint(0, kept), kept_hi=kept)
    elif op == "attend frame":
        kept = _log_int(rng, 1, 8191)
        case.update(batch=_log_int(rng, 1, 64), new_lo=1, new_hi=rng.choice([1, 1, 1, 2, 4]), kept_lo=rng.randint(0, kept), kept_hi=kept)
    elif op == "attend prompt":
        hi = _log_int(rng, 5, 2048)
        kept = rng.choice([0, _log_int(rng, 1, 4096)])
        batch = max(1, min(_log_int(rng, 1, 64), (8 * 2048 * 2048) // (hi * (hi + kept))))
        case.update(batch=batch, new_lo=rng.randint(1, hi), new_hi=hi, kept_lo=rng.randint(0, kept), kept_hi=kept)
    elif op == "update":
        rows = _log_int(rng, 2, 64)
        hi = _log_int(rng, 1, 1024)
        held = rng.randint(1, rows)
        case.update(layers=_log_int(rng, 1, 36), rows=rows, held=held, len_lo=rng.randint(0, hi), len_hi=hi,
                    fork=rng.choice([1, 1, 2, 3, 4]), ended=rng.randint(0, held // 2), room=rng.choice([0, 1, 16, 65]),
                    spare=rows * 5 + 8)
    else:
        rows = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, 1024)
        used = rows * (-(-hi // case["page"]))
        case.update(layers=_log_int(rng, 1, 36), rows=rows, len_lo=rng.randint(0, hi), len_hi=hi,
                    pool=used + _log_int(rng, 1, max(2, used)))
        # no more bytes than the largest listed pool
        page_bytes = 2 * kv * case["page"] * case["head_dim"]
        case["layers"] = max(1, min(case["layers"], (36 * 512 * 131072) // (page_bytes * case["pool"])))
    return case


def _pages_of(n, page):
    return -(-n // page)


def _lengths(case):
    """(new tokens, kept tokens) of every sequence."""
    rng = random.Random(case["ragged"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    kept = [rng.randint(case["kept_lo"], case["kept_hi"]) for _ in range(case["batch"])]
    return new, kept


def _plan(case):
    """The rows before an update or a compaction: lengths, page numbers of each row, pool size, parents."""
    rng = random.Random(case["ragged"])
    P, rows = case["page"], case["rows"]
    if case["op"] == "compact":
        lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(rows)]
        ids = rng.sample(range(case["pool"]), sum(_pages_of(n, P) for n in lens))
        parents, pool = None, case["pool"]
    else:
        lens = [rng.randint(case["len_lo"], case["len_hi"]) if b < case["held"] else 0 for b in range(rows)]
        used = sum(_pages_of(n, P) for n in lens)
        pool = used + case["spare"]
        ids = rng.sample(range(pool), used)
        if case["fork"] > 1:   # the held rows' continuations side by side
            parents = [b // case["fork"] if b // case["fork"] < case["held"] else -1 for b in range(rows)]
        else:                  # rows stay; the free ones start as copies of a row, some end
            parents = [b if b < case["held"] else rng.randrange(case["held"]) for b in range(rows)]
        for b in rng.sample(range(case["held"]), case["ended"]):
            parents[b] = -1
    table, at = [], 0
    for n in lens:
        table.append(ids[at:at + _pages_of(n, P)])
        at += _pages_of(n, P)
    return lens, table, pool, parents


def _wide(case, lens):
    """Width of the page table."""
    extra = case.get("room", 0)
    return max(1, _pages_of(max(lens) + extra, case["page"]) + 1)


# ------------------------------------------------------------------------------------------- inputs

def _random_codes(shape, gen):
    """E4M3 codes of normal values: a few large, most in the middle of the range, none NaN."""
    x = torch.empty(shape, dtype=torch.uint8, device=_DEV)
    flat = x.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=gen, device=_DEV) * 100).clamp(-_TOP, _TOP).to(_E4M3).view(torch.uint8)
    return x


def _random_scales(shape, gen):
    e = torch.randint(-9, -4, shape, generator=gen, device=_DEV, dtype=torch.int32)
    return ((e + 127) << 23).view(torch.float32)


def _tensor(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=_DEV)


def _table_tensor(rows, wide):
    return _tensor([r + [-1] * (wide - len(r)) for r in rows])


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    s = {"case": case, "op": case["op"]}
    if case["op"] in ("append", "attend"):
        new, kept = _lengths(case)
        ends = [a + b for a, b in zip(new, kept)]
        rng = random.Random(seed)
        n_pages = sum(_pages_of(n, P) for n in ends) + 3
        ids, rows = rng.sample(range(n_pages), n_pages - 3), []
        for n in ends:
            rows.append(ids[:_pages_of(n, P)])
            ids = ids[_pages_of(n, P):]
        layers, wide, lens = 1, max(len(r) for r in rows) + 1, kept
        s.update(cu=_tensor([0] + np.cumsum(new).tolist()), kept=_tensor(kept), ends=_tensor(ends), max_new=max(new),
                 max_end=max(ends))
        T = sum(new)
        if case["op"] == "append":
            # rows of the merged projection's output: K and V lie inside wider rows
            kv = torch.randn(T, 2 * H, D, generator=gen, device=_DEV)
            kv *= 0.25 + 4.0 * torch.rand(T, 2 * H, 1, generator=gen, device=_DEV)
            kv = kv.to(torch.bfloat16)
            s.update(k=kv[:, :H], v=kv[:, H:])
        else:
            s["q"] = torch.randn(T, case["q_heads"], D, generator=gen, device=_DEV).to(torch.bfloat16)
    else:
        lens, rows, n_pages, parents = _plan(case)
        layers, wide = case["layers"], _wide(case, lens)
        if parents is not None:
            s.update(parents=_tensor(parents), room=_tensor([case["room"] if p >= 0 else 0 for p in parents]))
    refs = [0] * n_pages
    for r in rows:
        for p in r:
            refs[p] += 1
    s.update(codes=_random_codes((layers, n_pages, 2, H, P, D), gen),
             scales=_random_scales((layers, n_pages, 2, H, P // _BLOCK), gen),
             table=_table_tensor(rows, wide), lens=_tensor(lens), refs=_tensor(refs))
    if own:
        import qwen3_prefill_delayed_gb300 as hra
        s["kv"] = hra.Kv8Cache(s["codes"], s["scales"], s["table"], s["lens"], s["refs"])
        if case["op"] in ("update", "compact"):
            s["next"] = s["kv"].empty_pages()
    return s


# ------------------------------------------------------------------------------------------- runs

def run(s):
    return _RUN[s["op"]](s)


def _append(s):
    if own:
        s["kv"].append(0, s["k"], s["v"], s["cu"], s["kept"], s["max_new"])
        return {"codes": s["codes"].view(_E4M3), "scales": s["scales"], "lens": s["lens"]}
    codes, scales, table, cu, kept = s["codes"][0], s["scales"][0], s["table"], s["cu"], s["kept"]
    P, T = codes.shape[3], s["k"].shape[0]
    t = torch.arange(T, device=_DEV)
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    pos = kept[seq] + t - cu[seq]
    page, slot = table[seq, pos // P].long(), pos % P
    block = page * (P // _BLOCK) + slot // _BLOCK                    # of the whole pool
    x = torch.stack([s["k"], s["v"]], 1).float()                     # [T, 2, H, D]
    top = x.abs().amax(3)                                            # [T, 2, H]
    n_blocks = codes.shape[0] * (P // _BLOCK)
    amax = torch.zeros(n_blocks, *top.shape[1:], device=_DEV)
    amax.scatter_reduce_(0, block[:, None, None].expand_as(top), top, "amax")
    fresh = _power(amax)
    # a block that already held tokens keeps a scale that they fit, and their codes follow it
    cont = (kept % _BLOCK != 0) & (cu[1:] > cu[:-1])
    page0 = table[torch.arange(kept.numel(), device=_DEV), kept // P].long().clamp_min(0)
    block0 = page0 * (P // _BLOCK) + kept % P // _BLOCK
    flat = scales.permute(0, 3, 1, 2).reshape(n_blocks, *top.shape[1:])   # [blocks, 2, H]
    before = flat[block0]
    after = torch.maximum(fresh[block0], before)
    after = torch.where(cont[:, None, None], after, fresh[block0])
    # untouched blocks keep their scale
    touched = torch.zeros(n_blocks, dtype=torch.bool, device=_DEV)
    touched[block] = True
    flat = torch.where(touched[:, None, None], fresh, flat)
    now = cont.nonzero().squeeze(1)
    flat[block0[now]] = after[now]
    scales.copy_(flat.view(codes.shape[0], P // _BLOCK, *top.shape[1:]).permute(0, 2, 3, 1))
    i = torch.arange(_BLOCK, device=_DEV)
    old_slot = (kept % P // _BLOCK * _BLOCK)[now, None] + i          # the whole block; new tokens overwrite theirs
    held = codes.view(_E4M3)[page0[now, None], :, :, old_slot].float()    # [n, 16, 2, H, D]
    again = _round8(held * (before[now] / after[now])[:, None, :, :, None])
    mine = i[None] < (kept % _BLOCK)[now, None]
    kept_codes = torch.where(mine[:, :, None, None, None], again.view(torch.uint8), held.to(_E4M3).view(torch.uint8))
    codes[page0[now, None], :, :, old_slot] = kept_codes
    codes[page, :, :, slot] = _round8(x * (1.0 / flat[block])[..., None]).view(torch.uint8)
    s["lens"].copy_(torch.where(cu[1:] > cu[:-1], kept + cu[1:] - cu[:-1], s["lens"]))
    return {"codes": s["codes"].view(_E4M3), "scales": s["scales"], "lens": s["lens"]}


def _power(a):
    """The smallest power of two s with a <= 448 s, at least 2^-126."""
    m, e = torch.frexp(a)
    e = (e - 9 + (m > 0.875)).clamp_min(-126).to(torch.int32)
    e = torch.where(a > 0, e, torch.full_like(e, -126))
    return ((e + 127) << 23).view(torch.float32)


def _round8(x):
    return x.clamp(-_TOP, _TOP).to(_E4M3)


def _attend(s):
    if own:
        return s["kv"].attend(0, s["q"], s["cu"], s["ends"], s["max_new"], s["max_end"])
    codes, scales, cu, ends, q = s["codes"][0].view(_E4M3), s["scales"][0], s["cu"].long(), s["ends"], s["q"]
    B, S, P, H, D = ends.numel(), s["max_end"], codes.shape[3], codes.shape[2], codes.shape[4]
    N, G, T = s["max_new"], q.shape[1] // H, q.shape[0]
    j = torch.arange(S, device=_DEV)
    page = s["table"][:, j // P].clamp_min(0).long()                      # [B, S]
    slot = (j % P).expand(B, S)
    unit = scales[page, :, :, slot // _BLOCK]                             # [B, S, 2, H]
    kv = codes[page, :, :, slot].float() * unit[..., None]                # [B, S, 2, H, D]
    there = j[None] < ends[:, None]
    kv = torch.where(there[:, :, None, None, None], kv, torch.zeros((), device=_DEV))
    k, v = kv[:, :, 0].permute(0, 2, 3, 1), kv[:, :, 1].transpose(1, 2)   # [B, H, D, S], [B, H, S, D]
    i = torch.arange(N, device=_DEV)
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp_max(T - 1)                            # [B, N]
    x = q[row].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    score = ((x @ k) * D ** -0.5).view(B, H, N, G, S)
    last = (ends - new)[:, None] + i                                      # the position of each new token
    seen = (j[None, None] <= last[..., None]) & there[:, None]            # [B, N, S]
    score = score.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, N * G, S) @ v).view(B, H, N, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    t = torch.arange(T, device=_DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)[seq, t - cu[seq]].to(torch.bfloat16)


def _update(s):
    if own:
        t, n, r = s["kv"].update(s["parents"], s["room"], out=s["next"])
        return {"codes": s["codes"].view(_E4M3), "scales": s["scales"], "table": t, "lens": n, "refs": r}
    codes, scales, table, parents = s["codes"], s["scales"], s["table"], s["parents"].long()
    P, rows, wide = codes.shape[4], table.shape[0], table.shape[1]
    src = parents.clamp_min(0)
    alive = parents >= 0
    lens = torch.where(alive, s["lens"][src], torch.zeros_like(s["lens"]))
    b = torch.arange(rows, device=_DEV)
    first = torch.full((rows,), rows, device=_DEV).scatter_reduce_(0, src[alive], b[alive], "amin")
    heir = alive & (first[src] == b)                      # the lowest child keeps the part-filled page
    i = torch.arange(wide, device=_DEV)
    old = torch.where(alive[:, None], table[src], torch.full_like(table, -1))
    full = i[None] < (lens // P)[:, None]                 # pages that nobody writes again
    keep = (old >= 0) & (full | heir[:, None])
    want = i[None] < -(-(lens + torch.where(alive, s["room"], 0)) // P)[:, None]
    fresh = want & ~keep
    refs = torch.zeros_like(s["refs"])
    refs.index_add_(0, old[keep].long(), torch.ones_like(old[keep]))
    free = (refs == 0).nonzero().squeeze(1)
    rank = (fresh.view(-1).cumsum(0) - 1).view(rows, wide)
    new = torch.where(keep, old, torch.full_like(old, -1))
    new = torch.where(fresh, free[rank.clamp_min(0)].to(torch.int32), new)
    refs.index_add_(0, new[fresh].long(), torch.ones_like(new[fresh]))
    copied = fresh & (old >= 0) & (i[None] * P < lens[:, None])
    a, z = old[copied].long(), new[copied].long()
    codes[:, z] = codes[:, a]
    scales[:, z] = scales[:, a]
    return {"codes": codes.view(_E4M3), "scales": scales, "table": new, "lens": lens, "refs": refs}


def _compact(s):
    if own:
        t, n, r = s["kv"].compact(out=s["next"])
        return {"codes": s["codes"].view(_E4M3), "scales": s["scales"], "table": t, "lens": n, "refs": r}
    codes, scales, refs, table = s["codes"], s["scales"], s["refs"], s["table"]
    used = refs > 0
    count = used.sum()
    ids = torch.arange(refs.numel(), device=_DEV)
    a = (used & (ids >= count)).nonzero().squeeze(1)      # moved ...
    z = (~used & (ids < count)).nonzero().squeeze(1)      # ... to the holes, in order
    to = ids.clone()
    to[a] = z
    new_refs = torch.zeros_like(refs)
    new_refs[to[used]] = refs[used]
    codes[:, z] = codes[:, a]
    scales[:, z] = scales[:, a]
    new = torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table)
    return {"codes": codes.view(_E4M3), "scales": scales, "table": new, "lens": s["lens"].clone(), "refs": new_refs}


_RUN = {"append": _append, "attend": _attend, "update": _update, "compact": _compact}


# ------------------------------------------------------------------------------------------- work

def work(case):
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] in ("append", "attend"):
        new, kept = _lengths(case)
        table = 4 * sum(_pages_of(a + b, P) for a, b in zip(new, kept)) + 12 * case["batch"]
    if case["op"] == "append":
        T = sum(new)
        blocks = sum(_pages_of(a + b, _BLOCK) - b // _BLOCK for a, b in zip(new, kept))
        # bf16 rows read, codes and scales written; a block that goes on: its scale read
        cont = sum(1 for a, b in zip(new, kept) if b % _BLOCK)
        return {"bytes": T * 2 * H * D * 3 + (blocks + cont) * 2 * H * 4 + table, "flops": T * 2 * H * D * 2}
    if case["op"] == "attend":
        tokens, T = sum(a + b for a, b in zip(new, kept)), sum(new)
        blocks = sum(_pages_of(a + b, _BLOCK) for a, b in zip(new, kept))
        seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, kept))
        return {"bytes": tokens * 2 * H * D + blocks * 2 * H * 4 + 2 * T * case["q_heads"] * D * 2 + table,
                "flops": 4 * seen * case["q_heads"] * D}
    lens, rows, pool, parents = _plan(case)
    page = 2 * H * (P * D + P // _BLOCK * 4)
    if case["op"] == "update":
        seen, copies = set(), 0
        for p in parents:
            if p >= 0:
                copies += p in seen and lens[p] % P != 0
                seen.add(p)
    else:
        used = sorted(x for r in rows for x in r)
        copies = sum(x >= len(used) for x in used)
    meta = 8 * (sum(map(len, rows)) + case["rows"] + pool)
    return {"bytes": 2 * copies * case["layers"] * page + meta, "flops": pool + sum(map(len, rows))}


# ------------------------------------------------------------------------------------------- 64 bits

def _grid(x):
    """The nearest E4M3 values of x (float64), ties to the even mantissa."""
    a = x.abs().clamp_max(_TOP)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -12))).clamp_min(-6.0)
    e = torch.where(a >= torch.exp2(e + 1), e + 1, torch.where(a < torch.exp2(e), (e - 1).clamp_min(-6.0), e))
    step = torch.exp2(e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp_max(_TOP), x)


def _values(codes):
    """E4M3 values of uint8 codes from the format's definition, float64."""
    c = torch.arange(256, dtype=torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    v[(c & 127) == 127] = float("nan")
    v = torch.where(c >= 128, -v, v)
    return v.to(codes.device)[codes.long()]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(s, case)
    if op == "attend":
        return _exact_attend(s, case)
    return _exact_pages(s, case)


def _exact_append(s, case):
    new, kept = _lengths(case)
    P, H = case["page"], case["kv_heads"]
    value, scale = _values(s["codes"][0]), s["scales"][0].double()
    x = torch.stack([s["k"], s["v"]], 1).double()
    table, at = s["table"].tolist(), 0
    for b, (n, first) in enumerate(zip(new, kept)):
        last = first + n
        pages = torch.tensor(table[b][:_pages_of(last, P)], device=_DEV)
        # this row's slots in order, in whole blocks: [blocks, 16, 2, H, D]
        row = value[pages].permute(0, 3, 1, 2, 4).reshape(-1, _BLOCK, 2, H, x.shape[3])
        unit = scale[pages].permute(0, 3, 1, 2).reshape(-1, 2, H)
        lo, hi = first // _BLOCK, _pages_of(last, _BLOCK)
        fill = torch.zeros((hi - lo) * _BLOCK, *x.shape[1:], dtype=torch.float64, device=_DEV)
        off = first - lo * _BLOCK
        fill[off:off + n] = x[at:at + n]
        fill = fill.view(hi - lo, _BLOCK, *x.shape[1:])
        top = fill.abs().amax(dim=(1, 4))
        e = torch.ceil(torch.log2((top / _TOP).clamp_min(2.0 ** -140)))
        e = torch.where(top > _TOP * torch.exp2(e), e + 1, torch.where(top <= _TOP * torch.exp2(e - 1), e - 1, e))
        u = torch.exp2(e.clamp_min(-126.0))
        if off:
            u[0] = torch.maximum(u[0], unit[lo])
            row[lo, :off] = _grid(row[lo, :off] * (unit[lo] / u[0])[None, :, :, None])
        unit[lo:hi] = u
        code = _grid(fill / u[:, None, :, :, None])
        is_new = torch.zeros((hi - lo) * _BLOCK, dtype=torch.bool, device=_DEV)
        is_new[off:off + n] = True
        row[lo:hi] = torch.where(is_new.view(hi - lo, _BLOCK, 1, 1, 1), code, row[lo:hi])
        value[pages] = row.view(len(pages), P, 2, H, -1).permute(0, 2, 3, 1, 4)
        scale[pages] = unit.view(len(pages), P // _BLOCK, 2, H).permute(0, 2, 3, 1)
        at += n
    return {"codes": value[None], "scales": scale[None], "lens": None}


def _exact_attend(s, case):
    new, kept = _lengths(case)
    P, H, D, G = case["page"], case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    if 4 * sum(a * (a + b) for a, b in zip(new, kept)) * case["q_heads"] * D > 4e12:
        return None
    table, out, at = s["table"].tolist(), [], 0
    for b, (n, before) in enumerate(zip(new, kept)):
        last = before + n
        pages = torch.tensor(table[b][:_pages_of(last, P)], device=_DEV)
        unit = s["scales"][0][pages].double().repeat_interleave(_BLOCK, dim=3)
        kv = (_values(s["codes"][0][pages]) * unit[..., None]).permute(1, 2, 0, 3, 4).reshape(2, H, -1, D)[:, :, :last]
        q = s["q"][at:at + n].double().view(n, H, G, D)
        z = torch.einsum("nhgd,hsd->hgns", q, kv[0]) / np.sqrt(D)
        late = torch.arange(last, device=_DEV)[None] > torch.arange(before, last, device=_DEV)[:, None]
        w = torch.softmax(z.masked_fill(late, float("-inf")), -1)
        out.append(torch.einsum("hgns,hsd->nhgd", w, kv[1]).reshape(n, H * G, D))
        at += n
    return torch.cat(out)


def _exact_pages(s, case):
    lens, rows, pool, parents = _plan(case)
    P, moves = case["page"], []
    if case["op"] == "compact":
        used = sorted(p for r in rows for p in r)
        holes = [p for p in range(len(used)) if p not in set(used)]
        moves = list(zip([p for p in used if p >= len(used)], holes))
    else:
        heirs, kept, want = set(), set(), []
        for p in parents:
            if p < 0:
                continue
            n = lens[p]
            share = n // P
            kept.update(rows[p][:share] if p in heirs else rows[p])
            here = share if p in heirs else len(rows[p])
            want += [(rows[p][k] if k < len(rows[p]) else None) for k in range(here, max(here, _pages_of(n + case["room"], P)))]
            heirs.add(p)
        free = [p for p in range(pool) if p not in kept]
        moves = [(a, z) for a, z in zip(want, free) if a is not None]
    codes, scales = s["codes"].clone(), s["scales"].clone()
    for a, z in moves:
        codes[:, z] = s["codes"][:, a]
        scales[:, z] = s["scales"][:, a]
    return {"codes": codes.view(_E4M3), "scales": scales, "table": None, "lens": None, "refs": None}
