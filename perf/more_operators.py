"""Measured cases of the paged 8-bit key/value cache where streams are long and prompts are shared.

Operators:
  window   causal grouped-query attention of new tokens that see the last `window` positions up to their own and the
           first `sinks` positions: single tokens of an audio frame, whole prompts, and prompt chunks;
  shared   attention of a batch whose groups of rows share the pages of a long prefix, which is read once for the group:
           single tokens of an audio frame, and steps of a few tokens;
  update   the page tables of the next step where a window bounds what is seen: the pages that no later token sees
           go back to the pool, rows are forked, freed and extended, shared part-filled pages copied in every layer.

``run`` computes them in elementary torch operations in fp32, or, where ``own`` is true, with the library's calls.
Lengths, parents and page numbers come from the case alone (its "ragged" number), so that ``work`` is exact; values
come from the seed.
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
        # one frame of one stream on the small model: latency alone
        {"name": "window frame short", "op": "window", "batch": 1, "new_lo": 1, "new_hi": 1, "kept_lo": 203, "kept_hi": 203,
         "window": 96, "sinks": 4, "released": 0, "ragged": 1, **tiny},
        # one frame of a full server whose streams run for minutes: the pages outside the window are back in the pool
        {"name": "window frame wide", "op": "window", "batch": 64, "new_lo": 1, "new_hi": 1, "kept_lo": 15, "kept_hi": 32767,
         "window": 2048, "sinks": 4, "released": 1, "ragged": 2, **full},
        # 8 long ragged prompts through a window of a quarter of their length
        {"name": "window prompts", "op": "window", "batch": 8, "new_lo": 1024, "new_hi": 2048, "kept_lo": 0, "kept_hi": 0,
         "window": 512, "sinks": 16, "released": 0, "ragged": 3, **full},
        # later chunks of very long prompts, 2 rows, odd sizes
        {"name": "window chunked", "op": "window", "batch": 2, "new_lo": 500, "new_hi": 1021, "kept_lo": 9001, "kept_hi": 16001,
         "window": 4001, "sinks": 7, "released": 0, "ragged": 4, **full},
        # four continuations of one short prompt on the small model: latency alone
        {"name": "shared frame short", "op": "shared", "groups": 1, "rows_lo": 4, "rows_hi": 4, "new_lo": 1, "new_hi": 1,
         "prefix_lo": 203, "prefix_hi": 203, "own_lo": 1, "own_hi": 40, "ragged": 5, **tiny},
        # 8 voices, four to eight streams each: a frame after their voice prompts
        {"name": "shared frame voices", "op": "shared", "groups": 8, "rows_lo": 4, "rows_hi": 8, "new_lo": 1, "new_hi": 1,
         "prefix_lo": 1024, "prefix_hi": 2112, "own_lo": 1, "own_hi": 700, "ragged": 6, **full},
        # a full server of one long prompt: 64 continuations
        {"name": "shared frame wide", "op": "shared", "groups": 1, "rows_lo": 64, "rows_hi": 64, "new_lo": 1, "new_hi": 1,
         "prefix_lo": 16001, "prefix_hi": 16001, "own_lo": 15, "own_hi": 1000, "ragged": 7, **full},
        # 32 rows take a few tokens each after one instruction prompt, some none
        {"name": "shared steps", "op": "shared", "groups": 1, "rows_lo": 32, "rows_hi": 32, "new_lo": 0, "new_hi": 12,
         "prefix_lo": 4099, "prefix_hi": 4099, "own_lo": 0, "own_hi": 200, "ragged": 8, **full},
        # one step of a server with a window: most rows take a token, a few pages fall out of their windows
        {"name": "update step", "op": "update", "layers": 36, "rows": 64, "held": 60, "len_lo": 1, "len_hi": 4096, "window": 512,
         "sinks": 4, "released": 1, "fork": 1, "ended": 6, "room": 1, "spare": 80, "ragged": 9, "kv_heads": 8, "head_dim": 128,
         "page": 64},
        # 8 long prompts after their prefill: what the window has left behind goes, and each gets three more continuations
        {"name": "update fork", "op": "update", "layers": 36, "rows": 32, "held": 8, "len_lo": 1024, "len_hi": 8192,
         "window": 1024, "sinks": 64, "released": 0, "fork": 4, "ended": 0, "room": 64, "spare": 80, "ragged": 10, "kv_heads": 8,
         "head_dim": 128, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["window frame", "window frame", "window prompt", "window prompt", "shared frame", "shared frame",
                     "shared steps", "update"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op.split()[0], "ragged": rng.randrange(1 << 20), "kv_heads": kv, "head_dim": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 64, 128])}
    if case["op"] != "update":
        case["q_heads"] = kv * rng.choice([1, 2, 4, 8] if kv < 8 else [1, 2, 4])
    if case["op"] in ("window", "update"):
        case.update(window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, _log_int(rng, 1, 300)]),
                    released=rng.choice([0, 1]))
    if op == "window frame":
        kept = _log_int(rng, 1, 32767)
        case.update(batch=_log_int(rng, 1, 64), new_lo=rng.choice([0, 1]), new_hi=rng.choice([1, 1, 1, 2, 4]),
                    kept_lo=rng.randint(0, kept), kept_hi=kept)
        case["window"] = min(case["window"], 2048)
    elif op == "window prompt":
        hi = _log_int(rng, 5, 2048)
        kept = rng.choice([0, _log_int(rng, 1, 16000)])
        # no more pairs of a token and a position than the largest listed case
        sees = min(hi + kept, case["window"] + case["sinks"])
        hi = min(hi, 6000000 // sees)
        batch = max(1, min(_log_int(rng, 1, 64), 6000000 // (hi * sees)))
        case.update(batch=batch, new_lo=rng.randint(0, hi), new_hi=hi, kept_lo=rng.randint(0, kept), kept_hi=kept)
    elif op == "shared frame":
        rows = _log_int(rng, 1, 64)
        prefix, mine = _log_int(rng, 1, 16001), _log_int(rng, 1, 1000)
        groups = _log_int(rng, 1, max(1, min(64 // rows, 16)))
        prefix = min(prefix, 32002 // groups)
        case.update(groups=groups, rows_lo=rng.randint(1, rows), rows_hi=rows, new_lo=rng.choice([0, 1]), new_hi=1,
                    prefix_lo=rng.randint(prefix // 2, prefix), prefix_hi=prefix, own_lo=rng.randint(0, mine), own_hi=mine)
    elif op == "shared steps":
        rows, hi = _log_int(rng, 1, 32), _log_int(rng, 2, 100)
        prefix, mine = _log_int(rng, 1, 4099), _log_int(rng, 1, 500)
        groups = _log_int(rng, 1, max(1, min(32 // rows, 8)))
        hi = min(hi, max(2, 6000000 // (groups * rows * (prefix + mine))))
        case.update(groups=groups, rows_lo=rng.randint(1, rows), rows_hi=rows, new_lo=rng.randint(0, hi), new_hi=hi,
                    prefix_lo=rng.randint(prefix // 2, prefix), prefix_hi=prefix, own_lo=rng.randint(0, mine), own_hi=mine)
    elif op == "update":
        rows = _log_int(rng, 2, 64)
        hi = _log_int(rng, 1, 4096 if rows <= 32 else 2048)
        held = rng.randint(1, rows)
        case.update(layers=_log_int(rng, 1, 36), rows=rows, held=held, len_lo=rng.randint(0, hi), len_hi=hi,
                    fork=rng.choice([1, 1, 2, 3, 4]), ended=rng.randint(0, held // 2), room=rng.choice([0, 1, 16, 65]),
                    spare=rows * 5 + 8)
        # no more bytes than the largest listed pools
        page_bytes = 2 * kv * case["page"] * case["head_dim"]
        pages = held * _pages_of(hi, case["page"]) + case["spare"]
        case["layers"] = max(1, min(case["layers"], (36 * 640 * 131072) // (page_bytes * pages)))
    return case


def _pages_of(n, page):
    return -(-n // page)


def _shared_pages(case, prefix):
    """Pages of a prefix that its group shares: the whole ones."""
    return prefix // case["page"]


def _lengths(case):
    """(new tokens, kept tokens) of every row; of shared prefixes also the rows of each group and the prefixes."""
    rng = random.Random(case["ragged"])
    if case["op"] == "window":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
        kept = [rng.randint(case["kept_lo"], case["kept_hi"]) for _ in range(case["batch"])]
        new[rng.randrange(case["batch"])] = case["new_hi"]   # a call has a token
        return new, kept
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["groups"])]
    prefix = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in rows]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(sum(rows))]
    new[rng.randrange(len(new))] = case["new_hi"]
    kept = [p + rng.randint(case["own_lo"], case["own_hi"]) for r, p in zip(rows, prefix) for _ in range(r)]
    return new, kept, rows, prefix


def _gone(case, length):
    """Pages [lo, hi) of a row of `length` positions that no token behind them sees."""
    lo = _pages_of(case["sinks"], case["page"])
    return lo, max(lo, (length - case["window"] + 1) // case["page"])


def _plan(case):
    """The rows before an update: lengths, page numbers of each row (-1: released before), pool size, parents."""
    rng = random.Random(case["ragged"])
    P, rows = case["page"], case["rows"]
    lens = [rng.randint(case["len_lo"], case["len_hi"]) if b < case["held"] else 0 for b in range(rows)]
    holes = []
    for n in lens:   # released when the row was a page or two shorter
        lo, hi = _gone(case, max(0, n - rng.randint(0, 2 * P))) if case["released"] else (0, 0)
        holes.append(range(lo, min(hi, _pages_of(n, P))))
    used = sum(_pages_of(n, P) - len(h) for n, h in zip(lens, holes))
    pool = used + case["spare"]
    if case["fork"] > 1:   # the held rows' continuations side by side
        parents = [b // case["fork"] if b // case["fork"] < case["held"] else -1 for b in range(rows)]
    else:                  # rows stay; the free ones start as copies of a row, some end
        parents = [b if b < case["held"] else rng.randrange(case["held"]) for b in range(rows)]
    for b in rng.sample(range(case["held"]), case["ended"]):
        parents[b] = -1
    ids = iter(rng.sample(range(pool), used))
    table = [[-1 if i in h else next(ids) for i in range(_pages_of(n, P))] for n, h in zip(lens, holes)]
    return lens, table, pool, parents


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
    H, D, P, op = case["kv_heads"], case["head_dim"], case["page"], case["op"]
    s = {"case": case, "op": op}
    if op == "update":
        lens, rows, n_pages, parents = _plan(case)
        layers, wide = case["layers"], _pages_of(max(lens) + case["room"], P) + 1
        s.update(parents=_tensor(parents), room=_tensor([case["room"] if p >= 0 else 0 for p in parents]))
    else:
        lengths = _lengths(case)
        new, lens = lengths[:2]
        ends = [a + b for a, b in zip(new, lens)]
        rng = random.Random(seed)
        if op == "window":   # where pages are released, those that the new tokens do not see
            lists = []
            for n, before, end in zip(new, lens, ends):
                lo, hi = _gone(case, before) if case["released"] else (0, 0)
                lists.append([i >= lo and i < hi for i in range(_pages_of(end, P))])
            count = sum(x.count(False) for x in lists)
            n_pages = count + 3
            ids = iter(rng.sample(range(n_pages), count))
            rows = [[-1 if gone else next(ids) for gone in x] for x in lists]
        else:
            per_group, prefix = lengths[2:]
            group_cu = [0] + np.cumsum(per_group).tolist()
            full = [_shared_pages(case, p) for p in prefix]
            of = [g for g, r in enumerate(per_group) for _ in range(r)]
            count = sum(full) + sum(_pages_of(e, P) - full[g] for e, g in zip(ends, of))
            n_pages = count + 3
            ids = iter(rng.sample(range(n_pages), count))
            common = [[next(ids) for _ in range(f)] for f in full]
            rows = [common[g] + [next(ids) for _ in range(_pages_of(e, P) - full[g])] for e, g in zip(ends, of)]
            s.update(group_cu=_tensor(group_cu), prefix=_tensor(prefix), max_prefix=max(prefix),
                     max_own=max(e - prefix[g] for e, g in zip(ends, of)))
        layers, wide, T = 1, max(len(r) for r in rows) + 1, sum(new)
        s.update(cu=_tensor([0] + np.cumsum(new).tolist()), ends=_tensor(ends), max_new=max(new), max_end=max(ends),
                 q=torch.randn(T, case["q_heads"], D, generator=gen, device=_DEV).to(torch.bfloat16))
    refs = [0] * n_pages
    for r in rows:
        for p in r:
            if p >= 0:
                refs[p] += 1
    s.update(codes=_random_codes((layers, n_pages, 2, H, P, D), gen),
             scales=_random_scales((layers, n_pages, 2, H, P // _BLOCK), gen),
             table=_table_tensor(rows, wide), lens=_tensor(lens), refs=_tensor(refs))
    if own:
        import qwen3_prefill_delayed_gb300 as hra
        s["kv"] = hra.Kv8Cache(s["codes"], s["scales"], s["table"], s["lens"], s["refs"])
        if op == "shared":
            s["reach"] = hra.Kv8Reach(groups=s["group_cu"], prefix=s["prefix"], max_prefix=s["max_prefix"], max_own=s["max_own"])
        else:
            s["reach"] = hra.Kv8Reach(window=case["window"], sinks=case["sinks"])
        if op == "update":
            s["next"] = s["kv"].empty_pages()
    return s


# ------------------------------------------------------------------------------------------- runs

def run(s):
    return _RUN[s["op"]](s)


def _gather(s, table, pos, there):
    """K and V (fp32) of positions pos [B, S] of the rows of table, zeros where not `there`: [B, H, D, S], [B, H, S, D]."""
    codes, scales = s["codes"][0].view(_E4M3), s["scales"][0]
    P = codes.shape[3]
    at = pos.clamp(0, table.shape[1] * P - 1)
    page = torch.gather(table, 1, at // P).clamp_min(0).long()
    slot = at % P
    unit = scales[page, :, :, slot // _BLOCK]                             # [B, S, 2, H]
    kv = codes[page, :, :, slot].float() * unit[..., None]                # [B, S, 2, H, D]
    kv = torch.where(there[:, :, None, None, None], kv, torch.zeros((), device=_DEV))
    return kv[:, :, 0].permute(0, 2, 3, 1), kv[:, :, 1].transpose(1, 2)


def _softmax(score):
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _padded(q, cu, N, H):
    """The tokens of every row as [B, H, N * G, D] in fp32, and their packed rows [B, N]."""
    T, nq, D = q.shape
    row = (cu[:-1, None] + torch.arange(N, device=_DEV)).clamp_max(T - 1)
    x = q[row].float().view(-1, N, H, nq // H, D)
    return x.permute(0, 2, 1, 3, 4).reshape(-1, H, N * (nq // H), D)


def _packed(out, cu, T):
    """[B, H, N, G, D] -> bf16 [T, H * G, D]."""
    B, H, N, G, D = out.shape
    t = torch.arange(T, device=_DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)[seq, t - cu[seq]].to(torch.bfloat16)


def _window(s):
    if own:
        return s["kv"].attend(0, s["q"], s["cu"], s["ends"], s["max_new"], s["max_end"], reach=s["reach"])
    case, cu, ends, q, N = s["case"], s["cu"].long(), s["ends"].long(), s["q"], s["max_new"]
    H, D, W = case["kv_heads"], case["head_dim"], case["window"]
    S = min(case["sinks"], s["max_end"])
    B, G, T = ends.numel(), q.shape[1] // H, q.shape[0]
    first = ends - (cu[1:] - cu[:-1])                                     # the first new token's position
    behind = min(W - 1, s["max_end"])
    near = (first - behind)[:, None] + torch.arange(behind + N, device=_DEV)
    pos = torch.cat([torch.arange(S, device=_DEV).expand(B, S), near], 1)
    there = (pos >= 0) & (pos < ends[:, None])
    there[:, S:] &= near >= S
    k, v = _gather(s, s["table"], pos, there)
    x = _padded(q, cu, N, H)
    score = ((x @ k) * D ** -0.5).view(B, H, N, G, -1)
    at = (first[:, None] + torch.arange(N, device=_DEV))[..., None]       # [B, N, 1]
    seen = there[:, None] & (pos[:, None] <= at) & ((pos[:, None] > at - W) | (pos[:, None] < S))
    score = score.masked_fill(~seen[:, None, :, None], float("-inf"))
    p = _softmax(score)
    return _packed((p.view(B, H, N * G, -1) @ v).view(B, H, N, G, D), cu, T)


def _shared(s):
    if own:
        return s["kv"].attend(0, s["q"], s["cu"], s["ends"], s["max_new"], s["max_end"], reach=s["reach"])
    case, cu, ends, q, N = s["case"], s["cu"].long(), s["ends"].long(), s["q"], s["max_new"]
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    G, T = q.shape[1] // H, q.shape[0]
    x = _padded(q, cu, N, H)
    new, kept, per_group, prefix = _lengths(case)                         # what the caller of the step knows
    first = ends - (cu[1:] - cu[:-1])
    out, lo = [], 0
    for rows, length in zip(per_group, prefix):
        hi, shared = lo + rows, length // P * P
        table, end = s["table"][lo:hi], ends[lo:hi]
        most = max(a + b for a, b in zip(new[lo:hi], kept[lo:hi])) - shared
        j = torch.arange(shared, device=_DEV)[None]
        k, v = _gather(s, table[:1], j, torch.ones_like(j, dtype=torch.bool))      # once for the group
        pos = (shared + torch.arange(most, device=_DEV)).expand(rows, most)
        there = pos < end[:, None]
        k1, v1 = _gather(s, table, pos, there)
        y = x[lo:hi]
        score = torch.cat([y @ k, y @ k1], -1) * D ** -0.5
        at = (first[lo:hi, None] + torch.arange(N, device=_DEV))[..., None]
        seen = there[:, None] & (pos[:, None] <= at)                      # [rows, N, most]
        score = score.view(rows, H, N, G, shared + most)
        score[..., shared:].masked_fill_(~seen[:, None, :, None], float("-inf"))
        p = _softmax(score).view(rows, H, N * G, shared + most)
        out.append((p[..., :shared] @ v + p[..., shared:] @ v1).view(rows, H, N, G, D))
        lo = hi
    return _packed(torch.cat(out), cu, T)


def _update(s):
    if own:
        t, n, r = s["kv"].update(s["parents"], s["room"], out=s["next"], reach=s["reach"])
        return {"codes": s["codes"].view(_E4M3), "scales": s["scales"], "table": t, "lens": n, "refs": r}
    case, codes, scales, table, parents = s["case"], s["codes"], s["scales"], s["table"], s["parents"].long()
    P, rows, wide = codes.shape[4], table.shape[0], table.shape[1]
    src = parents.clamp_min(0)
    alive = parents >= 0
    lens = torch.where(alive, s["lens"][src], torch.zeros_like(s["lens"]))
    b = torch.arange(rows, device=_DEV)
    first = torch.full((rows,), rows, device=_DEV).scatter_reduce_(0, src[alive], b[alive], "amin")
    heir = alive & (first[src] == b)                      # the lowest child keeps the part-filled page
    i = torch.arange(wide, device=_DEV)
    gone = (i[None] * P >= case["sinks"]) & ((i[None] + 1) * P <= (lens - case["window"] + 1)[:, None])
    old = torch.where(alive[:, None] & ~gone, table[src], torch.full_like(table, -1))
    full = i[None] < (lens // P)[:, None]                 # pages that nobody writes again
    keep = (old >= 0) & (full | heir[:, None])
    want = ~gone & (i[None] < -(-(lens + torch.where(alive, s["room"], 0)) // P)[:, None])
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


_RUN = {"window": _window, "shared": _shared, "update": _update}


# ------------------------------------------------------------------------------------------- work

def _seen(case, p):
    """Positions that a token at position p sees through the window."""
    return min(p + 1, case["window"]) + min(case["sinks"], max(0, p + 1 - case["window"]))


def work(case):
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "update":
        lens, rows, pool, parents = _plan(case)
        page = 2 * H * (P * D + P // _BLOCK * 4)
        seen, copies = set(), 0
        for p in parents:
            if p >= 0:
                n = lens[p]
                lo, hi = _gone(case, n)
                copies += p in seen and n % P != 0 and not lo <= n // P < hi
                seen.add(p)
        meta = 8 * (sum(map(len, rows)) + case["rows"] + pool)
        return {"bytes": 2 * copies * case["layers"] * page + meta, "flops": pool + sum(map(len, rows))}
    lengths = _lengths(case)
    new, kept = lengths[:2]
    T = sum(new)
    spans, pairs = [], 0     # [lo, hi) of positions that have to be read
    if case["op"] == "window":
        for n, k in zip(new, kept):
            if n:
                near = max(0, k - case["window"] + 1)
                spans += [(near, k + n), (0, min(case["sinks"], near))]
                pairs += sum(_seen(case, p) for p in range(k, k + n))
    else:
        at = 0
        for r, p in zip(*lengths[2:]):
            start = p // P * P
            if any(new[at:at + r]):
                spans.append((0, start))
            spans += [(start, k + n) for n, k in zip(new[at:at + r], kept[at:at + r]) if n]
            at += r
        pairs = sum(n * k + n * (n + 1) // 2 for n, k in zip(new, kept))
    tokens = sum(hi - lo for lo, hi in spans)
    blocks = sum(_pages_of(hi, _BLOCK) - lo // _BLOCK for lo, hi in spans if hi > lo)
    entries = sum(_pages_of(hi, P) - lo // P for lo, hi in spans if hi > lo)
    return {"bytes": tokens * 2 * H * D + blocks * 2 * H * 4 + 2 * T * case["q_heads"] * D * 2 + 4 * entries + 12 * len(new),
            "flops": 4 * pairs * case["q_heads"] * D}


# ------------------------------------------------------------------------------------------- 64 bits

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
    if case["op"] == "update":
        return _exact_update(s, case)
    return _exact_attend(s, case)


def _exact_attend(s, case):
    lengths = _lengths(case)
    new, kept = lengths[:2]
    P, H, D, G = case["page"], case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    W, S = case.get("window", 1 << 40), case.get("sinks", 0)
    spans = [a * min(a + b, a + W + S) for a, b in zip(new, kept)]
    if 4 * sum(spans) * case["q_heads"] * D > 4e12:
        return None
    table, out, at = s["table"].tolist(), [], 0
    for b, (n, before) in enumerate(zip(new, kept)):
        if n == 0:
            continue
        last = before + n
        near = max(0, before - W + 1)
        pos = list(range(min(S, near))) + list(range(near, last))     # what one of its tokens sees, in order
        j = torch.tensor(pos, device=_DEV)
        page = torch.tensor([table[b][i // P] for i in pos], device=_DEV)
        unit = s["scales"][0][page, :, :, j % P // _BLOCK].double()
        kv = (_values(s["codes"][0][page, :, :, j % P]) * unit[..., None]).permute(1, 2, 0, 3)   # [2, H, S, D]
        q = s["q"][at:at + n].double().view(n, H, G, D)
        z = torch.einsum("nhgd,hsd->hgns", q, kv[0]) / np.sqrt(D)
        i = torch.arange(before, last, device=_DEV)[:, None]
        hidden = (j[None] > i) | ((j[None] <= i - W) & (j[None] >= S))
        w = torch.softmax(z.masked_fill(hidden, float("-inf")), -1)
        out.append(torch.einsum("hgns,hsd->nhgd", w, kv[1]).reshape(n, H * G, D))
        at += n
    return torch.cat(out)


def _exact_update(s, case):
    lens, rows, pool, parents = _plan(case)
    P, heirs, kept, want = case["page"], set(), set(), []
    for p in parents:
        if p < 0:
            continue
        n = lens[p]
        lo, hi = _gone(case, n)
        mine = [-1 if lo <= i < hi else x for i, x in enumerate(rows[p])]
        for i in range(max(len(mine), _pages_of(n + case["room"], P))):
            have = mine[i] if i < len(mine) else -1
            if have >= 0 and (i < n // P or p not in heirs):
                kept.add(have)
            elif not lo <= i < hi and i * P < n + case["room"]:
                want.append(have if i * P < n else -1)
        heirs.add(p)
    free = [p for p in range(pool) if p not in kept]
    codes, scales = s["codes"].clone(), s["scales"].clone()
    for a, z in zip(want, free):
        if a >= 0:
            codes[:, z] = s["codes"][:, a]
            scales[:, z] = s["scales"][:, a]
    return {"codes": codes.view(_E4M3), "scales": scales, "table": None, "lens": None, "refs": None}
