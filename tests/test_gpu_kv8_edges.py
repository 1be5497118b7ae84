"""The paged 8-bit cache on the GPU at the edges of its contract, beyond tests/test_gpu_kv8.py: lengths after appends that are
cut short, rows without pages, not-a-numbers behind the causal mask, scales of zero, other streams."""
import pytest
import torch

import kv8_ref as R
from test_gpu_kv8 import BF16, build, check, cu_of, gpu, hra, i32, same  # noqa: F401  (hra: the fixture)

pytestmark = pytest.mark.gpu


def give_pages(c, width):
    """Every row of the CPU cache a page for each of its first `width` table entries."""
    free = [p for p in range(c["refs"].numel()) if not c["refs"][p]]
    for b in range(c["table"].shape[0]):
        for i in range(width):
            if c["table"][b, i] < 0:
                c["table"][b, i] = free.pop()
                c["refs"][c["table"][b, i]] = 1


# ----------------------------------------------------------------------------- what an append leaves as the length

@pytest.mark.parametrize("new,start,max_new", [([20, 3, 7], [5, 30, 16], 6), ([1, 40], [15, 0], 17), ([2, 2], [31, 7], 1)])
def test_tokens_beyond_max_new_are_not_counted(hra, new, start, max_new):  # noqa: F811
    H, D, P = 2, 64, 16
    c = build(start, H=H, D=D, P=P, width=4, spare=12, seed=1)
    give_pages(c, 4)
    T, cu = sum(new), cu_of(new)
    x = torch.randn(T, 2 * H, D, generator=torch.Generator().manual_seed(2)).to(BF16)
    kv, xg = gpu(hra, c), x.cuda()
    kv.append(0, xg[:, :H], xg[:, H:], i32(cu).cuda(), i32(start).cuda(), max_new)
    short = [min(n, max_new) for n in new]
    y = torch.cat([x[cu[b]:cu[b] + n] for b, n in enumerate(short)])
    R.append(c, 0, y[:, :H], y[:, H:], cu_of(short), start)
    assert c["lens"].tolist() == [s + n for s, n in zip(start, short)]
    same(kv, c)
    assert kv.device_error() == hra.DEVERR_POS_RANGE


@pytest.mark.parametrize("held,start,n,want", [(0, -3, 4, 0), (7, -3, 4, 1), (7, -3, 2, 0), (20, 32, 5, 20), (32, 40, 1, 32),
                                               (5, -2147483648, 3, 0), (9, 2147483647, 3, 9)])
def test_a_row_that_gets_nothing_holds_no_more_than_before(hra, held, start, n, want):  # noqa: F811
    c = build([held, 3], H=1, D=64, P=16, width=2, spare=4, seed=4)
    give_pages(c, 2)
    kv = gpu(hra, c)
    x = torch.randn(n + 2, 1, 64, generator=torch.Generator().manual_seed(5)).to(BF16)
    kv.append(0, x.cuda(), x.cuda(), i32([0, n, n + 2]).cuda(), i32([start, 3]).cuda(), n + 2)
    R.append(c, 0, x[n:], x[n:], [0, 0, 2], [0, 3])          # the other row's tokens are written
    c["lens"][0] = want
    same(kv, c)
    assert kv.device_error() == hra.DEVERR_POS_RANGE


def test_rows_without_pages_keep_their_length(hra):  # noqa: F811
    """No page for any new token: nothing is written or counted.  A page for some of them: the length covers all."""
    rows, W, P = 5, 40, 16
    c = build([0, 20, 0, 0, 17], H=1, D=64, P=P, width=W, spare=60, seed=6)
    free = [p for p in range(c["refs"].numel()) if not c["refs"][p]]
    c["table"][1] = -1                                      # held 20 positions, lost its pages
    c["table"][2, 38] = free[0]                             # the last of the new tokens' pages alone
    c["table"][3, 0] = 1 << 20                              # no page of the pool
    new, start = [1, 3, 620, 5, 4], [0, 20, 2, 0, 17]
    x = torch.randn(sum(new), 1, 64, generator=torch.Generator().manual_seed(7)).to(BF16)
    kv = gpu(hra, c)
    kv.append(0, x.cuda(), x.cuda(), i32(cu_of(new)).cuda(), i32(start).cuda(), max(new))
    R.append(c, 0, x, x, cu_of(new), start)
    c["lens"][:4] = i32([0, 20, 622, 0])
    same(kv, c)
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE
    kv.append(0, x[:1].cuda(), x[:1].cuda(), i32([0, 0, 1, 1, 1, 1]).cuda(), i32([0, 4, 0, 0, 0]).cuda(), 1)
    c["lens"][1] = 5                                        # written nowhere, before its end
    same(kv, c)


def test_a_freed_row_in_the_batch_stays_empty(hra):  # noqa: F811
    """A row that has ended and was freed takes part in no later step: its length stays 0, so an update that extends the others
    gives it no page."""
    c = build([20, 33, 18], H=1, D=64, P=16, width=4, spare=6, seed=8)
    c["scales"] = torch.nan_to_num(c["scales"], nan=0.5)
    kv = gpu(hra, c)
    kv.update(i32([0, -1, 2]).cuda(), i32([2, 0, 2]).cuda())
    x = torch.randn(3, 1, 64, generator=torch.Generator().manual_seed(9)).to(BF16).cuda()
    for step in range(2):
        kv.append(0, x, x, i32([0, 1, 2, 3]).cuda(), i32([20 + step, step, 18 + step]).cuda(), 1)
        assert kv.lens.tolist() == [21 + step, 0, 19 + step]
    kv.update()
    assert kv.page_table[1].tolist() == [-1] * 4


# ------------------------------------------------------------------------- not-a-numbers behind the causal mask

@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 16), (1, 1, 64, 32), (2, 3, 128, 64), (1, 8, 64, 16), (1, 2, 64, 128)])
@pytest.mark.parametrize("new,kept", [([2], [0]), ([4, 3], [29, 12]), ([2, 5], [15, 600]), ([40, 21], [0, 50]), ([130], [33]),
                                      ([70, 2], [2300, 2200]), ([4, 2], [1022, 60])])
@pytest.mark.parametrize("what", ["V", "K"])
def test_nan_reaches_only_the_rows_that_see_it(hra, H, G, D, P, new, kept, what):  # noqa: F811
    """A token whose K or V has a NaN: rows before it are what they would be without it, rows from it on have the formula's NaN
    (of V in its dimension alone)."""
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=sum(lens) + D)
    which, cu, T = (1 if what == "V" else 0), cu_of(new), sum(new)
    q = torch.randn(T, H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    want, bound = R.attend(c, 0, q, cu, lens)                # without the NaNs
    nan = torch.zeros(T, H * G, D, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in {n // 2, n - 1}:                            # two of the new tokens, the last one among them
            at, head, dim = kept[b] + i, i % H, (7 * i + 5) % D
            c["codes"][0, int(c["table"][b, at // P]), which, head, at % P, dim] = 0xFF if i & 1 else 0x7F
            nan[cu[b] + i:cu[b + 1], head * G:(head + 1) * G, dim if which else slice(None)] = True
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu).cuda(), i32(lens).cuda(), max(new), max(lens)).double().cpu()
    assert torch.equal(torch.isnan(got), nan)
    assert bool(((got - want).abs() <= bound)[~nan].all())
    assert kv.device_error() == 0


@pytest.mark.parametrize("new,kept", [([4, 3], [600, 12]), ([200, 64], [1000, 0])])
def test_tokens_that_are_nan_throughout(hra, new, kept):  # noqa: F811
    """K and V of a row's last cached token and of all its new ones are NaN: every output is, soon; of the other row's, none."""
    H, G, D, P = 2, 4, 128, 16
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=3)
    for pos in range(max(0, kept[0] - 1), lens[0]):
        c["codes"][0, int(c["table"][0, pos // P]), :, :, pos % P] = 0x7F
    q = torch.randn(sum(new), H * G, D, generator=torch.Generator().manual_seed(4)).to(BF16)
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max(new), max(lens)).double().cpu()
    assert bool(torch.isnan(got[:new[0]]).all())
    want, bound = R.attend({**c, "table": c["table"][1:]}, 0, q[new[0]:], [0, new[1]], lens[1:])
    assert bool(((got[new[0]:] - want).abs() <= bound).all())


# --------------------------------------------------------------------------------------------- scales of zero

@pytest.mark.parametrize("G,D", [(4, 128), (2, 64)])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [60, 30]])
@pytest.mark.parametrize("which", ["K", "V", "both", "all V"])
def test_a_scale_of_zero_makes_values_of_zero(hra, G, D, new, which):  # noqa: F811
    """As Kv8Cache.new fills them: such a block's keys have a score of 0 and count, its values are 0, however it is read."""
    lens = [200, 77]
    c = build(lens, H=2, D=D, P=32, seed=11)
    for b, blocks in ((0, (0, 4, 12)), (1, (1, 4))):
        for blk in blocks:
            s = c["scales"][0, int(c["table"][b, blk // 2]), :, :, blk % 2]
            if which in ("K", "both"):
                s[0] = 0
            if which in ("V", "both"):
                s[1] = 0
    if which == "all V":
        c["scales"][0, :, 1] = torch.where(torch.isnan(c["scales"][0, :, 1]), c["scales"][0, :, 1], torch.zeros(()))
    got = check(hra, c, new, lens, G)
    assert which != "all V" or bool((got == 0).all())


# ------------------------------------------------------------------- memory of calls on another stream than the current one

def freed_in_use(nbytes):
    """Address of a block that the current stream still writes after it went back to the allocator.  (The stream is busy for
    some 50 ms; what runs meanwhile has run before, since the first launch of a kernel loads it and may take as long.)"""
    x = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(100_000_000)
    x.fill_(1)
    return x.data_ptr()


@pytest.mark.parametrize("new", [1, 70])
def test_outputs_and_workspaces_are_memory_of_the_stream_they_are_written_on(hra, new):  # noqa: F811
    H, G, D = 2, 4, 128
    lens = [2500, 900]
    c = build(lens, H=H, D=D, P=16, seed=12)
    q = torch.randn(2 * new, H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    cu, n = i32([0, new, 2 * new]).cuda(), i32(lens).cuda()
    want = gpu(hra, c).attend(0, q, cu, n, new, 2500).clone()
    kv, side = gpu(hra, c), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    size = kv.attention_workspace_size(2, 2 * new, H * G, new, 2500)
    busy = [freed_in_use(size), freed_in_use(q.nbytes)]      # what the current stream's pool would hand out
    out = kv.attend(0, q, cu, n, new, 2500, stream=side)
    assert kv._attn_ws.buf.data_ptr() not in busy and out.data_ptr() not in busy
    assert not torch.cuda.current_stream().query()           # the current stream was still at work
    side.synchronize()
    assert torch.equal(out, want)
    # dropped while the side stream still writes it
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    out = kv.attend(0, q, cu, n, new, 2500, stream=side)
    at = out.data_ptr()
    del out
    assert torch.empty_like(q).data_ptr() != at and not side.query()
    # a workspace that another stream than its own uses goes back only when that one is done
    at = kv._attn_ws.buf.data_ptr()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    kv.attend(0, q, cu, n, new, 2500)                        # on the current stream
    kv._attn_ws.buf = None
    with torch.cuda.stream(side):
        assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != at
    assert not torch.cuda.current_stream().query()


def test_page_workspaces_are_memory_of_the_stream_they_are_used_on(hra):  # noqa: F811
    c = build([20, 17], L=1, H=1, D=64, P=16, rows=300, width=8, spare=30, seed=3, stale=0x22)
    c["scales"] = torch.nan_to_num(c["scales"], nan=0.5)
    kv, side = gpu(hra, c), torch.cuda.Stream()
    room = i32([30] * 2 + [0] * 298).cuda()
    gpu(hra, c).update(None, room)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    import ctypes
    busy = freed_in_use(hra.lib().hra_kv8_pages_workspace_size(ctypes.byref(kv.struct)))
    kv.update(None, room, stream=side)
    assert kv._pages_ws.buf.data_ptr() != busy and not torch.cuda.current_stream().query()
    side.synchronize()
    want = R.update(c, None, room.tolist())
    assert torch.equal(kv.page_table.cpu(), want[0]) and torch.equal(kv.refs.cpu(), want[2])


@pytest.fixture(scope="module")
def model(hra):  # noqa: F811
    import workloads as W
    d = W.tiny_dims()
    w = W.make_backbone(d, 21)
    return d, {"embed": w["embed"].cuda(), "final_norm": w["final_norm"].cuda(),
               "layers": [{k: v.cuda() for k, v in l.items()} for l in w["layers"]]}


@pytest.mark.parametrize("paged", [True, False])
def test_the_backbones_outputs_and_workspace_are_memory_of_the_call_s_stream(hra, model, paged):  # noqa: F811
    d, w = model
    toks = torch.randint(0, d.vocab, (2, 40), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    lens, results = [40, 23], []
    for other in (False, True):
        bb = hra.Backbone(d, w)
        if paged:
            cache = hra.Kv8Cache.new(d, 2, 64)
            cache.update(room=i32([64, 64]).cuda())
            need = hra.lib().hra_prefill_kv8_workspace_size(__import__("ctypes").byref(bb.dims), cache.ref, 2, 63, 40, 40)
        else:
            cache = hra.new_kv_cache(d, 2, 64, fill=0.0)
            need = bb.prefill_workspace_size(2, 63, 40)
        side = torch.cuda.Stream() if other else None
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        busy = [freed_in_use(need), freed_in_use(4 * d.hidden)] if other else []
        a = bb.prefill(toks, lens, cache, stream=side)
        assert bb.ws.buf.data_ptr() not in busy and a.data_ptr() not in busy
        b = bb.decode(a, lens, cache, stream=side)
        pos = i32([n + 1 for n in lens]).cuda() if side is None else torch.tensor([n + 1 for n in lens], dtype=torch.int32).pin_memory()
        if other:
            with torch.cuda.stream(side):
                pos = pos.cuda(non_blocking=True)
        c = bb.decode_dev(b, pos, 63, cache, stream=side)
        assert a.data_ptr() != b.data_ptr() != c.data_ptr()
        if other:
            assert not torch.cuda.current_stream().query()   # all of it while the current stream was at work
            side.synchronize()
        results.append((a.clone(), b.clone(), c.clone()))
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("paged", [True, False])
def test_a_captured_decode_keeps_its_workspace(hra, model, paged):  # noqa: F811
    """A later call needs a larger workspace; a graph captured before still has the one it was captured with.  (Its token sits
    at position 0 and attends itself alone, so what the prefill leaves in the cache does not matter.)"""
    d, w = model
    bb = hra.Backbone(d, w)
    if paged:
        cache = hra.Kv8Cache.new(d, 4, 96)
        cache.update(room=i32([96] * 4).cuda())
    else:
        cache = hra.new_kv_cache(d, 4, 96, fill=0.0)
    emb = torch.randn(1, d.hidden, generator=torch.Generator().manual_seed(2)).mul(0.05).to(BF16).cuda()
    pos, out = i32([0]).cuda(), torch.zeros(1, d.hidden, dtype=BF16, device="cuda")
    first = bb.decode_dev(emb, pos, 95, cache, advance=False).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bb.decode_dev(emb, pos, 95, cache, advance=False, out=out)
    small = bb.ws.buf.data_ptr(), bb.ws.buf.numel()
    toks = torch.randint(0, d.vocab, (4, 90), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    bb.prefill(toks[1:], [90, 80, 70], cache)
    assert bb.ws.buf.data_ptr() != small[0]
    torch.cuda.synchronize()
    fill = [torch.full((small[1],), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and all(bool((f == 3).all()) for f in fill)


# ------------------------------------------------------------------------------------- the object and its tensors

def test_the_tensors_of_a_cache_cannot_be_replaced(hra):  # noqa: F811
    """Its calls would go on reading the ones it was made of."""
    kv = gpu(hra, build([20], H=1, D=64, P=16))
    for name in ("codes", "scales", "page_table", "lens", "refs", "errors"):
        was = getattr(kv, name)
        with pytest.raises(hra.HraError):
            setattr(kv, name, was.clone())
        assert getattr(kv, name) is was
    kv.lens += 1                                             # in place: the same tensor
    assert kv.lens.tolist() == [21]
    bare = hra.Kv8Cache(kv.codes, kv.scales, kv.page_table, kv.lens)
    with pytest.raises(hra.HraError):
        bare.refs = kv.refs


def test_a_loop_s_cache_struct_is_the_cache_s(hra, model):  # noqa: F811
    """ARLoop.kv: the struct that describes the cache, of either kind."""
    import workloads as W
    d, w = model
    audio = W.make_audio(d, torch.Generator().manual_seed(8))
    head, bb = hra.AudioHead(d, audio["head_w"].cuda(), audio["code_emb"].cuda()), hra.Backbone(d, w)
    hid = torch.zeros(2, d.hidden, dtype=BF16, device="cuda")
    flat, paged = hra.new_kv_cache(d, 2, 32, fill=0.0), hra.Kv8Cache.new(d, 2, 32)
    loop = hra.ARLoop(bb, head, flat, hid, [3, 4], 31)
    assert loop.kv.base == flat.data_ptr() and (loop.kv.batch, loop.kv.n_slots) == (2, 32)
    loop = hra.ARLoop(bb, head, paged, hid, [3, 4], 31)
    assert loop.kv.codes == paged.codes.data_ptr() and loop.kv.rows == 2


# --------------------------------------------------------------------------------------- the path at its main shape

def test_one_layer_at_full_width(hra):  # noqa: F811
    """head_dim 128, 32 q and 8 kv heads, hidden 2560, over 512 rows: the keys and values that prefill writes are the bf16 path's,
    quantised; its last rows, those of a chunk after over 2048 positions, and a token's are a plain layer's over that cache."""
    import dataclasses

    import workloads as W
    from test_gpu_kv8_model import close, cpu, plain
    d = dataclasses.replace(W.full_dims(1), vocab=2048)
    assert (d.hidden, d.n_q_heads, d.n_kv_heads, d.head_dim) == (2560, 32, 8, 128)
    w = W.make_backbone(d, 31)
    bb = hra.Backbone(d, {"embed": w["embed"].cuda(), "final_norm": w["final_norm"].cuda(),
                          "layers": [{k: v.cuda() for k, v in l.items()} for l in w["layers"]]})
    g = torch.Generator().manual_seed(32)
    new, start = [2300, 613], [0, 0]
    toks = torch.randint(0, d.vocab, (2, 2300), generator=g, dtype=torch.int32)
    kv = hra.Kv8Cache.new(d, 2, 2560)
    kv.update(room=i32([2500, 900]).cuda())
    want, cu = cpu(kv), cu_of(new)
    out = bb.prefill(toks.cuda(), new, kv)
    flat = hra.new_kv_cache(d, 2, 2560, fill=0.0)
    bb.prefill(toks.cuda(), new, flat)
    k, v = (torch.cat([flat[0, b, i, :, :n].transpose(0, 1).cpu() for b, n in enumerate(new)]) for i in (0, 1))
    R.append(want, 0, k, v, cu, start)
    same(kv, want)
    # the last rows again, each as one token at the end of its row
    embed = lambda t: w["embed"][t.long()].double()  # noqa: E731
    last = torch.stack([toks[b, n - 1] for b, n in enumerate(new)])
    close(out, plain(d, w, embed(last), cpu(kv), [1, 1], [n - 1 for n in new]))
    # a chunk, every row through the whole layer
    start, new = new, [130, 64]
    toks = torch.randint(0, d.vocab, (2, 130), generator=g, dtype=torch.int32)
    c = cpu(kv)
    out = bb.prefill(toks.cuda(), new, kv, start_pos=start, full_last_layer=True)
    x = torch.cat([embed(toks[b, :n]) for b, n in enumerate(new)])
    close(out, plain(d, w, x, c, new, start)[[129, 193]])
    # a token
    start = [s + n for s, n in zip(start, new)]
    emb = torch.randn(2, d.hidden, generator=g).mul(0.05).to(BF16)
    c = cpu(kv)
    close(bb.decode(emb.cuda(), start, kv), plain(d, w, emb.double(), c, [1, 1], start))
    assert kv.device_error() == 0 and kv.lens.tolist() == [s + 1 for s in start]


def test_a_row_that_has_ended_leaves_the_batch(hra, model):  # noqa: F811
    """Freed and moved behind the live rows by one update; a smaller batch goes on as before and sets no error bit."""
    d, w = model
    bb = hra.Backbone(d, w)
    g = torch.Generator().manual_seed(41)
    toks = torch.randint(0, d.vocab, (4, 40), generator=g, dtype=torch.int32).cuda()
    lens, outs = [37, 12, 21, 30], []
    for ended in (False, True):
        kv = hra.Kv8Cache.new(d, 4, 64, page_size=16)
        kv.update(room=i32([n + 8 for n in lens]).cuda())
        bb.prefill(toks, lens, kv)
        rows = [0, 1, 2, 3]
        if ended:                                            # row 1: its pages are free, rows 2 and 3 move down
            rows = [0, 2, 3]
            kv.update(i32(rows + [-1]).cuda(), i32([8, 8, 8, 0]).cuda())
            assert kv.lens.tolist() == [37, 21, 30, 0] and kv.page_table[3].tolist() == [-1] * 4
        e = torch.Generator().manual_seed(42)
        for step in range(3):
            emb = torch.randn(4, d.hidden, generator=e).mul(0.05).to(BF16).cuda()
            out = bb.decode(emb[rows].contiguous(), [lens[r] + step for r in rows], kv)
            outs.append(out if ended else out[[0, 2, 3]])
        assert kv.device_error() == 0
        assert kv.lens.tolist() == ([40, 24, 33, 0] if ended else [n + 3 for n in lens])
    for a, b in zip(outs[:3], outs[3:]):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ queries of a wide range

@pytest.mark.parametrize("new", [[1, 1], [40, 9]])
def test_queries_whose_largest_element_lies_just_below_a_power_of_two(hra, new):  # noqa: F811
    """Mantissas of the largest element above 1.75, where q / s is least, and others down to 2^-15 of it that alone meet large
    keys.  Two E4M3 values may lose 2^-10 / 224 = 1.143 * 2^-18 of the largest (tests/test_kv8_edges.py), so a score may be off by
    8 / 7 of what kv8_ref.attend's split counts.  Its relative term expm1(w) of the worst score error w grows with w to at most
    expm1(8/7 w) <= 8/7 expm1(w) exp(w / 7): 1.3 times the split's share covers it while w <= 0.9."""
    kv_len = [300, 170]
    c = build(kv_len, H=1, D=64, P=16, seed=13)
    c["codes"][..., 0] &= 0x87                     # dim 0 of K and V: zero or subnormal
    T = sum(new)
    g = torch.Generator().manual_seed(14)
    q = torch.randn(T, 2, 64, generator=g) * 0.1
    mantissa = 1.7578125 + torch.arange(T * 2) % 31 * 0.0078125
    q[..., 0] = (0.125 * mantissa * torch.exp2(torch.arange(T * 2) % 15)).view(T, 2)
    q = q.to(BF16)
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(kv_len).cuda(), max(new), 300).double().cpu()
    want, bound = R.attend(c, 0, q, cu_of(new), kv_len)
    if 2 * max(new) > 16:
        bound = bound + 1.3 * (R.attend(c, 0, q, cu_of(new), kv_len, split=True)[1] - bound)
    assert bool(((got - want).abs() <= bound).all()) and kv.device_error() == 0


def test_a_scale_that_float32_rounds_to_zero_is_not_the_default(hra):  # noqa: F811
    kv = gpu(hra, build([20], H=2, D=64, P=16))
    q, cu, n = torch.ones(1, 2, 64, dtype=BF16, device="cuda"), i32([0, 1]).cuda(), i32([20]).cuda()
    for scale in (1e-46, -1e-46, 1e39, float("nan")):
        with pytest.raises(hra.HraError):
            kv.attend(0, q, cu, n, 1, 20, scale=scale)
    assert torch.equal(kv.attend(0, q, cu, n, 1, 20, scale=0.125), kv.attend(0, q, cu, n, 1, 20))


def test_streams_by_any_object_with_a_handle(hra):  # noqa: F811
    """A torch stream, another object with its handle, and CUDA's own handles of the default stream."""
    from types import SimpleNamespace
    c = build([600, 40], H=2, D=64, P=16, seed=51)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    cu, n = i32([0, 1, 2]).cuda(), i32([600, 40]).cuda()
    want = gpu(hra, c).attend(0, q, cu, n, 1, 600).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, SimpleNamespace(cuda_stream=side.cuda_stream), SimpleNamespace(cuda_stream=0), SimpleNamespace(cuda_stream=1),
                   SimpleNamespace(cuda_stream=2)):
        kv = gpu(hra, c)
        torch.cuda.synchronize()
        out = kv.attend(0, q, cu, n, 1, 600, stream=stream)
        kv.update(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kv.page_table.cpu(), c["table"])
    with pytest.raises(AttributeError):
        kv.attend(0, q, cu, n, 1, 600, stream=7)


def test_other_calls_outputs_are_memory_of_the_call_s_stream(hra, model):  # noqa: F811
    """The codebook step, a linear layer and a quantisation, with stream= by name or by position."""
    import workloads as W
    d, _ = model
    audio = W.make_audio(d, torch.Generator().manual_seed(8))
    head = hra.AudioHead(d, audio["head_w"].cuda(), audio["code_emb"].cuda())
    g = torch.Generator().manual_seed(9)
    hid = torch.randn(3, d.hidden, generator=g).mul(0.1).to(BF16).cuda()
    a, w = torch.randn(200, 256, generator=g).to(BF16).cuda(), torch.randn(384, 256, generator=g).to(BF16).cuda()
    scale = torch.ones(1, device="cuda")
    results = []
    for other in (False, True):
        side = torch.cuda.Stream() if other else None
        state = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
        state[:, 1] = -1
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        busy = [freed_in_use(n) for n in (3 * d.n_codebooks * 4, 3 * d.hidden * 2, 200 * 384 * 2, 200 * 256)] if other else []
        codes, emb, _ = head.step(hid, state, stream=side)
        x8 = hra.fp8_quantize(a, scale, side)
        if other:
            assert not torch.cuda.current_stream().query()
        y = hra.hra_linear(a, w, stream=side)                # (waits for its stream)
        assert not {codes.data_ptr(), emb.data_ptr(), x8.data_ptr(), y.data_ptr()} & set(busy)
        torch.cuda.synchronize()
        results.append([t.clone() for t in (codes, emb, x8, y)])
    assert all(torch.equal(p, q) for p, q in zip(*results))
