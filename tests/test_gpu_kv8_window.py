"""Attention through a window with sinks over the paged 8-bit cache, and page updates that drop what the window has left,
on the GPU against the plain 64-bit forms of tests/kv8_reach_ref.py."""
import random

import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_gpu_kv8 import build, cu_of, gpu, hra, i32  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def hide(c, new, lens, window, sinks, P, drop):
    """Every position that no new token sees holds NaN in K and V; drop: pages of nothing but such positions are no pages."""
    for b, (n, L) in enumerate(zip(new, lens)):
        lo = L - n - window + 1
        for pos in range(min(sinks, L), max(0, min(lo, L))):
            page = int(c["table"][b, pos // P])
            c["codes"][:, page, :, :, pos % P] = 0x7F
        if drop:
            for i in range(-(-L // P)):
                if W.gone(L - n, P, window, sinks, i):
                    c["table"][b, i] = -1


def check(hra, c, new, lens, G, window, sinks, max_len=None, errors=0, seed=3, scale=0.0, max_new=None, q=None):  # noqa: F811
    H, D = c["codes"].shape[3], c["codes"].shape[5]
    T = sum(new)
    if q is None:
        q = torch.randn(T, H * G, D, generator=torch.Generator().manual_seed(seed)).to(BF16)
    max_new = max_new or max(new)
    want, bound = W.attend(c, 0, q, cu_of(new), lens, window, sinks, scale=scale, split=max_new * G > 16)
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max_new, max(lens) if max_len is None else max_len,
                    scale=scale, reach=hra.Kv8Reach(window=window, sinks=sinks)).cpu()
    assert kv.device_error() == errors
    over = float(((got.double() - want).abs() - bound).max())
    assert over <= 0, f"{over:.3g} over the bound"      # (a NaN is not)
    return got


SHAPES = [(2, 4, 128, 64), (1, 1, 64, 16), (2, 3, 128, 32), (1, 16, 64, 16), (1, 8, 128, 128), (1, 9, 64, 64)]


@pytest.mark.parametrize("H,G,D,P", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 33), (96, 64), (5000, 0), (7, 5000)])
@pytest.mark.parametrize("lens", [[1, 2, 17, 63], [300, 0, 129, 1000]])
def test_single_tokens(hra, H, G, D, P, window, sinks, lens):  # noqa: F811
    c = build(lens, H=H, D=D, P=P, seed=sum(lens) + P)
    new = [1] * len(lens)
    hide(c, new, lens, window, sinks, P, drop=window % 2 == 0)
    check(hra, c, new, lens, G, window, sinks)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 2, 64, 16), (1, 16, 128, 32)])
@pytest.mark.parametrize("window,sinks", [(511, 1), (700, 0), (1500, 129), (2048, 4)])
def test_single_tokens_in_shares(hra, H, G, D, P, window, sinks):  # noqa: F811
    lens = [700, 3, 4049, 0, 512, 2047]
    c = build(lens, H=H, D=D, P=P, seed=window)
    hide(c, [1] * 6, lens, window, sinks, P, drop=True)
    check(hra, c, [1] * 6, lens, G, window, sinks)


@pytest.mark.parametrize("H,G,D,P", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (33, 20), (64, 64), (100, 0), (300, 70), (5000, 3)])
@pytest.mark.parametrize("new,kept", [([2, 1, 4], [30, 0, 100]), ([0, 33, 1, 130], [5, 0, 400, 64]), ([129, 64], [1, 391]),
                                      ([1, 2, 3, 300], [700, 0, 16, 1])])
def test_prompts(hra, H, G, D, P, window, sinks, new, kept):  # noqa: F811
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=sum(new))
    hide(c, new, lens, window, sinks, P, drop=window % 2 == 0)
    check(hra, c, new, lens, G, window, sinks)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (8, 3, 64, 16), (5, 16, 64, 32)])
@pytest.mark.parametrize("window,sinks", [(40, 17), (130, 0), (5000, 1)])
@pytest.mark.parametrize("rows", [64, 65, 90])
def test_many_prompts(hra, H, G, D, P, window, sinks, rows):  # noqa: F811
    """Both sides of the number of sequences and of items up to which a CTA looks for its own."""
    rng = random.Random(rows + G)
    new = [rng.choice([0, 1, rng.randrange(2, 30), rng.randrange(2, 60)]) for _ in range(rows)]
    new[0] = 40
    lens = [n + rng.choice([0, rng.randrange(200)]) for n in new]
    c = build(lens, H=H, D=D, P=P, seed=rows)
    hide(c, new, lens, window, sinks, P, drop=True)
    got = check(hra, c, new, lens, G, window, sinks)
    q = torch.randn(sum(new), H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    if window == 5000:
        plain = gpu(hra, c).attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max(new), max(lens)).cpu()
        assert torch.equal(plain, got)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 2, 64, 16), (1, 5, 128, 128)])
@pytest.mark.parametrize("window,sinks", [(2500, 0), (3001, 7), (1000, 2000), (200, 4)])
@pytest.mark.parametrize("new,kept", [([130], [5500]), ([33, 1, 90, 0, 2], [4100, 5000, 5, 40, 4047]), ([1, 200], [6000, 0])])
def test_prompts_in_shares(hra, H, G, D, P, window, sinks, new, kept):  # noqa: F811
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=sum(kept))
    hide(c, new, lens, window, sinks, P, drop=True)
    a = check(hra, c, new, lens, G, window, sinks)
    assert torch.equal(a, check(hra, c, new, lens, G, window, sinks))


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [40, 70]])
def test_a_window_of_everything_is_no_window(hra, new):  # noqa: F811
    lens = [500, 333]
    c = build(lens, H=2, D=128, P=32, seed=5)
    q = torch.randn(sum(new), 8, 128, generator=torch.Generator().manual_seed(1)).to(BF16)
    kv = gpu(hra, c)
    args = (0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max(new), 500)
    plain = kv.attend(*args).cpu()
    for window, sinks in ((500, 0), (1 << 30, 1 << 30), (501, 17)):
        assert torch.equal(plain, kv.attend(*args, reach=hra.Kv8Reach(window=window, sinks=sinks)).cpu())


@pytest.mark.parametrize("new,G", [([4, 3], 4), ([60, 40], 2), ([33], 8)])
def test_a_nan_reaches_only_the_tokens_that_see_it(hra, new, G):  # noqa: F811
    """V with a NaN at positions that enter and leave the tokens' windows: exactly the tokens that see one have it."""
    lens = [300 + n for n in new]
    P, window, sinks = 16, 50, 3
    c = build(lens, H=1, D=64, P=P, seed=2)
    marks = {}
    for b, n in enumerate(new):
        first = lens[b] - n
        marks[b] = [(first - window + 1 + n // 2, 5), (first + n // 3, 9), (1, 11) if b else (4, 11)]
        for pos, dim in marks[b]:
            c["codes"][0, int(c["table"][b, pos // P]), 1, 0, pos % P, dim] = 0x7F
    T = sum(new)
    q = torch.randn(T, G, 64, generator=torch.Generator().manual_seed(4)).to(BF16)
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max(new), max(lens),
                    reach=hra.Kv8Reach(window=window, sinks=sinks)).cpu()
    nan = torch.zeros(T, G, 64, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(n):
            p = lens[b] - n + i
            for pos, dim in marks[b]:
                nan[cu_of(new)[b] + i, :, dim] |= pos <= p and (pos > p - window or pos < sinks)
    assert torch.equal(torch.isnan(got), nan)
    clean = {k: v.clone() for k, v in c.items()}
    clean["codes"][clean["codes"] == 0x7F] = 0
    want, bound = W.attend(clean, 0, q, cu_of(new), lens, window, sinks, split=max(new) * G > 16)
    over = ((got.double() - want).abs() - bound)[~nan]
    assert float(over.max()) <= 0


@pytest.mark.parametrize("new,lens", [([1, 1, 1], [0, 5, 0]), ([4, 3], [2, 30]), ([40, 33], [5, 100]), ([70, 1], [66, 0])])
@pytest.mark.parametrize("window", [0, 20])
def test_rows_that_see_no_position_are_zero_whatever_their_q_is(hra, new, lens, window):  # noqa: F811
    c = build([max(1, n) for n in lens], H=1, D=64, P=16, seed=3)
    G, T, cu = 4, sum(new), cu_of(new)
    q = torch.randn(T, G, 64, generator=torch.Generator().manual_seed(6)).to(BF16)
    empty = torch.zeros(T, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(n):
            empty[cu[b] + i] = lens[b] - n + i < 0
    clean = q.clone()
    q[empty] = torch.tensor([float("nan"), float("inf")]).repeat(32).to(BF16)
    reach = hra.Kv8Reach(window=window) if window else None
    kv = gpu(hra, c)
    args = (i32(cu).cuda(), i32(lens).cuda(), max(new), max(lens))
    got, want = (kv.attend(0, x.cuda(), *args, reach=reach).cpu() for x in (q, clean))
    assert bool(empty.any()) and bool((got[empty] == 0).all()) and torch.equal(got, want)


@pytest.mark.parametrize("new", [1, 3, 6])
def test_more_rows_than_a_table_of_sequences_holds(hra, new):  # noqa: F811
    """1100 rows: single tokens, short chunks and prompts; beyond 1024 the single tokens' items go whole."""
    rng = random.Random(new)
    news = [rng.choice([0, new, rng.randrange(0, new + 1)]) for _ in range(1100)]
    lens = [n + rng.choice([0, rng.randrange(60), 700 if b % 300 == 0 else 5]) for b, n in enumerate(news)]
    c = build(lens, H=1, D=64, P=16, seed=new)
    hide(c, news, lens, 30, 5, 16, drop=True)
    check(hra, c, news, lens, 4, 30, 5)


def test_strided_queries_on_another_stream(hra):  # noqa: F811
    new, lens = [40, 1, 33], [340, 77, 33]
    c = build(lens, H=2, D=64, P=16, seed=9)
    hide(c, new, lens, 50, 7, 16, drop=False)
    q = torch.randn(sum(new), 11, 64, generator=torch.Generator().manual_seed(5)).to(BF16)
    want, bound = W.attend(c, 0, q[:, 2:10], cu_of(new), lens, 50, 7, split=True)
    kv, side = gpu(hra, c), torch.cuda.Stream()
    args = q.cuda()[:, 2:10], i32(cu_of(new)).cuda(), i32(lens).cuda(), 40, 340
    side.wait_stream(torch.cuda.current_stream())
    got = kv.attend(0, *args, reach=hra.Kv8Reach(window=50, sinks=7), stream=side)
    side.synchronize()
    assert float(((got.cpu().double() - want).abs() - bound).max()) <= 0 and kv.device_error() == 0


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("G", [3, 4, 16])
def test_a_nan_in_queries_stays_in_its_sequence(hra, window, G):  # noqa: F811
    """A tile's rows behind its sequence's last hold the next one's queries: nothing of them reaches an output."""
    new, lens = [40, 33, 5, 50], [340, 33, 90, 201]
    c = build(lens, H=2, D=64, P=16, seed=4)
    cu = cu_of(new)
    q = torch.randn(sum(new), 2 * G, 64, generator=torch.Generator().manual_seed(5)).to(BF16)
    kv = gpu(hra, c)
    reach = hra.Kv8Reach(window=window) if window else None
    args = i32(cu).cuda(), i32(lens).cuda(), 50, 340
    clean = kv.attend(0, q.cuda(), *args, reach=reach).cpu()
    for b in range(4):
        bad = q.clone()
        bad[cu[b]:cu[b + 1]] = float("nan")
        got = kv.attend(0, bad.cuda(), *args, reach=reach).cpu()
        mine = torch.zeros(sum(new), dtype=torch.bool)
        mine[cu[b]:cu[b + 1]] = True
        assert bool(torch.isnan(got[mine]).all()) and torch.equal(got[~mine], clean[~mine])


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_missing_pages_in_sight_are_reported(hra, new):  # noqa: F811
    lens = [200, 150]
    c = build(lens, H=1, D=64, P=16, seed=6)
    c["table"][0, 0], c["table"][1, 8] = -1, 1 << 20      # a sink's page and one inside the window
    check(hra, c, new, lens, 2, 60, 4, errors=hra.DEVERR_PAGE_RANGE)


@pytest.mark.parametrize("new", [[1, 1], [70, 5]])
def test_length_zero_and_clamped_lengths(hra, new):  # noqa: F811
    c = build([96, 96], H=1, D=64, P=16, width=6)
    check(hra, c, new, [100, -4], 2, 20, 3, max_len=96, errors=hra.DEVERR_POS_RANGE)


def test_tokens_beyond_max_new_get_no_output(hra):  # noqa: F811
    lens, new = [200, 90], [9, 2]
    c = build(lens, H=1, D=64, P=16)
    q = torch.randn(11, 2, 64, generator=torch.Generator().manual_seed(8)).to(BF16)
    kv = gpu(hra, c)
    for max_new in (2, 5):
        out = torch.full((11, 2, 64), 7.0, dtype=BF16, device="cuda")
        kv.attend(0, q.cuda(), i32([0, 9, 11]).cuda(), i32(lens).cuda(), max_new, 200, out=out,
                  reach=hra.Kv8Reach(window=30, sinks=2))
        assert kv.device_error() == hra.DEVERR_POS_RANGE
        want, bound = W.attend(c, 0, q, [0, 9, 11], lens, 30, 2)
        have = out.cpu()
        rows = list(range(max_new)) + [9, 10]
        assert float(((have.double() - want).abs() - bound)[rows].max()) <= 0
        assert bool((have[max_new:9] == 7).all())


def test_captured_and_replayed_as_streams_grow(hra):  # noqa: F811
    """One graph of append, update and attend through a window, replayed token after token: every step's attention is the plain
    one, and the pool's pages in use stay bounded while the streams grow."""
    H, G, D, P, window, sinks, rows = 2, 2, 64, 16, 40, 4, 3
    kv = hra.Kv8Cache.new(type("d", (), dict(n_layers=1, n_kv_heads=H, head_dim=D)), rows, 512, n_pages=rows * 6, page_size=P)
    g = torch.Generator().manual_seed(7)
    reach = hra.Kv8Reach(window=window, sinks=sinks)
    room, cu = i32([1] * rows).cuda(), i32(range(rows + 1)).cuda()
    k, v = (torch.zeros(rows, H, D, dtype=BF16, device="cuda") for _ in range(2))
    q = torch.zeros(rows, H * G, D, dtype=BF16, device="cuda")
    start, lens = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)

    def step():
        start.copy_(kv.lens)
        kv.update(room=room, reach=reach)
        kv.append(0, k, v, cu, start, 1)
        lens.copy_(kv.lens)
        kv.attend(0, q, cu, lens, 1, 512, out=out, reach=reach)

    step()
    torch.cuda.synchronize()
    kv.lens.zero_(), kv.refs.zero_(), kv.page_table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(130):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert int((kv.refs > 0).sum()) <= rows * 5 and kv.lens.cpu().tolist() == [t + 1] * rows
        if t in (0, 3, 39, 40, 41, 77, 129):
            c = {"codes": kv.codes.cpu(), "scales": kv.scales.cpu(), "table": kv.page_table.cpu()}
            want, bound = W.attend(c, 0, q.cpu(), list(range(rows + 1)), [t + 1] * rows, window, sinks)
            assert float(((out.cpu().double() - want).abs() - bound).max()) <= 0
    assert kv.device_error() == 0


# ------------------------------------------------------------------------------------------ pages

@pytest.mark.parametrize("rows,width,P,window,sinks,seed", [
    (6, 20, 16, 40, 4, 1), (6, 20, 16, 1, 0, 2), (9, 12, 32, 100, 33, 3), (5, 40, 16, 200, 500, 4), (4, 300, 16, 64, 16, 5),
    (64, 520, 16, 33, 1, 6)])
def test_update_in_a_chain(hra, rows, width, P, window, sinks, seed):  # noqa: F811
    rng = random.Random(seed)
    lens = [rng.randrange(width * P) if b < rows - 2 else 0 for b in range(rows)]
    c = build(lens, L=2, H=1, D=64, P=P, rows=rows, width=width, spare=rows * 8, seed=seed)
    kv = gpu(hra, c)
    reach = hra.Kv8Reach(window=window, sinks=sinks)
    for step in range(4):
        parents = [rng.randrange(-1, rows) if rng.random() < 0.5 else b for b in range(rows)]
        room = [rng.choice([0, 1, 5, P]) for _ in range(rows)]
        room = [r if p >= 0 and int(c["lens"][p]) + r <= width * P else 0 for r, p in zip(room, parents)]
        want = W.update(c, parents, room, window, sinks)
        kv.update(i32(parents).cuda(), i32(room).cuda(), reach=reach)
        if want is None:
            assert kv.device_error() == hra.DEVERR_PAGES_SPENT
            break
        table, lens_, refs, moves = want
        codes, scales = R.move(c, moves)
        # the tokens that room was for
        lens_ = torch.minimum(lens_ + i32(room) * (torch.rand(rows) < 0.7).int(), torch.tensor(width * P, dtype=torch.int32))
        torch.cuda.synchronize()
        assert torch.equal(kv.page_table.cpu(), table) and torch.equal(kv.refs.cpu(), refs)
        assert torch.equal(kv.codes.cpu(), codes) and torch.equal(kv.scales.cpu().view(torch.int32), scales.view(torch.int32))
        kv.lens.copy_(lens_)
        c = {"codes": codes, "scales": scales, "table": table, "lens": lens_, "refs": refs}
        assert kv.device_error() == 0


def test_update_frees_what_the_window_left_for_the_rows_that_need_it(hra):  # noqa: F811
    """A pool without one spare page: the pages that fall out of a window are the next step's fresh ones."""
    c = build([160, 31], L=1, H=1, D=64, P=16, rows=2, width=12, spare=0)
    kv = gpu(hra, c)
    kv.update(room=i32([1, 2]).cuda())
    assert kv.device_error() == hra.DEVERR_PAGES_SPENT
    kv.errors.zero_()
    want = W.update(c, [0, 1], [1, 2], 32, 16)
    kv.update(room=i32([1, 2]).cuda(), reach=hra.Kv8Reach(window=32, sinks=16))
    torch.cuda.synchronize()
    assert kv.device_error() == 0
    assert torch.equal(kv.page_table.cpu(), want[0]) and torch.equal(kv.refs.cpu(), want[2])
    assert kv.page_table.cpu()[0].tolist()[1:8] == [-1] * 7 and int(kv.page_table[0, 8]) >= 0
    table = kv.page_table.clone()
    # without a window holes get pages, as ever: 7 of them, and of the 12 pages 4 + 3 are listed
    kv.update(reach=hra.Kv8Reach())
    assert kv.device_error() == hra.DEVERR_PAGES_SPENT and torch.equal(kv.page_table, table)
