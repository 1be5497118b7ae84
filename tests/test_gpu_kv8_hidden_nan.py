"""Not-a-numbers that a token does not see, in prompts over the paged 8-bit cache: one V element at a time in tiles of every
fill, and queries that see absent pages alone; against the plain 64-bit forms of kv8_ref and kv8_reach_ref."""
import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_gpu_kv8 import build, cu_of, gpu, hra, i32  # noqa: F401
from test_gpu_kv8_shared import wide

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def one_mark_at_a_time(hra, new, lens, b, G, D, window, H=2, P=16):  # noqa: F811
    """V of the last token of sequence b, and through a window of a position that its later tokens have left, with a NaN in one
    dim of each 32: the tokens that see it have a NaN in that dim, and every other output is what it is without."""
    sinks, T, cu = (2 if window else 0), sum(new), cu_of(new)
    c = build(lens, H=H, D=D, P=P, seed=sum(lens) + D + G)
    q = torch.randn(T, H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    if window:
        want, bound = W.attend(c, 0, q, cu, lens, window, sinks, split=True)
    else:
        want, bound = R.attend(c, 0, q, cu, lens, split=True)
    kv, n, head = gpu(hra, c), new[b], H - 1
    args = (0, q.cuda(), i32(cu).cuda(), i32(lens).cuda(), max(new), max(lens))
    reach = hra.Kv8Reach(window=window, sinks=sinks) if window else None
    first = lens[b] - n
    for pos in [lens[b] - 1] + ([first - window + n // 2] if window else []):
        page = int(c["table"][b, pos // P])
        sees = [pos <= p and (not window or pos > p - window or pos < sinks) for p in range(first, lens[b])]
        assert any(sees) and not all(sees)
        for dim in range(5, D, 35):                      # one in each 32: 5, 40, 75, 110
            at = kv.codes[0, page, 1, head, pos % P, dim]
            kept = at.clone()
            at.fill_(0x7F)
            got = kv.attend(*args, reach=reach).cpu()
            at.copy_(kept)
            nan = torch.zeros(T, H * G, D, dtype=torch.bool)
            nan[cu[b]:cu[b + 1], head * G:(head + 1) * G, dim] = torch.tensor(sees)[:, None]
            assert torch.equal(torch.isnan(got), nan), (pos, dim)
            assert bool(((got.double() - want).abs() <= bound)[~nan].all()), (pos, dim)
    assert kv.device_error() == 0


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("G,D", [(4, 128), (4, 64)])
@pytest.mark.parametrize("n", [5, 8, 16, 24, 32, 40, 53])
def test_v_in_tiles_of_every_fill(hra, G, D, n, window):  # noqa: F811
    one_mark_at_a_time(hra, [n], [n + 40], 0, G, D, window)


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("G,D,n", [(1, 128, 17), (1, 128, 32), (1, 128, 33), (1, 64, 32), (1, 64, 64), (1, 128, 64), (1, 128, 65),
                                   (1, 128, 96), (1, 128, 97), (1, 128, 128), (1, 128, 129), (2, 128, 9), (3, 128, 6), (3, 128, 22),
                                   (3, 128, 42), (3, 64, 10), (5, 128, 4), (7, 64, 3), (8, 128, 4), (11, 128, 2), (16, 128, 2),
                                   (16, 64, 2), (16, 128, 5), (16, 128, 8), (16, 128, 9)])
def test_v_at_other_heads(hra, G, D, n, window):  # noqa: F811
    one_mark_at_a_time(hra, [n], [n + 40], 0, G, D, window, H=1, P=64)


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("G,D", [(4, 128), (2, 64)])
@pytest.mark.parametrize("new,b", [([40, 3], 1), ([3, 40, 12], 0), ([60, 9, 1], 1), ([40] + [1] * 65 + [10], 66),
                                   ([1, 0, 70] + [2] * 64, 2)])
def test_v_of_one_sequence_among_others(hra, G, D, new, b, window):  # noqa: F811
    """Short sequences beside prompts, with and without a list of the items."""
    one_mark_at_a_time(hra, new, [n + 40 for n in new], b, G, D, window, H=1)


# ------------------------------------------------------------------------- queries that see absent pages alone

def blind(c, new, lens, rows, window):
    """The packed tokens of which every position that they see is absent, once the pages of `rows` ({row: pages}) are."""
    for b, pages in rows.items():
        c["table"][b, pages] = -1
    P, out = c["codes"].shape[4], torch.zeros(sum(new), dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(n):
            p = lens[b] - n + i
            lo = max(0, p - window + 1) if window else 0
            out[cu_of(new)[b] + i] = all(int(c["table"][b, j // P]) < 0 for j in range(lo, p + 1))
    return out


@pytest.mark.parametrize("window", [0, 25])
@pytest.mark.parametrize("G,D", [(4, 64), (2, 128)])
@pytest.mark.parametrize("new,kept,rows", [
    ([40], [30], {0: slice(None)}), ([40, 33], [0, 100], {0: slice(0, 1)}), ([40, 33], [90, 7], {0: slice(None), 1: slice(1, 2)}),
    ([130], [5000], {0: slice(None)}), ([20] * 70, [9] * 70, {3: slice(None), 69: slice(0, 1)}), ([3, 2], [20, 60], {1: slice(None)})])
def test_queries_that_see_absent_pages_alone(hra, G, D, new, kept, rows, window):  # noqa: F811
    """They see no position, so they are 0 whatever they hold, and a page that is absent is reported."""
    lens, T = [a + b for a, b in zip(new, kept)], sum(new)
    c = build(lens, H=1, D=D, P=16, seed=5)
    none = blind(c, new, lens, rows, window)
    q = torch.randn(T, G, D, generator=torch.Generator().manual_seed(6)).to(BF16)
    clean = q.clone()
    q[none] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0]).repeat(D // 4).to(BF16)
    reach = hra.Kv8Reach(window=window) if window else None
    kv = gpu(hra, c)
    args = (i32(cu_of(new)).cuda(), i32(lens).cuda(), max(new), max(lens))
    got, want = (kv.attend(0, x.cuda(), *args, reach=reach).cpu() for x in (q, clean))
    assert bool(none.any()) and bool((got[none] == 0).all()) and torch.equal(got, want)
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 4]])
def test_queries_of_a_group_that_see_absent_pages_alone(hra, new):  # noqa: F811
    """The same over a shared prefix: of a row that shares pages none of which is there, and has none of its own."""
    lens = [128 + 40 + n for n in new]
    c = build(lens, H=1, D=64, P=16, seed=5, width=wide(1, 64, 16, 3, 1))
    c["table"][:, :8] = -1
    c["table"][1] = -1
    T, G, cu = sum(new), 4, cu_of(new)
    q = torch.randn(T, G, 64, generator=torch.Generator().manual_seed(6)).to(BF16)
    clean = q.clone()
    q[cu[1]:cu[2]] = float("nan")
    kv = gpu(hra, c)
    reach = hra.Kv8Reach(groups=i32([0, 3]).cuda(), prefix=i32([128]).cuda(), max_own=64)
    got, want = (kv.attend(0, x.cuda(), i32(cu).cuda(), i32(lens).cuda(), max(new), max(lens), reach=reach).cpu()
                 for x in (q, clean))
    assert bool((got[cu[1]:cu[2]] == 0).all()) and torch.equal(got, want)
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE
