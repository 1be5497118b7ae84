"""Attention of groups of rows that share the pages of a prefix, on the GPU against the plain 64-bit form of tests/kv8_ref.py
over the same tables, row by row."""
import random

import pytest
import torch

import kv8_ref as R
from test_gpu_kv8 import build, cu_of, gpu, hra, i32  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


LEAST = 96 << 20     # bytes that reading a prefix once has to save, by the call's bounds, before it is done


def wide(H, D, P, rows, groups):
    """Pages of a table row whose positions, as the bound of a prefix, make any call worth sharing."""
    return LEAST // (2 * H * D * P * max(1, rows - groups)) + 1


def shared(group_cu, prefix, lens, H, D, P, seed=0, **kw):
    """A cache whose rows of a group list their first row's pages for the prefix's whole pages."""
    c = build(lens, H=H, D=D, P=P, seed=seed, width=wide(H, D, P, len(lens), len(prefix)), **kw)
    for g, p in enumerate(prefix):
        for b in range(group_cu[g] + 1, group_cu[g + 1]):
            c["table"][b, :p // P] = c["table"][group_cu[g], :p // P]
    return c


def run(hra, c, kv, q, new, lens, group_cu, prefix, max_new=None, max_len=None, max_own=None, max_prefix=None, **kw):  # noqa: F811
    reach = hra.Kv8Reach(groups=i32(group_cu).cuda(), prefix=i32(prefix).cuda(), max_prefix=max_prefix or 1 << 30,
                         max_own=max_own)
    T = q.shape[0]
    out = torch.full((T + 2,) + q.shape[1:], 7.0, dtype=BF16, device="cuda")
    kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(lens).cuda(), max_new or max(new),
              max(lens) if max_len is None else max_len, out=out[:T], reach=reach, **kw)
    out = out.cpu()
    assert bool((out[T:] == 7).all())
    return out[:T]


def check(hra, c, new, lens, G, group_cu, prefix, errors=0, seed=3, **kw):  # noqa: F811
    H, D = c["codes"].shape[3], c["codes"].shape[5]
    T = sum(new)
    q = torch.randn(T, H * G + 1, D, generator=torch.Generator().manual_seed(seed)).to(BF16)[:, 1:]
    want, bound = R.attend(c, 0, q, cu_of(new), lens, split=True)
    kv = gpu(hra, c)
    for max_prefix in ((max(prefix), None) if "max_prefix" not in kw else (kw.pop("max_prefix"),)):   # row by row (mostly), and once
        before = hra.hra_launch_counter()
        got = run(hra, c, kv, q, new, lens, group_cu, prefix, max_prefix=max_prefix, **kw)
        kernels = hra.hra_launch_counter() - before
        over = float(((got.double() - want).abs() - bound).max())
        assert over <= 0, f"{over:.3g} over the bound"      # (a NaN is not)
        assert kv.device_error() == errors
        kv.errors.zero_()
    if max_prefix is None and len(prefix) < len(lens) and G * (kw.get("max_new") or max(new)) <= 64:
        assert kernels == 4                                 # read once
    return got


SHAPES = [(2, 4, 128, 64), (1, 1, 64, 16), (2, 3, 128, 32), (1, 16, 64, 16), (1, 8, 128, 128), (3, 5, 64, 32)]


@pytest.mark.parametrize("H,G,D,P", SHAPES)
@pytest.mark.parametrize("group_cu,prefix,own", [
    ([0, 4], [203], [1, 40, 17, 129]), ([0, 2], [129], [1, 1]), ([0, 3, 4, 7], [300, 64, 500], [5, 1, 300, 9, 1, 77, 2]),
    ([1, 4], [131], [90, 1, 2, 3, 700, 0, 1]), ([0, 0, 5, 5], [50, 260, 9], [3, 1, 1, 1, 40]), ([0, 2, 4], [0, 15], [6, 7, 8, 9])])
def test_single_tokens(hra, H, G, D, P, group_cu, prefix, own):  # noqa: F811
    lens = [o for o in own]
    for g, p in enumerate(prefix):
        for b in range(group_cu[g], group_cu[g + 1]):
            lens[b] = p + own[b]
    c = shared(group_cu, prefix, lens, H, D, P, seed=sum(lens) + P)
    check(hra, c, [1] * len(lens), lens, G, group_cu, prefix, max_own=max(own))


@pytest.mark.parametrize("H,G,D,P", SHAPES)
@pytest.mark.parametrize("new", [[2, 0, 4, 1], [4, 4, 4, 4], [0, 0, 3, 0]])
@pytest.mark.parametrize("prefix,own", [(200, [0, 3, 40, 130]), (1000, [300, 0, 0, 1])])
def test_steps(hra, H, G, D, P, new, prefix, own):  # noqa: F811
    lens = [prefix + o + n for o, n in zip(own, new)]
    c = shared([0, 4], [prefix], lens, H, D, P, seed=prefix + P)
    check(hra, c, new, lens, G, [0, 4], [prefix], max_own=max(own) + 4)


@pytest.mark.parametrize("G,new", [(1, [64, 3, 20]), (4, [16, 9, 1]), (4, [17, 1, 0]), (2, [31, 32, 7]), (2, [100, 5, 60])])
def test_steps_of_many_tokens(hra, G, new):  # noqa: F811
    """Both sides of the number of tokens from which the sequences' own tiles are taken."""
    own = [5, 80, 33]
    lens = [700 + o + n for o, n in zip(own, new)]
    c = shared([0, 3], [700], lens, 2, 64, 16, seed=G)
    check(hra, c, new, lens, G, [0, 3], [700], max_own=200)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 2, 64, 16)])
@pytest.mark.parametrize("rows,prefix", [(5, 4100), (40, 2050), (70, 600)])
def test_long_prefixes_and_many_rows(hra, H, G, D, P, rows, prefix):  # noqa: F811
    rng = random.Random(rows)
    lens = [prefix + rng.randrange(1, 60) for _ in range(rows)]
    lens[rows // 2] = prefix + 900
    c = shared([0, rows], [prefix], lens, H, D, P, seed=rows)
    a = check(hra, c, [1] * rows, lens, G, [0, rows], [prefix], max_own=900)
    assert torch.equal(a, check(hra, c, [1] * rows, lens, G, [0, rows], [prefix], max_own=900))   # again: the same sums
    # another bound: other parts, the same values
    check(hra, c, [1] * rows, lens, G, [0, rows], [prefix], max_own=1)


def test_many_groups(hra):  # noqa: F811
    rng = random.Random(4)
    group_cu, prefix, lens = [0], [], []
    for _ in range(150):
        r = rng.randrange(0, 4)
        p = rng.randrange(0, 100)
        group_cu.append(group_cu[-1] + r)
        prefix.append(p)
        lens += [p + rng.randrange(1, 30) for _ in range(r)]
    lens += [1, 50]      # rows of no group
    c = shared(group_cu, prefix, lens, 1, 64, 16, seed=1)
    check(hra, c, [1] * len(lens), lens, 4, group_cu, prefix)


def test_a_prefix_is_no_longer_than_what_its_rows_hold(hra):  # noqa: F811
    """Rows that hold less than the prefix, nothing, or fewer positions than new tokens: the group shares less or nothing."""
    for lens, new in (([300, 40, 300], [1, 1, 1]), ([300, 1, 300], [1, 1, 1]), ([300, 0, 300], [1, 1, 1]), ([64, 2, 64], [3, 3, 1]),
                      ([300, 0, 300], [1, 0, 1])):
        c = build([300, 300, 300], H=2, D=64, P=16, seed=2, width=wide(2, 64, 16, 3, 1))
        c["table"][1:, :18] = c["table"][0, :18]
        check(hra, c, new, lens, 4, [0, 3], [288], max_len=300)


@pytest.mark.parametrize("new", [[0, 1, 1, 0], [0, 0, 3, 2], [0, 2, 0, 0]])
def test_a_group_goes_on_without_its_first_rows(hra, new):  # noqa: F811
    """Rows that ended list no pages: the prefix is read through a row that has new tokens."""
    lens = [140 + n for n in new]
    c = shared([0, 4], [128], lens, 2, 64, 16, seed=9)
    c["table"][[b for b in range(4) if new[b] == 0]] = -1
    check(hra, c, new, [n if m else 0 for n, m in zip(lens, new)], 4, [0, 4], [128])


def test_prefixes_of_groups_without_new_tokens_do_not_count(hra):  # noqa: F811
    lens = [200, 180, 0, 0, 190]
    c = shared([0, 2, 4, 4], [128, 0, 0], lens, 1, 64, 16, seed=12)
    check(hra, c, [1, 1, 0, 0, 1], lens, 4, [0, 2, 4, 4], [128, 2 ** 31 - 1, 2 ** 31 - 1], max_prefix=1 << 30)


def test_more_rows_than_the_plan_holds_and_the_most_groups(hra):  # noqa: F811
    rows, rng = 1100, random.Random(2)
    group_cu = [min(g, 1000) + max(0, g - 1000) * 4 for g in range(1025)]     # 1000 groups of one row, 24 of four
    prefix = [rng.randrange(0, 70) for _ in range(1024)]
    lens = [1] * rows
    for g, p in enumerate(prefix):
        for b in range(group_cu[g], group_cu[g + 1]):
            lens[b] = p + rng.randrange(1, 40)
    c = shared(group_cu, prefix, lens, 1, 64, 16, seed=2)
    check(hra, c, [1] * rows, lens, 2, group_cu, prefix)


def test_group_numbers_outside_the_batch_are_clamped(hra):  # noqa: F811
    lens = [100, 90, 80, 120]
    c = build(lens, H=1, D=64, P=16, seed=2, width=wide(1, 64, 16, 4, 3))
    c["table"][1:, :4] = c["table"][0, :4]
    for group_cu, prefix in (([-3, 2, 9], [64, 64]), ([0, 3, 1, 4], [64, 64, 64]), ([0, 4], [-5]), ([7, 9], [64]), ([2, 0], [64])):
        check(hra, c, [1] * 4, lens, 2, group_cu, prefix, errors=hra.DEVERR_POS_RANGE, max_prefix=1 << 30)


def test_packed_rows_out_of_order_stay_inside_the_workspace(hra):  # noqa: F811
    """cu that claims rows twice: no result is promised, and nothing outside the output is written."""
    lens = [100, 90, 80, 120]
    c = build(lens, H=1, D=64, P=16, seed=2, width=wide(1, 64, 16, 4, 3))
    c["table"][1:, :4] = c["table"][0, :4]
    kv = gpu(hra, c)
    q = torch.randn(4, 2, 64).to(BF16).cuda()
    reach = hra.Kv8Reach(groups=i32([0, 2, 4]).cuda(), prefix=i32([64, 64]).cuda())
    for cu in ([0, 4, 0, 4, 0], [4, 3, 2, 1, 0], [-7, 100, 2, 3, 4], [0, 1, 1, 1, 99]):
        need = kv.attention_workspace_size(4, 4, 2, 4, 120, reach)
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        out = torch.full((6, 2, 64), 7.0, dtype=BF16, device="cuda")
        kv.attend(0, q, i32(cu).cuda(), i32(lens).cuda(), 4, 120, out=out[:4], workspace=ws[:need], reach=reach)
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0x5A).all()) and bool((out[4:] == 7).all())


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 4]])
def test_hidden_pages_and_clamped_lengths(hra, new):  # noqa: F811
    lens = [200, 180, 230]
    c = shared([0, 3], [128], lens, 1, 64, 16, seed=6)
    c["table"][:, 3] = -1
    c["table"][1, 9] = 1 << 20
    check(hra, c, new, lens, 2, [0, 3], [128], errors=hra.DEVERR_PAGE_RANGE)
    c = build([96, 96, 96], H=1, D=64, P=16, width=wide(1, 64, 16, 3, 1))
    c["table"][:, :2] = c["table"][0, :2]
    check(hra, c, new, [96, -70, 96], 2, [0, 3], [32], errors=hra.DEVERR_POS_RANGE, max_len=96)


def test_tokens_beyond_max_new_get_no_output(hra):  # noqa: F811
    lens, new = [200, 150], [9, 2]
    c = shared([0, 2], [128], lens, 1, 64, 16)
    q = torch.randn(11, 2, 64, generator=torch.Generator().manual_seed(8)).to(BF16)
    kv = gpu(hra, c)
    want, bound = R.attend(c, 0, q, [0, 9, 11], lens, split=True)
    for max_new in (2, 5):
        have = run(hra, c, kv, q, new, lens, [0, 2], [128], max_new=max_new, max_len=200)
        assert kv.device_error() == hra.DEVERR_POS_RANGE
        rows = list(range(max_new)) + [9, 10]
        assert float(((have.double() - want).abs() - bound)[rows].max()) <= 0
        assert bool((have[max_new:9] == 7).all())


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 2, 3]])
def test_a_nan_reaches_only_the_tokens_that_see_it(hra, new):  # noqa: F811
    lens = [128 + 40 + n for n in new]
    P, G = 16, 4
    c = shared([0, 3], [128], lens, 1, 64, P, seed=2)
    marks = [(1, 128 + 40, 5), (2, 128 + 40 + new[2] - 1, 9)]     # a row's first, and another's last new token
    for b, pos, dim in marks:
        c["codes"][0, int(c["table"][b, pos // P]), 1, 0, pos % P, dim] = 0x7F
    T = sum(new)
    q = torch.randn(T, G, 64, generator=torch.Generator().manual_seed(4)).to(BF16)
    q[0, 1, 7] = float("nan")
    got = run(hra, c, gpu(hra, c), q, new, lens, [0, 3], [128])
    nan = torch.zeros(T, G, 64, dtype=torch.bool)
    nan[0, 1] = True
    for b, pos, dim in marks:
        for i in range(new[b]):
            nan[cu_of(new)[b] + i, :, dim] |= pos <= lens[b] - new[b] + i
    assert torch.equal(torch.isnan(got), nan)
    c["codes"][c["codes"] == 0x7F] = 0
    q[0, 1, 7] = 0
    want, bound = R.attend(c, 0, q, cu_of(new), lens, split=True)
    assert float(((got.double() - want).abs() - bound)[~nan].max()) <= 0


@pytest.mark.parametrize("case", ["zero V", "tiny V", "huge K", "far V"])
def test_scales_far_apart(hra, case):  # noqa: F811
    """The prefix's and the row's own sums have maxima of their own: neither loses the other's terms."""
    for where in (0, 140):
        lens = [160, 150, 155]
        c = shared([0, 3], [128], lens, 1, 64, 16, seed=4)
        for b in range(3):
            page = int(c["table"][b, where // 16])
            if case == "zero V":
                c["codes"][0, page, 1] = 0
                c["scales"][0, page, 1] = 2.0 ** -126
            elif case == "tiny V":
                c["scales"][0, page, 1] = 2.0 ** -100
            elif case == "huge K":
                c["scales"][0, page, 0] = 2.0 ** -2
            else:
                c["scales"][0, page, 1] = 2.0 ** 40
        check(hra, c, [1] * 3, lens, 4, [0, 3], [128])
        check(hra, c, [3, 2, 4], lens, 4, [0, 3], [128])


def test_captured_and_replayed_with_other_groups(hra):  # noqa: F811
    """The device arrays are read at each replay: other groups, prefixes and lengths under the same bounds."""
    lens = [[300, 280, 290, 310], [200, 170, 290, 150]]
    groups = [([0, 4], [256]), ([0, 2], [160])]
    c = build([320] * 4, H=2, D=64, P=16, seed=7, width=wide(2, 64, 16, 4, 1))
    c["table"][1:, :16] = c["table"][0, :16]
    kv = gpu(hra, c)
    q = torch.randn(4, 8, 64, generator=torch.Generator().manual_seed(1)).to(BF16)
    cu, kl, qg = i32(range(5)).cuda(), i32(lens[0]).cuda(), q.cuda()
    g, p = i32(groups[0][0]).cuda(), i32(groups[0][1]).cuda()
    reach = hra.Kv8Reach(groups=g, prefix=p, max_own=200)
    out = torch.zeros_like(qg)
    ws = torch.empty(kv.attention_workspace_size(4, 4, 8, 1, 320, reach), dtype=torch.uint8, device="cuda")
    kv.attend(0, qg, cu, kl, 1, 320, out=out, workspace=ws, reach=reach)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend(0, qg, cu, kl, 1, 320, out=out, workspace=ws, reach=reach)
    for n, (gc, pf) in zip(lens, groups):
        kl.copy_(i32(n)), g.copy_(i32(gc)), p.copy_(i32(pf)), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, bound = R.attend(c, 0, q, list(range(5)), n, split=True)
        assert float(((out.cpu().double() - want).abs() - bound).max()) <= 0
    assert kv.device_error() == 0


def test_calls_at_once_with_workspaces_of_their_own(hra):  # noqa: F811
    lens = [3000 + i for i in range(8)]
    c = shared([0, 8], [2048], lens, 2, 128, 64, seed=3)
    kv = gpu(hra, c)
    reach = hra.Kv8Reach(groups=i32([0, 8]).cuda(), prefix=i32([2048]).cuda(), max_own=1000)
    cu, kl = i32(range(9)).cuda(), i32(lens).cuda()
    qs = [torch.randn(8, 8, 128, generator=torch.Generator().manual_seed(i)).to(BF16).cuda() for i in range(4)]
    alone = [kv.attend(0, q, cu, kl, 1, 3008, reach=reach) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    need = kv.attention_workspace_size(8, 8, 8, 1, 3008, reach)
    for _ in range(5):
        got = []
        for q, st in zip(qs, streams):
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            st.wait_stream(torch.cuda.current_stream())
            got.append((kv.attend(0, q, cu, kl, 1, 3008, workspace=ws, stream=st, reach=reach), ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, (b, _) in zip(alone, got))
