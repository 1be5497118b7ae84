"""The paged 8-bit cache on the GPU against the plain 64-bit forms of tests/kv8_ref.py: whole numbers, codes and scales
equal; attention within the bound that its roundings give (kv8_ref.attend)."""
import random

import pytest
import torch

import kv8_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def hra():
    import qwen3_prefill_delayed_gb300 as h
    h.lib()
    return h


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def build(lens, L=1, H=2, D=64, P=16, rows=None, width=None, spare=2, seed=0, stale=0x7F):
    """A CPU cache whose rows hold `lens` positions of random codes under random scales; every other slot holds the
    byte `stale` (0x7F: NaN) and every other scale NaN."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    rows = rows or len(lens)
    lens = list(lens) + [0] * (rows - len(lens))
    need = [-(-n // P) for n in lens]
    width = width or max(1, max(need))
    pages = sum(need) + spare
    ids = rng.sample(range(pages), sum(need))
    codes = torch.full((L, pages, 2, H, P, D), stale, dtype=torch.uint8)
    scales = torch.full((L, pages, 2, H, P // 16), float("nan"))
    table = torch.full((rows, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(need[b]):
            p = ids.pop()
            table[b, i] = p
            refs[p] = 1
            m = min(P, n - i * P)
            codes[:, p, :, :, :m] = R.e4m3_code(100 * torch.randn(L, 2, H, m, D, generator=g).double())
            e = torch.randint(-9, -4, (L, 2, H, -(-m // 16)), generator=g)
            scales[:, p, :, :, :-(-m // 16)] = torch.exp2(e.float())
    return {"codes": codes, "scales": scales, "table": table, "lens": i32(lens), "refs": refs}


def gpu(hra, c):
    return hra.Kv8Cache(*[c[k].cuda() for k in ("codes", "scales", "table", "lens", "refs")])


def same(kv, c):
    torch.cuda.synchronize()
    assert torch.equal(kv.codes.cpu(), c["codes"])
    assert torch.equal(kv.scales.cpu().view(torch.int32), c["scales"].view(torch.int32))
    assert torch.equal(kv.page_table.cpu(), c["table"]) and torch.equal(kv.lens.cpu(), c["lens"])


def cu_of(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("H,D,P", [(1, 64, 16), (2, 128, 64), (3, 128, 32), (8, 64, 128)])
@pytest.mark.parametrize("new,start", [
    ([1], [0]), ([1, 1, 1], [15, 16, 31]), ([5, 0, 33, 17], [0, 7, 3, 47]), ([16, 64, 1, 2], [16, 0, 63, 62]),
    ([100, 15], [29, 1])])
def test_append(hra, H, D, P, new, start):
    c = build(start, H=H, D=D, P=P, width=-(-160 // P), spare=40, seed=H + P)
    free = [p for p in range(c["refs"].numel()) if not c["refs"][p]]
    for b, (n, s) in enumerate(zip(new, start)):
        for i in range(-(-s // P), -(-(s + n) // P)):
            c["table"][b, i] = free.pop()
    g = torch.Generator().manual_seed(7)
    T = sum(new)
    # rows inside wider ones, magnitudes that raise some blocks' scales and not others'
    x = torch.randn(T, 2 * H + 1, D, generator=g) * torch.exp2(torch.randint(-6, 7, (T, 2 * H + 1, 1), generator=g).float())
    x = x.to(BF16)
    kv, xg = gpu(hra, c), x.cuda()
    kv.append(0, xg[:, :H], xg[:, H:2 * H], i32(cu_of(new)).cuda(), i32(start).cuda(), max(new))
    R.append(c, 0, x[:, :H], x[:, H:2 * H], cu_of(new), start)
    same(kv, c)
    assert kv.device_error() == 0


def test_append_special_values(hra):
    c = build([3], H=1, D=64, P=16, width=1, spare=0)
    x = torch.zeros(9, 1, 64)
    x[0, 0, 0] = float("inf")
    x[1, 0, 1] = float("nan")
    x[2, 0, 2] = -float("inf")
    x[3] = 3.3895313892515355e38
    x[4] = 1e-40
    x = x.to(BF16)
    kv = gpu(hra, c)
    kv.append(0, x.cuda(), torch.zeros_like(x).cuda(), i32([0, 9]).cuda(), i32([3]).cuda(), 9)
    R.append(c, 0, x, torch.zeros_like(x), [0, 9], [3])
    torch.cuda.synchronize()
    got = kv.codes.cpu()
    nan = (got & 127) == 127
    assert torch.equal(nan, (c["codes"] & 127) == 127)
    assert torch.equal(got.masked_fill(nan, 0), c["codes"].masked_fill(nan, 0))
    assert torch.equal(kv.scales.cpu(), c["scales"])


def test_append_all_zero_block_has_the_smallest_scale(hra):
    c = build([0], H=1, D=64, P=16, width=1, spare=1)
    c["table"][0, 0] = 0
    kv = gpu(hra, c)
    z = torch.zeros(2, 1, 64, dtype=BF16).cuda()
    kv.append(0, z, z, i32([0, 2]).cuda(), i32([0]).cuda(), 2)
    kv.append(0, z + 3, z, i32([0, 2]).cuda(), i32([2]).cuda(), 2)   # the block goes on with larger values
    torch.cuda.synchronize()
    assert float(kv.scales[0, 0, 1, 0, 0]) == 2.0 ** -126 and float(kv.scales[0, 0, 0, 0, 0]) == 2.0 ** -7
    assert kv.codes[0, 0, 0, 0, :4, 0].view(torch.float8_e4m3fn).float().cpu().tolist() == [0, 0, 384, 384]


def test_append_outside_positions_and_pages(hra):
    c = build([8, 8, 8, 8], H=1, D=64, P=16, width=2, spare=3)
    c["table"][1, 1] = 99            # no page of the pool
    c["table"][2, 1] = -1
    free = [p for p in range(c["refs"].numel()) if not c["refs"][p]]
    c["table"][0, 1] = free[0]
    c["table"][3, 1] = free[1]
    new, start = [12, 12, 12, 40], [8, 8, 8, 8]
    x = torch.randn(sum(new), 1, 64, generator=torch.Generator().manual_seed(3)).to(BF16)
    kv = gpu(hra, c)
    kv.append(0, x.cuda(), x.cuda(), i32(cu_of(new)).cuda(), i32(start).cuda(), 40)
    R.append(c, 0, x, x, cu_of(new), start)
    same(kv, c)
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE | hra.DEVERR_POS_RANGE
    kv.errors.zero_()
    kv.append(0, x[:4].cuda(), x[:4].cuda(), i32([0, 4]).cuda(), i32([-3]).cuda(), 4)
    assert kv.device_error() == hra.DEVERR_POS_RANGE
    c["lens"][0] = 1
    same(kv, c)


# --------------------------------------------------------------------------------------- attention

def check(hra, c, new, kv_len, G, layer=0, scale=0.0, seed=0, q_scale=1.0, max_len=None, errors=0, kv=None, q=None):
    H, D = c["codes"].shape[3], c["codes"].shape[5]
    g = torch.Generator().manual_seed(seed + 100)
    T, nq = sum(new), H * G
    if q is None:
        wide = (torch.randn(T + 2, nq + 1, D, generator=g) * q_scale).to(BF16)
        q, qg = wide[:T, :nq], wide.cuda()[:T, :nq]          # rows inside wider ones
    else:
        qg = q.cuda()
    kv = kv or gpu(hra, c)
    out = torch.full((T + 2, nq, D), 7.0, dtype=BF16).cuda()
    got = kv.attend(layer, qg, i32(cu_of(new)).cuda(), i32(kv_len).cuda(), max(new),
                    max(kv_len) if max_len is None else max_len, scale=scale, out=out[:T])
    torch.cuda.synchronize()
    want, bound = R.attend(c, layer, q, cu_of(new), kv_len, scale)
    off = (got.double().cpu() - want).abs()
    assert bool((out[T:] == 7.0).all())                      # rows behind the last are left as they were
    assert not bool(torch.isnan(got).any())
    worst = float((off / bound).max()) if T else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} of the bound"
    assert kv.device_error() == errors
    return got


@pytest.mark.parametrize("H,G,D,P", [(1, 1, 64, 16), (2, 2, 64, 16), (8, 4, 128, 64), (2, 8, 128, 128), (3, 5, 64, 32),
                                     (1, 16, 128, 16), (2, 7, 128, 32), (4, 3, 64, 64)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 63], [15, 16, 17, 64, 65, 300], [0, 5, 0, 129]])
def test_single_tokens(hra, H, G, D, P, lens):
    c = build(lens, H=H, D=D, P=P, seed=sum(lens) + P)
    check(hra, c, [1] * len(lens), lens, G)


@pytest.mark.parametrize("lens", [[1030], [700, 3, 2049, 0, 512], [4001] * 3])
@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 2, 64, 16)])
def test_single_tokens_long(hra, H, G, D, P, lens):
    c = build(lens, H=H, D=D, P=P, seed=len(lens))
    check(hra, c, [1] * len(lens), lens, G)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 1, 64, 16), (2, 3, 128, 32), (1, 16, 64, 16), (1, 8, 128, 128)])
@pytest.mark.parametrize("new,kept", [
    ([2, 1, 4], [30, 0, 100]), ([13], [0]), ([0, 33, 1, 130], [5, 0, 200, 64]), ([129, 64], [1, 191]),
    ([257], [300]), ([1, 2, 3, 300], [700, 0, 16, 1])])
def test_prompts(hra, H, G, D, P, new, kept):
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=sum(new))
    check(hra, c, new, lens, G)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 64), (1, 2, 64, 16), (1, 5, 128, 128)])
@pytest.mark.parametrize("new,kept", [
    ([130], [2500]), ([33, 1, 90, 0, 2], [2100, 3000, 5, 40, 2047]), ([70, 70], [2049, 4000]), ([1, 200], [5000, 0])])
def test_prompts_after_many_positions(hra, H, G, D, P, new, kept):
    """Long items in equal shares; single tokens beside them with many keys of their own."""
    lens = [a + b for a, b in zip(new, kept)]
    c = build(lens, H=H, D=D, P=P, seed=sum(kept))
    kv = gpu(hra, c)
    a = check(hra, c, new, lens, G, kv=kv)
    assert torch.equal(a, check(hra, c, new, lens, G, kv=kv))       # the shares' borders do not move
    assert bool(torch.isfinite(a).all())


def test_long_prompt_with_hidden_pages_and_rows_before_the_cache(hra):
    c = build([2300, 2100], H=2, D=64, P=16, seed=3)
    c["table"][0, 20:60], c["table"][1, :] = -1, 5000
    check(hra, c, [150, 40], [2300, 30], 2, max_len=2300, errors=hra.DEVERR_PAGE_RANGE)


def test_more_sequences_than_a_share_table_holds(hra):
    lens = [1 + (i * 37) % 70 for i in range(1100)]
    lens[500] = 1500
    c = build(lens, H=1, D=64, P=16, seed=3)
    check(hra, c, [1] * 1100, lens, 2)


def test_prompt_many_rows(hra):
    rng = random.Random(5)
    new = [rng.choice([0, 1, 2, 40, 77]) for _ in range(37)]
    kept = [rng.randrange(90) for _ in new]
    lens = [a + b for a, b in zip(new, kept)]
    check(hra, build(lens, H=1, D=64, P=16, seed=9), new, lens, 4)


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_rows_that_see_nothing(hra, new):
    # fewer cached positions than new tokens: the first ones sit before position 0
    lens = [0, 2]
    c = build([16, 16], H=2, D=64, P=16)
    got = check(hra, c, new, lens, 2, max_len=16)
    assert bool((got[:new[0]] == 0).all())


@pytest.mark.parametrize("new", [[1, 1], [70, 5]])
def test_length_zero_and_clamped_lengths(hra, new):
    c = build([96, 96], H=1, D=64, P=16, width=6)
    check(hra, c, new, [100, -4], 2, max_len=96, errors=hra.DEVERR_POS_RANGE)


@pytest.mark.parametrize("new", [[1, 1], [66, 12]])
def test_pages_outside_the_pool_are_hidden(hra, new):
    c = build([100, 90], H=2, D=128, P=16)
    c["table"][0, 2], c["table"][0, 5], c["table"][1, 0] = -1, 1 << 20, -7
    check(hra, c, new, [100, 90], 4, errors=hra.DEVERR_PAGE_RANGE)


@pytest.mark.parametrize("new", [[1], [50]])
@pytest.mark.parametrize("case", ["zero V", "tiny V", "zero K", "huge K", "far V"])
def test_scales_far_apart(hra, new, case):
    """Blocks whose scales differ by many powers of two: a block of zero or tiny V still counts in the softmax's sum,
    and one large V far down the softmax is not lost."""
    c = build([160], H=1, D=64, P=16, seed=4)
    page = [int(p) for p in c["table"][0]]
    if case == "zero V":
        c["codes"][0, page[:9], 1] = 0
        c["scales"][0, page[:9], 1] = 2.0 ** -126
    elif case == "tiny V":
        c["scales"][0, page[2:9], 1] = 2.0 ** -100
    elif case == "zero K":
        c["codes"][0, page[3:7], 0] = 0
        c["scales"][0, page[3:7], 0] = 2.0 ** -126
    elif case == "huge K":
        c["scales"][0, page[5], 0] = 2.0 ** -2
    else:
        c["scales"][0, page[4], 1] = 2.0 ** 40
        c["scales"][0, page[6], 0] = 2.0 ** -3
    check(hra, c, new, [160], 4)


@pytest.mark.parametrize("new", [[1], [40]])
def test_flat_tail(hra, new):
    """One key far above thousands of equal ones whose weights, taken together, count."""
    n = 4000
    c = build([n], H=1, D=64, P=64, seed=2)
    c["codes"][0, :, 0] = 0
    c["scales"][0, :, :] = 1.0 / 64
    c["codes"][0, :, 1] &= 0x7F
    c["codes"][0, :, 1] = c["codes"][0, :, 1].clamp(max=0x60)
    page, slot = int(c["table"][0, 3]), 5
    c["codes"][0, page, 0, 0, slot, 0] = int(R.e4m3_code(torch.tensor([288.0], dtype=torch.float64)))
    c["codes"][0, page, 1, 0, slot] = 0
    q = torch.zeros(new[0], 1, 64, dtype=BF16)
    q[:, :, 0] = 16.0                                        # score 16 * 4.5 / 8 = 9 against 0
    check(hra, c, new, [n], 1, q=q)


@pytest.mark.parametrize("new", [[1], [20]])
@pytest.mark.parametrize("q_scale", [2.0 ** -60, 2.0 ** 40, 8.0])
def test_query_magnitudes(hra, new, q_scale):
    c = build([90], H=1, D=64, P=16, seed=8)
    if q_scale > 2.0 ** 20:
        c["scales"][0, :, 0] *= 2.0 ** -42
    check(hra, c, new, [90], 2, q_scale=q_scale, scale=0.25)


@pytest.mark.parametrize("new", [[1, 1], [40, 40]])
def test_nan_stays_in_its_row(hra, new):
    c = build([64, 64], H=1, D=64, P=16)
    T = sum(new)
    q = torch.randn(T, 2, 64, generator=torch.Generator().manual_seed(1)).to(BF16)
    clean = q.clone()
    q[0, 0, 3] = float("nan")
    kv = gpu(hra, c)
    cu, kl = i32(cu_of(new)).cuda(), i32([64, 64]).cuda()
    a = kv.attend(0, q.cuda(), cu, kl, max(new), 64).cpu()
    b = kv.attend(0, clean.cuda(), cu, kl, max(new), 64).cpu()
    assert bool(torch.isnan(a[0, 0]).all())
    a[0, 0] = b[0, 0]
    assert torch.equal(a, b)


@pytest.mark.parametrize("new", [[1], [33]])
def test_layers_and_offsets_past_32_bits(hra, new):
    """A pool of more than 2^32 bytes: the row's pages lie at its end."""
    L, pages, H, P, D = 2, 8320, 8, 128, 128
    codes = torch.zeros(L, pages, 2, H, P, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(L, pages, 2, H, P // 16, device="cuda")
    assert codes.numel() > 2 ** 32
    small = build([200], L=2, H=H, D=D, P=P, width=2, spare=0, seed=3)
    ids = [pages - 1, pages - 3]
    for i in range(2):
        codes[:, ids[i]] = small["codes"][:, int(small["table"][0, i])].cuda()
        scales[:, ids[i]] = small["scales"][:, int(small["table"][0, i])].cuda()
    kv = hra.Kv8Cache(codes, scales, i32([ids]).cuda(), i32([200]).cuda())
    check(hra, small, new, [200], 4, layer=1, kv=kv)
    # and append writes there
    x = torch.randn(20, H, D, generator=torch.Generator().manual_seed(2)).to(BF16)
    kv.append(1, x.cuda(), x.cuda(), i32([0, 20]).cuda(), i32([195]).cuda(), 20)
    R.append(small, 1, x, x, [0, 20], [195])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(codes[:, ids[i]].cpu(), small["codes"][:, int(small["table"][0, i])])


def test_attention_is_repeatable_and_the_bound_only_splits(hra):
    lens = [900, 33, 2000, 64]
    c = build(lens, H=2, D=128, P=64, seed=6)
    kv = gpu(hra, c)
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(5)).to(BF16)
    a = check(hra, c, [1] * 4, lens, 4, kv=kv, q=q)
    b = check(hra, c, [1] * 4, lens, 4, kv=kv, q=q)
    assert torch.equal(a, b)
    check(hra, c, [1] * 4, lens, 4, kv=kv, q=q, max_len=kv.max_pages * 64)


# ------------------------------------------------------------------------------------------- pages

def random_rows(rows, W, P, pages, seed, L=2, H=1, D=64):
    """A valid state: some rows share full pages."""
    rng = random.Random(seed)
    lens = [rng.choice([0, 1, P - 1, P, P + 1, rng.randint(0, (W - 1) * P)]) for _ in range(rows)]
    c = build(lens, L=L, H=H, D=D, P=P, width=W, spare=pages, seed=seed, stale=0x35)
    c["scales"] = torch.nan_to_num(c["scales"], nan=0.5)
    return c


@pytest.mark.parametrize("rows,W,P,seed", [(1, 1, 16, 0), (5, 3, 16, 1), (16, 7, 32, 2), (40, 33, 16, 3), (64, 70, 16, 4)])
def test_update_in_a_chain(hra, rows, W, P, seed):
    """Forks, frees and reservations one after another, in place and out of place, against the plain form."""
    rng = random.Random(seed)
    c = random_rows(rows, W, P, rows * W, seed)
    kv = gpu(hra, c)
    for step in range(6):
        parents = None if step == 3 else [rng.choice([b, rng.randrange(rows), -1]) for b in range(rows)]
        lens = c["lens"].tolist()
        room = None if step == 4 else [
            rng.choice([0, 1, P, max(0, W * P - lens[parents[b] if parents else b])])
            if parents is None or parents[b] >= 0 else 5 for b in range(rows)]
        if room is not None:
            room = [min(r, W * P - lens[(parents[b] if parents else b)]) if parents is None or parents[b] >= 0 else r
                    for b, r in enumerate(room)]
        want = R.update(c, parents, room)
        assert want is not None
        out = kv.empty_pages() if step % 2 else None
        t, n, r = kv.update(None if parents is None else i32(parents).cuda(), None if room is None else i32(room).cuda(),
                            out=out)
        torch.cuda.synchronize()
        codes, scales = R.move(c, want[3])
        assert torch.equal(t.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(r.cpu(), want[2])
        if out is not None:   # the inputs are as they were
            assert torch.equal(kv.page_table.cpu(), c["table"]) and torch.equal(kv.refs.cpu(), c["refs"])
            for mine, new in zip((kv.page_table, kv.lens, kv.refs), out):
                mine.copy_(new)
        c.update(table=want[0], lens=want[1], refs=want[2], codes=codes, scales=scales)
        same(kv, c)
    assert kv.device_error() == 0
    want = R.compact(c)
    t, n, r = kv.compact()
    torch.cuda.synchronize()
    codes, scales = R.move(c, want[3])
    assert torch.equal(t.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(r.cpu(), want[2])
    assert torch.equal(kv.codes.cpu(), codes) and torch.equal(kv.scales.cpu(), scales)


def test_update_without_enough_pages_changes_nothing(hra):
    c = build([20, 17], L=1, H=1, D=64, P=16, rows=4, width=3, spare=3, stale=0x22)
    c["scales"] = torch.nan_to_num(c["scales"], nan=0.5)
    for parents, room in (([0, 1, 0, 1], [16, 16, 16, 16]), ([0, 1, -1, -1], [64, 0, 0, 0])):
        assert R.update(c, parents, room) is None
        kv = gpu(hra, c)
        for out in (None, kv.empty_pages()):
            t, n, r = kv.update(i32(parents).cuda(), i32(room).cuda(), out=out)
            assert kv.device_error() == hra.DEVERR_PAGES_SPENT
            assert torch.equal(t.cpu(), c["table"]) and torch.equal(n.cpu(), c["lens"]) and torch.equal(r.cpu(), c["refs"])
        same(kv, c)


def test_update_with_bad_numbers(hra):
    c = build([20, 17, 5], L=1, H=1, D=64, P=16, rows=3, width=3, spare=4, stale=0x22)
    c["scales"] = torch.nan_to_num(c["scales"], nan=0.5)
    c["table"][1, 0] = 1000
    c["lens"][2] = -4
    kv = gpu(hra, c)
    parents = [0, 1, 2]
    want = R.update(c, parents, [0, 0, -3])
    t, n, r = kv.update(i32(parents).cuda(), i32([0, 0, -3]).cuda(), out=kv.empty_pages())
    assert torch.equal(t.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(r.cpu(), want[2])
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE | hra.DEVERR_POS_RANGE
    kv.errors.zero_()
    want = R.update(c, [0, 7, -9], None)
    t, n, r = kv.update(i32([0, 7, -9]).cuda(), out=kv.empty_pages())
    assert torch.equal(t.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(r.cpu(), want[2])
    assert kv.device_error() == hra.DEVERR_PARENT_RANGE


@pytest.mark.parametrize("pages,used", [(1, 0), (1, 1), (40, 40), (2500, 1100), (2100, 3)])
def test_compact(hra, pages, used):
    rng = random.Random(pages)
    ids = rng.sample(range(pages), used)
    c = {"codes": torch.randint(0, 120, (2, pages, 2, 1, 16, 64), dtype=torch.uint8),
         "scales": torch.rand(2, pages, 2, 1, 1), "table": torch.full((4, max(1, used)), -1, dtype=torch.int32),
         "lens": i32([used * 16, 0, 3, 0]), "refs": torch.zeros(pages, dtype=torch.int32)}
    if used:
        c["table"][0] = i32(ids)
        c["table"][2, 0] = ids[0]
        c["refs"][ids] = 1
        c["refs"][ids[0]] = 2
    kv = gpu(hra, c)
    want = R.compact(c)
    t, n, r = kv.compact(out=kv.empty_pages())
    torch.cuda.synchronize()
    codes, scales = R.move(c, want[3])
    assert torch.equal(t.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(r.cpu(), want[2])
    assert torch.equal(kv.codes.cpu(), codes) and torch.equal(kv.scales.cpu(), scales)
    assert kv.device_error() == 0


# ------------------------------------------------------------------------------- used together

def test_run_together_on_a_side_stream(hra):
    """Two prompts appended and attended, each continued twice, single tokens, a row freed, the pool compacted: the
    outputs after every step are those of the plain forms on the same cache."""
    H, G, D, P, rows, W = 2, 4, 128, 16, 4, 8
    g = torch.Generator().manual_seed(11)
    c = {"codes": torch.zeros(2, 30, 2, H, P, D, dtype=torch.uint8), "scales": torch.zeros(2, 30, 2, H, 1),
         "table": torch.full((rows, W), -1, dtype=torch.int32), "lens": torch.zeros(rows, dtype=torch.int32),
         "refs": torch.zeros(30, dtype=torch.int32)}
    kv = gpu(hra, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def pages(parents, room):
        want = R.update(c, parents, room)
        with torch.cuda.stream(side):
            kv.update(i32(parents).cuda(), i32(room).cuda())
        codes, scales = R.move(c, want[3])
        c.update(table=want[0], lens=want[1], refs=want[2], codes=codes, scales=scales)

    def step(new):
        start = c["lens"].tolist()
        T = sum(new)
        with torch.cuda.stream(side):
            for layer in range(2):
                k, v = (torch.randn(T, H, D, generator=g).to(BF16) for _ in range(2))
                q = torch.randn(T, H * G, D, generator=g).to(BF16)
                cu, st = i32(cu_of(new)).cuda(), i32(start).cuda()
                lens = [s + n for s, n in zip(start, new)]
                kv.append(layer, k.cuda(), v.cuda(), cu, st, max(new))
                got = kv.attend(layer, q.cuda(), cu, i32(lens).cuda(), max(new), max(lens))
                R.append(c, layer, k, v, cu_of(new), start)
                want, bound = R.attend(c, layer, q, cu_of(new), lens)
                side.synchronize()
                assert bool(((got.double().cpu() - want).abs() <= bound).all())
        same(kv, c)

    pages([0, 1, -1, -1], [37, 20, 0, 0])
    step([37, 20, 0, 0])
    pages([0, 0, 1, 1], [3, 3, 3, 3])
    for _ in range(3):
        step([1, 1, 1, 1])
    pages([0, -1, 2, 3], [1, 0, 1, 20])
    with torch.cuda.stream(side):
        kv.compact()
    want = R.compact(c)
    codes, scales = R.move(c, want[3])
    c.update(table=want[0], lens=want[1], refs=want[2], codes=codes, scales=scales)
    step([1, 0, 1, 17])
    assert kv.device_error(stream=side) == 0


def test_captured_and_replayed(hra):
    """One captured frame (append + attend, lengths advancing on the device) replayed gives what eager calls give."""
    H, G, D, P = 2, 4, 128, 16
    c = build([20, 33], H=H, D=D, P=P, width=6, spare=12, seed=1)
    free = [p for p in range(c["refs"].numel()) if not c["refs"][p]]
    for b in range(2):
        for i in range(6):
            if c["table"][b, i] < 0:
                c["table"][b, i] = free.pop()
    a, z = gpu(hra, c), gpu(hra, c)
    cu = i32([0, 1, 2]).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn(2, n, D, generator=g, device="cuda").to(BF16) for n in (H, H, H * G))

    def frame(kv, pos, end, out):
        kv.append(0, k, v, cu, pos, 1)
        kv.attend(0, q, cu, end, 1, 90, out=out)
        pos += 1
        end += 1

    outs = [torch.zeros(2, H * G, D, dtype=BF16, device="cuda") for _ in range(2)]
    pos = [i32([20, 33]).cuda() for _ in range(2)]
    end = [i32([21, 34]).cuda() for _ in range(2)]
    z._attn_ws.get(1 << 24, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        frame(z, pos[1], end[1], outs[1])
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(25):
        frame(a, pos[0], end[0], outs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    assert torch.equal(a.codes, z.codes) and torch.equal(a.lens, z.lens) and a.lens.tolist() == [45, 58]


def test_wrapper_refusals(hra):
    c = build([20], H=2, D=64, P=16)
    kv = gpu(hra, c)
    cu, n = i32([0, 1]).cuda(), i32([20]).cuda()
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    for bad in (k.float(), k.cpu(), k[:, :1], torch.zeros(1, 2, 128, dtype=BF16, device="cuda"),
                torch.zeros(2, 2, 128, dtype=BF16, device="cuda")[:, :, ::2]):
        with pytest.raises(hra.HraError):
            kv.append(0, bad, k, cu, n, 1)
    with pytest.raises(hra.HraError):
        kv.append(0, k, k, i32([0, 1, 1]).cuda(), n, 1)
    with pytest.raises(hra.HraError):
        kv.append(0, k, k, cu.long(), n, 1)
    with pytest.raises(hra.HraError):
        kv.attend(0, torch.zeros(1, 3, 64, dtype=BF16, device="cuda"), cu, n, 1, 20)
    with pytest.raises(hra.HraError):
        kv.attend(0, k, cu, n, 1, 33)
    with pytest.raises(hra.HraError):
        kv.update(i32([0, 0]).cuda())
    with pytest.raises(hra.HraError):
        hra.Kv8Cache(kv.codes, kv.scales, kv.page_table, kv.lens).update()
    assert kv.attend(0, k[:0], i32([0, 0]).cuda(), n, 0, 20).shape == (0, 2, 64)


# ----------------------------------------------------------------------- calls at the edge of what is allowed

@pytest.mark.parametrize("G,max_len", [(2, 3000), (4, 3000), (2, 1500)])
def test_padded_rows_behind_a_short_sequence(hra, G, max_len):
    """batch * max_new = total_rows says nothing when the last rows are padding: a sequence of one token is answered."""
    kv_len = [40, max_len]
    c = build(kv_len, H=2, D=64, P=16, seed=5)
    kv = gpu(hra, c)
    q = torch.randn(64, 2 * G, 64, generator=torch.Generator().manual_seed(6)).to(BF16)
    out = torch.full((64, 2 * G, 64), 7.0, dtype=BF16).cuda()
    kv.attend(0, q.cuda(), i32([0, 32, 33]).cuda(), i32(kv_len).cuda(), 32, max_len, out=out)
    want, bound = R.attend(c, 0, q, [0, 32, 33], kv_len)
    assert bool(((out.double().cpu() - want).abs() <= bound)[:33].all())
    assert bool((out[33:] == 7.0).all()) and kv.device_error() == 0


@pytest.mark.parametrize("new,max_new,G,max_len", [([5, 3, 1], 2, 4, 130), ([5, 3], 2, 4, 700), ([70, 40], 50, 2, 300),
                                                   ([70, 9], 50, 2, 2500)])
def test_tokens_beyond_max_new_get_no_output(hra, new, max_new, G, max_len):
    kv_len = [max_len, 60, 20][:len(new)]
    c = build(kv_len, H=2, D=64, P=16, seed=7)
    kv = gpu(hra, c)
    T, cu = sum(new), cu_of(new)
    q = torch.randn(T, 2 * G, 64, generator=torch.Generator().manual_seed(8)).to(BF16)
    out = torch.full((T, 2 * G, 64), 7.0, dtype=BF16).cuda()
    kv.attend(0, q.cuda(), i32(cu).cuda(), i32(kv_len).cuda(), max_new, max_len, out=out)
    want, bound = R.attend(c, 0, q, cu, kv_len)
    ok = (out.double().cpu() - want).abs() <= bound
    for b, n in enumerate(new):
        m = cu[b] + min(n, max_new)
        assert bool(ok[cu[b]:m].all()) and bool((out[m:cu[b + 1]] == 7.0).all())
    assert kv.device_error() == hra.DEVERR_POS_RANGE


@pytest.mark.parametrize("max_len", [400, 2500])
def test_sequences_that_claim_the_same_rows_stay_inside_the_workspace(hra, max_len):
    """A cu that does not ascend asks for more tiles than the rows have: the list of tiles ends where its room ends."""
    B, T, G = 40, 200, 4
    c = build([300] * B, H=1, D=64, P=16, width=160, seed=9)
    kv = gpu(hra, c)
    cu = i32([0 if i % 2 == 0 else T for i in range(B + 1)]).cuda()
    q = torch.randn(T, G, 64, generator=torch.Generator().manual_seed(8)).to(BF16).cuda()
    size = kv.attention_workspace_size(B, T, G, T, max_len)
    room = torch.full((size + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 64, G, 64), 7.0, dtype=BF16).cuda()
    kv.attend(0, q, cu, i32([300] * B).cuda(), T, max_len, out=out[:T], workspace=room[:size])
    assert kv.device_error() == hra.DEVERR_POS_RANGE
    assert bool((room[size:] == 0x5A).all()) and bool((out[T:] == 7.0).all())


@pytest.mark.parametrize("G,far", [(8, 1500), (1, 2500)])
def test_prompts_of_more_sequences_than_a_list_chunk(hra, G, far):
    rng = random.Random(11)
    new = [rng.choice([0, 1, 3, 20]) for _ in range(1100)]
    new[3] = new[1090] = 40
    lens = [n + rng.randrange(50) for n in new]
    lens[1090] = far
    check(hra, build(lens, H=1, D=64, P=16, seed=12), new, lens, G)


@pytest.mark.parametrize("new", [[1, 1], [40, 9]])
def test_queries_with_elements_far_below_the_largest(hra, new):
    """One element of a q row 2^0 .. 2^14 times the others, which alone meet large keys: what the split of q into two E4M3
    values drops, 2^-18 of the largest (kv8_ref.attend, split)."""
    kv_len = [300, 170]
    c = build(kv_len, H=1, D=64, P=16, seed=13)
    c["codes"][..., 0] &= 0x87                     # dim 0 of K and V: zero or subnormal
    T = sum(new)
    g = torch.Generator().manual_seed(14)
    q = torch.randn(T, 2, 64, generator=g) * 0.1
    q[..., 0] = 0.2 * torch.exp2(torch.arange(T * 2) % 15).view(T, 2)
    q = q.to(BF16)
    kv = gpu(hra, c)
    got = kv.attend(0, q.cuda(), i32(cu_of(new)).cuda(), i32(kv_len).cuda(), max(new), 300)
    want, bound = R.attend(c, 0, q, cu_of(new), kv_len, split=2 * max(new) > 16)
    assert bool(((got.double().cpu() - want).abs() <= bound).all()) and kv.device_error() == 0


def test_a_captured_call_keeps_its_workspace(hra):
    """The object's workspace grows for a longer call; a graph captured before still has the one it was captured with."""
    c = build([900, 700], H=2, D=64, P=16, seed=15)
    kv = gpu(hra, c)
    g = torch.Generator().manual_seed(16)
    q = torch.randn(2, 4, 64, generator=g).to(BF16).cuda()
    cu, n = i32([0, 1, 2]).cuda(), i32([900, 700]).cuda()
    first = kv.attend(0, q, cu, n, 1, 900)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend(0, q, cu, n, 1, 900, out=out)
    small = kv._attn_ws.buf
    long = torch.randn(300, 4, 64, generator=g).to(BF16).cuda()
    kv.attend(0, long, i32([0, 290, 300]).cuda(), n, 290, 900)
    need = kv.attention_workspace_size(2, 300, 4, 290, 900)
    if small.numel() >= need:
        kv._attn_ws.get(2 * small.numel(), kv.device)
    assert kv._attn_ws.buf.data_ptr() != small.data_ptr() and kv._attn_ws.outgrown[-1] is small
    del small
    fill = [torch.full((kv._attn_ws.outgrown[-1].numel(),), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and all(bool((f == 3).all()) for f in fill)


@pytest.mark.parametrize("rows,W,P,seed", [(90, 300, 16, 5), (70, 500, 16, 6), (2100, 20, 16, 7)])
def test_update_of_large_tables_in_a_chain(hra, rows, W, P, seed):
    """Tables and pools whose plan takes several CTAs."""
    test_update_in_a_chain(hra, rows, W, P, seed)


def test_large_update_without_enough_pages_changes_nothing(hra):
    c = build([20, 17], L=1, H=1, D=64, P=16, rows=1500, width=40, spare=3000, stale=0x22)
    kv = gpu(hra, c)
    for parents, room in (([0] * 1500, [16] + [40] * 1499), ([0, 1] + [-1] * 1498, [641] + [0] * 1499)):
        assert R.update(c, parents, room) is None
        for out in (None, kv.empty_pages()):
            kv.errors.zero_()
            t, n, r = kv.update(i32(parents).cuda(), i32(room).cuda(), out=out)
            assert kv.device_error() == hra.DEVERR_PAGES_SPENT
            assert torch.equal(t.cpu(), c["table"]) and torch.equal(n.cpu(), c["lens"]) and torch.equal(r.cpu(), c["refs"])


@pytest.mark.parametrize("pages,used", [(40000, 9000), (40001, 33000), (33000, 0), (33000, 33000)])
def test_compact_of_a_large_pool(hra, pages, used):
    test_compact(hra, pages, used)


@pytest.mark.parametrize("new,kept", [([1, 1, 1], [900, 3, 60]), ([2, 45, 9], [300, 80, 0]), ([100, 40], [2500, 10])])
def test_rows_and_outputs_at_16_bytes(hra, new, kept):
    """Rows 16 bytes off a 32-byte border, q strides that are odd multiples of 16 bytes, an output that starts at 16."""
    H, G, D = 2, 4, 128
    kv_len = [a + b for a, b in zip(new, kept)]
    c = build(kv_len, H=H, D=D, P=16, seed=21)
    kv = gpu(hra, c)
    T, cu = sum(new), cu_of(new)
    flat = torch.randn(8 + T * (H * G * D + 8), generator=torch.Generator().manual_seed(22)).to(BF16)
    q = torch.as_strided(flat, (T, H * G, D), (H * G * D + 8, D, 1), 8)
    qg = torch.as_strided(flat.cuda(), (T, H * G, D), (H * G * D + 8, D, 1), 8)
    buf = torch.full((16 + T * H * G * D,), 7.0, dtype=BF16, device="cuda")
    out = buf[8:8 + T * H * G * D].view(T, H * G, D)
    kv.attend(0, qg, i32(cu).cuda(), i32(kv_len).cuda(), max(new), max(kv_len), out=out)
    want, bound = R.attend(c, 0, q, cu, kv_len)
    assert bool(((out.double().cpu() - want).abs() <= bound).all())
    assert bool((buf[:8] == 7.0).all()) and bool((buf[-8:] == 7.0).all()) and kv.device_error() == 0


def test_calls_at_once_with_workspaces_of_their_own(hra):
    c = build([3000, 500, 40], H=2, D=128, P=16, seed=23)
    kv = gpu(hra, c)
    g = torch.Generator().manual_seed(24)
    one = torch.randn(3, 8, 128, generator=g).to(BF16).cuda()
    many = torch.randn(160, 8, 128, generator=g).to(BF16).cuda()
    calls = [(one, i32([0, 1, 2, 3]).cuda(), 1), (many, i32([0, 90, 150, 160]).cuda(), 90)]
    n = i32([3000, 500, 40]).cuda()
    want = [kv.attend(0, q, cu, n, m, 3000).clone() for q, cu, m in calls]
    ws = [torch.empty(kv.attention_workspace_size(3, q.shape[0], 8, m, 3000), dtype=torch.uint8, device="cuda") for q, _, m in calls]
    out = [torch.empty_like(q) for q, _, _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, cu, m), w, o, s in zip(calls, ws, out, streams):
            kv.attend(0, q, cu, n, m, 3000, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and kv.device_error() == 0


@pytest.mark.parametrize("rows,W", [(6, 5), (1500, 24)])
def test_update_and_compact_captured_and_replayed(hra, rows, W):
    """One captured step of forks, reservations and a compaction, replayed with other parents and rooms each time."""
    P = 16
    rng = random.Random(rows)
    c = random_rows(rows, W, P, rows * W, 31)
    kv = gpu(hra, c)
    parents, room = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    kv.update(torch.arange(rows, dtype=torch.int32, device="cuda"), out=kv.empty_pages())     # the workspace
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kv.update(parents, room)
        kv.compact()
    for _ in range(4):
        p = [rng.choice([b, rng.randrange(rows), -1]) for b in range(rows)]
        lens = c["lens"].tolist()
        m = [min(rng.choice([0, 1, P]), W * P - lens[x]) if x >= 0 else 0 for x in p]
        parents.copy_(i32(p))
        room.copy_(i32(m))
        graph.replay()
        for f, args in ((R.update, (p, m)), (R.compact, ())):
            want = f(c, *args)
            codes, scales = R.move(c, want[3])
            c.update(table=want[0], lens=want[1], refs=want[2], codes=codes, scales=scales)
        same(kv, c)
        assert torch.equal(kv.refs.cpu(), c["refs"])
    assert kv.device_error() == 0
