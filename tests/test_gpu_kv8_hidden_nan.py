"""Not-a-numbers that a token does not see, in prompts over the paged 8-bit cache: one V element at a time in tiles of every
fill, against the plain 64-bit forms of kv8_ref and kv8_reach_ref."""
import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_gpu_kv8 import build, cu_of, gpu, hra, i32  # noqa: F401

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
