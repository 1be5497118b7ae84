"""Prompts of mixed lengths over the paged 8-bit cache: whole items or equal shares by the lengths that the call finds on the device,
against the plain 64-bit forms of kv8_ref and kv8_reach_ref; captured calls replayed with lengths that ask for the other; and steps of
many tokens behind prefixes that are and are not worth sharing."""
import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_gpu_kv8 import build, cu_of, gpu, hra, i32  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Call:
    """A call with a workspace of its own, whose list says at its head how many (query tile, sequence) pairs there are and whether
    they go in equal shares."""

    def __init__(self, hra, c, new, lens, G, window=0, max_len=None):  # noqa: F811
        self.hra, self.c, self.new, self.lens, self.window = hra, c, new, lens, window
        H, D = c["codes"].shape[3], c["codes"].shape[5]
        T = sum(new)
        self.q = torch.randn(T, H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16)
        self.kv, self.qg = gpu(hra, c), self.q.cuda()
        self.cu, self.kl = i32(cu_of(new)).cuda(), i32(lens).cuda()
        self.most = max_len or max(lens)
        self.reach = hra.Kv8Reach(window=window) if window else None
        need = self.kv.attention_workspace_size(len(new), T, H * G, max(new), self.most, self.reach)
        self.ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
        self.out = torch.empty_like(self.qg)

    def run(self):
        self.kv.attend(0, self.qg, self.cu, self.kl, max(self.new), self.most, out=self.out, workspace=self.ws, reach=self.reach)

    def check(self, new=None, lens=None):
        new, lens = new or self.new, lens or self.lens
        args = (self.c, 0, self.q, cu_of(new), lens)
        want, bound = W.attend(*args, self.window, 0, split=True) if self.window else R.attend(*args, split=True)
        got, n = self.out.cpu()[:sum(new)].double(), sum(new)
        assert float(((got - want[:n]).abs() - bound[:n]).max()) <= 0 and self.kv.device_error() == 0
        return got

    def shares(self):
        return int(self.ws[:8].view(torch.int32)[1])


# as many items as CTAs, all of one length or one sequence far longer; a few sequences among which one is long; few items after many
# positions, and short ones, whose bounds leave nothing open
CASES = [([20] * 38, [2500] * 38, 8, 4, 0), ([20] * 38, [3200] + [0] * 37, 8, 4, 1), ([64] * 9, [2500] + [7] * 8, 8, 4, 1),
         ([130], [5500], 1, 4, 1), ([20] * 38, [300] * 38, 8, 4, 0), ([40, 1, 33, 0, 2], [2000, 1900, 5, 40, 1999], 1, 16, 1),
         ([130, 64], [0, 2400], 2, 2, 1)]


@pytest.mark.parametrize("new,kept,H,G,shares", CASES)
def test_the_choice_follows_the_lengths(hra, new, kept, H, G, shares):  # noqa: F811
    lens = [a + b for a, b in zip(new, kept)]
    call = Call(hra, build(lens, H=H, D=64, P=64, seed=len(new)), new, lens, G)
    call.run()
    torch.cuda.synchronize()
    assert call.shares() == shares
    first = call.check()
    for _ in range(3):
        call.run()
        assert torch.equal(first, call.out.cpu().double())      # and nothing of it by chance


@pytest.mark.parametrize("H,G,D", [(2, 4, 128), (1, 3, 64), (5, 1, 64)])
@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("new,kept", [([90, 17, 50, 70], [0, 2000, 5, 300]), ([30] * 12, [2600] + [0] * 11),
                                      ([300, 20, 1], [1300, 10, 1999])])
def test_mixed_lengths(hra, H, G, D, window, new, kept):  # noqa: F811
    lens = [a + b for a, b in zip(new, kept)]
    call = Call(hra, build(lens, H=H, D=D, P=32, seed=sum(new)), new, lens, G, window)
    call.run()
    call.check()


@pytest.mark.parametrize("rows,shares", [(1100, 1), (2600, 0)])
def test_more_sequences_than_one_turn_of_the_list(hra, rows, shares):  # noqa: F811
    """More than 1024 sequences, and more pairs than are weighed; one long prompt among them."""
    new = [1 if b % 9 else 0 for b in range(rows)]
    new[rows - 40], new[3] = 40, 70
    lens = [n + (b % 5) for b, n in enumerate(new)]
    lens[rows - 40] += 3000
    call = Call(hra, build(lens, H=1, D=64, P=64, seed=rows), new, lens, 16)
    call.run()
    call.check()
    assert call.shares() == shares


def test_replays_choose_anew(hra):  # noqa: F811
    """One captured call, replayed with other lengths under its bounds: shares, whole items, and shares again."""
    new = [20] * 38
    long, even = [3220] + [20] * 37, [1720] * 38
    c = build([max(a, b) for a, b in zip(long, even)], H=8, D=64, P=64, seed=1)
    call = Call(hra, c, new, long, 4, max_len=3220)
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for lens, shares in ((long, 1), (even, 0), (long, 1)):
        call.kl.copy_(i32(lens))
        call.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert call.shares() == shares
        call.check(lens=lens)


@pytest.mark.parametrize("H,new,lens", [(2, [40, 10], [0, 0]), (2, [40, 10], [30, 0]), (2, [40, 10], [-5, 10]), (8, [20] * 38, [0] * 38),
                                        (8, [20] * 38, [30, -1] * 19), (8, [20, 0] * 19, [64, 0] * 19)])
def test_lengths_far_below_the_bound(hra, H, new, lens):  # noqa: F811
    """Bounds of a long call, of which little is left: rows with new tokens that hold fewer positions or none."""
    c = build([64] * len(new), H=H, D=64, P=16, seed=2, width=400)
    call = Call(hra, c, new, lens, 4, max_len=6400)
    call.run()
    torch.cuda.synchronize()
    want, bound = R.attend(c, 0, call.q, cu_of(new), lens, split=True)
    assert float(((call.out.cpu().double() - want).abs() - bound).max()) <= 0
    assert call.shares() == (len(new) == 2)


@pytest.mark.parametrize("n,prefix,kernels", [(16, 1024, 0), (8, 1024, 0), (4, 1024, 4), (8, 4096, 4)])
def test_steps_of_many_tokens_share_long_prefixes_alone(hra, n, prefix, kernels):  # noqa: F811
    """Many tokens behind a prefix that is not long for them: the call with groups is the one without, launches among it."""
    H, G, D, P, rows = 8, 4, 128, 64, 64
    c = build([prefix], H=H, D=D, P=P, seed=n, spare=rows + 1)
    used = [int(x) for x in c["table"][0]]
    free = [x for x in range(c["refs"].numel()) if x not in used]
    c["codes"][0, free] = c["codes"][0, used[0]].clone()
    c["scales"][0, free] = c["scales"][0, used[0]].clone()
    c["table"] = torch.tensor([used + [free[b]] for b in range(rows)], dtype=torch.int32)
    c["lens"] = i32([prefix + n] * rows)
    kv = gpu(hra, c)
    q = torch.randn(rows * n, H * G, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    args = (0, q, i32(range(0, rows * n + 1, n)).cuda(), i32([prefix + n] * rows).cuda(), n, prefix + n)
    reach = hra.Kv8Reach(groups=i32([0, rows]).cuda(), prefix=i32([prefix]).cuda(), max_prefix=prefix, max_own=n)
    before = hra.hra_launch_counter()
    plain = kv.attend(*args)
    middle = hra.hra_launch_counter()
    got = kv.attend(*args, reach=reach)
    after = hra.hra_launch_counter()
    if kernels:
        assert after - middle == kernels
        want, bound = R.attend({**c, "table": c["table"][-1:]}, 0, q.cpu()[-n:], [0, n], [prefix + n], split=True)   # the last row
        assert float(((got.cpu()[-n:].double() - want).abs() - bound).max()) <= 0
    else:
        assert after - middle == middle - before and torch.equal(got, plain)
