"""What a call over the paged 8-bit cache reads (Kv8Reach) without a GPU: refusals, workspace sizes, the index arithmetic of its
kernels, and the plain forms the GPU tests compare with."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_kv8 import FAKE, ROOT, _cache, _empty, hra  # noqa: F401


def reach(hra, **kw):  # noqa: F811
    f = dict(group_cu=None, prefix=None, groups=0, max_prefix=0, max_own=0, window=0, sinks=0)
    f.update(kw)
    return hra.HraKv8Reach(*[f[n] for n, _ in hra.HraKv8Reach._fields_])


GROUPS = dict(group_cu=FAKE, prefix=FAKE, groups=2, max_prefix=32, max_own=8)
BAD = [(dict(window=-1), -1), (dict(sinks=-1, window=4), -1), (dict(sinks=1), -1), (dict(window=(1 << 30) + 1), -4),
       (dict(window=1, sinks=(1 << 30) + 1), -4), (dict(groups=-1), -1), (dict(GROUPS, group_cu=None), -1),
       (dict(GROUPS, prefix=None), -1), (dict(GROUPS, group_cu=FAKE + 2), -1), (dict(GROUPS, prefix=FAKE + 1), -1),
       (dict(GROUPS, groups=5), -1), (dict(GROUPS, max_prefix=-1), -1), (dict(GROUPS, max_own=-1), -1),
       (dict(GROUPS, window=3), -2), (dict(GROUPS, groups=1025), -2)]


def _attend(hra, cache, r, total=3, ws_bytes=1 << 40, ws=0x8000000, **kw):  # noqa: F811
    f = dict(layer=0, q=FAKE, stride=256, nq=4, scale=0.0, cu=FAKE, kv_len=FAKE, batch=4, max_new=2, max_len=40, out=0x40000)
    f.update(kw)
    return hra.lib().hra_kv8_attention_reach(ctypes.byref(cache), f["layer"], f["q"], f["stride"], f["nq"], f["scale"], f["cu"],
                                             f["kv_len"], f["batch"], total, f["max_new"], f["max_len"],
                                             ctypes.byref(r) if r is not None else None, f["out"], ws, ws_bytes, None)


@pytest.mark.parametrize("bad,rc", BAD)
def test_bad_reaches_are_refused(hra, bad, rc):  # noqa: F811
    L, c, r = hra.lib(), _cache(hra), reach(hra, **bad)
    assert _attend(hra, c, r) == rc
    assert L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), 4, 3, 4, 2, 40, ctypes.byref(r)) == 0
    if bad.get("groups", 0) == 0:
        assert L.hra_kv8_update_reach(ctypes.byref(c), FAKE, FAKE, ctypes.byref(r), 0x20000, 0x30000, 0x40000, 0x50000, 1 << 40,
                                      None) == rc


def test_other_refusals_are_those_of_the_calls_without(hra):  # noqa: F811
    c, r = _cache(hra), reach(hra, window=8, sinks=2)
    for kw, rc in ((dict(layer=2), -1), (dict(q=None), -1), (dict(nq=3), -2), (dict(batch=5), -1), (dict(max_new=4), -1),
                   (dict(max_len=65), -4), (dict(out=None), -1), (dict(ws=None), -1), (dict(ws_bytes=0), -3)):
        assert _attend(hra, c, r, **kw) == rc and _attend(hra, c, None, **kw) == rc, kw
    assert _attend(hra, c, r, total=0, max_new=0, q=None, out=None) == 0
    # pages are dropped by a window alone
    assert hra.lib().hra_kv8_update_reach(ctypes.byref(c), FAKE, FAKE, ctypes.byref(reach(hra, **GROUPS)), 0x20000, 0x30000,
                                          0x40000, 0x50000, 1 << 40, None) == -1


def test_group_arrays_inside_what_the_call_writes_are_refused(hra):  # noqa: F811
    L, c = hra.lib(), _cache(hra)
    r = reach(hra, **dict(GROUPS, group_cu=0x100000, prefix=0x200000))
    need = L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), 4, 3, 4, 2, 40, ctypes.byref(r))
    for kw in (dict(ws=0x100000 - 16), dict(ws=0x200000), dict(out=0x100000), dict(out=0x200000 - 16)):
        assert _attend(hra, c, r, ws_bytes=need, **kw) == -1, kw


def test_wrapper_refusals(hra):  # noqa: F811
    z = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(window=-1), dict(sinks=2), dict(window=(1 << 30) + 1), dict(groups=z), dict(prefix=z[:2]), dict(max_own=3),
               dict(groups=z, prefix=z[:2]), dict(groups=z, prefix=z), dict(groups=z, prefix=z[:2], window=4),
               dict(groups=z, prefix=z[:2], max_prefix=-1)):
        with pytest.raises(hra.HraError):
            hra.Kv8Reach(**kw)
    assert hra.Kv8Reach(window=5, sinks=1).struct.window == 5
    assert hra.Kv8Reach().struct.window == 0
    with pytest.raises(hra.HraError):
        hra._reach(hra.Kv8Reach(window=5), torch.zeros(1))        # the bf16 cache has none
    with pytest.raises(hra.HraError):
        hra._reach((5, 1), torch.zeros(1))
    assert hra._reach(None, torch.zeros(1)) is None


def test_workspaces_never_fall_when_a_call_grows(hra):  # noqa: F811
    c = _cache(hra, rows=4096, max_pages=4096)
    L = hra.lib()

    def size(batch, total, nq, max_new, max_len, groups, max_prefix, max_own):
        r = reach(hra, group_cu=FAKE if groups else None, prefix=FAKE if groups else None, groups=groups, max_prefix=max_prefix,
                  max_own=max_own)
        return L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), batch, total, nq, max_new, max_len, ctypes.byref(r))

    grow = [[2, 5, 600, 4096], [5, 100, 200000], [2, 8, 32], [1, 3, 9, 100], [0, 513, 60000], [0, 1, 2], [0, 15, 16, 9000, 1 << 30],
            [0, 200, 1 << 30]]
    rng = random.Random(2)
    seen = 0
    for _ in range(4000):
        at = [rng.randrange(len(g)) for g in grow]
        args = [g[i] for g, i in zip(grow, at)]
        if args[3] > args[1]:
            continue
        n = size(*args)
        assert n > 0, args
        for k in range(len(grow)):
            if at[k] + 1 < len(grow[k]):
                more = args[:k] + [grow[k][at[k] + 1]] + args[k + 1:]
                if more[3] <= more[1]:
                    assert size(*more) >= n, (args, more)
                    seen += 1
        # a window alone needs what the call without one does
        w = reach(hra, window=7)
        assert L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), *args[:5], ctypes.byref(w)) == \
            L.hra_kv8_attention_workspace_size(ctypes.byref(c), *args[:5])
    assert seen > 1000


def test_prompts_need_no_room_for_what_they_do_not_share(hra):  # noqa: F811
    """Prompts too long to share a prefix: the scratch is that of as many rows with as many tokens as share one at most."""
    c = _cache(hra, rows=64, max_pages=4096)
    L = hra.lib()
    for total in (2000, 16384, 1 << 20):
        r = reach(hra, **dict(GROUPS, max_prefix=4096, max_own=4096))
        with_groups = L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), 8, total, 4, 2000, 8192, ctypes.byref(r))
        without = L.hra_kv8_attention_workspace_size(ctypes.byref(c), 8, total, 4, 2000, 8192)
        assert 0 < with_groups - without < 64 << 20, total


HARNESS = r"""
#include <cstdio>
#include <algorithm>
#include <vector>
#include "kv8.cuh"
using namespace hra;
int main() {
    // the units of a window's tokens: every position that some token from `first` on sees lies in one, each once, in order, and
    // every unit up to the last token's holds such a position
    for (int per : {16, 64}) for (int window : {0, 1, 2, 15, 16, 17, 63, 64, 65, 200, 1 << 30})
        for (int sinks : {0, 1, 15, 16, 17, 64, 100, 1 << 30}) for (int first = -3; first < 300; ++first) {
            if (window == 0 && sinks) continue;
            const int n = 3, keys = std::max(0, first + n);
            const Kv8Skip s = kv8_skip(first, window, sinks, per);
            const int all = (keys + per - 1) / per, units = std::max(all, 1) - s.by;
            if (s.from < 0 || s.by < 0 || units < 1) { std::printf("skip %d %d %d %d\n", per, window, sinks, first); return 1; }
            std::vector<int> have(all + 1, 0);
            int last = -1;
            for (int i = 0; i < units; ++i) {
                const int u = kv8_unit_at(s, i);
                if (u <= last || u > all) { std::printf("order %d %d %d %d\n", per, window, sinks, first); return 1; }
                last = u;
                have[u] = 1;
            }
            for (int u = 0; u < all; ++u) {
                bool seen = false;
                for (int j = u * per; j < std::min(keys, (u + 1) * per); ++j)
                    for (int p = std::max(first, 0); p < keys; ++p)
                        seen |= j <= p && (window == 0 || j > p - window || j < sinks);
                if (seen != (have[u] != 0) && first >= 0) { std::printf("seen %d %d %d %d %d\n", per, window, sinks, first, u); return 1; }
            }
        }
    // a row's own positions: the parts' units cover the blocks behind the prefix once
    for (int kv_len : {0, 1, 16, 63, 64, 65, 200, 1000, 5000}) for (int n : {0, 1, 3, 20}) for (int tokens : {1, 2, 8})
        for (int most : {1, 3, 64}) for (int prefix : {0, 16, 64, 160}) for (int splits : {1, 2, 8}) for (int least : {1, 2}) {
            if (prefix > std::max(0, kv_len - n)) continue;
            int got = 0;
            for (int t = 0; t * tokens < std::max(1, std::min(n, most)); ++t) {
                const Kv8Own o = kv8_own(kv_len, n, t, tokens, most, prefix, splits, least);
                if (o.tokens < 0 || o.tokens > tokens || o.t0 != t * tokens) { std::printf("tokens\n"); return 1; }
                got += o.tokens;
                if (o.parts < 1 || o.parts > splits || o.per < 1) { std::printf("parts %d %d\n", o.parts, splits); return 1; }
                const int end = std::max(0, kv_len - n + o.t0 + o.tokens);
                if (o.keys != end || o.blocks != std::max(0, (end + 15) / 16 - prefix / 16)) { std::printf("blocks\n"); return 1; }
                const int units = std::max(1, (o.blocks + 7) / 8);
                if (o.parts * o.per < units || (o.parts - 1) * o.per >= units) { std::printf("cover\n"); return 1; }
            }
            if (got != std::min(n, most)) { std::printf("all tokens %d %d\n", got, n); return 1; }
        }
    for (int len : {0, 5, 1 << 30}) for (int w : {0, 1, 1 << 30}) for (int s : {0, 1 << 30}) {
        const int m = kv8_most_seen(len, w, s, 100);
        if (m < 0 || m > len || (w == 0 && m != len)) { std::printf("most\n"); return 1; }
    }
    std::printf("ok\n");
    return 0;
}
"""


def run_harness(tmp_path, text):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src = tmp_path / "h.cpp"
    src.write_text(text)
    exe = tmp_path / "h"
    inc = os.path.join(ROOT, "qwen3_prefill_delayed_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", inc,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


def test_index_arithmetic(tmp_path):
    run_harness(tmp_path, HARNESS)


DIVISIONS = r"""
#include <cstdio>
#include "kv8.cuh"
using namespace hra;
int main() {
    const int ends[] = {1, 2, 3, 7, 8, 100, 1023, 1024, 1025, 65535, (1 << 30) - 1, 1 << 30};
    for (int d : ends) {
        const Kv8Div by = kv8_div(d);
        auto right = [&](long long i) { return i < 0 || i > 0x7FFFFFFF || kv8_over(by, (int)i) == (int)i / d; };
        for (long long i = 0; i < 5000; ++i)
            if (!right(i) || !right(0x7FFFFFFFLL - i)) return printf("%lld / %d\n", i, d), 1;
        for (long long q = 0x7FFFFFFFLL / d; q > 0; q = q * 3 / 4)
            for (int e = -1; e <= 1; ++e)
                if (!right(q * d + e)) return printf("%lld / %d\n", q * d + e, d), 1;
    }
    for (int d = 1; d <= 1024; ++d)
        for (long long i = 0; i < 0x80000000LL; i += 104729)
            if (kv8_over(kv8_div(d), (int)i) != (int)i / d) return printf("%lld / %d\n", i, d), 1;
    puts("ok");
    return 0;
}
"""


def test_divisions_without_one(tmp_path):
    run_harness(tmp_path, DIVISIONS)


# ---- the plain forms themselves

def filled(lens, rows_wide, H=1, P=16, D=64, seed=0):
    c = _empty(1, sum(-(-n // P) for n in lens) + 1, H, P, D, len(lens), rows_wide)
    g = torch.Generator().manual_seed(seed)
    page = 0
    for b, n in enumerate(lens):
        for i in range(-(-n // P)):
            c["table"][b, i] = page
            page += 1
        x = torch.randn(n, H, D, generator=g).to(torch.bfloat16)
        R.append(c, 0, x, -2 * x, [0] * (b + 1) + [n] * (len(lens) - b), [0] * len(lens))
    return c


def test_reference_window():
    lens = [40, 7]
    c = filled(lens, 4)
    q = torch.randn(8, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cu = [0, 5, 8]
    # a window of everything is none
    a, _ = R.attend(c, 0, q, cu, lens)
    for window, sinks in ((40, 0), (1, 1000), (1000, 3)):
        assert torch.allclose(a, W.attend(c, 0, q, cu, lens, window, sinks)[0], atol=1e-12)
    # a window of one position returns its V
    v = R.values(c, 0, 0, 40)[0][1]
    o, _ = W.attend(c, 0, q, cu, lens, 1, 0)
    assert torch.allclose(o[:5], v[35:40].expand(5, 1, 64).reshape(5, 1, 64).repeat(1, 2, 1), atol=1e-12)
    # what lies behind the window changes nothing, and a sink does
    w1, _ = W.attend(c, 0, q, cu, lens, 10, 2)
    d = {k: x.clone() for k, x in c.items()}
    d["codes"][0, 0, :, :, 2:16] ^= 1
    assert torch.equal(w1[:5], W.attend(d, 0, q, cu, lens, 10, 2)[0][:5])
    d["codes"][0, 0, :, :, 1] ^= 1
    assert not torch.equal(w1[:5], W.attend(d, 0, q, cu, lens, 10, 2)[0][:5])


def test_reference_update_drops_what_no_later_token_sees():
    c = _empty(1, 12, 1, 16, 64, 2, 8)
    c["table"][0, :6] = torch.tensor([7, 3, 9, 1, 5, 8])
    c["lens"][0] = 90
    table, lens, refs, moves = W.update(c, [0, 0], [0, 10], 40, 17)
    # page 2 holds 32 .. 47, and position 90 sees from 51 on; page 1 holds the last sink
    assert table.tolist() == [[7, 3, -1, 1, 5, 8, -1, -1], [7, 3, -1, 1, 5, 0, 2, -1]]
    assert moves == [(8, 0)] and lens.tolist() == [90, 90] and int(refs.sum()) == 11
    for n in range(0, 200):
        for i in range(12):
            sees = any(j > p - 40 or j < 17 for p in range(n, n + 60) for j in range(i * 16, min(i * 16 + 16, p + 1)))
            if (i + 1) * 16 <= n:
                assert sees == (not W.gone(n, 16, 40, 17, i))
