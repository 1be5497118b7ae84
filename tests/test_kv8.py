"""The paged 8-bit cache without a GPU: refusals of its entry points, the index arithmetic of its kernels against the
buffers' sizes (bad page numbers and positions among it), and the plain forms the GPU tests compare with."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

import kv8_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hra():
    import qwen3_prefill_delayed_gb300 as h
    if not os.path.exists(h.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("no nvcc to build the library")
        from qwen3_prefill_delayed_gb300 import _build
        _build.build()
    h.lib()
    return h


FAKE = 0x10000   # aligned, never dereferenced: every call below is refused or has nothing to do


def _cache(hra, **kw):
    f = dict(codes=FAKE, scales=FAKE, page_table=FAKE, lens=FAKE, refs=FAKE, errors=FAKE, n_layers=2, n_pages=8,
             n_kv_heads=2, head_dim=64, page_size=16, rows=4, max_pages=4)
    f.update(kw)
    return hra.HraKv8Cache(*[f[n] for n, _ in hra.HraKv8Cache._fields_])


BAD_CACHE = [(dict(codes=None), -1), (dict(codes=FAKE + 8), -1), (dict(scales=None), -1), (dict(scales=FAKE + 4), -1),
             (dict(page_table=None), -1), (dict(page_table=FAKE + 2), -1), (dict(lens=None), -1), (dict(errors=None), -1),
             (dict(refs=FAKE + 1), -1), (dict(n_layers=0), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1),
             (dict(rows=0), -1), (dict(max_pages=-1), -1), (dict(head_dim=96), -2), (dict(page_size=8), -2),
             (dict(page_size=48), -2), (dict(page_size=256), -2), (dict(n_kv_heads=1025), -2), (dict(rows=65536), -2),
             (dict(max_pages=1 << 27), -2), (dict(n_pages=(1 << 28) + 1), -2), (dict(n_pages=1 << 25), -2),
             (dict(rows=65535, max_pages=20000), -2)]


def _append(hra, cache, layer=0, k=FAKE, v=FAKE, stride=128, cu=FAKE, start=FAKE, batch=2, total=3, max_new=2):
    return hra.lib().hra_kv8_append(ctypes.byref(cache) if cache is not None else None, layer, k, v, stride, cu, start,
                                    batch, total, max_new, None)


def _attend(hra, cache, layer=0, q=FAKE, stride=256, nq=4, scale=0.0, cu=FAKE, kv_len=FAKE, batch=2, total=3, max_new=2,
            max_len=40, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return hra.lib().hra_kv8_attention(ctypes.byref(cache) if cache is not None else None, layer, q, stride, nq, scale,
                                       cu, kv_len, batch, total, max_new, max_len, out, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,rc", BAD_CACHE)
def test_bad_cache_refused(hra, bad, rc):
    c = _cache(hra, **bad)
    L = hra.lib()
    assert _append(hra, c) == rc
    assert _attend(hra, c) == rc
    assert L.hra_kv8_update(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == rc
    assert L.hra_kv8_compact(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == rc
    assert L.hra_kv8_attention_workspace_size(ctypes.byref(c), 2, 3, 4, 2, 40) == 0
    assert L.hra_kv8_pages_workspace_size(ctypes.byref(c)) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(layer=-1), -1), (dict(layer=2), -1), (dict(k=None), -1), (dict(v=FAKE + 8), -1), (dict(stride=120), -1),
    (dict(stride=132), -1), (dict(cu=None), -1), (dict(start=FAKE + 2), -1), (dict(batch=0), -1), (dict(batch=5), -1),
    (dict(total=-1), -1), (dict(max_new=0), -1), (dict(max_new=4), -1), (dict(max_new=-1), -1),
    (dict(total=(1 << 30) + 1), -4)])
def test_append_refusals(hra, kw, rc):
    assert _append(hra, _cache(hra), **kw) == rc


def test_nothing_to_do(hra):
    # no rows at all: nothing is enqueued, and the row tensors may be null
    assert _append(hra, _cache(hra), k=None, v=None, total=0, max_new=0) == 0
    assert _attend(hra, _cache(hra), q=None, out=None, total=0, max_new=0) == 0
    assert _append(hra, None) == -1 and _attend(hra, None) == -1


@pytest.mark.parametrize("kw,rc", [
    (dict(layer=2), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(stride=248), -1), (dict(stride=260), -1),
    (dict(nq=3), -2), (dict(nq=0), -2), (dict(nq=34, stride=34 * 64), -2), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(scale=-1.0), -1), (dict(cu=None), -1), (dict(kv_len=None), -1),
    (dict(batch=5), -1), (dict(max_new=4), -1), (dict(max_len=-1), -4), (dict(max_len=65), -4), (dict(out=None), -1),
    (dict(out=FAKE + 4), -1), (dict(ws=None), -1), (dict(ws_bytes=0), -3)])
def test_attention_refusals(hra, kw, rc):
    assert _attend(hra, _cache(hra), **kw) == rc


def test_pages_refusals(hra):
    L = hra.lib()
    c = _cache(hra)
    need = L.hra_kv8_pages_workspace_size(ctypes.byref(c))
    assert need >= 4 * (4 * 4 + 3 * 4 + 2 * 8)
    table, lens, refs, ws = 0x20000, 0x30000, 0x40000, 0x50000

    def up(c=c, parents=FAKE, room=FAKE, table=table, lens=lens, refs=refs, ws=ws, n=need):
        return L.hra_kv8_update(ctypes.byref(c), parents, room, table, lens, refs, ws, n, None)

    def co(c=c, table=table, lens=lens, refs=refs, ws=ws, n=need):
        return L.hra_kv8_compact(ctypes.byref(c), table, lens, refs, ws, n, None)

    for f in (up, co):
        assert f(n=need - 1) == -3
        assert f(table=None) == -1 and f(lens=FAKE + 1) == -1 and f(refs=None) == -1 and f(ws=FAKE + 4) == -1
        assert f(c=_cache(hra, refs=None)) == -1
        # outputs that overlap the inputs without being them
        assert f(table=FAKE + 4) == -1 and f(lens=FAKE + 4) == -1 and f(refs=FAKE - 4) == -1
    assert up(parents=FAKE + 2) == -1 and up(room=FAKE + 1) == -1


def test_wrapper_refuses_cpu_tensors(hra):
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(hra.HraError):
        hra.Kv8Cache(z(1, 2, 2, 1, 16, 64, dt=torch.uint8), z(1, 2, 2, 1, 1, dt=torch.float32), z(1, 2), z(1), z(2))
    with pytest.raises(hra.HraError):
        hra.Kv8Cache(z(1, 2, 2, 1, 16, 64, dt=torch.uint8), z(1, 2, 2, 1, 2, dt=torch.float32), z(1, 2), z(1), z(2))


HARNESS = r"""
#include <cstdio>
#include <cstring>
#include <cstdlib>
#include <vector>
#include "kv8.cuh"
using namespace hra;
int main() {
    long long n = 0;
    for (int hd : {64, 128}) for (int ps : {16, 32, 64, 128}) for (int kv : {1, 3, 8}) for (int pages : {1, 5, 70000}) {
        Kv8View c{};
        c.n_pages = pages; c.n_kv = kv; c.head_dim = hd; c.page_size = ps; c.max_pages = 4;
        for (c.page_shift = 0; (1 << c.page_shift) < ps; ++c.page_shift) {}
        int32_t table[8] = {0, pages - 1, pages, -1, -2147483647 - 1, 2147483647, pages / 2, pages + 1};
        c.table = table;
        const long long codes = 2LL * pages * kv * ps * hd, scales = 2LL * pages * kv * (ps / 16);
        const int pos[] = {-2147483647 - 1, -1, 0, 1, 15, 16, ps - 1, ps, 2 * ps - 1, 2 * ps, 3 * ps, 4 * ps - 1, 4 * ps,
                           4 * ps + 1, 1 << 30, 2147483647};
        for (int row = 0; row < 2; ++row) for (int p : pos) {
            const int page = kv8_page_of(c, row, p);
            const bool in = p >= 0 && p < 4 * ps;
            const int want = in ? table[row * 4 + p / ps] : -1;
            const bool ok = want >= 0 && want < pages;
            if (page != (ok ? want : -1)) { std::printf("page %d %d %d\n", row, p, page); return 1; }
            if (page < 0) continue;
            for (int w = 0; w < 2; ++w) for (int h = 0; h < kv; ++h) {
                const int slot = p % ps;
                const long long a = kv8_code_at(c, page, w, h, slot), s = kv8_scale_at(c, page, w, h, slot);
                const long long base = (((long long)page * 2 + w) * kv + h);
                if (a != (base * ps + slot) * hd || a < 0 || a + hd > codes) { std::printf("code\n"); return 1; }
                if (s != base * (ps / 16) + slot / 16 || s < 0 || s >= scales) { std::printf("scale\n"); return 1; }
                ++n;
            }
        }
    }
    // packed rows never leave the tensor, whatever cu holds
    const int32_t cus[] = {-5, 0, 3, 7, 8, 9, 2147483647, -2147483647 - 1};
    for (int32_t x : cus) for (int32_t y : cus) {
        const int32_t cu[2] = {x, y};
        int lo, m;
        kv8_rows(cu, 0, 8, lo, m);
        if (lo < 0 || m < 0 || lo + m > 8) { std::printf("rows\n"); return 1; }
        if (x >= 0 && y >= x && y <= 8 && (lo != x || m != y - x)) { std::printf("rows value\n"); return 1; }
    }
    // every finite bf16 magnitude: the smallest power of two (>= 2^-126) that holds it
    for (uint32_t b = 0; b < 0x7F80; ++b) {
        const uint32_t bits = b << 16;
        float a, s;
        std::memcpy(&a, &bits, 4);
        const uint32_t sb = kv8_scale_bits(bits);
        std::memcpy(&s, &sb, 4);
        if ((sb & 0x7FFFFF) || sb == 0 || (double)a > 448.0 * s) { std::printf("scale bits %x\n", b); return 1; }
        if (sb > (1u << 23) && (double)a <= 448.0 * (s * 0.5)) { std::printf("scale bits %x not smallest\n", b); return 1; }
    }
    for (int k = 1; k < 200; ++k) for (int first = 0; first < 32; ++first) {
        const int blocks = (first + k - 1) / 16 - first / 16 + 1;
        if (blocks > kv8_max_blocks(k)) { std::printf("blocks\n"); return 1; }
    }
    std::printf("ok %lld\n", n);
    return 0;
}
"""


def test_index_arithmetic_stays_in_the_buffers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src = tmp_path / "h.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "h"
    inc = os.path.join(ROOT, "qwen3_prefill_delayed_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", inc,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


# ---- the plain forms themselves

def test_reference_codes_are_nearest():
    x = torch.cat([torch.linspace(-460, 460, 4001, dtype=torch.float64), R._POS, -R._POS, (R._POS[1:] + R._POS[:-1]) / 2]).float().double()
    c = R.e4m3_code(x)
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(c, want)
    assert int(R.e4m3_code(torch.tensor([float("nan")], dtype=torch.float64))[0]) & 127 == 127


def _empty(L, pages, H, P, D, rows, W):
    return {"codes": torch.zeros(L, pages, 2, H, P, D, dtype=torch.uint8),
            "scales": torch.zeros(L, pages, 2, H, P // 16), "table": torch.full((rows, W), -1, dtype=torch.int32),
            "lens": torch.zeros(rows, dtype=torch.int32), "refs": torch.zeros(pages, dtype=torch.int32)}


def test_reference_append_round_trip():
    g = torch.Generator().manual_seed(1)
    c = _empty(1, 3, 2, 16, 64, 1, 3)
    c["table"][0] = torch.tensor([2, 0, 1])
    x = torch.randn(40, 2, 64, generator=g).to(torch.bfloat16)
    R.append(c, 0, x, -x, [0, 40], [0])
    kv, there = R.values(c, 0, 0, 40)
    assert bool(there.all()) and int(c["lens"][0]) == 40
    # half a step of E4M3, or of its subnormals under the block's scale (at most 2^-9 * max / 224 there)
    assert float((kv[0] - x.double()).abs().max()) <= float(x.double().abs().max()) * 2.0 ** -4
    assert torch.equal(kv[0], -kv[1])
    # token by token: the same scales; the codes agree but for the second rounding of subnormals
    d = _empty(1, 3, 2, 16, 64, 1, 3)
    d["table"][0] = c["table"][0]
    for t in range(40):
        R.append(d, 0, x[t:t + 1], -x[t:t + 1], [0, 1], [t])
    assert torch.equal(c["scales"], d["scales"])
    kd, _ = R.values(d, 0, 0, 40)
    assert float((kd - kv).abs().max()) <= 2.0 ** -9 * float(c["scales"].max())


def test_reference_update_and_compact():
    c = _empty(1, 12, 1, 16, 64, 4, 4)
    c["table"][0, :2] = torch.tensor([5, 9])
    c["table"][1, :1] = torch.tensor([3])
    c["lens"][:2] = torch.tensor([20, 16])
    for p in (5, 9, 3):
        c["refs"][p] = 1
    table, lens, refs, moves = R.update(c, [0, 0, 1, -1], [1, 13, 0, 7])
    assert table.tolist() == [[5, 9, -1, -1], [5, 0, 1, -1], [3, -1, -1, -1], [-1] * 4]
    assert lens.tolist() == [20, 20, 16, 0] and moves == [(9, 0)]
    assert refs[5] == 2 and refs[9] == 1 and refs[0] == 1 and refs[1] == 1 and int(refs.sum()) == 6
    c.update(table=table, lens=lens, refs=refs)
    table, lens, refs, moves = R.compact(c)
    assert moves == [(5, 2), (9, 4)] and table.tolist()[1] == [2, 0, 1, -1] and table.tolist()[0] == [2, 4, -1, -1]
    assert refs.tolist() == [1, 1, 2, 1, 1] + [0] * 7
    assert R.update(c, None, [0, 0, 200, 0]) is None


def test_attention_workspace_never_falls_when_a_call_grows(hra):
    c = _cache(hra, rows=4096, max_pages=4096)
    size = lambda *a: hra.lib().hra_kv8_attention_workspace_size(ctypes.byref(c), *a)  # noqa: E731
    grow = [[1, 2, 600, 1024, 1025, 4096], [1, 100, 5000, 200000], [2, 4, 16, 32], [1, 2, 9, 100, 5000, 200000],
            [0, 100, 512, 513, 2048, 2049, 60000]]

    def walk(i, args):
        if i == len(grow):
            return {tuple(args): size(*args)} if args[3] <= args[1] else {}
        out = {}
        for v in grow[i]:
            out.update(walk(i + 1, args + [v]))
        return out

    sizes = walk(0, [])
    assert all(n > 0 for n in sizes.values())
    for args, n in sizes.items():
        for i, values in enumerate(grow):
            j = values.index(args[i]) + 1
            more = args[:i] + (values[j],) + args[i + 1:] if j < len(values) else args
            assert more not in sizes or sizes[more] >= n, (args, more)


def test_page_outputs_that_overlap_are_refused(hra):
    L = hra.lib()
    c = _cache(hra, rows=4, max_pages=4, n_pages=4, page_table=0x10000, lens=0x11000, refs=0x12000)
    need = L.hra_kv8_pages_workspace_size(ctypes.byref(c))
    ok = dict(table=0x20000, lens=0x30000, refs=0x40000, ws=0x50000)
    for f in (lambda **k: L.hra_kv8_update(ctypes.byref(c), FAKE, FAKE, k["table"], k["lens"], k["refs"], k["ws"], need, None),
              lambda **k: L.hra_kv8_compact(ctypes.byref(c), k["table"], k["lens"], k["refs"], k["ws"], need, None)):
        for bad in (dict(refs=0x30000), dict(lens=0x20000 + 60), dict(lens=0x10000), dict(refs=0x11000), dict(table=0x12000),
                    dict(ws=0x20000), dict(ws=0x11000), dict(ws=0x40000 - 16), dict(table=0x10004)):
            assert f(**{**ok, **bad}) == -1, bad
