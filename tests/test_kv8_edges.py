"""The paged 8-bit cache without a GPU: calls that its entry points have to refuse, and arithmetic of its kernels, beyond
tests/test_kv8.py."""
import ctypes

import pytest

from test_kv8 import FAKE, _append, _attend, _cache, hra  # noqa: F401  (hra: the fixture)

LENS = 0x40000


@pytest.mark.parametrize("kw", [dict(start=LENS), dict(start=LENS + 4), dict(start=LENS - 4), dict(start=LENS + 12), dict(cu=LENS),
                                dict(cu=LENS - 8), dict(cu=LENS + 12)])
def test_append_refuses_start_and_cu_inside_lens(hra, kw):  # noqa: F811
    """The call writes lens while other CTAs of the row still read start and cu."""
    c = _cache(hra, lens=LENS)                       # four rows: 16 bytes; start 8 bytes, cu 12
    assert _append(hra, c, **{**dict(cu=FAKE, start=FAKE), **kw}) == -1


RING = r"""
#include <cstdio>
#include "kv8.cuh"
int main() {   // a warp's turns: stages requested and not yet taken, at the wait of every turn
    for (int stages = 2; stages < 5; ++stages) for (int step = 1; step < 12; step += 5) for (int blk0 = 0; blk0 < 9; ++blk0)
        for (int blk1 = 0; blk1 < 60; ++blk1) {
            int ahead = blk0, under_way = 0;
            auto request = [&] { if (ahead < blk1) ++under_way; ahead += step; };
            for (int s = 0; s < stages - 1; ++s) request();
            for (int blk = blk0; blk < blk1; blk += step) {
                request();
                if (under_way != hra::kv8_turns_left(blk, blk1, step, stages)) { std::printf("%d %d\n", blk, blk1); return 1; }
                --under_way;
            }
            if (under_way != 0 || hra::kv8_turns_left(blk1, blk1, step, stages) != 0) return 2;
        }
    return 0;
}
"""


def test_a_ring_knows_its_copies_under_way(tmp_path):
    """What the single-token kernel waits for before it gives up."""
    import os
    import shutil
    import subprocess

    from test_kv8 import ROOT
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    (tmp_path / "r.cpp").write_text(RING)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "qwen3_prefill_delayed_gb300", "csrc"),
                    str(tmp_path / "r.cpp"), "-o", str(tmp_path / "r")], check=True)
    r = subprocess.run([str(tmp_path / "r")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_page_calls_refuse_parents_and_room_inside_the_workspace(hra):  # noqa: F811
    L = hra.lib()
    c = _cache(hra, page_table=0x10000, lens=0x11000, refs=0x12000)
    need = L.hra_kv8_pages_workspace_size(ctypes.byref(c))
    ws = 0x50000
    for parents, room in ((ws, FAKE), (FAKE, ws + 4), (ws - 4, None), (None, ws + need - 4)):
        assert L.hra_kv8_update(ctypes.byref(c), parents, room, 0x20000, 0x30000, 0x40000, ws, need, None) == -1


def test_a_path_without_the_8_bit_cache_says_so(hra):  # noqa: F811
    """FP8 and NVFP4 prefill take the bf16 tensor alone, and check their cache here."""
    from types import SimpleNamespace
    paged = hra.Kv8Cache.__new__(hra.Kv8Cache)
    with pytest.raises(hra.HraError):
        hra.Backbone.kv(SimpleNamespace(d=None), paged)


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    """The build of one small source and a binding, in a folder of its own."""
    from qwen3_prefill_delayed_gb300 import _build
    try:
        _build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src = tmp_path / "binding.cpp"
    src.write_text("extern \"C\" int answer() { return 42; }\n")
    for name, value in (("SOURCES", ["noalloc.cu"]), ("BUILD", str(tmp_path / "build")), ("LIB", str(tmp_path / "libhra.so")),
                        ("BINDING", str(tmp_path / "binding.so")), ("BINDING_SRC", str(src))):
        monkeypatch.setattr(_build, name, value)
    return _build, src, tmp_path


@pytest.mark.parametrize("why", ["source", "compiler", "torch"])
def test_the_library_is_built_where_the_binding_cannot_be(small_build, monkeypatch, why):
    build, src, tmp = small_build
    if why == "source":
        src.write_text("#error no headers\n")
    elif why == "compiler":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda n: str(tmp / "no-such-compiler") if n == "g++" else which(n))
    else:
        def missing(out):
            raise ImportError("No module named 'torch'")
        monkeypatch.setattr(build, "_binding_command", missing)
    with pytest.raises(RuntimeError, match="8-bit cache"):
        build.build()
    assert (tmp / "libhra.so").exists() and not (tmp / "binding.so").exists()


def test_the_binding_follows_torch(small_build, monkeypatch):
    import torch
    build, _, tmp = small_build
    build.build()
    first = (tmp / "binding.so").stat().st_mtime_ns
    build.build()
    assert (tmp / "binding.so").stat().st_mtime_ns == first
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert (tmp / "binding.so").stat().st_mtime_ns != first


def test_what_two_e4m3_values_keep_of_a_query():
    """q as e4m3(q / s) + e4m3(the rest) under the largest element's scale, for every bf16 magnitude and every mantissa of the
    largest: exact from 2^-9.8 of it on, below off by 2^-17.8 of it at most."""
    import torch

    import kv8_ref as R
    e4m3 = lambda x: x.float().to(torch.float8_e4m3fn).double()  # noqa: E731
    every = (torch.arange(0x7F80, dtype=torch.int32) << 16).view(torch.float32).double()
    worst = 0.0
    for top in [m * 2.0 ** e for m in range(128, 256) for e in (-90, -7, 60)] + [2.0 ** -126, 255 * 2.0 ** -133]:
        s = R.scale_of(top)
        x = every[every <= top]
        v = (x / s).half()                                   # as the kernel forms it
        hi = e4m3(v)
        lo = e4m3(v - hi.half())
        off = ((hi + lo) * s - x).abs() / top
        assert float(off[x >= top * 2.0 ** -9.8].max()) == 0.0
        worst = max(worst, float(off.max()))
    assert 2.0 ** -18 < worst <= 2.0 ** -17.8


@pytest.mark.parametrize("off", [0, 512 * 2 - 16, -(3 * 256 * 2 - 16)])
def test_attention_refuses_an_output_over_its_queries(hra, off):  # noqa: F811
    # three rows: of q 512 elements apart and 256 long, of the output 256
    assert _attend(hra, _cache(hra), q=0x100000, stride=512, out=0x100000 + off) == -1
