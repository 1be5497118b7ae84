"""A Kv8Reach keeps what its calls read: its attributes cannot be replaced under the struct that holds their values and addresses; and
workspaces sized for the largest call of a reach do for every smaller one."""
import ctypes
import gc
import weakref

import pytest
import torch

from test_abi import _dims
from test_kv8 import FAKE, _cache, hra  # noqa: F401


def refuses_changes(hra, r):  # noqa: F811
    before = bytes(r.struct)
    held = dict(r.__dict__)
    for name, value in (("window", 9), ("sinks", 3), ("groups", torch.zeros(2, dtype=torch.int32)),
                        ("prefix", torch.zeros(1, dtype=torch.int32)), ("groups", 5), ("struct", None), ("ref", None), ("at", 0)):
        if name in held:
            with pytest.raises(hra.HraError, match=name):
                setattr(r, name, value)
            with pytest.raises(hra.HraError, match=name):
                delattr(r, name)
    assert bytes(r.struct) == before and all(r.__dict__[k] is v for k, v in held.items())


def test_a_window_cannot_be_changed_under_its_struct(hra):  # noqa: F811
    r = hra.Kv8Reach(window=5, sinks=1)
    refuses_changes(hra, r)
    r.window = r.window                                   # nothing new
    assert r.struct.window == 5 and r.struct.sinks == 1


@pytest.mark.gpu
def test_groups_cannot_be_changed_under_their_struct(hra):  # noqa: F811
    g, p = torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([64], dtype=torch.int32).cuda()
    r = hra.Kv8Reach(groups=g, prefix=p, max_prefix=64)
    refuses_changes(hra, r)
    assert r.groups is g and r.prefix is p and (r.struct.group_cu, r.struct.prefix) == (g.data_ptr(), p.data_ptr())
    other = hra.Kv8Reach(groups=g, prefix=p.clone(), max_prefix=64)
    assert other.struct.prefix != r.struct.prefix


def test_workspaces_never_fall_with_more_heads_or_tokens(hra):  # noqa: F811
    """Every number of q heads a kv head, beside the other arguments that the tiles of a sequence depend on."""
    c, L = _cache(hra, rows=4096, max_pages=4096), hra.lib()

    def size(batch, total, heads, max_new, max_own, groups=1):
        r = hra.HraKv8Reach(FAKE, FAKE, groups, 9000, max_own, 0, 0)
        return L.hra_kv8_attention_reach_workspace_size(ctypes.byref(c), batch, total, 2 * heads, max_new, 60000, ctypes.byref(r))

    for batch, total in ((1, 70), (5, 70), (64, 2000), (4096, 9000)):
        for max_own in (0, 300, 9000):
            for most in [*range(1, 70), 100, 1000]:
                if most > total:
                    continue
                sizes = [size(batch, total, g, most, max_own) for g in range(1, 17)]
                assert all(sizes) and sizes == sorted(sizes), (batch, total, max_own, most)
            for g in range(1, 17):
                sizes = [size(batch, total, g, most, max_own) for most in range(1, 71)]
                assert sizes == sorted(sizes), (batch, total, max_own, g)
                sizes = [size(batch, total + i, g, 20, max_own) for i in range(0, 200, 7)]
                assert sizes == sorted(sizes), (batch, total, max_own, g)


def test_group_arrays_inside_what_a_frame_writes_are_refused(hra):  # noqa: F811
    """The codebook step's outputs, state and workspace too: they are written before the attention reads the groups."""
    L, d = hra.lib(), _dims(hra)
    layers = (hra.HraLayerWeights * d.n_layers)()
    for layer in layers:
        for f, _ in hra.HraLayerWeights._fields_:
            setattr(layer, f, FAKE)
    w = hra.HraWeights(FAKE, layers, FAKE)
    c = _cache(hra, n_layers=d.n_layers, n_kv_heads=d.n_kv_heads, head_dim=d.head_dim)
    at = {n: (i + 16) << 28 for i, n in enumerate(("state", "hidden", "pos", "codes", "next_emb", "done", "bws", "cws"))}
    size = {"state": 32, "hidden": 4 * d.hidden, "pos": 8, "codes": 8 * d.n_codebooks, "next_emb": 4 * d.hidden, "done": 8,
            "bws": 1 << 24, "cws": 1 << 24}

    def frame(group_cu, prefix):
        r = hra.HraKv8Reach(group_cu, prefix, 1, 32, 8, 0, 0)
        return L.hra_ar_frame_kv8_reach(ctypes.byref(d), ctypes.byref(w), FAKE, FAKE, at["state"], None, None, None, at["hidden"],
                                        at["pos"], 7, 2, ctypes.byref(c), ctypes.byref(r), at["codes"], at["next_emb"], at["done"],
                                        at["bws"], size["bws"], at["cws"], size["cws"], None)

    for name in at:
        for where in (at[name], at[name] + size[name] - 4, at[name] - 4):
            assert frame(where, 0x9000000) == -1, name
            if where >= at[name]:
                assert frame(0x9000000, where) == -1, name
    assert L.hra_launch_counter() == 0


def test_a_captured_loop_keeps_the_reach_that_it_reads(hra, monkeypatch):  # noqa: F811
    """Replays read the groups at the addresses that were captured, whatever the loop's reach is by then."""
    class Graph:
        def __enter__(self):
            return self

        def __exit__(self, *a):
            pass

    loop = hra.ARLoop.__new__(hra.ARLoop)
    loop.hidden, loop.B, loop.bb = torch.zeros(1), 1, type("B", (), {"d": _dims(hra)})
    loop.reach = hra.Kv8Reach(window=5)
    for name in ("Stream", "current_stream", "CUDAGraph", "graph"):
        monkeypatch.setattr(torch.cuda, name, lambda *a, **k: type("S", (Graph,), {"wait_stream": lambda *a: None})())
    monkeypatch.setattr(hra.ARLoop, "frame", lambda *a, **k: None)
    loop.capture(2)
    alive = weakref.ref(loop.reach)
    loop.reach = None
    gc.collect()
    assert alive() is not None
    loop.reach = hra.Kv8Reach(window=7)
    loop.capture(2)                                       # the next graph reads the next one
    gc.collect()
    assert alive() is None
