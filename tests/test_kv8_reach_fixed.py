"""A Kv8Reach keeps what its calls read: its attributes cannot be replaced under the struct that holds their values and addresses."""
import pytest
import torch

from test_kv8 import hra  # noqa: F401


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
