"""The paged 8-bit cache without a GPU: calls that its entry points have to refuse, and arithmetic of its kernels, beyond
tests/test_kv8.py."""
import ctypes

import pytest

from test_kv8 import FAKE, _append, _cache, hra  # noqa: F401  (hra: the fixture)

LENS = 0x40000


@pytest.mark.parametrize("kw", [dict(start=LENS), dict(start=LENS + 4), dict(start=LENS - 4), dict(start=LENS + 12), dict(cu=LENS),
                                dict(cu=LENS - 8), dict(cu=LENS + 12)])
def test_append_refuses_start_and_cu_inside_lens(hra, kw):  # noqa: F811
    """The call writes lens while other CTAs of the row still read start and cu."""
    c = _cache(hra, lens=LENS)                       # four rows: 16 bytes; start 8 bytes, cu 12
    assert _append(hra, c, **{**dict(cu=FAKE, start=FAKE), **kw}) == -1
