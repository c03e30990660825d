"""Calls whose launch would pass 2^32 threads, the most a grid takes in one dimension, are refused on the host."""
import ctypes

import pytest

from tests.test_abi import E_SHAPE, E_WS, FAKE
from tests.test_kv_options import option
from tests.test_serving_abi import cache, q, seqs  # noqa: F401


@pytest.mark.parametrize("heads,new,kernel", [(64, 1, 0), (64, 1, 1), (64, 40, 2), (16, 17, 1)])
def test_attention(q, heads, new, kernel):  # noqa: F811
    batch = 1 << 20
    c, s = cache(q, heads=heads, dim=64), seqs(q, batch=batch, tokens=batch)
    st = q.lib().q4gsw_kv_attention_ex(ctypes.byref(c), ctypes.byref(s), FAKE * 8, heads * 64, q.F16, heads, new, 100, 0, 0.0,
                                       FAKE * 12, None, 0, option(q, kernel), None)
    assert st == E_SHAPE


def test_join(q):  # noqa: F811
    """Splits of a call with far more token rows than its sequences' bounds."""
    c, s = cache(q, heads=1, dim=64), seqs(q, batch=1, tokens=1 << 22)
    f = q.lib().q4gsw_kv_attention
    go = lambda s, hq: f(ctypes.byref(c), ctypes.byref(s), FAKE * 8, hq * 64, q.F16, hq, 1, 4096, 0, 0.0, FAKE * 12, None, 0, None)
    assert go(s, 4) == E_SHAPE
    assert go(seqs(q, batch=1, tokens=1000), 4) == E_WS      # the same splits, a workspace is due
