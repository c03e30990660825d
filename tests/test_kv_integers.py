"""Sizes that do not fit the library's 32-bit arguments are refused by the Python calls instead of
being taken modulo 2^32.  On the host: nothing here reaches a HIP call."""
import pytest
import torch

from tests.test_abi import FAKE
from tests.test_serving_abi import cache, q  # noqa: F401

BIG = 2 ** 32 + 64


def test_sizes_past_32_bits(q):  # noqa: F811
    c = q.KvCache(cache(q, heads=2, dim=64, data=FAKE), torch.empty(0, dtype=torch.uint8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    args = (c, torch.zeros(3, 4, 64), i32(1, 2), i32(2), i32(1))
    for bad in (dict(max_new=BIG), dict(max_ctx=BIG), dict(window=BIG), dict(window=2 ** 31), dict(window=-BIG)):
        with pytest.raises(ValueError):
            q.kv_attention(*args, **{**dict(max_new=3, max_ctx=3), **bad})
    sizes = dict(batch=1, tokens=3, hq=4, max_new=3, max_ctx=64)
    for bad in ("batch", "hq", "max_new", "max_ctx"):
        with pytest.raises(ValueError):
            q.kv_attention_workspace_bytes(c, **{**sizes, bad: BIG if bad != "hq" else 2 ** 32 + 4})
        with pytest.raises(ValueError):
            q.kv_attention_plan(c, **{**sizes, bad: BIG if bad != "hq" else 2 ** 32 + 4}, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.kv_attention_plan(c, **sizes, dtype=torch.float16, window=BIG)
    for bad in ((1, BIG, 1, 64), (1, 64, BIG, 64), (1, 64, 1, BIG)):
        with pytest.raises(ValueError):
            q.kv_cache(*bad)
    assert q.kv_attention_plan(c, **sizes, dtype=torch.float16, window=2 ** 31 - 1)["splits"] == 1
    for small in (dict(max_new=-1), dict(max_ctx=-1)):
        with pytest.raises(q.Q4gswError):
            q.kv_attention_plan(c, **{**sizes, **small}, dtype=torch.float16)
