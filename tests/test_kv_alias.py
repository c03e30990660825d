"""Outputs of the cache's calls over the arrays that describe the sequences are refused on the host."""
import ctypes

import pytest

from tests.test_abi import E_ALIAS, FAKE
from tests.test_serving_abi import cache, q, seqs  # noqa: F401

BATCH, COLS, LD = 3, 4, 9
PLACES = {"table": (FAKE * 20, (2 * LD + COLS) * 4), "cu": (FAKE * 21, (BATCH + 1) * 4), "lens": (FAKE * 22, BATCH * 4)}


@pytest.mark.parametrize("name", list(PLACES))
@pytest.mark.parametrize("end", ["first", "last"])
def test_outputs_over_the_sequences(q, name, end):  # noqa: F811
    at, size = PLACES[name]
    hit = at if end == "first" else at + (size - 1) // 16 * 16
    r, lib = ctypes.byref, q.lib()
    s = seqs(q, batch=BATCH, cols=COLS, ld=LD, tokens=5, **{n: p for n, (p, _) in PLACES.items()})
    c = cache(q)
    attend = lambda out=FAKE * 9, ws=FAKE * 10, n=0, ctx=64: lib.q4gsw_kv_attention(
        r(c), r(s), FAKE * 8, 512, q.F16, 4, 2, ctx, 0, 0.0, out, ws, n, None)
    assert attend(out=hit) == E_ALIAS
    need = ctypes.c_uint64()
    assert lib.q4gsw_kv_attention_workspace_bytes(r(c), BATCH, 5, 4, 2, 5000, r(need)) == 0 and need.value > 0
    assert attend(ws=at & ~255, n=need.value, ctx=5000) == E_ALIAS
    for k, v in ((hit, FAKE * 9), (FAKE * 9, hit)):
        assert lib.q4gsw_kv_read(r(c), r(s), k, v, None) == E_ALIAS
    over = cache(q, data=at & ~15)
    assert lib.q4gsw_kv_append(r(over), r(s), FAKE * 8, 256, FAKE * 9, 256, q.F16, None) == E_ALIAS
