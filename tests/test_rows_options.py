"""The int8 linear on ready rows with per-call options, on the host: nothing here reaches a HIP call."""
import ctypes

from tests.test_abi import E_NULL, E_WS, FAKE, S_OK, fake_desc
from tests.test_serving_abi import q  # noqa: F401


def test_splits_reach_the_plan(q):  # noqa: F811
    """The workspace is that of linear_dq8ca less the rows', whatever the splits."""
    f, wsb, rb = q.lib().q4gsw_linear_dq8ca_rows_ex, q.lib().q4gsw_dq8ca_rows_workspace_bytes_ex, q.lib().q4gsw_dq8ca_rows_bytes
    n, whole, rows = (ctypes.c_uint64() for _ in range(3))
    d, r = fake_desc(q, 256, 1024, 64, 1), ctypes.byref
    assert rb(100, 1024, r(rows)) == S_OK
    assert q.lib().q4gsw_dq8ca_rows_workspace_bytes(r(d), 100, r(n)) == S_OK
    plain = n.value
    assert wsb(r(d), 100, None, r(n)) == S_OK and n.value == plain
    sizes = []
    for splits in (1, 2, 4):
        o = ctypes.pointer(q.binding.Options(0, 0, splits))
        assert wsb(r(d), 100, o, r(n)) == S_OK
        assert q.lib().q4gsw_workspace_bytes_ex(q.OP_DQ8CA, r(d), 100, q.F16, o, r(whole)) == S_OK
        assert whole.value - rows.value == n.value
        sizes.append(n.value)
        if n.value:
            assert f(r(d), FAKE * 8, rows.value, 100, FAKE * 9, FAKE * 10, n.value - 1, o, None) == E_WS
    assert sizes[0] == 0 and sizes[2] == 2 * sizes[1] > 0
    bad = ctypes.pointer(q.binding.Options(0, 0, -1))
    refused = q.lib().q4gsw_workspace_bytes_ex(q.OP_DQ8CA, r(d), 100, q.F16, bad, r(whole))
    assert refused != S_OK and wsb(r(d), 100, bad, r(n)) == refused
    assert f(r(d), FAKE * 8, rows.value, 100, FAKE * 9, None, 0, bad, None) == refused
    assert wsb(r(d), 100, None, None) == E_NULL
