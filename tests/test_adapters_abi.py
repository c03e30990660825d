"""Refusals of the calls for adapters of many requests, on the host: every call here fails validation before
any HIP call, so made-up device addresses are safe."""
import ctypes

import pytest
import torch

from tests.test_abi import E_ALIAS, E_BUF, E_DESC, E_DTYPE, E_NULL, E_SHAPE, E_WS, FAKE, S_OK, fake_desc
from tests.test_serving_abi import E_ALIGN, q  # noqa: F401

X, SLOT, Y, OUT, WS, A, B, SET = (FAKE * i for i in range(60, 68))


def desc(q, n=256, k=512, slots=4, rank=16, dtype=None, reserved=0, data=SET, short=0):  # noqa: F811
    d = q.binding.AdaptersDesc(n, k, slots, rank, q.BF16 if dtype is None else dtype, reserved, data, 0)
    need = ctypes.c_uint64()
    if q.lib().q4gsw_adapters_bytes(ctypes.byref(d), ctypes.byref(need)) == S_OK:
        d.bytes = need.value - short
    return d


def test_bytes(q):  # noqa: F811
    f, n = q.lib().q4gsw_adapters_bytes, ctypes.c_uint64()
    r = ctypes.byref
    assert f(r(desc(q)), r(n)) == S_OK and n.value == 4 * 16 * (256 + 512) * 2 + 256
    assert f(r(desc(q, n=1, k=33, slots=1, rank=17)), r(n)) == S_OK and n.value == 32 * (32 + 64) * 2 + 256
    assert f(r(desc(q)), None) == E_NULL
    assert f(None, r(n)) == E_NULL
    for bad in (dict(n=0), dict(k=0), dict(n=(1 << 30) + 1), dict(k=-1), dict(slots=0), dict(slots=(1 << 20) + 1), dict(rank=0),
                dict(rank=65), dict(reserved=1)):
        assert f(r(desc(q, **bad)), r(n)) == E_SHAPE, bad
    for dt in (q.F32, 3, -1):
        assert f(r(desc(q, dtype=dt)), r(n)) == E_DTYPE


def test_load_refusals(q):  # noqa: F811
    f = q.lib().q4gsw_adapters_load

    def go(d=None, slot=0, a=A, b=B, dt=q.F32, rank=16, alpha=1.0):
        return f(ctypes.byref(d if d is not None else desc(q)), slot, a, b, dt, rank, alpha, None)

    assert go(desc(q, data=None)) == E_NULL
    assert go(desc(q, short=1)) == E_BUF
    assert go(desc(q, data=SET + 8)) == E_ALIGN
    assert go(a=None) == E_NULL
    assert go(b=None) == E_NULL
    for slot in (-1, 4):
        assert go(slot=slot) == E_SHAPE
    for rank in (0, 17, -3):
        assert go(rank=rank) == E_SHAPE
    for alpha in (float("nan"), float("inf")):
        assert go(alpha=alpha) == E_SHAPE
    assert go(dt=3) == E_DTYPE
    assert go(a=SET + 64) == E_ALIAS
    assert go(b=SET - 64) == E_ALIAS


def test_add_refusals(q):  # noqa: F811
    lib, r = q.lib(), ctypes.byref
    n = ctypes.c_uint64()
    assert lib.q4gsw_adapters_workspace_bytes(r(desc(q)), None, 40, q.F32, r(n)) == S_OK and n.value > 0
    need = n.value
    assert lib.q4gsw_adapters_workspace_bytes(r(desc(q)), None, 40, q.F32, None) == E_NULL
    assert lib.q4gsw_adapters_workspace_bytes(r(desc(q)), None, 0, q.F32, r(n)) == E_SHAPE
    assert lib.q4gsw_adapters_workspace_bytes(r(desc(q)), None, 40, 5, r(n)) == E_DTYPE

    def go(d=None, x=X, dt=q.F32, M=40, slot=SLOT, y=Y, out=OUT, ws=WS, wb=need):
        return lib.q4gsw_adapters_add(r(d if d is not None else desc(q)), x, dt, M, slot, y, out, ws, wb, None)

    assert go(desc(q, short=1)) == E_BUF
    for name in ("x", "slot", "y", "out"):
        assert go(**{name: None}) == E_NULL, name
    assert go(M=0) == E_SHAPE
    assert go(M=(1 << 23) + 1) == E_SHAPE
    assert go(desc(q, n=1 << 28), M=1 << 20) == E_SHAPE              # a launch past 2^32 threads
    assert go(dt=3) == E_DTYPE
    assert go(ws=None, wb=0) == E_WS
    assert go(wb=need - 1) == E_WS
    assert go(ws=WS + 16) == E_WS
    assert go(out=X) == E_ALIAS
    assert go(out=Y + 16) == E_ALIAS                                 # shifted, not in place
    assert go(out=SLOT) == E_ALIAS
    assert go(out=SET) == E_ALIAS
    assert go(out=WS) == E_ALIAS
    for name in ("x", "slot", "y"):
        assert go(**{name: WS}) == E_ALIAS, name
    assert go(ws=SET) == E_ALIAS


def test_fwd_refusals(q):  # noqa: F811
    lib, r = q.lib(), ctypes.byref
    n = ctypes.c_uint64()
    w = fake_desc(q, 256, 512, 64, 1, flags=1)
    wsb = lib.q4gsw_adapters_workspace_bytes
    assert wsb(r(desc(q)), r(w), 40, q.BF16, r(n)) == S_OK
    need = n.value
    assert need >= 1
    assert wsb(r(desc(q, n=255)), r(w), 40, q.BF16, r(n)) == E_SHAPE
    assert wsb(r(desc(q, k=256)), r(w), 40, q.BF16, r(n)) == E_SHAPE

    def go(w=w, d=None, x=X, dt=q.BF16, M=40, slot=SLOT, y=Y, ws=WS, wb=need):
        return lib.q4gsw_adapters_fwd(r(w), r(d if d is not None else desc(q)), x, dt, M, slot, y, ws, wb, None)

    bad = fake_desc(q, 256, 512, 64, 1)
    bad.magic = 0
    assert go(w=bad) == E_DESC
    assert wsb(r(desc(q)), r(bad), 40, q.BF16, r(n)) == E_DESC
    assert go(d=desc(q, n=255)) == E_SHAPE
    assert go(d=desc(q, k=480)) == E_SHAPE
    assert go(d=desc(q, short=1)) == E_BUF
    for name in ("x", "slot", "y"):
        assert go(**{name: None}) == E_NULL, name
    assert go(M=0) == E_SHAPE
    assert go(dt=3) == E_DTYPE
    assert go(wb=need - 1) == E_WS
    assert go(ws=WS + 16) == E_WS
    for name in ("x", "slot", "ws"):
        assert go(**{name: Y}) == E_ALIAS, name
    assert go(y=SET + 256) == E_ALIAS
    assert go(ws=SET) == E_ALIAS
    assert go(ws=SLOT) == E_ALIAS


def test_binding_refuses_tensors_of_the_wrong_kind(q):  # noqa: F811
    s = q.Adapters(desc(q, n=24, k=40), torch.empty(0, dtype=torch.uint8))
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    x, y = torch.zeros(3, 40), torch.zeros(3, 24)
    for bad in (torch.zeros(3, 41), torch.zeros(3), x.to(torch.int32)):
        with pytest.raises(ValueError):
            q.adapters_add(y, bad, s, i32(3))
    for bad in (i32(2), i32(3).long(), i32(3, 1)):
        with pytest.raises(ValueError):
            q.adapters_add(y, x, s, bad)
    for bad in (y.half(), torch.zeros(3, 25), torch.zeros(2, 24)):
        with pytest.raises(ValueError):
            q.adapters_add(bad, x, s, i32(3))
        with pytest.raises(ValueError):
            q.adapters_add(y, x, s, i32(3), out=bad)
    a, b = torch.zeros(4, 40), torch.zeros(24, 4)
    for bad in ((a[:, :9], b), (a, b[:, :3]), (a, b.half()), (a.to(torch.int32), b.to(torch.int32)), (a[0], b), (a, b.t())):
        with pytest.raises(ValueError):
            q.adapters_load(s, 0, *bad, 1.0)
    with pytest.raises(ValueError):
        q.adapters_load(s, 1 << 31, a, b, 1.0)
    with pytest.raises(ValueError):
        q.adapters(4, 16, 24, 40, torch.float32)
    with pytest.raises(ValueError):
        q.adapters(1 << 32, 16, 24, 40)
    with pytest.raises(ValueError):
        q.adapters(4, 16, 24, 40, device="cpu")


def test_a_weight_on_another_device(q):  # noqa: F811
    """adapters_fwd launches on the device of the set and x; a weight elsewhere is refused before that."""
    class Elsewhere:
        def get_device(self):
            return 1

    s = q.Adapters(desc(q, n=256, k=512), torch.empty(0, dtype=torch.uint8))
    w = q.PackedWeight(fake_desc(q, 256, 512, 64, 1, flags=1), Elsewhere())
    with pytest.raises(ValueError, match="w must be on"):
        q.adapters_fwd(w, torch.zeros(3, 512), s, torch.zeros(3, dtype=torch.int32))
