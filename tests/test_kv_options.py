"""The kernel choice and the plan of kv_attention, on the host: nothing here reaches a HIP call."""
import ctypes

import pytest

from tests.test_abi import E_ALIAS, E_DTYPE, E_NULL, E_SHAPE, FAKE, S_OK
from tests.test_serving_abi import cache, q, seqs  # noqa: F401

E_ROUTE = 11


def option(q, kernel, reserved=0):
    return ctypes.pointer(q.binding.KvOptions(kernel, reserved))


def test_plan(q):  # noqa: F811
    f, info, c = q.lib().q4gsw_kv_attention_plan, q.binding.KvPlanInfo(), cache(q)
    go = lambda new=40, win=0, dt=2, opts=None, out=info, hq=8: f(
        ctypes.byref(c), 3, 3 * new, hq, new, 1000, win, dt, opts, ctypes.byref(out) if out is not None else None)
    assert go() == S_OK and info.kernel == 1 and info.waves in (4, 8) and info.splits >= 1
    assert go(opts=option(q, 2)) == S_OK and info.kernel == 2
    assert go(opts=option(q, 1)) == S_OK and info.kernel == 1
    assert go(out=None) == E_NULL
    assert go(win=-1) == E_SHAPE
    assert go(hq=7) == E_SHAPE
    assert go(dt=9) == E_DTYPE
    assert go(opts=option(q, 3)) == E_ROUTE
    assert go(opts=option(q, -1)) == E_ROUTE
    assert go(opts=option(q, 1, 1)) == E_SHAPE
    assert go(new=8, opts=option(q, 2)) == E_ROUTE            # 32 rows a cache head
    assert go(new=9, opts=option(q, 2)) == S_OK


def test_either_kernel_fits_the_workspace(q):  # noqa: F811
    """kv_attention_workspace_bytes covers both kernels and every window (an aliasing output is refused
    only after the workspace check)."""
    f, wsb = q.lib().q4gsw_kv_attention_ex, q.lib().q4gsw_kv_attention_workspace_bytes
    n, c = ctypes.c_uint64(), cache(q, heads=1)
    for new in (9, 40, 300, 2000):
        for ctx in (300, 2500, 9000, 131072):
            for batch in (1, 9, 100):
                if new > ctx:
                    continue
                s = seqs(q, batch=batch, tokens=new * batch)
                assert wsb(ctypes.byref(c), batch, new * batch, 4, new, ctx, ctypes.byref(n)) == S_OK
                for win in (0, 1, 500, 4096):
                    for opts in (None, option(q, 1), option(q, 2)):
                        for dt in (q.F16, q.BF16):
                            st = f(ctypes.byref(c), ctypes.byref(s), FAKE * 8, 512, dt, 4, new, ctx, win, 0.0, FAKE * 8,
                                   FAKE * 10, n.value, opts, None)
                            assert st == E_ALIAS, (new, ctx, batch, win, st)


def test_forced_kernel_names(q):  # noqa: F811
    with pytest.raises(KeyError):
        with q.forced_kv_kernel("other"):
            pass
    with q.forced_kv_kernel("many_rows"):
        assert q.binding._local.kv.contents.kernel == 2
    assert getattr(q.binding._local, "kv", None) is None


def test_a_cache_on_the_cpu_is_refused(q):  # noqa: F811
    with pytest.raises(ValueError):
        q.kv_cache(2, 64, 1, 64, device="cpu")
