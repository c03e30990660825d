"""Refusals of the decoder serving calls, on the host: every call here fails validation (or has
nothing to do) before any HIP call, so made-up device addresses are safe."""
import ctypes
import os

import pytest
import torch

from tests.test_abi import E_ALIAS, E_BUF, E_DESC, E_DTYPE, E_GROUP, E_NULL, E_SHAPE, E_WS, FAKE, S_OK, fake_desc

E_ALIGN = 13


@pytest.fixture(scope="module")
def q():
    from bit_group_quantized_q4gsw_amd import build as qbuild
    if not os.path.exists(qbuild.LIB):
        qbuild.build()
    import bit_group_quantized_q4gsw_amd as q
    return q


def cache(q, pages=10, page=64, heads=2, dim=128, data=FAKE, short=0, reserved=0):
    c = q.binding.KvCacheDesc(pages, page, heads, dim, reserved, data, 0)
    n = ctypes.c_uint64()
    if q.lib().q4gsw_kv_bytes(ctypes.byref(c), ctypes.byref(n)) == S_OK:
        c.bytes = n.value - short
    return c


def seqs(q, batch=3, cols=4, tokens=5, table=FAKE * 2, cu=FAKE * 3, lens=FAKE * 4, ld=None):
    return q.binding.KvSeqs(table, cols if ld is None else ld, cols, batch, cu, lens, tokens)


def test_new_status_name(q):
    assert "16 bytes" in q.status_str(E_ALIGN)


def test_kv_bytes(q):
    f, n = q.lib().q4gsw_kv_bytes, ctypes.c_uint64()
    assert f(ctypes.byref(cache(q)), ctypes.byref(n)) == S_OK
    assert n.value == 10 * 2 * 64 * 2 * (128 // 2 + 2 * 128 // 32)       # codes and scales of keys and values
    assert f(ctypes.byref(cache(q)), None) == E_NULL
    assert f(None, ctypes.byref(n)) == E_NULL
    for bad in (dict(pages=0), dict(pages=-1), dict(page=16), dict(page=48), dict(page=8192), dict(heads=0),
                dict(heads=70000), dict(dim=32), dict(dim=100), dict(dim=512), dict(reserved=1)):
        assert f(ctypes.byref(cache(q, **bad)), ctypes.byref(n)) == E_SHAPE, bad


def test_kv_append_refusals(q):
    f = q.lib().q4gsw_kv_append
    k, v = FAKE * 8, FAKE * 9

    def go(c=None, s=None, k=k, k_ld=256, v=v, v_ld=256, dt=q.F16):
        return f(ctypes.byref(c if c is not None else cache(q)), ctypes.byref(s if s is not None else seqs(q)), k, k_ld, v,
                 v_ld, dt, None)

    assert go(cache(q, data=None)) == E_NULL
    assert go(cache(q, short=1)) == E_BUF
    assert go(cache(q, data=FAKE + 8)) == E_ALIGN
    assert go(cache(q, dim=80)) == E_SHAPE
    assert go(s=seqs(q, batch=0)) == E_SHAPE
    assert go(s=seqs(q, tokens=-1)) == E_SHAPE
    assert go(s=seqs(q, ld=3)) == E_SHAPE                     # overlapping table rows
    assert go(s=seqs(q, cu=None)) == E_NULL
    assert go(s=seqs(q, lens=None)) == E_NULL
    assert go(s=seqs(q, table=None)) == E_NULL
    assert go(k=None) == E_NULL
    assert go(v=None) == E_NULL
    assert go(dt=7) == E_DTYPE
    assert go(k_ld=255) == E_SHAPE                            # rows overlap
    assert go(k_ld=260) == E_ALIGN                            # 520-byte pitch
    assert go(k=k + 8) == E_ALIGN
    assert go(v=v + 2) == E_ALIGN
    assert go(k=FAKE + 256) == E_ALIAS                        # inside the cache
    assert go(v=FAKE - 512) == E_ALIAS                        # runs into it
    assert go(s=seqs(q, tokens=0), k=None, v=None) == S_OK    # nothing to store: no HIP call


def test_kv_read_refusals(q):
    f = q.lib().q4gsw_kv_read
    c, s = cache(q), seqs(q)
    assert f(ctypes.byref(c), ctypes.byref(s), None, FAKE * 8, None) == E_NULL
    assert f(ctypes.byref(c), ctypes.byref(s), FAKE * 8 + 4, FAKE * 9, None) == E_ALIGN
    assert f(ctypes.byref(c), ctypes.byref(s), FAKE * 8, FAKE * 8 + 64, None) == E_ALIAS
    assert f(ctypes.byref(c), ctypes.byref(s), FAKE + 64, FAKE * 8, None) == E_ALIAS
    assert f(ctypes.byref(c), ctypes.byref(seqs(q, tokens=0)), None, None, None) == S_OK


def test_kv_attention_refusals(q):
    f, wsb = q.lib().q4gsw_kv_attention, q.lib().q4gsw_kv_attention_workspace_bytes
    n = ctypes.c_uint64()
    c = cache(q)
    assert wsb(ctypes.byref(c), 3, 5, 8, 2, 100000, ctypes.byref(n)) == S_OK
    need = n.value
    assert need > 0
    assert wsb(ctypes.byref(c), 3, 5, 8, 2, 100000, None) == E_NULL
    assert wsb(ctypes.byref(c), 3, 5, 8, 2, 64, ctypes.byref(n)) == S_OK and n.value == 0
    for bad in ((0, 5, 8, 2, 9), (3, -1, 8, 2, 9), (3, 5, 7, 2, 9), (3, 5, 0, 2, 9), (3, 5, 8, 0, 9), (3, 5, 8, 2, -1)):
        assert wsb(ctypes.byref(c), *bad, ctypes.byref(n)) == E_SHAPE, bad

    qq, out, ws = FAKE * 8, FAKE * 9, FAKE * 10

    def go(c=None, s=None, x=qq, ld=1024, dt=q.F16, hq=8, new=2, ctx=100000, win=0, cap=0.0, out=out, ws=ws, wb=need):
        return f(ctypes.byref(c if c is not None else cache(q)), ctypes.byref(s if s is not None else seqs(q)), x, ld, dt, hq,
                 new, ctx, win, cap, out, ws, wb, None)

    nan, inf = float("nan"), float("inf")
    assert go(cache(q, short=1)) == E_BUF
    assert go(hq=7) == E_SHAPE
    assert go(new=0) == E_SHAPE
    assert go(ctx=-1) == E_SHAPE
    assert go(win=-1) == E_SHAPE
    for cap in (nan, inf, -1.0, 1e-38, 1e38):
        assert go(cap=cap) == E_SHAPE, cap
    assert go(dt=3) == E_DTYPE
    assert go(x=None) == E_NULL
    assert go(out=None) == E_NULL
    assert go(ld=1023) == E_SHAPE
    assert go(ld=1028) == E_ALIGN
    assert go(x=qq + 2) == E_ALIGN
    assert go(out=out + 4) == E_ALIGN
    assert go(ws=None, wb=0) == E_WS
    assert go(wb=need - 1) == E_WS
    assert go(ws=ws + 16) == E_WS
    assert go(out=qq + 1024) == E_ALIAS
    assert go(out=FAKE + 1024) == E_ALIAS
    assert go(ws=qq) == E_ALIAS
    assert go(ws=out) == E_ALIAS
    assert go(ws=FAKE) == E_ALIAS
    assert go(s=seqs(q, tokens=0), x=None, out=None, ws=None, wb=0) == S_OK


def test_window_never_needs_more_workspace(q):
    """kv_attention is given one workspace for every window: a narrower span must pass validation with
    it (an aliasing output is refused only after the workspace check)."""
    f, wsb = q.lib().q4gsw_kv_attention, q.lib().q4gsw_kv_attention_workspace_bytes
    n = ctypes.c_uint64()
    c = cache(q, heads=1)
    for new in (1, 5, 40, 300):
        for ctx in (64, 600, 1000, 5000, 131072):
            for batch in (1, 7, 100):
                if new > ctx:
                    continue
                s = seqs(q, batch=batch, tokens=new * batch)
                assert wsb(ctypes.byref(c), batch, new * batch, 4, new, ctx, ctypes.byref(n)) == S_OK
                for win in (1, 33, 500, 2000, 4096, 100000):
                    st = f(ctypes.byref(c), ctypes.byref(s), FAKE * 8, 512, q.F16, 4, new, ctx, win, 0.0, FAKE * 8,
                           FAKE * 10, n.value, None)
                    assert st == E_ALIAS, (new, ctx, batch, win, st)


def test_norm_refusals(q):
    f, rb = q.lib().q4gsw_rmsnorm_dq8ca, q.lib().q4gsw_dq8ca_rows_bytes
    n = ctypes.c_uint64()
    assert rb(4, 300, ctypes.byref(n)) == S_OK
    need = n.value
    assert need >= 4 * 384 + 4 * 8
    assert rb(4, 300, None) == E_NULL
    assert rb(0, 300, ctypes.byref(n)) == E_SHAPE
    assert rb(4, 0, ctypes.byref(n)) == E_SHAPE
    x, res, w, h, rows, val = (FAKE * i for i in range(8, 14))

    def go(x=x, xt=q.F16, res=res, w=w, rt=q.F32, M=4, K=300, eps=1e-6, h=h, rows=rows, rb=need, val=val):
        return f(x, xt, res, w, rt, M, K, eps, h, rows, rb, val, None)

    assert go(x=None) == E_NULL
    assert go(w=None) == E_NULL
    assert go(rows=None) == E_NULL
    assert go(M=0) == E_SHAPE
    assert go(K=0) == E_SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert go(eps=eps) == E_SHAPE
    assert go(xt=5) == E_DTYPE
    assert go(rt=-1) == E_DTYPE
    assert go(rb=need - 1) == E_BUF
    assert go(rows=rows + 128) == E_ALIGN
    assert go(h=x + 16) == E_ALIAS
    assert go(h=res + 16) == E_ALIAS                          # shifted, not in place
    assert go(h=w) == E_ALIAS
    assert go(val=h + 64) == E_ALIAS
    assert go(val=x) == E_ALIAS
    assert go(val=res) == E_ALIAS
    assert go(rows=val) == E_ALIAS
    assert go(rows=res) == E_ALIAS


def test_rows_linear_refusals(q):
    f, wsb = q.lib().q4gsw_linear_dq8ca_rows, q.lib().q4gsw_dq8ca_rows_workspace_bytes
    rb = q.lib().q4gsw_dq8ca_rows_bytes
    n = ctypes.c_uint64()
    d = fake_desc(q, 256, 512, 64, 1, flags=1)
    r = ctypes.byref
    assert rb(100, 512, r(n)) == S_OK
    need = n.value
    assert wsb(r(d), 100, r(n)) == S_OK
    wneed = n.value
    assert wneed > 0
    rows, y, ws = FAKE * 8, FAKE * 9, FAKE * 10
    assert wsb(r(d), 100, None) == E_NULL
    assert wsb(r(fake_desc(q, 256, 512, 16, 1)), 100, r(n)) == E_GROUP
    bad = fake_desc(q, 256, 512, 64, 1)
    bad.magic = 0
    assert f(r(bad), rows, need, 100, y, ws, wneed, None) == E_DESC
    assert f(r(d), None, need, 100, y, ws, wneed, None) == E_NULL
    assert f(r(d), rows, need, 100, None, ws, wneed, None) == E_NULL
    assert f(r(d), rows, need, 0, y, ws, wneed, None) == E_SHAPE
    assert f(r(d), rows, need - 1, 100, y, ws, wneed, None) == E_BUF
    assert f(r(d), rows + 64, need, 100, y, ws, wneed, None) == E_ALIGN
    assert f(r(d), rows, need, 100, y, None, 0, None) == E_WS
    assert f(r(d), rows, need, 100, rows + 256, ws, wneed, None) == E_ALIAS
    assert f(r(d), rows, need, 100, y, rows, wneed, None) == E_ALIAS
    assert f(r(d), rows, need, 100, y, y, wneed, None) == E_ALIAS
    assert f(r(d), rows, need, 100, FAKE * 4 + 512, ws, wneed, None) == E_ALIAS


def test_binding_refuses_tensors_of_the_wrong_kind(q):
    """The Python calls check dtypes, shapes and devices before the library is asked (a cache object
    on the CPU stands in: nothing is launched)."""
    c = q.KvCache(cache(q, heads=2, dim=64, data=FAKE), torch.empty(0, dtype=torch.uint8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    k = torch.zeros(3, 2, 64)
    ok = dict(table=i32(1, 2), cu=i32(2), lens=i32(1))
    for bad in (dict(table=i32(2, 2)), dict(table=torch.zeros(1, 2)), dict(cu=i32(3)), dict(lens=i32(1).long()),
                dict(table=i32(1, 4)[:, ::2])):
        with pytest.raises(ValueError):
            q.kv_append(c, k, k, **{**ok, **bad})
    for x in (k[:, :1], k[..., :32], k.to(torch.int32), k[0]):
        with pytest.raises(ValueError):
            q.kv_append(c, x, k, **ok)
    with pytest.raises(ValueError):
        q.kv_append(c, k, k.half(), **ok)
    with pytest.raises(ValueError):
        q.kv_append(c, k, k[:2], **ok)
    with pytest.raises(ValueError):
        q.kv_attention(c, torch.zeros(3, 4, 32), max_new=1, max_ctx=1, **ok)
    with pytest.raises(ValueError):
        q.kv_attention(c, torch.zeros(3, 4, 64), max_new=1, max_ctx=1, out=torch.zeros(3, 4, 64).half(), **ok)
    with pytest.raises(ValueError):
        q.kv_read(c, tokens=3, out=(k, k.half()), **ok)
    with pytest.raises(ValueError):
        q.rmsnorm_dq8ca(torch.zeros(3, 4), torch.ones(4), 1e-6)
    with pytest.raises(ValueError):
        q.linear_dq8ca_rows(q.PackedWeight(fake_desc(q, 256, 512, 64), torch.empty(0)), q.Dq8caRows(3, 256, torch.empty(0)))
