"""Refusals of the calls for trees of drafted tokens, on the host: every call here fails validation before
any HIP call, so made-up device addresses are safe."""
import ctypes
import itertools

import pytest
import torch

from tests.test_abi import E_ALIAS, E_BUF, E_DTYPE, E_NULL, E_SHAPE, E_WS, FAKE, S_OK
from tests.test_serving_abi import E_ALIGN, cache, q, seqs  # noqa: F401

UP, X, OUT, WS, LEAF, KEPT, PATH = (FAKE * i for i in range(40, 47))


def test_tree_attention_refusals(q):  # noqa: F811
    lib, r = q.lib(), ctypes.byref
    n = ctypes.c_uint64()
    c = cache(q)
    wsb = lib.q4gsw_kv_tree_attention_workspace_bytes
    assert wsb(r(c), 3, 5, 8, 2, 100000, r(n)) == S_OK and n.value > 0
    need = n.value
    assert wsb(r(c), 3, 5, 8, 2, 100000, None) == E_NULL
    assert wsb(r(c), 3, 5, 8, 512, 100000, r(n)) == S_OK
    assert wsb(r(c), 3, 5, 8, 513, 100000, r(n)) == E_SHAPE
    assert wsb(r(c), 0, 5, 8, 2, 9, r(n)) == E_SHAPE

    def go(c=None, s=None, up=UP, x=X, ld=1024, dt=q.F16, hq=8, new=2, ctx=100000, win=0, cap=0.0, out=OUT, ws=WS, wb=need):
        c, s = c if c is not None else cache(q), s if s is not None else seqs(q)
        args = (r(c), r(s), up, x, ld, dt, hq, new, ctx, win, cap, out, ws, wb)
        st = lib.q4gsw_kv_tree_attention(*args, None)
        assert st == lib.q4gsw_kv_tree_attention_ex(*args, None, None)
        return st

    assert go(cache(q, short=1)) == E_BUF
    assert go(up=None) == E_NULL
    assert go(x=None) == E_NULL
    assert go(out=None) == E_NULL
    assert go(new=513) == E_SHAPE
    assert go(new=0) == E_SHAPE
    assert go(hq=7) == E_SHAPE
    assert go(win=-1) == E_SHAPE
    assert go(cap=-1.0) == E_SHAPE
    assert go(dt=3) == E_DTYPE
    assert go(ld=1028) == E_ALIGN
    assert go(ws=None, wb=0) == E_WS
    assert go(out=UP) == E_ALIAS
    assert go(out=UP + 16) == E_ALIAS
    assert go(ws=UP) == E_ALIAS
    assert go(out=X) == E_ALIAS
    assert go(s=seqs(q, tokens=0), up=None, x=None, out=None, ws=None, wb=0) == S_OK
    opts = q.binding.KvOptions(9, 0)
    s = seqs(q)
    assert lib.q4gsw_kv_tree_attention_ex(r(c), r(s), UP, X, 1024, q.F16, 8, 2, 9, 0, 0.0, OUT, WS, need, r(opts), None) == 11
    # no kernel of many rows up to 32 rows
    opts.kernel = 4
    assert lib.q4gsw_kv_tree_attention_ex(r(c), r(s), UP, X, 1024, q.F16, 8, 2, 9, 0, 0.0, OUT, WS, need, r(opts), None) == 11
    opts.kernel = 2
    assert lib.q4gsw_kv_tree_attention_ex(r(c), r(s), UP, X, 1024, q.F16, 8, 2, 9, 0, 0.0, OUT, WS, need, r(opts), None) == 11


def test_a_window_never_needs_more_workspace(q):  # noqa: F811
    lib, r = q.lib(), ctypes.byref
    n = ctypes.c_uint64()
    opts = q.binding.KvOptions(0, 0)
    for heads, dim, new, kernel in itertools.product((1, 3), (64, 128, 256), (1, 5, 16, 64, 300, 512), (0, 1, 2, 3)):
        if kernel == 2 and 4 * new <= 32:
            continue
        c = cache(q, heads=heads, dim=dim)
        opts.kernel = kernel
        for ctx, batch in itertools.product((600, 5000, 131072), (1, 7, 100)):
            s = seqs(q, batch=batch, tokens=new * batch)
            assert lib.q4gsw_kv_tree_attention_workspace_bytes(r(c), batch, new * batch, 4 * heads, new, ctx, r(n)) == S_OK
            for win, dt in itertools.product((0, 1, 500, 4096, 100000), (q.F16, q.BF16)):
                st = lib.q4gsw_kv_tree_attention_ex(r(c), r(s), FAKE * 200, X, 4 * heads * dim, dt, 4 * heads, new, ctx, win, 0.0, X,
                                                    FAKE * 100, n.value, r(opts), None)
                assert st == E_ALIAS, (heads, dim, kernel, new, ctx, batch, win, st)


def caches(q, *each):  # noqa: F811
    return (q.binding.KvCacheDesc * len(each))(*each)


def test_keep_refusals(q):  # noqa: F811
    f, r = q.lib().q4gsw_kv_keep, ctypes.byref

    def go(cs=None, count=None, s=None, up=UP, leaf=LEAF, new=16, kept=KEPT, path=PATH):
        cs = cs if cs is not None else caches(q, cache(q))
        s = s if s is not None else seqs(q)
        return f(cs, len(cs) if count is None else count, r(s), up, leaf, new, kept, path, None)

    assert f(None, 1, r(seqs(q)), UP, LEAF, 16, KEPT, PATH, None) == E_NULL
    for count in (0, -1, 129):
        assert go(count=count) == E_SHAPE
    far = lambda i, **kw: cache(q, data=FAKE * (60 + i), **kw)  # noqa: E731
    assert go(caches(q, cache(q), far(1, heads=4))) == E_SHAPE
    assert go(caches(q, cache(q), far(1, dim=64))) == E_SHAPE
    assert go(caches(q, cache(q), far(1, page=128))) == E_SHAPE
    assert go(caches(q, cache(q), far(1, pages=11))) == E_SHAPE
    assert go(caches(q, cache(q), far(1, short=1))) == E_BUF
    assert go(caches(q, cache(q), cache(q, data=None))) == E_NULL
    assert go(caches(q, cache(q, data=FAKE + 8))) == E_ALIGN
    assert go(caches(q, far(1), far(2), far(1))) == E_ALIAS                  # the same cache twice
    assert go(s=seqs(q, batch=0)) == E_SHAPE
    assert go(s=seqs(q, cu=None)) == E_NULL
    assert go(new=0) == E_SHAPE
    assert go(new=513) == E_SHAPE
    assert go(up=None) == E_NULL
    assert go(leaf=None) == E_NULL
    assert go(kept=None) == E_NULL
    assert go(kept=PATH) == E_ALIAS
    assert go(kept=FAKE * 4) == E_ALIAS                                      # lens in place
    assert go(kept=FAKE * 3) == E_ALIAS
    assert go(kept=LEAF) == E_ALIAS
    assert go(path=UP) == E_ALIAS
    assert go(path=FAKE * 2) == E_ALIAS
    assert go(kept=FAKE + 64) == E_ALIAS
    assert go(path=FAKE + 64) == E_ALIAS
    assert go(up=FAKE + 64) == E_ALIAS
    assert go(leaf=FAKE + 64) == E_ALIAS
    assert go(caches(q, cache(q, data=FAKE * 4))) == E_ALIAS                 # over lens


def test_binding_refuses_tensors_of_the_wrong_kind(q):  # noqa: F811
    c = q.KvCache(cache(q, heads=2, dim=64, data=FAKE), torch.empty(0, dtype=torch.uint8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 4, 64)
    ok = dict(table=i32(1, 2), cu=i32(2), lens=i32(1), max_new=3)
    for up in (None, i32(2), i32(4), i32(3).long(), i32(3, 1), torch.zeros(3)):
        with pytest.raises(ValueError):
            q.kv_tree_attention(c, x, up, max_ctx=9, **ok)
    for leaf in (i32(2), i32(1).long(), i32(1, 1)):
        with pytest.raises(ValueError):
            q.kv_keep(c, i32(3), leaf, **ok)
    for up in (i32(3).long(), i32(3, 1)):
        with pytest.raises(ValueError):
            q.kv_keep(c, up, i32(1), **ok)
    for kw in (dict(kept=i32(2)), dict(kept=i32(1).long()), dict(path=i32(1, 4)), dict(path=i32(3, 1).t()[:, ::1].float())):
        with pytest.raises(ValueError):
            q.kv_keep(c, i32(3), i32(1), **kw, **ok)
    with pytest.raises(ValueError):
        q.kv_keep([], i32(3), i32(1), **ok)
    for new in (0, -1, 1 << 31):
        with pytest.raises(ValueError):
            q.kv_keep(c, i32(3), i32(1), **{**ok, "max_new": new})
