"""Refusals of logits_adjust on the host: every call here fails validation before any HIP call, so made-up
device addresses are safe."""
import ctypes

import pytest
import torch

from tests.test_abi import E_ALIAS, E_DTYPE, E_NULL, E_SHAPE, FAKE, S_OK
from tests.test_serving_abi import q  # noqa: F401

NAMES = ["cu", "history", "history_len", "prompt_len", "ids", "parents", "repetition", "presence", "frequency", "bias_ids",
         "bias", "mask"]
AT = {n: FAKE * (80 + i) for i, n in enumerate(NAMES)}
X, OUT = FAKE * 100, FAKE * 101


def rules(q, **kw):  # noqa: F811
    r = q.binding.LogitsRules()
    base = dict(batch=3, max_new=16, history_ld=50, history_cols=40, bias_ld=12, bias_cols=10, mask_ld=32, **AT)
    for k, v in {**base, **kw}.items():
        setattr(r, k, v)
    return r


def test_layout(q):  # noqa: F811
    """The packed bytes of the binding are the structure."""
    values = dict(batch=3, max_new=16, cu=1, history=2, history_ld=50, history_cols=40, bias_cols=10, history_len=3, prompt_len=4,
                  ids=5, parents=6, repetition=7, presence=8, frequency=9, bias_ids=10, bias=11, bias_ld=12, mask=13, mask_ld=32)
    r = rules(q, **values)
    assert bytes(r) == q.binding._pack_rules(*(values[n] for n, _ in q.binding.LogitsRules._fields_))


def test_refusals(q):  # noqa: F811
    def go(x=X, dt=q.F32, rows=20, v=1000, ld=1000, out=OUT, out_ld=1000, **kw):
        return q.lib().q4gsw_logits_adjust(x, dt, rows, v, ld, ctypes.byref(rules(q, **kw)), out, out_ld, None)

    assert q.lib().q4gsw_logits_adjust(X, q.F32, 20, 1000, 1000, None, OUT, 1000, None) == E_NULL
    assert go(x=None) == E_NULL
    assert go(out=None) == E_NULL
    for kw in (dict(rows=-1), dict(rows=(1 << 23) + 1), dict(v=0), dict(v=1001), dict(out_ld=999), dict(ld=999), dict(batch=0),
               dict(batch=-1), dict(max_new=0), dict(max_new=513), dict(history_ld=39), dict(history_cols=-1), dict(bias_ld=9),
               dict(bias_cols=-1), dict(mask_ld=31), dict(cu=None, parents=None), dict(rows=1 << 23, v=1 << 26, ld=1 << 26,
                                                                                      out_ld=1 << 26, mask=None)):
        assert go(**kw) == E_SHAPE, kw
    assert go(dt=3) == E_DTYPE
    assert go(history_len=None) == E_NULL
    assert go(bias=None) == E_NULL
    assert go(cu=None, batch=20) == E_NULL                      # parents without cu
    assert go(ids=None) == E_NULL                               # parents without ids
    for name in NAMES:
        assert go(out=AT[name]) == E_ALIAS, name
    assert go(out=X + 4000) == E_ALIAS
    assert go(out=X, out_ld=1004) == E_ALIAS                    # in place, but of another pitch
    assert go(rows=0, x=None, out=None) == S_OK


def test_binding_refuses_tensors_of_the_wrong_kind(q):  # noqa: F811
    with pytest.raises(ValueError):
        q.logits_adjust(torch.zeros(3, 40))                     # not on a GPU
    x = torch.zeros(3, 40, device="meta")
    for bad in (x, x[0], x.long()):
        with pytest.raises(ValueError):
            q.logits_adjust(bad)


def test_histories_whose_counts_would_not_fit(q):  # noqa: F811
    """A token is counted in 29 bits with its path's: histories of up to 2^28 tokens."""
    def go(cols):
        r = rules(q, batch=1, history=FAKE << 20, history_cols=cols, history_ld=1 << 30, bias_ids=None, bias=None)
        # an output over the mask: what passes the sizes is refused for that, before any launch
        return q.lib().q4gsw_logits_adjust(X, q.F32, 1, 1000, 1000, ctypes.byref(r), AT["mask"], 1000, None)

    assert go(1 << 28) == E_ALIAS
    for cols in ((1 << 28) + 1, 1 << 29, 1 << 30):
        assert go(cols) == E_SHAPE, cols
