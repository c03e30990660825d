"""The C++ marshalling of the serving calls, without a GPU: what is not regular is left to Python."""
import pytest
import torch

import bit_group_quantized_q4gsw_amd as q


def host():
    q.lib()
    return q.binding._host


def test_calls_that_are_not_regular_are_left_to_python():
    h = host()
    d = q.binding.KvCacheDesc(4, 32, 2, 64, 0, None, 0)
    a = q.binding.ctypes.addressof(d)
    x, i = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    where = (table, i[:2], i[:1])
    for dev in (-1, 0):                                     # CPU tensors, whatever the device is said to be
        assert h.attention(a, dev, x, None, *where, 3, 3, 0, 0.0, None, None) is None
        assert h.attention(a, dev, x, i, *where, 3, 3, 0, 0.0, x, None) is None
        assert h.append(a, dev, x, x, *where) is None
        assert h.read(a, dev, *where, 3) is None
        assert h.keep([a], dev, i, i[:1], *where, 3, None, None) is None
        assert h.adapters(None, a, dev, x[:, 0], i, x[:, 0], None, None) is None
    for bad in (None, 3, "x", [None], 1.5):
        assert h.logits(bad, *[None] * 14) is None
        assert h.append(a, 0, bad, bad, *where) is None
        assert h.append(bad if bad != 3 else None, 0, x, x, *where) is None
        assert h.keep(bad, 0, i, i[:1], *where, 3, None, None) is None
        if bad is not None:
            assert h.adapters(bad if bad != 3 else "3", a, 0, x, i, x, None, None) is None
        assert h.attention(a, 1 << 40, bad, None, *where, bad, 3, 0, 0.0, None, None) is None
    assert h.logits(torch.zeros(2, 5), None, 1, *[None] * 12) is None
    assert h.logits(torch.zeros(2, 5, device="meta"), None, 1, *[None] * 12) is None
    assert h.logits(torch.zeros(2, 5).to_sparse(), None, 1, *[None] * 12) is None


@pytest.mark.parametrize("name", ["attention", "append", "read", "keep", "adapters", "logits", "open"])
def test_a_wrong_number_of_arguments(name):
    with pytest.raises(TypeError):
        getattr(host(), name)(1, 2)


def test_a_handle_without_the_calls():
    with pytest.raises(ImportError):
        host().open(q.binding.ctypes.CDLL(None)._handle, None, None)
    q.binding._host.open(q.lib()._handle, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
