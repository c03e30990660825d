"""linear_dq8ca_rows follows the calling thread's plan, as linear_dq8ca does."""
import ctypes

import pytest
import torch

from synthetic_inputs import make_linear
from tests.gpu_helpers import lib, pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 2, 3])
def test_forced_splits(splits):
    """With several splits the partials go to the workspace and the workspace query counts them; with
    one nothing is written there.  A group's int32 sum is exact; either result has a rounding of 2^-24 a
    group and a split, and the test's sizes those of the values and scales."""
    q = lib()
    print(f"dq8ca rows splits={splits}", flush=True)
    M, N, K = 40, 256, 1024
    pw = pack(q, make_linear(M, K, N, 64, "f32", "f16", seed=1).w)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(2)).cuda()
    rows, _, values = q.rmsnorm_dq8ca(x, torch.ones(K, device="cuda"), 1e-6, values=torch.empty(M, K, device="cuda"))
    with q.forced_plan(splits=1):
        one = q.linear_dq8ca_rows(pw, rows)
    codes, scales = q.unpack(pw)
    dense = (codes.float() - 8) * scales.float().repeat_interleave(64, 0).T
    size = values.abs().double() @ dense.abs().double().T
    ws = torch.full((4 << 20,), 0xAB, dtype=torch.uint8, device="cuda")
    with q.forced_plan(splits=splits):
        assert q.plan(q.OP_DQ8CA, pw, M, torch.float32)["splits"] == splits
        y = q.linear_dq8ca_rows(pw, rows, workspace=ws)
    torch.cuda.synchronize()
    need = ctypes.c_uint64()
    with q.forced_plan(splits=splits):
        assert q.lib().q4gsw_dq8ca_rows_workspace_bytes_ex(pw.ref(), M, q.binding._opts(), ctypes.byref(need)) == 0
    touched = (ws != 0xAB).nonzero()
    end = int(touched[-1]) + 1 if touched.numel() else 0
    assert need.value * (splits - 1) / splits < end <= need.value if splits > 1 else end == need.value == 0
    assert bool(((y - one).abs().double() <= 2 * (K // 64 + splits + 6) * 2.0 ** -24 * size).all())
