"""rmsnorm_dq8ca and linear_dq8ca_rows on the GPU against their definitions.

h and the codes are decided by steps that are taken as defined, so h and the values' codes must be
equal; a value is code * scale in fp32, its scale two fp32 roundings (the norm's factor and the
product) from the definition: 3 roundings of 2^-24 in all.
"""
import pytest
import torch

from oracle import oracle as O
from synthetic_inputs import make_linear
from tests.gpu_helpers import THREADS, assert_within, lib, pack
from tests.serving_model import norm_rows

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

CASES = [
    # rows, cols, x, residual's type
    (1, 1, F32, F32), (3, 64, F32, F32), (4, 2048, F32, F32), (5, 300, BF16, F16), (2, 301, F16, BF16),
    (130, 1000, F32, BF16), (7, 8192, BF16, BF16), (3, 8200, F16, F32), (2, 16384, F32, F16), (2, 40000, BF16, BF16),
]


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("m,k,xt,rt", CASES)
def test_norm(m, k, xt, rt, with_residual):
    q = lib()
    print(f"norm m={m} k={k} {xt} {rt} residual={with_residual}", flush=True)
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=g).to(xt)
    res = (3 * torch.randn(m, k, generator=g)).to(rt) if with_residual else None
    w = (1 + 0.2 * torch.randn(k, generator=g)).to(rt)
    if m > 2:
        x[1], x[2] = 0, x[2].abs()
        if with_residual:
            res[1], res[2] = 0, res[2].abs()
    h = torch.empty(m, k, dtype=rt, device="cuda")
    values = torch.empty(m, k, device="cuda")
    rows, gh, gv = q.rmsnorm_dq8ca(x.cuda(), w.cuda(), 1e-6, residual=res.cuda() if with_residual else None, h=h,
                                   values=values)
    torch.cuda.synchronize()
    wh, codes, zero, row, wv = norm_rows(x, res, w, 1e-6)
    assert torch.equal(gh.cpu().double(), wh)
    err = (gv.cpu().double() - wv).abs()
    assert (err <= 3.1 * 2.0 ** -24 * wv.abs()).all(), float((err / wv.abs().clamp(min=1e-30)).max())
    # the rows themselves: codes in layout order, padding, scale and minus the zero point
    ld = (k + 127) // 128 * 128
    up = lambda n: (n + 255) // 256 * 256
    buf = rows.buffer.cpu()
    got = buf[:m * ld].view(torch.int8).view(m, ld // 8, 8)
    want = torch.zeros(m, ld, dtype=torch.int8)
    want[:, :k] = codes.to(torch.int8)
    assert torch.equal(got, want.view(m, ld // 8, 8)[:, :, [0, 4, 1, 5, 2, 6, 3, 7]])
    nz = buf[up(m * ld) + up(4 * m):up(m * ld) + up(4 * m) + 4 * m].view(torch.int32)
    assert torch.equal(nz.double(), -zero[:, 0])


def test_in_place_residual_and_optional_outputs():
    q = lib()
    print("norm in place", flush=True)
    g = torch.Generator().manual_seed(2)
    for k in (512, 500):
        x, res = torch.randn(9, k, generator=g).cuda(), torch.randn(9, k, generator=g).cuda()
        w = torch.rand(k, generator=g).cuda()
        rows, h, values = q.rmsnorm_dq8ca(x, w, 1e-5, residual=res)
        assert values is None and torch.equal(h, x + res)
        again = q.rmsnorm_dq8ca(x, w, 1e-5, residual=res, h=res)[0]
        assert torch.equal(again.buffer[:9 * 512], rows.buffer[:9 * 512])
        assert torch.equal(res, h)
        assert q.rmsnorm_dq8ca(x, w, 1e-5)[1] is None


def test_misaligned_input_takes_the_element_path():
    q = lib()
    print("norm misaligned", flush=True)
    x = torch.randn(4 * 256 + 1, generator=torch.Generator().manual_seed(1)).cuda()
    w = torch.ones(256, device="cuda")
    a = torch.empty(4, 256, device="cuda")
    b = torch.empty(4, 256, device="cuda")
    q.rmsnorm_dq8ca(x[1:].view(4, 256), w, 1e-6, values=a)
    q.rmsnorm_dq8ca(x[1:].view(4, 256).clone(), w, 1e-6, values=b)
    # the sum of squares is added up in another order: at most the scale's last bits differ
    assert ((a - b).abs() <= 4 * 2.0 ** -24 * b.abs()).all()


@pytest.mark.parametrize("m,k,n,gs", [(1, 64, 96, 32), (130, 512, 256, 64), (9, 2048, 512, 32), (257, 192, 128, 64)])
def test_rows_feed_the_int8_linear(m, k, n, gs):
    """linear_dq8ca_rows against a 64-bit product of the values the rows stand for; one rows buffer
    serves several weights."""
    q = lib()
    print(f"rows linear m={m} k={k} n={n} gs={gs}", flush=True)
    case = make_linear(m, k, n, gs, "bf16", "f16", seed=m + n)
    pw = pack(q, case.w)
    w = torch.rand(k, generator=torch.Generator().manual_seed(3)).to(BF16)
    values = torch.empty(m, k, device="cuda")
    rows, _, _ = q.rmsnorm_dq8ca(case.x.cuda(), w.cuda(), 1e-6, values=values)
    y = q.linear_dq8ca_rows(pw, rows)
    torch.cuda.synchronize()
    ref, norm = O.linear_fwd(values.cpu(), case.w.codes, case.w.scales, gs, threads=THREADS)
    splits = q.plan(q.OP_DQ8CA, pw, m, BF16)["splits"]
    # groups' sums and splits in fp32, the row scale, and the roundings of `values`
    assert_within(y, ref, norm, max(1e-5, (k // gs + splits + 6) * 2.0 ** -24), "rows linear")
    assert torch.equal(q.linear_dq8ca_rows(pw, rows), y)
