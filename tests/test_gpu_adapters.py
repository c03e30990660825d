"""Adapters of many requests beside one projection, on the GPU against the formula in 64 bits.

The bound, element by element.  Products of 16-bit parts are exact in fp32, so t = x A^T is off by its sums'
roundings, K 2^-24 sum |x| |A|, and, where fp16 factors meet rows of another type, by 2^-21 of the row's
largest value times sum |A| (22 bits of it are kept: 2^-22, and once more for values that round
across a power of two).  t then loses 2^-21 of its row's largest where the factors are fp16 (2^-24 else, below the
sums' roundings) and alpha's product 2^-24; sums over the rank add rank 2^-24, the join with y one rounding
of the result.
"""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E = 2.0 ** -24


def factors(slots, rank, n, k, dtype, seed, ranks=None):
    """[(A, B, alpha)] of every slot, of ranks up to `rank`."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i in range(slots):
        r = rank if ranks is None else ranks[i % len(ranks)]
        out.append(((torch.randn(r, k, generator=g) * k ** -0.5).to(dtype), torch.randn(n, r, generator=g).to(dtype), 0.5 + i / 4))
    return out


def make(q, adapters, rank, n, k, dtype):
    s = q.adapters(len(adapters), rank, n, k, dtype)
    s.buffer.fill_(0xFF)                                       # what a slot holds before it is loaded
    for i, (a, b, alpha) in enumerate(adapters):
        q.adapters_load(s, i, a.cuda(), b.cuda(), alpha)
    return s


def formula(y, x, adapters, slots, dtype):
    """(out, bound) in 64 bits."""
    out, x = y.double().clone(), x.double()
    bound = torch.zeros_like(out)
    for m, i in enumerate(slots):
        if not 0 <= i < len(adapters):
            continue
        a, b, alpha = adapters[i]
        a, b = a.to(dtype).double(), b.to(dtype).double()
        t = a @ x[m]
        et = len(x[m]) * E * (a.abs() @ x[m].abs()) + 2.0 ** -21 * x[m].abs().max() * a.abs().sum(1)
        et = et + 2.0 ** -21 * t.abs().max() + (len(t) + 1) * E * t.abs()
        out[m] += alpha * (b @ t)
        bound[m] = abs(alpha) * (b.abs() @ et)
    return out, bound + 2 * E * out.abs() + 1e-30


def check(got, want, bound, label):
    g = got.cpu().double()
    assert torch.isfinite(g).all(), label
    worst = float(((g - want).abs() / bound).max())
    print(f"{label}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1, label


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def some_slots(m, n, seed, runs=False):
    g = torch.Generator().manual_seed(seed)
    s = torch.randint(-1, n + 1, (m,), generator=g)            # -1 and n: no adapter
    if runs:
        s = s.sort().values
    return s.tolist()


CASES = [
    # rows, K, N, rank, slots, x, factors, runs
    (1, 32, 32, 1, 1, BF16, BF16, False),
    (1, 4096, 130, 32, 3, BF16, F16, False),                   # one launch: t in every workgroup
    (3, 1024, 2049, 16, 2, F16, BF16, False),
    (16, 256, 516, 20, 16, F32, F16, False),
    (9, 512, 64, 16, 9, BF16, BF16, False),
    (4, 2080, 100, 16, 2, F32, BF16, False),                   # just past it
    (1, 2048, 2048, 16, 8, F32, BF16, False),
    (2, 100, 7, 5, 3, F16, F16, False),
    (15, 33, 1, 16, 4, F32, F16, False),
    (16, 256, 130, 17, 20, BF16, F16, False),
    (17, 288, 128, 33, 5, F16, BF16, False),
    (65, 4160, 96, 64, 70, F32, F16, False),
    (64, 1, 513, 8, 3, BF16, BF16, False),
    (100, 8192, 160, 48, 100, BF16, BF16, False),
    (300, 640, 512, 16, 9, F32, BF16, False),                  # unlike adapters in the tiles of a long call
    (300, 640, 516, 20, 3, F16, F16, True),
    (4100, 64, 1024, 16, 6, BF16, BF16, True),                 # wide column groups
    (4100, 40, 1030, 64, 6, F32, F16, False),
    (2064, 96, 2050, 33, 2, BF16, F16, True),
]


@pytest.mark.parametrize("m,k,n,rank,slots,xtype,ftype,runs", CASES)
def test_against_the_formula(m, k, n, rank, slots, xtype, ftype, runs):
    q = lib()
    label = f"adapters m={m} k={k} n={n} rank={rank} slots={slots} {xtype} {ftype}"
    print(label, flush=True)
    ad = factors(slots, rank, n, k, ftype, seed=k)
    s = make(q, ad, rank, n, k, ftype)
    g = torch.Generator().manual_seed(m)
    x, y, at = torch.randn(m, k, generator=g).to(xtype), torch.randn(m, n, generator=g), some_slots(m, slots, n, runs)
    want, bound = formula(y, x, ad, at, ftype)
    need = q.adapters_workspace_bytes(s, m, xtype)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    yd = y.cuda()
    got = q.adapters_add(yd, x.cuda(), s, ints(at), workspace=ws)
    check(got, want, bound, label)
    assert torch.equal(yd.cpu(), y)
    again = q.adapters_add(yd, x.cuda(), s, ints(at), out=yd)                  # in place
    assert again is yd and torch.equal(again, got)


@pytest.mark.parametrize("ftype", [F16, BF16])
@pytest.mark.parametrize("xtype", [F16, BF16, F32])
@pytest.mark.parametrize("k", [96, 99, 100])
def test_types_and_alignment(k, xtype, ftype):
    """Every pair of types, rows of whole quads and octets or not, x and out off their alignment."""
    q = lib()
    m, n, rank = 19, 36, 12
    ad = factors(4, rank, n, k, ftype, seed=1)
    s = make(q, ad, rank, n, k, ftype)
    g = torch.Generator().manual_seed(2)
    x, y, at = torch.randn(m, k, generator=g).to(xtype), torch.randn(m, n, generator=g), some_slots(m, 4, 3)
    want, bound = formula(y, x, ad, at, ftype)
    first = q.adapters_add(y.cuda(), x.cuda(), s, ints(at))
    check(first, want, bound, f"{k} {xtype} {ftype}")
    xo = torch.empty(m * k + 1, dtype=xtype, device="cuda")[1:].view(m, k).copy_(x)
    yo = torch.empty(m * n + 1, device="cuda")[1:].view(m, n).copy_(y)
    oo = torch.empty(m * n + 3, device="cuda")[3:].view(m, n)
    q.adapters_add(yo, xo, s, ints(at), out=oo)
    assert torch.equal(oo, first)


@pytest.mark.parametrize("src", [F16, BF16, F32])
@pytest.mark.parametrize("ftype", [F16, BF16])
def test_loading(ftype, src):
    """Factors of unlike ranks and any source type, rounded once; a slot loaded again."""
    q = lib()
    m, n, k, rank = 40, 70, 130, 40
    ad = factors(6, rank, n, k, src, seed=5, ranks=[1, 40, 16, 7, 33, 15])
    s = make(q, ad, rank, n, k, ftype)
    new = factors(1, 3, n, k, src, seed=6)[0]
    q.adapters_load(s, 1, new[0].cuda(), new[1].cuda(), new[2])                # a smaller rank over a larger one
    ad[1] = new
    g = torch.Generator().manual_seed(2)
    x, y, at = torch.randn(m, k, generator=g), torch.randn(m, n, generator=g), [i % 6 for i in range(m)]
    want, bound = formula(y, x, ad, at, ftype)
    check(q.adapters_add(y.cuda(), x.cuda(), s, ints(at)), want, bound, f"{src} in {ftype}")


def test_an_empty_set_adds_nothing():
    q = lib()
    s = q.adapters(3, 20, 50, 70, BF16)
    x, y = torch.randn(9, 70).cuda(), torch.randn(9, 50).cuda()
    assert torch.equal(q.adapters_add(y, x, s, ints([0, 1, 2, -1, 3, 2 ** 31 - 1, -2 ** 31, 0, 1])), y)


@pytest.mark.parametrize("ftype", [F16, BF16])
@pytest.mark.parametrize("xtype", [F16, BF16, F32])
def test_rows_are_their_own(xtype, ftype):
    """What is not finite in one row, or in one request's adapter, stays in the rows that are concerned."""
    q = lib()
    m, n, k, rank = 16, 64, 64, 16
    ad = factors(3, rank, n, k, ftype, seed=5)
    bad = (ad[2][0].clone(), ad[2][1].clone(), 1.0)
    bad[0][3, 5], bad[1][7, 2] = float("inf"), float("nan")
    s = make(q, ad[:2] + [bad], rank, n, k, ftype)
    x, y, at = torch.randn(m, k).to(xtype), torch.randn(m, n), [0, 1, 2, -1] * 4
    want, bound = formula(y, x, ad, at, ftype)
    x[0, 9], x[5, 63], x[3, 2] = float("nan"), float("inf"), float("nan")        # row 3 has no adapter
    got = q.adapters_add(y.cuda(), x.cuda(), s, ints(at)).cpu()
    broken = torch.tensor([i in (0, 5) or at[i] == 2 for i in range(m)])
    assert not got[broken].isfinite().all(1).any()
    check(got[~broken], want[~broken], bound[~broken], f"{xtype} {ftype}")
    assert torch.equal(got[3], y[3])


@pytest.mark.parametrize("ftype", [F16, BF16])
def test_ranges(ftype):
    """Rows far above and below fp16's range, and within a row values of unlike size."""
    q = lib()
    m, n, k, rank = 6, 40, 600, 9
    ad = factors(2, rank, n, k, ftype, seed=5)
    s = make(q, ad, rank, n, k, ftype)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(m, k, generator=g) * torch.tensor([1e-30, 1e-12, 1.0, 1e5, 1e12, 1e30])[:, None]
    x[2] *= torch.logspace(-9, 6, k)
    at = [0, 1, 0, 1, 0, 1]
    y = torch.zeros(m, n)
    want, bound = formula(y, x, ad, at, ftype)
    check(q.adapters_add(y.cuda(), x.cuda(), s, ints(at)), want, bound, f"{ftype}")
    x = x.to(BF16)
    want, bound = formula(y, x, ad, at, ftype)
    check(q.adapters_add(y.cuda(), x.cuda(), s, ints(at)), want, bound, f"{ftype} bf16 rows")


@pytest.mark.parametrize("m,xtype", [(1, BF16), (8, F32), (64, BF16), (300, F16), (2048, BF16)])
def test_beside_the_linear(m, xtype):
    """adapters_fwd is linear_fwd with the term of adapters_add, bit for bit."""
    q = lib()
    n, k, rank = 256, 512, 16
    g = torch.Generator().manual_seed(m)
    w = q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
               (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)
    ad = factors(5, rank, n, k, BF16, seed=1)
    s = make(q, ad, rank, n, k, BF16)
    x, at = torch.randn(m, k, generator=g).to(xtype), some_slots(m, 5, 1)
    y = q.linear_fwd(w, x.cuda())
    ws = torch.full((q.adapters_workspace_bytes(s, m, xtype, w),), 0xFF, dtype=torch.uint8, device="cuda")
    got = q.adapters_fwd(w, x.cuda(), s, ints(at), workspace=ws)
    assert torch.equal(got, q.adapters_add(y, x.cuda(), s, ints(at)))
    want, bound = formula(y.cpu(), x, ad, at, BF16)
    check(got, want, bound, f"beside the linear {m}")


def test_against_the_training_adapter():
    """A served adapter gives what adapter_fwd gives for the same factors."""
    q = lib()
    m, n, k, rank = 33, 128, 256, 8
    g = torch.Generator().manual_seed(1)
    w = q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
               (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)
    a, b, alpha = factors(1, rank, n, k, BF16, seed=1)[0]
    x = torch.randn(m, k, generator=g).to(BF16).cuda()
    want, _ = q.adapter_fwd(w, x, a.float().cuda(), b.float().cuda(), alpha)
    s = make(q, [(a, b, alpha)], rank, n, k, BF16)
    got = q.adapters_fwd(w, x, s, ints([0] * m))
    # two fp32 computations of sums of 256 and 8 products, values of some ten
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-4)


def test_captured_and_replayed():
    """Replays follow the slots and the factors that the tensors hold then."""
    q = lib()
    m, n, k, rank = 37, 96, 320, 16
    s = make(q, factors(4, rank, n, k, BF16, seed=1), rank, n, k, BF16)
    g = torch.Generator().manual_seed(2)
    x, y = torch.randn(m, k, generator=g).cuda(), torch.randn(m, n, generator=g).cuda()
    at, out = ints([0] * m), torch.empty(m, n, device="cuda")
    ws = torch.empty(q.adapters_workspace_bytes(s, m, F32), dtype=torch.uint8, device="cuda")
    call = lambda: q.adapters_add(y, x, s, at, out=out, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        ad = factors(4, rank, n, k, BF16, seed=10 + step)
        for i, (a, b, alpha) in enumerate(ad):
            q.adapters_load(s, i, a.cuda(), b.cuda(), alpha)
        now = some_slots(m, 4, step)
        at.copy_(ints(now))
        graph.replay()
        torch.cuda.synchronize()
        want, bound = formula(y.cpu(), x.cpu(), ad, now, BF16)
        check(out, want, bound, f"replay {step}")


@pytest.mark.parametrize("ftype", [F16, BF16])
@pytest.mark.parametrize("m,n,k,rank,slots,xtype", [
    (9, 64, 512, 5, 3, BF16),
    (17, 96, 1024, 16, 20, F16),
    (33, 65, 640, 24, 40, BF16),                   # odd columns, a tile with one row
    (64, 2050, 2048, 33, 70, F32),
    (50, 1000, 4096, 64, 8, F16),
    (200, 512, 4480, 16, 3, BF16),                 # three chunks of K
    (31, 320, 8192, 48, 64, F32),
])
def test_in_the_sum_of_a_split_linear(m, n, k, rank, slots, xtype, ftype):
    """Where the linear splits K, adapters_fwd adds the terms in the launch that sums the splits: the same values."""
    q = lib()
    g = torch.Generator().manual_seed(m)
    w = q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
               (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)
    ad = factors(slots, rank, n, k, ftype, seed=1, ranks=[rank, 1 + rank // 2])
    s = make(q, ad, rank, n, k, ftype)
    x, at = torch.randn(m, k, generator=g).to(xtype), some_slots(m, slots, 1)
    y = q.linear_fwd(w, x.cuda())
    ws = torch.full((q.adapters_workspace_bytes(s, m, xtype, w),), 0xFF, dtype=torch.uint8, device="cuda")
    got = q.adapters_fwd(w, x.cuda(), s, ints(at), workspace=ws)
    assert torch.equal(got, q.adapters_add(y, x.cuda(), s, ints(at)))
    want, bound = formula(y.cpu(), x, ad, at, ftype)
    check(got, want, bound, f"split {m} {n} {k}")
    # a row's term that is not finite stays in its row
    x[m // 2, 3] = float("nan")
    got = q.adapters_fwd(w, x.cuda(), s, ints(at))
    keep = torch.arange(m) != m // 2
    assert torch.equal(got.cpu()[keep], q.adapters_add(y, x.cuda(), s, ints(at)).cpu()[keep])


@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (5, 100, 96), (40, 2052, 2048), (40, 333, 1024), (1100, 260, 64)])
def test_rows_that_are_not_aligned(m, n, k):
    """y and out one element past an aligned address: the same values, and nothing beside them."""
    q = lib()
    g = torch.Generator().manual_seed(n)
    ad = factors(4, 8, n, k, F16, seed=2)
    s = make(q, ad, 8, n, k, F16)
    w = q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
               (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)
    x, y, at = torch.randn(m, k, generator=g).to(BF16).cuda(), torch.randn(m, n, generator=g).cuda(), ints(some_slots(m, 4, 1))

    def moved(t):
        return torch.cat([t.new_full((1,), 3.0), t.flatten()])[1:].view(t.shape)

    def room():
        return torch.full((m * n + 1 + 8,), 9.0, device="cuda")
    out = room()
    got = q.adapters_add(moved(y), x, s, at, out=out[1:1 + m * n].view(m, n))
    assert torch.equal(got, q.adapters_add(y, x, s, at))
    assert (out[:1] == 9).all() and (out[1 + m * n:] == 9).all()           # nothing beside the rows
    out = room()
    got = q.adapters_fwd(w, x, s, at, out=out[1:1 + m * n].view(m, n))
    assert torch.equal(got, q.adapters_fwd(w, x, s, at))
    assert (out[:1] == 9).all() and (out[1 + m * n:] == 9).all()


def packed(q, n, k, g):
    return q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
                  (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)


@pytest.mark.parametrize("rank", [16, 32])
@pytest.mark.parametrize("m", [1, 4])
@pytest.mark.parametrize("n", [261888, 261889, 262144, 262400])
def test_few_rows_of_an_output_layer(n, m, rank):
    """Outputs as wide as a vocabulary, on both sides of the change from narrow column groups to wide ones: every column of
    an `out` that holds NaN before, in place, and beside the linear."""
    q = lib()
    k = 64
    ad = factors(2, rank, n, k, BF16, seed=rank)
    s = make(q, ad, rank, n, k, BF16)
    g = torch.Generator().manual_seed(m)
    x, y, at = torch.randn(m, k, generator=g).to(BF16), torch.randn(m, n, generator=g), [i % 2 for i in range(m)]
    want, bound = formula(y, x, ad, at, BF16)
    out = torch.full((m, n), float("nan"), device="cuda")
    got = q.adapters_add(y.cuda(), x.cuda(), s, ints(at), out=out)
    check(got, want, bound, f"wide add m={m} n={n} rank={rank}")
    yd = y.cuda()
    assert torch.equal(q.adapters_add(yd, x.cuda(), s, ints(at), out=yd), got)
    w = packed(q, n, k, g)
    base = q.linear_fwd(w, x.cuda())
    out.fill_(float("nan"))
    got = q.adapters_fwd(w, x.cuda(), s, ints(at), out=out)
    want, bound = formula(base.cpu(), x, ad, at, BF16)
    check(got, want, bound, f"wide fwd m={m} n={n} rank={rank}")


@pytest.mark.parametrize("k", [2080, 4096, 8192])
@pytest.mark.parametrize("xtype,ftype", [(BF16, BF16), (F32, F16), (F16, BF16)])
def test_one_row_off_its_alignment(k, xtype, ftype):
    """Sums are in an order that depends on the sizes alone: a row of x at any address gives the same bits, whichever launches
    may load it."""
    q = lib()
    n, rank = 70, 16
    ad = factors(2, rank, n, k, ftype, seed=k)
    s = make(q, ad, rank, n, k, ftype)
    g = torch.Generator().manual_seed(k)
    x, y, at = torch.randn(1, k, generator=g).to(xtype), torch.randn(1, n, generator=g), [1]
    want, bound = formula(y, x, ad, at, ftype)
    first = q.adapters_add(y.cuda(), x.cuda(), s, ints(at))
    check(first, want, bound, f"aligned {k} {xtype} {ftype}")
    xo = torch.empty(k + 1, dtype=xtype, device="cuda")[1:].view(1, k).copy_(x)
    assert torch.equal(q.adapters_add(y.cuda(), xo, s, ints(at)), first)


@pytest.mark.parametrize("m,k,n,rank,slots,xtype,ftype", [
    (1, 2048, 130, 32, 3, BF16, F16), (1, 4096, 16384, 16, 2, BF16, BF16), (1, 4096, 16385, 16, 2, F16, BF16),
    (1, 4104, 65, 16, 2, F32, BF16), (2, 1024, 8192, 17, 3, F16, F16), (2, 1024, 8193, 17, 3, F32, BF16), (5, 384, 33, 20, 5, F32, F16),
    (16, 128, 516, 20, 16, BF16, F16), (16, 120, 516, 17, 3, F16, BF16), (16, 256, 1, 9, 16, F32, F16), (16, 264, 40, 9, 16, BF16, BF16)])
def test_one_launch_and_just_past_it(m, k, n, rank, slots, xtype, ftype):
    """Few rows up to 128 KB of factors and 256 column groups, and past them; `out` holds NaN before."""
    q = lib()
    ad = factors(slots, rank, n, k, ftype, seed=k)
    s = make(q, ad, rank, n, k, ftype)
    g = torch.Generator().manual_seed(m)
    x, y, at = torch.randn(m, k, generator=g).to(xtype), torch.randn(m, n, generator=g), some_slots(m, slots, n)
    want, bound = formula(y, x, ad, at, ftype)
    yd, out = y.cuda(), torch.full((m, n), float("nan"), device="cuda")
    check(q.adapters_add(yd, x.cuda(), s, ints(at), out=out), want, bound, f"{m} x {k} -> {n} rank {rank}")
    assert torch.equal(q.adapters_add(yd, x.cuda(), s, ints(at), out=yd), out)
