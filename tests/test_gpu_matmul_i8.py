"""Products of 8-bit integer matrices with scales per token and channel against
the fp64 definition.  The integer sum is exact; it is rounded to fp32, the two
products round once each (3 u, u = 2^-24), and bf16 storage rounds by 2^-8."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# fp32: one more rounding is counted than is made, for the product of the bounds
TOL = {"bf16": 2.0 ** -8 + 4 * U, "f32": 4 * U}


@pytest.fixture(scope="module")
def stp():
    import token_indexed_sparse_staple_b200 as m
    return m


@pytest.fixture(scope="module")
def ctx(stp):
    c = stp.staple_context_create(0)
    yield c
    stp.staple_context_destroy(c)


def operands(T, N, K, seed, full_range=False):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lo = -128 if full_range else -127
    a, b = (torch.randint(lo, 128, (r, K), generator=g, device="cuda", dtype=torch.int8)
            for r in (T, N))
    sa, sb = (torch.rand(r, generator=g, device="cuda") * 0.02 + 1e-4 for r in (T, N))
    return a, sa, b, sb


def run(stp, ctx, dtype, a, sa, b, sb, stream=None, y=None):
    import torch
    T, K = a.shape
    N = b.shape[0]
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    if y is None:
        y = torch.full((T + 2, N), 7.0, dtype=td, device="cuda")[1:T + 1]
    stp.staple_matmul_i8(ctx, stp.STAPLE_BF16 if dtype == "bf16" else stp.STAPLE_F32, T, N, K, a,
                         sa, b, sb, y, stream=stream)
    return y


def check(y, a, sa, b, sb, dtype):
    import torch
    # (fp64 products on the GPU for the large ones: the sums are exact there too)
    want = ((a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :])
    err = (y.double() - want).abs()
    bad = ~(err <= TOL[dtype] * want.abs())
    assert not bool(bad.any()), (int(bad.sum()), float(err.max()), bad.nonzero()[:4].tolist())


SHAPES = [(1, 1, 16), (1, 128, 256), (1, 8192, 2048), (2, 7, 48), (16, 129, 144), (17, 4096, 4096),
          (64, 11008, 4096), (64, 4096, 11008), (33, 1000, 1040), (100, 260, 8208), (128, 515, 528),
          (200, 2048, 8192), (256, 640, 512), (257, 640, 512), (300, 130, 12288), (700, 33, 16),
          (4096, 2048, 2048), (5000, 1023, 272), (2500, 4100, 160), (1537, 3001, 1552),
          (19000, 40, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, N, K", SHAPES)
def test_matches_the_definition(stp, ctx, T, N, K, dtype):
    import torch
    ops = operands(T, N, K, T + N + K, full_range=True)
    y = run(stp, ctx, dtype, *ops)
    check(y, *ops, dtype)
    full = y._base if y._base is not None else y
    assert (full[0] == 7).all() and (full[-1] == 7).all()
    assert stp.staple_get_error(ctx) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, N, K", [(129, 16384, 512), (200, 22016, 1040), (256, 12345, 528),
                                     (600, 9600, 2048), (1000, 2052, 784), (130, 600, 4112),
                                     (600, 200, 4096), (1100, 515, 8192)])
def test_either_kernel_above_half_a_tile_of_tokens(stp, ctx, T, N, K, dtype):
    """Both sides of the choice between the tiles and the split kernel, with rows,
    channels and k that no tile divides, at an output address of the element's size."""
    import torch
    ops = operands(T, N, K, T + K, full_range=True)
    check(run(stp, ctx, dtype, *ops), *ops, dtype)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((T * N + 2,), 7.0, dtype=td, device="cuda")
    y = buf[1:1 + T * N].view(T, N)
    run(stp, ctx, dtype, *ops, y=y)
    check(y, *ops, dtype)
    assert buf[0] == 7 and buf[-1] == 7
    assert stp.staple_get_error(ctx) == 0


def test_against_the_numpy_definition(stp, ctx):
    for dtype in ("bf16", "f32"):
        a, sa, b, sb = operands(19, 37, 80, 3)
        y = run(stp, ctx, dtype, a, sa, b, sb).double().cpu().numpy()
        want = bo.matmul_i8(*(t.cpu().numpy() for t in (a, sa, b, sb)))
        assert (np.abs(y - want) <= TOL[dtype] * np.abs(want)).all()


@pytest.mark.parametrize("T, N", [(3, 200), (300, 12800)])
def test_the_largest_sums_are_exact(stp, ctx, T, N):
    """-128 * -128 over the largest K, and the same with one product short."""
    import torch
    K = 131056
    a = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    b[1::2, K - 1] = 0
    sa, sb = torch.ones(T, device="cuda"), torch.full((N,), 2.0 ** -14, device="cuda")
    y = run(stp, ctx, "f32", a, sa, b, sb)
    assert (y[:, 0::2] == K).all() and (y[:, 1::2] == K - 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, N, K", [(5, 96, 64), (600, 9600, 64)])
def test_outputs_at_any_element_aligned_address(stp, ctx, dtype, T, N, K):
    import torch
    ops = operands(T, N, K, 5)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((T * N + 2,), 7.0, dtype=td, device="cuda")
    y = buf[1:1 + T * N].view(T, N)
    run(stp, ctx, dtype, *ops, y=y)
    check(y, *ops, dtype)
    assert buf[0] == 7 and buf[-1] == 7
    # scales at addresses that only fp32 alignment allows
    a, sa, b, sb = ops
    sa2, sb2 = (torch.cat([s[:1], s])[1:] for s in (sa, sb))
    y2 = run(stp, ctx, dtype, a, sa2, b, sb2)
    assert torch.equal(y2, y)


def test_non_finite_scales_reach_their_rows_and_channels_only(stp, ctx):
    import torch
    for T, N in ((9, 140), (400, 12800)):
        a, sa, b, sb = operands(T, N, 128, 1)
        a[4] = 0
        sa[4] = float("inf")      # what staple_quant_rows gives for such a row
        sa[6] = float("nan")
        sb[130] = float("nan")
        y = run(stp, ctx, "f32", a, sa, b, sb)
        bad = torch.isnan(y)
        want = torch.zeros_like(bad)
        want[4], want[6], want[:, 130] = True, True, True
        assert torch.equal(bad, want)


def test_streams_graphs_and_repeats(stp, ctx):
    import torch
    cases = [operands(T, N, K, T) for T, N, K in ((1, 8192, 2048), (64, 4096, 4096),
                                                  (1000, 9000, 512))]
    want = [run(stp, ctx, "bf16", *c).clone() for c in cases]
    ys = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):            # different shapes side by side on the SMs
        for c, y, s in zip(cases, ys, streams):
            run(stp, ctx, "bf16", *c, stream=s, y=y)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)
        y.zero_()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        for c, y in zip(cases, ys):
            run(stp, ctx, "bf16", *c, stream=s, y=y)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)
    assert stp.staple_get_error(ctx) == 0


def test_quantised_product_of_float_rows(stp, ctx):
    """staple_quant_rows on both operands, then the product: off from the fp64
    product of the unquantised rows by at most half a step of each operand,
    sa/2 sum|b| + sb/2 sum|a| + K sa sb / 4."""
    import torch
    T, N, K = 70, 300, 1040
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn((N, K), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    q = []
    for m in (x, w):
        v = torch.empty(m.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(m.shape[0], device="cuda")
        stp.staple_quant_rows(ctx, stp.STAPLE_BF16, *m.shape, m, v, s)
        q += [v, s]
    y = run(stp, ctx, "f32", *q)
    xd, wd, sx, sw = x.double(), w.double(), q[1].double()[:, None], q[3].double()[None, :]
    want = xd @ wd.t()
    tol = (sx / 2 * wd.abs().sum(1)[None, :] + sw / 2 * xd.abs().sum(1)[:, None] + K * sx * sw / 4)
    assert ((y.double() - want).abs() <= tol * 1.0001).all()


def test_an_empty_batch(stp, ctx):
    stp.staple_matmul_i8(ctx, stp.STAPLE_BF16, 0, 8, 16, None, None, None, None, None)


@pytest.mark.parametrize("T, N", [(300, 9472), (3, 8192), (64, 200)])
def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(stp, ctx, T, N):
    """The longest K makes the first sum take tens of microseconds at least (a
    pair of SMs 280, a block of a full split 150, a block of a cluster of 8
    about 20), so a limit of 10 us runs out in the first wait for an
    accumulator; the same context then computes the product."""
    import torch
    a, sa, b, sb = operands(T, N, 131056, 7)
    assert stp.staple_get_error(ctx) == 0
    stp.staple_set_wait_limit(ctx, 10_000)
    try:
        run(stp, ctx, "bf16", a, sa, b, sb)
        err = stp.staple_get_error(ctx)
    finally:
        stp.staple_set_wait_limit(ctx, 4_000_000_000)
    assert err == stp.STAPLE_ETIMEOUT, stp.staple_status_string(err)
    y = run(stp, ctx, "f32", a, sa, b, sb)
    assert stp.staple_get_error(ctx) == 0
    rows = torch.arange(0, T, max(1, T // 5), device="cuda")      # some tokens are enough
    want = ((a[rows].double() @ b.double().t()) * sa[rows].double()[:, None]
            * sb.double()[None, :])
    assert ((y[rows].double() - want).abs() <= TOL["f32"] * want.abs()).all()
