"""Rows quantised to 8-bit integers: bit for bit the exact quotient's rounding,
ties, zeros, subnormal scales, infinities and NaN included."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stp():
    import token_indexed_sparse_staple_b200 as m
    return m


@pytest.fixture(scope="module")
def ctx(stp):
    c = stp.staple_context_create(0)
    yield c
    stp.staple_context_destroy(c)


def run(stp, ctx, x, offset=0):
    """x: CUDA tensor [T][D]; q, scale as numpy, guards around q checked."""
    import torch
    T, D = x.shape
    dt = stp.STAPLE_BF16 if x.dtype == torch.bfloat16 else stp.STAPLE_F32
    qb = torch.full((T * D + offset + 8,), 99, dtype=torch.int8, device="cuda")
    q = qb[offset:offset + T * D]
    scale = torch.full((T + 1,), 5.0, device="cuda")
    stp.staple_quant_rows(ctx, dt, T, D, x, q, scale)
    torch.cuda.synchronize()
    assert (qb[:offset] == 99).all() and (qb[offset + T * D:] == 99).all() and scale[T] == 5
    return q.view(T, D).cpu().numpy(), scale[:T].cpu().numpy()


def check(stp, ctx, x, offset=0):
    q, s = run(stp, ctx, x, offset)
    wq, ws = bo.quant_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(s, ws)
    np.testing.assert_array_equal(q, wq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, D", [(1, 1), (1, 8), (3, 7), (5, 64), (1001, 24), (257, 100),
                                  (64, 4096), (2, 8192), (300, 1111), (3, 11008), (2, 20001),
                                  (2, 32768), (1, 32767)])
def test_matches_the_definition(stp, ctx, T, D, dtype):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(T * D)
    x = torch.randn((T, D), generator=g, device="cuda")
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    check(stp, ctx, x)
    if T * D < 1 << 20:
        check(stp, ctx, x, offset=3)      # q at an odd address
        flat = torch.zeros(T * D + 1, dtype=x.dtype, device="cuda")
        y = flat[1:].view(T, D)           # x only element-aligned
        y.copy_(x)
        check(stp, ctx, y)


def test_ties_and_their_neighbours(stp, ctx):
    """max = 127 s with s a power of two times an odd factor: every k + 1/2 is a
    tie where s is a power of two; one fp32 step beside it is not."""
    import torch
    rows = []
    for s in (1.0, 2.0 ** -20, 2.0 ** 30, 2.0 ** -59, 2.0 ** -66, 2.0 ** -100, 2.0 ** 118):
        half = (np.arange(-126, 127) + 0.5) * s
        for step in (0, 1, -1):
            v = half.astype(np.float32)
            if step:
                v = np.nextafter(v, np.float32(np.inf * step), dtype=np.float32)
            rows.append(np.concatenate([[np.float32(127 * s)], v, [0.0, -0.0]]))
    check(stp, ctx, torch.from_numpy(np.array(rows, dtype=np.float32)).cuda())


def test_random_scales_close_to_ties(stp, ctx):
    """Quotients within a few fp32 steps of k + 1/2 for scales of full precision."""
    import torch
    r = np.random.default_rng(0)
    T, D = 256, 512
    amax = (r.random(T) + 0.5).astype(np.float32) * np.float32(2.0) ** r.integers(-50, 50, T)
    amax = amax.astype(np.float32)
    s = (amax / np.float32(127)).astype(np.float64)
    k = r.integers(-126, 126, size=(T, D)) + 0.5
    x = (k * s[:, None]).astype(np.float32)
    x = (x.view(np.int32) + r.integers(-2, 3, size=(T, D)).astype(np.int32)).view(np.float32)
    x[:, 0] = amax
    check(stp, ctx, torch.from_numpy(x).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_subnormals_infinities_and_nans(stp, ctx, dtype):
    import torch
    D = 64
    x = np.zeros((9, D), dtype=np.float32)
    x[1, 3] = np.inf
    x[2, 5] = -np.inf
    x[2, 6] = np.nan
    x[3, 63] = np.nan
    x[4] = np.linspace(-1, 1, D) * 2.0 ** -126
    x[5, :40] = np.arange(40) * 2.0 ** -149         # the scale underflows to 0 or one step
    x[6] = np.linspace(-190, 190, D).round() * 2.0 ** -149   # scale 2^-149: clamped
    x[7] = 3.0e38 * np.linspace(-1, 1, D)
    x[8, 0] = 1e-30
    t = torch.from_numpy(x).cuda()
    check(stp, ctx, t.to(torch.bfloat16) if dtype == "bf16" else t)


def test_empty(stp, ctx):
    stp.staple_quant_rows(ctx, stp.STAPLE_BF16, 0, 64, None, None, None)
