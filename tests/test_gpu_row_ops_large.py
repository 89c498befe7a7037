"""The operators around the layer at the far end of their sizes: rows of nearly 2^31
elements, and tensors of more than 2^31, whose last rows lie behind offsets that 32
bits do not hold.  Some rows of each are checked against the fp64 definitions.

Tolerances, with u = 2^-24 and h = half a step of bf16 (2^-8): dropout rounds the
scale and its product (3 u) and the sum (u) in fp32, then the output (h).  A sum over
a row takes at most 32 adds per thread, 5 across a warp and 16 across warps, 53 u of
the sum of the absolute values; 64 u covers it with the roundings of its terms."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
SEED, OFFSET, SITE = 0x0123456789ABCDEF, 5, 3


@pytest.fixture(scope="module")
def stp():
    import token_indexed_sparse_staple_b200 as m
    return m


@pytest.fixture(scope="module")
def ctx(stp):
    c = stp.staple_context_create(0)
    yield c
    stp.staple_context_destroy(c)


@pytest.fixture(autouse=True)
def give_memory_back():
    import torch
    yield
    torch.cuda.empty_cache()


def random_bf16(shape, seed):
    """bf16 values of either sign and 2^-7 to 2^9 in size, made in place as bit patterns:
    sign, mantissa and four bits of the exponent as drawn, the exponent from 120 on."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = torch.empty(shape, dtype=torch.int16, device="cuda")
    v.random_(-2 ** 15, 2 ** 15, generator=g)
    v &= 0x07FF - 0x8000
    v += 120 << 7
    return v.view(torch.bfloat16)


def np64(t):
    return t.detach().double().cpu().numpy()


def rng_state():
    import torch
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")


def factors(first_group, n, p):
    """The factors of n elements from a group's first on."""
    thr = int(np.floor(p * 65536 + 0.5))
    draws = []
    for g in range(first_group, first_group + -(-n // 8)):
        hi = OFFSET + SITE
        w = bo.philox4x32((g & bo.MASK32, g >> 32, hi & bo.MASK32, hi >> 32),
                          (SEED & bo.MASK32, SEED >> 32))
        for v in w:
            draws += [v & 0xFFFF, v >> 16]
    return np.where(np.array(draws[:n]) >= thr, 65536.0 / (65536 - thr), 0.0)


def within(got, want, tol, what):
    assert np.isfinite(got).all(), what
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[-1][:4])


# D - 1 + 32 passes 2^31 for the last three of these, and 2^31 - 32 is whole vectors
@pytest.mark.parametrize("D", [2 ** 31 - 33, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 9, 2 ** 31 - 1])
def test_dropout_of_the_longest_rows(stp, ctx, D):
    import torch
    x = random_bf16((1, D), 1)
    out = torch.full_like(x, float("nan"))
    stp.staple_dropout(ctx, stp.STAPLE_BF16, 1, D, x, stp.make_drop(0.0, None), out)
    assert torch.equal(out, x)
    out.fill_(float("nan"))
    rng, p = rng_state(), 0.25
    stp.staple_dropout(ctx, stp.STAPLE_BF16, 1, D, x, stp.make_drop(p, rng, SITE), out)
    for e0 in (0, D // 16 * 8, (D - 2000) // 8 * 8):
        n = min(2000, D - e0)
        want = np64(x[0, e0:e0 + n]) * factors(e0 // 8, n, p)
        within(np64(out[0, e0:e0 + n]), want, (H + 4 * U) * np.abs(want), e0)
    kept = int((out != 0).sum())      # every element was written: a NaN counts as kept
    assert not bool(torch.isnan(out).any())
    assert abs(kept / D - (1 - p)) < 1e-4      # 10 standard deviations


@pytest.mark.parametrize("D", [16384, 16383])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_and_dropout_behind_two_to_the_31(stp, ctx, D, rms):
    import torch
    T, p, eps = 131200, 0.25, 1e-5
    assert T * D > 2 ** 31 + D
    rows = [0, 2 ** 31 // D - 1, 2 ** 31 // D, 2 ** 31 // D + 1, T - 1]
    G = -(-D // 8)
    f = np.stack([factors(t * G, D, p) for t in rows])
    rng = rng_state()
    drop = stp.make_drop(p, rng, SITE)
    kind = stp.STAPLE_NORM_RMS if rms else stp.STAPLE_NORM_LAYER
    BF = stp.STAPLE_BF16
    x, res = random_bf16((T, D), 1), random_bf16((T, D), 2)
    w = random_bf16(D, 3)
    s, y = (torch.full_like(x, float("nan")) for _ in range(2))
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    stp.staple_norm_fwd(ctx, BF, kind, T, D, x, y, weight=w, eps=eps, residual=res, drop=drop,
                        sum=s, mean=mean, rstd=rstd)
    xr, rr, sr, wr = np64(x[rows]), np64(res[rows]), np64(s[rows]), np64(w)
    within(sr, rr + f * xr, H * np.abs(rr + f * xr) + 4 * U * (np.abs(f * xr) + np.abs(rr)), "sum")
    want, mu, rs = bo.norm_fwd(sr, wr, None, eps, rms)
    m1, c = np.abs(sr).mean(axis=1), np.abs(sr - mu[:, None])
    dvar = 64 * U * ((c * c).mean(axis=1) + 2 * c.mean(axis=1) * m1 + eps)
    within(np64(y[rows]), want, H * np.abs(want) + np.abs(wr) * rs[:, None] * 64 * U * m1[:, None]
           + np.abs(want) * ((dvar * rs ** 2)[:, None] + 10 * U), "y")
    # dropout by itself, over x's place
    out = y
    stp.staple_dropout(ctx, BF, T, D, x, drop, out, residual=res)
    assert torch.equal(out, s)
    del x, y, out
    # backward: the gradient into res's place
    dy, dsum_in = random_bf16((T, D), 4), res
    dx = torch.full_like(dy, float("nan"))
    dw, db = (torch.empty(D, device="cuda") for _ in range(2))
    wsb = stp.staple_norm_workspace_bytes(T, D)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ar = np64(dsum_in[rows])
    stp.staple_norm_bwd(ctx, BF, kind, T, D, dy, s, rstd, dsum_in, mean=mean, weight=w,
                        dsum_in=dsum_in, drop=drop, dx=dx, dw=dw, db=db, workspace=ws,
                        workspace_bytes=wsb)
    dyr, mu, rs = np64(dy[rows]), np64(mean[rows]), np64(rstd[rows])
    ds = bo.norm_bwd(dyr, sr, mu, rs, wr, rms)[0] + ar
    gw = np.abs(dyr * wr)
    xh = np.abs((sr - (0.0 if rms else mu[:, None])) * rs[:, None])
    tol = 64 * U * rs[:, None] * (gw + (0 if rms else gw.mean(axis=1, keepdims=True))
                                  + xh * (gw * xh).mean(axis=1, keepdims=True))
    tol += U * (np.abs(ar) + np.abs(ds))
    within(np64(dsum_in[rows]), ds, H * np.abs(ds) + tol * (1 + H), "dsum")
    within(np64(dx[rows]), f * ds, H * np.abs(f * ds) + f * (tol * (1 + H) + 3 * U * np.abs(ds)), "dx")
    # dw and db over all rows: every row of a block's share is added in turn, and a block
    # has at least T / 640 rows and at most all of T / 148 (148 blocks and more); then at
    # most 20 blocks in each of 32 slices; xhat and its product round 4 times
    n = -(-T // 148) + 20 + 32 + 4
    for which, got in (("dw", dw), ("db", db)):
        total, size = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
        for t in range(0, T, 4100):
            v = dy[t:t + 4100].double()
            if which == "dw":
                m = 0.0 if rms else mean[t:t + 4100, None].double()
                v *= (s[t:t + 4100].double() - m) * rstd[t:t + 4100, None].double()
            total += v.sum(dim=0)
            size += v.abs_().sum(dim=0)
        within(np64(got), np64(total), n * U * np64(size), which)
    assert stp.staple_get_error(ctx) == 0


@pytest.mark.parametrize("D", [32768, 32761])
def test_rows_to_8_bits_behind_two_to_the_31(stp, ctx, D):
    import torch
    T = 65700
    assert T * D > 2 ** 31 + D
    x = random_bf16((T, D), 1)
    q = torch.full((T, D), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((T,), float("nan"), device="cuda")
    stp.staple_quant_rows(ctx, stp.STAPLE_BF16, T, D, x, q, scale)
    for t in (0, 2 ** 31 // D, 2 ** 31 // D + 1, T - 1):
        wq, ws = bo.quant_rows(x[t:t + 1].float().cpu().numpy())
        assert (q[t].cpu().numpy() == wq[0]).all() and float(scale[t]) == float(ws[0]), t


def i8(shape, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=torch.int8, device="cuda").random_(-128, 128, generator=g)


# outputs (by TMA and by element), channels and tokens behind 2^31; each kernel
@pytest.mark.parametrize("T, N, K", [(131200, 16400, 32), (131200, 16401, 32), (1, 17000, 131056),
                                     (64, 17000, 131056), (300, 17000, 131056), (17000, 64, 131056),
                                     (17000, 520, 131056)])
def test_8_bit_product_behind_two_to_the_31(stp, ctx, T, N, K):
    import torch
    assert max(T * N, N * K, T * K) > 2 ** 31
    a, b = i8((T, K), 1), i8((N, K), 2)
    sa, sb = torch.rand(T, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    stp.staple_matmul_i8(ctx, stp.STAPLE_BF16, T, N, K, a, sa, b, sb, y)
    rows, cols = (torch.cat([torch.arange(0, min(n, 40)), torch.arange(max(n - 40, 0), n)]).cuda()
                  for n in (T, N))
    # (integer sums below 2^31 are exact in fp64; rounded to fp32, multiplied twice, stored)
    want = ((a[rows].double() @ b[cols].double().t()) * sa[rows].double()[:, None]
            * sb[cols].double()[None, :])
    got = y[rows][:, cols].double()
    assert bool(((got - want).abs() <= (H + 4 * U) * want.abs()).all())
    assert not bool(torch.isnan(y).any())
    assert stp.staple_get_error(ctx) == 0
