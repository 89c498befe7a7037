"""The operators around the layer at the far end of their sizes: rows of nearly 2^31
elements.  Parts of them are checked against the fp64 definitions.

Tolerances, with u = 2^-24 and h = half a step of bf16 (2^-8): dropout rounds the
scale and its product (3 u) and the sum (u) in fp32, then the output (h)."""
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
