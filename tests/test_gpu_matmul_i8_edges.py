"""8-bit products whose last column tile holds an odd number of 32-column blocks,
with several tiles per pair of SMs: the blocks of such a tile and of the next one
leave by TMA from the same two staging boxes.

The integer sum is exact; it is rounded to fp32 and multiplied twice (3 u, u =
2^-24, and one more for the product of the bounds), and bf16 storage rounds by
2^-8."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
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


# 1, 3, 5 and 7 blocks in the last column tile, whole and cut; 320 tiles and more, so
# that every pair has four at least, and few k, so that the next sum is ready at once
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, N, K", [
    (16384, 1024 + 32, 64), (16384, 1024 + 8, 64), (16384, 1024 + 96, 16), (16384, 1024 + 72, 64),
    (16384, 1024 + 160, 64), (16384, 1024 + 136, 128), (16384, 1024 + 224, 64),
    (16001, 1024 + 200, 48), (100000, 16, 16), (100000, 96, 32), (4096, 8192 + 32, 128)])
def test_every_block_leaves_with_its_own_values(stp, ctx, T, N, K, dtype):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(T + N + K)
    a, b = (torch.randint(-128, 128, (r, K), generator=g, device="cuda", dtype=torch.int8)
            for r in (T, N))
    sa, sb = (torch.rand(r, generator=g, device="cuda") * 0.02 + 1e-4 for r in (T, N))
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    y = torch.full((T, N), float("nan"), dtype=td, device="cuda")
    dt = stp.STAPLE_BF16 if dtype == "bf16" else stp.STAPLE_F32

    def run(out):
        stp.staple_matmul_i8(ctx, dt, T, N, K, a, sa, b, sb, out)

    run(y)
    for r in range(0, T, 16384):     # (fp64 sums on the GPU, exact too)
        want = (a[r:r + 16384].double() @ b.double().t()) * sa[r:r + 16384].double()[:, None] * sb.double()
        err = (y[r:r + 16384].double() - want).abs()
        bad = ~(err <= TOL[dtype] * want.abs())
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    again = torch.empty_like(y)
    for _ in range(20):
        again.fill_(float("nan"))
        run(again)
        assert torch.equal(again, y)
    assert stp.staple_get_error(ctx) == 0


@pytest.mark.parametrize("T, D, F", [(2560, 64, 1040), (9216, 544, 272)])
def test_i8_layer_of_such_widths(stp, ctx, T, D, F):
    """2F, or D, with an odd number of blocks in the last tile of many."""
    from tests.test_gpu_block import I8Layer
    m = I8Layer(stp, ctx, T, D, F, V=50)
    m.run(m.embed("table"))
    m.check(True, False)
    assert stp.staple_get_error(ctx) == 0
