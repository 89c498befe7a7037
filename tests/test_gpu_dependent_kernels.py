"""What the kernel in front of a call writes is what the call reads, although the call's
kernel may start before that one has ended."""
from __future__ import annotations

import pytest

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


def replayed(calls, stream, graph):
    """calls() on the stream, at once or through a captured graph."""
    import torch
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                calls()
            g.replay()
        else:
            calls()
    torch.cuda.synchronize()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T, N, K", [(1, 2048, 512), (40, 2048, 512), (40, 256, 8192),
                                     (4096, 6144, 128)])
def test_a_product_reads_scales_written_just_before_it(stp, ctx, T, N, K, graph):
    """One token, the split kernel alone and in clusters, and tiles."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(T + N)
    a, b = (torch.randint(-127, 128, (r, K), generator=g, device="cuda", dtype=torch.int8)
            for r in (T, N))
    kept = [[torch.rand(r, generator=g, device="cuda") + 0.1 for r in (T, N)] for _ in range(2)]
    sa, sb = (torch.empty(r, device="cuda") for r in (T, N))
    want, got = (torch.empty((n, T, N), dtype=torch.bfloat16, device="cuda") for n in (2, 10))

    def call(i, out):
        sa.copy_(kept[i][0])
        sb.copy_(kept[i][1])
        stp.staple_matmul_i8(ctx, stp.STAPLE_BF16, T, N, K, a, sa, b, sb, out)

    for i in range(2):
        call(i, want[i])
        torch.cuda.synchronize()
        ref = ((a.double() @ b.double().t()) * kept[i][0].double()[:, None]
               * kept[i][1].double()[None, :])
        tol = 2.0 ** -8 + 4 * 2.0 ** -24       # fp32 three times, then bf16
        assert bool(((want[i].double() - ref).abs() <= tol * ref.abs()).all())
    assert not torch.equal(*want)
    replayed(lambda: [call(i % 2, got[i]) for i in range(10)], torch.cuda.Stream(), graph)
    for i in range(10):
        assert torch.equal(got[i], want[i % 2])


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T, D", [(3, 64), (300, 2048), (300, 1001)])
def test_dropout_reads_the_state_written_just_before_it(stp, ctx, T, D, graph):
    """The norm forward and backward and dropout on its own, each behind an update of
    {seed, offset} on the same stream: the masks are those of the updated state."""
    import torch

    from oracle import block_oracle as bo
    p, n, seed, site = 0.5, 6, 1234567, 2
    x = torch.rand((T, D), device="cuda") + 1.0          # dropped elements alone are zero
    rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
    drop = stp.make_drop(p, rng, site)
    f32 = stp.STAPLE_F32
    s, y, o, dx = (torch.empty((n, T, D), device="cuda") for _ in range(4))
    rstd = torch.ones(T, device="cuda")
    dsum_in = torch.full((T, D), 1e6, device="cuda")      # so that ds is nowhere zero

    def calls():
        for i in range(n):
            rng[1] += 1
            stp.staple_norm_fwd(ctx, f32, stp.STAPLE_NORM_RMS, T, D, x, y[i], drop=drop, sum=s[i])
            rng[1] += 1
            stp.staple_dropout(ctx, f32, T, D, x, drop, o[i])
            rng[1] += 1
            stp.staple_norm_bwd(ctx, f32, stp.STAPLE_NORM_RMS, T, D, x, x, rstd, None,
                                dsum_in=dsum_in, drop=drop, dx=dx[i])

    replayed(calls, torch.cuda.Stream(), graph)
    for i in range(n):
        for k, got in enumerate((s[i], o[i], dx[i])):
            keep = bo.dropout_factors(T, D, p, seed, 3 * i + k + 1, site) != 0
            assert ((got != 0).cpu().numpy() == keep).all(), (i, k)


def test_quantise_layer_on_another_stream(stp, ctx):
    """The weights are written on the current stream, behind a wait, and so are the reads
    of a tensor whose memory the copy then gets; the copy is read there afterwards."""
    import torch

    from token_indexed_sparse_staple_b200.stack import LayerWeights, quantise_layer
    F, D = 512, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    src = [torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
           for s in ((F, D), (F, D), (D, F))]
    want = quantise_layer(ctx, LayerWeights(*src))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        w = [torch.zeros_like(s) for s in src]
        old = torch.full((2 * F, D), 5, dtype=torch.int8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)        # about 10 ms
        for a, b in zip(w, src):
            a.copy_(b)
        kept = old.clone()
        del old
        q = quantise_layer(ctx, LayerWeights(*w), stream=stream)
        got = [t.clone() for t in (q.w_gate_up, q.gate_up_scale, q.w_down, q.down_scale)]
        torch.cuda.synchronize()
        assert (kept == 5).all()
        for a, b in zip(got, (want.w_gate_up, want.gate_up_scale, want.w_down, want.down_scale)):
            assert torch.equal(a, b)
