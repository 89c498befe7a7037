"""The operators around the layer together, as a model uses them: the 8-bit
layer, and the training and decode stacks as residual streams with norms and
dropout.  Each layer is checked against the fp64 definitions on its own inputs
as the GPU produced them."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import synthetic as syn
from oracle import block_oracle as bo
from tests.helpers import TOL, assert_close, dev, f64
from tests.test_gpu_stack import _build, _f64b, _stack_inputs

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


class I8Layer:
    def __init__(self, stp, ctx, T, D, F, V, seed=1):
        import torch

        from token_indexed_sparse_staple_b200.stack import LayerWeights, quantise_layer
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def rnd(*s, std):
            return (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.stp, self.ctx, self.T, self.D, self.F, self.V = stp, ctx, T, D, F, V
        self.x = rnd(T, D, std=1.0)
        w = LayerWeights(rnd(F, D, std=D ** -0.5), rnd(F, D, std=D ** -0.5), rnd(D, F, std=F ** -0.5))
        self.q = quantise_layer(ctx, w)
        self.E = rnd(V, F, std=1.0)
        self.ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.y = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.wsb = stp.staple_ffn_i8_workspace_bytes(T, D, F)
        self.ws = torch.full((max(self.wsb, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def embed(self, mode, flags=0):
        s = self.stp
        return (s.make_embed(s.STAPLE_EMBED_NONE) if mode == "none" else
                s.make_embed(s.STAPLE_EMBED_TABLE, self.E, self.F, self.ids, self.V, flags))

    def run(self, embed, x=None, y=None, stream=None):
        q = self.q
        self.stp.staple_ffn_fwd_i8(self.ctx, self.T, self.D, self.F, self.x if x is None else x,
                                   embed, q.w_gate_up, q.gate_up_scale, q.w_down, q.down_scale,
                                   self.y if y is None else y, self.ws, self.wsb, stream=stream)

    def check(self, e_on: bool, stem: bool):
        """The definition with its roundings, as intervals.  Up to its rounding
        to bf16, g (and u) is a sum of integers rounded to fp32 and multiplied
        twice: off by 3 * 2^-24.  SiLU by the fast exponential (2 + 1.2 |g| fp32
        steps) and the fast division (2 steps), under 2^-18 for |g| < 20.  An
        interval that straddles a rounding boundary takes in both sides; all
        others collapse.  The row's scale and the integers follow, and y is off
        by the integers' intervals and its own rounding (2^-8 and 4 * 2^-24)."""
        def bf16(v):
            return f64(_to_bf16(v))

        def widen(lo, hi, rel):
            return lo - rel * np.abs(lo), hi + rel * np.abs(hi)

        eps = 2.0 ** -18
        xq, xs = bo.quant_rows(self.x.float().cpu().numpy())
        gu = bo.matmul_i8(xq, xs, f64(self.q.w_gate_up), f64(self.q.gate_up_scale))
        wd = f64(self.q.w_down) * f64(self.q.down_scale)[:, None]
        e = f64(self.E)[self.ids.cpu().numpy()] if e_on else 0.0

        def z_interval(e):
            g, u = gu[:, :self.F], gu[:, self.F:]
            assert np.abs(g).max() < 20
            glo, ghi = (bf16(v) for v in widen(g, g, 3 * 2.0 ** -24))
            hlo = hhi = e + np.zeros_like(g)
            if not stem:
                ulo, uhi = (bf16(v) for v in widen(u, u, 3 * 2.0 ** -24))
                r = 2.0 ** -23 * (np.abs(u) + np.abs(e))
                hlo, hhi = ulo + e - r, uhi + e + r
            silu = np.stack([v / (1 + np.exp(-v)) for v in (glo, ghi)])
            slo, shi = widen(silu.min(axis=0), silu.max(axis=0), eps)
            c = np.stack([slo * hlo, slo * hhi, shi * hlo, shi * hhi])
            return tuple(bf16(v) for v in widen(c.min(axis=0), c.max(axis=0), 2.0 ** -23))

        zlo, zhi = z_interval(e)
        small = np.where(zlo * zhi <= 0, 0.0, np.minimum(np.abs(zlo), np.abs(zhi)))
        big = np.maximum(np.abs(zlo), np.abs(zhi))
        s = np.stack([m.max(axis=1, keepdims=True).astype(np.float32) / np.float32(127)
                      for m in (small, big)]).astype(np.float64)
        q = np.clip(np.rint(np.stack([zlo / s[0], zlo / s[1], zhi / s[0], zhi / s[1]])), -127, 127)
        v = np.stack([q * s[0], q * s[1]]).reshape(8, *zlo.shape)
        vlo, vhi = v.min(axis=0), v.max(axis=0)
        y = (vlo + vhi) / 2 @ wd.T
        radius = (vhi - vlo) / 2 @ np.abs(wd).T
        tol = radius + (2.0 ** -8 + 4 * 2.0 ** -24) * (np.abs(y) + radius) + 1e-12
        got = f64(self.y)
        assert np.isfinite(got).all()
        bad = np.abs(got - y) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(got - y) / tol).max()))
        # the check can tell the layer without its rows from the layer with them
        if e_on and not stem:
            zl, zh = z_interval(0.0 * e)
            assert (np.abs((zl + zh) / 2 @ wd.T - y) > tol).mean() > 0.5


def _to_bf16(v):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v)).to(torch.bfloat16)


@pytest.mark.parametrize("T, D, F", [(1, 64, 128), (1, 2048, 8192), (64, 512, 1040), (17, 1040, 272),
                                     (300, 256, 512), (700, 512, 2048), (64, 4096, 11008)])
def test_i8_layer(stp, ctx, T, D, F):
    m = I8Layer(stp, ctx, T, D, F, V=50)
    m.run(m.embed("table"))
    m.check(True, False)
    m.run(m.embed("none"))
    m.check(False, False)
    m.run(None)
    m.check(False, False)
    m.run(m.embed("table", stp.STAPLE_EMBED_REPLACE_UP))
    m.check(True, True)
    # in place
    x = m.x.clone()
    m.run(m.embed("table"))
    m.run(m.embed("table"), x=x, y=x)
    import torch
    assert torch.equal(x, m.y)
    assert stp.staple_get_error(ctx) == 0


def test_i8_layer_reports_an_id_out_of_range(stp, ctx):
    import torch
    m = I8Layer(stp, ctx, 40, 128, 256, V=10)
    m.ids[7] = 10
    m.run(m.embed("table"))
    assert stp.staple_get_error(ctx) == stp.STAPLE_EIDRANGE
    m.ids[7] = 3
    m.run(m.embed("table"))
    torch.cuda.synchronize()
    m.check(True, False)
    assert stp.staple_get_error(ctx) == 0


def test_i8_layer_keeps_a_bad_row_to_itself(stp, ctx):
    import torch
    m = I8Layer(stp, ctx, 30, 128, 256, V=10)
    m.run(m.embed("table"))
    good = m.y.clone()
    m.x[5, 3] = float("nan")
    m.x[9, 0] = float("inf")
    m.run(m.embed("table"))
    rows = torch.ones(30, dtype=torch.bool, device="cuda")
    rows[5], rows[9] = False, False
    assert torch.equal(m.y[rows], good[rows])
    assert torch.isnan(m.y[~rows]).all()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,D,F", [(1, 256, 512), (1, 1024, 8192), (7, 1024, 2048)])
def test_i8_layer_reads_weights_written_just_before_it(stp, ctx, T, D, F, graph):
    """The layer's kernels start early and may load weights early; weights that the
    work in front of the call writes on the same stream are still the ones read."""
    import torch
    a, b = (I8Layer(stp, ctx, T, D, F, 64, seed=s) for s in (1, 2))
    e = a.embed("table")
    names = ("w_gate_up", "gate_up_scale", "w_down", "down_scale")
    want, saved = [], [{n: getattr(l.q, n).clone() for n in names} for l in (a, b)]
    for s in saved:
        for n in names:
            getattr(a.q, n).copy_(s[n])
        torch.cuda.synchronize()
        a.run(e)
        torch.cuda.synchronize()
        want.append(a.y.clone())
    assert not torch.equal(*want)
    got = torch.full((8, T, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def alternate(stream):
        for i in range(8):
            for n in names:
                getattr(a.q, n).copy_(saved[i % 2][n])
            a.run(e, y=got[i], stream=stream)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                alternate(st)
            g.replay()
        else:
            alternate(st)
    torch.cuda.synchronize()
    for i in range(8):
        assert torch.equal(got[i], want[i % 2])


@pytest.mark.parametrize("i8, norms", [(False, True), (True, False), (True, True)])
def test_decode_stack_runs_the_same_operators(stp, ctx, i8, norms):
    """A captured step of the stack equals the same public calls made one by
    one, bit for bit; each of those is checked against its definition in its
    own test, and so is a layer of the step here."""
    import torch

    from token_indexed_sparse_staple_b200.stack import DecodeStack, NormWeights, quantise_layer
    L, G, T, D, F, V = 4, 4, 33, 128, 256, 1000
    layers, groups = _stack_inputs(L, G, D, F, V)
    freq = syn.calibration_freq(V, n_tokens=1 << 18)
    W, tables = _build(stp, ctx, layers, groups, V, F, G, freq)
    try:
        W8 = [quantise_layer(ctx, w) if i8 and l % 2 == 0 else w for l, w in enumerate(W)]
        nw = None
        if norms:
            nw = [NormWeights(dev(syn.bf16_normal((D,), 0.3, 900 + l)[0], "bf16"),
                              dev(syn.bf16_normal((D,), 0.3, 910 + l)[0], "bf16"),
                              stp.STAPLE_NORM_LAYER if l % 2 else stp.STAPLE_NORM_RMS)
                  for l in range(L)]
        s = DecodeStack(ctx, W8, tables, T, D, F, V, norms=nw)
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            s.run(st)
        torch.cuda.synchronize()
        s.capture(st)
        for rep in range(2):
            ids = syn.zipf_ids(T, V, 1.1, seed=80 + rep)
            s.ids_buf.copy_(torch.from_numpy(ids))
            s.xs[0].copy_(dev(syn.bf16_normal((T, D), 1.0, 90 + rep)[0], "bf16"))
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                s.replay()
            torch.cuda.synchronize()
            assert stp.staple_get_error(ctx) == 0
            x = s.xs[0]
            n, y = torch.empty_like(x), torch.empty_like(x)
            for l in range(L):
                inp = x
                if norms:
                    stp.staple_norm_fwd(ctx, stp.STAPLE_BF16, nw[l].kind, T, D, x, n,
                                        weight=nw[l].weight, bias=nw[l].bias, eps=nw[l].eps)
                    inp = n
                if i8 and l % 2 == 0:
                    q = W8[l]
                    stp.staple_ffn_fwd_i8(ctx, T, D, F, inp, s.r.embed(l), q.w_gate_up,
                                          q.gate_up_scale, q.w_down, q.down_scale, y, s.ws8, s.wsb8)
                else:
                    w = W[l]
                    stp.staple_ffn_fwd(ctx, stp.STAPLE_BF16, T, D, F, inp, s.r.embed(l), w.w_gate,
                                       w.w_up, w.w_down, s.z, y, None, None, s.ws, s.wsb)
                    fw = oracle.ffn_forward(f64(inp), ids, *(_f64b(a) for a in layers[l]))
                    assert_close(f64(y), fw["y"], TOL["bf16"], f"layer {l}")
                if norms:
                    nx = torch.empty_like(x)
                    stp.staple_dropout(ctx, stp.STAPLE_BF16, T, D, y, stp.make_drop(0.0, None), nx,
                                       residual=x)
                    x = nx
                else:
                    x = y.clone()
                assert torch.equal(x, s.xs[l + 1]), l
        s.release()
    finally:
        tables.close()


def test_layers_side_by_side_on_streams_of_their_own(stp, ctx):
    """8-bit layers of one token, of clusters and of tiles beside the bf16 decode
    kernel and a norm's backward pass: each gives what it gives alone."""
    import torch
    layers = [I8Layer(stp, ctx, T, D, F, 64, seed=T) for T, D, F in
              ((1, 1024, 4096), (64, 2048, 8192), (64, 1024, 12288), (200, 1024, 8192))]
    embeds = [m.embed("table") for m in layers]
    m = layers[1]
    T, D, F = m.T, m.D, m.F
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    wg, wu, wd = ((torch.randn(s, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
                  for s in ((F, D), (F, D), (D, F)))
    z = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    wsb = stp.staple_workspace_bytes(T, D, F)
    ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
    rows = 4000
    dy, s_in = ((torch.randn((rows, D), generator=g, device="cuda")).to(torch.bfloat16)
                for _ in range(2))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y0 = torch.empty_like(s_in)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    stp.staple_norm_fwd(ctx, stp.STAPLE_BF16, stp.STAPLE_NORM_LAYER, rows, D, s_in, y0, weight=w,
                        mean=mean, rstd=rstd)
    nwb = stp.staple_norm_workspace_bytes(rows, D)
    nws = torch.zeros(nwb, dtype=torch.uint8, device="cuda")
    dw, db = (torch.empty(D, device="cuda") for _ in range(2))
    dx = torch.empty_like(dy)
    bf_y = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")

    def bf16(st):
        stp.staple_ffn_fwd(ctx, stp.STAPLE_BF16, T, D, F, m.x, embeds[1], wg, wu, wd, z, bf_y, None,
                           None, ws, wsb, stream=st)

    def norm(st):
        stp.staple_norm_bwd(ctx, stp.STAPLE_BF16, stp.STAPLE_NORM_LAYER, rows, D, dy, s_in, rstd,
                            dx, mean=mean, weight=w, dw=dw, db=db, workspace=nws,
                            workspace_bytes=nwb, stream=st)

    jobs = [(lambda st, m=m, e=e: m.run(e, stream=st), m.y) for m, e in zip(layers, embeds)]
    jobs += [(bf16, bf_y), (norm, dx)]
    want = []
    for run, out in jobs:
        run(None)
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for _, out in jobs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(8):
            for (run, _), st in zip(jobs, streams):
                run(st)
        torch.cuda.synchronize()
        for (_, out), w0 in zip(jobs, want):
            assert torch.equal(out, w0)
    assert stp.staple_get_error(ctx) == 0


def test_train_stack_as_a_residual_stream(stp, ctx):
    import torch

    from token_indexed_sparse_staple_b200.stack import NormWeights, TrainStack
    L, G, T, D, F, V, p = 4, 2, 300, 128, 256, 1000, 0.2
    layers, groups = _stack_inputs(L, G, D, F, V)
    freq = syn.calibration_freq(V, n_tokens=1 << 18)
    W, tables = _build(stp, ctx, layers, groups, V, F, G, freq)
    try:
        nw = [NormWeights(dev(syn.bf16_normal((D,), 0.3, 900 + l)[0], "bf16"),
                          dev(syn.bf16_normal((D,), 0.3, 910 + l)[0], "bf16") if l % 2 else None,
                          stp.STAPLE_NORM_LAYER if l % 2 else stp.STAPLE_NORM_RMS)
              for l in range(L)]
        rng = torch.tensor([1234567, 0], dtype=torch.int64, device="cuda")
        s = TrainStack(ctx, W, tables, T, D, F, V, keep_dy=True, norms=nw, dropout=p, rng=rng)
        for step in range(2):
            ids = syn.zipf_ids(T, V, 1.1, seed=50 + step)
            x0 = dev(syn.bf16_normal((T, D), 1.0, 60 + step)[0], "bf16")
            dyt = dev(syn.bf16_normal((T, D), 1.0, 70 + step)[0], "bf16")
            r = s.step(torch.from_numpy(ids).cuda(), x0, dyt)
            s.host_ready.synchronize()
            torch.cuda.synchronize()
            assert stp.staple_get_error(ctx) == 0
            U, b, tol = int(r.U.item()), s.b, TOL["bf16"]
            offset = step * L
            fac = [bo.dropout_factors(T, D, p, 1234567, offset, l) for l in range(L)]
            dres = f64(dyt)
            for l in reversed(range(L)):
                x = f64(b.xs[l])
                nwt = f64(nw[l].weight)
                nb = None if nw[l].bias is None else f64(nw[l].bias)
                rms = nw[l].kind == stp.STAPLE_NORM_RMS
                n, mean, rstd = bo.norm_fwd(x, nwt, nb, nw[l].eps, rms)
                assert_close(f64(s.n[l]), n, tol, f"n {l}")
                wg, wu, wd, E = (_f64b(a) for a in layers[l])
                fw = oracle.ffn_forward(f64(s.n[l]), ids, wg, wu, wd, E)
                assert_close(f64(b.xs[l + 1]), x + fac[l] * fw["y"], tol, f"x {l + 1}")
                dy = f64(b.dy[l])
                assert_close(dy, fac[l] * dres, tol, f"dy {l}")
                bw = oracle.ffn_backward(dy, f64(s.n[l]), ids, wg, wu, wd, fw)
                assert_close(b.host_dE[l].numpy()[:U].astype(np.float64), bw["dE"], tol, f"dE {l}")
                assert_close(f64(b.dW[l][2]), bw["dW_down"], tol, f"dW_down {l}")
                ds, dw, db = bo.norm_bwd(bw["dx"], x, mean, rstd, nwt, rms)
                assert_close(f64(s.dnorm[l][0]), dw, tol, f"dnorm weight {l}")
                assert_close(f64(s.dnorm[l][1]), db, tol, f"dnorm bias {l}")
                assert_close(f64(s.dstream[l]), ds + dres, tol, f"stream gradient {l}")
                dres = f64(s.dstream[l])
            assert s.dx0.data_ptr() == s.dstream[0].data_ptr()
            rng[1] += L
    finally:
        tables.close()
