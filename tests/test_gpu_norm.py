"""The norm with residual add and dropout in front of it, its backward pass,
and dropout on its own, against their fp64 definitions on the same inputs.

Tolerances, with u = 2^-24 (half a step of fp32) and h = half a step of the
output type (bf16 2^-8, fp32 2^-24), relative to the value: an output is off by
at most h |value| for its rounding, plus the fp32 arithmetic before it.  A sum
over a row is taken in at most 32 adds per thread, 5 across a warp and 16
across warps, so it is off by at most 53 u times the sum of the absolute
values; with the few roundings of the terms themselves, 64 u covers each sum
and each chain of products below."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-5


@pytest.fixture(scope="module")
def stp():
    import token_indexed_sparse_staple_b200 as m
    return m


@pytest.fixture(scope="module")
def ctx(stp):
    c = stp.staple_context_create(0)
    yield c
    stp.staple_context_destroy(c)


def tdt(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def rnd(shape, dtype, seed, std=1.0, mean=0.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(tdt(dtype))


def np64(t):
    return t.detach().double().cpu().numpy()


def rng_state(seed=0x0123456789ABCDEF, offset=5):
    import torch
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def within(got, want, tol, what):
    err = np.abs(got - want)
    assert np.isfinite(got).all(), what
    bad = err > tol
    assert not bad.any(), (what, int(bad.sum()), float((err / np.maximum(tol, 1e-300)).max()))


class Norm:
    """One forward and backward pass with every optional piece chosen."""

    def __init__(self, stp, ctx, T, D, dtype, rms, add, p, affine, seed=1, offset_elems=0):
        import torch
        self.stp, self.ctx, self.T, self.D, self.dtype, self.rms = stp, ctx, T, D, dtype, rms
        self.dt = stp.STAPLE_BF16 if dtype == "bf16" else stp.STAPLE_F32
        self.kind = stp.STAPLE_NORM_RMS if rms else stp.STAPLE_NORM_LAYER
        self.p, self.site = p, 3
        self.rng = rng_state()
        self.drop = stp.make_drop(p, self.rng, self.site) if p > 0 else None

        def place(t):
            # the same values at an address that is only element-aligned
            if not offset_elems:
                return t
            buf = torch.empty(t.numel() + offset_elems, dtype=t.dtype, device="cuda")
            v = buf[offset_elems:].view(t.shape)
            v.copy_(t)
            return v

        self.x = place(rnd((T, D), dtype, seed))
        self.res = place(rnd((T, D), dtype, seed + 1, 1.5, 0.2)) if add else None
        self.w = place(rnd(D, dtype, seed + 2, 0.2, 1.0)) if affine else None
        self.b = place(rnd(D, dtype, seed + 3, 0.2)) if affine else None
        self.dy = place(rnd((T, D), dtype, seed + 4, 0.5))
        self.dsum_in = place(rnd((T, D), dtype, seed + 5, 0.5)) if add else None
        new = lambda *s, d=tdt(dtype): torch.full(s, float("nan"), dtype=d, device="cuda")
        f32 = torch.float32
        self.y = place(new(T, D))
        self.sum = place(new(T, D)) if add or p > 0 else None
        self.mean, self.rstd = new(T, d=f32), new(T, d=f32)
        self.dsum, self.dx = place(new(T, D)), place(new(T, D))
        self.dw, self.db = new(D, d=f32), new(D, d=f32)
        self.wsb = stp.staple_norm_workspace_bytes(T, D)
        self.ws = torch.full((max(self.wsb, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def fwd(self, stream=None):
        self.stp.staple_norm_fwd(self.ctx, self.dt, self.kind, self.T, self.D, self.x, self.y,
                                 weight=self.w, bias=self.b, eps=EPS, residual=self.res,
                                 drop=self.drop, sum=self.sum, mean=self.mean, rstd=self.rstd,
                                 stream=stream)

    def bwd(self, stream=None):
        s = self.sum if self.sum is not None else self.x
        self.stp.staple_norm_bwd(self.ctx, self.dt, self.kind, self.T, self.D, self.dy, s,
                                 self.rstd, self.dsum, mean=self.mean, weight=self.w,
                                 dsum_in=self.dsum_in, drop=self.drop, dx=self.dx, dw=self.dw,
                                 db=self.db, workspace=self.ws, workspace_bytes=self.wsb,
                                 stream=stream)

    def factors(self):
        seed, offset = (int(v) & (2 ** 64 - 1) for v in self.rng.cpu().tolist())
        return bo.dropout_factors(self.T, self.D, self.p, seed, offset, self.site)

    def check_fwd(self):
        h = HALF[self.dtype]
        x = np64(self.x)
        if self.sum is not None:
            f = self.factors() if self.p > 0 else 1.0
            res = np64(self.res) if self.res is not None else 0.0
            s = np64(self.sum)
            want = res + x * f
            # scale and product rounded in fp32 (3 u), the add (u), the storage
            within(s, want, h * np.abs(want) + 4 * U * (np.abs(x * f) + np.abs(res)), "sum")
        else:
            s = x
        w, b = (None if t is None else np64(t) for t in (self.w, self.b))
        y, mean, rstd = bo.norm_fwd(s, w, b, EPS, self.rms)
        m1 = np.abs(s).mean(axis=1)
        within(np64(self.mean), mean, 64 * U * m1, "mean")
        c = np.abs(s - mean[:, None])
        # the variance's terms carry the mean's error: d(var) <= 2 |c| 64 u m1, averaged
        dvar = 64 * U * ((c * c).mean(axis=1) + 2 * c.mean(axis=1) * m1 + EPS)
        within(np64(self.rstd), rstd, rstd * (dvar * rstd ** 2 + 4 * U), "rstd")
        aw = 1.0 if w is None else np.abs(w)
        core = np.abs(y - (0.0 if b is None else b))
        tol = (h * np.abs(y) + aw * rstd[:, None] * 64 * U * m1[:, None]
               + core * ((dvar * rstd ** 2)[:, None] + 8 * U) + 2 * U * np.abs(y))
        within(np64(self.y), y, tol, "y")

    def check_bwd(self):
        h = HALF[self.dtype]
        s = np64(self.sum if self.sum is not None else self.x)
        dy, mean, rstd = np64(self.dy), np64(self.mean), np64(self.rstd)
        w = None if self.w is None else np64(self.w)
        ds, dw, db = bo.norm_bwd(dy, s, mean, rstd, w, self.rms)
        mu = 0.0 if self.rms else mean[:, None]
        xh = np.abs((s - mu) * rstd[:, None])
        gw = np.abs(dy if w is None else dy * w)
        tol = 64 * U * rstd[:, None] * (gw + (0 if self.rms else gw.mean(axis=1, keepdims=True))
                                        + xh * (gw * xh).mean(axis=1, keepdims=True))
        if self.dsum_in is not None:
            a = np64(self.dsum_in)
            ds = ds + a
            tol = tol + U * (np.abs(a) + np.abs(ds))
        within(np64(self.dsum), ds, h * np.abs(ds) + tol * (1 + h), "dsum")
        f = self.factors() if self.p > 0 else 1.0
        within(np64(self.dx), ds * f, h * np.abs(ds * f) + f * (tol * (1 + h) + 3 * U * np.abs(ds)),
               "dx")
        # dw, db: rows add up one after another in a block (at least
        # min(T, 148) row groups share them), over at most 256 row groups of a
        # block, 80 blocks and 8 slices; xhat and the product add 4 u
        n = -(-self.T // 148) + 8 + 256 + 80 + 8
        within(np64(self.dw), dw, (n + 4) * U * (np.abs(dy) * xh).sum(axis=0), "dw")
        within(np64(self.db), db, (n + 4) * U * np.abs(dy).sum(axis=0), "db")


SHAPES = [(1, 1), (2, 2), (1, 8), (3, 7), (5, 64), (4099, 24), (257, 100), (2, 4096), (33, 2048),
          (64, 4096), (300, 2561), (700, 1023), (1, 5000), (17, 8192), (9, 12288), (3, 16384),
          (2, 16383), (1200, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, D", SHAPES)
def test_forward_and_backward(stp, ctx, T, D, dtype):
    # every optional piece on, then off; LayerNorm and RMSNorm
    for rms, add, p, affine in ((False, True, 0.1, True), (True, False, 0.0, False),
                                (True, True, 0.0, True), (False, False, 0.5, False)):
        n = Norm(stp, ctx, T, D, dtype, rms, add, p, affine, seed=T + D)
        n.fwd()
        n.check_fwd()
        n.bwd()
        n.check_bwd()
    assert stp.staple_get_error(ctx) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_element_aligned_pointers(stp, ctx, dtype):
    n = Norm(stp, ctx, 37, 512, dtype, False, True, 0.2, True, offset_elems=1)
    n.fwd()
    n.check_fwd()
    n.bwd()
    n.check_bwd()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [256, 101])
def test_outputs_may_share_the_inputs_memory(stp, ctx, dtype, D):
    a = Norm(stp, ctx, 50, D, dtype, False, True, 0.1, True)
    a.fwd()
    a.bwd()
    b = Norm(stp, ctx, 50, D, dtype, False, True, 0.1, True)
    b.sum, b.y = b.res, b.x
    b.fwd()
    b.dsum, b.dx = b.dsum_in, b.dy
    b.bwd()
    import torch
    for k in ("sum", "y", "mean", "rstd", "dsum", "dx", "dw", "db"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_runs_repeat_bit_for_bit_and_streams_do_not_matter(stp, ctx):
    import torch
    a = Norm(stp, ctx, 3000, 1024, "bf16", False, True, 0.1, True)
    a.fwd()
    a.bwd()
    torch.cuda.synchronize()
    first = {k: getattr(a, k).clone() for k in ("sum", "y", "dsum", "dx", "dw", "db")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for k in first:
        getattr(a, k).fill_(float("nan"))
    s.wait_stream(torch.cuda.current_stream())
    a.fwd(stream=s)
    a.bwd(stream=s)
    torch.cuda.synchronize()
    for k, v in first.items():
        assert torch.equal(getattr(a, k), v), k


def test_two_streams_with_their_own_workspaces(stp, ctx):
    import torch
    pair = [Norm(stp, ctx, 2000, 768, "bf16", r, True, 0.1, True, seed=9 + r) for r in (0, 1)]
    st = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(5):
        for n, s in zip(pair, st):
            n.fwd(stream=s)
            n.bwd(stream=s)
    torch.cuda.synchronize()
    for n in pair:
        n.check_fwd()
        n.check_bwd()


def test_captured_graph_draws_new_masks_when_the_offset_moves(stp, ctx):
    import torch
    n = Norm(stp, ctx, 130, 200, "bf16", False, True, 0.3, True)
    n.fwd()
    n.bwd()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        n.fwd(stream=s)
        n.bwd(stream=s)
    masks = []
    for _ in range(3):
        n.rng[1] += 1
        g.replay()
        torch.cuda.synchronize()
        n.check_fwd()
        n.check_bwd()
        masks.append((n.dx == 0).clone())
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])


def test_empty_batch(stp, ctx):
    import torch
    dw, db = (torch.full((16,), float("nan"), device="cuda") for _ in range(2))
    stp.staple_norm_fwd(ctx, stp.STAPLE_BF16, stp.STAPLE_NORM_LAYER, 0, 16, None, None)
    stp.staple_norm_bwd(ctx, stp.STAPLE_BF16, stp.STAPLE_NORM_LAYER, 0, 16, None, None, None, None,
                        dw=dw, db=db)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


def test_rows_beside_the_batch_stay_as_they_were(stp, ctx):
    import torch
    for dtype, D in (("bf16", 72), ("f32", 45)):
        n = Norm(stp, ctx, 21, D, dtype, False, True, 0.1, True)
        guard = {}
        for k in ("y", "sum", "dsum", "dx"):
            buf = torch.full((23, D), 7.0, dtype=tdt(dtype), device="cuda")
            guard[k] = buf
            setattr(n, k, buf[1:22])
        n.fwd()
        n.check_fwd()
        n.bwd()
        n.check_bwd()
        for k, buf in guard.items():
            assert (buf[0] == 7).all() and (buf[22] == 7).all(), k


def test_a_nan_or_infinity_stays_in_its_row(stp, ctx):
    import torch
    n = Norm(stp, ctx, 40, 96, "f32", False, True, 0.0, True)
    n.x[3, 5] = float("nan")
    n.x[8, 95] = float("inf")
    n.fwd()
    bad = ~torch.isfinite(n.y).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [3, 8]
    # what dropout drops is zero whatever it held
    x = torch.full((4, 64), float("nan"), device="cuda")
    out = torch.empty_like(x)
    stp.staple_dropout(ctx, stp.STAPLE_F32, 4, 64, x, stp.make_drop(1.0, rng_state()), out)
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, D", [(1, 1), (3, 8), (257, 1001), (64, 4096), (5, 100000), (1000, 24)])
@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 1.0])
def test_dropout(stp, ctx, T, D, dtype, p):
    import torch
    dt = stp.STAPLE_BF16 if dtype == "bf16" else stp.STAPLE_F32
    x, res = rnd((T, D), dtype, 4), rnd((T, D), dtype, 5)
    rng = rng_state(-3, (1 << 62) + 1)
    drop = stp.make_drop(p, rng, 9)
    f = bo.dropout_factors(T, D, p, 2 ** 64 - 3, (1 << 62) + 1, 9)
    for residual in (None, res):
        out = torch.full_like(x, float("nan"))
        stp.staple_dropout(ctx, dt, T, D, x, drop, out, residual=residual)
        a = np64(x) * f
        r = 0.0 if residual is None else np64(residual)
        within(np64(out), a + r, HALF[dtype] * np.abs(a + r) + 4 * U * (np.abs(a) + np.abs(r)),
               "out")
    # in place
    y = x.clone()
    stp.staple_dropout(ctx, dt, T, D, y, drop, y, residual=res)
    assert torch.equal(y, out)


def test_dropout_gradient_against_differences(stp, ctx):
    """out is linear in x, so the difference over a step of 1 is the gradient."""
    import torch
    T, D = 6, 40
    drop = stp.make_drop(0.4, rng_state(), 1)
    x, res, dout = (rnd((T, D), "f32", s) for s in (1, 2, 3))
    dx = torch.empty_like(x)
    stp.staple_dropout(ctx, stp.STAPLE_F32, T, D, dout, drop, dx)
    outs = []
    for step in (0.0, 1.0):
        o = torch.empty_like(x)
        stp.staple_dropout(ctx, stp.STAPLE_F32, T, D, x + step, drop, o, residual=res)
        outs.append(np64(o))
    grad = (outs[1] - outs[0]) * np64(dout)
    # each out is a sum of terms below 16, rounded a few times in fp32
    within(np64(dx), grad, 64 * U * 16 * np.abs(np64(dout)), "dx")


def test_kernel_gradient_against_differences(stp, ctx):
    """ds of the fp32 kernel against central differences of its own forward
    pass.  The two differ by the truncation of the difference, which the fp64
    definition gives at the same step, and by the rounding of y over the step:
    each y is off by at most 200 u max(1, |y|, |w| rstd mean|s|)."""
    T, D, h = 4, 24, 2.0 ** -6
    n = Norm(stp, ctx, T, D, "f32", False, False, 0.0, True)
    n.fwd()
    n.bwd()
    ds, dy, x0, w, b = np64(n.dsum), np64(n.dy), n.x.clone(), np64(n.w), np64(n.b)
    y0, m1 = np64(n.y), np.abs(np64(x0)).mean(axis=1, keepdims=True)
    ty = 200 * U * np.maximum(np.maximum(1.0, np.abs(y0) + 2 * h * np.abs(w)),
                              np.abs(w) * np64(n.rstd)[:, None] * m1 * 2)
    rounding = (ty * np.abs(dy)).sum(axis=1) / h
    got, trunc = np.empty((T, D)), np.empty((T, D))
    for d in range(D):
        ys, ref = [], []
        for sgn in (1, -1):
            n.x.copy_(x0)
            n.x[:, d] += sgn * h
            n.fwd()
            ys.append((np64(n.y) * dy).sum(axis=1))
            ref.append((bo.norm_fwd(np64(n.x), w, b, EPS)[0] * dy).sum(axis=1))
        got[:, d] = (ys[0] - ys[1]) / (2 * h)
        trunc[:, d] = (ref[0] - ref[1]) / (2 * h)
    exact = bo.norm_bwd(dy, np64(x0), np64(n.mean), np64(n.rstd), w)[0]
    within(got, ds, np.abs(trunc - exact) + rounding[:, None] + 1e-5, "ds")
    assert rounding.max() < 0.1 * np.abs(ds).max()     # the test can tell
