"""Argument checks of the operators around the layer, without a GPU: every bad
argument is refused before the device is touched.  The context is a block of
zeros that no refusal may look into; the same call with good arguments gets as
far as choosing the device and fails there (STAPLE_ECUDA), so a refusal that
went missing would show."""
import ctypes as C

import pytest

import token_indexed_sparse_staple_b200 as stp
from token_indexed_sparse_staple_b200 import _lib

OK_PTR, ODD = 0x10000, 0x10001     # never read: nothing launches
BF, F32 = stp.STAPLE_BF16, stp.STAPLE_F32


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the good calls would launch")
    from token_indexed_sparse_staple_b200 import build
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def ctx():
    buf = (C.c_uint8 * 4096)()
    yield C.addressof(buf)


def drop(p=0.1, rng=OK_PTR):
    return C.byref(_lib.staple_drop(p, 0, rng))


def check(fn, good: dict, bad: list):
    assert fn(*good.values()) == stp.STAPLE_ECUDA, "good arguments were refused"
    for change, want in bad:
        args = dict(good, **change)
        assert list(args) == list(good)
        assert fn(*args.values()) == want, change


E, U = stp.STAPLE_EINVAL, stp.STAPLE_EUNSUPPORTED
ROWS = [(dict(ctx=None), E), (dict(dtype=2), E), (dict(T=-1), E), (dict(D=0), E), (dict(D=-8), E)]


def test_norm_fwd(lib, ctx):
    good = dict(ctx=ctx, dtype=BF, kind=0, T=4, D=10, x=OK_PTR, residual=OK_PTR, drop=drop(),
                weight=OK_PTR, bias=None, eps=1e-5, sum=OK_PTR + 64, y=OK_PTR, mean=None,
                rstd=OK_PTR, stream=None)
    check(lib.staple_norm_fwd, good, ROWS + [
        (dict(kind=2), E), (dict(D=16385), U), (dict(x=None), E), (dict(y=None), E),
        (dict(x=ODD), E), (dict(weight=ODD), E), (dict(bias=ODD), E), (dict(residual=ODD), E),
        (dict(rstd=OK_PTR + 2), E), (dict(mean=ODD), E), (dict(sum=None), E),
        (dict(sum=None, residual=None), E), (dict(sum=None, drop=None), E),
        (dict(sum=OK_PTR), E),                       # sum is y
        (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(eps=float("inf")), E),
        (dict(drop=drop(-0.1)), E), (dict(drop=drop(1.5)), E), (dict(drop=drop(float("nan"))), E),
        (dict(drop=drop(0.1, None)), E), (dict(drop=drop(0.1, OK_PTR + 4)), E),
        (dict(T=0), stp.STAPLE_OK),
    ])
    # neither residual nor dropout: no sum is needed
    assert lib.staple_norm_fwd(*dict(good, residual=None, drop=drop(0.0, None),
                                     sum=None).values()) == stp.STAPLE_ECUDA


def test_norm_bwd(lib, ctx):
    ws = stp.staple_norm_workspace_bytes(4, 10)
    assert ws >= 4 * 2 * 10 * 4
    good = dict(ctx=ctx, dtype=F32, kind=0, T=4, D=10, dy=OK_PTR, s=OK_PTR, weight=None,
                mean=OK_PTR, rstd=OK_PTR, dsum_in=None, drop=drop(), dsum=OK_PTR, dx=OK_PTR + 64,
                dw=OK_PTR, db=OK_PTR, workspace=OK_PTR, wsb=ws, stream=None)
    check(lib.staple_norm_bwd, good, ROWS + [
        (dict(kind=-1), E), (dict(D=16385), U), (dict(dy=None), E), (dict(s=None), E),
        (dict(rstd=None), E), (dict(mean=None), E), (dict(mean=ODD), E), (dict(s=OK_PTR + 2), E),
        (dict(weight=ODD), E), (dict(dsum_in=ODD), E), (dict(dsum=ODD), E), (dict(dx=ODD), E),
        (dict(dw=ODD), E), (dict(db=ODD), E), (dict(dx=OK_PTR), E),
        (dict(dsum=None, dx=None, dw=None, db=None), E),
        (dict(workspace=None), E), (dict(workspace=OK_PTR + 4), E), (dict(wsb=4 * 2 * 10 * 4 - 1), E),
        (dict(drop=drop(2.0)), E),
    ])
    f = lib.staple_norm_bwd
    assert f(*dict(good, kind=1, mean=None).values()) == stp.STAPLE_ECUDA       # RMSNorm
    assert f(*dict(good, dw=None, db=None, workspace=None, wsb=0).values()) == stp.STAPLE_ECUDA


def test_norm_workspace_sizes(lib):
    w = stp.staple_norm_workspace_bytes
    assert w(0, 10) == 0 and w(-1, 10) == 0 and w(4, 0) == 0 and w(4, 16385) == 0
    assert w(1 << 20, 16384) == w(1 << 30, 16384)     # bounded by the blocks, not by T
    for T, D in ((1, 1), (7, 1001), (640, 64), (641, 64)):
        assert w(T, D) % 256 == 0 and w(T, D) >= min(T, 640) * 8 * D


def test_dropout(lib, ctx):
    good = dict(ctx=ctx, dtype=BF, T=4, D=100000, x=OK_PTR, residual=None, drop=drop(1.0),
                out=OK_PTR, stream=None)
    check(lib.staple_dropout, good, ROWS + [
        (dict(x=None), E), (dict(out=None), E), (dict(x=ODD), E), (dict(residual=ODD), E),
        (dict(drop=None), E), (dict(drop=drop(1.01)), E), (dict(drop=drop(0.5, None)), E),
        (dict(T=0), stp.STAPLE_OK),
    ])


def test_quant_rows(lib, ctx):
    good = dict(ctx=ctx, dtype=BF, T=4, D=32768, x=OK_PTR, q=ODD, scale=OK_PTR, stream=None)
    check(lib.staple_quant_rows, good, ROWS + [
        (dict(D=32769), U), (dict(x=None), E), (dict(q=None), E), (dict(scale=None), E),
        (dict(x=ODD), E), (dict(scale=OK_PTR + 2), E), (dict(T=0), stp.STAPLE_OK),
    ])


def test_matmul_i8(lib, ctx):
    good = dict(ctx=ctx, dtype=F32, T=3, N=5, K=32, a=OK_PTR, a_scale=OK_PTR, b=OK_PTR,
                b_scale=OK_PTR + 4, y=OK_PTR + 4, stream=None)
    check(lib.staple_matmul_i8, good, [
        (dict(ctx=None), E), (dict(dtype=2), E), (dict(T=-1), E), (dict(N=0), E), (dict(N=-1), E),
        (dict(K=0), E), (dict(K=8), E), (dict(K=-16), E), (dict(K=33), E), (dict(K=131072), U),
        (dict(a=None), E), (dict(b=None), E), (dict(a_scale=None), E), (dict(b_scale=None), E),
        (dict(y=None), E), (dict(a=OK_PTR + 8), E), (dict(b=ODD), E), (dict(a_scale=OK_PTR + 2), E),
        (dict(b_scale=ODD), E), (dict(y=OK_PTR + 2), E), (dict(T=0), stp.STAPLE_OK),
    ])


def test_ffn_fwd_i8(lib, ctx):
    ws = stp.staple_ffn_i8_workspace_bytes(5, 32, 48)
    assert ws >= 5 * (32 + 2 * 48 * 2 + 48 + 8) and ws % 256 == 0
    w = stp.staple_ffn_i8_workspace_bytes
    assert w(-1, 32, 48) == 0 and w(5, 8, 48) == 0 and w(5, 32, 40) == 0 and w(5, 32784, 48) == 0
    e = stp.make_embed(stp.STAPLE_EMBED_TABLE, OK_PTR, 48, OK_PTR, 10)
    good = dict(ctx=ctx, T=5, D=32, F=48, x=OK_PTR, embed=C.byref(e), w_gate_up=OK_PTR, gus=OK_PTR,
                w_down=OK_PTR, ds=OK_PTR + 4, y=OK_PTR, workspace=OK_PTR, wsb=ws, stream=None)
    bad_pitch = stp.make_embed(stp.STAPLE_EMBED_TABLE, OK_PTR, 40, OK_PTR, 10)
    bad_base = stp.make_embed(stp.STAPLE_EMBED_TABLE, OK_PTR + 2, 48, OK_PTR, 10)
    stem_none = stp.make_embed(stp.STAPLE_EMBED_NONE, flags=stp.STAPLE_EMBED_REPLACE_UP)
    check(lib.staple_ffn_fwd_i8, good, [
        (dict(ctx=None), E), (dict(T=-1), E), (dict(D=24), E), (dict(F=40), E), (dict(F=0), E),
        (dict(D=32784), U), (dict(F=32784), U), (dict(x=None), E), (dict(x=OK_PTR + 8), E),
        (dict(y=None), E), (dict(w_gate_up=None), E), (dict(w_down=OK_PTR + 4), E),
        (dict(gus=None), E), (dict(ds=ODD), E), (dict(workspace=None), E),
        (dict(workspace=OK_PTR + 16), E), (dict(wsb=ws - 1), E), (dict(embed=C.byref(bad_pitch)), E),
        (dict(embed=C.byref(bad_base)), E), (dict(embed=C.byref(stem_none)), E),
        (dict(T=0), stp.STAPLE_OK),
    ])
    assert lib.staple_ffn_fwd_i8(*dict(good, embed=None).values()) == stp.STAPLE_ECUDA
