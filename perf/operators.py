"""The operators around the FFN layer of a transformer block, as timed cases.

Training:  s = residual + dropout(x), y = norm(s), and the backward pass of
both, with dropout from a counter-based generator whose mask is never stored.
Serving:   the same norm for a few tokens, rows quantised to 8-bit integers
with one scale each, and the product of such rows with 8-bit weights.

own = False: the operators' plain form in elementary torch operations.
own = True:  the calls a user makes of token_indexed_sparse_staple_b200.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a single new token's norm between two layers of a decode step
        {"name": "norm_fwd_one_token", "op": "norm_fwd", "kind": "layer", "dtype": "bf16",
         "T": 1, "D": 4096, "p": 0.0, "add": True, "bias": True, "stats": False},
        # the training step of the 1B-shaped layer: 4 x 4096 tokens, residual and dropout
        {"name": "norm_fwd_train", "op": "norm_fwd", "kind": "rms", "dtype": "bf16",
         "T": 16384, "D": 2048, "p": 0.1, "add": True, "bias": False, "stats": True},
        # a ragged fp32 batch with a row length that no vector load divides
        {"name": "norm_fwd_odd_f32", "op": "norm_fwd", "kind": "layer", "dtype": "f32",
         "T": 1537, "D": 1023, "p": 0.0, "add": False, "bias": True, "stats": True},
        # the backward pass of the 1B-shaped training step, residual and dropout
        {"name": "norm_bwd_train", "op": "norm_bwd", "kind": "layer", "dtype": "bf16",
         "T": 16384, "D": 2048, "p": 0.1, "add": True, "bias": True},
        # a short fp32 fine-tuning batch with odd sizes
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "kind": "rms", "dtype": "f32",
         "T": 333, "D": 2561, "p": 0.0, "add": False, "bias": False},
        # dropout and residual after the FFN of a training step at the 7B width
        {"name": "dropout_train", "op": "dropout", "dtype": "bf16",
         "T": 8192, "D": 4096, "p": 0.1, "add": True},
        # the gradient of a small odd batch: the same mask applied to it
        {"name": "dropout_odd_f32", "op": "dropout", "dtype": "f32",
         "T": 257, "D": 1001, "p": 0.25, "add": False},
        # a decode batch's activations before an 8-bit product
        {"name": "quant_decode", "op": "quant_rows", "dtype": "bf16", "T": 64, "D": 4096},
        # a prompt's FFN activations at the 1B width of d_ff
        {"name": "quant_prompt", "op": "quant_rows", "dtype": "bf16", "T": 16384, "D": 8192},
        # one new token times the 1B-shaped up-projection
        {"name": "matmul_i8_one_token", "op": "matmul_i8", "dtype": "bf16",
         "T": 1, "N": 8192, "K": 2048},
        # a decode batch times the 7B-shaped gate projection
        {"name": "matmul_i8_decode", "op": "matmul_i8", "dtype": "bf16",
         "T": 64, "N": 11008, "K": 4096},
        # a prompt batch times the 1B-shaped gate projection
        {"name": "matmul_i8_prompt", "op": "matmul_i8", "dtype": "bf16",
         "T": 16384, "N": 8192, "K": 2048},
    ]


_MAX_ELEMS = {"norm_fwd": 1 << 25, "norm_bwd": 1 << 25, "dropout": 1 << 25, "quant_rows": 1 << 27}
_MAX_MACS = 16384 * 8192 * 2048


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "dropout", "quant_rows", "matmul_i8"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "matmul_i8":
        K = 16 * _log(rng, 1, 700)
        N = _log(rng, 1, 16384)
        T = min(_log(rng, 1, 16384), max(1, _MAX_MACS // (K * N)))
        return {"op": op, "dtype": dtype, "T": T, "N": N, "K": K}
    D = _log(rng, 1, 12288)
    if rng.random() < 0.5:
        D = max(8, D // 8 * 8)
    T = min(_log(rng, 1, 32768), _MAX_ELEMS[op] // D // (1 if dtype == "bf16" else 2))
    case = {"op": op, "dtype": dtype, "T": T, "D": D}
    if op == "quant_rows":
        return case
    case["add"] = rng.random() < 0.6
    case["p"] = rng.choice([0.0, 0.1, 0.25, 0.5]) if op != "dropout" else rng.choice([0.1, 0.25, 0.5])
    if op in ("norm_fwd", "norm_bwd"):
        case["kind"] = rng.choice(["layer", "rms"])
        case["bias"] = rng.random() < 0.5
    if op == "norm_fwd":
        case["stats"] = rng.random() < 0.7
    return case


EPS = 1e-5


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(*shape, dtype=_DT[case["dtype"]], std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    op, T = case["op"], case["T"]
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if op == "matmul_i8":
        N, K = case["N"], case["K"]
        for name, rows, std in (("a", T, 1.0), ("b", N, 0.02)):
            v = torch.randn((rows, K), generator=g, device="cuda") * std
            s = v.abs().amax(dim=1) / 127.0
            st[name] = torch.round(v / s[:, None]).clamp(-127, 127).to(torch.int8)
            st[name + "_scale"] = s
            del v
        st["y"] = torch.empty((T, N), dtype=dt, device="cuda")
    elif op == "quant_rows":
        D = case["D"]
        x = torch.randn((T, D), generator=g, device="cuda")
        # some channels of real activations are much larger than the rest
        x *= torch.where(torch.rand(D, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        st["x"] = x.to(dt)
        st["q"] = torch.empty((T, D), dtype=torch.int8, device="cuda")
        st["scale"] = torch.empty(T, dtype=torch.float32, device="cuda")
    else:
        D = case["D"]
        st["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % (1 << 62), 7 + 12 * (seed % 1000)],
                                 dtype=torch.int64, device="cuda")
        st["site"] = seed % 5
        if op != "dropout":
            st["weight"] = rnd(D, std=0.1, mean=1.0)
            st["bias"] = rnd(D, std=0.1) if case["bias"] else None
        if op == "norm_bwd":
            st["dy"] = rnd(T, D, std=0.01)
            st["sum"] = rnd(T, D, std=1.5, mean=0.1)
            st["dsum_in"] = rnd(T, D, std=0.01) if case["add"] else None
            s = st["sum"].float()
            mean = s.mean(dim=1) if case["kind"] == "layer" else torch.zeros(T, device="cuda")
            var = ((s - mean[:, None]) ** 2).mean(dim=1)
            st["mean"], st["rstd"] = mean, 1.0 / torch.sqrt(var + EPS)
            st["dsum"] = torch.empty((T, D), dtype=dt, device="cuda")
            st["dx"] = torch.empty((T, D), dtype=dt, device="cuda") if case["p"] > 0 else None
            st["dw"] = torch.empty(D, dtype=torch.float32, device="cuda")
            st["db"] = torch.empty(D, dtype=torch.float32, device="cuda") if case["bias"] else None
        else:
            st["x"] = rnd(T, D, std=1.0)
            st["residual"] = rnd(T, D, std=1.5, mean=0.1) if case["add"] else None
            st["out"] = torch.empty((T, D), dtype=dt, device="cuda")
            if op == "norm_fwd":
                st["sum"] = (torch.empty((T, D), dtype=dt, device="cuda")
                             if case["add"] or case["p"] > 0 else None)
                st["mean"], st["rstd"] = ((torch.empty(T, device="cuda") for _ in range(2))
                                          if case["stats"] else (None, None))
    if own:
        import token_indexed_sparse_staple_b200 as stp
        st["ctx"] = _context(stp)
        st["dt"] = stp.STAPLE_BF16 if case["dtype"] == "bf16" else stp.STAPLE_F32
        if op in ("norm_fwd", "norm_bwd"):
            st["kind"] = stp.STAPLE_NORM_LAYER if case["kind"] == "layer" else stp.STAPLE_NORM_RMS
        if "rng" in st:
            st["drop"] = (stp.make_drop(case["p"], st["rng"], st["site"])
                          if case["p"] > 0 else None)
        if op == "norm_bwd":
            st["wsb"] = stp.staple_norm_workspace_bytes(T, case["D"])
            st["ws"] = torch.zeros(max(st["wsb"], 1), dtype=torch.uint8, device="cuda")
    return st


_ctx = None


def _context(stp):
    """The library context: one per process, as a user's program keeps it."""
    global _ctx
    if _ctx is None:
        _ctx = stp.staple_context_create(0)
    return _ctx


# ----------------------------------------------------------------- own calls

def run(state):
    if own:
        return _run_own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "dropout": _plain_dropout,
            "quant_rows": _plain_quant, "matmul_i8": _plain_matmul}[state["case"]["op"]](state)


def _run_own(st):
    import token_indexed_sparse_staple_b200 as stp
    case = st["case"]
    op, T = case["op"], case["T"]
    if op == "norm_fwd":
        stp.staple_norm_fwd(st["ctx"], st["dt"], st["kind"], T, case["D"], st["x"], st["out"],
                            weight=st["weight"], bias=st["bias"], eps=EPS,
                            residual=st["residual"], drop=st["drop"], sum=st["sum"],
                            mean=st["mean"], rstd=st["rstd"])
        return _norm_fwd_outputs(case, st["out"], st["sum"], st["mean"], st["rstd"])
    if op == "norm_bwd":
        stp.staple_norm_bwd(st["ctx"], st["dt"], st["kind"], T, case["D"], st["dy"], st["sum"],
                            st["rstd"], st["dsum"], mean=st["mean"], weight=st["weight"],
                            dsum_in=st["dsum_in"], drop=st["drop"], dx=st["dx"], dw=st["dw"],
                            db=st["db"], workspace=st["ws"], workspace_bytes=st["wsb"])
        return _norm_bwd_outputs(case, st["dsum"], st["dx"], st["dw"], st["db"])
    if op == "dropout":
        stp.staple_dropout(st["ctx"], st["dt"], T, case["D"], st["x"], st["drop"], st["out"],
                           residual=st["residual"])
        return st["out"]
    if op == "quant_rows":
        stp.staple_quant_rows(st["ctx"], st["dt"], T, case["D"], st["x"], st["q"], st["scale"])
        return st["q"], st["scale"]
    stp.staple_matmul_i8(st["ctx"], st["dt"], T, case["N"], case["K"], st["a"], st["a_scale"],
                         st["b"], st["b_scale"], st["y"])
    return st["y"]


def _norm_fwd_outputs(case, y, s, mean, rstd):
    out = {"y": y}
    if case["add"] or case["p"] > 0:
        out["sum"] = s
    if case["stats"]:
        out["mean"], out["rstd"] = mean, rstd
    return out


def _norm_bwd_outputs(case, dsum, dx, dw, db):
    out = {"dsum": dsum, "dw": dw}
    if case["p"] > 0:
        out["dx"] = dx
    if case["bias"]:
        out["db"] = db
    return out


# --------------------------------------------------------------- plain forms

def _plain_philox16(rng, site, T, D):
    """[T][D] 16-bit draws of Philox4x32-10 (Salmon et al., SC 2011): key = the
    seed's two words; the counter's low half numbers the row's groups of eight
    elements, its high half is offset + site.  Element i of a group is the low
    (even i) or high (odd i) half of output word i / 2."""
    M = 0xFFFFFFFF
    G = (D + 7) // 8
    n = torch.arange(T * G, dtype=torch.int64, device=rng.device)
    hi = (rng[1] + site).expand_as(n)
    c0, c1, c2, c3 = n & M, (n >> 32) & M, hi & M, (hi >> 32) & M
    k0, k1 = rng[0] & M, (rng[0] >> 32) & M
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # wraps modulo 2^64
        c0, c1, c2, c3 = (((p1 >> 32) & M) ^ c1 ^ k0, p1 & M, ((p0 >> 32) & M) ^ c3 ^ k1, p0 & M)
        k0, k1 = (k0 + 0x9E3779B9) & M, (k1 + 0xBB67AE85) & M
    u = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16,
                     c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], dim=1)
    return u.reshape(T, G * 8)[:, :D]


def _plain_drop(x, case, st):
    """x in 32 bits, dropped with probability round(p 2^16) / 2^16 and scaled."""
    if not case["p"] > 0:
        return x
    thr = int(round(case["p"] * 65536))
    keep = _plain_philox16(st["rng"], st["site"], case["T"], case["D"]) >= thr
    return torch.where(keep, x * (65536.0 / (65536 - thr)), 0.0)


def _plain_norm_fwd(st):
    case = st["case"]
    dt = st["x"].dtype
    s = _plain_drop(st["x"].float(), case, st)
    if case["add"]:
        s = st["residual"].float() + s
    s_out = s.to(dt)
    s = s_out.float()               # the norm sees the stored sum
    mean = s.mean(dim=1) if case["kind"] == "layer" else torch.zeros(s.shape[0], device=s.device)
    c = s - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + EPS)
    y = c * rstd[:, None] * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return _norm_fwd_outputs(case, y.to(dt), s_out, mean, rstd)


def _plain_norm_bwd(st):
    case = st["case"]
    dt = st["dy"].dtype
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xhat = (st["sum"].float() - st["mean"][:, None]) * rstd
    wdy = dy * st["weight"].float()
    c2 = (wdy * xhat).mean(dim=1, keepdim=True)
    ds = wdy - xhat * c2
    if case["kind"] == "layer":
        ds = ds - wdy.mean(dim=1, keepdim=True)
    ds = ds * rstd
    if case["add"]:
        ds = ds + st["dsum_in"].float()
    dx = _plain_drop(ds, case, st)
    return _norm_bwd_outputs(case, ds.to(dt), dx.to(dt), (dy * xhat).sum(dim=0), dy.sum(dim=0))


def _plain_dropout(st):
    y = _plain_drop(st["x"].float(), st["case"], st)
    if st["residual"] is not None:
        y = st["residual"].float() + y
    return y.to(st["x"].dtype)


def _plain_quant(st):
    x = st["x"].double()            # quotients next to a half need 64 bits
    scale = (x.abs().amax(dim=1) / 127.0).float()
    q = torch.round(x / scale.double()[:, None]).clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, 0.0)
    return q.to(torch.int8), scale


def _plain_matmul(st):
    acc = st["a"].double() @ st["b"].double().t()    # exact: sums below 2^53
    y = acc.float() * st["a_scale"][:, None] * st["b_scale"][None, :]
    return y.to(st["y"].dtype)


# ---------------------------------------------------------------------- work

def work(case):
    op, T = case["op"], case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "matmul_i8":
        N, K = case["N"], case["K"]
        return {"bytes": T * K + N * K + 4 * (T + N) + e * T * N, "flops": 2 * T * N * K}
    D = case["D"]
    if op == "quant_rows":
        return {"bytes": T * D * (e + 1) + 4 * T, "flops": 4 * T * D}
    if op == "dropout":
        return {"bytes": T * D * e * (3 if case["add"] else 2), "flops": 3 * T * D}
    params = D * (2 if case["bias"] else 1)
    if op == "norm_fwd":
        tensors = 2 + (1 if case["add"] else 0) + (1 if case["add"] or case["p"] > 0 else 0)
        return {"bytes": T * D * e * tensors + params * e + (8 * T if case["stats"] else 0),
                "flops": 8 * T * D}
    tensors = 3 + (1 if case["add"] else 0) + (1 if case["p"] > 0 else 0)
    return {"bytes": T * D * e * tensors + 8 * T + D * e + 4 * params, "flops": 14 * T * D}


# --------------------------------------------------------------------- exact

def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _exact_keep(st, T, D, p):
    """The dropout's factors in 64 bits, row by row of the definition."""
    thr = int(round(p * 65536))
    seed, offset = (int(v) & (2 ** 64 - 1) for v in st["rng"].cpu().tolist())
    ctr_hi = (offset + st["site"]) % 2 ** 64
    G = -(-D // 8)
    ctr = np.arange(T * G, dtype=np.uint64)
    lo32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    v = [ctr & lo32, ctr >> sh, np.full_like(ctr, ctr_hi & 0xFFFFFFFF),
         np.full_like(ctr, ctr_hi >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        a = v[0] * np.uint64(0xD2511F53)
        b = v[2] * np.uint64(0xCD9E8D57)
        ka = np.uint64((key[0] + r * 0x9E3779B9) % 2 ** 32)
        kb = np.uint64((key[1] + r * 0xBB67AE85) % 2 ** 32)
        v = [(b >> sh) ^ v[1] ^ ka, b & lo32, (a >> sh) ^ v[3] ^ kb, a & lo32]
    u = np.empty((T * G, 8), dtype=np.int64)
    for j in range(4):
        u[:, 2 * j] = (v[j] & np.uint64(0xFFFF)).astype(np.int64)
        u[:, 2 * j + 1] = (v[j] >> np.uint64(16)).astype(np.int64)
    u = u.reshape(T, G * 8)[:, :D]
    return np.where(u >= thr, 65536.0 / max(65536 - thr, 1), 0.0)


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "matmul_i8":
        # scaled operands in 64 bits; the sum is taken over k in four parts
        a = st["a"].to(torch.float64) * st["a_scale"].to(torch.float64).unsqueeze(1)
        b = st["b"].to(torch.float64) * st["b_scale"].to(torch.float64).unsqueeze(1)
        y = torch.zeros((T, case["N"]), dtype=torch.float64, device=a.device)
        step = -(-case["K"] // 4)
        for k in range(0, case["K"], step):
            y += torch.einsum("tk,nk->tn", a[:, k:k + step], b[:, k:k + step])
        return y
    D = case["D"]
    if op == "quant_rows":
        x = st["x"].detach().float().cpu().numpy()
        amax = np.max(np.abs(x), axis=1)
        scale = amax / np.float32(127)
        q = np.zeros((T, D), dtype=np.int8)
        for i in range(0, T, 512):      # blocks of rows keep the 64-bit copies small
            s = scale[i:i + 512].astype(np.float64)[:, None]
            with np.errstate(divide="ignore", invalid="ignore"):
                r = np.rint(x[i:i + 512].astype(np.float64) / s)
            q[i:i + 512] = np.where(s > 0, np.clip(np.nan_to_num(r), -127, 127), 0).astype(np.int8)
        return torch.from_numpy(q), torch.from_numpy(scale)
    keep = _exact_keep(st, T, D, case["p"]) if case["p"] > 0 else 1.0
    if op == "dropout":
        y = _np(st["x"]) * keep
        if case["add"]:
            y = y + _np(st["residual"])
        return torch.from_numpy(y)
    w = _np(st["weight"])
    rms = case["kind"] == "rms"
    if op == "norm_fwd":
        s = _np(st["x"]) * keep
        if case["add"]:
            s = s + _np(st["residual"])
        # the sum is stored in its type, and the norm is defined on what is stored
        stored = (torch.from_numpy(s).to(st["x"].dtype).double().numpy()
                  if case["add"] or case["p"] > 0 else s)
        mean = np.zeros(T) if rms else stored.sum(axis=1) / D
        dev = stored - mean[:, None]
        rstd = (np.einsum("td,td->t", dev, dev) / D + EPS) ** -0.5
        y = dev * (rstd[:, None] * w[None, :])
        if case["bias"]:
            y += _np(st["bias"])[None, :]
        return _norm_fwd_outputs(case, torch.from_numpy(y), torch.from_numpy(s),
                                 torch.from_numpy(mean), torch.from_numpy(rstd))
    dy, rstd = _np(st["dy"]), _np(st["rstd"])
    xhat = (_np(st["sum"]) - _np(st["mean"])[:, None]) * rstd[:, None]
    gw = dy * w[None, :]
    proj = np.einsum("td,td->t", gw, xhat) / D
    ds = gw - xhat * proj[:, None]
    if not rms:
        ds -= gw.sum(axis=1, keepdims=True) / D
    ds *= rstd[:, None]
    if case["add"]:
        ds += _np(st["dsum_in"])
    return _norm_bwd_outputs(case, torch.from_numpy(ds), torch.from_numpy(ds * keep),
                             torch.from_numpy(np.einsum("td,td->d", dy, xhat)),
                             torch.from_numpy(dy.sum(axis=0)))
