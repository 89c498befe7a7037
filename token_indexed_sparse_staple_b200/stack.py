"""Stacks of STAPLE layers driven through the C ABI: the per-step
orchestration of several augmented layers (host logic only; every step of
the computation runs in the library's kernels).

- x_{l+1} = y_l, and every layer sees the same token ids.  So the batch is
  deduplicated once per step, and one inverse map serves every layer
  (retrieval-path table, Prefill row: dedup once, reuse the inverse map).
- Tables are grouped G adjacent layers per host row, token-major: host array
  [V][G][F] per group (retrieval-path table, Decode row).  One gather per
  group fetches the rows of all G layers.  Later groups are gathered on
  prefetch streams while earlier layers compute, and a layer waits only for
  its own group (Decode row: synchronise when a group is first consumed).
- Training: the backward pass runs the layers in reverse.  Each layer's U
  table-gradient rows go back to host memory on a copy stream while the next
  layer's backward runs.  By default the copy engine moves exactly U rows:
  U reaches pinned host memory right after the dedup, long before the
  backward needs it.  SM stores over the host link (staple_embed_grad_to_host,
  which reads U on the device and so also works inside a captured graph)
  would occupy every SM's store path with slow posted writes and stall the
  concurrent GEMMs' epilogues.  The next step's dedup
  and first-group gather run during this step's backward (successive batches
  are pipelined: retrieval-path table, Prefill row).  No table optimizer runs
  here, so nothing the prefetch reads changes in between.
- Decode: one step (dedup, group gathers, all layers) is captured once in a
  multi-stream CUDA graph and replayed (Decode row: grouped lookups and the
  model in one multi-stream CUDA graph).

- With `norms`, a stack is the residual stream of a pre-norm transformer's
  FFN sublayers instead of the bare chain:
      x_{l+1} = x_l + dropout(FFN_l(norm_l(x_l)))
  Each residual add, its dropout and the next layer's norm are one kernel, and
  so are the backward pass of a norm, the residual's gradient and the dropout
  in front of it.  No dropout mask is stored: the backward pass draws it again
  from the step's {seed, offset} and the layer's site.
- Decode layers may have their weights in 8 bits (LayerWeightsI8).

torch supplies device memory, pinned host memory, streams and events.
"""
from __future__ import annotations

from dataclasses import dataclass

import token_indexed_sparse_staple_b200 as stp


@dataclass
class LayerWeights:
    w_gate: object   # [F][D] bf16
    w_up: object     # [F][D] bf16
    w_down: object   # [D][F] bf16


@dataclass
class LayerWeightsI8:
    """A decode layer's weights in 8 bits, one scale per row."""
    w_gate_up: object      # [2F][D] int8: W_gate's rows, then W_up's
    gate_up_scale: object  # [2F] fp32
    w_down: object         # [D][F] int8
    down_scale: object     # [D] fp32


def quantise_layer(ctx, w: LayerWeights, stream=None) -> LayerWeightsI8:
    """The 8-bit copy of a layer's bf16 weights, made on `stream` (default:
    torch's current stream).  With another stream, that one first waits for the
    current stream, where the weights were made and the copy's memory is
    allocated (memory that work still queued there may have used before), and the
    current stream then waits for the copy."""
    import torch
    current = torch.cuda.current_stream()
    st = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream or current
    F, D = w.w_gate.shape
    gu = torch.empty((2 * F, D), dtype=torch.int8, device="cuda")
    gus = torch.empty(2 * F, dtype=torch.float32, device="cuda")
    down = torch.empty((D, F), dtype=torch.int8, device="cuda")
    ds = torch.empty(D, dtype=torch.float32, device="cuda")
    if st != current:
        st.wait_stream(current)
    for src, q, s in ((w.w_gate, gu[:F], gus[:F]), (w.w_up, gu[F:], gus[F:]), (w.w_down, down, ds)):
        stp.staple_quant_rows(ctx, stp.STAPLE_BF16, *src.shape, src, q, s, stream=st)
    if st != current:
        current.wait_stream(st)
    return LayerWeightsI8(gu, gus, down, ds)


@dataclass
class NormWeights:
    """The norm in front of a layer."""
    weight: object = None            # [D] bf16, or None (ones)
    bias: object = None              # [D] bf16, or None (zeros)
    kind: int = stp.STAPLE_NORM_RMS
    eps: float = 1e-5


class GroupedTables:
    """The host tables of L layers, G layers per host row: group k is a
    page-locked [V][G * F] bf16 array (layer G*k + j in columns [j F, (j+1) F)),
    registered with the library, each with its own hot-row cache."""

    def __init__(self, ctx, host_groups, V: int, F: int, G: int, freq, frac: float):
        self.ctx, self.V, self.F, self.G = ctx, V, F, G
        self.host = list(host_groups)
        self.handles, self.caches = [], []
        try:
            for t in self.host:
                h = stp.staple_table_register(ctx, t, t.numel() * t.element_size(), V, F, G,
                                              stp.STAPLE_BF16, stp.STAPLE_TABLE_HOST_PINNED)
                self.handles.append(h)
                self.caches.append(stp.staple_cache_build(ctx, h, freq, frac))
        except Exception:
            self.close()
            raise

    @property
    def n_groups(self) -> int:
        return len(self.host)

    def close(self):
        for c in self.caches:
            stp.staple_cache_free(c)
        for h in self.handles:
            stp.staple_table_unregister(h)
        self.caches, self.handles = [], []


class Retrieval:
    """One step's retrieval state: a dedup and, per group, the probe results
    and the gathered rows [T][G * F]."""

    def __init__(self, T: int, F: int, G: int, n_groups: int):
        import torch
        i32 = dict(dtype=torch.int32, device="cuda")
        self.T, self.F, self.G = T, F, G
        self.unique, self.inverse, self.sorted_pos = (torch.empty(max(T, 1), **i32) for _ in range(3))
        self.seg, self.U = torch.empty(T + 1, **i32), torch.empty(1, **i32)
        self.slot = [torch.empty(max(T, 1), **i32) for _ in range(n_groups)]
        self.miss = [torch.empty(max(T, 1), **i32) for _ in range(n_groups)]
        self.mc = [torch.empty(1, **i32) for _ in range(n_groups)]
        self.rows = [torch.empty((max(T, 1), G * F), dtype=torch.bfloat16, device="cuda")
                     for _ in range(n_groups)]
        self.ready = [torch.cuda.Event() for _ in range(n_groups)]
        self.free = torch.cuda.Event()   # recorded after the last reader of this step
        self.U_host = torch.zeros(1, dtype=torch.int32, pin_memory=True)
        self.U_known = torch.cuda.Event()  # U_host holds this step's U

    def embed(self, layer: int):
        """The embed argument of layer `layer`: its G-slice of its group's rows,
        indexed by the inverse map."""
        g, j = divmod(layer, self.G)
        base = self.rows[g].data_ptr() + j * self.F * self.rows[g].element_size()
        return stp.make_embed(stp.STAPLE_EMBED_ROWS, base, self.G * self.F, self.inverse, self.T)


def issue_dedup(ctx, r: Retrieval, ids, V: int, stream, u_to_host: bool = True):
    """The batch's dedup on `stream`; with u_to_host, U is also copied to pinned
    host memory (the training stack reads it there; a decode step does not,
    and the copy would sit between the dedup and the first gather)."""
    import torch
    stp.staple_dedup(ctx, ids, r.T, V, r.unique, r.inverse, r.seg, r.sorted_pos, r.U,
                     stream=stream)
    if u_to_host:
        with torch.cuda.stream(stream):
            r.U_host.copy_(r.U, non_blocking=True)   # 4 bytes; read by the host much later
        r.U_known.record(stream)


def issue_group(ctx, r: Retrieval, tables: GroupedTables, g: int, stream, side):
    stp.staple_gather_unique_rows(ctx, tables.caches[g], tables.handles[g], r.unique, r.U, r.T,
                                  r.slot[g], r.miss[g], r.mc[g], r.rows[g], stream=stream,
                                  side=side)
    r.ready[g].record(stream)


# --------------------------------------------------------------------------
# Training stack
# --------------------------------------------------------------------------

@dataclass
class TrainBuffers:
    xs: list                       # x_0 .. x_L: [T][D] bf16 (x_{l+1} = y_l)
    z: list
    g: list
    h: list                        # per layer [T][F] bf16, saved for the backward
    dy: list                       # [T][D] bf16 gradients passed down (two alternating, or L)
    dgh: object                    # [T][2F] bf16, one layer at a time
    dE: list                       # two fp32 [T][F] buffers alternating (copy-out overlap)
    dE_copied: list                # events: the copy of dE[i] to the host has been issued and run
    dW: list                       # per layer (dW_gate, dW_up, dW_down) fp32
    host_dE: list                  # per layer page-locked fp32 [T][F]
    host_unique: list              # per layer page-locked int32 [T]
    host_U: list                   # per layer page-locked int32 [1]
    ws: object
    wsb: int


class TrainStack:
    """L augmented layers, forward and full backward per step, with dE of
    every layer returned to host memory."""

    def __init__(self, ctx, weights: list, tables: GroupedTables, T: int, D: int, F: int, V: int,
                 freeze_up: bool = False, keep_dy: bool = False, de_return: str = "dma",
                 norms=None, dropout: float = 0.0, rng=None):
        """keep_dy keeps every layer's incoming gradient (L buffers instead of
        two alternating ones), so each layer can be checked on its own inputs
        (with norms the residual stream's gradients too, in dstream).
        de_return: "dma" (copy engine, U known on the host) or "kernel"
        (staple_embed_grad_to_host, U read on the device).
        norms: one NormWeights per layer, which makes the stack the residual
        stream described above; dropout is then the probability of the
        dropouts in front of the residual adds, drawn from rng, a device int64
        tensor {seed, offset} that the caller advances by L after each step
        (site l is layer l's).  The gradients of x_0 and of the norms are in
        dx0 and dnorm[l] = (dw, db) after a step."""
        assert de_return in ("dma", "kernel")
        self.de_return = de_return
        import torch
        self.ctx, self.W, self.tables = ctx, weights, tables
        self.T, self.D, self.F, self.V, self.G = T, D, F, V, tables.G
        self.L = len(weights)
        assert self.L == tables.n_groups * self.G
        self.freeze_up = freeze_up
        bf = dict(dtype=torch.bfloat16, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")
        L = self.L
        wsb = stp.staple_workspace_bytes(T, D, F)
        self.b = TrainBuffers(
            xs=[torch.empty((T, D), **bf) for _ in range(L + 1)],
            z=[torch.empty((T, F), **bf) for _ in range(L)],
            g=[torch.empty((T, F), **bf) for _ in range(L)],
            h=[torch.empty((T, F), **bf) for _ in range(L)],
            dy=[torch.empty((T, D), **bf) for _ in range(L if keep_dy else 2)],
            dgh=torch.empty((T, 2 * F), **bf),
            dE=[torch.empty((T, F), **f32) for _ in range(2)],
            dE_copied=[torch.cuda.Event() for _ in range(2)],
            dW=[(torch.empty((F, D), **f32), None if freeze_up else torch.empty((F, D), **f32),
                 torch.empty((D, F), **f32)) for _ in range(L)],
            host_dE=[torch.empty((T, F), dtype=torch.float32).pin_memory() for _ in range(L)],
            host_unique=[torch.empty(T, dtype=torch.int32).pin_memory() for _ in range(L)],
            host_U=[torch.zeros(1, dtype=torch.int32).pin_memory() for _ in range(L)],
            ws=torch.zeros(max(wsb, 256), dtype=torch.uint8, device="cuda"), wsb=wsb)
        self.norms = list(norms) if norms is not None else None
        if self.norms is not None:
            assert len(self.norms) == L
            assert dropout == 0.0 or rng is not None
            self.rng = rng
            self.drops = [stp.make_drop(dropout, rng, l) for l in range(L)]
            self.n = [torch.empty((T, D), **bf) for _ in range(L)]      # the layers' inputs
            self.y = torch.empty((T, D), **bf)                          # a layer's output
            self.mean, self.rstd = ([torch.empty(T, **f32) for _ in range(L)] for _ in range(2))
            self.dnorm = [(torch.empty(D, **f32), torch.empty(D, **f32)) for _ in range(L)]
            self.dn = torch.empty((T, D), **bf)                         # gradient of norm_l's output
            self.dstream = [torch.empty((T, D), **bf) for _ in range(L if keep_dy else 2)]
            self.dx0 = None
            self.nws = torch.empty(max(stp.staple_norm_workspace_bytes(T, D), 16),
                                   dtype=torch.uint8, device="cuda")
        else:
            assert dropout == 0.0
        self.retr = [Retrieval(T, F, self.G, tables.n_groups) for _ in range(2)]
        self.pf, self.pf_side, self.copy = (torch.cuda.Stream() for _ in range(3))
        self.host_ready = torch.cuda.Event()   # the last step's dE rows are in host memory
        self.step_no = 0
        self._primed = None   # (step, ids) whose dedup + group 0 are in flight

    def _prefetch_head(self, r: Retrieval, ids):
        """Dedup and group 0 of a step, on the prefetch streams, once the
        previous user of `r` is done with it."""
        self.pf.wait_event(r.free)
        issue_dedup(self.ctx, r, ids, self.V, self.pf)
        issue_group(self.ctx, r, self.tables, 0, self.pf, self.pf_side)

    def _norm_fwd(self, l: int, x, st, **kw):
        nw = self.norms[l]
        stp.staple_norm_fwd(self.ctx, stp.STAPLE_BF16, nw.kind, self.T, self.D, x, self.n[l],
                            weight=nw.weight, bias=nw.bias, eps=nw.eps, mean=self.mean[l],
                            rstd=self.rstd[l], stream=st, **kw)

    def step(self, ids, x0, dy_top, next_ids=None, stream=None):
        """One training step on `stream` (default: torch's current stream).
        ids [T] int32, x0 [T][D] and dy_top [T][D] bf16 on the device.
        next_ids, when given, lets the next step's dedup and first gather run
        during this step's backward; the next step then uses those ids (its
        own `ids` argument is not read again).  Returns the Retrieval used
        (its U_dev, unique ids and hit/miss maps stay valid until the step
        after next).  The step's dE rows reach host memory when host_ready
        completes (wait on it before reading host_dE): later work on `stream`,
        such as the next step's forward, does not wait for the last layer's
        copy-out, since no table optimizer runs between the steps here."""
        import torch
        st = stream or torch.cuda.current_stream()
        b, T, D, F = self.b, self.T, self.D, self.F
        r = self.retr[self.step_no % 2]
        if self._primed is None or self._primed[0] != self.step_no:
            self.pf.wait_stream(st)               # ids may come from this stream
            self._prefetch_head(r, ids)
        for gi in range(1, self.tables.n_groups):
            issue_group(self.ctx, r, self.tables, gi, self.pf, self.pf_side)
        if x0.data_ptr() != b.xs[0].data_ptr():
            with torch.cuda.stream(st):
                b.xs[0].copy_(x0)
        # forward
        if self.norms is not None:
            self._norm_fwd(0, b.xs[0], st)
        for l in range(self.L):
            gi = l // self.G
            if l % self.G == 0:
                st.wait_event(r.ready[gi])
            w = self.W[l]
            x, y = (b.xs[l], b.xs[l + 1]) if self.norms is None else (self.n[l], self.y)
            stp.staple_ffn_fwd(self.ctx, stp.STAPLE_BF16, T, D, F, x, r.embed(l), w.w_gate,
                               w.w_up, w.w_down, b.z[l], y, b.g[l], b.h[l], b.ws, b.wsb,
                               stream=st)
            if self.norms is None:
                continue
            if l + 1 < self.L:     # the residual add and the next layer's norm
                self._norm_fwd(l + 1, self.y, st, residual=b.xs[l], drop=self.drops[l],
                               sum=b.xs[l + 1])
            else:
                stp.staple_dropout(self.ctx, stp.STAPLE_BF16, T, D, self.y, self.drops[l],
                                   b.xs[l + 1], residual=b.xs[l], stream=st)
        # the next step's dedup and first group while the backward runs
        if next_ids is not None:
            rn = self.retr[(self.step_no + 1) % 2]
            self.pf.wait_stream(st)
            self._prefetch_head(rn, next_ids)
            self._primed = (self.step_no + 1, next_ids)
        # backward, layers in reverse
        if self.de_return == "dma":
            r.U_known.synchronize()               # completed long ago: the dedup ran first
            U = int(r.U_host[0])
        dy = dy_top
        if self.norms is not None:
            # the stream's gradient dres and, dropped, the top layer's dy
            dres, dy = dy_top, b.dy[(self.L - 1) % len(b.dy)]
            stp.staple_dropout(self.ctx, stp.STAPLE_BF16, T, D, dres, self.drops[self.L - 1], dy,
                               stream=st)
        for l in reversed(range(self.L)):
            w = self.W[l]
            k = l % 2
            st.wait_event(b.dE_copied[k])          # dE[k]'s previous copy-out is done
            stp.staple_embed_bwd(self.ctx, stp.STAPLE_BF16, T, D, F, dy, b.g[l], b.h[l], w.w_down,
                                 r.sorted_pos, r.inverse, r.seg, r.U, b.dgh, b.dE[k], b.ws, b.wsb,
                                 stream=st)
            self.copy.wait_stream(st)
            if self.de_return == "dma":
                with torch.cuda.stream(self.copy):
                    b.host_dE[l][:U].copy_(b.dE[k][:U], non_blocking=True)
                    b.host_unique[l][:U].copy_(r.unique[:U], non_blocking=True)
                b.host_U[l][0] = U
            else:
                stp.staple_embed_grad_to_host(self.ctx, F, T, b.dE[k], r.unique, r.U,
                                              b.host_dE[l], b.host_unique[l], b.host_U[l],
                                              stream=self.copy)
            b.dE_copied[k].record(self.copy)
            dwg, dwu, dwd = b.dW[l]
            if self.norms is None:
                dx = b.dy[l % len(b.dy)]   # the gradient layer l passes down (layer l-1's dy)
                stp.staple_ffn_bwd(self.ctx, stp.STAPLE_BF16, T, D, F, dy, b.xs[l], b.z[l], b.dgh,
                                   w.w_gate, w.w_up, dx, dwg, dwu, dwd, stream=st)
                dy = dx
                continue
            stp.staple_ffn_bwd(self.ctx, stp.STAPLE_BF16, T, D, F, dy, self.n[l], b.z[l], b.dgh,
                               w.w_gate, w.w_up, self.dn, dwg, dwu, dwd, stream=st)
            # through norm_l, joined by the residual's gradient; then, for the
            # layer below, its dropout
            dy = b.dy[(l - 1) % len(b.dy)] if l > 0 else None
            out = self.dstream[l % len(self.dstream)]
            nw = self.norms[l]
            dw, db = self.dnorm[l]
            stp.staple_norm_bwd(self.ctx, stp.STAPLE_BF16, nw.kind, T, D, self.dn, b.xs[l],
                                self.rstd[l], out, mean=self.mean[l], weight=nw.weight,
                                dsum_in=dres, drop=self.drops[l - 1] if l > 0 else None, dx=dy,
                                dw=dw, db=db, workspace=self.nws,
                                workspace_bytes=self.nws.numel(), stream=st)
            dres = out
        if self.norms is not None:
            self.dx0 = dres
        r.free.record(self.copy)                   # after the last reader (layer 0's copy-out)
        self.host_ready.record(self.copy)
        self.step_no += 1
        return r


# --------------------------------------------------------------------------
# Decode stack
# --------------------------------------------------------------------------

class DecodeStack:
    """L augmented layers at decode sizes (T <= 256): one step = dedup,
    group gathers on prefetch streams, the L fused decode layers.  capture()
    records a step into a CUDA graph; replay() runs it for the ids currently
    in `ids_buf`.  Layers are LayerWeights or LayerWeightsI8.  norms: one
    NormWeights per layer, which makes the stack the residual stream
    x_{l+1} = x_l + FFN_l(norm_l(x_l))."""

    def __init__(self, ctx, weights: list, tables: GroupedTables, T: int, D: int, F: int, V: int,
                 norms=None):
        import torch
        self.ctx, self.W, self.tables = ctx, weights, tables
        self.T, self.D, self.F, self.V, self.G = T, D, F, V, tables.G
        self.L = len(weights)
        assert self.L == tables.n_groups * self.G
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.ids_buf = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.xs = [torch.empty((T, D), **bf) for _ in range(self.L + 1)]
        self.z = torch.empty((T, F), **bf)
        self.wsb = stp.staple_workspace_bytes(T, D, F)
        self.ws = torch.zeros(self.wsb, dtype=torch.uint8, device="cuda")
        if any(isinstance(w, LayerWeightsI8) for w in weights):
            self.wsb8 = stp.staple_ffn_i8_workspace_bytes(T, D, F)
            self.ws8 = torch.empty(max(self.wsb8, 256), dtype=torch.uint8, device="cuda")
        self.norms = list(norms) if norms is not None else None
        if self.norms is not None:
            assert len(self.norms) == self.L
            self.n, self.y = torch.empty((T, D), **bf), torch.empty((T, D), **bf)
            self.no_drop = stp.make_drop(0.0, None)
        self.r = Retrieval(T, F, self.G, tables.n_groups)
        self.pf, self.pf_side = torch.cuda.Stream(), torch.cuda.Stream()
        self.graph = None

    def run(self, stream=None):
        """One step for ids_buf and xs[0]; y of the last layer in xs[L]."""
        import torch
        st = stream or torch.cuda.current_stream()
        r = self.r
        self.pf.wait_stream(st)
        issue_dedup(self.ctx, r, self.ids_buf, self.V, self.pf, u_to_host=False)
        for gi in range(self.tables.n_groups):
            issue_group(self.ctx, r, self.tables, gi, self.pf, self.pf_side)
        T, D = self.T, self.D
        if self.norms is not None:
            self._norm_fwd(0, self.xs[0], st)
        for l in range(self.L):
            if l % self.G == 0:
                st.wait_event(r.ready[l // self.G])
            if self.norms is None:
                self._layer(l, self.xs[l], self.xs[l + 1], st)
                continue
            self._layer(l, self.n, self.y, st)
            if l + 1 < self.L:     # the residual add and the next layer's norm
                self._norm_fwd(l + 1, self.y, st, residual=self.xs[l], sum=self.xs[l + 1])
            else:
                stp.staple_dropout(self.ctx, stp.STAPLE_BF16, T, D, self.y, self.no_drop,
                                   self.xs[l + 1], residual=self.xs[l], stream=st)
        st.wait_stream(self.pf)                    # join the prefetch streams (graph capture)

    def _norm_fwd(self, l: int, x, st, **kw):
        nw = self.norms[l]
        stp.staple_norm_fwd(self.ctx, stp.STAPLE_BF16, nw.kind, self.T, self.D, x, self.n,
                            weight=nw.weight, bias=nw.bias, eps=nw.eps, stream=st, **kw)

    def _layer(self, l: int, x, y, st):
        w = self.W[l]
        if isinstance(w, LayerWeightsI8):
            stp.staple_ffn_fwd_i8(self.ctx, self.T, self.D, self.F, x, self.r.embed(l), w.w_gate_up,
                                  w.gate_up_scale, w.w_down, w.down_scale, y, self.ws8, self.wsb8,
                                  stream=st)
        else:
            stp.staple_ffn_fwd(self.ctx, stp.STAPLE_BF16, self.T, self.D, self.F, x,
                               self.r.embed(l), w.w_gate, w.w_up, w.w_down, self.z, y, None, None,
                               self.ws, self.wsb, stream=st)

    def capture(self, stream, ids_src=None, x_src=None):
        """Record a step into a CUDA graph (kept for replay() and returned).
        With ids_src / x_src the graph first copies them into ids_buf /
        xs[0], so that a set of graphs feeds recorded inputs with no copy
        outside the graphs."""
        import torch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            if ids_src is not None:
                self.ids_buf.copy_(ids_src)
            if x_src is not None:
                self.xs[0].copy_(x_src)
            self.run(stream)
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()

    def release(self):
        self.graph = None
