// The norm in front of a layer, with the residual add and the dropout that
// come before it fused in, and its backward pass.
//
//   s = residual + dropout(x),  y = (s - mean) rstd w + b
//   LayerNorm: mean = sum(s) / D, rstd = 1 / sqrt(sum((s - mean)^2) / D + eps)
//   RMSNorm:   mean = 0,          rstd = 1 / sqrt(sum(s^2) / D + eps)
//
//   xhat = (s - mean) rstd,  gw = dy w
//   ds = rstd (gw - mean(gw) [LayerNorm only] - xhat mean(gw xhat)) + dsum_in
//   dx = dropout'(ds),  dw = sum_t dy xhat,  db = sum_t dy
//
// Both directions are bound by memory: each tensor is read or written once.
// A row stays in registers between its loads and its stores, so the variance
// is summed from the deviations (two passes over registers, none over
// memory).  Sums, means and rstd are fp32.  The backward pass adds dw and db
// up in registers over the rows of a persistent block; the blocks' sums meet
// in a second small kernel in block order, so the result does not depend on
// timing.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "rows.cuh"

namespace stp {

namespace {

struct FwdParams {
  const void* x;
  const void* res;
  const void* w;
  const void* b;
  void* sum;
  void* y;
  float* mean;
  float* rstd;
  DropParams drop;
  int32_t T, D, tpr;
  float eps;
  bool rms;
};

// Forward.  One read of x and the residual, one write of the sum and y; a block
// holds whole rows.  In captured runs 16384 x 2048 bf16 with residual takes 44.0 us
// without dropout (6.1 TB/s, 0.94 of a copy) and 47 to 49 with it (0.85 to 0.88: the
// generator's integer products share the issue slots), 1 x 4096 2.7 us, 1537 x 1023
// fp32 7.4 from memory and 5.9 from L2.
template <bool BF16, int NV, RowLayout L, bool DROP>
// (bf16: 64 registers, so that 32 warps share an SM)
__global__ void __launch_bounds__(512, BF16 ? 2 : 1) norm_fwd_kernel(const FwdParams p) {
  __shared__ float red[2][32];
  const int rpb = blockDim.x / p.tpr;
  const int rg = threadIdx.x / p.tpr, t = threadIdx.x - rg * p.tpr;
  const int64_t row = int64_t(blockIdx.x) * rpb + rg;
  const bool row_ok = row < p.T;
  const int G = (p.D + kGroup - 1) / kGroup;
  const int64_t base = row * p.D;
  wait_prior_kernels();
  Raw8<BF16> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Span e = span<L>(i, t, p.tpr, p.D);
    xr[i] = rr[i] = zero_raw8<BF16>();
    if (row_ok && e.n > 0) {
      xr[i] = load_raw8<BF16, L>(p.x, base, e);
      if (p.res) rr[i] = load_raw8<BF16, L>(p.res, base, e);
    }
  }
  // With few rows the weight and bias come from memory like the row itself:
  // load them with it, not after its sums.
  constexpr bool EARLY = NV == 1;
  Raw8<BF16> w0 = ones_raw8<BF16>(), b0 = zero_raw8<BF16>();
  if (EARLY) {
    const Span e = span<L>(0, t, p.tpr, p.D);
    if (p.w && e.n > 0) w0 = load_raw8<BF16, L>(p.w, 0, e);
    if (p.b && e.n > 0) b0 = load_raw8<BF16, L>(p.b, 0, e);
  }
  F2 v[NV][4];
  F2 s1 = f2(0.0f);
  constexpr int B = NV < 2 ? 1 : 2;      // (more at a time would not fit the registers)
  uint4 u[B];
  const int draws = L == VEC ? t : stride_group(t, p.tpr);
  DropKey key{};
  if (DROP) key = drop_key(p.drop);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Span s = span<L>(i, t, p.tpr, p.D);
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = xr[i].get(j);
    if (DROP && i % B == 0)
      philox_n<B>(key, uint64_t(row) * uint64_t(G) + (draws + i * p.tpr), uint32_t(p.tpr), u);
    if (DROP && L == VEC) drop8(u[i % B], p.drop.below, p.drop.scale, e);
    if (DROP && L == STRIDE)
      drop8_kept(stride_keep(u[i % B], p.drop.below, t, p.tpr), p.drop.scale, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = f2(e[2 * j], e[2 * j + 1]);
    if (p.sum) {
      // the norm sees the sum as stored, which is what the backward pass reads
      // (a missing residual is zeros)
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_get(v[i][j] + pair(rr[i], j), e[2 * j], e[2 * j + 1]);
      const Raw8<BF16> sr = pack_raw8<BF16>(e);
      if (row_ok && s.n > 0) store_raw8<BF16, L>(p.sum, base, s, sr);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = pair(sr, j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s1 = s1 + v[i][j];   // elements past D are zero
  }
  const float inv_d = 1.0f / float(p.D);
  float mean = 0.0f;
  if (!p.rms) {
    float lo, hi;
    f2_get(s1, lo, hi);
    float a[1] = {lo + hi};
    row_sum(a, p.tpr, red[0]);
    mean = a[0] * inv_d;
  }
  F2 s2 = f2(0.0f);
  const F2 nmean = f2(-mean);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int left = span<L>(i, t, p.tpr, p.D).n;
    if (L == VEC ? left > 0 : left == kGroup) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i][j] = v[i][j] + nmean;
        s2 = fma2(v[i][j], v[i][j], s2);
      }
    } else if (left > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // eight that the row's end cuts: nothing past D counts
        float lo, hi;
        f2_get(v[i][j] + nmean, lo, hi);
        v[i][j] = f2(2 * j < left ? lo : 0.0f, 2 * j + 1 < left ? hi : 0.0f);
        s2 = fma2(v[i][j], v[i][j], s2);
      }
    }
  }
  float lo, hi;
  f2_get(s2, lo, hi);
  float a[1] = {lo + hi};
  row_sum(a, p.tpr, red[1]);
  const float rstd = 1.0f / sqrtf(a[0] * inv_d + p.eps);
  if (!row_ok) return;
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const F2 rs = f2(rstd);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Span e = span<L>(i, t, p.tpr, p.D);
    if (e.n <= 0) break;
    // (a missing weight is ones, a missing bias is zeros)
    Raw8<BF16> w = w0, b = b0;
    if (!EARLY && p.w) w = load_raw8<BF16, L>(p.w, 0, e);
    if (!EARLY && p.b) b = load_raw8<BF16, L>(p.b, 0, e);
    float o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f2_get(fma2(v[i][j] * rs, pair(w, j), pair(b, j)), o[2 * j], o[2 * j + 1]);
    store_raw8<BF16, L>(p.y, base, e, pack_raw8<BF16>(o));
  }
}

struct BwdParams {
  const void* dy;
  const void* s;
  const void* w;
  const float* mean;
  const float* rstd;
  const void* dsum_in;
  void* dsum;
  void* dx;
  float* part;           // [blocks][2][D]: dw, db of each block; NULL: not wanted
  DropParams drop;
  int32_t T, D, tpr;
  bool rms;
};

// A row of one or two elements has next to no gradient: gw, its mean and its
// projection cancel down to their last bits (eps rstd^2 of gw remains).  This
// kernel, which takes such rows, therefore rounds each product and sum of the
// formula by itself; a fused multiply-add would leave another remainder than
// the formula's terms do.
//
// NV groups per thread and row, R rows in flight per thread.
template <bool BF16, int NV, int R, RowLayout L, bool DROP>
__global__ void __launch_bounds__(512, NV == 1 && R == 1 ? 2 : 1)
    norm_bwd_kernel(const BwdParams p) {
  __shared__ float red[2][2 * R * 32];
  extern __shared__ float s_acc[];   // row groups' dw, db (several row groups per block)
  const int rpb = blockDim.x / p.tpr;
  const int rg = threadIdx.x / p.tpr, t = threadIdx.x - rg * p.tpr;
  const int G = (p.D + kGroup - 1) / kGroup;
  const float inv_d = 1.0f / float(p.D);
  float aw[NV][8], ab[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[i][j] = ab[i][j] = 0.0f;
  wait_prior_kernels();
  if (p.part) release_dependents();
  const int draws = L == VEC ? t : stride_group(t, p.tpr);
  DropKey key{};
  if (DROP) key = drop_key(p.drop);
  int buf = 0;
  const int64_t step = int64_t(gridDim.x) * rpb * R;
  for (int64_t r0 = int64_t(blockIdx.x) * rpb * R; r0 < p.T; r0 += step, buf ^= 1) {
    Raw8<BF16> dyr[R][NV], sr[R][NV];
    float mu[R], rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + rg * R + r;
      const bool ok = row < p.T;
      mu[r] = ok && !p.rms ? p.mean[row] : 0.0f;
      rs[r] = ok ? p.rstd[row] : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Span e = span<L>(i, t, p.tpr, p.D);
        dyr[r][i] = sr[r][i] = zero_raw8<BF16>();
        if (ok && e.n > 0) {
          dyr[r][i] = load_raw8<BF16, L>(p.dy, row * p.D, e);
          sr[r][i] = load_raw8<BF16, L>(p.s, row * p.D, e);
        }
      }
    }
    float c[2 * R];
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) c[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Span e = span<L>(i, t, p.tpr, p.D);
      Raw8<BF16> w = ones_raw8<BF16>();      // (a missing weight)
      if (p.w && e.n > 0) w = load_raw8<BF16, L>(p.w, 0, e);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dy = dyr[r][i].get(j);        // zero past the row's end
          const float xh = (sr[r][i].get(j) - mu[r]) * rs[r];
          const float gw = dy * w.get(j);
          aw[i][j] = fmaf(dy, xh, aw[i][j]);
          ab[i][j] += dy;
          c[2 * r] += gw;
          c[2 * r + 1] = __fadd_rn(c[2 * r + 1], __fmul_rn(gw, xh));
        }
    }
    row_sum(c, p.tpr, red[buf]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Span e = span<L>(i, t, p.tpr, p.D);
      uint32_t keep[R];
      if constexpr (DROP && L == STRIDE) {
        // (by every lane, whatever it has of the row)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t n = (r0 + rg * R + r) * G + (draws + i * p.tpr);
          keep[r] = p.dx ? stride_keep(philox(key, uint64_t(n)), p.drop.below, t, p.tpr) : 0u;
        }
      }
      if (e.n <= 0) continue;
      Raw8<BF16> w = ones_raw8<BF16>();
      if (p.w) w = load_raw8<BF16, L>(p.w, 0, e);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = r0 + rg * R + r;
        if (row >= p.T) break;
        const float c1 = p.rms ? 0.0f : c[2 * r] * inv_d, c2 = c[2 * r + 1] * inv_d;
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dy = dyr[r][i].get(j);
          const float xh = (sr[r][i].get(j) - mu[r]) * rs[r];
          const float gw = dy * w.get(j);
          d[j] = __fsub_rn(__fsub_rn(gw, __fmul_rn(xh, c2)), c1) * rs[r];
        }
        if (p.dsum_in) {
          const Raw8<BF16> a = load_raw8<BF16, L>(p.dsum_in, row * p.D, e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += a.get(j);
        }
        if (p.dsum) store_raw8<BF16, L>(p.dsum, row * p.D, e, pack_raw8<BF16>(d));
        if (p.dx) {
          // from the fp32 gradient, not from the rounded dsum
          if constexpr (DROP && L == STRIDE)
            drop8_kept(keep[r], p.drop.scale, d);
          else if (DROP)
            drop8(philox(key, uint64_t(row) * uint64_t(G) + (t + i * p.tpr)), p.drop.below,
                  p.drop.scale, d);
          store_raw8<BF16, L>(p.dx, row * p.D, e, pack_raw8<BF16>(d));
        }
      }
    }
  }
  if (!p.part) return;
  // the block's row groups add up in group order
  float* out = p.part + int64_t(blockIdx.x) * 2 * p.D;
  if (rpb > 1) {
    // [row group][2][tpr * NV * 8] floats
    const int cols = p.tpr * NV * kGroup;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Span sp = span<L>(i, t, p.tpr, p.D);
        const int e = sp.off + j * sp.step;
        s_acc[(rg * 2 + 0) * cols + e] = aw[i][j];
        s_acc[(rg * 2 + 1) * cols + e] = ab[i][j];
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * p.D; k += blockDim.x) {
      const int which = k >= p.D, e = k - which * p.D;
      float s = 0.0f;
      for (int q = 0; q < rpb; ++q) s += s_acc[(q * 2 + which) * cols + e];
      out[k] = s;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Span sp = span<L>(i, t, p.tpr, p.D);
      const int e = sp.off + j * sp.step;
      if (j < sp.n) {
        out[e] = aw[i][j];
        out[p.D + e] = ab[i][j];
      }
    }
}

// The same backward pass for rows of whole 16-byte words, with the rows
// arriving by bulk asynchronous copies: tpr threads (whole warps) share a row
// and walk the rows on their own, each group of threads with a ring of `stages`
// rows per input tensor in shared memory, refilled by its first thread.  The
// loads of the next rows are in flight while a row is summed and written, so
// the memory stays busy through the two sums; groups meet only in their own
// named barrier.
//
// The stage that a group refills after the barrier of row i is the one of row
// i - 1: by then every thread of the group has left row i - 1 behind.
//
// 16384 x 2048 bf16 with residual takes 77 to 81 us with dropout (335.9 MB, 4.2 to
// 4.3 TB/s) and 59 to 62 without (268.8 MB, 4.3 to 4.5 TB/s) in captured runs, dw and
// db included: bound by issue and the latency of a row's chain at 16 warps per SM
// (with dropout 56 % of the issue slots, 43 instructions per element against 29
// without).  The plain kernel above took 117 us.
//
// NV groups of eight per thread and row.  With two, what both passes use (gw
// and xhat) stays in registers beside the 32 partial sums of dw and db; with
// four (rows beyond 8192 elements) it is read and formed again.
struct RingParams {
  BwdParams b;
  int32_t stages, tensors;   // tensors: 2, or 3 with dsum_in
  int32_t row_bytes;
  int32_t* err;
  uint64_t wait_ns;
};

constexpr int kRingMaxGroups = 8;    // row groups per block
constexpr int kRingMaxStages = 4;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void group_sync(int rg, int tpr) {
  if (tpr == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(rg + 1), "r"(tpr) : "memory");
}

template <bool BF16, int NV, bool DROP>
__global__ void __launch_bounds__(512) norm_bwd_ring_kernel(const RingParams rp) {
  // what both passes use stays in registers where the partial sums leave room
  constexpr bool KEEP = NV <= 2;
  const BwdParams& p = rp.b;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kRingMaxGroups][kRingMaxStages];
  __shared__ float2 red[2][16];       // [parity][warp]
  __shared__ int abort_flag;
  const int rpb = blockDim.x / p.tpr;
  const int rg = threadIdx.x / p.tpr, t = threadIdx.x - rg * p.tpr;
  const int G = p.D / kGroup;
  const int S = rp.stages, nt = rp.tensors;
  const int64_t stage_bytes = int64_t(rp.row_bytes) * nt;
  uint8_t* ring = smem + rg * S * stage_bytes;
  uint64_t* full = bars[rg];
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0) {
    for (int g = 0; g < rpb; ++g)
      for (int s = 0; s < S; ++s) mbar_init(&bars[g][s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  wait_prior_kernels();
  if (p.part) release_dependents();
  const int64_t row0 = int64_t(blockIdx.x) * rpb + rg, step = int64_t(gridDim.x) * rpb;
  int issued = 0;      // (the filling thread's) fills so far, in ring order
  auto fill = [&](int64_t row, int s) {
    ++issued;
    uint8_t* dst = ring + s * stage_bytes;
    const int64_t off = row * rp.row_bytes;
    mbar_arrive_expect_tx(&full[s], uint32_t(stage_bytes));
    bulk_load(dst, static_cast<const uint8_t*>(p.dy) + off, rp.row_bytes, &full[s]);
    bulk_load(dst + rp.row_bytes, static_cast<const uint8_t*>(p.s) + off, rp.row_bytes, &full[s]);
    if (nt > 2)
      bulk_load(dst + 2 * int64_t(rp.row_bytes), static_cast<const uint8_t*>(p.dsum_in) + off,
                rp.row_bytes, &full[s]);
  };
  if (t == 0)
    for (int s = 0; s < S; ++s)
      if (row0 + s * step < p.T) fill(row0 + s * step, s);
  const float inv_d = 1.0f / float(p.D);
  F2 aw[NV][4], ab[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) aw[i][j] = ab[i][j] = f2(0.0f);
  // (a missing weight is multiplied as ones, a missing gradient added as
  // zeros below: a test per pair would put a branch around each)
  F2 ws[KEEP ? NV : 1][4];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Raw8<BF16> w = ones_raw8<BF16>();
      if (p.w && t + i * p.tpr < G)
        w = load_raw8<BF16, VEC>(p.w, 0, span<VEC>(i, t, p.tpr, p.D));
#pragma unroll
      for (int j = 0; j < 4; ++j) ws[i][j] = pair(w, j);
    }
  }
  DropKey key{};
  if (DROP) key = drop_key(p.drop);
  int st = 0, par = 0;
  uint32_t ph = 0;
  // a row's mean and rstd are loaded a row ahead, out of the way of its sums
  float mu_next = 0.0f, rs_next = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= p.T) return;
    if (!p.rms) mu_next = p.mean[row];
    rs_next = p.rstd[row];
  };
  fetch(row0);
  for (int64_t row = row0; row < p.T; row += step, par ^= 1) {
    const float mu = mu_next, rs = rs_next;
    fetch(row + step);
    // After a wait that ran out the group goes on with what the stage holds
    // (its outputs are then undefined); the flag ends every later wait, and no
    // stage is filled again.
    mbar_wait(&full[st], ph, abort, rp.err, rp.wait_ns);
    const uint8_t* src = ring + st * stage_bytes;
    F2 c1 = f2(0.0f), c2 = f2(0.0f);
    const F2 nmu = f2(-mu), rs2 = f2(rs);
    F2 gws[KEEP ? NV : 1][4], xhs[KEEP ? NV : 1][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = t + i * p.tpr;
      const Span at = span<VEC>(i, t, p.tpr, p.D);
      if (g < G) {
        const Raw8<BF16> dyr = load_raw8<BF16, VEC>(src, 0, at);
        const Raw8<BF16> sr = load_raw8<BF16, VEC>(src + rp.row_bytes, 0, at);
        Raw8<BF16> w = ones_raw8<BF16>();
        if (!KEEP && p.w) w = load_raw8<BF16, VEC>(p.w, 0, at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 dy = pair(dyr, j), xh = (pair(sr, j) + nmu) * rs2;
          const F2 gw = dy * (KEEP ? ws[KEEP ? i : 0][j] : pair(w, j));
          aw[i][j] = fma2(dy, xh, aw[i][j]);
          ab[i][j] = ab[i][j] + dy;
          c1 = c1 + gw;
          c2 = fma2(gw, xh, c2);
          if (KEEP) {
            gws[KEEP ? i : 0][j] = gw;
            xhs[KEEP ? i : 0][j] = xh;
          }
        }
      }
    }
    float a0, a1, b0, b1;
    f2_get(c1, a0, a1);
    f2_get(c2, b0, b1);
    a0 += a1;
    b0 += b1;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      a0 += __shfl_xor_sync(0xffffffffu, a0, m);
      b0 += __shfl_xor_sync(0xffffffffu, b0, m);
    }
    if (p.tpr > 32) {
      const int warp = threadIdx.x >> 5, wpr = p.tpr >> 5, w0 = warp / wpr * wpr;
      if ((threadIdx.x & 31) == 0) red[par][warp] = make_float2(a0, b0);
      group_sync(rg, p.tpr);
      a0 = b0 = 0.0f;
      for (int k = 0; k < wpr; ++k) {
        const float2 v = red[par][w0 + k];
        a0 += v.x;
        b0 += v.y;
      }
    } else {
      __syncwarp();
    }
    // row - step is behind every thread of the group: its stage takes the
    // row S - 1 steps ahead of this one
    if (t == 0 && row != row0 && row + (S - 1) * step < p.T && !*abort)
      fill(row + (S - 1) * step, st == 0 ? S - 1 : st - 1);
    uint4 u[NV];
    if (DROP) philox_n<NV>(key, uint64_t(row) * uint64_t(G) + t, uint32_t(p.tpr), u);
    const F2 nc1 = f2(p.rms ? 0.0f : -a0 * inv_d), nc2 = f2(-b0 * inv_d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = t + i * p.tpr;
      if (g >= G) break;
      const Span at = span<VEC>(i, t, p.tpr, p.D);
      Raw8<BF16> dyr, sr, w = ones_raw8<BF16>(), add = zero_raw8<BF16>();
      if (!KEEP) {
        dyr = load_raw8<BF16, VEC>(src, 0, at);
        sr = load_raw8<BF16, VEC>(src + rp.row_bytes, 0, at);
        if (p.w) w = load_raw8<BF16, VEC>(p.w, 0, at);
      }
      if (nt > 2) add = load_raw8<BF16, VEC>(src + 2 * int64_t(rp.row_bytes), 0, at);
      float d[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        F2 gw, xh;
        if constexpr (KEEP) {
          gw = gws[i][j];
          xh = xhs[i][j];
        } else {
          xh = (pair(sr, j) + nmu) * rs2;
          gw = pair(dyr, j) * pair(w, j);
        }
        const F2 ds = fma2(fma2(xh, nc2, gw + nc1), rs2, pair(add, j));
        f2_get(ds, d[2 * j], d[2 * j + 1]);
      }
      if (p.dsum) store_raw8<BF16, VEC>(p.dsum, row * p.D, at, pack_raw8<BF16>(d));
      if (p.dx) {
        // from the fp32 gradient, not from the rounded dsum
        if (DROP) drop8(u[i], p.drop.below, p.drop.scale, d);
        store_raw8<BF16, VEC>(p.dx, row * p.D, at, pack_raw8<BF16>(d));
      }
    }
    if (++st == S) {
      st = 0;
      ph ^= 1;
    }
  }
  // every fill was waited for above, unless a wait ran out: then let the
  // copies in flight land before the shared memory goes away
  if (*abort && t == 0) drain_ring(full, S, issued % S, uint32_t(issued / S) & 1, issued);
  if (!p.part) return;
  float* out = p.part + int64_t(blockIdx.x) * 2 * p.D;
  if (rpb == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = t + i * p.tpr;
      if (g >= G) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        f2_get(aw[i][j], lo, hi);
        *reinterpret_cast<float2*>(out + g * kGroup + 2 * j) = make_float2(lo, hi);
        f2_get(ab[i][j], lo, hi);
        *reinterpret_cast<float2*>(out + p.D + g * kGroup + 2 * j) = make_float2(lo, hi);
      }
    }
    return;
  }
  // the block's row groups add up in group order, [row group][2][D] floats
  // over the rings, which no copy writes any more
  __syncthreads();
  float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int g = t + i * p.tpr;
    if (g >= G) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      f2_get(aw[i][j], lo, hi);
      *reinterpret_cast<float2*>(acc + (rg * 2 + 0) * p.D + g * kGroup + 2 * j) = make_float2(lo, hi);
      f2_get(ab[i][j], lo, hi);
      *reinterpret_cast<float2*>(acc + (rg * 2 + 1) * p.D + g * kGroup + 2 * j) = make_float2(lo, hi);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * p.D; k += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < rpb; ++q) s += acc[q * 2 * p.D + k];
    out[k] = s;
  }
}

// dw[d], db[d] = sums over the blocks of the backward kernel, in block order
// within each of 32 slices, then over the slices in order.  Block: 32 columns
// x 32 slices.
constexpr int kWgCols = 32, kWgSlices = 32;
__global__ void __launch_bounds__(kWgCols* kWgSlices)
    norm_wgrad_kernel(const float* part, int blocks, int D, float* dw, float* db) {
  __shared__ float s[kWgSlices][kWgCols];
  wait_prior_kernels();   // the partial sums are written
  const int cx = threadIdx.x % kWgCols, sl = threadIdx.x / kWgCols;
  const int d = blockIdx.x * kWgCols + cx;
  float* dst = blockIdx.y ? db : dw;
  if (!dst) return;
  float a = 0.0f;
  if (d < D) {
    const float* src = part + int64_t(blockIdx.y) * D + d;
#pragma unroll 8
    for (int k = sl; k < blocks; k += kWgSlices) a += src[int64_t(k) * 2 * D];
  }
  s[sl][cx] = a;
  __syncthreads();
  if (sl == 0 && d < D) {
#pragma unroll
    for (int k = 1; k < kWgSlices; ++k) a += s[k][cx];
    dst[d] = a;
  }
}

inline int cdiv(int64_t a, int64_t b) { return int((a + b - 1) / b); }

// Groups per thread of the forward kernel: with few rows one, so that a row is
// as many threads wide as it can be and its chain of loads and sums as short;
// with many four, so that the two sums across threads cost little per element
// and each thread has four loads per tensor in flight.
int row_groups_per_thread(int G, int T, int num_sms) {
  if (G > 1024) return 4;
  if (T <= 2 * num_sms) return G > 512 ? 2 : 1;
  return G > 64 ? 4 : (G > 32 ? 2 : 1);
}

bool vec_ok(int D, std::initializer_list<const void*> ps) {
  if (D % kGroup) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}

template <bool BF16, int NV>
staple_status fwd_go(const FwdParams& p, bool vec, int grid, int block, cudaStream_t st) {
  void (*kern)(FwdParams);
  if (p.drop.rng)
    kern = vec ? norm_fwd_kernel<BF16, NV, VEC, true> : norm_fwd_kernel<BF16, NV, STRIDE, true>;
  else
    kern = vec ? norm_fwd_kernel<BF16, NV, VEC, false> : norm_fwd_kernel<BF16, NV, STRIDE, false>;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("norm_fwd", st,
             ce = launch_dependent(kern, dim3(unsigned(grid)), unsigned(block), 0, st, 1, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16>
staple_status fwd_nv(const FwdParams& p, int nv, bool vec, int grid, int block, cudaStream_t st) {
  switch (nv) {
    case 1: return fwd_go<BF16, 1>(p, vec, grid, block, st);
    case 2: return fwd_go<BF16, 2>(p, vec, grid, block, st);
    default: return fwd_go<BF16, 4>(p, vec, grid, block, st);
  }
}

// Rows in flight per thread of the plain backward kernel: as many as its
// registers hold, one where there are too few rows to go round the SMs.
constexpr int rows_in_flight(bool bf16, int nv) {
  return nv == 1 ? (bf16 ? 4 : 2) : (nv == 2 && bf16 ? 2 : 1);
}

template <bool BF16, int NV, int R>
staple_status bwd_go(const BwdParams& p, bool vec, int grid, int block, size_t smem,
                     cudaStream_t st) {
  void (*kern)(BwdParams) = p.drop.rng ? norm_bwd_kernel<BF16, NV, R, STRIDE, true>
                                       : norm_bwd_kernel<BF16, NV, R, STRIDE, false>;
  // whole vectors come here only from rows too short for the ring kernel, and
  // from fp32 rows too long for it
  if constexpr (NV == 1 || (NV == 4 && !BF16))
    if (vec)
      kern = p.drop.rng ? norm_bwd_kernel<BF16, NV, R, VEC, true>
                        : norm_bwd_kernel<BF16, NV, R, VEC, false>;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("norm_bwd", st,
             ce = launch_dependent(kern, dim3(unsigned(grid)), unsigned(block), smem, st, 1, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16>
staple_status bwd_nv(const BwdParams& p, int nv, int R, bool vec, int grid, int block, size_t smem,
                     cudaStream_t st) {
  if (nv == 1 && R > 1)
    return bwd_go<BF16, 1, rows_in_flight(BF16, 1)>(p, vec, grid, block, smem, st);
  if (BF16 && nv == 2 && R > 1) return bwd_go<BF16, 2, 2>(p, vec, grid, block, smem, st);
  switch (nv) {
    case 1: return bwd_go<BF16, 1, 1>(p, vec, grid, block, smem, st);
    case 2: return bwd_go<BF16, 2, 1>(p, vec, grid, block, smem, st);
    default: return bwd_go<BF16, 4, 1>(p, vec, grid, block, smem, st);
  }
}

// The ring kernel's launch: block, stages, blocks per SM and shared memory;
// false where the rows do not suit it (then the plain kernel runs).
struct RingPlan {
  int nv, tpr, rpb, stages, per_sm;
  size_t smem;
};
bool plan_ring(int D, int es, int tensors, RingPlan* out) {
  const int G = D / kGroup;
  RingPlan r{};
  // (four only where two would need more than 512 threads)
  r.nv = G > 1024 ? 4 : (G > 32 ? 2 : 1);
  r.tpr = std::max(32, threads_per_row(G, r.nv));
  // one block of 512 threads per SM: fewer blocks leave fewer partial sums of
  // dw and db (16384 x 2048: 77.8 us, against 80.5 with two blocks of 256)
  r.rpb = std::min(kRingMaxGroups, std::max(1, 512 / r.tpr));
  const size_t row_stage = size_t(D) * es * tensors * r.rpb;
  for (r.per_sm = std::max(1, 512 / (r.rpb * r.tpr)); r.per_sm >= 1; --r.per_sm) {
    // 228 KB per SM, of which each block's share loses 1 KB to the system and
    // under 1 KB to static arrays; 227 KB at most per block
    const size_t avail = std::min<size_t>(size_t(228) * 1024 / r.per_sm - 2048, 226 * 1024);
    r.stages = int(std::min<size_t>(kRingMaxStages, avail / row_stage));
    if (r.stages >= 2) {
      r.smem = row_stage * r.stages;
      *out = r;
      return true;
    }
  }
  return false;
}

template <bool BF16, int NV, bool DROP>
staple_status ring_go(const DeviceInfo& di, const RingParams& p, int grid, int block, size_t smem,
                      cudaStream_t st) {
  auto kern = norm_bwd_ring_kernel<BF16, NV, DROP>;
  // set once per device, so that no attribute call happens during a capture
  static std::atomic<uint64_t> attr_done{0};
  const uint64_t bit = uint64_t(1) << (di.device & 63);
  if (!(attr_done.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) !=
        cudaSuccess)
      return STAPLE_ECUDA;
    attr_done.fetch_or(bit);
  }
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("norm_bwd", st,
             ce = launch_dependent(kern, dim3(unsigned(grid)), unsigned(block), smem, st, 1, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16, bool DROP>
staple_status ring_nv(const DeviceInfo& di, const RingParams& p, int nv, int grid, int block,
                      size_t smem, cudaStream_t st) {
  switch (nv) {
    case 1: return ring_go<BF16, 1, DROP>(di, p, grid, block, smem, st);
    case 2: return ring_go<BF16, 2, DROP>(di, p, grid, block, smem, st);
    default: return ring_go<BF16, 4, DROP>(di, p, grid, block, smem, st);
  }
}

DropParams drop_params(const staple_drop* d) {
  DropParams r{};
  if (!d) return r;
  const uint32_t thr = uint32_t(d->p * 65536.0 + 0.5);
  if (thr == 0) return r;
  r.below = uint32_t((uint64_t(thr) << 16) - 1);
  r.rng = static_cast<const uint64_t*>(d->rng);
  r.site = d->site;
  r.scale = thr < 65536 ? float(65536.0 / double(65536 - thr)) : 0.0f;
  return r;
}

// Dropout with an optional residual on its own: unit n is group g of row t.
// Bound by HBM: 8192 x 4096 bf16 with residual takes 33.5 us a call among others (6.0
// TB/s, 0.93 of a copy), 32 in a captured run; the ten rounds per eight elements fit
// beside it.
// VEC: D % 8 == 0, so n alone gives the address.
struct DropoutParams {
  const void* x;
  const void* res;
  void* out;
  DropParams drop;
  int64_t units;
  int32_t D, G, tpr, per_row;
};

template <bool BF16, RowLayout L, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutParams p) {
  wait_prior_kernels();
  // VEC: a unit is eight elements.  STRIDE: a row has `per_row` units, tpr of them
  // (a warp's lanes, or fewer for short rows) side by side.
  const int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (L == VEC && u >= p.units) return;
  int64_t off = u * kGroup, draw = u;
  Span s{0, 1, kGroup};
  const int t = L == VEC ? 0 : threadIdx.x & (p.tpr - 1);
  if (L == STRIDE) {
    const int64_t row = u / p.per_row;
    const int g = int(u - row * p.per_row);
    s.off = (g - t) * kGroup + t;
    s.step = p.tpr;
    // (not (D - off + tpr - 1) / tpr, which leaves 32 bits for D within tpr of 2^31)
    s.n = u < p.units && s.off < p.D ? min(kGroup, (p.D - 1 - s.off) / p.tpr + 1) : 0;
    off = row * p.D;
    draw = row * p.G + g;
  }
  const Raw8<BF16> xr = load_raw8<BF16, L>(p.x, off, s);
  Raw8<BF16> rr = zero_raw8<BF16>();
  if (p.res) rr = load_raw8<BF16, L>(p.res, off, s);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = xr.get(j);
  if (DROP) {
    const uint4 draws = philox(drop_key(p.drop), uint64_t(draw));
    if constexpr (L == VEC) drop8(draws, p.drop.below, p.drop.scale, v);
    else drop8_kept(stride_keep(draws, p.drop.below, t, p.tpr), p.drop.scale, v);
  }
  if (p.res)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += rr.get(j);
  store_raw8<BF16, L>(p.out, off, s, pack_raw8<BF16>(v));
}

template <bool BF16, RowLayout L>
staple_status dropout_go(const DropoutParams& p, cudaStream_t st) {
  const unsigned grid = unsigned((p.units + 255) / 256);
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("dropout", st,
             ce = launch_dependent(p.drop.rng ? dropout_kernel<BF16, L, true>
                                              : dropout_kernel<BF16, L, false>,
                                   dim3(grid), 256, 0, st, 1, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

}  // namespace

size_t norm_workspace_bytes(int T, int D) {
  return size_t(std::min(T, kNormMaxBlocks)) * 2 * size_t(D) * sizeof(float);
}

staple_status launch_norm_fwd(const DeviceInfo& di, bool bf16, bool rms, int T, int D, const void* x, const void* res,
                              const staple_drop* drop, const void* w, const void* b, float eps,
                              void* sum, void* y, float* mean, float* rstd, cudaStream_t st) {
  if (T == 0) return STAPLE_OK;
  FwdParams p{x, res, w, b, sum, y, mean, rstd, drop_params(drop), T, D, 0, eps, rms};
  const int G = groups_of(D);
  const int nv = row_groups_per_thread(G, T, di.num_sms);
  p.tpr = threads_per_row(G, nv);
  const int rpb = std::max(1, 128 / p.tpr);
  const int grid = cdiv(T, rpb), block = rpb * p.tpr;
  const bool vec = vec_ok(D, {x, res, w, b, sum, y});
  return bf16 ? fwd_nv<true>(p, nv, vec, grid, block, st)
              : fwd_nv<false>(p, nv, vec, grid, block, st);
}

staple_status launch_norm_bwd(const DeviceInfo& di, bool bf16, bool rms, int T, int D,
                              const void* dy, const void* s, const void* w, const float* mean,
                              const float* rstd, const void* dsum_in, const staple_drop* drop,
                              void* dsum, void* dx, float* dw, float* db, float* part,
                              int32_t* err, cudaStream_t st) {
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, size_t(D) * 4, st) != cudaSuccess) return STAPLE_ECUDA;
    if (db && cudaMemsetAsync(db, 0, size_t(D) * 4, st) != cudaSuccess) return STAPLE_ECUDA;
    return STAPLE_OK;
  }
  BwdParams p{dy, s, w, mean, rstd, dsum_in, dsum, dx, (dw || db) ? part : nullptr,
              drop_params(drop), T, D, 0, rms};
  const int G = groups_of(D);
  const bool vec = vec_ok(D, {dy, s, w, dsum_in, dsum, dx});
  staple_status r;
  int grid;
  RingPlan rp;
  if (vec && G >= 32 && plan_ring(D, bf16 ? 2 : 4, dsum_in ? 3 : 2, &rp)) {
    p.tpr = rp.tpr;
    grid = std::min(std::min(cdiv(T, rp.rpb), kNormMaxBlocks), di.num_sms * rp.per_sm);
    const RingParams q{p, rp.stages, dsum_in ? 3 : 2, D * (bf16 ? 2 : 4), err, di.wait_ns};
    const int block = rp.rpb * rp.tpr;
    if (bf16)
      r = p.drop.rng ? ring_nv<true, true>(di, q, rp.nv, grid, block, rp.smem, st)
                     : ring_nv<true, false>(di, q, rp.nv, grid, block, rp.smem, st);
    else
      r = p.drop.rng ? ring_nv<false, true>(di, q, rp.nv, grid, block, rp.smem, st)
                     : ring_nv<false, false>(di, q, rp.nv, grid, block, rp.smem, st);
  } else {
    const int nv = G <= 512 ? 1 : (G <= 1024 ? 2 : 4);
    p.tpr = threads_per_row(G, nv);
    const int rpb = std::max(1, 256 / p.tpr);
    const int block = rpb * p.tpr;
    const int blocks = di.num_sms * std::max(1, 1024 / block);
    const int R = T <= 4 * int64_t(blocks) * rpb ? 1 : rows_in_flight(bf16, nv);
    grid = std::min(std::min(cdiv(T, int64_t(rpb) * R), kNormMaxBlocks), blocks);
    const size_t smem = rpb > 1 ? size_t(rpb) * 2 * p.tpr * nv * kGroup * sizeof(float) : 0;
    r = bf16 ? bwd_nv<true>(p, nv, R, vec, grid, block, smem, st)
             : bwd_nv<false>(p, nv, R, vec, grid, block, smem, st);
  }
  if (r != STAPLE_OK || !p.part) return r;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("norm_wgrad", st,
             ce = launch_dependent(norm_wgrad_kernel, dim3(unsigned(cdiv(D, kWgCols)), 2),
                                   kWgCols * kWgSlices, 0, st, 1, part, grid, D, dw, db));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

staple_status launch_dropout(bool bf16, int T, int D, const void* x, const void* res,
                             const staple_drop* drop, void* out, cudaStream_t st) {
  if (T == 0) return STAPLE_OK;
  DropoutParams p{x, res, out, drop_params(drop), 0, D, groups_of(D), 0, 0};
  const bool vec = vec_ok(D, {x, res, out});
  p.tpr = std::min(32, threads_per_row(p.G, 1));
  p.per_row = vec ? p.G : (p.G + p.tpr - 1) / p.tpr * p.tpr;
  p.units = int64_t(T) * p.per_row;
  if (bf16) return vec ? dropout_go<true, VEC>(p, st) : dropout_go<true, STRIDE>(p, st);
  return vec ? dropout_go<false, VEC>(p, st) : dropout_go<false, STRIDE>(p, st);
}

}  // namespace stp
