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

template <bool BF16, int NV, bool VEC, bool DROP>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const FwdParams p) {
  __shared__ float red[2][32];
  const int rpb = blockDim.x / p.tpr;
  const int rg = threadIdx.x / p.tpr, t = threadIdx.x - rg * p.tpr;
  const int64_t row = int64_t(blockIdx.x) * rpb + rg;
  const bool row_ok = row < p.T;
  const int G = (p.D + kGroup - 1) / kGroup;
  const int64_t base = row * p.D;
  Raw8<BF16> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int g = t + i * p.tpr;
    xr[i] = rr[i] = zero_raw8<BF16>();
    if (row_ok && g < G) {
      const int e = g * kGroup, n = min(kGroup, p.D - e);
      xr[i] = load_raw8<BF16, VEC>(p.x, base + e, n);
      if (p.res) rr[i] = load_raw8<BF16, VEC>(p.res, base + e, n);
    }
  }
  float v[NV][8];
  float s1[1] = {0.0f};
  DropKey key{};
  if (DROP) key = drop_key(p.drop);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int g = t + i * p.tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = xr[i].get(j);
    if (DROP) drop8(key, uint64_t(row) * uint64_t(G) + g, p.drop.thr, p.drop.scale, v[i]);
    if (p.res)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += rr[i].get(j);
    if (p.sum) {
      // the norm sees the sum as stored, which is what the backward pass reads
      const Raw8<BF16> sr = pack_raw8<BF16>(v[i]);
      if (row_ok && g < G)
        store_raw8<BF16, VEC>(p.sum, base + g * kGroup, min(kGroup, p.D - g * kGroup), sr);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = sr.get(j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s1[0] += v[i][j];   // elements past D are zero
  }
  const float inv_d = 1.0f / float(p.D);
  float mean = 0.0f;
  if (!p.rms) {
    row_sum(s1, p.tpr, red[0]);
    mean = s1[0] * inv_d;
  }
  float s2[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int left = p.D - (t + i * p.tpr) * kGroup;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) s2[0] = fmaf(v[i][j] - mean, v[i][j] - mean, s2[0]);
  }
  row_sum(s2, p.tpr, red[1]);
  const float rstd = 1.0f / sqrtf(s2[0] * inv_d + p.eps);
  if (!row_ok) return;
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int g = t + i * p.tpr;
    if (g >= G) break;
    const int e = g * kGroup, n = min(kGroup, p.D - e);
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (v[i][j] - mean) * rstd;
    if (p.w) {
      const Raw8<BF16> w = load_raw8<BF16, VEC>(p.w, e, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= w.get(j);
    }
    if (p.b) {
      const Raw8<BF16> b = load_raw8<BF16, VEC>(p.b, e, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += b.get(j);
    }
    store_raw8<BF16, VEC>(p.y, base + e, n, pack_raw8<BF16>(o));
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

// NV groups per thread and row, R rows in flight per thread.
template <bool BF16, int NV, int R, bool VEC, bool DROP>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const BwdParams p) {
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
        const int g = t + i * p.tpr;
        dyr[r][i] = sr[r][i] = zero_raw8<BF16>();
        if (ok && g < G) {
          const int e = g * kGroup, n = min(kGroup, p.D - e);
          dyr[r][i] = load_raw8<BF16, VEC>(p.dy, row * p.D + e, n);
          sr[r][i] = load_raw8<BF16, VEC>(p.s, row * p.D + e, n);
        }
      }
    }
    float c[2 * R];
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) c[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = t + i * p.tpr;
      Raw8<BF16> w = zero_raw8<BF16>();
      if (p.w && g < G)
        w = load_raw8<BF16, VEC>(p.w, g * kGroup, min(kGroup, p.D - g * kGroup));
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dy = dyr[r][i].get(j);        // zero past the row's end
          const float xh = (sr[r][i].get(j) - mu[r]) * rs[r];
          const float gw = p.w ? dy * w.get(j) : dy;
          aw[i][j] = fmaf(dy, xh, aw[i][j]);
          ab[i][j] += dy;
          c[2 * r] += gw;
          c[2 * r + 1] = fmaf(gw, xh, c[2 * r + 1]);
        }
    }
    row_sum(c, p.tpr, red[buf]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = t + i * p.tpr;
      if (g >= G) break;
      const int e = g * kGroup, n = min(kGroup, p.D - e);
      Raw8<BF16> w = zero_raw8<BF16>();
      if (p.w) w = load_raw8<BF16, VEC>(p.w, e, n);
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
          const float gw = p.w ? dy * w.get(j) : dy;
          d[j] = (gw - c1 - xh * c2) * rs[r];
        }
        if (p.dsum_in) {
          const Raw8<BF16> a = load_raw8<BF16, VEC>(p.dsum_in, row * p.D + e, n);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += a.get(j);
        }
        if (p.dsum) store_raw8<BF16, VEC>(p.dsum, row * p.D + e, n, pack_raw8<BF16>(d));
        if (p.dx) {
          // from the fp32 gradient, not from the rounded dsum
          if (DROP) drop8(key, uint64_t(row) * uint64_t(G) + g, p.drop.thr, p.drop.scale, d);
          store_raw8<BF16, VEC>(p.dx, row * p.D + e, n, pack_raw8<BF16>(d));
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
        const int e = (t + i * p.tpr) * kGroup + j;
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
      const int e = (t + i * p.tpr) * kGroup + j;
      if (e < p.D) {
        out[e] = aw[i][j];
        out[p.D + e] = ab[i][j];
      }
    }
}

// dw[d], db[d] = sums over the blocks of the backward kernel, in block order
// within each of 8 slices, then over the slices in order.  Block: 32 columns
// x 8 slices.
constexpr int kWgCols = 32, kWgSlices = 8;
__global__ void __launch_bounds__(kWgCols* kWgSlices)
    norm_wgrad_kernel(const float* part, int blocks, int D, float* dw, float* db) {
  __shared__ float s[kWgSlices][kWgCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partial sums are written
  const int cx = threadIdx.x % kWgCols, sl = threadIdx.x / kWgCols;
  const int d = blockIdx.x * kWgCols + cx;
  float* dst = blockIdx.y ? db : dw;
  if (!dst) return;
  float a = 0.0f;
  if (d < D) {
    const float* src = part + int64_t(blockIdx.y) * D + d;
#pragma unroll 4
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

bool vec_ok(int D, std::initializer_list<const void*> ps) {
  if (D % kGroup) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}

template <bool BF16, int NV, bool VEC>
staple_status fwd_go(const FwdParams& p, int grid, int block, cudaStream_t st) {
  if (p.drop.rng)
    STP_LAUNCH("norm_fwd", st, norm_fwd_kernel<BF16, NV, VEC, true><<<grid, block, 0, st>>>(p));
  else
    STP_LAUNCH("norm_fwd", st, norm_fwd_kernel<BF16, NV, VEC, false><<<grid, block, 0, st>>>(p));
  return cudaGetLastError() == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16, bool VEC>
staple_status fwd_nv(const FwdParams& p, int nv, int grid, int block, cudaStream_t st) {
  switch (nv) {
    case 1: return fwd_go<BF16, 1, VEC>(p, grid, block, st);
    case 2: return fwd_go<BF16, 2, VEC>(p, grid, block, st);
    default: return fwd_go<BF16, 4, VEC>(p, grid, block, st);
  }
}

constexpr int rows_in_flight(bool bf16, int nv) { return nv == 1 ? (bf16 ? 4 : 2) : (nv == 2 && bf16 ? 2 : 1); }

template <bool BF16, int NV, bool VEC, bool DROP>
staple_status bwd_go(const BwdParams& p, int grid, int block, size_t smem, cudaStream_t st) {
  STP_LAUNCH("norm_bwd", st,
             norm_bwd_kernel<BF16, NV, rows_in_flight(BF16, NV), VEC, DROP>
             <<<grid, block, smem, st>>>(p));
  return cudaGetLastError() == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16, bool VEC, bool DROP>
staple_status bwd_nv(const BwdParams& p, int nv, int grid, int block, size_t smem,
                     cudaStream_t st) {
  switch (nv) {
    case 1: return bwd_go<BF16, 1, VEC, DROP>(p, grid, block, smem, st);
    case 2: return bwd_go<BF16, 2, VEC, DROP>(p, grid, block, smem, st);
    default: return bwd_go<BF16, 4, VEC, DROP>(p, grid, block, smem, st);
  }
}

DropParams drop_params(const staple_drop* d) {
  DropParams r{};
  if (!d) return r;
  r.thr = uint32_t(d->p * 65536.0 + 0.5);
  if (r.thr == 0) return r;
  r.rng = static_cast<const uint64_t*>(d->rng);
  r.site = d->site;
  r.scale = r.thr < 65536 ? float(65536.0 / double(65536 - r.thr)) : 0.0f;
  return r;
}

// Dropout with an optional residual on its own: unit n is group g of row t.
// VEC: D % 8 == 0, so n alone gives the address.
struct DropoutParams {
  const void* x;
  const void* res;
  void* out;
  DropParams drop;
  int64_t units;
  int32_t D, G;
};

template <bool BF16, bool VEC, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutParams p) {
  const int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (u >= p.units) return;
  int64_t off = u * kGroup;
  int n = kGroup;
  if (!VEC) {
    const int64_t row = u / p.G;
    const int e = int(u - row * p.G) * kGroup;
    off = row * p.D + e;
    n = min(kGroup, p.D - e);
  }
  const Raw8<BF16> xr = load_raw8<BF16, VEC>(p.x, off, n);
  Raw8<BF16> rr = zero_raw8<BF16>();
  if (p.res) rr = load_raw8<BF16, VEC>(p.res, off, n);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = xr.get(j);
  if (DROP) drop8(drop_key(p.drop), uint64_t(u), p.drop.thr, p.drop.scale, v);
  if (p.res)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += rr.get(j);
  store_raw8<BF16, VEC>(p.out, off, n, pack_raw8<BF16>(v));
}

template <bool BF16, bool VEC>
staple_status dropout_go(const DropoutParams& p, cudaStream_t st) {
  const unsigned grid = unsigned((p.units + 255) / 256);
  if (p.drop.rng)
    STP_LAUNCH("dropout", st, dropout_kernel<BF16, VEC, true><<<grid, 256, 0, st>>>(p));
  else
    STP_LAUNCH("dropout", st, dropout_kernel<BF16, VEC, false><<<grid, 256, 0, st>>>(p));
  return cudaGetLastError() == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

}  // namespace

size_t norm_workspace_bytes(int T, int D) {
  return size_t(std::min(T, kNormMaxBlocks)) * 2 * size_t(D) * sizeof(float);
}

staple_status launch_norm_fwd(bool bf16, bool rms, int T, int D, const void* x, const void* res,
                              const staple_drop* drop, const void* w, const void* b, float eps,
                              void* sum, void* y, float* mean, float* rstd, cudaStream_t st) {
  if (T == 0) return STAPLE_OK;
  FwdParams p{x, res, w, b, sum, y, mean, rstd, drop_params(drop), T, D, 0, eps, rms};
  const int G = groups_of(D);
  const int nv = G <= 512 ? 1 : (G <= 1024 ? 2 : 4);
  p.tpr = threads_per_row(G, nv);
  const int rpb = std::max(1, 256 / p.tpr);
  const int grid = cdiv(T, rpb), block = rpb * p.tpr;
  const bool vec = vec_ok(D, {x, res, w, b, sum, y});
  if (bf16) return vec ? fwd_nv<true, true>(p, nv, grid, block, st)
                       : fwd_nv<true, false>(p, nv, grid, block, st);
  return vec ? fwd_nv<false, true>(p, nv, grid, block, st)
             : fwd_nv<false, false>(p, nv, grid, block, st);
}

staple_status launch_norm_bwd(const DeviceInfo& di, bool bf16, bool rms, int T, int D,
                              const void* dy, const void* s, const void* w, const float* mean,
                              const float* rstd, const void* dsum_in, const staple_drop* drop,
                              void* dsum, void* dx, float* dw, float* db, float* part,
                              cudaStream_t st) {
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, size_t(D) * 4, st) != cudaSuccess) return STAPLE_ECUDA;
    if (db && cudaMemsetAsync(db, 0, size_t(D) * 4, st) != cudaSuccess) return STAPLE_ECUDA;
    return STAPLE_OK;
  }
  BwdParams p{dy, s, w, mean, rstd, dsum_in, dsum, dx, (dw || db) ? part : nullptr,
              drop_params(drop), T, D, 0, rms};
  const int G = groups_of(D);
  const int nv = G <= 512 ? 1 : (G <= 1024 ? 2 : 4);
  p.tpr = threads_per_row(G, nv);
  const int rpb = std::max(1, 256 / p.tpr);
  const int block = rpb * p.tpr;
  const int R = rows_in_flight(bf16, nv);
  const int grid = std::min(std::min(cdiv(T, int64_t(rpb) * R), kNormMaxBlocks),
                            di.num_sms * std::max(1, 512 / block));
  const size_t smem = rpb > 1 ? size_t(rpb) * 2 * p.tpr * nv * kGroup * sizeof(float) : 0;
  const bool vec = vec_ok(D, {dy, s, w, dsum_in, dsum, dx});
  staple_status r;
  if (bf16)
    r = vec ? (p.drop.rng ? bwd_nv<true, true, true>(p, nv, grid, block, smem, st)
                          : bwd_nv<true, true, false>(p, nv, grid, block, smem, st))
            : (p.drop.rng ? bwd_nv<true, false, true>(p, nv, grid, block, smem, st)
                          : bwd_nv<true, false, false>(p, nv, grid, block, smem, st));
  else
    r = vec ? (p.drop.rng ? bwd_nv<false, true, true>(p, nv, grid, block, smem, st)
                          : bwd_nv<false, true, false>(p, nv, grid, block, smem, st))
            : (p.drop.rng ? bwd_nv<false, false, true>(p, nv, grid, block, smem, st)
                          : bwd_nv<false, false, false>(p, nv, grid, block, smem, st));
  if (r != STAPLE_OK || !p.part) return r;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cdiv(D, kWgCols), 2);
  cfg.blockDim = dim3(kWgCols * kWgSlices);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t ce = cudaSuccess;
  const float* cpart = part;
  STP_LAUNCH("norm_wgrad", st,
             ce = cudaLaunchKernelEx(&cfg, norm_wgrad_kernel, cpart, grid, D, dw, db));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

staple_status launch_dropout(bool bf16, int T, int D, const void* x, const void* res,
                             const staple_drop* drop, void* out, cudaStream_t st) {
  if (T == 0) return STAPLE_OK;
  DropoutParams p{x, res, out, drop_params(drop), 0, D, groups_of(D)};
  p.units = int64_t(T) * p.G;
  const bool vec = vec_ok(D, {x, res, out});
  if (bf16) return vec ? dropout_go<true, true>(p, st) : dropout_go<true, false>(p, st);
  return vec ? dropout_go<false, true>(p, st) : dropout_go<false, false>(p, st);
}

}  // namespace stp
