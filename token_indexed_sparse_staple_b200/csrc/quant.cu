// Rows quantised to 8-bit integers with one scale each, the operands of
// staple_matmul_i8:
//
//   scale = fp32(max |x| / 127),  q = x / scale rounded to nearest even
//
// Bound by memory: a row is read once (it stays in registers between the
// maximum and the rounding) and its bytes written once.  16384 x 8192 bf16 takes
// 64.4 us a call among others (403 MB, 6.25 TB/s, 0.97 of a copy), 61 in a captured
// run; 64 x 4096 takes 1.7 us in a captured run of many.
//
// The quotient is rounded exactly, ties included, at the price of a
// multiplication: q0 = rint(x * (1 / scale)) by adding 1.5 * 2^23, whose sum
// holds q0 in its low byte, and the remainder r = x - q0 scale, which one fma
// gives exactly wherever it matters (near a tie both terms are multiples of
// 2^(e-24), for scale in [2^e, 2^(e+1)), and |r| < 2^e).  |r| < scale / 2
// shows that q0 is the nearest integer; a group of eight with any other
// element (a tie, or a product rounded across one) is divided in fp64, where
// a quotient of two fp32 numbers cannot be rounded onto a half it does not
// equal.
#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace stp {

namespace {

struct QuantParams {
  const void* x;
  int8_t* q;
  float* scale;
  int32_t T, D, tpr;
  bool release;              // the next kernel is part of the same call
  // GATE: x holds g [T][pitch] and, `up` elements further on, u (0: none)
  int64_t pitch;
  int32_t up;
  const uint16_t* e_base;    // E rows; NULL: none
  int64_t e_pitch, e_rows;
  const int32_t* e_index;
  int32_t* err;
};

constexpr float kRintMagic = 12582912.0f;   // 1.5 * 2^23
// Below this maximum (2^-60) the reciprocal of the scale or the remainder
// could leave the normal range: those rows divide in fp64.
constexpr float kTiny = 8.67361738e-19f;

__device__ __forceinline__ uint32_t q_exact(float x, double scale) {
  double d = rint(double(x) / scale);
  d = fmin(fmax(d, -127.0), 127.0);   // a subnormal scale may be far below max / 127
  return uint32_t(int(d)) & 0xffu;
}

// The same for a row of ordinary scale, without a division.  The candidate q is
// off by one at most, and only where x lies within 2^-13 scales of a tie.  There
// r = x - q scale is exact: x is at least half the scale's power of two 2^e, so x
// and q scale are multiples of 2^(e-24), and |r| < 2^e.  (For a smaller x, whose
// quotient is below 1/2, the nearest is 0; a candidate of 1 gives an |r| that
// rounds to half the scale or more, and goes to 0 either way.)
__device__ __forceinline__ uint32_t q_near(float x, float inv, float scale) {
  const float m = fmaf(x, inv, kRintMagic);
  float q = m - kRintMagic;
  const float r = fmaf(-scale, q, x), half = 0.5f * scale;
  const bool odd = __float_as_uint(m) & 1u;
  if (fabsf(r) > half || (fabsf(r) == half && odd)) q += copysignf(1.0f, r);
  return uint32_t(int(q)) & 0xffu;
}

// A group's eight bytes.
template <RowLayout L>
__device__ __forceinline__ void store8(int8_t* row, const Span& s, uint32_t lo, uint32_t hi) {
  int8_t* dst = row + s.off;
  if constexpr (L == VEC) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < s.n) dst[j * s.step] = int8_t((j < 4 ? lo >> (8 * j) : hi >> (8 * j - 32)) & 0xffu);
  }
}

__device__ __forceinline__ float gated(float g, float u, float e) {
  return g * sigmoid_f(g) * (u + e);
}

// GATE: the row is not x but the layer's gated product z = SiLU(g) (u + E),
// rounded to bf16 as the layer stores it, which thus never goes to memory.
template <bool BF16, int NV, RowLayout L, bool GATE>
// (bf16: 64 registers, so that 32 warps share an SM)
__global__ void __launch_bounds__(GATE ? 1024 : 512, BF16 && !GATE ? 2 : 1)
    quant_rows_kernel(const QuantParams p) {
  __shared__ uint32_t red[32];
  const int rpb = blockDim.x / p.tpr;
  const int rg = threadIdx.x / p.tpr, t = threadIdx.x - rg * p.tpr;
  const int64_t row = int64_t(blockIdx.x) * rpb + rg;
  const bool row_ok = row < p.T;
  const int64_t base = row * p.D;
  if constexpr (!GATE) {
    wait_prior_kernels();
    if (p.release) release_dependents();
  }
  // E is there before the product in front has run: that one releases this kernel
  // only after it has itself waited for all before it, and does not write E or the
  // ids.
  const uint16_t* e_row = nullptr;
  if (GATE && row_ok && p.e_base) {
    const int64_t idx = p.e_index[row];
    if (idx < 0 || idx >= p.e_rows) report(p.err, STAPLE_EIDRANGE);
    else e_row = p.e_base + idx * p.e_pitch;
  }
  // (eight groups per thread leave no registers to hold it)
  constexpr bool kEarlyE = GATE && NV <= 4;
  Raw8<true> early[kEarlyE ? NV : 1];
  if constexpr (kEarlyE) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Span s = span<L>(i, t, p.tpr, p.D);
      early[i] = e_row && s.n > 0 ? load_raw8<true, VEC>(e_row, 0, s) : zero_raw8<true>();
    }
  }
  if constexpr (GATE) {
    wait_prior_kernels();
    if (p.release) release_dependents();
  }
  auto load_group = [&](const Span& s, int i) {
    if constexpr (GATE) {
      const Raw8<true> gr = load_raw8<true, VEC>(p.x, row * p.pitch, s);
      Raw8<true> ur = zero_raw8<true>(), er = zero_raw8<true>();
      if (p.up) ur = load_raw8<true, VEC>(p.x, row * p.pitch + p.up, s);
      if constexpr (kEarlyE) er = early[i];
      else if (e_row) er = load_raw8<true, VEC>(e_row, 0, s);
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = gated(gr.get(j), ur.get(j), er.get(j));
      return pack_raw8<true>(z);
    } else {
      return load_raw8<BF16, L>(p.x, base, s);
    }
  };
  Raw8<BF16> xr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Span s = span<L>(i, t, p.tpr, p.D);
    xr[i] = row_ok && s.n > 0 ? load_group(s, i) : zero_raw8<BF16>();
  }
  // the largest |x| as bits: a NaN is above the infinity, which is above
  // every finite number
  uint32_t m = 0;
  if constexpr (BF16) {
    // two bf16 magnitudes at a time as 16-bit integers
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __vmaxu2(m, xr[i].w[j] & 0x7fff7fffu);
    m = max(m << 16, m & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, xr[i].w[j] & 0x7fffffffu);
  }
  if (p.tpr >= 32) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (p.tpr > 32) {
      const int warp = threadIdx.x >> 5, wpr = p.tpr >> 5;
      if ((threadIdx.x & 31) == 0) red[warp] = m;
      __syncthreads();
      const int w0 = warp / wpr * wpr;
      for (int j = 0; j < wpr; ++j) m = max(m, red[w0 + j]);
    }
  } else {
    for (int k = p.tpr >> 1; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
  }
  if (!row_ok) return;
  const float amax = __uint_as_float(m);
  const float scale = amax / 127.0f;
  const bool finite = m < 0x7f800000u;
  if (t == 0) p.scale[row] = scale;
  // (an approximate reciprocal will do: the remainder decides)
  const float inv1 = __fdividef(1.0f, scale);
  const F2 inv = f2(inv1), nscale = f2(-scale);
  const F2 magic = f2(kRintMagic), nmagic = f2(-kRintMagic);
  const bool fast = finite && amax >= kTiny;
  const float half = fast ? 0.5f * scale : 0.0f;
  uint32_t redo = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Span s = span<L>(i, t, p.tpr, p.D);
    if (s.n <= 0) break;
    float worst = 0.0f;
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const F2 x = pair(xr[i], j);
      const F2 m = fma2(x, inv, magic);
      float r0, r1, s0, s1;
      f2_get(fma2(m + nmagic, nscale, x), r0, r1);
      f2_get(m, s0, s1);
      worst = fmaxf(worst, fmaxf(fabsf(r0), fabsf(r1)));
      b[2 * j] = __float_as_uint(s0);
      b[2 * j + 1] = __float_as_uint(s1);
    }
    // the low bytes of four words
    const uint32_t lo =
        __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    const uint32_t hi =
        __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    store8<L>(p.q + base, s, lo, hi);
    if (!(worst < half)) redo |= 1u << i;
  }
  // groups with an element at a tie (and all of a row that is tiny, zero or not
  // finite), behind the others so that no branch stands between their loads
  // and stores; one at a time
  while (redo) {
    const int i = __ffs(int(redo)) - 1;
    redo &= redo - 1;
    const Span s = span<L>(i, t, p.tpr, p.D);
    Raw8<BF16> x = xr[0];
    if constexpr (NV == 8) {     // (read again: fewer registers)
      x = load_group(s, 0);
    } else {
#pragma unroll
      for (int k = 1; k < NV; ++k)
        if (k == i) x = xr[k];
    }
    uint32_t lo = 0, hi = 0;
    if (fast) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo |= q_near(x.get(j), inv1, scale) << (8 * j);
        hi |= q_near(x.get(j + 4), inv1, scale) << (8 * j);
      }
      store8<L>(p.q + base, s, lo, hi);
      continue;
    }
#pragma unroll 1
    for (int j = 0; j < kGroup; ++j) {
      const uint32_t v = finite && scale > 0.0f ? q_exact(x.get(0), double(scale)) : 0u;
      // the bytes enter at the top, the elements leave at the bottom
      lo = __funnelshift_r(lo, hi, 8);
      hi = hi >> 8 | v << 24;
      if constexpr (BF16) {
#pragma unroll
        for (int k = 0; k < 3; ++k) x.w[k] = __funnelshift_r(x.w[k], x.w[k + 1], 16);
        x.w[3] >>= 16;
      } else {
#pragma unroll
        for (int k = 0; k < 7; ++k) x.w[k] = x.w[k + 1];
      }
    }
    store8<L>(p.q + base, s, lo, hi);
  }
}

template <bool BF16, RowLayout L, bool GATE>
cudaError_t go(const DeviceInfo& di, QuantParams p, cudaStream_t st) {
  // few rows: as many threads per row as there are groups; many: up to eight
  // groups per thread, whose loads are in flight together and whose maximum
  // is found with few instructions per element (16384 x 8192 bf16: 125 us with
  // two, 80 with four, 73 with eight)
  const int G = groups_of(p.D);
  // (GATE's three loads per group want more threads: 64 x 4096 x 11008 as a
  // layer takes 35.7 us with 704 per row, 37.0 with 352)
  const int per = G / (GATE ? 2 : 1);
  const int few = per > 2048 ? 8 : (per > 1024 ? 4 : (G > 512 ? 2 : 1));
  const int many = G > 128 ? 8 : (G > 64 ? 4 : (G > 32 ? 2 : 1));
  const int nv = p.T <= 2 * di.num_sms ? few : many;
  p.tpr = threads_per_row(G, nv);
  const int rpb = std::max(1, 128 / p.tpr);
  const dim3 grid(unsigned((int64_t(p.T) + rpb - 1) / rpb));
  const unsigned block = unsigned(rpb * p.tpr);
  switch (nv) {
    case 1: return launch_dependent(quant_rows_kernel<BF16, 1, L, GATE>, grid, block, 0, st, 1, p);
    case 2: return launch_dependent(quant_rows_kernel<BF16, 2, L, GATE>, grid, block, 0, st, 1, p);
    case 4: return launch_dependent(quant_rows_kernel<BF16, 4, L, GATE>, grid, block, 0, st, 1, p);
    default: return launch_dependent(quant_rows_kernel<BF16, 8, L, GATE>, grid, block, 0, st, 1, p);
  }
}

}  // namespace

staple_status launch_quant_rows(const DeviceInfo& di, bool bf16, int T, int D, const void* x,
                                int8_t* q, float* scale, cudaStream_t st, bool release) {
  if (T == 0) return STAPLE_OK;
  QuantParams p{};
  p.release = release;
  p.x = x;
  p.q = q;
  p.scale = scale;
  p.T = T;
  p.D = D;
  const bool vec = D % kGroup == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(q) & 7u) == 0;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("quant_rows", st,
             ce = bf16 ? (vec ? go<true, VEC, false>(di, p, st) : go<true, STRIDE, false>(di, p, st))
                       : (vec ? go<false, VEC, false>(di, p, st) : go<false, STRIDE, false>(di, p, st)));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

staple_status launch_gate_quant(const DeviceInfo& di, int T, int F, const void* gu, bool up,
                                const staple_embed* e, int8_t* q, float* scale, int32_t* err,
                                cudaStream_t st) {
  if (T == 0) return STAPLE_OK;
  QuantParams p{};
  p.release = true;
  p.x = gu;
  p.q = q;
  p.scale = scale;
  p.T = T;
  p.D = F;
  p.pitch = up ? 2 * int64_t(F) : F;
  p.up = up ? F : 0;
  if (e && e->mode != STAPLE_EMBED_NONE) {
    p.e_base = static_cast<const uint16_t*>(e->base);
    p.e_pitch = e->row_pitch;
    p.e_rows = e->n_rows;
    p.e_index = e->index;
  }
  p.err = err;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("gate_quant", st, ce = (go<true, VEC, true>(di, p, st)));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

}  // namespace stp
