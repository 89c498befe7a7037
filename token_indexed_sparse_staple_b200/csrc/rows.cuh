// Row helpers of the norm, dropout and quantisation kernels: groups of eight
// consecutive elements of a row, sums over the threads that share a row, and
// the dropout's counter-based random numbers.
#pragma once

#include "common.cuh"
#include "dependent.cuh"

namespace stp {

constexpr int kGroup = 8;   // elements a thread handles together

// Eight consecutive elements as they lie in memory: four 32-bit words of bf16
// pairs, or eight fp32 words.
template <bool BF16>
struct Raw8 {
  uint32_t w[BF16 ? 4 : 8];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return (i & 1) ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
    else return __uint_as_float(w[i]);
  }
};

// How a thread's eight elements lie in a row.  VEC: side by side, on a 16-byte
// boundary, all within the row.  STRIDE: one from each of eight runs of tpr
// elements, so that a warp's loads are side by side, for rows of an odd length.
enum RowLayout { VEC, STRIDE };

// The elements of thread t's i-th eight: off + j * step for j < n, where n may
// be zero or less.
struct Span {
  int off, step, n;
};
template <RowLayout L>
__device__ __forceinline__ Span span(int i, int t, int tpr, int D) {
  if constexpr (L == STRIDE) {
    const int off = i * kGroup * tpr + t;
    return Span{off, tpr, off < D ? min(kGroup, (D - off + tpr - 1) / tpr) : 0};
  } else {
    const int off = (t + i * tpr) * kGroup;
    return Span{off, 1, min(kGroup, D - off)};
  }
}

// Load the n <= 8 elements base[row + off + j * step]; the rest are zero.
// Plain (coherent) loads: the outputs of these kernels may share the inputs'
// memory.
template <bool BF16, RowLayout L>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void* base, int64_t row, const Span& s) {
  Raw8<BF16> r;
  const int64_t off = row + s.off;
  if constexpr (L == VEC) {
    if constexpr (BF16) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(base) + off);
      const uint4 a = p[0], b = p[1];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
  } else if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    const int step = s.step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < s.n ? p[2 * i * step] : 0u;
      const uint32_t hi = 2 * i + 1 < s.n ? p[(2 * i + 1) * step] : 0u;
      r.w[i] = lo | (hi << 16);
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(base) + off;
    const int step = s.step;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < s.n ? p[i * step] : 0u;
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> zero_raw8() {
  Raw8<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 4 : 8); ++i) r.w[i] = 0u;
  return r;
}

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> ones_raw8() {
  Raw8<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 4 : 8); ++i) r.w[i] = BF16 ? 0x3f803f80u : 0x3f800000u;
  return r;
}

// Eight floats rounded to the element type (bf16: to nearest even, the
// storage rounding of every bf16 tensor of the library).
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> pack_raw8(const float (&v)[8]) {
  Raw8<BF16> r;
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_bf2(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  }
  return r;
}

template <bool BF16, RowLayout L>
__device__ __forceinline__ void store_raw8(void* base, int64_t row, const Span& s,
                                           const Raw8<BF16>& r) {
  const int64_t off = row + s.off;
  if constexpr (L == VEC) {
    if constexpr (BF16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) =
          make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else {
      uint4* p = reinterpret_cast<uint4*>(static_cast<uint32_t*>(base) + off);
      p[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
      p[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    }
  } else if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + off;
    const int step = s.step;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < s.n) p[i * step] = uint16_t((i & 1) ? r.w[i >> 1] >> 16 : r.w[i >> 1] & 0xffffu);
  } else {
    uint32_t* p = static_cast<uint32_t*>(base) + off;
    const int step = s.step;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < s.n) p[i * step] = r.w[i];
  }
}

// Groups of a row of D elements.
inline int groups_of(int D) { return int((int64_t(D) + kGroup - 1) / kGroup); }

// Threads per row for nv groups per thread: a power of two up to 32, else
// whole warps.
inline int threads_per_row(int groups, int nv) {
  const int need = (groups + nv - 1) / nv;
  if (need > 32) return (need + 31) / 32 * 32;
  int t = 1;
  while (t < need) t <<= 1;
  return t;
}

// Threads that share a row: tpr of them, either a power of two up to 32
// (several rows per warp) or a multiple of 32 (whole warps).  Sums of N
// values over a row's threads, the same in each of them and in an order that
// depends on tpr alone.  red: N * 32 floats, free for the call (a caller that
// uses it again puts a block barrier, or another array, in between).  Every
// thread of the block calls it.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float* red) {
  const int width = tpr < 32 ? tpr : 32;
  for (int m = width >> 1; m > 0; m >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, wpr = tpr >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + warp] = v[k];
  __syncthreads();
  const int w0 = warp / wpr * wpr;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = red[k * 32 + w0];
    for (int j = 1; j < wpr; ++j) s += red[k * 32 + w0 + j];
    v[k] = s;
  }
}

// ---------------------------------------------------------------------------
// Dropout: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011).  One call gives 128 bits, a 16-bit
// draw for each element of a group of eight, so the generator costs ten rounds
// per eight elements.  Group g of row t has the counter (t * ceil(D / 8) + g)
// in its low 64 bits and offset + site in its high 64 bits; the key is the
// seed.  An element is kept when its draw is >= thr = round(p * 2^16).  The
// mask depends on nothing else: not on the kernel, its launch shape or the
// element type, so the backward pass and every fused form draw the same one.
// ---------------------------------------------------------------------------
struct DropParams {
  const uint64_t* rng;   // device {seed, offset}; NULL: no dropout
  uint64_t site;
  uint32_t below;        // thr * 2^16 - 1: a draw in a word's high half is kept if word > below
  float scale;           // 65536 / (65536 - thr)
};

struct DropKey {
  uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ DropKey drop_key(const DropParams& d) {
  // Ordinary loads, after the caller's wait: the kernel in front may have just moved
  // the offset on, and a read-only load (__ldg) need not stay behind the wait.  (It
  // gains nothing either: 16384 x 2048 bf16 with dropout 47.1 us forward and 77.3
  // backward, with read-only loads 47.6 and 77.8.)
  const unsigned long long* r = reinterpret_cast<const unsigned long long*>(d.rng);
  const uint64_t seed = r[0], hi = r[1] + d.site;
  return DropKey{uint32_t(seed), uint32_t(seed >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}

__device__ __forceinline__ uint4 philox(const DropKey& k, uint64_t n) {
  uint32_t c0 = uint32_t(n), c1 = uint32_t(n >> 32), c2 = k.c2, c3 = k.c3;
  uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
    c1 = uint32_t(p1);
    c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
    c3 = uint32_t(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The draws of N groups n0, n0 + step, ..., round by round: the key's schedule
// is then worked out once for all of them, and no chain of ten rounds leaves
// the warp waiting for its own results.
template <int N>
__device__ __forceinline__ void philox_n(const DropKey& k, uint64_t n0, uint32_t step,
                                         uint4 (&u)[N]) {
  uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t n = n0 + uint64_t(i) * step;
    u[i] = make_uint4(uint32_t(n), uint32_t(n >> 32), k.c2, k.c3);
  }
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t p0 = uint64_t(u[i].x) * 0xD2511F53u, p1 = uint64_t(u[i].z) * 0xCD9E8D57u;
      u[i] = make_uint4(uint32_t(p1 >> 32) ^ u[i].y ^ k0, uint32_t(p1),
                        uint32_t(p0 >> 32) ^ u[i].w ^ k1, uint32_t(p0));
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// v[i] = kept ? v[i] * scale : 0 for eight elements with the draws u.  A dropped
// element is zero whatever it held (an infinity or a NaN included).  A draw in
// the high half is compared without taking it out of its word; thr = 2^16
// makes `below` the largest word, which no word exceeds.
__device__ __forceinline__ void drop8(const uint4& u, uint32_t below, float scale, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t draw = (i & 1) ? w[i >> 1] : w[i >> 1] << 16;
    v[i] = draw > below ? v[i] * scale : 0.0f;
  }
}

// Strided eights: the 8 * 32 elements of a warp's lanes (of a row's threads where
// those are fewer) are as many whole groups, so each lane draws one group's eight,
// in any order, and passes on a byte of which are kept.  (Whole groups per thread,
// element by element, want no exchange but spread each of a warp's loads and
// stores over 32 sectors: with dropout the norm of 16384 x 1023 fp32 took 122 us
// forward and 133 backward, so 63 and 80; bf16 83 and 142, so 74 and 89.)  The
// group that thread t draws, counted from the first of its i-th eights:
__device__ __forceinline__ int stride_group(int t, int tpr) {
  return tpr < 32 ? t : ((t & 31) >> 2) * (tpr >> 3) + ((t & ~31) >> 3) + (t & 3);
}

// ... and what thread t keeps of its eight, given its own draws; every lane of the
// warp takes part.
__device__ __forceinline__ uint32_t stride_keep(const uint4& u, uint32_t below, int t, int tpr) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t draw = (i & 1) ? w[i >> 1] : w[i >> 1] << 16;
    mine |= draw > below ? 1u << i : 0u;
  }
  const int width = min(tpr, 32), at = t & (width - 1);
  uint32_t keep = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int k = j * width + at;      // of the lanes' elements in order
    keep |= (__shfl_sync(0xffffffffu, mine, k >> 3, width) >> (k & 7) & 1u) << j;
  }
  return keep;
}

__device__ __forceinline__ void drop8_kept(uint32_t keep, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = keep >> i & 1u ? v[i] * scale : 0.0f;
}

// ---------------------------------------------------------------------------
// Pairs of floats (fma.rn.f32x2 and friends): two IEEE operations in one
// instruction, which the row kernels need because they are close to bound by
// instruction issue.
// ---------------------------------------------------------------------------
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void f2_get(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Elements 2j and 2j + 1 of a group.
template <bool BF16>
__device__ __forceinline__ F2 pair(const Raw8<BF16>& r, int j) {
  return f2(r.get(2 * j), r.get(2 * j + 1));
}

}  // namespace stp
