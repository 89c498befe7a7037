// Product of 8-bit integer matrices with a scale per token and per output
// channel, on the tensor cores:
//
//   y[t][n] = float(sum_k a[t][k] b[n][k]) * a_scale[t] * b_scale[n]
//
// a [T][K] and b [N][K] are read in place by TMA (both K-major) into
// 128-byte-swizzled shared-memory stages; tcgen05.mma.kind::i8 adds the
// products up in int32, which is exact (K < 2^17, so a sum stays inside 32
// bits), in tensor memory.  The epilogue rounds the sum to fp32, multiplies by
// the two scales and rounds to the output type: three roundings of fp32 and
// one of storage.
//
// Three kernels:
//  * tiles: many tokens.  Tokens take the MMA's M side; a pair of SMs shares a
//    256 x 256 tile (cta_group::2), each holding half of either operand, so
//    that an operand byte is fetched from L2 and read from shared memory once
//    for twice the products of a 128 x 256 tile.  Persistent pairs, two
//    accumulators in tensor memory so that a tile's epilogue runs beside the
//    next tile's products.  Bound by the tensor cores.
//  * split: few tiles (decode, or narrow outputs).  The weights take the M
//    side and up to 256 tokens the N side, so a block is a stream of weights;
//    bound by HBM.  Where k is split too, the blocks of a cluster add their
//    integer sums through distributed shared memory: no partial sums in
//    memory, no counters, and integer adds give the same result in any order.
//  * dots: a single token, on the CUDA cores; bound by HBM and by launching.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dependent.cuh"
#include "internal.h"
#include "tmap.h"

namespace stp {

namespace {

namespace i8 {

constexpr int BK = 128;   // bytes (= k values) per 128-byte-swizzled row

// One lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n"
               : "=r"(p));
  return p;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, signed 8-bit inputs, int32
// accumulator; K = 32 per instruction.  PAIR: one instruction over the shared
// and tensor memories of two SMs, M = 256.  The whole warp calls it with the
// same operands and the elected lane issues it: a loop that only one lane runs
// moves every operand into the uniform registers anew, which took 100 cycles
// per instruction here, more than a 128 x 64 x 32 product takes (49).
template <bool PAIR>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                     uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// Every thread of every block of the cluster; shared-memory writes before it
// are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" :::
                   "memory");
}
// The cluster address of this block's shared-memory word in block `rank`.
__device__ __forceinline__ uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

// The pair's forms of the wrappers in common.cuh.  A load lands in the shared
// memory of the block that issues it and counts on a barrier that may be the
// other block's; a commit arrives on the same barrier of both blocks.
__device__ __forceinline__ void pair_load_2d(const CUtensorMap* map, uint32_t bar, void* dst,
                                             int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Instruction descriptor for kind::i8: int32 accumulator, signed A and B, both
// K-major.
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (2u << 4)                      // D format: s32
         | (1u << 7)                    // A format: s8
         | (1u << 10)                   // B format: s8
         | (uint32_t(N >> 3) << 17)     // N / 8
         | (uint32_t(M >> 4) << 24);    // M / 16
}

// bulk_wait_read0() for all but the last committed group.
__device__ __forceinline__ void bulk_wait_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

struct Params {
  int32_t T, N, K;
  // The kernel in front may still be writing the scales when this one starts, so they
  // are loaded after the wait and by ordinary loads: a read-only load (__ldg) is for
  // what nothing writes while the kernel runs, and need not stay behind the wait.
  const float* a_scale;
  const float* b_scale;
  void* y;
  int32_t* err;
  uint64_t wait_ns;
  bool release;          // the next kernel is part of the same call
  bool weights_ready;    // b may be read before wait_prior_kernels() (split and dot)
  // tiles
  int32_t tiles_t, tiles_n, group_t;
  bool tma_out;
  // split
  int32_t tokens;        // tokens per tile, rounded up to 16 (the MMA's N)
  int32_t cols;          // tensor-memory columns (a power of two >= 32)
  int32_t rows;          // channels per tile, a multiple of 8 up to 128
  int32_t stages, units; // 256-byte k units in all
  bool vec_out;
};

// ---------------------------------------------------------------- tiles

constexpr int BM = 128, BN = 256, STAGES = 6, kThreads = 192;
// per block and stage: 128 of the pair's 256 tokens and 128 of its 256 channels
constexpr int HALF_STAGE = 128 * BK, STAGE_BYTES = 2 * HALF_STAGE;
// One warp's staged 32 x 32 outputs: two blocks of bf16, or one of fp32.
constexpr int kOutBox = 32 * 32 * 4;
// One block per SM, whatever the output type: two would not share the 512
// columns of tensor memory, and the one that waits for them must not hold
// shared memory that another kernel could use.
constexpr int kTilesSmem = 226 * 1024;
static_assert(1024 + STAGES * STAGE_BYTES + 4 * kOutBox + 4 * BN * 4 + 256 <= kTilesSmem, "shared memory");

__device__ __forceinline__ void tile_coords(int t, const Params& p, int& mb, int& nb) {
  const int per_group = p.group_t * p.tiles_n;
  const int g = t / per_group, first = g * p.group_t;
  const int rows = min(p.group_t, p.tiles_t - first);
  const int r = t - g * per_group;
  mb = first + r % rows;
  nb = r / rows;
}

// 16384 x 8192 x 2048 takes 165 us in captured runs with pauses between them (3.33 P
// op/s, 0.97 of twice the measured bf16 rate) and 205 to 211 back to back, where the 1
// kW cap holds the clock near 1.6 GHz; 128 x 256 tiles on single SMs took 189 and 229
// when these took 170 and 209.  With fp32 outputs a captured run takes 210 us.
//
// Blocks 2i and 2i + 1 are a pair; the even one leads: it waits for both
// blocks' loads and issues the products.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmO, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * HALF_STAGE;
  uint8_t* s_out = sB + STAGES * HALF_STAGE;
  float* s_scale = reinterpret_cast<float*>(s_out + 4 * kOutBox);   // [4 warps][256]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + 4 * BN);   // the leader's are used
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;                                     // the leader's are used
  uint64_t* dbar = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dbar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(blockIdx.x & 1u);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);      // four epilogue warps in either block
    }
    mbar_init(dbar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) pair_tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // the other block's barriers are set up too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int ntiles = p.tiles_t * p.tiles_n, kblocks = (p.K + BK - 1) / BK;
  const int first = int(blockIdx.x >> 1), step = int(gridDim.x >> 1);
  wait_prior_kernels();
  if (p.release) release_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step) {
        int mb, nb;
        tile_coords(t, p, mb, nb);
        const int m0 = mb * 2 * BM + rank * BM, n0 = nb * BN + rank * 128;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.err, p.wait_ns)) {
            ok = false;
            break;
          }
          // (the other block's bytes may be counted before this: the phase
          // cannot end without the arrival)
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * STAGE_BYTES);
          const uint32_t bar = map_peer(smem_u32(&full[stage]), 0);
          pair_load_2d(&tmA, bar, sA + stage * HALF_STAGE, kb * BK, m0);
          pair_load_2d(&tmB, bar, sB + stage * HALF_STAGE, kb * BK, n0);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (rank == 0) {
        drain_ring(full, STAGES, stage, phase, issued);
      } else if (!ok) {
        // the leader counts this block's loads; after a wait that ran out,
        // give those in flight the time to land
        for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < kDrainNs;) {
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t elected = elect_one();
      const uint64_t a0 = sw128_desc(smem_u32(sA), 16, 1024);
      const uint64_t b0 = sw128_desc(smem_u32(sB), 16, 1024);
      int stage = 0, iter = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step, ++iter) {
        const int buf = iter & 1;
        ok = mbar_wait(&tempty[buf], (uint32_t(iter >> 1) & 1) ^ 1, abort_flag, p.err, p.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t dacc = tmem_base + uint32_t(buf * BN);
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait(&full[stage], phase, abort_flag, p.err, p.wait_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = a0 + uint64_t(stage * (HALF_STAGE >> 4));
          const uint64_t b = b0 + uint64_t(stage * (HALF_STAGE >> 4));
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)   // 32 bytes further on: 2 in the address field
            umma<true>(dacc, a + 2 * k, b + 2 * k, idesc(2 * BM, BN), (kb | k) ? 1u : 0u, elected);
          if (elected) pair_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok && elected) pair_commit(&tfull[buf]);
      }
      if (elected) pair_commit(dbar);
      __syncwarp();
      mbar_drain(dbar, 0);
    }
  } else {
    const int q = warp & 3;
    uint8_t* box = s_out + q * kOutBox;
    float* scales = s_scale + q * BN;      // the tile's channel scales, a copy per warp
    int iter = 0;
    // bf16 has two boxes, taken in turn from the first tile to the last: a tile at the
    // right edge may end on either, and the wait below leaves the newest store in flight
    int turn = 0;
    const uint32_t free_bar[2] = {map_peer(smem_u32(&tempty[0]), 0), map_peer(smem_u32(&tempty[1]), 0)};
    for (int t = first; t < ntiles; t += step, ++iter) {
      const int buf = iter & 1;
      int mb, nb;
      tile_coords(t, p, mb, nb);
      const int m0 = mb * 2 * BM + rank * BM + q * 32, m = m0 + lane;
      const float sa = m < p.T ? p.a_scale[m] : 0.0f;
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) {
        const int n = nb * BN + i * 32 + lane;
        scales[i * 32 + lane] = n < p.N ? p.b_scale[n] : 0.0f;
      }
      __syncwarp();
      const bool ok = mbar_wait(&tfull[buf], uint32_t(iter >> 1) & 1, abort_flag, p.err, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(buf * BN);
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int n = nb * BN + c * 32;
        if (n >= p.N) break;          // the same for the whole warp
        uint8_t* stg = box + (BF16 ? turn * (kOutBox / 2) : 0);
        turn ^= 1;
        uint32_t r[32];
        tmem_ld32(tacc + c * 32, r);
        tmem_ld_wait(r);
        float v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 sb = *reinterpret_cast<const float4*>(scales + c * 32 + 4 * i);
          v[4 * i] = float(int(r[4 * i])) * sa * sb.x;
          v[4 * i + 1] = float(int(r[4 * i + 1])) * sa * sb.y;
          v[4 * i + 2] = float(int(r[4 * i + 2])) * sa * sb.z;
          v[4 * i + 3] = float(int(r[4 * i + 3])) * sa * sb.w;
        }
        // stage the 32 x 32 block, swizzled as the TMA store expects it (and
        // free of bank conflicts either way)
        if (p.tma_out && lane == 0) {
          // (bf16: the store from the other box may still be on its way out)
          if constexpr (BF16) bulk_wait_read1();
          else bulk_wait_read0();
        }
        __syncwarp();
        if constexpr (BF16) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pack_bf2(v[8 * k], v[8 * k + 1]), pack_bf2(v[8 * k + 2], v[8 * k + 3]),
                           pack_bf2(v[8 * k + 4], v[8 * k + 5]),
                           pack_bf2(v[8 * k + 6], v[8 * k + 7]));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
        if (p.tma_out) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmO, stg, n, m0);
            bulk_commit();
          }
        } else {
          // rows that TMA cannot address (pitch not a multiple of 16 bytes):
          // one row at a time, a warp's 32 columns side by side
          __syncwarp();
          const int rows = min(32, p.T - m0);
          if (n + lane < p.N)
            for (int i = 0; i < rows; ++i) {
              const int64_t o = int64_t(m0 + i) * p.N + n + lane;
              if constexpr (BF16)
                static_cast<uint16_t*>(p.y)[o] = *reinterpret_cast<const uint16_t*>(
                    stg + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
              else
                static_cast<float*>(p.y)[o] = *reinterpret_cast<const float*>(
                    stg + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
            }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(free_bar[buf]);
    }
    if (p.tma_out && lane == 0) bulk_wait0();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // the products, which read both blocks' memory, are over
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tmem_base, 512);
  cluster_sync();
}

// ---------------------------------------------------------------- split

// The bound is HBM, so the tiles are cut to keep every SM streaming: a tile is
// `rows` channels high, not 128 (the MMA's M stays 128; what it computes of
// the rows that no copy wrote is not read), and the height is chosen so that
// the tiles are as many as the SMs.  Only outputs too narrow for that, or with
// so many tokens that their re-reading from L2 would cost more, split k too.
// 64 x 11008 x 4096 takes 12.0 us in a captured run over weights enough that they come
// from memory (45.1 MB, 7.0 us at a copy's rate), 9.6 where one or two sets of them
// stay in L2; 64 x 8192 x 2048 takes 7.8 from memory.
constexpr int kUnit = 2 * BK;               // 256 bytes of each row per stage
constexpr int kMaxTokens = 256, kMaxStages = 24;

__device__ __forceinline__ void st_cluster(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// Channels n .. n + 3 of one token, of which `left` are this tile's.
template <bool BF16>
__device__ __forceinline__ void store4(const Params& p, int t, int n, int left,
                                       const float (&v)[4]) {
  const int64_t o = int64_t(t) * p.N + n;
  if (p.vec_out && left >= 4) {
    if constexpr (BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + o) =
          make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + o) =
          make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) {
      if constexpr (BF16)
        static_cast<uint16_t*>(p.y)[o + i] = uint16_t(pack_bf2(v[i], 0.0f) & 0xffffu);
      else
        static_cast<float*>(p.y)[o + i] = v[i];
    }
}

// Block = 6 warps: 0 loads, 1 MMAs, 2..5 drain the accumulator.  blockIdx.x =
// tile * C + rank in the cluster; blockIdx.y = token tile.
template <bool BF16, int C>
__global__ void __launch_bounds__(kThreads)
    split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_i;
  __shared__ float s_scale[kMaxTokens];
  volatile int* abort_flag = &abort_i;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {          // the maps' way into the cache is the longest: first
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  const uint32_t rank = blockIdx.x % C;
  const int n0 = int(blockIdx.x / C) * p.rows, t0 = int(blockIdx.y) * kMaxTokens;
  const int S = p.stages;
  // a k block of 128 bytes: weights, tokens (the tokens' tiles start on 1 KB
  // boundaries as both are multiples of eight rows)
  const int w_bytes = p.rows * BK, x_bytes = p.tokens * BK;
  const int stage_bytes = 2 * (w_bytes + x_bytes);
  // this block's k units
  const int u0 = p.units * int(rank) / C, u1 = p.units * (int(rank) + 1) / C;
  const int len = u1 - u0, first = min(S, len);   // units, fills of the first lap
  // Tiles start at different units of k (the sum does not mind): in step, all
  // blocks would read the same tokens' lines from L2 at the same time.
  const int shift = int(blockIdx.x / C) % len;
  auto unit = [&](int i) { return u0 + (i + shift < len ? i + shift : i + shift - len); };
  const uint64_t policy = l2_policy_evict_first();
  auto load_w = [&](int i, int stage) {
    uint8_t* w = smem + stage * stage_bytes;
    for (int h = 0; h < 2; ++h) {
      const int k = unit(i) * kUnit + h * BK;     // past K: zeros
      // weights that no other token tile reads need not stay in L2
      if (gridDim.y == 1)
        tma_load_2d_hint(&tmW, &full[stage], w + h * w_bytes, k, n0, policy);
      else
        tma_load_2d(&tmW, &full[stage], w + h * w_bytes, k, n0);
    }
  };
  auto load_x = [&](int i, int stage) {
    uint8_t* x = smem + stage * stage_bytes + 2 * w_bytes;
    for (int h = 0; h < 2; ++h)
      tma_load_2d(&tmX, &full[stage], x + h * x_bytes, unit(i) * kUnit + h * BK, t0);
  };
  // Warp 0 sets the barriers up and sends the first ring of loads out before
  // the block's set-up barrier.
  if (warp == 0) {
    if (lane < S) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], 1);
    }
    if (lane == 0) {
      mbar_init(&tfull, 1);
      abort_i = 0;
    }
    fence_barrier_init();
    if (lane < first) mbar_arrive_expect_tx(&full[lane], stage_bytes);
    __syncwarp();
    // In the 8-bit layer the first ring of weights is on its way while the kernel in
    // front finishes: 64 x 4096 x 11008 37 us with it and the gate's early E, 40
    // without; prefetching the weights behind the ring into L2 too gained nothing.
    if (p.weights_ready && lane == 0)
      for (int s = 0; s < first; ++s) load_w(s, s);
    __syncwarp();
    wait_prior_kernels();
    if (lane == 0)
      for (int s = 0; s < first; ++s) {
        if (!p.weights_ready) load_w(s, s);
        load_x(s, s);
      }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, p.cols);
    tmem_relinquish();
  }
  if (warp != 0) wait_prior_kernels();
  if (p.release) release_dependents();
  const int tokens = min(p.tokens, p.T - t0);
  const int channels = min(p.rows, p.N - n0);
  // The scales are fetched now: at the end their latency would count.  One
  // block: a thread has one channel; a cluster: four (see the sums below).
  const int row = (warp & 3) * 32 + lane;   // this thread's accumulator row (warps 2..5)
  float sb[C == 1 ? 1 : 4];
  if constexpr (C == 1) {
    sb[0] = row < channels ? p.b_scale[n0 + row] : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sb[i] = lane * 4 + i < channels ? p.b_scale[n0 + lane * 4 + i] : 0.0f;
  }
  if (warp >= 2)
    for (int t = threadIdx.x - 64; t < tokens; t += kThreads - 64)
      s_scale[t] = p.a_scale[t0 + t];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = first;
      uint32_t phase = 0;
      for (; issued < len; ++issued) {
        if (!mbar_wait(&empty[stage], phase, abort_flag, p.err, p.wait_ns)) break;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        load_w(issued, stage);
        load_x(issued, stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      drain_ring(full, S, issued % S, uint32_t(issued / S) & 1, issued);
    }
  } else if (warp == 1) {
    const uint32_t id = idesc(BM, p.tokens), elected = elect_one();
    const uint64_t d0 = sw128_desc(smem_u32(smem), 16, 1024);
    const uint32_t dw = uint32_t(w_bytes) >> 4, dx = uint32_t(x_bytes) >> 4;
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < len; ++i) {
      const bool ok = mbar_wait(&full[stage], phase, abort_flag, p.err, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t w = d0 + uint64_t(uint32_t(stage * stage_bytes) >> 4), x = w + 2 * dw;
#pragma unroll
      for (int k = 0; k < 8; ++k)   // 32 bytes further on: 2 in the address field
        umma<false>(tmem_base, w + (k >> 2) * dw + (k & 3) * 2, x + (k >> 2) * dx + (k & 3) * 2, id,
             (i | k) ? 1u : 0u, elected);
      if (elected) umma_commit(&empty[stage]);
      if (++stage == S) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (elected) umma_commit(&tfull);
  }
  __syncwarp();
  // every product of this block is in tensor memory, and its stages are free
  mbar_wait(&tfull, 0, abort_flag, p.err, p.wait_ns);
  if (*abort_flag && warp == 1) mbar_drain(&tfull, 0);
  __syncwarp();
  tc_fence_after();
  const uint32_t tacc = tmem_base + (uint32_t((warp & 3) * 32) << 16);
  if constexpr (C == 1) {
    // thread = channel: a warp writes 32 neighbouring channels of one token
    if (warp >= 2 && (warp & 3) * 32 < channels) {
      const size_t es = BF16 ? 2 : 4, pitch = size_t(p.N) * es;
      uint8_t* y = static_cast<uint8_t*>(p.y) + size_t(t0) * pitch + size_t(n0 + row) * es;
      const bool row_ok = row < channels;
      for (int c = 0; c < tokens; c += 16, y += 16 * pitch) {
        uint32_t r[16];
        tmem_ld16(tacc + c, r);
        tmem_ld_wait16(r);
        const int n = row_ok ? tokens - c : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = float(int(r[i])) * s_scale[c + i] * sb[0];
          if (i < n) {
            if constexpr (BF16)
              *reinterpret_cast<uint16_t*>(y + i * pitch) = uint16_t(pack_bf2(v, 0.0f) & 0xffffu);
            else
              *reinterpret_cast<float*>(y + i * pitch) = v;
          }
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, p.cols);
  } else {
    // Rank r adds the sums of tokens r, r + C, ... of the tile: every block sends
    // them there from its tensor memory, [rank][token / C][128], over the stages,
    // which are free once the block's products are done.  (Fetched by rank r from
    // every block's own memory instead: 64 x 2048 x 8192 8.9 us, so 8.2.)
    cluster_sync();
    int32_t* sums = reinterpret_cast<int32_t*>(smem);
    const int per = p.tokens / C;
    if (warp >= 2 && (warp & 3) * 32 < channels) {
      uint32_t to[C];
#pragma unroll
      for (int r = 0; r < C; ++r) to[r] = map_peer(smem_u32(sums + int(rank) * per * BM + row), r);
      for (int c = 0; c < p.tokens; c += 16) {
        uint32_t r[16];
        tmem_ld16(tacc + c, r);
        tmem_ld_wait16(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) st_cluster(to[i % C] + (c + i) / C * (BM * 4), r[i]);
      }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, p.cols);
    // one warp per token, four channels per lane
    const int n = n0 + lane * 4;
    for (int j = warp; j < per; j += kThreads / 32) {
      const int t = int(rank) + C * j;
      if (t >= tokens) break;
      int4 v = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const int4 u = *reinterpret_cast<const int4*>(sums + (r * per + j) * BM + lane * 4);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const float sa = s_scale[t];
      const float f[4] = {float(v.x) * sa * sb[0], float(v.y) * sa * sb[1],
                          float(v.z) * sa * sb[2], float(v.w) * sa * sb[3]};
      store4<BF16>(p, t0 + t, n, channels - lane * 4, f);
    }
  }
}

// ---------------------------------------------------------------- dots

// One token: each warp streams two channels' weights straight into registers,
// 16 bytes per lane, against the token's bytes (which the L1 keeps), with the
// four-way integer dot product of the CUDA cores.  Nothing is set up: no tensor
// maps, barriers or tensor memory, whose 1.5 us before the first load the split
// kernel has no work to hide behind here.  ksplit warps of a block share a pair
// of channels where there are too few channels to keep HBM busy.  In a captured
// run, beside two tokens in the split kernel: 8192 x 2048 4.4 us (6.4), 2048 x
// 8192 4.4 (7.1), 11008 x 4096 9.7 (10.8).  Given two tokens the two kernels were
// even, given four the split kernel won.
constexpr int kDotThreads = 256, kDotWarps = kDotThreads / 32, kDotRows = 2;
constexpr int kDotChunks = 4;              // chunks of 512 bytes in flight per row

// 16 bytes of weights, read once; the loads stay in this order, ahead of what
// uses them.
__device__ __forceinline__ int4 load_weights(const int8_t* p, bool ok) {
  int4 v = make_int4(0, 0, 0, 0);
  if (ok)
    asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kDotThreads)
    dot_kernel(const int8_t* a, const int8_t* b, const Params p, int ksplit) {
  __shared__ int part[kDotWarps][kDotRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kw = warp % ksplit;
  const int n0 = (int(blockIdx.x) * (kDotWarps / ksplit) + warp / ksplit) * kDotRows;
  if (!p.weights_ready) wait_prior_kernels();
  int acc[kDotRows] = {};
  const int8_t* row[kDotRows];
#pragma unroll
  for (int r = 0; r < kDotRows; ++r) row[r] = b + int64_t(min(n0 + r, p.N - 1)) * p.K;
  // warp kw of a pair of channels takes every ksplit-th run of chunks
  constexpr int kRun = kDotChunks * 512;
  for (int kr = kw * kRun; kr < p.K; kr += ksplit * kRun) {
    const int k0 = kr + lane * 16;
    int4 w[kDotChunks][kDotRows];
#pragma unroll
    for (int u = 0; u < kDotChunks; ++u)
#pragma unroll
      for (int r = 0; r < kDotRows; ++r)
        w[u][r] = load_weights(row[r] + k0 + u * 512, k0 + u * 512 < p.K);
    // the first weights are on their way while the kernel in front finishes: in the
    // 8-bit layer of one token (2048 -> 8192 -> 2048) 19 -> 15 us
    if (p.weights_ready && kr == kw * kRun) wait_prior_kernels();
#pragma unroll
    for (int u = 0; u < kDotChunks; ++u) {
      const int k = k0 + u * 512;
      const int4 x = k < p.K ? *reinterpret_cast<const int4*>(a + k) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kDotRows; ++r) {
        acc[r] = __dp4a(w[u][r].x, x.x, acc[r]);
        acc[r] = __dp4a(w[u][r].y, x.y, acc[r]);
        acc[r] = __dp4a(w[u][r].z, x.z, acc[r]);
        acc[r] = __dp4a(w[u][r].w, x.w, acc[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kDotRows; ++r) {
    const int s = __reduce_add_sync(0xffffffffu, acc[r]);
    if (lane == 0) part[warp][r] = s;
  }
  if (ksplit > 1) __syncthreads();
  else __syncwarp();
  if (p.weights_ready) wait_prior_kernels();    // (a warp without a run has not waited yet)
  if (p.release) release_dependents();
  const int n = n0 + lane;
  if (kw == 0 && lane < kDotRows && n < p.N) {
    int s = 0;
    for (int k = 0; k < ksplit; ++k) s += part[warp + k][lane];
    const float v = float(s) * p.a_scale[0] * p.b_scale[n];
    if constexpr (BF16)
      static_cast<uint16_t*>(p.y)[n] = uint16_t(pack_bf2(v, 0.0f) & 0xffffu);
    else
      static_cast<float*>(p.y)[n] = v;
  }
}

inline int cdiv(int64_t a, int64_t b) { return int((a + b - 1) / b); }

}  // namespace i8

// How a few-tiles product is cut.
struct SplitPlan {
  int cluster, rows, stages, smem;
  double us;           // of the whole launch, estimated; see tiles_us
};

// Beside 1.5 KB of static arrays and the 1 KB that each block takes; a quantiser's
// block (the kernel in front in the 8-bit layer) still fits in what is left of 228.
constexpr int kSplitSmemMax = 223 * 1024;

// Every candidate cluster size with the tile height that fills the SMs (w
// blocks each), and the estimated time on one SM in us: its share of the
// weights at its share of HBM (43.6 KB per us) with the tokens' rows once more
// per tile at about 2.5 times that from L2, at least 0.3 per unit to issue its
// products, 1 for each further block per SM, and the sum over a cluster.
// Measured in a captured run: 64 x 4096 x 11008 takes 12.3 us in clusters of
// 4 (128 rows) against 17.7 without (32 rows); 64 x 11008 x 4096 takes 12.0
// without (80 rows) against 13.2 in pairs; 128 x 8192 x 8192 takes 17.7 in
// pairs against 20.1 without.  Over 65 shapes of 2 to 256 tokens the choice was
// the best or 1 % behind it on average, 13 % at most.  Clusters do not pack all
// SMs (33 of 4 and 15 of 8 fit at one block per SM).
SplitPlan plan_split(int num_sms, int N, int units, int tokens, int tiles_t, int cols) {
  SplitPlan best{};
  double best_us = 1e30;
  for (int c = 1; c <= 8 && c <= units; c *= 2) {
    const int sms = std::max(1, num_sms * (c == 1 ? 16 : (c == 2 ? 15 : (c == 4 ? 14 : 13))) / 16);
    const int64_t cells = int64_t(tiles_t) * c;
    const int w = i8::cdiv(i8::cdiv(N, i8::BM) * cells, sms);
    const int64_t tiles = std::max<int64_t>(1, int64_t(w) * sms / cells);
    const int rows = std::min<int>(i8::BM, std::max<int>(16, i8::cdiv(i8::cdiv(N, tiles), 8) * 8));
    const int per_block = i8::cdiv(units, c);
    const double unit_us = std::max(0.3, (rows + 0.4 * tokens) * i8::kUnit / 43600.0);
    const double us = w * per_block * unit_us + (w - 1) + (c > 1 ? 0.6 + 0.2 * c : 0.0);
    if (us >= best_us) continue;
    // two blocks per SM at most: more would have too few stages each
    const int stage = 2 * (rows + tokens) * i8::BK;
    // an MMA reads 128 rows from where a tile starts, in the last stage past
    // its end too
    const int sums = c > 1 ? tokens * i8::BM * 4 : 0;
    const int over = std::max(0, i8::BM * i8::BK + rows * i8::BK - stage);
    int stages = 0;
    for (int fit = std::min(w, 512 / cols > 1 ? 2 : 1); fit >= 1 && stages < std::min(3, per_block); --fit)
      stages = std::min(std::min(per_block, i8::kMaxStages),
                        (std::min(228 * 1024 / fit - 4096, kSplitSmemMax) - 1024 - over) / stage);
    const int want = std::max(stages * stage + over, sums) + 1024;
    // Blocks that share an SM share its 512 columns of tensor memory, and a
    // block that waits for columns could wait for a cluster whose other blocks
    // wait for it: so no block takes a smaller part of the SM's 228 KB than of
    // its columns, and none fits beside a tiled GEMM block (at least 193.25 KB
    // and all columns).  A cluster's blocks do not fit beside a block of the
    // decode kernel either (147 KB or more, all columns): its blocks wait for
    // one another as a cluster's do, and the two could wait in a circle.
    const int share = std::max(int(int64_t(cols) * 228 * 1024 / 512) - 1024,
                               (c > 1 ? 84 : 36) * 1024);
    best_us = us;
    const double total = 4.0 +
                         w * per_block * std::max(0.3, (rows + 0.15 * tokens) * i8::kUnit / 43600.0) +
                         (c == 1 ? 0.025 : 0.02) * tokens * w;
    best = SplitPlan{c, rows, stages, std::max(want, share), total};
  }
  return best;
}

// The time of the pair's tiles, to choose between the two kernels above half a
// tile's 256 tokens (below, the split kernel wins): a start and an end, and per
// round of tiles its k and its epilogue.  This and the split estimate (a start and
// an end, the units, the tokens' epilogue) were fitted to captured runs of 110
// shapes (160 to 4096 tokens, N 512 to 28672, K 64 to 28672) and pick the faster
// or one within 5 % each time.  Split against tiles: 192 x 8192 x 2048 11.7 / 12.4
// us, 192 x 16384 x 2048 15.2 / 13.6, 256 x 22016 x 4096 48.4 / 28.2, 256 x 4096 x
// 11008 19.8 / 31.3, 512 x 8192 x 2048 17.6 / 13.0, 1024 x 2048 x 8192 22.7 / 25.4.
double tiles_us(int pairs, int64_t tiles, int K) {
  return 7.0 + (0.3 * i8::cdiv(K, i8::BK) + 0.5) * i8::cdiv(tiles, pairs);
}

template <typename K>
bool opt_in(K kern, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (done.load() & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  done.fetch_or(bit);
  return true;
}

int tile_pairs(const DeviceInfo& di) { return std::max(1, (di.num_sms - di.sm_reserve) / 2); }

template <bool BF16>
staple_status go_tiles(const DeviceInfo& di, const CUtensorMap& a, const CUtensorMap& b,
                       const CUtensorMap& o, const i8::Params& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = i8::tiles_kernel<BF16>;
  if (!opt_in(kern, i8::kTilesSmem, di.device, done)) return STAPLE_ECUDA;
  const int ntiles = p.tiles_t * p.tiles_n;
  const int per = i8::cdiv(ntiles, tile_pairs(di));
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("matmul_i8", st,
             ce = launch_dependent(kern, dim3(2 * unsigned(i8::cdiv(ntiles, per))), i8::kThreads,
                                   i8::kTilesSmem, st, 2, a, b, o, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16, int C>
staple_status go_split(const DeviceInfo& di, const CUtensorMap& w, const CUtensorMap& x,
                       const i8::Params& p, int tiles_t, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = i8::split_kernel<BF16, C>;
  if (!opt_in(kern, kSplitSmemMax, di.device, done)) return STAPLE_ECUDA;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("matmul_i8_split", st,
             ce = launch_dependent(kern, dim3(unsigned(i8::cdiv(p.N, p.rows)) * C, unsigned(tiles_t)),
                                   i8::kThreads, size_t(smem), st, C, w, x, p));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

template <bool BF16>
staple_status go_split_c(const DeviceInfo& di, const CUtensorMap& w, const CUtensorMap& x,
                         const i8::Params& p, const SplitPlan& pl, int tiles_t, cudaStream_t st) {
  switch (pl.cluster) {
    case 1: return go_split<BF16, 1>(di, w, x, p, tiles_t, pl.smem, st);
    case 2: return go_split<BF16, 2>(di, w, x, p, tiles_t, pl.smem, st);
    case 4: return go_split<BF16, 4>(di, w, x, p, tiles_t, pl.smem, st);
    default: return go_split<BF16, 8>(di, w, x, p, tiles_t, pl.smem, st);
  }
}

template <bool BF16>
staple_status go_dot(const DeviceInfo& di, const int8_t* a, const int8_t* b, const i8::Params& p,
                     cudaStream_t st) {
  // warps enough that their loads (128 bytes per lane) cover HBM's latency
  const int pairs = i8::cdiv(p.N, i8::kDotRows);
  int ksplit = 1;
  while (ksplit < i8::kDotWarps && int64_t(pairs) * ksplit < int64_t(di.num_sms) * 16 &&
         ksplit * i8::kDotChunks * 512 < p.K)
    ksplit *= 2;
  cudaError_t ce = cudaSuccess;
  STP_LAUNCH("matmul_i8_dot", st,
             ce = launch_dependent(i8::dot_kernel<BF16>,
                                   dim3(unsigned(i8::cdiv(pairs, i8::kDotWarps / ksplit))),
                                   i8::kDotThreads, 0, st, 1, a, b, p, ksplit));
  return ce == cudaSuccess ? STAPLE_OK : STAPLE_ECUDA;
}

}  // namespace

staple_status launch_matmul_i8(const DeviceInfo& di, bool bf16, int T, int N, int K,
                               const int8_t* a, const float* a_scale, const int8_t* b,
                               const float* b_scale, void* y, int32_t* err, cudaStream_t st,
                               bool release, bool weights_ready) {
  if (T == 0) return STAPLE_OK;
  // tiles are counted in 32 bits
  if (int64_t(i8::cdiv(T, 2 * i8::BM)) * i8::cdiv(N, i8::BN) > INT32_MAX / 2)
    return STAPLE_EUNSUPPORTED;
  const int es = bf16 ? 2 : 4;
  i8::Params p{};
  p.T = T;
  p.N = N;
  p.K = K;
  p.a_scale = a_scale;
  p.b_scale = b_scale;
  p.y = y;
  p.err = err;
  p.wait_ns = di.wait_ns;
  p.release = release;
  p.weights_ready = weights_ready;
  if (T == 1)
    return bf16 ? go_dot<true>(di, a, b, p, st) : go_dot<false>(di, a, b, p, st);
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap ma, mb, mo;
  p.tiles_t = i8::cdiv(T, 2 * i8::BM);
  p.tiles_n = i8::cdiv(N, i8::BN);
  const int tiles_t = i8::cdiv(T, i8::kMaxTokens);
  p.tokens = std::min(i8::kMaxTokens, i8::cdiv(T, 16) * 16);
  p.cols = 32;
  while (p.cols < p.tokens) p.cols <<= 1;
  p.units = i8::cdiv(K, i8::kUnit);
  const int64_t tiles = int64_t(p.tiles_t) * p.tiles_n;
  const int pairs = tile_pairs(di);
  // (with many tiles there is nothing to weigh)
  SplitPlan pl{};
  bool by_tiles = T > i8::BM && tiles > 4 * int64_t(pairs);
  if (!by_tiles) {
    pl = plan_split(di.num_sms, N, p.units, p.tokens, tiles_t, p.cols);
    by_tiles = T > i8::BM && tiles_us(pairs, tiles, K) < pl.us;
  }
  if (by_tiles) {
    p.group_t = 8;
    p.tma_out = (int64_t(N) * es) % 16 == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
    if (!tensor_map_2d(&ma, u8, 1, a, K, T, K, i8::BK, i8::BM, sw) ||
        !tensor_map_2d(&mb, u8, 1, b, K, N, K, i8::BK, 128, sw))
      return STAPLE_ECUDA;
    mo = ma;
    if (p.tma_out &&
        !tensor_map_2d(&mo, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                       es, y, N, T, N, 32, 32,
                       bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
      return STAPLE_ECUDA;
    return bf16 ? go_tiles<true>(di, ma, mb, mo, p, st) : go_tiles<false>(di, ma, mb, mo, p, st);
  }
  p.vec_out = (N % 4) == 0 && (reinterpret_cast<uintptr_t>(y) & uintptr_t(4 * es - 1)) == 0;
  p.rows = pl.rows;
  p.stages = pl.stages;
  if (!tensor_map_2d(&mb, u8, 1, b, K, N, K, i8::BK, uint32_t(p.rows), sw) ||
      !tensor_map_2d(&ma, u8, 1, a, K, T, K, i8::BK, uint32_t(p.tokens), sw))
    return STAPLE_ECUDA;
  return bf16 ? go_split_c<true>(di, mb, ma, p, pl, tiles_t, st)
              : go_split_c<false>(di, mb, ma, p, pl, tiles_t, st);
}

}  // namespace stp
