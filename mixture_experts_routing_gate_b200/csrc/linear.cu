// The linear projection with its epilogue: y = act(x . w^T + bias) + residual, x [T, K] and w [N, K] bf16,
// fp32 accumulation, y bf16 or fp32.
//
// Two kernels.  Up to 16 tokens the weights are read for at most sixteen columns of products, so what counts
// is the weight stream (linear_stream_kernel, mma.sync); above, the products are tiles on the tcgen05 tensor
// cores (linear_gemm_kernel).  Both add the bias, apply the activation and add the residual to the fp32
// accumulators, which are rounded once.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "serving.h"
#include "stream.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------------------------------------
// the epilogue
// ------------------------------------------------------------------------------------------------
// NaN goes through every branch.  silu and the tanh form of gelu are z / (1 + e^-a) (no cancellation for
// negative z); the exact gelu uses erfc for the same reason.  The fast exponential's error grows with its argument (2^-20
// at z = -10), far below a bf16 output's rounding, not below an fp32 one's: kExact takes the accurate one.
template <int kAct, bool kExact>
__device__ __forceinline__ float activate(float z) {
  auto e = [](float a) { return kExact ? expf(a) : __expf(a); };
  if (kAct == MOE_ACT_RELU) return z < 0.f ? 0.f : z;
  if (kAct == MOE_ACT_SILU) return __fdiv_rn(z, 1.f + e(-z));
  if (kAct == MOE_ACT_GELU) return 0.5f * z * erfcf(-0.70710678f * z);
  if (kAct == MOE_ACT_GELU_TANH) return __fdiv_rn(z, 1.f + e(-1.5957691f * (z + 0.044715f * z * z * z)));
  return z;
}

// Eight consecutive outputs (columns c .. c + 7 of row t) in two steps, so that a caller can have the loads of
// several under way: what the epilogue reads, then what it computes and writes.  Whole vectors where the rows
// are aligned, single elements at the edge of N and elsewhere.
__device__ __forceinline__ bool whole8(const LinearParams& p, long c) { return c + 8 <= p.N; }

__device__ __forceinline__ void load_bias8(const LinearParams& p, long c, float (&b)[8]) {
  if (p.bias != nullptr && p.bias_vec && whole8(p, c)) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.bias + c)), y = __ldg(reinterpret_cast<const float4*>(p.bias + c) + 1);
    b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
    b[4] = y.x; b[5] = y.y; b[6] = y.z; b[7] = y.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = p.bias != nullptr && c + i < p.N ? __ldg(p.bias + c + i) : 0.f;
  }
}
__device__ __forceinline__ uint4 load_residual8(const LinearParams& p, int t, long c) {
  if (p.residual == nullptr || !p.residual_vec || !whole8(p, c)) return make_uint4(0u, 0u, 0u, 0u);
  return *reinterpret_cast<const uint4*>(p.residual + (size_t)t * p.ldr + c);
}

template <int kAct, bool kExact>
__device__ __forceinline__ void finish8(const LinearParams& p, int t, long c, const float (&z)[8], const float (&bias)[8],
                                        const uint4& res) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate<kAct, kExact>(z[i] + bias[i]);
  const bool whole = whole8(p, c);
  if (p.residual != nullptr) {
    if (whole && p.residual_vec) {
      const uint32_t w[4] = {res.x, res.y, res.z, res.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const __nv_bfloat16* r = p.residual + (size_t)t * p.ldr + c;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.N) v[i] += __bfloat162float(r[i]);
    }
  }
  if (p.out_fp32) {
    float* y = static_cast<float*>(p.y) + (size_t)t * p.ldy + c;
    if (whole && p.y_vec) {
      reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.N) y[i] = v[i];
    }
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + (size_t)t * p.ldy + c;
    if (whole && p.y_vec) {
      *reinterpret_cast<uint4*>(y) = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                                                bf16x2_bits(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.N) y[i] = __float2bfloat16_rn(v[i]);
    }
  }
}

// f(std::integral_constant) for the descriptor's activation: one branch for a whole block of outputs.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

// ------------------------------------------------------------------------------------------------
// up to 16 tokens: a weight stream
//
// Work is cut into stages of 64 weight rows x 128 elements of k (16 KB), numbered tile by tile, and every
// CTA takes an equal run of them, whatever the number of tiles: 112 tiles of 64 rows on 148 SMs would keep a
// quarter of them idle.  (7168 x 7168, one token: 21 us in a graph, of which the weights' bytes need 16.)  A tile that spans several CTAs is added up by the last of them to arrive, from
// fp32 partials in the workspace and in the order of the CTAs, so results do not depend on scheduling
// and no CTA waits for another.
//
// One thread keeps TMA copies in flight into a ring of about 180 KB, sixteen warps compute: two groups taking
// alternate stages (the ring has an even number of slots, so a slot always belongs to one group), in each
// group four warps along k times two along the rows.  The weights are the 16-row operand of mma.sync
// m16n8k16, the tokens its columns; thread t of a quad holds 8 consecutive elements of k for both, so a
// weight fragment is one conflict-free 16-byte load from TMA's 128-byte swizzle and a token fragment one
// 16-byte load from L1 or L2, a stage ahead.
// ------------------------------------------------------------------------------------------------
constexpr int kStreamWarps = 16, kStreamConsumers = kStreamWarps * 32, kStreamThreads = kStreamConsumers + 32;
constexpr int kStreamRows = 64, kStreamK = 128, kStreamBytes = kStreamRows * kStreamK * 2;
constexpr int kStreamMaxStages = 12;
constexpr int kStreamPitch = kStreamRows + 4;   // floats per token column of the exchange (bank = 8 t + g)

template <int kNT>
struct StreamSmem {
  uint64_t full[kStreamMaxStages], empty[kStreamMaxStages];
  int abort, last;
  int issued;   // stages whose copies the producer has started
  alignas(16) float red[8][8 * kNT][kStreamPitch];
};

__device__ __forceinline__ void stream_sync() {   // the consumer warps, whole
  __syncwarp();
  asm volatile("bar.sync 1, 512;" ::: "memory");
}
static_assert(kStreamConsumers == 512, "the named barrier's thread count");

// First stage of CTA c of G, and the CTA that has stage u, of U stages dealt in equal runs.
// (A stage is 16 KB of weights, so their number fits an int.)
__device__ __forceinline__ int run_start(int U, int c, int G) { return (int)((long)U * c / G); }
__device__ __forceinline__ int run_owner(int U, int u, int G) { return (int)((((long)u + 1) * G - 1) / U); }

template <int kNT>
__global__ void __launch_bounds__(kStreamThreads, 1)
    linear_stream_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ LinearParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* sm = reinterpret_cast<StreamSmem<kNT>*>(ring + p.stages * kStreamBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int G = (int)gridDim.x, ns = (p.K + kStreamK - 1) / kStreamK;
  const int U = (p.N + kStreamRows - 1) / kStreamRows * ns;
  const int u0 = run_start(U, blockIdx.x, G), u1 = run_start(U, blockIdx.x + 1, G);
  volatile int* abort = &sm->abort;
  if (tid < p.stages) {
    mbar_init(&sm->full[tid], 1);
    mbar_init(&sm->empty[tid], 8);
    fence_barrier_init();
  }
  if (tid == 0) {
    sm->abort = 0;
    sm->issued = 0;
    tma_prefetch_desc(&map_w);
  }
  __syncthreads();
  pdl_begin();

  if (warp == kStreamWarps) {
    if (lane == 0 && p.test_stall != kStallCopies) {
      const int most = p.test_stall == kStallLater ? 5 : 0x7fffffff;
      int slot = 0, issued = 0;
      uint32_t ph = 0;
      int row = u0 / ns * kStreamRows, k = u0 % ns * kStreamK;
      for (int u = u0; u < u1 && issued < most; ++u) {
        // A consumer whose wait was given up goes on and frees stages whose fill may be under way, but has seen
        // `abort` set before: a second fill would arm the barrier twice.
        if (!mbar_wait(&sm->empty[slot], ph ^ 1, abort, p.ew, 501) || *abort) break;
        uint8_t* dst = ring + slot * kStreamBytes;
        mbar_arrive_expect_tx(&sm->full[slot], kStreamBytes);   // whole boxes: zeros past K and N
        tma_load_2d(dst, &map_w, &sm->full[slot], k, row);
        tma_load_2d(dst + kStreamBytes / 2, &map_w, &sm->full[slot], k + 64, row);
        ++issued;
        if ((k += kStreamK) >= p.K) {
          k = 0;
          row += kStreamRows;
        }
        if (++slot == p.stages) {
          slot = 0;
          ph ^= 1;
        }
      }
      sm->issued = issued;
    }
  } else {
    const int grp = warp >> 3, wk = warp & 3, wr = (warp >> 2) & 1, g = lane >> 2, t = lane & 3;
    const uint32_t ring_addr = smem_u32(ring);
    uint4 nxt[kNT];
    auto fetch = [&](int u) {   // this warp's 32 elements of k of stage u, for token columns g and g + 8
      const int k = u % ns * kStreamK + wk * 32 + t * 8;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        nxt[nt] = g + 8 * nt < p.T && k < p.K
                      ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)(g + 8 * nt) * p.ldx + k))
                      : make_uint4(0u, 0u, 0u, 0u);
    };
    int slot = grp % p.stages;
    uint32_t ph = 0;
    if (u0 + grp < u1) fetch(u0 + grp);
    for (int u = u0; u < u1;) {
      const int tile = u / ns, end = min((tile + 1) * ns, u1);
      const bool starts = u == tile * ns, ends = end == (tile + 1) * ns;
      float acc[2][kNT][4] = {};
      for (int s = u + ((u - u0 + grp) & 1); s < end; s += 2) {   // the group's stages: those of its parity from u0
        uint4 cur[kNT];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) cur[nt] = nxt[nt];
        if (s + 2 < u1) fetch(s + 2);
        if (!mbar_try_wait(&sm->full[slot], ph) && !*abort) mbar_wait(&sm->full[slot], ph, abort, p.ew, 502);
        __syncwarp();
        // elements [32 wk, 32 wk + 32) are half of 64-element column wk / 2
        const uint32_t at = ring_addr + slot * kStreamBytes + (wk >> 1) * (kStreamBytes / 2) +
                            (wr * 32 + g) * 128 + ((((wk & 1) * 4 + t) ^ g) << 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 lo = lds128(at + i * 16 * 128), hi = lds128(at + (i * 16 + 8) * 128);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma_16816<false>(acc[i][nt], lo.x, hi.x, lo.y, hi.y, cur[nt].x, cur[nt].y);
            mma_16816<false>(acc[i][nt], lo.z, hi.z, lo.w, hi.w, cur[nt].z, cur[nt].w);
          }
        }
        mbar_arrive_after_reads(&sm->empty[slot]);
        slot += 2;
        if (slot >= p.stages) {
          slot -= p.stages;
          ph ^= 1;
        }
      }
      stream_sync();   // the exchange buffer is free
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float* c = &sm->red[grp * 4 + wk][nt * 8 + 2 * t][wr * 32 + i * 16 + g];
          c[0] = acc[i][nt][0];
          c[kStreamPitch] = acc[i][nt][1];
          c[8] = acc[i][nt][2];
          c[kStreamPitch + 8] = acc[i][nt][3];
        }
      stream_sync();
      // thread: eight rows of one token's column
      const int col = tid >> 3, r8 = (tid & 7) * 8;
      const bool in = col < p.T;
      const long c8 = (long)tile * kStreamRows + r8;
      float z[8] = {};
      if (in) {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float4* src = reinterpret_cast<const float4*>(&sm->red[w][col][r8]);
          const float4 a = src[0], b = src[1];
          z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
          z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
        }
      }
      bool finish = in;
      if (!(starts && ends)) {
        // a slot per CTA for the tile it continues and one for the tile it leaves unfinished
        const int c0 = run_owner(U, tile * ns, G), c1 = run_owner(U, (tile + 1) * ns - 1, G);
        constexpr int kSlot = kStreamRows * 16;
        auto place = [&](int c) { return p.scratch + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kSlot + col * kStreamRows + r8; };
        if (in) {
          float4* dst = reinterpret_cast<float4*>(place(blockIdx.x));
          dst[0] = make_float4(z[0], z[1], z[2], z[3]);
          dst[1] = make_float4(z[4], z[5], z[6], z[7]);
          __threadfence();
        }
        stream_sync();
        if (tid == 0) {
          const int last = atomicAdd(&p.gc->linear_done[c0], 1) == c1 - c0;
          if (last) p.gc->linear_done[c0] = 0;
          __threadfence();
          sm->last = last;
        }
        stream_sync();
        finish = in && sm->last;
        if (finish) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float4* src = reinterpret_cast<const float4*>(place(c));
            const float4 a = __ldcg(src), b = __ldcg(src + 1);
            z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
            z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
          }
        }
      }
      if (finish && c8 < p.N) {
        float b[8];
        load_bias8(p, c8, b);
        const uint4 res = load_residual8(p, col, c8);
        with_activation(p.act, [&](auto act) { finish8<decltype(act)::value, true>(p, col, c8, z, b, res); });
      }
      u = end;
    }
  }
  __syncwarp();
  __syncthreads();
  if (*abort && tid == kStreamConsumers) {   // every copy already started lands before the CTA leaves
    for (int i = sm->issued > p.stages ? sm->issued - p.stages : 0; i < sm->issued; ++i)
      mbar_wait(&sm->full[i % p.stages], (i / p.stages) & 1, nullptr, nullptr, 0, 200000000LL);
  }
}

// ------------------------------------------------------------------------------------------------
// more tokens: tiles on the tcgen05 tensor cores
//
// A CTA's tile is 128 tokens (the MMA's M, a TMEM lane each) by kN = 64 or 128 features (its N).  kPair: clusters
// of two CTAs share MMAs of M = 256 by kN = 256 (cta_group::2): each loads its 128 tokens and half of the weight
// rows, 32 KB for 64 elements of k, half of what two single CTAs load for the same products.  Persistent and
// warp-specialised: warp 0 TMA, warp 1 MMA (even CTA), eight epilogue warps, two accumulators in TMEM so that
// a tile's epilogue runs beside the next tile's MMAs.  The epilogue brings 32 x 32 blocks through shared
// memory (pitch 36: 16-byte accesses free of bank conflicts both ways) so that a lane finishes eight
// consecutive features of a row and stores 16 bytes; what it reads (bias, residual) is loaded before the
// block's accumulators are, since its latency, not its arithmetic, bounded the tile.
//
// Measured: 16384 x 5120 x 5120 1.15 to 1.25 PFLOP/s, 0.83 to 0.91 of cuBLAS's sustained rate; the loads are then
// 9 to 9.8 TB/s from L2 to all SMs, which bounds it.  64 x 7168 onto 129280 fp32 logits 341 to 406 us (288 at the
// measured bandwidth).
//
// splits > 1 (fewer tiles than SMs; single CTAs): K is cut over a cluster of 2, 4 or 8 CTAs.  Each leaves its
// fp32 tile in shared memory, and each adds up and finishes its share of the columns from all of them
// through distributed shared memory, in the order of the slices.
// ------------------------------------------------------------------------------------------------
constexpr int kGemmStagesMax = 12;
constexpr int kEpiWarps = 8;
constexpr int kLinThreads = 64 + kEpiWarps * 32;
constexpr int kEpiPitch = 36;
constexpr int kSplitPitch = 132;   // floats per row of a cut tile in shared memory

struct LinGemmSmem {
  uint64_t full[kGemmStagesMax], empty[kGemmStagesMax];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued;   // stages that the producer has filled
  alignas(16) float stage[kEpiWarps][32 * kEpiPitch];
};

template <bool kPair, int kN>
struct LinTile {
  static constexpr int kBN = kN;
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kBBytes = kBN / kCtas * 128;
};

// Unit w: tile and slice of k.  Tiles run through groups of eight token blocks, all of a group's token blocks
// for one feature block before the next, so that what runs at a time shares weights and tokens in L2.
struct LinUnit {
  int m, n, k0, k1, tile, split;
};
__device__ __forceinline__ LinUnit lin_unit(const LinearParams& p, int w) {
  LinUnit u;
  u.tile = w / p.splits;
  u.split = w - u.tile * p.splits;
  const int nk = (p.K + 63) / 64, group = 8 * p.n_tiles, gi = u.tile / group, r = u.tile - gi * group;
  const int rows = min(8, p.m_tiles - gi * 8);
  u.n = r / rows;
  u.m = gi * 8 + (r - u.n * rows);
  u.k0 = (int)((long)nk * u.split / p.splits);
  u.k1 = (int)((long)nk * (u.split + 1) / p.splits);
  return u;
}

// kPromote (fp32 outputs; bf16 ones round 2^-8, five hundred times as much): the tensor cores add into the fp32 accumulator with truncation, a bias that grows
// with the number of steps -- 8e-6 of the result after 7168 products.  So K is accumulated in chunks of
// kPromoteSteps * 64, alternating between the two accumulators, and the epilogue warps add the chunks in
// registers, rounding to nearest.
constexpr int kPromoteSteps = 8;
template <bool kPair, int kN, bool kPromote>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ LinearParams p) {
  using L = LinTile<kPair, kN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Batches below 128 tokens load and stage only x_box rows of x: the MMA then reads the weights (or the next
  // stage, or the barriers) as its other rows, whose accumulators are never read.
  const int a_bytes = p.x_box * 128, stage_bytes = a_bytes + L::kBBytes;
  auto* sm = reinterpret_cast<LinGemmSmem*>(smem + p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int first = kPair ? blockIdx.x >> 1 : blockIdx.x, step = kPair ? gridDim.x >> 1 : gridDim.x;
  const int units = p.m_tiles * p.n_tiles * p.splits;
  volatile int* abort = &sm->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm->acc_full[a], 1);
      mbar_init(&sm->acc_empty[a], L::kCtas * kEpiWarps);
    }
    mbar_init(&sm->drain, 1);
    sm->abort = 0;
    sm->issued = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&sm->tmem_base, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sm->tmem_base, 512);
      tmem_relinquish();
    }
  }
  pdl_begin();
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // both CTAs' barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      int issued = 0;
      const int most = p.test_stall == kStallLater ? 3 : 0x7fffffff;
      const uint32_t full_leader = kPair ? cluster_addr(&sm->full[0], 0) : 0u;   // + 8 * stage
      bool ok = p.test_stall != kStallCopies;
      for (int w = first; w < units && ok; w += step) {
        const LinUnit u = lin_unit(p, w);
        const int row_x = (u.m * L::kCtas + (int)rank) * 128, row_w = u.n * L::kBN + (int)rank * (L::kBN / L::kCtas);
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (issued == most || !mbar_wait(&sm->empty[st], ph ^ 1, abort, p.ew, 511)) {
            ok = false;
            break;
          }
          ++issued;
          uint8_t* sa = smem + st * stage_bytes;
          if (leader) mbar_arrive_expect_tx(&sm->full[st], L::kCtas * stage_bytes);   // whole boxes: zeros outside
          if (kPair) {
            tma_load_2d_pair(sa, &map_x, full_leader + 8u * st, kb * 64, row_x);
            tma_load_2d_pair(sa + a_bytes, &map_w, full_leader + 8u * st, kb * 64, row_w);
          } else {
            tma_load_2d(sa, &map_x, &sm->full[st], kb * 64, row_x);
            tma_load_2d(sa + a_bytes, &map_w, &sm->full[st], kb * 64, row_w);
          }
          if (++st == p.stages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      sm->issued = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_bf16_f32(128 * L::kCtas, L::kBN);
      int st = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      auto finish_acc = [&]() {
        if (kPair) umma_commit_pair_both(&sm->acc_full[acc]);
        else umma_commit(&sm->acc_full[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_ph ^= 1;
        }
      };
      for (int w = first; w < units && ok; w += step) {
        const LinUnit u = lin_unit(p, w);
        uint32_t d = 0;
        for (int kb = u.k0; kb < u.k1; ++kb) {
          const bool start = kb == u.k0 || (kPromote && (kb - u.k0) % kPromoteSteps == 0);
          if (start) {   // a new accumulator
            if (kb != u.k0) finish_acc();
            if (!mbar_wait(&sm->acc_empty[acc], acc_ph ^ 1, abort, p.ew, 512)) {
              ok = false;
              break;
            }
            tc_fence_after();
            d = tmem + acc * L::kBN;
          }
          if (!mbar_wait(&sm->full[st], ph, abort, p.ew, 513)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + st * stage_bytes);
          const uint64_t a = sdesc_kmajor_sw128(sa), b = sdesc_kmajor_sw128(sa + a_bytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t accumulate = !start || kk != 0;
            if (kPair) umma_bf16_pair(d, a + 2 * kk, b + 2 * kk, idesc, accumulate);
            else umma_bf16(d, a + 2 * kk, b + 2 * kk, idesc, accumulate);
          }
          if (kPair) umma_commit_pair_both(&sm->empty[st]);
          else umma_commit(&sm->empty[st]);
          if (++st == p.stages) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        finish_acc();
      }
      if (!ok) {
        if (kPair) umma_commit_pair(&sm->drain);
        else umma_commit(&sm->drain);
        mbar_wait(&sm->drain, 0, nullptr, nullptr, 0, 200000000LL);
      }
    }
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    const int q = warp & 3, part = (warp - 2) >> 2;   // TMEM lane quadrant; 32-column blocks part, part + 2, ...
    float* stage = sm->stage[warp - 2];
    const uint32_t acc_empty_leader = kPair ? cluster_addr(&sm->acc_empty[0], 0) : 0u;   // + 8 * buffer
    int acc = 0;
    uint32_t acc_ph = 0;
    for (int w = first; w < units; w += step) {
      const LinUnit u = lin_unit(p, w);
      const int row0 = (u.m * L::kCtas + (int)rank) * 128 + q * 32;   // the warp's first token
      const long col0 = (long)u.n * L::kBN;
      uint32_t taddr = 0;
      auto await_acc = [&]() {
        const bool got = mbar_wait_warp(&sm->acc_full[acc], acc_ph, abort, p.ew, 514);
        (void)mbar_try_wait(&sm->acc_full[acc], acc_ph);   // every lane observes the completed phase
        tc_fence_after();
        taddr = tmem + acc * L::kBN + ((uint32_t)(q * 32) << 16);
        return got;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair) mbar_arrive_remote(acc_empty_leader + 8u * acc);
          else mbar_arrive(&sm->acc_empty[acc]);
        }
        if (++acc == 2) {
          acc = 0;
          acc_ph ^= 1;
        }
      };
      auto load_block = [&](int blk, float (&v)[32]) {
        tmem_ld16(taddr + blk * 32, *reinterpret_cast<float(*)[16]>(&v[0]));
        tmem_ld16(taddr + blk * 32 + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
        tmem_ld_wait();
      };
      constexpr int kMine = L::kBN / 64;   // 32-column blocks of this warp
      float sum[kPromote ? kMine : 1][32];
      bool have = await_acc();
      if constexpr (kPromote) {
        const int chunks = (u.k1 - u.k0 + kPromoteSteps - 1) / kPromoteSteps;
#pragma unroll
        for (int b = 0; b < kMine; ++b)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[b][i] = 0.f;
        for (int c = 0; c < chunks && have; ++c) {
          if (c > 0) have = await_acc();
#pragma unroll
          for (int b = 0; b < kMine; ++b) {
            float v[32];
            load_block(part + 2 * b, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[b][i] += v[i];
          }
          release();
        }
      }
      if (!have) break;
      // block b of the warp's columns, as accumulated
      auto block = [&](int b, float (&v)[32]) {
        if constexpr (kPromote) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = sum[b][i];
        } else {
          load_block(part + 2 * b, v);
        }
      };
      if (!kPair && p.splits > 1) {   // the stages are drained: the tile takes their place
        float* dst = reinterpret_cast<float*>(smem) + (q * 32 + lane) * kSplitPitch;
#pragma unroll
        for (int b = 0; b < kMine; ++b) {
          float v[32];
          block(b, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(dst + (part + 2 * b) * 32 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        break;   // one unit a CTA
      }
      with_activation(p.act, [&](auto act) {
#pragma unroll(kPromote ? kMine : 1)
        for (int b = 0; b < kMine; ++b) {
          const long c = col0 + (part + 2 * b) * 32, c8 = c + (lane & 3) * 8;
          if (row0 >= p.T || c >= p.N) break;   // warp-uniform: nothing of this block (or later ones) is kept
          const bool in = c8 < p.N;
          float b8[8];
          uint4 res[4];
          load_bias8(p, c8, b8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = row0 + (lane >> 2) + 8 * i;
            res[i] = in && t < p.T ? load_residual8(p, t, c8) : make_uint4(0u, 0u, 0u, 0u);
          }
          float v[32];
          block(b, v);
          if (!kPromote && b == kMine - 1) release();
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(stage + lane * kEpiPitch + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = (lane >> 2) + 8 * i;
            const float4* src = reinterpret_cast<const float4*>(stage + r * kEpiPitch + (lane & 3) * 8);
            const float4 lo = src[0], hi = src[1];
            const float z[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            if (in && row0 + r < p.T) finish8<decltype(act)::value, kPromote>(p, row0 + r, c8, z, b8, res[i]);
          }
          __syncwarp();
        }
      });
      // blocks past T or N were not loaded: the accumulator is released here
      if (!kPromote && (row0 >= p.T || col0 + (part + 2 * (kMine - 1)) * 32 >= p.N)) release();
    }
  }

  if (!kPair && p.splits > 1) {
    __syncwarp();
    cluster_sync();   // every slice's tile is in shared memory
    if (warp >= 2) {
      const LinUnit u = lin_unit(p, blockIdx.x);
      const int width = L::kBN / p.splits, per_row = width / 8, rows = min(128, p.T - u.m * 128);
      with_activation(p.act, [&](auto act) {
        for (int i = (int)threadIdx.x - 64; i < rows * per_row; i += kEpiWarps * 32) {
          const int r = i / per_row, c = u.split * width + (i - r * per_row) * 8;
          const long c8 = (long)u.n * L::kBN + c;
          if (c8 >= p.N) continue;
          const int t = u.m * 128 + r;
          float z[8] = {}, b8[8];
          load_bias8(p, c8, b8);
          const uint4 res = load_residual8(p, t, c8);
          const float* mine = reinterpret_cast<const float*>(smem) + r * kSplitPitch + c;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if (s >= p.splits) break;
            const uint32_t src = cluster_addr(mine, s);
            const float4 lo = ld_cluster_v4(src), hi = ld_cluster_v4(src + 16);
            z[0] += lo.x; z[1] += lo.y; z[2] += lo.z; z[3] += lo.w;
            z[4] += hi.x; z[5] += hi.y; z[6] += hi.z; z[7] += hi.w;
          }
          finish8<decltype(act)::value, kPromote>(p, t, c8, z, b8, res);
        }
      });
    }
    __syncwarp();
    cluster_sync();   // nobody reads this CTA's tile any more
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  // A wait was given up: every load already started lands before a CTA leaves (a pair's, on the even CTA's barriers).
  if (*abort && leader && threadIdx.x == 0)
    for (int i = sm->issued > p.stages ? sm->issued - p.stages : 0; i < sm->issued; ++i)
      mbar_wait(&sm->full[i % p.stages], (i / p.stages) & 1, nullptr, nullptr, 0, 200000000LL);
  __syncwarp();
  if (kPair) cluster_sync();  // no remote signal or MMA of either CTA is outstanding past this point
  if (*abort) {
    // a wait ran out: give any TMA copy this CTA may still have in flight time to land
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000LL) {
    }
  }
  tc_fence_after();
  if (warp == 1) {
    if (kPair) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

template <bool kPair, int kN, bool kPromote>
cudaError_t launch_gemm(const CUtensorMap& map_x, const CUtensorMap& map_w, LinearParams p, int num_sms,
                        cudaStream_t stream) {
  using L = LinTile<kPair, kN>;
  auto kernel = linear_gemm_kernel<kPair, kN, kPromote>;
  const size_t stage = (size_t)p.x_box * 128 + L::kBBytes;
  p.stages = (int)std::min<size_t>(kGemmStagesMax, (227 * 1024 - 1024 - sizeof(LinGemmSmem)) / stage);
  const size_t smem = 1024 + p.stages * stage + sizeof(LinGemmSmem);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const int units = p.m_tiles * p.n_tiles * p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L::kCtas * (num_sms / L::kCtas));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  const int cluster = kPair ? 2 : p.splits;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  int slots = num_sms / L::kCtas, active = 0;
  if (kPair && cudaOccupancyMaxActiveClusters(&active, kernel, &cfg) == cudaSuccess && active > 0 && active < slots)
    slots = active;
  (void)cudaGetLastError();
  cfg.gridDim = dim3(p.splits > 1 ? units : L::kCtas * std::min(units, slots));
  cfg.numAttrs = n + pdl_attr(attr + n);
  return cudaLaunchKernelEx(&cfg, kernel, map_x, map_w, p);
}

template <int kNT>
cudaError_t launch_stream(const CUtensorMap& map_w, LinearParams p, int num_sms, cudaStream_t stream) {
  auto kernel = linear_stream_kernel<kNT>;
  p.stages = (int)std::min<size_t>(kStreamMaxStages, (227 * 1024 - 1024 - sizeof(StreamSmem<kNT>)) / kStreamBytes) & ~1;
  const size_t smem = 1024 + (size_t)p.stages * kStreamBytes + sizeof(StreamSmem<kNT>);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const long U = (long)((p.N + kStreamRows - 1) / kStreamRows) * ((p.K + kStreamK - 1) / kStreamK);
  return launch_pdl(kernel, dim3((unsigned)std::min<long>(num_sms, U)), dim3(kStreamThreads), smem, stream, map_w, p);
}

}  // namespace

LinearPlan linear_plan(int T, int K, int N, int num_sms) {
  LinearPlan plan{};
  if (T <= kLinearStreamTokens) {
    plan.kind = LinearPlan::kStream;
    plan.w_box = kStreamRows;
    plan.scratch_floats = (size_t)num_sms * 2 * kStreamRows * 16;
    return plan;
  }
  // Time of a choice, in loads of 32 KB by every SM at once (about 0.48 us: L2 gives all SMs together some
  // 10 TB/s, which bounds these tiles before the tensor cores do).  A step is 64 elements of k; a unit of
  // work also has its pipeline's fill and its epilogue, a cut one the join.  A cluster of 4 or 8 CTAs needs
  // that many free SMs in one GPC, so fewer of those fit at a time.
  //
  // All candidates measured in graphs on 14 shapes of 17 to 4096 tokens: the choice is the fastest in 13 (64 x 7168
  // x 7168: 128 columns cut in two 27 us, 64 uncut 42, pairs 46; 300 x 7168 x 7168: pairs 48, 128 columns 82; 1024 x
  // 7168 x 2048: 128 columns 45, pairs 46), and not for 128 x 5120 x 1536 (128 columns cut in eight 20.1 us, 64 in
  // four 15.4).
  const long nk = (K + 63) / 64;
  double best = 0;
  for (int kind = 0; kind < 3; ++kind) {
    const bool pair = kind == 2;
    const int rows = pair ? 256 : 128, cols = pair ? 256 : kind == 1 ? 128 : 64;
    const long m = ((long)T + rows - 1) / rows, n = ((long)N + cols - 1) / cols;
    const double step = pair ? 1.0 : std::max(0.25, (std::min(T, 128) + cols) / 256.0);
    for (int s = 1; s <= (pair ? 1 : 8) && s <= nk; s *= 2) {
      const long slots = pair ? num_sms / 2 : s <= 2 ? num_sms : s == 4 ? num_sms * 6 / 7 : num_sms * 3 / 4;
      const long units = m * n * s;
      if (s > 1 && units > slots) break;   // K is cut only to fill the SMs once
      const double unit = ((nk + s - 1) / s) * step + (pair ? 12 : 8) + (s > 1 ? 3 : 0);
      const double cost = ((units + slots - 1) / slots) * unit;
      if (best == 0 || cost < best) {
        best = cost;
        plan.kind = pair ? LinearPlan::kPair : LinearPlan::kSolo;
        plan.m_tiles = (int)m;
        plan.n_tiles = (int)n;
        plan.splits = s;
        plan.w_box = pair ? 128 : cols;
        plan.x_box = pair || T > 64 ? 128 : T > 32 ? 64 : 32;
      }
    }
  }
  return plan;
}

cudaError_t launch_linear(const LinearPlan& plan, const CUtensorMap& map_x, const CUtensorMap& map_w, LinearParams p,
                          int num_sms, cudaStream_t stream) {
  p.m_tiles = plan.m_tiles;
  p.n_tiles = plan.n_tiles;
  p.splits = plan.splits;
  p.x_box = plan.x_box;
  if (plan.kind == LinearPlan::kStream)
    return p.T <= 8 ? launch_stream<1>(map_w, p, num_sms, stream) : launch_stream<2>(map_w, p, num_sms, stream);
  auto gemm = [&](auto promote) {
    constexpr bool kPromote = decltype(promote)::value;
    if (plan.kind == LinearPlan::kPair) return launch_gemm<true, 256, kPromote>(map_x, map_w, p, num_sms, stream);
    return plan.w_box == 128 ? launch_gemm<false, 128, kPromote>(map_x, map_w, p, num_sms, stream)
                             : launch_gemm<false, 64, kPromote>(map_x, map_w, p, num_sms, stream);
  };
  return p.out_fp32 ? gemm(std::true_type{}) : gemm(std::false_type{});
}

}  // namespace moe
