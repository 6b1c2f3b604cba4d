// The whole MoE layer for a few tokens (decode batches of at most 16) in one launch.
//
//   l = x . Wg^T (+ offset), s = affinity(l), experts = group-limited top-k of s + bias (or the token-id
//   table's row), w = s / sum(s) * scale;  h_e = silu(x w1_e^T) * (x w3_e^T);  y = sum_j w_j h w2^T + shared.
//
// What bounds it: the weights of the chosen experts, read once -- every weight meets one to sixteen tokens,
// far below the flops per byte at which the tensor cores would matter.  So the kernel is a weight stream:
//
// * one CTA per SM, all resident at once (cooperative launch).  Two producer warps keep TMA copies of 8 KB in
//   flight into two rings of together 136 (MXFP4) or 160 KB of shared memory, two groups of eight consumer warps
//   compute, each on tiles of its own.  At 44 bytes/ns per SM the rings hold about 4 us of the stream, more
//   than the memory latency, so the stream does not stop between the phases.  (Copies of single rows, 1 KB,
//   cost about 65 ns each whoever issues them and held the stream at 2 TB/s.)
// * two router warps turn the logits into the lists of experts while the consumers work on the shared
//   expert, whose weights need no routing: the selection's latency (it runs once, on code and data that are
//   not cached) is hidden.
// * the products run on mma.sync with the weight rows as the 16-row operand and the tokens as the 8 columns
//   of one or two tiles, so each weight is read from shared memory once.  The reduction index is permuted
//   alike for both operands (thread t of a quad holds 8 consecutive elements), so that a weight fragment is
//   one conflict-free shared load from TMA's 128-byte swizzle and a token fragment one 16-byte load from
//   global memory (L1 or L2; a stage ahead), whatever the token's row.  The eight warps of a group split a
//   stage along k; the accumulators of a tile are added through shared memory in warp order: nothing depends
//   on scheduling.  (All sixteen on one tile, in alternate stages, met at barriers twice as often.)
// * in the up projections rows 0-7 of an MMA are w1's and rows 8-15 w3's, so gate and value of a feature meet
//   in one accumulator tile.  A CTA starts on down-projection tiles of an expert as soon as all of that
//   expert's h is written (a counter per expert), with no barrier between the projections; CTAs that had one
//   up tile less take more of the first down tiles.
//
// bf16 weights: tiles of 16 rows, 512 elements of k a stage, bf16 MMAs; h is held in two bf16 parts, in columns that
// few tokens leave free (beside one rounded part: no time up to 8 tokens, 387 -> 403 us at 16; the error of y
// against 64 bits 2.4e-3 -> 1.7e-3, its own rounding).  Measured (floor at the measured copy bandwidth in
// brackets): d = 7168, I = 2048, 9 experts, one token 136 us (122); d = 5120, I = 1536, 16 tokens on 384 unevenly
// popular experts 320 to 405 us, by the experts drawn (278); d = 256, one token 18 us.
//
// MXFP4 weights: what travels is a quarter, so the arithmetic of decoding is what has to be cheap.  The
// hardware's E2M1 -> f16 conversion takes 73 codes/clock/SM (measured; the stream brings 44), where placing
// the bits by shifts and logic, 15 operations for 8 codes, takes 34 and bounded the first form of this kernel
// at 1.4 TB/s.  So the MMAs are f16: the activations of each block of 32 are scaled by a power of two to below
// 2^15 and held in f16 (exact for bf16 values down to 2^-31 of the block's largest, off by 2^-39 of it
// at most below), and the block's scale and the weights' UE8M0 scale multiply the fp32 accumulators of its 32
// elements.  An up tile is 32 features, one block of h, whose scale its epilogue can therefore choose; tiles
// are 64 rows, 512 codes of k a stage, so a token fragment serves four MMA row tiles.  Measured: d = 7168, I =
// 2048, one token 75 to 79 us (33), eight tokens 350 to 362 us (206); half of the issue slots are used, so what is left is in
// the consumers' instructions and waits.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "serving.h"
#include "stream.cuh"

namespace moe {

namespace {

constexpr int kGroups = 2, kGroupWarps = 8, kGroupThreads = kGroupWarps * 32;   // a group has a ring and tiles
constexpr int kConsumerWarps = kGroups * kGroupWarps, kConsumers = kConsumerWarps * 32;
constexpr int kRouterWarps = 2;
constexpr int kRouters = kRouterWarps * 32;
constexpr int kDecThreads = kConsumers + kGroups * 32 + kRouters;
constexpr int kMaxStages = 8;        // of a ring
constexpr int kMaxT = kDecodeMaxTokens;
constexpr int kMaxS = kMaxT * kMaxRouteTopk;
constexpr int kMaxAct = kMaxS + 1;  // active experts: the shared one and at most one per slot
constexpr int kMaxE = 512;
constexpr int kGateRows = 16;       // router rows per unit of the logit phase
constexpr int kGatePitch = 20;      // floats per token column of its exchange (bank = 8 t + g)
static_assert(kMaxT <= 16, "two column tiles of eight tokens, token masks of 16 bits");
static_assert(kMaxAct <= sizeof(GridCounters::ready) / sizeof(int), "a counter for every active expert");

// A stage holds kChunk elements of k of kRows weight rows as two blocks (up: w1's and w3's rows), each as TMA
// writes a box of 128 bytes x kRows / 2 x kCols in the 128-byte swizzle -- the 16-byte unit u of row r of
// column c lies at c * (kRows / 2) * 128 + r * 128 + ((u ^ (r & 7)) << 4) -- and, for MXFP4, 16 bytes of
// scales of each row.
template <bool kFp4>
struct Stage {
  static constexpr int kRowTiles = kFp4 ? 4 : 1;
  static constexpr int kRows = 16 * kRowTiles;
  static constexpr int kUp = kRows / 2;                    // features of an up tile
  static constexpr int kChunk = 512;
  static constexpr int kCols = kFp4 ? 2 : 8;               // of 256 codes or 64 bf16
  static constexpr int kColBytes = kRows / 2 * 128;
  static constexpr int kBlock = kCols * kColBytes;
  static constexpr int kSOff = 2 * kBlock;
  static constexpr int kBytes = kSOff + (kFp4 ? kRows * 16 : 0);
  static constexpr int kRedPitch = kRows + 4;              // floats per token column (bank = 8 t + g)
  // exchange buffers: two let a tile's sums run beside the next tile; the four-bit tiles of 9 to 16 tokens
  // leave room for one
  static constexpr int red_bufs(int nt) { return kFp4 && nt == 2 ? 1 : 2; }
};

template <bool kFp4, int kNT>
struct DecodeSmem {
  uint64_t full[kGroups][kMaxStages];
  uint64_t empty[kGroups][kMaxStages];
  uint64_t routed, weighted;        // the lists below are complete; the slots' weights are too
  int abort;
  int n_act;                        // the lists' experts as published with `routed` (0 before); follows `abort`
  int last;
  int up_done[kGroups];             // warps that wrote their part of an up tile's h, over the group's tiles so far
  int issued[kGroups];              // stages whose copies a group's producer has started
  int n_listed;                     // active experts, the shared one first
  int sel_e[kMaxS];
  float sel_w[kMaxS];
  int dup[kMaxS];                   // the token already chose this expert in an earlier slot
  int row_of_slot[kMaxS];
  int tok_of_row[kMaxS + kMaxT];
  float row_w[kMaxS + kMaxT];
  int act_e[kMaxAct], act_off[kMaxAct], act_n[kMaxAct];
  uint32_t mask[kMaxE];             // tokens of each expert
  int off_of[kMaxE];                // first row of each active expert
  float bias[kMaxE], offset[kMaxE]; // the router's (zeros where there is none)
  float scores[kRouterWarps][kMaxE];
  // exchange buffers of the groups; the router logits' exchange takes the first 16 * 8 kNT * kGatePitch floats
  alignas(16) float red[kGroups][Stage<kFp4>::red_bufs(kNT)][kGroupWarps * 8 * kNT * Stage<kFp4>::kRedPitch];
};

// The warps of a group that write h of an up tile with n tokens: a token at a time (MXFP4), or four.
template <bool kFp4>
__device__ __forceinline__ int up_writers(int n) { return kFp4 ? min(n, kGroupWarps) : (n + 3) / 4; }

// Barriers of whole warps: lanes that waited on their own rejoin first.
__device__ __forceinline__ void consumer_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, 512;" ::: "memory");
}
__device__ __forceinline__ void router_sync() {
  __syncwarp();
  asm volatile("bar.sync 2, 64;" ::: "memory");
}
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("bar.sync %0, 256;" ::"r"(3 + group) : "memory");
}
static_assert(kConsumers == 512 && kRouters == 64 && kGroupThreads == 256, "the named barriers' thread counts");

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_add(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int atom_acquire_add(int* p, int v) {
  int old;
  asm volatile("atom.acquire.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
// 16 bytes global -> shared past L1, and this lane's arrival on a barrier once its copies so far landed.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Waits until `*counter` reaches `target`.  Bounded as mbar_wait is.
__device__ __forceinline__ bool grid_wait(const int* counter, int target, volatile int* abort, ErrorWord* ew, int site) {
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(counter) >= target) return true;
    if ((it & 63) == 0) {
      if (*abort) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        record_error(ew, MOE_ERR_TIMEOUT, site);
        *abort = 1;
        return false;
      }
    }
  }
}

// A consumer's wait: the usual, successful test inline; after an abort no waiting at all.  A warp that gives up
// the wait for the lists publishes empty ones (the shared expert alone) in n_act, the word behind `abort`, unless
// the router has just published its own: all warps go by the same lists.  (It is here, and not where the lists
// are waited for, since what is added between two tiles costs the four-bit layer 3 to 5 us of 75.)
constexpr int kListsSite = 409;
__device__ __noinline__ void stage_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, ErrorWord* ew, int site) {
  const bool got = !*abort && mbar_wait(bar, parity, abort, ew, site);
  if (!got && site == kListsSite) {
    if (atomicCAS(const_cast<int*>(abort) + 1, 0, 1) == 0) mbar_arrive(bar);
    __threadfence_block();
  }
}
__device__ __forceinline__ void stage_wait(uint64_t* bar, uint32_t parity, volatile int* abort, ErrorWord* ew, int site) {
  if (!mbar_try_wait(bar, parity)) stage_wait_slow(bar, parity, abort, ew, site);
  __syncwarp();
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void step(int by, int stages) {
    for (slot += by; slot >= stages; slot -= stages) phase ^= 1;
  }
};

// The tiles of a group as (active expert, block of rows); groups are numbered over the grid, `self` of `all`.  Up
// projections: every all-th tile.  Down projections (early > 0): the `early` first rounds are taken by the
// groups from `first` on alone, which had one up tile less than the others; then every all-th.
struct TileIter {
  int j, a, blk, nb, self, all, early, first;
  __device__ TileIter(int nb_, int self_, int all_, int early_ = 0, int first_ = 0)
      : nb(nb_), self(self_), all(all_), early(early_), first(first_) {
    if (early > 0 && self >= first) {
      set(self - first);
    } else {
      const int before = early * (all - first);
      early = 0;
      set(before + self);
    }
  }
  __device__ void set(int j_) {
    j = j_;
    a = j / nb;
    blk = j - a * nb;
  }
  __device__ void next() {
    if (early > 1) {
      --early;
      set(j + all - first);
    } else if (early == 1) {   // j = (early rounds - 1) * (all - first) + self - first
      early = 0;
      set(j + all);
    } else {
      set(j + all);
    }
  }
};
// The down projections' iterator: groups of index >= (up tiles) % all had one up tile less, worth d / I down
// tiles.
__device__ __forceinline__ TileIter down_tiles(const DecodeParams& p, int n_act, int nb_up, int nb_down, int self, int all) {
  const int m = (int)((long)n_act * nb_up % all);
  return TileIter(nb_down, self, all, m == 0 ? 0 : (p.d + p.I / 2) / p.I, m);
}

// ------------------------------------------------------------------------------------------------
// phase 1: partial router logits
// ------------------------------------------------------------------------------------------------
// Unit u: 16 router rows x one slice of k, its blocks of 32 dealt to the warps.  The fp32 weights are split
// exactly into three bf16 parts (hi + mid + lo), whose products with the bf16 activations are exact in fp32.
template <int kNT>
__device__ __forceinline__ void gate_partials(const DecodeParams& p, float* red, int warp, int lane) {
  const int groups = p.E / kGateRows, units = groups * p.gate_splits, nb = p.d / 32;
  const int g = lane >> 2, t = lane & 3, tid = warp * 32 + lane;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int grp = u % groups, sp = u / groups;
    const int b1 = (sp + 1) * nb / p.gate_splits;
    const float* w0 = p.w_gate + (size_t)(grp * kGateRows + g) * p.d + t * 8;
    float acc[kNT][4] = {};
    for (int b = sp * nb / p.gate_splits + warp; b < b1; b += kConsumerWarps) {
      float w[2][8];
      uint4 x[kNT];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4* src = reinterpret_cast<const float4*>(w0 + (size_t)r * 8 * p.d + b * 32);
        *reinterpret_cast<float4*>(&w[r][0]) = __ldg(src);
        *reinterpret_cast<float4*>(&w[r][4]) = __ldg(src + 1);
      }
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        x[nt] = g + 8 * nt < p.T ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)(g + 8 * nt) * p.d + b * 32 + t * 8))
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
      for (int plane = 0; plane < 3; ++plane) {
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[r][i] = bf16x2_bits(w[r][2 * i], w[r][2 * i + 1]);
            w[r][2 * i] -= __uint_as_float(a[r][i] << 16);
            w[r][2 * i + 1] -= __uint_as_float(a[r][i] & 0xffff0000u);
          }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          mma_16816<false>(acc[nt], a[0][0], a[1][0], a[0][1], a[1][1], x[nt].x, x[nt].y);
          mma_16816<false>(acc[nt], a[0][2], a[1][2], a[0][3], a[1][3], x[nt].z, x[nt].w);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float* c = red + (warp * 8 * kNT + nt * 8 + 2 * t) * kGatePitch + g;
      c[0] = acc[nt][0];
      c[kGatePitch] = acc[nt][1];
      c[8] = acc[nt][2];
      c[kGatePitch + 8] = acc[nt][3];
    }
    consumer_sync();
    const int c = tid >> 4, r = tid & 15;
    if (c < p.T) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kConsumerWarps; ++i) v += red[(i * 8 * kNT + c) * kGatePitch + r];
      p.partial[((size_t)sp * p.T + c) * p.E + grp * kGateRows + r] = v;
    }
    consumer_sync();
  }
}

// The power of two that brings a block whose largest magnitude has the biased exponent eb below 2^15, and its
// inverse.  (Zero, tiny and infinite blocks included: eb is at least 15, and 255 leaves infinities and NaN.)
__device__ __forceinline__ float block_up(int eb) { return __uint_as_float((uint32_t)(268 - max(eb, 15)) << 23); }
__device__ __forceinline__ float block_down(int eb) { return __uint_as_float((uint32_t)(max(eb, 15) - 14) << 23); }

// x in f16 blocks of 32 with their scales (MXFP4), spread over the grid.
__device__ __forceinline__ void scale_tokens(const DecodeParams& p, int tid) {
  const int n = p.T * p.d / 8;   // a multiple of 4: the four threads of a block are all in
  for (int i = blockIdx.x * kConsumers + tid; i < n; i += gridDim.x * kConsumers) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.x) + i);
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(q[j] & 0x7fffu, (q[j] >> 16) & 0x7fffu));
    const uint32_t group = 0xfu << (threadIdx.x & 28);
    m = max(m, __shfl_xor_sync(group, m, 1));
    m = max(m, __shfl_xor_sync(group, m, 2));
    const int eb = (int)(m >> 7);
    const float up = block_up(eb);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 r = __floats2half2_rn(__uint_as_float(q[j] << 16) * up, __uint_as_float(q[j] & 0xffff0000u) * up);
      h[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
    reinterpret_cast<uint4*>(p.x16)[i] = make_uint4(h[0], h[1], h[2], h[3]);
    if ((i & 3) == 0) p.x_scale[i >> 2] = block_down(eb);
  }
}

// ------------------------------------------------------------------------------------------------
// phase 2: selection, one warp per token
// ------------------------------------------------------------------------------------------------
// Affinities with the accurate exponential and division: the selection compares these values.  The affinity
// of -inf is 0 in both, so lanes need no bounds and their experts' chains of instructions interleave.
__device__ __forceinline__ float affinity_softplus(float l) {
  return sqrtf(fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))));
}
__device__ __forceinline__ float affinity_sigmoid(float l) { return __fdiv_rn(1.f, 1.f + expf(-l)); }

// An unsigned key that orders as the float does; never 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return max((b & 0x80000000u) ? ~b : b | 0x80000000u, 1u);
}

// Lane l holds experts 128 q + 4 l + r as i = 4 q + r, ascending in i.
template <int PL>
__device__ __forceinline__ void select_experts(const DecodeParams& p, const float* bias, const float* offset, int* sel_e,
                                               float* sel_w, float* scores, int t, bool report, int lane) {
  auto expert = [&](int i) { return (i >> 2) * 128 + 4 * lane + (i & 3); };
  float sc[PL];
  uint32_t key[PL];
  // the partial logits of up to eight slices in one round of loads: under the weight stream a round takes
  // about 2 us
  constexpr int kRound = 32 / PL * 2;
#pragma unroll
  for (int i = 0; i < PL; ++i) sc[i] = 0.f;
  for (int s0 = 0; s0 < p.gate_splits; s0 += kRound) {
    float4 v[kRound][PL / 4];
#pragma unroll
    for (int s = 0; s < kRound; ++s)
#pragma unroll
      for (int q = 0; q < PL / 4; ++q) {
        v[s][q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 + s < p.gate_splits && expert(4 * q) < p.E)
          v[s][q] = __ldcg(reinterpret_cast<const float4*>(p.partial + ((size_t)(s0 + s) * p.T + t) * p.E + expert(4 * q)));
      }
#pragma unroll
    for (int s = 0; s < kRound; ++s)
#pragma unroll
      for (int q = 0; q < PL / 4; ++q) {
        sc[4 * q] += v[s][q].x;
        sc[4 * q + 1] += v[s][q].y;
        sc[4 * q + 2] += v[s][q].z;
        sc[4 * q + 3] += v[s][q].w;
      }
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = expert(i);
    sc[i] = e < p.E ? sc[i] + offset[e] : -INFINITY;
  }
  if (p.score_func == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, sc[i]);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      sc[i] = expert(i) < p.E ? expf(sc[i] - m) : 0.f;
      z += sc[i];
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int i = 0; i < PL; ++i) sc[i] = __fdiv_rn(sc[i], z);
  } else if (p.score_func == MOE_SCORE_SQRT_SOFTPLUS) {
#pragma unroll
    for (int i = 0; i < PL; ++i) sc[i] = affinity_softplus(sc[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) sc[i] = affinity_sigmoid(sc[i]);
  }

  int my_e = 0;          // lane j holds slot j's expert and unbiased score
  float my_s = 0.f;
  if (p.token_ids != nullptr) {
    int tok = p.token_ids[t];
    if (tok < 0 || tok >= p.vocab) {
      if (report && lane == 0) record_error(p.ew, MOE_ERR_DEVICE, tok);
      tok = tok < 0 ? 0 : p.vocab - 1;
    }
    if (lane < p.k) {
      my_e = p.tid2eid[(size_t)tok * p.k + lane];
      if (my_e < 0 || my_e >= p.E) {
        if (report) record_error(p.ew, MOE_ERR_DEVICE, my_e);
        my_e = my_e < 0 ? 0 : p.E - 1;
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (expert(i) < p.E) scores[expert(i)] = sc[i];
    __syncwarp();
    my_s = scores[my_e];
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = expert(i);
      const float b = e < p.E ? __fadd_rn(sc[i], bias[e]) : 0.f;
      if (e < p.E) scores[e] = b;
      key[i] = e < p.E ? order_key(b) : 0u;
    }
    __syncwarp();
    if (p.G > 1 && p.g < p.G) {
      // group scores: the sum of a group's two best biased scores (the best alone without a bias), by
      // L lanes per group; then the g best groups (equal scores: the lower group)
      int L = 32;
      while (L * p.G > 32) L >>= 1;
      const int grp = lane / L, per = p.E / p.G;
      float m1 = -INFINITY, m2 = -INFINITY;
      if (grp < p.G) {
        for (int i = lane % L; i < per; i += L) {
          const float b = scores[grp * per + i];
          m2 = fmaxf(m2, fminf(m1, b));
          m1 = fmaxf(m1, b);
        }
      }
      for (int o = 1; o < L; o <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
        const float n1 = fmaxf(m1, o1);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = n1;
      }
      const float gs = p.bias != nullptr ? __fadd_rn(m1, m2) : m1;
      int better = 0;
      for (int j = 0; j < p.G; ++j) {
        const float gj = __shfl_sync(0xffffffffu, gs, j * L);
        better += (gj > gs || (gj == gs && j < grp)) ? 1 : 0;
      }
      const uint32_t kept = __ballot_sync(0xffffffffu, grp < p.G && better < p.g);
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int e = expert(i);
        if (e < p.E && !((kept >> ((e / per) * L)) & 1u)) key[i] = 0u;
      }
    }
    // k rounds of a warp-wide maximum (equal scores: the lower expert)
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (key[i] > best) {
          best = key[i];
          at = expert(i);
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int e = __reduce_min_sync(0xffffffffu, top != 0u && best == top ? at : 0x7fffffff);
      const int ec = e < p.E ? e : 0;   // no candidate left (scores that are not numbers): stays in range
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (expert(i) == ec) {
          mine = sc[i];
          key[i] = 0u;
        }
      const float s = __shfl_sync(0xffffffffu, mine, (ec & 127) >> 2);
      if (lane == j) {
        my_e = ec;
        my_s = s;
      }
    }
  }
  float total = 0.f;
  for (int j = 0; j < p.k; ++j) total = __fadd_rn(total, __shfl_sync(0xffffffffu, my_s, j));
  if (lane < p.k) {
    float w = my_s;
    if (p.renorm) w = __fdiv_rn(w, total);
    w = __fmul_rn(w, p.route_scale);
    sel_e[t * p.k + lane] = my_e;
    sel_w[t * p.k + lane] = w;
  }
}

// The lists of active experts and their token rows, by the router warps.  Active expert 0 is the shared one
// with every token, the routed ones follow by index; an expert's rows are its tokens in order.  A token that
// names an expert twice (a table may) has one row there.  sm->mask is zero on entry and on exit.
template <typename Smem>
__device__ __forceinline__ void build_lists(const DecodeParams& p, Smem* sm, int rt, int lane) {
  const int S = p.T * p.k;
  for (int s = rt; s < S; s += kRouters) {
    const int e = sm->sel_e[s], t = s / p.k;
    int d = 0;
    for (int q = t * p.k; q < s; ++q) d |= sm->sel_e[q] == e;
    sm->dup[s] = d;
    atomicOr(&sm->mask[e], 1u << t);
  }
  router_sync();
  if (rt < 32) {
    // lane l: experts [l per, (l + 1) per): how many are active (high half) and their rows (low half)
    const int per = (p.E + 31) / 32, e0 = min(lane * per, p.E), e1 = min(e0 + per, p.E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
      const uint32_t m = sm->mask[e];
      mine += m != 0u ? 0x10000 + __popc(m) : 0;
    }
    int run = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) sm->n_listed = 1 + (run >> 16);
    run -= mine;
    for (int e = e0; e < e1; ++e) {
      const uint32_t m = sm->mask[e];
      if (m != 0u) {
        const int a = 1 + (run >> 16), off = p.T + (run & 0xffff);
        sm->act_e[a] = e;
        sm->act_n[a] = __popc(m);
        sm->act_off[a] = off;
        sm->off_of[e] = off;
        run += 0x10000 + __popc(m);
      }
    }
  }
  router_sync();
  for (int s = rt; s < S; s += kRouters) {
    const int e = sm->sel_e[s], t = s / p.k;
    const int row = sm->off_of[e] + __popc(sm->mask[e] & ((1u << t) - 1u));
    sm->row_of_slot[s] = row;
    if (!sm->dup[s]) {
      float w = 0.f;
      for (int q = t * p.k; q < (t + 1) * p.k; ++q)
        if (sm->sel_e[q] == e) w += sm->sel_w[q];
      sm->tok_of_row[row] = t;
      sm->row_w[row] = w;
    }
  }
  router_sync();
  for (int s = rt; s < S; s += kRouters) sm->mask[sm->sel_e[s]] = 0u;
  router_sync();
}

// The lists are there for all (unless a consumer that gave up has published empty ones).
template <typename Smem>
__device__ __forceinline__ void publish_lists(Smem* sm) {
  __threadfence_block();
  if (atomicCAS(&sm->n_act, 0, sm->n_listed) == 0) mbar_arrive(&sm->routed);
}

// The router warps: selection and lists, then the CTA's reports of finished up tiles.
//
// A round trip to L2 takes about 2 us under the weight stream, so up to two tokens are selected by every CTA
// for itself, one per warp, from the partial logits of the whole grid.  More tokens are dealt to the first
// CTAs, one each, and their choices read back after one more counter: 16 tokens 6 a warp took 34 us.
template <bool kFp4, typename Smem>
__device__ __forceinline__ void route(const DecodeParams& p, Smem* sm, int rw, int lane) {
  if (p.test_stall == kStallRouter) return;
  volatile int* abort = &sm->abort;
  const int rt = rw * 32 + lane, S = p.T * p.k;
  const bool dealt = p.T > kRouterWarps && (int)gridDim.x >= p.T;
  for (int e = rt; e < p.E; e += kRouters) {
    sm->bias[e] = p.bias != nullptr ? p.bias[e] : 0.f;
    sm->offset[e] = p.logit_offset != nullptr ? p.logit_offset[e] : 0.f;
  }
  router_sync();
  const bool report = dealt || blockIdx.x == 0;   // bad ids: once, by the CTA that selects the token
  auto select = [&](int t) {
    if (p.E <= 256) select_experts<8>(p, sm->bias, sm->offset, sm->sel_e, sm->sel_w, sm->scores[rw], t, report, lane);
    else select_experts<16>(p, sm->bias, sm->offset, sm->sel_e, sm->sel_w, sm->scores[rw], t, report, lane);
  };
  // The table names a hash-routed token's experts before there are logits: their weights are then needed by
  // the combine alone (unless h carries them).
  const bool early = p.token_ids != nullptr && !p.weight_in_expert;
  if (early) {
    for (int s = rt; s < S; s += kRouters) {
      const int tok = min(max(p.token_ids[s / p.k], 0), p.vocab - 1);   // bad ids are reported by the selection below
      sm->sel_e[s] = min(max(p.tid2eid[(size_t)tok * p.k + s % p.k], 0), p.E - 1);
      sm->sel_w[s] = 0.f;
    }
    router_sync();
    build_lists(p, sm, rt, lane);
    if (rt == 0) publish_lists(sm);
  }
  if (lane == 0) grid_wait(&p.gc->arrive[0], (int)gridDim.x, abort, p.ew, 404);
  __syncwarp();
  if (!dealt) {
    for (int t = rw; t < p.T; t += kRouterWarps) select(t);
  } else {
    if (rw == 0 && (int)blockIdx.x < p.T) {
      const int t = blockIdx.x;
      select(t);
      __syncwarp();
      if (lane < p.k) {
        p.route_e[t * p.k + lane] = sm->sel_e[t * p.k + lane];
        p.route_w[t * p.k + lane] = sm->sel_w[t * p.k + lane];
      }
      __syncwarp();
      if (lane == 0) red_release_add(&p.gc->arrive[3], 1);
    }
    router_sync();
    if (lane == 0) grid_wait(&p.gc->arrive[3], p.T, abort, p.ew, 410);
    __syncwarp();
    for (int s = rt; s < S; s += kRouters) {
      sm->sel_e[s] = *abort ? 0 : __ldcg(p.route_e + s);   // after an abort the scratch may hold anything
      sm->sel_w[s] = __ldcg(p.route_w + s);
    }
  }
  router_sync();
  if (!early) {
    build_lists(p, sm, rt, lane);
    if (rt == 0) publish_lists(sm);
  }
  if (rt == 0) mbar_arrive(&sm->weighted);
  if (blockIdx.x == 0) {
    for (int s = rt; s < S; s += kRouters) {
      if (p.weights_out != nullptr) p.weights_out[s] = sm->sel_w[s];
      if (p.indices_out != nullptr) p.indices_out[s] = sm->sel_e[s];
    }
    if (p.counts_out != nullptr)
      for (int e = rt; e < p.E; e += kRouters) {
        int c = 0;
        for (int s = 0; s < S; ++s) c += sm->sel_e[s] == e;
        p.counts_out[e] = c;
      }
  }
  // Reports of finished up tiles, kept off the consumers' path: a release at GPU scope waits for the writes
  // before it, 1 to 2 us under the stream.
  if (lane == 0) {   // a router warp for each group
    const int nb = p.I / Stage<kFp4>::kUp;
    const long long t0 = clock64();
    int seen = 0;   // n_listed: n_act is published by one of these lanes, for the others
    for (TileIter it(nb, (int)blockIdx.x * kGroups + rw, (int)gridDim.x * kGroups); it.a < sm->n_listed;) {
      // a tile's writers are all past the tile before it, so the count passes each tile's total in turn
      const int done = *(volatile int*)&sm->up_done[rw];
      int tiles = 0;
      for (; it.a < sm->n_listed && done >= seen + up_writers<kFp4>(sm->act_n[it.a]); it.next()) {
        if (tiles++ == 0) __threadfence();
        seen += up_writers<kFp4>(sm->act_n[it.a]);
        atomicAdd(&p.gc->ready[it.a], 1);
      }
      if (tiles > 0) {
        atomicAdd(&p.gc->arrive[1], tiles);
      } else {
        __nanosleep(100);
        if (*abort || clock64() - t0 > 2 * kWaitLimitCycles) break;
      }
    }
  }
}
static_assert(kRouterWarps == kGroups, "one reports for each group");

// ------------------------------------------------------------------------------------------------
// consumers: one stage into the warp's accumulators
// ------------------------------------------------------------------------------------------------
// The warp's 64 elements of a stage's token rows (rows g and g + 8 of the tile's): two blocks of 32, of which
// thread t holds 8 elements each; MXFP4: and the blocks' scales of the token columns 2t, 2t + 1 (+ 8).
template <bool kFp4, int kNT>
struct TokenFrags {
  uint4 v[kNT][2];
  float2 scale[kFp4 ? kNT : 1][2];   // .x, .y: the two blocks; of columns 2t and 2t + 1
};

// Four f16 pairs of the eight E2M1 codes of w.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

// Bits 7 of the bytes of `bad` are set where one of four block scales lies outside [2, 252]: s + 3 is then below
// 5 modulo 256 (a carry out of a byte comes from such a scale too; other bits are not defined).
__device__ __forceinline__ void note_scales(uint32_t s, uint32_t& bad) {
  const uint32_t t = s + 0x03030303u;
  bad |= (t - 0x05050505u) & ~t;
}
// Those clamped and reported.
__device__ __noinline__ uint32_t clamp_scales(uint32_t s4, ErrorWord* ew) {
  uint32_t r = 0u;
  for (int i = 0; i < 32; i += 8) {
    uint32_t s = (s4 >> i) & 0xFFu;
    if (s < 2u || s > 252u) {
      record_error(ew, MOE_ERR_DEVICE, 0x10000 + (int)s);
      s = s < 2u ? 2u : 252u;
    }
    r |= s << i;
  }
  return r;
}

// w: the warp's place in its group of eight, which takes elements [64 w, 64 w + 64) of the stage.
template <bool kFp4, bool kDown, int NT, int kNT>
__device__ __forceinline__ void consume_stage(uint32_t stage, int w, int lane, const TokenFrags<kFp4, kNT>& tok,
                                              float (&acc)[Stage<kFp4>::kRowTiles][kNT][4], ErrorWord* ew) {
  using S = Stage<kFp4>;
  const int g = lane >> 2, t = lane & 3;
  if constexpr (!kFp4) {
    const uint32_t wr = stage + w * S::kColBytes + g * 128;   // the warp's elements are column w
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const uint32_t at = wr + (((kb * 4 + t) ^ g) << 4);
      const uint4 lo = lds128(at), hi = lds128(at + S::kBlock);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = tok.v[nt][kb];
        mma_16816<false>(acc[0][nt], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
        mma_16816<false>(acc[0][nt], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
      }
    }
  } else {
    // row tile i: rows 8 i + g of both blocks (up), or rows 16 i + g and 16 i + 8 + g (down)
    constexpr int kHi = kDown ? 8 : S::kRows / 2;                 // from a low row to its high row, in scale rows
    constexpr uint32_t kHiBytes = kDown ? 8 * 128 : S::kBlock;
    uint32_t sc[S::kRowTiles], bad = 0u;
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i) {
      const uint32_t at = stage + S::kSOff + ((kDown ? 16 : 8) * i + g) * 16 + w * 2;
      sc[i] = lds16(at) | (lds16(at + kHi * 16) << 16);
      note_scales(sc[i], bad);
    }
    if ((bad & 0x80808080u) != 0u) {
#pragma unroll
      for (int i = 0; i < S::kRowTiles; ++i) sc[i] = clamp_scales(sc[i], ew);
    }
    const uint32_t col = stage + (w >> 2) * S::kColBytes + g * 128 + t * 4;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const uint32_t unit = ((2 * (w & 3) + kb) ^ g) << 4;
#pragma unroll
      for (int i = 0; i < S::kRowTiles; ++i) {
        const uint32_t at = col + unit + (kDown ? (i >> 1) * S::kBlock + (i & 1) * 16 * 128 : i * 8 * 128);
        uint32_t lo[4], hi[4];
        e2m1_to_f16(lds32(at), lo);
        e2m1_to_f16(lds32(at + kHiBytes), hi);
        const float f_lo = __uint_as_float((kb == 0 ? sc[i] << 23 : sc[i] << 15) & 0x7f800000u);
        const float f_hi = __uint_as_float((kb == 0 ? sc[i] << 7 : sc[i] >> 1) & 0x7f800000u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 b = tok.v[nt][kb];
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816<true>(part, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
          mma_16816<true>(part, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
          const float s0 = kb == 0 ? tok.scale[nt][0].x : tok.scale[nt][0].y;
          const float s1 = kb == 0 ? tok.scale[nt][1].x : tok.scale[nt][1].y;
          acc[i][nt][0] = fmaf(part[0] * s0, f_lo, acc[i][nt][0]);
          acc[i][nt][1] = fmaf(part[1] * s1, f_lo, acc[i][nt][1]);
          acc[i][nt][2] = fmaf(part[2] * s0, f_hi, acc[i][nt][2]);
          acc[i][nt][3] = fmaf(part[3] * s1, f_hi, acc[i][nt][3]);
        }
      }
    }
  }
}

// As consume_stage for bf16, with two sets of token fragments: each weight fragment meets both.
template <int kNT, typename Frags>
__device__ __forceinline__ void consume_stage_two(uint32_t stage, int w, int lane, const Frags& first, const Frags& second,
                                                  float (&acc)[kNT][4], float (&acc2)[kNT][4]) {
  using S = Stage<false>;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t wr = stage + w * S::kColBytes + g * 128;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const uint32_t at = wr + (((kb * 4 + t) ^ g) << 4);
    const uint4 lo = lds128(at), hi = lds128(at + S::kBlock);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const uint4 b = first.v[nt][kb], c = second.v[nt][kb];
      mma_16816<false>(acc[nt], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
      mma_16816<false>(acc[nt], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
      mma_16816<false>(acc2[nt], lo.x, hi.x, lo.y, hi.y, c.x, c.y);
      mma_16816<false>(acc2[nt], lo.z, hi.z, lo.w, hi.w, c.z, c.w);
    }
  }
}

// The warp's accumulators of a tile into the exchange buffer, [warp][token column][row].
template <bool kFp4, int kNT>
__device__ __forceinline__ void put_partials(float* red, int warp, int lane,
                                             const float (&acc)[Stage<kFp4>::kRowTiles][kNT][4], int nt_used) {
  using S = Stage<kFp4>;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    if (nt >= nt_used) break;
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i) {
      float* c = red + (warp * 8 * kNT + nt * 8 + 2 * t) * S::kRedPitch + i * 16 + g;
      c[0] = acc[i][nt][0];
      c[S::kRedPitch] = acc[i][nt][1];
      c[8] = acc[i][nt][2];
      c[S::kRedPitch + 8] = acc[i][nt][3];
    }
  }
}
template <bool kFp4, int kNT>
__device__ __forceinline__ float sum_partials(const float* red, int col, int row) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kGroupWarps; ++w) v += red[(w * 8 * kNT + col) * Stage<kFp4>::kRedPitch + row];
  return v;
}

// ------------------------------------------------------------------------------------------------
// a group's weight stream: TMA copies by lane 0 and, for MXFP4, the scales by cp.async of all 32 lanes (then the
// full barriers count their 32 arrivals too)
// ------------------------------------------------------------------------------------------------
template <bool kFp4, typename Smem>
__device__ __forceinline__ void produce(const DecodeParams& p, const CUtensorMap* map_w1, const CUtensorMap* map_w3,
                                        const CUtensorMap* map_w2, Smem* sm, uint8_t* ring, int grp, int lane) {
  using S = Stage<kFp4>;
  const int self = (int)blockIdx.x * kGroups + grp, all = (int)gridDim.x * kGroups;
  uint64_t *full = sm->full[grp], *empty = sm->empty[grp];
  if (p.test_stall == kStallCopies) return;
  volatile int* abort = &sm->abort;
  constexpr int kColElems = S::kChunk / S::kCols;
  const int most = p.test_stall == kStallLater || (p.test_stall == kStallOneCta && blockIdx.x == 0) ? 5 : 0x7fffffff;
  RingPos pos;
  int issued = 0;
  bool ok = true, routed = false;
  // A free stage to fill: none once a wait has been given up.
  auto free_stage = [&]() {
    int ok = 0;
    if (!kFp4 || lane == 0) ok = mbar_wait(&empty[pos.slot], pos.phase ^ 1, abort, p.ew, 401) && !*abort;
    return (kFp4 ? __shfl_sync(0xffffffffu, ok, 0) : ok) != 0;
  };
  auto tile = [&](bool down, int e, int blk) {
    const int K = down ? p.I : p.d;
    const int row = down ? e * p.d + blk * S::kRows : e * p.I + blk * S::kUp;
    const CUtensorMap *m0 = down ? map_w2 : map_w1, *m1 = down ? map_w2 : map_w3;
    const int row1 = down ? row + S::kRows / 2 : row;
    for (int k0 = 0; k0 < K; k0 += S::kChunk) {
      if (issued == most || !free_stage()) return false;
      uint64_t* bar = &full[pos.slot];
      uint8_t* dst = ring + pos.slot * S::kBytes;
      if (kFp4) {
        const uint8_t* s0 = down ? p.w2s : p.w1s;
        const uint8_t* s1 = down ? p.w2s : p.w3s;
        cp_async16(smem_u32(dst + S::kSOff + lane * 16), s0 + ((size_t)(row + lane) * K + k0) / 32);
        cp_async16(smem_u32(dst + S::kSOff + (32 + lane) * 16), s1 + ((size_t)(row1 + lane) * K + k0) / 32);
        cp_async_arrive(bar);
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, 2 * S::kBlock);   // whole boxes: what lies past K is filled with zeros
        tma_load_3d(dst, m0, bar, 0, row, k0 / kColElems);
        tma_load_3d(dst + S::kBlock, m1, bar, 0, row1, k0 / kColElems);
      }
      ++issued;
      pos.step(1, p.stages);
    }
    return true;
  };
  const int nb1 = p.I / S::kUp, nb2 = p.d / S::kRows;
  for (TileIter it(nb1, self, all); ok; it.next()) {
    if (it.a > 0 && !routed) {
      ok = kFp4 ? mbar_wait_warp(&sm->routed, 0, abort, p.ew, 403) : mbar_wait(&sm->routed, 0, abort, p.ew, 403);
      routed = true;
      if (!ok) break;
    }
    if (routed && it.a >= sm->n_act) break;
    ok = tile(false, it.a == 0 ? p.E : sm->act_e[it.a], it.blk);
  }
  if (ok)
    for (TileIter it = down_tiles(p, sm->n_act, nb1, nb2, self, all); ok && it.a < sm->n_act; it.next())
      ok = tile(true, it.a == 0 ? p.E : sm->act_e[it.a], it.blk);
  if (lane == 0) sm->issued[grp] = issued;
}

// After an abort: every copy that the group's producer warp has started lands before the CTA leaves.
template <typename Smem>
__device__ __forceinline__ void drain(Smem* sm, int stages, int grp, int lane) {
  cp_async_wait_all();
  if (lane == 0) {
    const int issued = sm->issued[grp];
    for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
      mbar_wait(&sm->full[grp][i % stages], (i / stages) & 1, nullptr, nullptr, 0, 200000000LL);
  }
  __syncwarp();
}

// ------------------------------------------------------------------------------------------------
// the kernel
// ------------------------------------------------------------------------------------------------
// kNT: column tiles of eight tokens (1 for batches of at most 8, whose fragments then take half the registers).
template <bool kFp4, int kNT>
__global__ void __launch_bounds__(kDecThreads, 1)
    layer_decode_kernel(const __grid_constant__ CUtensorMap map_w1, const __grid_constant__ CUtensorMap map_w3,
                        const __grid_constant__ CUtensorMap map_w2, const __grid_constant__ DecodeParams p) {
  using S = Stage<kFp4>;
  using Smem = DecodeSmem<kFp4, kNT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem* sm = reinterpret_cast<Smem*>(ring + kGroups * p.stages * S::kBytes);
  static_assert(offsetof(Smem, n_act) == offsetof(Smem, abort) + sizeof(int), "where stage_wait_slow finds it");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  if (tid < kGroups * p.stages) {
    mbar_init(&sm->full[tid / p.stages][tid % p.stages], kFp4 ? 1 + 32 : 1);
    mbar_init(&sm->empty[tid / p.stages][tid % p.stages], kGroupWarps);
    fence_barrier_init();
  }
  if (tid == kConsumers) {
    mbar_init(&sm->routed, 1);
    mbar_init(&sm->weighted, 1);
    sm->abort = 0;
    sm->n_act = 0;
    for (int i = 0; i < kGroups; ++i) sm->up_done[i] = sm->issued[i] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_w1);
    tma_prefetch_desc(&map_w3);
    tma_prefetch_desc(&map_w2);
  }
  for (int i = tid; i < kMaxE; i += kDecThreads) {
    sm->mask[i] = 0u;
    if (i < kMaxS) sm->sel_e[i] = 0;
    if (i < p.T) {
      sm->tok_of_row[i] = i;
      sm->row_w[i] = 1.f;
    }
  }
  if (tid == 0) {
    sm->act_e[0] = p.E;
    sm->act_off[0] = 0;
    sm->act_n[0] = p.T;
  }
  __syncthreads();

  // Every wait below is bounded.  After one was given up the consumers go on over whatever lies in the ring, so
  // that they keep meeting at the same barriers; what they free then may still be under way, so the producers fill
  // nothing any more once `abort` is set (a consumer that gave up has seen it set before it frees the stage).
  // The lists that they go by are published once, by the router or (empty) by the first that gave up waiting for
  // them.  The combine is left out after an abort, and the producers see their copies land.
  volatile int* abort = &sm->abort;
  const int G = (int)gridDim.x;
  if (warp >= kConsumerWarps && warp < kConsumerWarps + kGroups) {
    const int grp = warp - kConsumerWarps;
    if (kFp4 || lane == 0) produce<kFp4>(p, &map_w1, &map_w3, &map_w2, sm, ring + grp * p.stages * S::kBytes, grp, lane);
  } else if (warp >= kConsumerWarps + kGroups) {
    route<kFp4>(p, sm, warp - kConsumerWarps - kGroups, lane);
    if (lane == 0) red_release_add(&p.gc->done, 1);
  } else {
    gate_partials<kNT>(p, sm->red[0][0], warp, lane);
    if (kFp4) scale_tokens(p, tid);
    consumer_sync();
    if (tid == 0) {
      red_release_add(&p.gc->arrive[0], 1);
      if (kFp4) grid_wait(&p.gc->arrive[0], G, abort, p.ew, 408);
    }
    if (kFp4) consumer_sync();   // x16 is written

    RingPos pos;                 // the next stage
    int buf = 0;
    bool routed = false;
    const int grp = warp >> 3, w8 = warp & 7, g = lane >> 2, t = lane & 3, gtid = tid & (kGroupThreads - 1);
    const int self = (int)blockIdx.x * kGroups + grp, all = G * kGroups;
    const uint32_t ring_addr = smem_u32(ring + grp * p.stages * S::kBytes);
    uint64_t *full = sm->full[grp], *empty = sm->empty[grp];
    const int nb1 = p.I / S::kUp, nb2 = p.d / S::kRows;
    auto run_phase = [&](auto down_tag, TileIter it) {
      constexpr bool kDown = decltype(down_tag)::value, kTwo = S::red_bufs(kNT) == 2;
      const int K = kDown ? p.I : p.d, ns = (K + S::kChunk - 1) / S::kChunk;
      const uint16_t* rows[kNT];               // the tile's token rows, bf16 or (MXFP4) f16, at this warp's part
      [[maybe_unused]] const float* scales[kFp4 ? kNT : 1][2];
      // Fragments of the next kSets stages, each set loaded again as soon as its stage is done.  Two where the
      // registers hold them: an L2 round trip under the stream is longer than a stage.
      constexpr int kSets = kFp4 ? 1 : 2;
      TokenFrags<kFp4, kNT> frags[kSets];
      // bf16 experts' h is held in two bf16 parts, 16 bits together.  The columns that an expert's few tokens leave
      // free take the second parts: of up to 4 tokens in columns 4 to 7; of up to 8 tokens, with two column tiles,
      // in the second.  More tokens need both sets of fragments for a stage: the other set holds the second
      // parts (one column tile), or tokens 8 to 15 with theirs.  The sums of the two parts are kept apart and
      // added at a tile's end: a token's result does not depend on how many others its expert has.
      constexpr bool kParts = kDown && !kFp4;
      int cols = 0;   // tokens of the tile entered
      int ready_a = -1;
      bool all_ready = !kDown;
      // Whether the iterator stands on a tile (waits for the lists at the first routed one).
      auto live = [&]() {
        if (it.a > 0 && !routed) {
          stage_wait(&sm->routed, 0, abort, p.ew, kListsSite);
          routed = true;
        }
        return it.a == 0 || it.a < sm->n_act;
      };
      auto enter = [&]() {
        if (!all_ready && it.a != ready_a) {   // all of this expert's h is written?
          int done = 0;
          if (lane == 0) {
            done = ld_acquire(&p.gc->arrive[1]) >= sm->n_act * nb1;
            if (!done) grid_wait(&p.gc->ready[it.a], nb1, abort, p.ew, 402);
          }
          all_ready = __shfl_sync(0xffffffffu, done, 0) != 0;
          ready_a = it.a;
        }
        const int n = sm->act_n[it.a], r0 = sm->act_off[it.a];
        const uint16_t* base = kDown ? p.h : kFp4 ? p.x16 : reinterpret_cast<const uint16_t*>(p.x);
        auto place = [&](int c) { return kDown ? r0 + c : sm->tok_of_row[r0 + c]; };
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          if constexpr (kParts) {   // one pointer: an expert's rows of h follow each other
            const int col = n <= 4 ? g & 3 : g;
            rows[0] = col < n ? base + (size_t)(r0 + col) * K + (n <= 4 && g >= 4 ? p.h_lo : 0) + w8 * 64 + t * 8 : nullptr;
            cols = n;
            break;
          }
          rows[nt] = g + 8 * nt < n ? base + (size_t)place(g + 8 * nt) * K + w8 * 64 + t * 8 : nullptr;
          if constexpr (kFp4) {
            const float* sbase = kDown ? p.h_scale : p.x_scale;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 2 * t + c + 8 * nt;
              scales[nt][c] = col < n ? sbase + (size_t)place(col) * (K / 32) + w8 * 2 : nullptr;
            }
          }
        }
      };
      // those of stage s of the tile entered (zeros past its end); h in parts: or its other set
      auto fetch = [&](int s, TokenFrags<kFp4, kNT>& nxt, bool other = false) {
        const bool in = s * S::kChunk + w8 * 64 < K;
        if constexpr (kParts) {
          const uint16_t* at = rows[0] + s * S::kChunk;
          if (other) at += kNT == 1 ? p.h_lo : 8 * K;
          const bool have = in && rows[0] != nullptr && (kNT == 1 || !other || g + 8 < cols);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)   // written during this kernel: read from L2
              nxt.v[nt][kb] = have && (nt == 0 || cols > 4)
                                  ? __ldcg(reinterpret_cast<const uint4*>(at + (nt == 0 ? 0 : p.h_lo)) + kb * 4)
                                  : make_uint4(0u, 0u, 0u, 0u);
        } else {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            nxt.v[nt][0] = nxt.v[nt][1] = make_uint4(0u, 0u, 0u, 0u);
            if (in && rows[nt] != nullptr) {
              const uint4* at = reinterpret_cast<const uint4*>(rows[nt] + s * S::kChunk);
#pragma unroll
              for (int kb = 0; kb < 2; ++kb)   // written during this kernel, except x itself: read from L2
                nxt.v[nt][kb] = kDown || kFp4 ? __ldcg(at + kb * 4) : __ldg(at + kb * 4);
            }
            if constexpr (kFp4) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                nxt.scale[nt][c] = in && scales[nt][c] != nullptr
                                       ? __ldcg(reinterpret_cast<const float2*>(scales[nt][c] + s * (S::kChunk / 32)))
                                       : make_float2(0.f, 0.f);
            }
          }
        }
      };
      auto fetch_first = [&]() {
        fetch(0, frags[0]);
        const bool both = kParts && cols > 4 * kNT;
        if (kSets == 2) fetch(both ? 0 : 1, frags[kSets - 1], both);
      };
      bool more = live();
      if (more) {
        enter();
        fetch_first();
      }
      while (more) {
        const int n = sm->act_n[it.a], r0 = sm->act_off[it.a], a = it.a, blk = it.blk;
        float acc[S::kRowTiles][kNT][4] = {};
        auto one_stage = [&](int s, TokenFrags<kFp4, kNT>& tok) {
          stage_wait(&full[pos.slot], pos.phase, abort, p.ew, kDown ? 406 : 405);
          if (kFp4 || s * S::kChunk + w8 * 64 < K) {
            const uint32_t stage = ring_addr + pos.slot * S::kBytes;
            if (kNT == 1 || n <= (kParts ? 4 : 8)) consume_stage<kFp4, kDown, 1, kNT>(stage, w8, lane, tok, acc, p.ew);
            else consume_stage<kFp4, kDown, kNT, kNT>(stage, w8, lane, tok, acc, p.ew);
          }
          if (s + kSets < ns) fetch(s + kSets, tok);
          mbar_arrive_after_reads(&empty[pos.slot]);
          pos.step(1, p.stages);
        };
        if (!kParts || n <= 4 * kNT) {
          for (int s = 0; s < ns; s += kSets) {
            one_stage(s, frags[0]);
            if (kSets == 2 && s + 1 < ns) one_stage(s + 1, frags[kSets - 1]);
          }
          if constexpr (kParts) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[0][0][i] += n <= 4 ? __shfl_xor_sync(0xffffffffu, acc[0][0][i], 2) : acc[0][kNT - 1][i];
          }
        } else if constexpr (kParts) {
          float acc2[kNT][4] = {};
          for (int s = 0; s < ns; ++s) {
            stage_wait(&full[pos.slot], pos.phase, abort, p.ew, 406);
            if (s * S::kChunk + w8 * 64 < K)
              consume_stage_two<kNT>(ring_addr + pos.slot * S::kBytes, w8, lane, frags[0], frags[kSets - 1], acc[0], acc2);
            if (s + 1 < ns) {
              fetch(s + 1, frags[0]);
              fetch(s + 1, frags[kSets - 1], true);
            }
            mbar_arrive_after_reads(&empty[pos.slot]);
            pos.step(1, p.stages);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[0][0][i] += kNT == 1 ? acc2[0][i] : acc[0][kNT - 1][i];
            if (kNT == 2) acc[0][kNT - 1][i] = acc2[0][i] + acc2[kNT - 1][i];
          }
        }
        // the next tile's first fragments are under way while this one is added up
        it.next();
        more = live();
        if (more) {
          enter();
          fetch_first();
        }
        float* red = sm->red[grp][buf];
        if (kTwo) buf ^= 1;   // the barrier of the next tile keeps its writes behind this tile's reads
        put_partials<kFp4, kNT>(red, w8, lane, acc, n <= 8 ? 1 : 2);
        group_sync(grp);
        if constexpr (kDown) {
          for (int i = gtid; i < n * S::kRows; i += kGroupThreads) {
            const int c = i / S::kRows, r = i % S::kRows;
            p.out[(size_t)(r0 + c) * p.d + blk * S::kRows + r] = sum_partials<kFp4, kNT>(red, c, r);
          }
        } else {
          // feature f of token c: gate and value sums, eight rows apart in their row tile
          const int f = gtid % S::kUp;
          for (int c = gtid / S::kUp; c < n; c += kGroupThreads / S::kUp) {
            const int r = (f >> 3) * 16 + (f & 7);
            const float w = p.weight_in_expert && a > 0 ? sm->row_w[r0 + c] : 1.f;
            const float h =
                swiglu(sum_partials<kFp4, kNT>(red, c, r), sum_partials<kFp4, kNT>(red, c, r + 8), p.swiglu_limit, w);
            uint16_t* dst = p.h + (size_t)(r0 + c) * p.I + blk * S::kUp + f;
            if constexpr (kFp4) {   // a warp holds one token's block of 32: its scale, then f16
              const int eb = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu) >> 23);
              const __half v = __float2half_rn(h * block_up(eb));
              *dst = *reinterpret_cast<const uint16_t*>(&v);
              if (lane == 0) p.h_scale[(size_t)(r0 + c) * (p.I / 32) + blk] = block_down(eb);
            } else {
              const __nv_bfloat16 v = __float2bfloat16_rn(h);
              *dst = *reinterpret_cast<const uint16_t*>(&v);
              const float rest = h - __bfloat162float(v);   // NaN for an infinite h, whose first part says enough
              const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
              dst[p.h_lo] = *reinterpret_cast<const uint16_t*>(&lo);
            }
          }
          // the router warps report the tile once all its writers are here
          if (w8 < up_writers<kFp4>(n)) {
            __threadfence_block();
            __syncwarp();
            if (lane == 0) atomicAdd(&sm->up_done[grp], 1);
          }
        }
        if (!kTwo) group_sync(grp);
      }
    };
    run_phase(std::false_type{}, TileIter(nb1, self, all));
    run_phase(std::true_type{}, down_tiles(p, sm->n_act, nb1, nb2, self, all));
    consumer_sync();
    if (tid == 0) {   // after an abort too: the other CTAs are not kept waiting
      red_release_add(&p.gc->arrive[2], 1);
      grid_wait(&p.gc->arrive[2], G, abort, p.ew, 407);
    }
    const bool weighted = mbar_wait(&sm->weighted, 0, abort, p.ew, 411);
    consumer_sync();

    // ---------------- combine, slot order then the shared expert ----------------
    const int d4 = p.d / 4;
    for (int i = weighted && !*abort ? blockIdx.x * kConsumers + tid : p.T * d4; i < p.T * d4; i += G * kConsumers) {
      const int t = i / d4, f = (i - t * d4) * 4;
      float4 v[kMaxRouteTopk];
#pragma unroll
      for (int j = 0; j < kMaxRouteTopk; ++j)
        if (j < p.k) v[j] = __ldcg(reinterpret_cast<const float4*>(p.out + (size_t)sm->row_of_slot[t * p.k + j] * p.d + f));
      const float4 sh = __ldcg(reinterpret_cast<const float4*>(p.out + (size_t)t * p.d + f));
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kMaxRouteTopk; ++j)
        if (j < p.k) {
          const int s = t * p.k + j;
          if (p.weight_in_expert && sm->dup[s]) continue;   // its weight is in the first slot's row
          const float w = p.weight_in_expert ? 1.f : sm->sel_w[s];
          y.x = fmaf(w, v[j].x, y.x);
          y.y = fmaf(w, v[j].y, y.y);
          y.z = fmaf(w, v[j].z, y.z);
          y.w = fmaf(w, v[j].w, y.w);
        }
      *reinterpret_cast<uint2*>(p.y + (size_t)t * p.d + f) =
          make_uint2(bf16x2_bits(y.x + sh.x, y.y + sh.y), bf16x2_bits(y.z + sh.z, y.w + sh.w));
    }
  }
  // The last CTA to get here leaves the grid's counters at zero.  Nobody waits on them any more, but a tile's
  // report that nobody waited for (it is passed over once the total is there) must not land behind the zeros.
  // So the lanes that report have arrived on `done` themselves, by a release behind their reports, which the last
  // CTA's arrival acquires; the other counters' sums it has waited for.
  __syncwarp();
  __syncthreads();
  if (*abort && warp >= kConsumerWarps && warp < kConsumerWarps + kGroups)
    drain(sm, p.stages, warp - kConsumerWarps, lane);
  if (tid == 0) {
    if (*abort) __threadfence();   // it may not have waited
    sm->last = atom_acquire_add(&p.gc->done, 1) == (1 + kRouterWarps) * G - 1;
  }
  __syncthreads();
  if (sm->last) {
    if (tid < kMaxAct) p.gc->ready[tid] = 0;
    if (tid < 4) p.gc->arrive[tid] = 0;
    if (tid == 4) p.gc->done = 0;
  }
}

}  // namespace

int decode_gate_splits(int E, int d) {
  // at most one unit of 16 router rows per SM of a B200, at least 128 elements of k each, and no more slices
  // than the selection reads at once
  return std::max(1, std::min({d / 128, 148 / (E / kGateRows), 8}));
}

cudaError_t launch_layer_decode(const CUtensorMap& w1, const CUtensorMap& w3, const CUtensorMap& w2, DecodeParams p,
                                bool fp4, int num_sms, cudaStream_t stream) {
  const size_t smem = 227 * 1024;
  const size_t stage = fp4 ? Stage<true>::kBytes : Stage<false>::kBytes;
  const size_t fixed = fp4 ? (p.T <= 8 ? sizeof(DecodeSmem<true, 1>) : sizeof(DecodeSmem<true, 2>))
                           : (p.T <= 8 ? sizeof(DecodeSmem<false, 1>) : sizeof(DecodeSmem<false, 2>));
  p.stages = (int)std::min<size_t>(kMaxStages, (smem - 1024 - fixed) / stage / kGroups);   // of each group's ring
  auto kernel = fp4 ? (p.T <= 8 ? layer_decode_kernel<true, 1> : layer_decode_kernel<true, 2>)
                    : (p.T <= 8 ? layer_decode_kernel<false, 1> : layer_decode_kernel<false, 2>);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  // no more CTAs than any phase has work for: small layers pay for each arrival at the barriers
  const long tiles = (long)(std::min(p.T * p.k, p.E) + 1) * std::max(p.I / (fp4 ? 32 : 8), p.d / (fp4 ? 64 : 16));
  const int units = p.E / kGateRows * p.gate_splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long>(num_sms, std::max<long>(tiles, units)));
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, w1, w3, w2, p);
}

}  // namespace moe
