// The whole MoE layer for a few tokens (decode batches of at most 16) in one launch.
//
//   l = x . Wg^T (+ offset), s = affinity(l), experts = group-limited top-k of s + bias (or the token-id
//   table's row), w = s / sum(s) * scale;  h_e = silu(x w1_e^T) * (x w3_e^T);  y = sum_j w_j h w2^T + shared.
//
// What bounds it: the weights of the chosen experts, read once -- every weight meets one to sixteen tokens,
// far below the flops per byte at which the tensor cores would matter.  So the kernel is a weight stream:
//
// * one CTA per SM, all resident at once (cooperative launch), 17 warps: one producer thread keeps TMA copies
//   of 8 rows x 1 KB in flight into a ring of about 180 KB of shared memory, sixteen consumer warps compute.
//   At 44 bytes/ns per SM the ring holds 4 us of the stream, more than the memory latency and more than a
//   grid barrier, so the stream does not stop between the phases: the shared expert's first weights are
//   loaded while the gate is computed, and the down projection's while the grid finishes the up projection.
//   Copies of single rows (1 KB) cost about 65 ns each whoever issues them and held the stream at 2 TB/s.
// * the products run on mma.sync m16n8k16 with the weight rows as the 16-row operand and the tokens as the
//   8 columns: at most two column tiles, so each weight is read from shared memory once.  The reduction
//   index is permuted alike for both operands (thread t of a quad holds 8 consecutive elements), so that
//   a weight fragment is one conflict-free 16-byte shared load from TMA's 128-byte swizzle and a token
//   fragment one 16-byte load from global memory (L1 or L2; loaded a stage ahead), whatever the token's row.
//   Eight warps split a stage along k, the two groups of eight take alternate stages; the fp32 accumulators
//   of a tile are added through shared memory in warp order: nothing depends on scheduling.
// * an up-projection tile is 8 features: rows 0-7 of the MMA are w1's, rows 8-15 w3's, so gate and value of
//   a feature meet in one accumulator tile.  A down-projection tile is 16 output features of one expert.
// * four phases between three grid barriers: partial router logits (K split over the CTAs), then every CTA
//   selects the experts of all tokens for itself (a few KB from L2; cheaper than another barrier), up
//   projections into h (bf16 in the workspace), down projections into fp32 rows, combine in slot order.
//
// MXFP4 weights: the packed codes and their scales are what travels.  A code's four bits become bf16 by
// placing sign, exponent and mantissa bits (E2M1 is bf16's format with fewer bits, off by 2^126) and one
// exact multiply; the block's UE8M0 scale multiplies the fp32 accumulators of its 32 elements, so the
// weights are exact and the activations keep their bf16 values.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kConsumerWarps = 16;   // two groups of eight taking alternate stages
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kDecThreads = kConsumers + 32;
constexpr int kMaxStages = 24;
constexpr int kMaxT = kDecodeMaxTokens;
constexpr int kMaxS = kMaxT * kMaxRouteTopk;
constexpr int kMaxAct = kMaxS + 1;  // active experts: the shared one and at most one per slot
constexpr int kRedPitch = 20;       // floats per token column of the warp-partial exchange (bank = 8 t + g)
constexpr int kRedFloats = kConsumerWarps * kMaxT * kRedPitch;
constexpr int kGateRows = 16;       // router rows per unit of the logit phase
static_assert(2 * kRedFloats >= kConsumerWarps * 512, "the selection's scores share the exchange buffer");
static_assert(kMaxT <= 16, "two column tiles of eight tokens");

struct DecodeSmem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t routed;                  // the lists below are complete
  int abort;
  int n_act;                        // active experts, the shared one first
  int sel_e[kMaxS];
  float sel_w[kMaxS];
  int dup[kMaxS];                   // the token already chose this expert in an earlier slot
  int first[kMaxS], cnt[kMaxS];     // no earlier slot has the expert; its distinct tokens
  int row_of_slot[kMaxS];
  int tok_of_row[kMaxS + kMaxT];
  float row_w[kMaxS + kMaxT];
  int act_e[kMaxAct], act_off[kMaxAct], act_n[kMaxAct];
  alignas(16) float red[2][kRedFloats];
};

// The consumer warps' barrier.  It takes whole warps, so lanes that waited on their own rejoin first.
__device__ __forceinline__ void consumer_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, 512;" ::: "memory");
}
static_assert(kConsumers == 512, "the named barrier's thread count");

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_add(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// 16 bytes global -> shared past L1, and this lane's arrival on a barrier once its copies so far landed.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits until `*counter` reaches `target` (every CTA of the grid arrived).  Bounded as mbar_wait is.
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

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// ------------------------------------------------------------------------------------------------
// stage layout
// ------------------------------------------------------------------------------------------------
// A stage holds kChunk elements of k of 16 weight rows: two blocks of 8 rows, each as TMA writes a box of
// 128 bytes x 8 rows x kBoxes in the 128-byte swizzle -- the 16-byte unit u of row r of box b lies at
// b * 1024 + r * 128 + ((u ^ r) << 4) -- and, for MXFP4, the rows' scales.
template <bool kFp4>
struct Stage {
  static constexpr int kChunk = kFp4 ? 1024 : 512;
  static constexpr int kBoxes = kFp4 ? 4 : 8;                  // of 256 codes or 64 bf16
  static constexpr int kBlock = kBoxes * 1024;
  static constexpr int kSPitch = kFp4 ? 48 : 0;                // scale rows (32 bytes)
  static constexpr int kSOff = 2 * kBlock;
  static constexpr int kBytes = (kSOff + 16 * kSPitch + 1023) & ~1023;
};

struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void step(int by, int stages) {
    for (slot += by; slot >= stages; slot -= stages) phase ^= 1;
  }
};

// Tile j of a phase as (active expert, block of rows), stepped by the grid without a division.
struct TileIter {
  int j, a, blk, step_a, step_b, nb;
  __device__ TileIter(int nb_) : j(blockIdx.x), a(j / nb_), blk(j % nb_), step_a(gridDim.x / nb_), step_b(gridDim.x % nb_), nb(nb_) {}
  __device__ void next() {
    j += gridDim.x;
    a += step_a;
    blk += step_b;
    if (blk >= nb) {
      blk -= nb;
      ++a;
    }
  }
};

// ------------------------------------------------------------------------------------------------
// phase 1: partial router logits
// ------------------------------------------------------------------------------------------------
// Sums each of the N values over the warp: halves of the array are exchanged until one value is left
// per lane (N - 1 shuffles for N <= 32 and a few more), so lane l ends with the sums of values
// [first, first + max(1, N / 32)).
template <int N>
__device__ __forceinline__ int reduce_transposed(float (&v)[N], int lane) {
  int first = 0;
  int cnt = N;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (cnt > 1) {
      const int half = cnt / 2;
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < half) {
          const float send = up ? v[i] : v[i + half];
          const float keep = up ? v[i + half] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      }
      first += up ? half : 0;
      cnt = half;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    }
  }
  return first;
}

// Unit u: 16 router rows x one slice of k.  Four warps take 4 rows each, on each quarter of the slice.
// Tokens t0 to t0 + TT - 1.
template <int TT>
__device__ __forceinline__ void gate_partials(const DecodeParams& p, int t0, float* red, int warp, int lane) {
  const int groups = p.E / kGateRows, units = groups * p.gate_splits;
  const int nb = p.d / 128;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int grp = u % groups, sp = u / groups;
    const int rsub = warp & 3, ksub = warp >> 2;
    const int q0 = sp * nb / p.gate_splits, q1 = (sp + 1) * nb / p.gate_splits;
    const int b0 = q0 + ((q1 - q0) * ksub >> 2), b1 = q0 + ((q1 - q0) * (ksub + 1) >> 2);
    const int e0 = grp * kGateRows + rsub * 4;
    float acc[4 * TT];
#pragma unroll
    for (int i = 0; i < 4 * TT; ++i) acc[i] = 0.f;
#pragma unroll 2
    for (int b = b0; b < b1; ++b) {
      const int k = b * 128 + lane * 4;
      float4 w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r] = __ldg(reinterpret_cast<const float4*>(p.w_gate + (size_t)(e0 + r) * p.d + k));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t0 + t < p.T) {
          const uint2 xv = __ldg(reinterpret_cast<const uint2*>(p.x + (size_t)(t0 + t) * p.d + k));
          const float x0 = __uint_as_float(xv.x << 16), x1 = __uint_as_float(xv.x & 0xffff0000u);
          const float x2 = __uint_as_float(xv.y << 16), x3 = __uint_as_float(xv.y & 0xffff0000u);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float a = acc[t * 4 + r];
            a = fmaf(w[r].x, x0, a);
            a = fmaf(w[r].y, x1, a);
            a = fmaf(w[r].z, x2, a);
            acc[t * 4 + r] = fmaf(w[r].w, x3, a);
          }
        }
      }
    }
    const int first = reduce_transposed<4 * TT>(acc, lane);
    constexpr int kPer = 4 * TT > 32 ? 4 * TT / 32 : 1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) red[warp * 64 + first + i] = acc[i];   // lanes with equal `first` agree
    consumer_sync();
    const int tid = warp * 32 + lane;
    if (tid < kGateRows * TT) {
      const int t = tid / kGateRows, row = tid % kGateRows;
      if (t0 + t < p.T) {
        const int at = (row >> 2) * 64 + t * 4 + (row & 3);
        p.partial[((size_t)sp * p.T + t0 + t) * p.E + grp * kGateRows + row] =
            (red[at] + red[at + 4 * 64]) + (red[at + 8 * 64] + red[at + 12 * 64]);
      }
    }
    consumer_sync();
  }
}

// ------------------------------------------------------------------------------------------------
// phase 2: selection, one warp per token
// ------------------------------------------------------------------------------------------------
// Affinity with the accurate exponential and division: the selection compares these values.
__device__ __forceinline__ float affinity_rn(float l, int score_func) {
  if (score_func == MOE_SCORE_SQRT_SOFTPLUS) return sqrtf(fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))));
  return __fdiv_rn(1.f, 1.f + expf(-l));
}

// An unsigned key that orders as the float does; never 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return max((b & 0x80000000u) ? ~b : b | 0x80000000u, 1u);
}

template <int PL>   // experts per lane: e = lane + 32 i
__device__ __forceinline__ void select_experts(const DecodeParams& p, DecodeSmem* sm, float* scores, int t, int lane) {
  float sc[PL];
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) sc[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.gate_splits; ++s) {
    const float* src = p.partial + ((size_t)s * p.T + t) * p.E;
#pragma unroll
    for (int i = 0; i < PL; ++i) sc[i] += __ldcg(src + min(lane + 32 * i, p.E - 1));
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    if (p.logit_offset != nullptr) sc[i] += __ldg(p.logit_offset + min(e, p.E - 1));
    if (e >= p.E) sc[i] = -INFINITY;
  }
  if (p.score_func == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, sc[i]);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      sc[i] = lane + 32 * i < p.E ? expf(sc[i] - m) : 0.f;
      z += sc[i];
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int i = 0; i < PL; ++i) sc[i] = __fdiv_rn(sc[i], z);
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i < p.E) sc[i] = affinity_rn(sc[i], p.score_func);
  }

  int my_e = 0;          // lane j holds slot j's expert and unbiased score
  float my_s = 0.f;
  if (p.token_ids != nullptr) {
    int tok = p.token_ids[t];
    if (tok < 0 || tok >= p.vocab) {
      if (blockIdx.x == 0 && lane == 0) record_error(p.ew, MOE_ERR_DEVICE, tok);
      tok = tok < 0 ? 0 : p.vocab - 1;
    }
    if (lane < p.k) {
      my_e = p.tid2eid[(size_t)tok * p.k + lane];
      if (my_e < 0 || my_e >= p.E) {
        if (blockIdx.x == 0) record_error(p.ew, MOE_ERR_DEVICE, my_e);
        my_e = my_e < 0 ? 0 : p.E - 1;
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i < p.E) scores[lane + 32 * i] = sc[i];
    __syncwarp();
    my_s = scores[my_e];
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      const float b = e < p.E ? __fadd_rn(sc[i], p.bias != nullptr ? p.bias[e] : 0.f) : 0.f;
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
        const int e = lane + 32 * i;
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
          at = lane + 32 * i;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int e = __reduce_min_sync(0xffffffffu, top != 0u && best == top ? at : 0x7fffffff);
      const int ec = e < p.E ? e : 0;   // no candidate left (scores that are not numbers): stays in range
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i == ec) {
          mine = sc[i];
          key[i] = 0u;
        }
      const float s = __shfl_sync(0xffffffffu, mine, ec & 31);
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
    sm->sel_e[t * p.k + lane] = my_e;
    sm->sel_w[t * p.k + lane] = w;
  }
}

// The lists of active experts and their token rows, by the consumer threads (at most 128 slots).  Active
// expert 0 is the shared one with every token; the routed ones follow in the order of their first slot.
// A token that names an expert twice (a table may) has one row there.
__device__ __forceinline__ void build_lists(const DecodeParams& p, DecodeSmem* sm, int tid) {
  const int S = p.T * p.k;
  const bool live = tid < S;
  const int t = live ? tid / p.k : 0, e = live ? sm->sel_e[tid] : -1;
  if (live) {
    int d = 0;
    for (int s = t * p.k; s < tid; ++s) d |= sm->sel_e[s] == e;
    sm->dup[tid] = d;
  }
  consumer_sync();
  int n = 0, rank = 0, s0 = tid;
  float wsum = 0.f;
  if (live) {
    for (int s = S - 1; s >= 0; --s) {
      if (sm->sel_e[s] != e) continue;
      s0 = s < s0 ? s : s0;
      if (!sm->dup[s]) {
        ++n;
        rank += s < t * p.k;
      }
    }
    for (int s = t * p.k; s < (t + 1) * p.k; ++s)
      if (sm->sel_e[s] == e) wsum += sm->sel_w[s];
    sm->first[tid] = s0 == tid;
    sm->cnt[tid] = n;
  }
  consumer_sync();
  if (live) {
    int order = 1, off = p.T;
    for (int s = 0; s < s0; ++s)
      if (sm->first[s]) {
        ++order;
        off += sm->cnt[s];
      }
    const int row = off + rank;
    sm->row_of_slot[tid] = row;
    if (!sm->dup[tid]) {
      sm->tok_of_row[row] = t;
      sm->row_w[row] = wsum;
    }
    if (s0 == tid) {
      sm->act_e[order] = e;
      sm->act_off[order] = off;
      sm->act_n[order] = n;
    }
  } else if (tid == kConsumers - 1) {
    int c = 1;
    for (int s = 0; s < S; ++s) c += sm->first[s];
    sm->n_act = c;
    sm->act_e[0] = p.E;
    sm->act_off[0] = 0;
    sm->act_n[0] = p.T;
  } else if (tid >= kMaxS && tid < kMaxS + p.T) {
    sm->tok_of_row[tid - kMaxS] = tid - kMaxS;
    sm->row_w[tid - kMaxS] = 1.f;
  }
}
static_assert(kMaxS + kMaxT < kConsumers - 1, "the list threads do not overlap");

// ------------------------------------------------------------------------------------------------
// consumers: one stage into the warp's accumulators
// ------------------------------------------------------------------------------------------------
// Four bf16 pairs of the eight E2M1 codes of w, pair i holding codes i and i + 4: the sign bit to bit
// 15, exponent and mantissa to bits 8-6, which is the value times 2^-126 (subnormals included), then an
// exact multiply by 2^126.
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t k126 = 0x7E807E80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = w << (12 - 4 * i);
    const uint32_t b = (y & 0x80008000u) | ((y >> 6) & 0x01C001C0u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&k126));
    v[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Block scales in [2, 252]; others are clamped and reported.
__device__ __forceinline__ uint32_t checked_scales(uint32_t s4, ErrorWord* ew) {
  if (__vminu4(s4, 0xFCFCFCFCu) != s4 || __vmaxu4(s4, 0x02020202u) != s4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s = (s4 >> (8 * i)) & 0xFFu;
      if (s < 2u || s > 252u) record_error(ew, MOE_ERR_DEVICE, 0x10000 + (int)s);
    }
    s4 = __vmaxu4(__vminu4(s4, 0xFCFCFCFCu), 0x02020202u);
  }
  return s4;
}

// The warp's token fragments of one stage: 16 bytes of each of its kBlocks blocks of 32 elements, for
// token columns g and g + 8.
template <bool kFp4, int kNT>
struct TokenFrags {
  static constexpr int kBlocks = kFp4 ? 4 : 2;
  uint4 v[kNT][kBlocks];
  // row: the columns' rows or null; k: first element of the warp's part, K: elements of a row
  template <bool kDown>
  __device__ __forceinline__ void load(const __nv_bfloat16* const (&row)[kNT], int k, int K, int t) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int kb = 0; kb < kBlocks; ++kb) {
        v[nt][kb] = make_uint4(0u, 0u, 0u, 0u);
        if (k < K && row[nt] != nullptr) {
          const uint4* at = reinterpret_cast<const uint4*>(row[nt] + k + kb * 32 + t * 8);
          v[nt][kb] = kDown ? __ldcg(at) : __ldg(at);   // h is written during this kernel: read from L2
        }
      }
  }
};

// kPaired: the token rows already hold each octet in the order 0 4 1 5 2 6 3 7 (MXFP4's h).
// w: the warp's place in its group of eight.
template <bool kFp4, bool kPaired, int NT, int kNT>
__device__ __forceinline__ void consume_stage(uint32_t stage, int w, int lane, const TokenFrags<kFp4, kNT>& tok,
                                              float (&acc)[kNT][4], ErrorWord* ew) {
  using S = Stage<kFp4>;
  const int g = lane >> 2, t = lane & 3;
  if (!kFp4) {
    const uint32_t wr = stage + w * 1024 + g * 128;   // the warp's 64 elements are box w
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const uint32_t at = wr + (((kb * 4 + t) ^ g) << 4);
      const uint4 lo = lds128(at), hi = lds128(at + S::kBlock);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = tok.v[nt][kb];
        mma_bf16(acc[nt], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
        mma_bf16(acc[nt], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
      }
    }
  } else {
    // the warp's 128 elements are half of box w / 2
    const uint32_t wr = stage + (w >> 1) * 1024 + g * 128 + t * 4, sr = stage + S::kSOff + g * S::kSPitch + w * 4;
    const uint32_t s_lo = checked_scales(lds32(sr), ew), s_hi = checked_scales(lds32(sr + 8 * S::kSPitch), ew);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      const uint32_t at = wr + ((((w & 1) * 4 + kb) ^ g) << 4);
      uint32_t lo[4], hi[4];
      e2m1_pairs(lds32(at), lo);
      e2m1_pairs(lds32(at + S::kBlock), hi);
      const float f_lo = __uint_as_float(((s_lo >> (8 * kb)) & 0xFFu) << 23);
      const float f_hi = __uint_as_float(((s_hi >> (8 * kb)) & 0xFFu) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint4 b = tok.v[nt][kb];
        if (!kPaired)
          b = make_uint4(__byte_perm(b.x, b.z, 0x5410), __byte_perm(b.x, b.z, 0x7632), __byte_perm(b.y, b.w, 0x5410),
                         __byte_perm(b.y, b.w, 0x7632));
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16(part, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
        mma_bf16(part, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
        acc[nt][0] = fmaf(part[0], f_lo, acc[nt][0]);
        acc[nt][1] = fmaf(part[1], f_lo, acc[nt][1]);
        acc[nt][2] = fmaf(part[2], f_hi, acc[nt][2]);
        acc[nt][3] = fmaf(part[3], f_hi, acc[nt][3]);
      }
    }
  }
}

// The warp's accumulators of a tile into the exchange buffer, [warp][token column][kRedPitch rows].
template <int kNT>
__device__ __forceinline__ void put_partials(float* red, int warp, int lane, const float (&acc)[kNT][4], int nt_used) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    if (nt >= nt_used) break;
    float* c = red + (warp * kMaxT + nt * 8 + 2 * t) * kRedPitch + g;
    c[0] = acc[nt][0];
    c[kRedPitch] = acc[nt][1];
    c[8] = acc[nt][2];
    c[kRedPitch + 8] = acc[nt][3];
  }
}
__device__ __forceinline__ float sum_partials(const float* red, int col, int row) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) v += red[(w * kMaxT + col) * kRedPitch + row];
  return v;
}

// ------------------------------------------------------------------------------------------------
// the kernel
// ------------------------------------------------------------------------------------------------
// The weight stream: TMA copies by lane 0 and, for MXFP4, the scales by cp.async of all 32 lanes (then the
// full barriers count their 32 arrivals too).
template <bool kFp4>
__device__ __forceinline__ void produce(const DecodeParams& p, const CUtensorMap* map_w1, const CUtensorMap* map_w3,
                                        const CUtensorMap* map_w2, DecodeSmem* sm, uint8_t* ring, int lane) {
  using S = Stage<kFp4>;
  if (p.test_stall) return;
  volatile int* abort = &sm->abort;
  constexpr int kBox = kFp4 ? 256 : 64;
  RingPos pos;
  int issued = 0;
  bool ok = true, routed = false;
  auto tile = [&](bool down, int a, int blk) {
    const int K = down ? p.I : p.d, e = sm->act_e[a];
    const int row = down ? e * p.d + blk * 16 : e * p.I + blk * 8;
    const CUtensorMap *m0 = down ? map_w2 : map_w1, *m1 = down ? map_w2 : map_w3;
    for (int k0 = 0; k0 < K; k0 += S::kChunk) {
      uint64_t* bar = &sm->full[pos.slot];
      uint8_t* dst = ring + pos.slot * S::kBytes;
      if (kFp4) {
        if (!mbar_wait_warp(&sm->empty[pos.slot], pos.phase ^ 1, abort, p.ew, 401)) return false;
        const int r = lane >> 1, half = lane & 1;
        const uint8_t* ws = down ? p.w2s : (r < 8 ? p.w1s : p.w3s);
        if (k0 + half * 512 < K)
          cp_async16(smem_u32(dst + S::kSOff + r * S::kSPitch + half * 16),
                     ws + ((size_t)(row + (down ? r : r & 7)) * K + k0) / 32 + half * 16);
        cp_async_arrive(bar);
      } else if (lane == 0) {
        if (!mbar_wait(&sm->empty[pos.slot], pos.phase ^ 1, abort, p.ew, 401)) return false;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, 2 * S::kBlock);   // whole boxes: what lies past K is filled with zeros
        tma_load_3d(dst, m0, bar, 0, row, k0 / kBox);
        tma_load_3d(dst + S::kBlock, m1, bar, 0, down ? row + 8 : row, k0 / kBox);
      }
      ++issued;
      pos.step(1, p.stages);
    }
    return true;
  };
  const int nb1 = p.I / 8, nb2 = p.d / 16;
  for (TileIter it(nb1); ok; it.next()) {
    if (it.a > 0 && !routed) {
      ok = kFp4 ? mbar_wait_warp(&sm->routed, 0, abort, p.ew, 403) : mbar_wait(&sm->routed, 0, abort, p.ew, 403);
      routed = true;
      if (!ok) break;
    }
    if (routed && it.a >= sm->n_act) break;
    ok = tile(false, it.a, it.blk);
  }
  if (ok)
    for (TileIter it(nb2); ok && it.a < sm->n_act; it.next()) ok = tile(true, it.a, it.blk);
  if (!ok) {   // let every copy already issued land before the CTA leaves
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
      mbar_wait(&sm->full[i % p.stages], (i / p.stages) & 1, nullptr, nullptr, 0, 200000000LL);
  }
}

// kNT: column tiles of eight tokens (1 for batches of at most 8, whose fragments then take half the registers).
template <bool kFp4, int kNT>
__global__ void __launch_bounds__(kDecThreads, 1)
    layer_decode_kernel(const __grid_constant__ CUtensorMap map_w1, const __grid_constant__ CUtensorMap map_w3,
                        const __grid_constant__ CUtensorMap map_w2, const __grid_constant__ DecodeParams p) {
  using S = Stage<kFp4>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DecodeSmem* sm = reinterpret_cast<DecodeSmem*>(ring + p.stages * S::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sm->full[i], kFp4 ? 1 + 32 : 1);
      mbar_init(&sm->empty[i], 8);
    }
    mbar_init(&sm->routed, 1);
    sm->abort = 0;
    sm->act_e[0] = p.E;
    fence_barrier_init();
    tma_prefetch_desc(&map_w1);
    tma_prefetch_desc(&map_w3);
    tma_prefetch_desc(&map_w2);
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    if (kFp4 || lane == 0) produce<kFp4>(p, &map_w1, &map_w3, &map_w2, sm, ring, lane);
    __syncwarp();   // lanes without work wait here, not at the CTA's barrier
  } else {
    volatile int* abort = &sm->abort;
    const int G = (int)gridDim.x;
    // Every wait below is bounded; after one has run out the threads go on over whatever lies in shared
    // memory (all indices stay in range), so that they keep meeting at the same barriers.
    // ---------------- phase 1 and 2: routing ----------------
    float* red0 = sm->red[0];
    if (p.T == 1)
      gate_partials<1>(p, 0, red0, warp, lane);
    else
      for (int t0 = 0; t0 < p.T; t0 += 4) gate_partials<4>(p, t0, red0, warp, lane);
    __threadfence();
    consumer_sync();
    if (tid == 0) {
      red_release_add(&p.ew->decode_arrive[0], 1);
      grid_wait(&p.ew->decode_arrive[0], G, abort, p.ew, 404);
    }
    consumer_sync();
    if (warp < p.T) {
      if (p.E <= 256) select_experts<8>(p, sm, red0 + warp * 512, warp, lane);
      else select_experts<16>(p, sm, red0 + warp * 512, warp, lane);
    }
    consumer_sync();
    build_lists(p, sm, tid);
    consumer_sync();
    if (tid == 0) mbar_arrive(&sm->routed);
    if (blockIdx.x == 0) {
      const int n = p.T * p.k;
      if (tid < n && p.weights_out != nullptr) p.weights_out[tid] = sm->sel_w[tid];
      if (tid < n && p.indices_out != nullptr) p.indices_out[tid] = sm->sel_e[tid];
      if (p.counts_out != nullptr && tid < p.E) {
        int c = 0;
        for (int s = 0; s < n; ++s) c += sm->sel_e[s] == tid;
        p.counts_out[tid] = c;
      }
    }

    // ---------------- phase 3 and 4: up and down projections ----------------
    int count = 0, buf = 0;      // stages of the tiles so far (the groups take turns)
    RingPos pos;                 // and where the next one lies
    const uint32_t ring_addr = smem_u32(ring);
    const int grp = warp >> 3, w8 = warp & 7, g = lane >> 2, t = lane & 3;
    const int part = S::kChunk / 8;          // elements of a stage that this warp takes
    auto run_phase = [&](auto down_tag) {
      constexpr bool kDown = decltype(down_tag)::value;
      const int K = kDown ? p.I : p.d, nb = kDown ? p.d / 16 : p.I / 8, na = sm->n_act;
      const int ns = (K + S::kChunk - 1) / S::kChunk;
      // the warp's next stage, whose token fragments are loaded ahead: tile, stage in it, stages before it
      TileIter ahead(nb);
      int ahead_s = (grp ^ count) & 1, ahead_count = count;
      const __nv_bfloat16* rows[kNT] = {};
      TokenFrags<kFp4, kNT> cur, nxt;
      auto rows_of = [&](int a) {
        const int n = sm->act_n[a], r0 = sm->act_off[a];
        auto row = [&](int c) -> const __nv_bfloat16* {
          if (c >= n) return nullptr;
          return kDown ? p.h + (size_t)(r0 + c) * p.I : p.x + (size_t)sm->tok_of_row[r0 + c] * p.d;
        };
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) rows[nt] = row(g + 8 * nt);
      };
      auto fetch = [&](bool first) {
        bool moved = first;
        while (ahead_s >= ns) {          // past the tile's end: the warp's first stage of the next one
          ahead_count += ns;
          ahead.next();
          ahead_s = (grp ^ ahead_count) & 1;
          moved = true;
        }
        if (ahead.a >= na) return;
        if (moved) rows_of(ahead.a);
        nxt.template load<kDown>(rows, ahead_s * S::kChunk + w8 * part, K, t);
        ahead_s += 2;
      };
      fetch(true);
      for (TileIter it(nb); it.a < na; it.next()) {
        const int n = sm->act_n[it.a], r0 = sm->act_off[it.a];
        float acc[kNT][4] = {};
        RingPos mine = pos;
        if ((grp ^ count) & 1) mine.step(1, p.stages);
        for (int s = (grp ^ count) & 1; s < ns; s += 2, mine.step(2, p.stages)) {
          cur = nxt;
          fetch(false);
          const int slot = mine.slot;
          if (!*abort) mbar_wait(&sm->full[slot], mine.phase, abort, p.ew, kDown ? 406 : 405);
          __syncwarp();
          if (s * S::kChunk + w8 * part < K) {
            if (kNT == 1 || n <= 8) consume_stage<kFp4, kDown, 1>(ring_addr + slot * S::kBytes, w8, lane, cur, acc, p.ew);
            else consume_stage<kFp4, kDown, kNT>(ring_addr + slot * S::kBytes, w8, lane, cur, acc, p.ew);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->empty[slot]);
        }
        count += ns;
        pos.step(ns, p.stages);
        float* red = sm->red[buf];
        buf ^= 1;   // the barrier of the next tile keeps its writes behind this tile's reads
        put_partials(red, warp, lane, acc, n <= 8 ? 1 : 2);
        consumer_sync();
        if (kDown) {
          const int c = tid >> 4, r = tid & 15;
          if (c < n) p.out[(size_t)(r0 + c) * p.d + it.blk * 16 + r] = sum_partials(red, c, r);
        } else {
          const int c = tid >> 3, f = tid & 7;
          if (c < n) {
            const float gate = sum_partials(red, c, f), val = sum_partials(red, c, f + 8);
            const float w = p.weight_in_expert && it.a > 0 ? sm->row_w[r0 + c] : 1.f;
            const int at = kFp4 ? (f < 4 ? 2 * f : 2 * f - 7) : f;   // MXFP4: the octet's order 0 4 1 5 2 6 3 7
            p.h[(size_t)(r0 + c) * p.I + it.blk * 8 + at] = __float2bfloat16_rn(swiglu(gate, val, p.swiglu_limit, w));
          }
        }
      }
    };
    // all CTAs past a phase before the next reads its rows
    auto grid_barrier = [&](int which, int site) {
      __threadfence();
      consumer_sync();
      if (tid == 0) {
        red_release_add(&p.ew->decode_arrive[which], 1);
        grid_wait(&p.ew->decode_arrive[which], G, abort, p.ew, site);
      }
      consumer_sync();
    };
    run_phase(std::false_type{});
    grid_barrier(1, 402);
    run_phase(std::true_type{});
    grid_barrier(2, 407);

    // ---------------- phase 5: combine, slot order then the shared expert ----------------
    const int d4 = p.d / 4;
    for (int i = blockIdx.x * kConsumers + tid; i < p.T * d4; i += G * kConsumers) {
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
  // the last CTA to get here leaves the grid's counters at zero (nobody waits on them any more)
  __syncwarp();
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&p.ew->decode_done, 1) == (int)gridDim.x - 1) {
      p.ew->decode_arrive[0] = p.ew->decode_arrive[1] = p.ew->decode_arrive[2] = 0;
      p.ew->decode_done = 0;
    }
  }
}

}  // namespace

int decode_gate_splits(int E, int d) {
  // about one unit of 16 router rows per SM of a B200, at least 128 elements of k each
  return std::max(1, std::min(d / 128, 148 / (E / kGateRows)));
}

cudaError_t launch_layer_decode(const CUtensorMap& w1, const CUtensorMap& w3, const CUtensorMap& w2, DecodeParams p,
                                bool fp4, int num_sms, cudaStream_t stream) {
  const size_t smem = 227 * 1024;
  const size_t stage = fp4 ? Stage<true>::kBytes : Stage<false>::kBytes;
  // An even number: a slot then always belongs to the same group of consumer warps, which waits for each of
  // its fills in turn.  With an odd one the groups would share a slot, and the group of its second fill,
  // running ahead inside a long tile, would take a first fill that has not landed for its own (a barrier's
  // parity tells two successive phases apart, not three).
  p.stages = (int)std::min<size_t>(kMaxStages, (smem - 1024 - sizeof(DecodeSmem)) / stage) & ~1;
  auto kernel = fp4 ? (p.T <= 8 ? layer_decode_kernel<true, 1> : layer_decode_kernel<true, 2>)
                    : (p.T <= 8 ? layer_decode_kernel<false, 1> : layer_decode_kernel<false, 2>);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  // no more CTAs than any phase has work for: small layers pay for each arrival at the barriers
  const long tiles = (long)(std::min(p.T * p.k, p.E) + 1) * std::max(p.I / 8, p.d / 16);
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
