// Parameter blocks and declarations of the serving kernels: the layer for a few tokens (decode.cu) and the linear
// projection (linear.cu).
#pragma once

#include "kernels.h"

namespace moe {

// The control words behind the error word at the head of a workspace, all zero between calls.
struct GridCounters {
  int arrive[4];        // the one-launch layer's grid counters: logits, up tiles, down, tokens
  int done;             //   CTAs and their reporting lanes finished
  int ready[144];       //   up tiles finished, per active expert
  int linear_done[512]; // the linear projection's parts of a tile finished
};
constexpr size_t kErrorBytes = 256, kControlBytes = 4096;   // ErrorWord; both together
static_assert(kErrorBytes + sizeof(GridCounters) <= kControlBytes, "the workspace's first region");

// What the failure-detection test hook makes a serving kernel do.
enum Stall {
  kStallCopies = 1,   // the producers issue no copies
  kStallRouter = 2,   // the router warps build no lists
  kStallLater = 3,    // the producers issue a few stages of copies each (inside a tile), and no more
  kStallOneCta = 4    // those of the first CTA alone
};

// The whole layer for a few tokens (decode.cu).
constexpr int kDecodeMaxTokens = MOE_DECODE_MAX_TOKENS;
struct DecodeParams {
  int T, d, E, G, g, k, I;
  int score_func, renorm;
  float route_scale, swiglu_limit;
  int weight_in_expert;       // routed rows of h carry their weights, the combine adds unweighted rows
  int vocab;                  // > 0 with token_ids and tid2eid: the token-id table routes
  int gate_splits;            // slices of k of the router logits
  int stages;                 // of a weight ring (set by the launcher)
  int test_stall;             // failure-detection test hook, one of Stall (0 outside the test build)
  const int32_t* token_ids;   // [T] or null
  const int32_t* tid2eid;     // [vocab, k]
  const float* w_gate;        // [E, d]
  const float* bias;          // [E] or null
  const float* logit_offset;  // [E] or null
  const __nv_bfloat16* x;     // [T, d]
  const uint8_t *w1, *w3, *w2;     // bf16 rows, or packed E2M1 codes
  const uint8_t *w1s, *w3s, *w2s;  // UE8M0 block scales (MXFP4), else null
  float* partial;             // [gate_splits, T, E] scratch
  uint16_t* x16;              // MXFP4: [T, d] scratch, x in f16 blocks of 32, and
  float* x_scale;             //   their scales [T, d / 32]
  uint16_t* h;                // [T + T * k, I] scratch (bf16; MXFP4: f16 blocks): shared rows first, then the experts'
  long long h_lo;             // bf16: elements from h to its second parts (h = first + second, 16 bits)
  float* h_scale;             // MXFP4: [T + T * k, I / 32] scratch
  int32_t* route_e;           // [T * k] scratch: the selection, handed round the grid
  float* route_w;             // [T * k]
  float* out;                 // [T + T * k, d] scratch
  __nv_bfloat16* y;           // [T, d]
  float* weights_out;         // [T, k] or null
  int32_t* indices_out;       // [T, k] or null
  int32_t* counts_out;        // [E] or null
  ErrorWord* ew;
  GridCounters* gc;
};
int decode_gate_splits(int E, int d);
// w1 / w3 / w2: the stacked expert matrices as [128 bytes, rows, bytes of a row / 128] in boxes of
// 128 bytes x 8 rows x 8 (bf16) or 128 bytes x 32 rows x 2 (packed codes), 128-byte swizzle.
cudaError_t launch_layer_decode(const CUtensorMap& w1, const CUtensorMap& w3, const CUtensorMap& w2, DecodeParams p,
                                bool fp4, int num_sms, cudaStream_t stream);

// The linear projection (linear.cu).
constexpr int kLinearStreamTokens = 16;   // batches up to this run as a weight stream
struct LinearParams {
  int T, K, N;
  int act, out_fp32;
  int y_vec, residual_vec, bias_vec;  // rows of y / residual, and bias, start on 16-byte boundaries
  int stages;                 // set by the launcher
  int m_tiles, n_tiles, splits;
  int x_box;                  // rows of x per tile in shared memory
  int test_stall;             // as DecodeParams::test_stall (kStallCopies, kStallLater)
  long long ldx, ldy, ldr;    // elements
  const __nv_bfloat16* x;
  const float* bias;          // [N] or null
  const __nv_bfloat16* residual;  // or null
  void* y;
  float* scratch;
  ErrorWord* ew;
  GridCounters* gc;
};
// How a projection of T tokens runs: as a weight stream, or in tiles of CTA pairs or of single CTAs, these with
// K cut over a cluster of `splits`.  x_box, w_box: rows per box of the
// tensor maps (64 elements of k wide).
struct LinearPlan {
  enum Kind { kStream, kSolo, kPair } kind;
  int m_tiles, n_tiles, splits;
  int x_box, w_box;
  size_t scratch_floats;
};
LinearPlan linear_plan(int T, int K, int N, int num_sms);
cudaError_t launch_linear(const LinearPlan& plan, const CUtensorMap& map_x, const CUtensorMap& map_w, LinearParams p,
                          int num_sms, cudaStream_t stream);

}  // namespace moe
