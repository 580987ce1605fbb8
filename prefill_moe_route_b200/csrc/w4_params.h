// w4_params.h -- what the few-token operators' host code (api_w4.cu) hands to their
// kernels (linear.cu, layer.cu).
#pragma once
#include "internal.h"

namespace moe {

#ifdef __CUDACC__
#define MOE_HD __host__ __device__
#else
#define MOE_HD
#endif
namespace w4 {
// `total` units cut into n shares as even as whole units allow, the larger
// ones first: share c takes [begin(c), begin(c + 1)), unit u is in share of(u).
struct Shares {
  int n, base, rem;
  MOE_HD Shares() {}
  MOE_HD Shares(int total, int count) : n(count), base(total / count), rem(total % count) {}
  MOE_HD Shares(int count, int quotient, int remainder) : n(count), base(quotient), rem(remainder) {}
  MOE_HD int begin(int c) const { return c * base + (c < rem ? c : rem); }
  MOE_HD int of(int u) const {
    const int big = rem * (base + 1);
    return u < big ? u / (base + 1) : rem + (u - big) / base;
  }
};
}  // namespace w4

// Parameters of the few-token product y = x W^T on MXFP4 weights (linear.cu).
struct LinearParams {
  const uint16_t* x;        // bf16, rows ldx elements apart
  const float* bias;        // may be null
  const uint8_t* wcodes;    // packed weights, 8192-byte blocks [N/128][K/128]
  const uint8_t* wsf;       // packed weight scales: 512-byte blocks [N/128][K/128]
  uint8_t* xop;             // from 9 tokens on, on large weights from 5: operand blocks and scale blocks [token tile][K/128]
  uint8_t* xsf;
  void* out;                // rows ldo elements apart
  uint32_t* part;           // [grid][tokens per tile][128] parts of tiles cut between shares, zero between calls
  int32_t* status;
  w4::Shares shares;        // of row tiles x token tiles x KU units
  int64_t ldx, ldo;
  int M, N, K, KC, KU, TT;  // K chunks of 128, units along K, token tiles
  int out_f32;
  int test_withhold;        // test knob: leave the last share's part unpublished
  uint64_t timeout_ns;
};

// Parameters of the few-token MoE layer (layer.cu).
struct LayerParams {
  const uint16_t* x;        // bf16, rows ldx elements apart
  const uint16_t* norm_w;   // bf16 [H], or null: no norm
  const uint16_t* router_w; // bf16 [E][H]
  const float* bias;        // fp32 [E], or null
  const uint8_t *s13, *s2, *ss13, *ss2;   // packed weight scales: routed, shared
  uint16_t* out;            // bf16, rows ldo elements apart
  int32_t* ids_out;         // [M][topk], or null
  float* wts_out;           // [M][topk], or null
  int32_t* status;
  int32_t* sync;            // [0] next task, [2] CTAs that have routed: zero between calls; [1] pieces of mid tiles stored: k_layer_head zeroes it
  uint32_t *part1, *part2;  // parts of cut tiles: [grid][gate, up of the tokens][128], [grid][tokens][128]; zero between calls
  uint32_t *sig, *rstd;     // sigmoids of the logits [M][E], the norm's factors [M], as parts (zero between calls)
  uint8_t *xop, *xsf;       // the tokens' operand blocks and scale blocks [H/128]
  uint8_t *mop, *msf;       // mid's, one per GEMM1 tile (up to 4 tokens: inverted words, scales a word each)
  int64_t ldx, ldo;
  int M, H, I, S, E, topk;  // S: the shared expert's width, 0 without one
  int nc;                   // operand columns: 16 up to 8 tokens, else 32
  int residual, test_withhold;
  float scale, eps;
  uint64_t timeout_ns;
  uint64_t test_hold_ns;    // test knob: the last CTA waits this long between its first ticket and its routing
};

}  // namespace moe
