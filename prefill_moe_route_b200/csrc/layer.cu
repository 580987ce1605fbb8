// layer.cu -- a whole mixture-of-experts layer for a few tokens (M <= 16) in
// two launches: RMS norm, router product, top-k, SwiGLU experts on MXFP4
// weights with bf16 activations, an always-used shared expert, the residual.
//
//   k_layer_head     the router's logits (bf16 MMAs, nothing rounded) and the
//                    norm's sums of squares, cut along K, to sigmoids; and the tokens as
//                    tensor-core operand columns (w4.cuh) of x * norm weight.  The
//                    norm's 1 / rms is a factor of the token, applied to the sums.
//   k_layer_experts  one CTA an SM.  Each routes the tokens from the sigmoids (the
//                    same everywhere), then streams weights: GEMM1 over the selected
//                    experts' gate and up rows, SwiGLU, mid as operand columns
//                    scaled by the routing weight, and GEMM2, in which the experts
//                    follow one another along K: one accumulation per 128 rows of
//                    out is the routing-weighted sum over all experts (columns of
//                    tokens that did not choose an expert are zero).
//
// Bound: the selected experts' weight bytes, for few tokens the chain of hand-overs
// between router, routing, GEMM1, mid and GEMM2.  H = 6144, E = 256, top-8: 16
// tokens with I = 512 take 83 us (66 experts, 4.1 TB/s: GEMM1 streams at 5.7, GEMM2 at
// 5.2, 8 us lie between), 4 tokens with I = 256 25.8 us (26 experts, 2.7 TB/s), 1
// token 15.9 us (1.6 TB/s).  All times in this file are those of calls replayed from a
// CUDA graph; calls made one by one take 0.5 us more.  Both products are cut into shares of equal bytes (as in
// linear.cu, parts of a cut tile meet in the share that starts it, in K order), one
// a CTA: twice as many, smaller ones cost more in parts than they balance (16 tokens
// 85.0 us, 4 tokens 28.6).  Shares are tasks that the CTAs draw from one counter,
// all of GEMM1 before all of GEMM2, and a task waits for earlier ones only, so the
// kernel ends however many of its CTAs run at once.  A CTA's weight stream runs
// ahead into its GEMM2 task while mid is still on its way, a ring's length (sending
// more for L2 then: 16 tokens 85.0 us, it stands before the operands).
#include <algorithm>
#include <type_traits>

#include "w4.cuh"

namespace moe {
namespace layer {

using namespace w4;

// What other kernels may write is read through L2 (__ldcg) throughout: these
// blocks can be resident, beside others that fill their SM's L1, long before
// the kernel whose results they wait for has ended.

constexpr int HEAD_THREADS = 256;
constexpr int HEAD_SLICES = 8;     // CTAs along K of 8 experts' logits (8 / 4, us: 1 token of H = 6144 16.9 / 18.1, 16 tokens 83.1 / 85.7)
constexpr int GROUP = 4;           // tokens whose sums one warp keeps
constexpr int MAX_GROUPS = 4;
// warps: 0 weights, 1 MMA, 2 operands, 3 routing, then four a group of tokens for the sums
constexpr int MAX_THREADS = 128 + 128 * MAX_GROUPS;
constexpr int STAGES = 5;          // as many as fit (5 / 4 / 3, us: 4 tokens of H = 6144 26.4 / 27.3 / 28.8, 16 tokens 83.1 / 86.5 / 92.4)
constexpr int SF_SLOTS = 4;        // TMEM scale slots of 16 columns: two weight blocks, two operand blocks
constexpr int TASKS = 4;           // task ring
constexpr int MAX_M = 16;
constexpr int MAX_SLOTS = 256;     // distinct experts of a call: M * topk at most
constexpr int MIN_SHARE = 2;       // units a share holds at least (1 / 2 / 4, us: 1 token of H = 6144 16.9 / 16.9 / 17.4, 4 small ones 9.9 / 10.0 / 10.7)

template <int NC>
struct Cfg {                       // NC: operand columns, two per token
  static constexpr int MT = NC / 2;
  static constexpr int B_TILE = NC * 128;
  static constexpr int A_BYTES = 2 * A_TILE, B_BYTES = 2 * B_TILE, SF_BYTES = 2 * SF_BLOCK;
  static constexpr int STAGE = A_BYTES + B_BYTES + 2 * SF_BYTES;
  static constexpr int SF_COL0 = 4 * NC;         // two buffers of two accumulators (gate, up)
  static constexpr int TMEM_COLS = 256;
  static_assert(SF_COL0 + SF_SLOTS * 16 <= TMEM_COLS, "tensor memory");
};

struct Smem {
  uint64_t full[STAGES], empty[STAGES], accf[2], acce[2], tfull[TASKS], tempty[TASKS], listed;
  uint32_t tmem;
  int abort_flag;
  int first_task, task[TASKS];
  float rstd[MAX_M];
  int ids[MAX_M * kMaxTopk];
  float wts[MAX_M * kMaxTopk];
  uint32_t mask[kMaxE / 32];       // selected experts
  alignas(16) uint8_t choice[kMaxE][MAX_M];   // by expert and token: 1 + which choice of the token's, 0: none
  uint16_t dlist[MAX_SLOTS];
};

template <int NC>
constexpr int smem_bytes() { return STAGES * Cfg<NC>::STAGE + (int)sizeof(Smem) + 1024; }
static_assert(smem_bytes<16>() <= 232448 && smem_bytes<32>() <= 232448, "shared memory");

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// D += A B, 16 x 8 x 16, bf16 in, fp32 sums.  (The router product is small: two
// dependent launches' latency is what counts here, not the tensor rate.)
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One 128-K chunk of the tokens as operand columns: 16 lanes a token.
__device__ __forceinline__ void split_chunk(const LayerParams& p, int kc) {
  const int t = threadIdx.x >> 4, g8 = threadIdx.x & 15, k = kc * 128 + g8 * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (t < p.M) {
    unpack8(__ldcg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ldx + k)), v);
    if (p.norm_w) {
      float g[8];
      unpack8(__ldcg(reinterpret_cast<const uint4*>(p.norm_w + k)), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g[i];
    }
  }
  uint32_t am = 0;   // largest magnitude's bits; a NaN's are above an infinity's
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  if (t >= p.M) return;
  const int s = split_exp(__uint_as_float(am));
  const float inv = s == SPLIT_NAN ? __int_as_float(0x7FC00000) : exp2i(-s);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_f16x2(f16x2_of(v[2 * i], v[2 * i + 1], inv), hi[i], lo[i]);
  uint8_t* tile = p.xop + (int64_t)kc * p.nc * 128;
  uint8_t* sf = p.xsf + (int64_t)kc * SF_BLOCK;
  const int mt = p.nc / 2;
  *reinterpret_cast<uint2*>(tile + tile_byte(t, g8 * 8)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
  *reinterpret_cast<uint2*>(tile + tile_byte(mt + t, g8 * 8)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  if ((g8 & 3) == 0) {
    sf[sf_byte(t, g8 >> 2)] = static_cast<uint8_t>(split_code_hi(s));
    sf[sf_byte(mt + t, g8 >> 2)] = static_cast<uint8_t>(split_code_lo(s));
  }
}

// Clusters of HEAD_SLICES CTAs.  The first ceil(E / 8): the logits of 8 experts, a
// slice of K a CTA, a warp every 32nd block of 32 K; the slices meet in rank 0.
// The other clusters: one operand chunk a CTA.
// A thread holds 8 consecutive K of token g, of token g + 8 and of expert g (g =
// lane / 4): two MMAs' fragments with K permuted the same way on both sides.
// The norm weight multiplies the router weight; the product of two 8-bit
// significands is two bf16 exactly, so nothing is rounded before the sums.
// NORM: with the norm; HIGH: more than 8 tokens.  64 registers: two of these
// blocks leave an SM room for one of k_layer_experts, whose start they overlap.
template <bool NORM, bool HIGH>
__global__ void __cluster_dims__(HEAD_SLICES, 1, 1) __launch_bounds__(HEAD_THREADS, HIGH ? 3 : 4) k_layer_head(const LayerParams p) {
  constexpr int BATCH = 3;   // blocks in flight
  __shared__ float sd[8][16][8], sq[8][16];
  __shared__ float cs[HEAD_SLICES][16 * 8 + 16];   // rank 0's: every slice's sums
  __shared__ uint64_t arrived;                     // rank 0's: their bytes
  const int M = p.M, H = p.H, E = p.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nlogit = (E + 7) / 8 * HEAD_SLICES;
  const bool logits = blockIdx.x < nlogit;         // the same for a whole cluster
  const int eg = blockIdx.x / HEAD_SLICES, slice = blockIdx.x % HEAD_SLICES;
  const int g = lane >> 2, kq = (lane & 3) * 8, nblk = H / 32;
  const bool e_ok = eg * 8 + g < E, t0 = g < M, t1 = HIGH && g + 8 < M;
  const uint16_t* wr = p.router_w + (int64_t)(e_ok ? eg * 8 + g : 0) * H + kq;
  const uint16_t* x0 = p.x + (int64_t)(t0 ? g : 0) * p.ldx + kq;
  const uint16_t* x1 = p.x + (int64_t)(t1 ? g + 8 : 0) * p.ldx + kq;
  if (logits) {
    if (threadIdx.x == 0) {
      mbar_init(&arrived, 1);
      fence_mbar_init();
      mbar_arrive_expect_tx(&arrived, HEAD_SLICES * (NORM ? 144 : 128) * 4);
    }
    __syncthreads();
    cluster_arrive_release();   // ready for the others' stores (waited for before they are made)
    if (e_ok && (lane & 3) == 0)   // the router's rows start for L2 while the kernel before ends
      for (int b = slice * 8 + warp; b < nblk; b += 8 * HEAD_SLICES) prefetch_l2_line(wr + b * 32);
  }
  have(wr); have(x0); have(x1);
  pdl_wait();
  // What k_layer_experts uses before this kernel's end (tickets, the count of routed
  // CTAs, empty sigmoids) was left ready by the call before, whose kernels have ended;
  // the count of mid's pieces it uses behind this kernel's end.
  if (blockIdx.x + 1 == gridDim.x && threadIdx.x == 0) p.sync[1] = 0;
  pdl_launch_dependents();
  if (!logits) {
    if (blockIdx.x - nlogit < H / 128) split_chunk(p, blockIdx.x - nlogit);
    if (M <= GROUP) {   // mid's words are empty until they are made
      const int64_t tiles = (int64_t)min(E, M * p.topk) * (p.I / 128) + p.S / 128, step = (int64_t)(gridDim.x - nlogit) * HEAD_THREADS;
      const int64_t first = (int64_t)(blockIdx.x - nlogit) * HEAD_THREADS + threadIdx.x;
      const uint4 empty = make_uint4(0u, 0u, 0u, 0u);
      for (int64_t i = first; i < tiles * (16 * 128 / 16); i += step) __stcg(reinterpret_cast<uint4*>(p.mop) + i, empty);
      for (int64_t i = first; i < tiles * (SF_BLOCK / 16); i += step) __stcg(reinterpret_cast<uint4*>(p.msf) + i, empty);
    }
    return;
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float d[4] = {0.f, 0.f, 0.f, 0.f}, ss0 = 0.0f, ss1 = 0.0f;
#pragma unroll 1
  for (int b0 = slice * 8 + warp; b0 < nblk; b0 += 8 * HEAD_SLICES * BATCH) {
    uint4 w[BATCH], gw[BATCH], xa[BATCH], xb[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int b = b0 + i * 8 * HEAD_SLICES;
      const bool in = b < nblk;
      w[i] = in && e_ok ? __ldcg(reinterpret_cast<const uint4*>(wr + b * 32)) : zero;
      if (NORM) gw[i] = in ? __ldcg(reinterpret_cast<const uint4*>(p.norm_w + kq + b * 32)) : zero;
      xa[i] = in && t0 ? __ldcg(reinterpret_cast<const uint4*>(x0 + b * 32)) : zero;
      xb[i] = HIGH && in && t1 ? __ldcg(reinterpret_cast<const uint4*>(x1 + b * 32)) : zero;
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t a[4] = {xa[i].x, xa[i].y, xa[i].z, xa[i].w}, c[4] = {xb[i].x, xb[i].y, xb[i].z, xb[i].w};
      uint32_t bh[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if (NORM) {
        float wf[8], gf[8];
        unpack8(w[i], wf);
        unpack8(gw[i], gf);
        uint32_t bl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float q0 = wf[2 * j] * gf[2 * j], q1 = wf[2 * j + 1] * gf[2 * j + 1];
          bh[j] = pack_bf16x2(q0, q1);
          bl[j] = pack_bf16x2(q0 - __uint_as_float(bh[j] << 16), q1 - __uint_as_float(bh[j] & 0xFFFF0000u));
        }
        mma_16816(d, a[0], c[0], a[1], c[1], bl[0], bl[1]);
        mma_16816(d, a[2], c[2], a[3], c[3], bl[2], bl[3]);
        float f[8];
        unpack8(xa[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss0 = fmaf(f[j], f[j], ss0);
        if (HIGH) {
          unpack8(xb[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) ss1 = fmaf(f[j], f[j], ss1);
        }
      }
      mma_16816(d, a[0], c[0], a[1], c[1], bh[0], bh[1]);
      mma_16816(d, a[2], c[2], a[3], c[3], bh[2], bh[3]);
    }
  }
  *reinterpret_cast<float2*>(&sd[warp][g][(lane & 3) * 2]) = make_float2(d[0], d[1]);
  *reinterpret_cast<float2*>(&sd[warp][g + 8][(lane & 3) * 2]) = make_float2(d[2], d[3]);
  if (NORM) {
#pragma unroll
    for (int o = 1; o <= 2; o *= 2) {
      ss0 += __shfl_xor_sync(0xFFFFFFFFu, ss0, o);
      ss1 += __shfl_xor_sync(0xFFFFFFFFu, ss1, o);
    }
    if ((lane & 3) == 0) { sq[warp][g] = ss0; sq[warp][g + 8] = ss1; }
  }
  __syncthreads();
  cluster_wait_acquire();
  if (threadIdx.x < (NORM ? 128 + 16 : 128)) {
    const int i = threadIdx.x;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum += i < 128 ? sd[q][i >> 3][i & 7] : sq[q][i - 128];
    st_async_cluster_f32(mapa_shared(smem_u32(&cs[slice][i]), 0), sum, mapa_shared(smem_u32(&arrived), 0));
  }
  if (slice != 0 || threadIdx.x >= 128) return;
  // The other slices wait for nothing more, so their sums do come; this block may
  // not end before them.  The limit is far beyond that of k_layer_experts, which
  // finds no sigmoids and says so.
  const uint64_t deadline = globaltimer() + p.timeout_ns + 10000000000ull;
  for (uint32_t spins = 0; !mbar_try_wait_cluster(&arrived, 0);)
    if ((++spins & 255u) == 0 && globaltimer() > deadline) return;
  const int t = threadIdx.x >> 3, e = eg * 8 + (threadIdx.x & 7);
  if (t >= M) return;
  float dot = 0.0f, sum = 0.0f, rstd = 1.0f;
#pragma unroll
  for (int q = 0; q < HEAD_SLICES; ++q) { dot += cs[q][threadIdx.x]; sum += NORM ? cs[q][128 + t] : 0.0f; }
  if (NORM) rstd = 1.0f / sqrtf(sum / (float)H + p.eps);
  if (e < E) part_put(p.sig + t * E + e, sigmoid_spec(dot * rstd));
  if (eg == 0 && (threadIdx.x & 7) == 0) part_put(p.rstd + t, rstd);
}

// Routes token t with one warp from its experts' sigmoids, which it waits for:
// the top k of sigmoid + bias in k rounds (a tie going to the lower expert),
// weights as in route_token_warp.  Every CTA runs this once, cold, so the code
// is kept short.  False: the wait ran out.
template <int KPER>
__device__ __forceinline__ bool pick(const LayerParams& p, int t, int* ids, float* wts, float* rstd, uint32_t* mask,
                                     uint8_t* choice, float* ssig, uint64_t deadline) {
  const int lane = threadIdx.x & 31, E = p.E, k = p.topk;
  uint32_t key[KPER];
  {
    float bias[KPER];
    uint32_t w[KPER], r = 0;
#pragma unroll
    for (int i = 0; i < KPER; ++i) bias[i] = p.bias && lane + 32 * i < E ? __ldcg(p.bias + lane + 32 * i) : 0.0f;
    for (uint32_t spins = 0;;) {
      r = part_peek(p.rstd + t);
      bool all = r != 0u;
#pragma unroll
      for (int i = 0; i < KPER; ++i) w[i] = lane + 32 * i < E ? part_peek(p.sig + t * E + lane + 32 * i) : 1u;
#pragma unroll
      for (int i = 0; i < KPER; ++i) all &= w[i] != 0u;
      if (__all_sync(0xFFFFFFFFu, all)) break;
      if ((++spins & 15u) == 0 && __any_sync(0xFFFFFFFFu, globaltimer() > deadline)) return false;
    }
#pragma unroll
    for (int i = 0; i < KPER; ++i) {
      const float sg = part_value(w[i]);
      ssig[lane + 32 * i] = sg;
      key[i] = lane + 32 * i < E ? float_order_key(p.bias ? __fadd_rn(sg, bias[i]) : sg) : 0u;
    }
    if (lane == 0) *rstd = part_value(r);
  }
  __syncwarp();
  float denom = 0.0f, mine = 0.0f;
  int id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t b[KPER];   // tournament: the lower of equal keys' experts is on the left
    int x[KPER];
#pragma unroll
    for (int i = 0; i < KPER; ++i) { b[i] = key[i]; x[i] = i; }
#pragma unroll
    for (int w = 1; w < KPER; w *= 2)
#pragma unroll
      for (int i = 0; i < KPER; i += 2 * w)
        if (b[i + w] > b[i]) { b[i] = b[i + w]; x[i] = x[i + w]; }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, b[0]);
    const int e = (int)__reduce_min_sync(0xFFFFFFFFu, b[0] == top ? (uint32_t)(lane + 32 * x[0]) : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < KPER; ++i)
      if (lane + 32 * i == e) key[i] = 0u;   // taken (below every key of a number or a NaN)
    const float s = ssig[e];
    denom = __fadd_rn(denom, s);
    if (lane == j) { id = e; mine = s; }
  }
  if (lane < k) {
    ids[lane] = id;
    wts[lane] = __fmul_rn(__fdiv_rn(mine, denom), p.scale);
    choice[id * MAX_M + t] = static_cast<uint8_t>(lane + 1);
    atomicOr(mask + (id >> 5), 1u << (id & 31));
  }
  return true;
}

// NC: operand columns; TG: tokens a warp's group holds (1 and 2 for as many
// tokens, else GROUP): the sums of a tile are spread over four warps a group, so
// that the code is short and a tile's epilogue takes as long for 16 tokens as for 4.
// WORDS: mid is handed over as inverted words (as the parts of sums are), which
// two warps bring into the ring; else as bytes behind a counter, by bulk copies.
// Words save the writer's fence, the counter's trip and the copy's start, but
// every reader polls all it needs.  Words against counter (us): 1 token 17.0 /
// 18.1, 4 small ones 10.0 / 10.5, 4 of H = 6144 26.5 / 27.3, 5 ragged 17.4 / 16.9.
// At most 128 registers there: two blocks of the next call's k_layer_head start
// beside this one (with 142 registers one; 4 tokens of H = 6144 27.4 us).
template <int NC, int TG, bool WORDS>
__global__ void __launch_bounds__(WORDS ? 256 : NC == 32 ? MAX_THREADS : 384, WORDS ? 2 : 1)
k_layer_experts(const __grid_constant__ CUtensorMap tmW13, const __grid_constant__ CUtensorMap tmW2,
                const __grid_constant__ CUtensorMap tmS13, const __grid_constant__ CUtensorMap tmS2, const LayerParams p) {
  using C = Cfg<NC>;
  constexpr int MT = C::MT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* abuf = base;                              // [STAGES][2][A_TILE]
  uint8_t* bbuf = abuf + STAGES * C::A_BYTES;        // [STAGES][2][B_TILE]
  uint8_t* asf = bbuf + STAGES * C::B_BYTES;         // [STAGES][2][512]
  uint8_t* bsf = asf + STAGES * C::SF_BYTES;         // [STAGES][2][512]
  Smem& S = *reinterpret_cast<Smem*>(bsf + STAGES * C::SF_BYTES);
  volatile int* abort_flag = &S.abort_flag;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int M = p.M, E = p.E, topk = p.topk, KC = p.H / 128, HT = p.H / 128, J = p.I / 128, JS = p.S / 128;

  const int groups = (M + TG - 1) / TG, epi_warps = 4 * groups;   // the block has 4 + epi_warps warps
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&S.full[s], 2); mbar_init(&S.empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&S.accf[b], 1); mbar_init(&S.acce[b], epi_warps); }
    for (int t = 0; t < TASKS; ++t) { mbar_init(&S.tfull[t], 1); mbar_init(&S.tempty[t], (WORDS ? 3 : 2) + epi_warps); }
    mbar_init(&S.listed, 1 + epi_warps);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmW13); tma_prefetch_desc(&tmW2);
    if (JS) { tma_prefetch_desc(&tmS13); tma_prefetch_desc(&tmS2); }
  }
  if (warp == 4) { tmem_alloc(&S.tmem, C::TMEM_COLS); tmem_relinquish(); }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kMaxE / 32) S.mask[threadIdx.x - 64] = 0u;
  for (int i = threadIdx.x; i < E; i += blockDim.x)
    reinterpret_cast<uint4*>(S.choice)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // k_layer_head's blocks are all running: its sigmoids are waited for one by
  // one, its end (pdl_wait) only by the reader of the operand columns.
  pdl_launch_dependents();
  const uint64_t deadline = globaltimer() + p.timeout_ns;
  auto fail = [&](uint32_t site) { wait_ran_out(p.status, abort_flag, 9u << 24 | site << 20); };
  int ticket = 0;
  if (threadIdx.x == 0) ticket = atomicAdd(p.sync, 1);   // in flight while routing runs
  if (p.test_hold_ns && blockIdx.x + 1 == gridDim.x) {   // test knob: a CTA that routes late
    const uint64_t until = globaltimer() + p.test_hold_ns;
    while (globaltimer() < until) { }
  }
  if (warp < M) {   // one token a warp: there are at least M warps
    float* scratch = reinterpret_cast<float*>(abuf) + warp * kMaxE;   // in the idle ring
    int* ids = S.ids + warp * topk;
    float* wts = S.wts + warp * topk;
    if (!(E <= 256 ? pick<8>(p, warp, ids, wts, S.rstd + warp, S.mask, S.choice[0], scratch, deadline)
                   : pick<kMaxE / 32>(p, warp, ids, wts, S.rstd + warp, S.mask, S.choice[0], scratch, deadline)))
      fail(10);
    fence_proxy_async_smem();   // the ring's next writers are asynchronous copies
  }
  if (threadIdx.x == 0) S.first_task = ticket;
  __syncthreads();
  if (*abort_flag) {   // no routing, no work
    if (warp == 4) tmem_dealloc(S.tmem, C::TMEM_COLS);
    return;
  }
  const uint32_t mword = lane < kMaxE / 32 ? S.mask[lane] : 0u;
  int ndist;
  const int before = warp_exclusive_scan(__popc(mword), &ndist);
  if (warp >= 3) {   // the selected experts, ascending: for the weight stream and the sums
    for (int i = warp - 3; i < (E + 31) / 32; i += 1 + epi_warps) {
      const uint32_t m = __shfl_sync(0xFFFFFFFFu, mword, i);
      const int n = __shfl_sync(0xFFFFFFFFu, before, i) + __popc(m & ((1u << lane) - 1u));
      if ((m >> lane) & 1u) S.dlist[n] = static_cast<uint16_t>(32 * i + lane);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.listed);
  }
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem, 0);
  // GEMM1: tile i (a gate and an up tile; the shared expert's first) is chunk i
  // of GEMM2's K.  A unit is 128 K of a GEMM1 tile or two chunks of a GEMM2 tile.
  const int tiles1 = JS + ndist * J, CU = (tiles1 + 1) / 2;
  const int U1 = tiles1 * KC, U2 = HT * CU, G = gridDim.x;
  auto cut = [&](int units) -> Shares {
    const int n = min(G, (units + MIN_SHARE - 1) / MIN_SHARE), q = quick_div(units, n);
    return Shares(n, q, units - q * n);
  };
  const Shares sh1 = cut(U1), sh2 = cut(U2);
  struct Where { int e, j, iw; bool shared; };
  auto where = [&](int i) -> Where {
    if (i < JS) return {0, i, JS, true};
    const int r = i - JS, slot = quick_div(r, J);
    return {(int)S.dlist[slot], r - slot * J, J, false};
  };
  auto drain = [&]() { const uint64_t until = globaltimer() + 2000000ull; while (globaltimer() < until) { } };
  // Ticket -> product (1, 2; 0: no more tasks), its share and units [u0, u1), units per tile.
  struct Task { int gemm, share, len, u0, u1; };
  auto task_of = [&](int t) -> Task {   // a share waits for later ones: they are drawn before it
    if (t < sh1.n) { const int c = sh1.n - 1 - t; return {1, c, KC, sh1.begin(c), sh1.begin(c + 1)}; }
    if (t < sh1.n + sh2.n) { const int c = sh1.n + sh2.n - 1 - t; return {2, c, CU, sh2.begin(c), sh2.begin(c + 1)}; }
    return {0, 0, 1, 0, 0};
  };
  // The other roles take the tasks in the order that the weight stream drew
  // them: the first as it is, the later ones from a ring.
  auto next_task = [&](int n, Task* k) -> bool {   // a whole warp
    int t = S.first_task;
    if (n > 0) {
      const int r = (n - 1) % TASKS;
      if (!mbar_wait(&S.tfull[r], ((n - 1) / TASKS) & 1, deadline, abort_flag)) { fail(1); return false; }
      __syncwarp();
      t = S.task[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tempty[r]);
    }
    *k = task_of(t);
    return k->gemm != 0;
  };

  auto choices_out = [&]() {   // a warp
    if (blockIdx.x == 0)
      for (int q = lane; q < M * topk; q += 32) {
        if (p.ids_out) p.ids_out[q] = S.ids[q];
        if (p.wts_out) p.wts_out[q] = S.wts[q];
      }
  };

  // The sigmoids are empty again for the next call once no CTA can still look for
  // them: each counts itself behind its routing (a ticket would not do, the first is
  // drawn before it and may be past the tasks), and the last one empties them.
  auto routed = [&]() {   // a warp
    int n = 0;
    if (lane == 0) n = add_acq_rel_gpu(p.sync + 2, 1);
    if (__shfl_sync(0xFFFFFFFFu, n, 0) != G - 1) return;
    if (lane == 0) __stcg(p.sync + 2, 0);
    for (int i = lane; i < M * E; i += 32) __stcg(p.sig + i, 0u);
    if (lane < M) __stcg(p.rstd + lane, 0u);
  };

  if (warp == 0) {
    // ------------------------------------------------ weights and their scales
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = mbar_wait(&S.listed, 0, deadline, abort_flag);
      if (!ok) fail(11);
      for (int n = 0; ok; ++n) {
        if (n > 0) {
          const int r = (n - 1) % TASKS;
          if (!mbar_wait(&S.tempty[r], (((n - 1) / TASKS) & 1) ^ 1, deadline, abort_flag)) { fail(2); ok = false; break; }
          S.task[r] = ticket;
          mbar_arrive(&S.tfull[r]);
        }
        const Task k = task_of(ticket);
        if (!k.gemm) break;
        ticket = atomicAdd(p.sync, 1);
        int tile = quick_div(k.u0, k.len), i = k.u0 - tile * k.len;
        Where w = where(k.gemm == 1 ? tile : 0);
        for (int u = k.u0; u < k.u1; ++u) {
          if (!mbar_wait(&S.empty[st], ph ^ 1, deadline, abort_flag)) { fail(3); ok = false; break; }
          uint8_t* a = abuf + st * C::A_BYTES;
          uint8_t* sf = asf + st * C::SF_BYTES;
          if (k.gemm == 1) {
            mbar_arrive_expect_tx(&S.full[st], 2 * (CODE_BLOCK + SF_BLOCK));
            const CUtensorMap* map = w.shared ? &tmS13 : &tmW13;
            const uint8_t* s = (w.shared ? p.ss13 : p.s13) + (((int64_t)w.e * 2 * w.iw + w.j) * KC + i) * SF_BLOCK;
            tma_load_3d(a, map, &S.full[st], i * 128, w.j * 128, w.e);
            tma_load_3d(a + A_TILE, map, &S.full[st], i * 128, (w.iw + w.j) * 128, w.e);
            bulk_load(sf, s, SF_BLOCK, &S.full[st]);
            bulk_load(sf + SF_BLOCK, s + (int64_t)w.iw * KC * SF_BLOCK, SF_BLOCK, &S.full[st]);
          } else {
            const int nk = min(2, tiles1 - 2 * i);
            mbar_arrive_expect_tx(&S.full[st], nk * (CODE_BLOCK + SF_BLOCK));
            for (int c = 0; c < nk; ++c) {
              const Where v = where(2 * i + c);
              tma_load_3d(a + c * A_TILE, v.shared ? &tmS2 : &tmW2, &S.full[st], v.j * 128, tile * 128, v.e);
              bulk_load(sf + c * SF_BLOCK,
                        (v.shared ? p.ss2 : p.s2) + (((int64_t)v.e * HT + tile) * v.iw + v.j) * SF_BLOCK, SF_BLOCK, &S.full[st]);
            }
          }
          if (++st == STAGES) { st = 0; ph ^= 1; }
          if (++i == k.len) {
            i = 0;
            ++tile;
            if (k.gemm == 1 && u + 1 < k.u1) w = where(tile);
          }
        }
      }
      // every CTA draws one ticket past the tasks: the last one ends the count
      if (ticket == sh1.n + sh2.n + G - 1) __stcg(p.sync, 0);
      if (!ok) drain();
      if (blockIdx.x == 0) report_used_up(p.status);   // here it holds nobody up
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (the whole warp, one lane issues)
    constexpr uint32_t IDESC = idesc_block_scaled(FMT8_E2M1, FMT8_E4M3, NC);
    int st = 0, slot = 0, seg = 0;
    uint32_t ph = 0;
    bool ok = true;
    Task k;
    for (int n = 0; ok && (ok = next_task(n, &k)); ++n) {
      int i = k.u0 - quick_div(k.u0, k.len) * k.len;
      bool first = true;
      const int nu = k.u1 - k.u0;
      const bool one = k.gemm == 1;
      for (int x = 0; x < nu; ++x) {
        const int b = seg & 1;
        if (first && !mbar_wait(&S.acce[b], ((seg >> 1) & 1) ^ 1, deadline, abort_flag)) { fail(4); ok = false; break; }
        if (!mbar_wait(&S.full[st], ph, deadline, abort_flag)) { fail(5); ok = false; break; }
        __syncwarp();
        tc_fence_after();
        const uint32_t d = tmem + b * 2 * NC;
        const bool last = i + 1 == k.len || x + 1 == nu;
        if (elect_one()) {
          const uint32_t sf = tmem + C::SF_COL0 + slot * 16;
          const uint32_t a0 = smem_u32(abuf + st * C::A_BYTES), b0 = smem_u32(bbuf + st * C::B_BYTES);
          const uint32_t fa = smem_u32(asf + st * C::SF_BYTES), fb = smem_u32(bsf + st * C::SF_BYTES);
          const uint32_t acc = first ? 0u : 1u;
          if (one) {   // gate and up tiles share the tokens' columns
            tc_cp_sf(sf, sdesc_sf(fa));
            tc_cp_sf(sf + 4, sdesc_sf(fa + SF_BLOCK));
            tc_cp_sf(sf + 8, sdesc_sf(fb));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint32_t id = idesc_with_sf(IDESC, ks, ks);
              const uint64_t bd = sdesc_sw128(b0 + ks * 32);
              mma_mxf8f6f4(d, sdesc_sw128(a0 + ks * 32), bd, id, sf, sf + 8, acc | (ks > 0));
              mma_mxf8f6f4(d + NC, sdesc_sw128(a0 + A_TILE + ks * 32), bd, id, sf + 4, sf + 8, acc | (ks > 0));
            }
          } else {
            const int nk = min(2, tiles1 - 2 * i);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c >= nk) break;
              tc_cp_sf(sf + c * 4, sdesc_sf(fa + c * SF_BLOCK));
              tc_cp_sf(sf + 8 + c * 4, sdesc_sf(fb + c * SF_BLOCK));
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_mxf8f6f4(d, sdesc_sw128(a0 + c * A_TILE + ks * 32), sdesc_sw128(b0 + c * C::B_TILE + ks * 32),
                             idesc_with_sf(IDESC, ks, ks), sf + c * 4, sf + 8 + c * 4, acc | (c > 0 || ks > 0));
            }
          }
          tc_commit(&S.empty[st]);
          if (last) tc_commit(&S.accf[b]);
        }
        __syncwarp();
        slot = (slot + 1) % SF_SLOTS;
        first = last;
        if (last) ++seg;
        if (++st == STAGES) { st = 0; ph ^= 1; }
        if (++i == k.len) i = 0;
      }
    }
    if (*abort_flag) drain();
    __syncwarp();
  } else if (warp == 2 || (WORDS && warp == 3)) {
    // ------------------------------------------------ operand columns: the tokens', then mid's
    int st = 0;
    uint32_t ph = 0;
    bool ok = true, mid_ready = WORDS;
    Task k;
    if (WORDS && warp == 3) { routed(); choices_out(); }
    pdl_wait();   // the tokens' columns are there: a kernel's end orders its stores before bulk copies too
    for (int n = 0; ok && (ok = next_task(n, &k)); ++n) {
      if constexpr (WORDS) {
        const int nu = k.u1 - k.u0;
        if (k.gemm == 2) {
          // A unit's live columns, 16 bytes a lane and load, and their scales; units
          // alternate between the two warps, each with two on their way (three and
          // four: the same times).
          constexpr int MX = TG, NLD = 4 * MX * 8 / 32, WD = 2;   // columns of a chunk / 2, loads of a unit
          struct Unit { uint4 d[NLD], s; } w[WD];
          const int half = warp - 2;
          auto column = [&](int r) { const int c = r % (2 * MX); return c < MX ? c : MT - MX + c; };   // of row r of 4 MX
          auto there = [&](int i, int r) { return 2 * i + r / (2 * MX) < tiles1 && (column(r) & (MT - 1)) < M; };
          auto fetch = [&](Unit& v, int i) {
#pragma unroll
            for (int j = 0; j < NLD; ++j) {
              const int r = (lane >> 3) + 4 * j;
              v.d[j] = there(i, r) ? words_peek(reinterpret_cast<const uint32_t*>(p.mop + (2 * (int64_t)i + r / (2 * MX)) * C::B_TILE + column(r) * 128 + (lane & 7) * 16))
                                   : make_uint4(1u, 1u, 1u, 1u);
            }
            v.s = 2 * i + (lane >> 4) < tiles1 && (lane & (MT - 1)) < M
                      ? words_peek(reinterpret_cast<const uint32_t*>(p.msf + (2 * (int64_t)i + (lane >> 4)) * SF_BLOCK + (lane & 15) * 16))
                      : make_uint4(1u, 1u, 1u, 1u);
          };
          auto whole = [&](const Unit& v) {
            bool all = v.s.x && v.s.y && v.s.z && v.s.w;
#pragma unroll
            for (int j = 0; j < NLD; ++j) all &= v.d[j].x && v.d[j].y && v.d[j].z && v.d[j].w;
            return __all_sync(0xFFFFFFFFu, all);
          };
          const int i0 = k.u0 - quick_div(k.u0, k.len) * k.len;
          int id[WD];
#pragma unroll
          for (int d = 0; d < WD; ++d) {
            id[d] = i0 + half + 2 * d;
            while (id[d] >= k.len) id[d] -= k.len;
            if (half + 2 * d < nu) fetch(w[d], id[d]);
          }
          for (int x0 = half; x0 < nu && ok; x0 += 2 * WD) {
#pragma unroll
            for (int d = 0; d < WD; ++d) {
              const int x = x0 + 2 * d;
              if (x >= nu) break;
              uint32_t spins = 0;
              while (ok && !whole(w[d])) {
                if ((++spins & 15u) == 0 && __any_sync(0xFFFFFFFFu, *abort_flag || globaltimer() > deadline)) { fail(6); ok = false; }
                else fetch(w[d], id[d]);
              }
              int s = st + x;
              uint32_t sph = ph;
              while (s >= STAGES) { s -= STAGES; sph ^= 1; }
              if (!ok || !mbar_wait(&S.empty[s], sph ^ 1, deadline, abort_flag)) { fail(7); ok = false; break; }
              __syncwarp();
#pragma unroll
              for (int j = 0; j < NLD; ++j) {
                const int r = (lane >> 3) + 4 * j;
                if (there(id[d], r))
                  *reinterpret_cast<uint4*>(bbuf + s * C::B_BYTES + r / (2 * MX) * C::B_TILE + column(r) * 128 + (lane & 7) * 16) =
                      make_uint4(~w[d].d[j].x, ~w[d].d[j].y, ~w[d].d[j].z, ~w[d].d[j].w);
              }
              *reinterpret_cast<uint32_t*>(bsf + s * C::SF_BYTES + (lane >> 4) * SF_BLOCK + (lane & 15) * 16) =
                  ~(__byte_perm(__byte_perm(w[d].s.x, w[d].s.y, 0x0040), __byte_perm(w[d].s.z, w[d].s.w, 0x0040), 0x5410));
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&S.full[s]);
              if (x + 2 * WD < nu) {
                id[d] += 2 * WD;
                while (id[d] >= k.len) id[d] -= k.len;
                fetch(w[d], id[d]);
              }
            }
          }
        }
        if (k.gemm == 2 || warp == 3) {
          st += nu;
          while (st >= STAGES) { st -= STAGES; ph ^= 1; }
          continue;
        }
      }
      if (k.gemm == 2 && !mid_ready) {
        // every GEMM1 tile's warps have stored their piece of mid
        uint32_t spins = 0;
        while (ld_acquire_gpu(p.sync + 1) < epi_warps * tiles1) {
          if ((++spins & 15u) == 0 && (*abort_flag || globaltimer() > deadline)) { fail(6); ok = false; break; }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        fence_proxy_async_global();
        mid_ready = true;
      }
      if (lane == 0) {
        int i = k.u0 - quick_div(k.u0, k.len) * k.len;
        for (int u = k.u0; u < k.u1; ++u) {
          if (!mbar_wait(&S.empty[st], ph ^ 1, deadline, abort_flag)) { fail(7); ok = false; break; }
          const int nk = k.gemm == 1 ? 1 : min(2, tiles1 - 2 * i);
          const int64_t blk = k.gemm == 1 ? i : 2 * i;
          mbar_arrive_expect_tx(&S.full[st], nk * (C::B_TILE + SF_BLOCK));
          bulk_load(bbuf + st * C::B_BYTES, (k.gemm == 1 ? p.xop : p.mop) + blk * C::B_TILE, nk * C::B_TILE, &S.full[st]);
          bulk_load(bsf + st * C::SF_BYTES, (k.gemm == 1 ? p.xsf : p.msf) + blk * SF_BLOCK, nk * SF_BLOCK, &S.full[st]);
          if (++st == STAGES) { st = 0; ph ^= 1; }
          if (++i == k.len) i = 0;
        }
      }
      st = __shfl_sync(0xFFFFFFFFu, st, 0);
      ph = __shfl_sync(0xFFFFFFFFu, ph, 0);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
    if (*abort_flag) drain();
    __syncwarp();
  } else if (warp == 3) {
    routed();
    choices_out();
  } else {
    // ------------------------------------------------ sums
    const int q = warp & 3, row = 32 * q + lane;   // TMEM lane quarter = warp % 4
    const int t0 = (warp - 4) / 4 * TG;            // this warp's tokens t0 .. t0 + TG - 1
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16) + t0;
    int seg = 0;
    bool ok = mbar_wait(&S.listed, 0, deadline, abort_flag);
    if (!ok) fail(11);
    __syncwarp();
    Task k;
    // Adds the later shares' parts [share + 1, c1] of NV values per row, in K
    // order, to v; value i is token t0 + i % TG's.
    auto live = [&](int i) { return t0 + (i & (TG - 1)) < M; };
    // Parts in flight: about what a tile has; more is more code that runs cold (16 / TG
    // of them and these, us: 16 tokens 83.1 / 82.5, 1 token 17.0 / 16.8)
    constexpr int CB = NC == 32 ? 2 : TG == GROUP ? 3 : 8;
    auto peek = [&](const uint32_t* part, int cb, int c1, auto& w, auto nv_const) {   // parts cb .. c1, CB at most
      constexpr int NV = decltype(nv_const)::value;
#pragma unroll
      for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          w[c][i] = live(i) && cb + c <= c1 ? part_peek(part + (cb + c) * (MAX_GROUPS * NV * 128) + i * 128) : 1u;
    };
    auto gather = [&](uint32_t* part, int share, int c1, auto& v, auto& w, auto nv_const) -> bool {   // w: the first batch
      constexpr int NV = decltype(nv_const)::value;
      uint32_t spins = 0;
      bool in_time = true;
#pragma unroll 1
      for (int cb = share + 1; cb <= c1;) {
        bool all = true;
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
          for (int i = 0; i < NV; ++i) all &= w[c][i] != 0u;
        if (all) {
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            if (cb + c > c1) break;
            uint32_t* src = part + (cb + c) * (MAX_GROUPS * NV * 128);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              v[i] += part_value(w[c][i]);
              if (live(i)) __stcg(src + i * 128, 0u);   // empty again for the next call
            }
          }
          cb += CB;
          if (cb > c1) break;
        } else if ((++spins & 15u) == 0 && (*abort_flag || globaltimer() > deadline)) {
          fail(8);
          in_time = false;
          break;
        }
        peek(part, cb, c1, w, nv_const);
      }
      return __all_sync(0xFFFFFFFFu, in_time);   // lanes wait for different words: they give up together
    };
    // [share][group][value][row]
    uint32_t* part1 = p.part1 + t0 * 2 * 128 + row;
    uint32_t* part2 = p.part2 + t0 * 128 + row;
    for (int n = 0; ok && next_task(n, &k); ++n) {
      for (int u = k.u0; u < k.u1 && ok; ++seg) {
        const int tile = quick_div(u, k.len), tb = tile * k.len, te = tb + k.len, ue = min(te, k.u1);
        const bool mine = u == tb;   // this share starts the tile and so finishes it
        const int c1 = mine ? (k.gemm == 1 ? sh1 : sh2).of(te - 1) : k.share;
        const int b = seg & 1;
        // most parts are there before this share's own sum is: look for them first
        uint32_t pw[CB][2 * TG];
        if (k.gemm == 1) peek(part1, k.share + 1, c1, pw, std::integral_constant<int, 2 * TG>());
        else peek(part2, k.share + 1, c1, pw, std::integral_constant<int, TG>());
        if (!mbar_wait(&S.accf[b], (seg >> 1) & 1, deadline, abort_flag)) { fail(9); ok = false; break; }
        __syncwarp();
        tc_fence_after();
        const uint32_t acc = tl + b * 2 * NC;
        float v[2 * TG];   // gate of token t0 + t, then up; or out
        {
          float a[TG], c[TG], d[TG], e[TG];   // a token's two columns, of each accumulator
          tmem_ld(acc, a);
          tmem_ld(acc + MT, c);
          if (k.gemm == 1) {
            tmem_ld(acc + NC, d);
            tmem_ld(acc + NC + MT, e);
          }
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < TG; ++t) { v[t] = a[t] + c[t]; v[TG + t] = d[t] + e[t]; }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.acce[b]);
        if (k.gemm == 1) {
          if (!mine) {
            uint32_t* dst = part1 + k.share * (MAX_GROUPS * 2 * TG * 128);
#pragma unroll
            for (int i = 0; i < 2 * TG; ++i)
              if (live(i)) part_put(dst + i * 128, v[i]);
          } else {
            const Where w = where(tile);
            float wt[TG];   // routing weights; 0: the token did not choose the expert
#pragma unroll
            for (int t = 0; t < TG; ++t) wt[t] = w.shared && live(t) ? 1.0f : 0.0f;
            if (!w.shared) {
#pragma unroll
              for (int t = 0; t < TG; ++t) {
                const int c = S.choice[w.e][(t0 + t) & (MAX_M - 1)];
                if (c) wt[t] = S.wts[(t0 + t) * topk + c - 1];
              }
            }
            ok = gather(part1, k.share, c1, v, pw, std::integral_constant<int, 2 * TG>());
            if (!ok) break;
            float m[TG];
            int s[TG];
#pragma unroll
            for (int t = 0; t < TG; ++t) {
              const float r = S.rstd[min(t0 + t, MAX_M - 1)], g = v[t] * r, h = v[TG + t] * r;
              // past -80 the quotient's divisor would overflow; there silu(g) is g e^g
              const float x = __expf(g < -80.0f ? g : -g);
              const float silu = g < -80.0f ? g * x : __fdividef(g, 1.0f + x);
              m[t] = wt[t] != 0.0f ? wt[t] * (silu * h) : 0.0f;   // a select: an absent token's sums count for nothing
              // a block of 32 rows is this warp's rows of the tile
              s[t] = split_exp(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m[t]) & 0x7FFFFFFFu)));
              m[t] *= s[t] == SPLIT_NAN ? __int_as_float(0x7FC00000) : exp2i(-s[t]);
            }
            uint8_t* dst = p.mop + (int64_t)tile * C::B_TILE;
            uint8_t* sf = p.msf + (int64_t)tile * SF_BLOCK;
#pragma unroll
            for (int t = 0; t < TG; t += 2) {
              uint32_t hi, lo;
              split_f16x2(f16x2_of(m[t], m[TG > 1 ? t + 1 : t], 1.0f), hi, lo);
              if constexpr (WORDS) {
                // bytes of four rows (lanes) by four columns (hi and lo of two tokens),
                // transposed: a lane stores four rows of one column as one word
                uint32_t w = hi | lo << 16, o = __shfl_xor_sync(0xFFFFFFFFu, w, 2);
                w = lane & 2 ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
                o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
                w = lane & 1 ? __byte_perm(o, w, 0x7351) : __byte_perm(w, o, 0x6240);
                const int tok = t0 + t + (lane & 1), col = (lane & 2 ? MT : 0) + tok;
                if (!(p.test_withhold && tile == 0) && (TG > 1 || !(lane & 1)) && tok < M) {
                  word_put(reinterpret_cast<uint32_t*>(dst + tile_byte(col, row & ~3)), w);
                  if (lane < 4)   // this block of 32 rows' scale, a word of its own
                    word_put(reinterpret_cast<uint32_t*>(sf + 16 * col) + q,
                             static_cast<uint32_t>(lane & 2 ? split_code_lo(lane & 1 ? s[TG > 1 ? t + 1 : t] : s[t])
                                                            : split_code_hi(lane & 1 ? s[TG > 1 ? t + 1 : t] : s[t])));
                }
                continue;
              }
#pragma unroll
              for (int o = 0; o < min(2, TG); ++o)
                if (live(t + o)) {
                  dst[tile_byte(t0 + t + o, row)] = static_cast<uint8_t>(hi >> (8 * o));
                  dst[tile_byte(MT + t0 + t + o, row)] = static_cast<uint8_t>(lo >> (8 * o));
                  if (lane == 0) {
                    sf[sf_byte(t0 + t + o, q)] = static_cast<uint8_t>(split_code_hi(s[t + o]));
                    sf[sf_byte(MT + t0 + t + o, q)] = static_cast<uint8_t>(split_code_lo(s[t + o]));
                  }
                }
            }
            if constexpr (!WORDS) {
              __syncwarp();   // the release below covers the warp's stores
              if (lane == 0 && !(p.test_withhold && tile == 0)) red_release_gpu(p.sync + 1, 1);
            }
          }
        } else {
          if (!mine) {
            uint32_t* dst = part2 + k.share * (MAX_GROUPS * TG * 128);
#pragma unroll
            for (int i = 0; i < TG; ++i)
              if (live(i)) part_put(dst + i * 128, v[i]);
          } else {
            const int h = tile * 128 + row;
            float r[TG];
#pragma unroll
            for (int t = 0; t < TG; ++t)
              r[t] = p.residual && live(t) ? __uint_as_float((uint32_t)__ldcg(p.x + (t0 + t) * p.ldx + h) << 16) : 0.0f;
            ok = gather(part2, k.share, c1, v, pw, std::integral_constant<int, TG>());
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < TG; ++t)
              if (live(t)) p.out[(t0 + t) * p.ldo + h] = bf16_bits(v[t] + r[t]);
          }
        }
        u = ue;
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

static cudaLaunchConfig_t config(int grid, int threads, int smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int NC, int TG, bool WORDS>
static cudaError_t launch_experts(const CUtensorMap* m, const LayerParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = set_up_kernel(k_layer_experts<NC, TG, WORDS>, smem_bytes<NC>(), &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(grid, 128 + 128 * ((p.M + TG - 1) / TG), smem_bytes<NC>(), st, &attr);
  return cudaLaunchKernelEx(&cfg, k_layer_experts<NC, TG, WORDS>, m[0], m[1], m[2], m[3], p);
}

template <bool NORM, bool HIGH>
static cudaError_t launch_head(const LayerParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = set_up_kernel(k_layer_head<NORM, HIGH>, 0, &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const int chunks = (p.H / 128 + HEAD_SLICES - 1) / HEAD_SLICES * HEAD_SLICES;   // whole clusters
  const cudaLaunchConfig_t cfg = config((p.E + 7) / 8 * HEAD_SLICES + chunks, HEAD_THREADS, 0, st, &attr);
  return cudaLaunchKernelEx(&cfg, k_layer_head<NORM, HIGH>, p);
}

}  // namespace layer

cudaError_t launch_layer_w4(const CUtensorMap* maps, const LayerParams& p, int sms, cudaStream_t st) {
  using namespace layer;
  const cudaError_t e = p.norm_w ? (p.M > 8 ? launch_head<true, true>(p, st) : launch_head<true, false>(p, st))
                                 : (p.M > 8 ? launch_head<false, true>(p, st) : launch_head<false, false>(p, st));
  if (e != cudaSuccess) return e;
  if (p.M == 1) return launch_experts<16, 1, true>(maps, p, sms, st);
  if (p.M == 2) return launch_experts<16, 2, true>(maps, p, sms, st);
  if (p.M <= GROUP) return launch_experts<16, GROUP, true>(maps, p, sms, st);
  if (p.M <= 8) return launch_experts<16, GROUP, false>(maps, p, sms, st);
  return launch_experts<32, GROUP, false>(maps, p, sms, st);
}

}  // namespace moe
