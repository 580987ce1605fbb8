// layer.cu -- a whole mixture-of-experts layer for a few tokens (M <= 16) in
// two launches: RMS norm, router product, top-k, SwiGLU experts on MXFP4
// weights with bf16 activations, an always-used shared expert, the residual.
//
//   k_layer_head     two experts' router logits a CTA (fp32 products of bf16),
//                    the norm's statistics on the way, sigmoid and selection
//                    keys; and the tokens as tensor-core operand columns
//                    (w4.cuh) of x * norm weight.  The norm's 1 / rms is a factor
//                    of the token, applied to the sums.
//   k_layer_experts  one CTA an SM.  Each picks the top k from the keys (the same
//                    everywhere), then streams weights: GEMM1 over the selected
//                    experts' gate and up rows, SwiGLU, mid as operand columns
//                    scaled by the routing weight, and GEMM2, in which the experts
//                    follow one another along K: one accumulation per 128 rows of
//                    out is the routing-weighted sum over all experts (columns of
//                    tokens that did not choose an expert are zero).
//
// Bound: the selected experts' weight bytes.  Both products are cut into
// shares of equal bytes (as in linear.cu, parts of a cut tile meet in the share
// that starts it, in K order).  Shares are tasks that the CTAs draw from one
// counter, all of GEMM1 before all of GEMM2, and a task waits for earlier ones
// only, so the kernel ends however many of its CTAs run at once.  A CTA's
// weight stream runs ahead into its GEMM2 task while mid is still on its way.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "w4.cuh"

namespace moe {
namespace layer {

using namespace w4;

constexpr int HEAD_THREADS = 256;
constexpr int THREADS = 256;       // warps: 0 weights, 1 MMA, 2 operands, 3 routing only, 4-7 sums
constexpr int STAGES = 5;
constexpr int SF_SLOTS = 4;        // TMEM scale slots of 16 columns: two weight blocks, two operand blocks
constexpr int TASKS = 4;           // task ring
constexpr int MAX_M = 16;
constexpr int MAX_SLOTS = 256;     // distinct experts of a call: M * topk at most
constexpr int MIN_SHARE = 2;       // units a share holds at least (a share may not be empty)

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
  uint64_t full[STAGES], empty[STAGES], accf[2], acce[2], tfull[TASKS], tempty[TASKS];
  uint32_t tmem;
  int abort_flag, ndist;
  int task[TASKS];
  float rstd[MAX_M];
  int ids[MAX_M * kMaxTopk];
  float wts[MAX_M * kMaxTopk];
  uint8_t mark[kMaxE];
  uint16_t dlist[MAX_SLOTS];
};

template <int NC>
constexpr int smem_bytes() { return STAGES * Cfg<NC>::STAGE + (int)sizeof(Smem) + 1024; }
static_assert(smem_bytes<16>() <= 232448 && smem_bytes<32>() <= 232448, "shared memory");

// Sums of R values over the warp, value lane >> (5 - log2 R) in each lane.
template <int R>
__device__ __forceinline__ float warp_sums(float (&v)[R]) {
  const int lane = threadIdx.x & 31;
  int off = 16;
#pragma unroll
  for (int n = R / 2; n >= 1; n /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, off);
    }
  }
  float r = v[0];
#pragma unroll
  for (; off >= 1; off /= 2) r += __shfl_xor_sync(0xFFFFFFFFu, r, off);
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// MT: the tokens' accumulators a thread keeps (M rounded up to a power of two).
template <int MT>
__global__ void __launch_bounds__(HEAD_THREADS) k_layer_head(const LayerParams p) {
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) { p.sync[0] = 0; p.sync[1] = 0; }
  pdl_launch_dependents();
  const int M = p.M, H = p.H, E = p.E, KC = H / 128, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int e0 = 2 * blockIdx.x;

  // ---- the tokens' operand columns: 16 lanes a chunk of one token
  for (int kc = blockIdx.x; kc < KC; kc += gridDim.x) {
    const int t = tid >> 4, g8 = tid & 15, k = kc * 128 + g8 * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (t < M) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ldx + k)), v);
      if (p.norm_w) {
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm_w + k)), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= g[i];
      }
    }
    uint32_t am = 0;   // largest magnitude's bits; a NaN's are above an infinity's
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    if (t < M) {
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
  }
  if (e0 >= E && blockIdx.x != 0) return;

  // ---- two experts' logits and the sums of squares
  float dot[2 * MT], ss[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) { dot[2 * i] = dot[2 * i + 1] = 0.0f; ss[i] = 0.0f; }
  const uint16_t* r0 = p.router_w + (int64_t)min(e0, E - 1) * H;
  const uint16_t* r1 = p.router_w + (int64_t)min(e0 + 1, E - 1) * H;
#pragma unroll 2
  for (int k = tid * 8; k < H; k += HEAD_THREADS * 8) {
    float a[8], b[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(r0 + k)), a);
    unpack8(__ldg(reinterpret_cast<const uint4*>(r1 + k)), b);
    if (p.norm_w) {
      float g[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm_w + k)), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) { a[i] *= g[i]; b[i] *= g[i]; }   // exact: 8-bit significands
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (t >= M) break;
      float v[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ldx + k)), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot[2 * t] = fmaf(v[i], a[i], dot[2 * t]);
        dot[2 * t + 1] = fmaf(v[i], b[i], dot[2 * t + 1]);
        ss[t] = fmaf(v[i], v[i], ss[t]);
      }
    }
  }
  __shared__ float sd[8][2 * MT], sq[8][MT];
  const float d = warp_sums(dot), q = warp_sums(ss);
  if (lane % (32 / (2 * MT)) == 0) sd[warp][lane / (32 / (2 * MT))] = d;
  if (lane % (32 / MT) == 0) sq[warp][lane / (32 / MT)] = q;
  __syncthreads();
  if (tid < 2 * M) {
    const int t = tid >> 1, e = e0 + (tid & 1);
    float dsum = 0.0f, qsum = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) { dsum += sd[w][tid]; qsum += sq[w][t]; }
    const float rstd = p.norm_w ? 1.0f / sqrtf(qsum / (float)H + p.eps) : 1.0f;
    if (e < E) {
      const float sg = sigmoid_spec(dsum * rstd);
      p.sig[t * E + e] = sg;
      p.key[t * E + e] = float_order_key(p.bias ? __fadd_rn(sg, __ldg(p.bias + e)) : sg);
    }
    if (blockIdx.x == 0 && (tid & 1) == 0) p.rstd[t] = rstd;
  }
}

// The top k of one token from its selection keys, a warp: k rounds, a tie
// going to the lower expert; weights as in route_token_warp.
template <int KPER>
__device__ __forceinline__ void pick(const uint32_t* keys, const float* sig, int E, int k, float scale, int* ids,
                                     float* wts) {
  const int lane = threadIdx.x & 31;
  uint32_t key[KPER];
  float sg[KPER];
#pragma unroll
  for (int i = 0; i < KPER; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < E ? __ldcg(keys + e) : 0u;
    sg[i] = e < E ? __ldcg(sig + e) : 0.0f;
  }
  float denom = 0.0f, mine = 0.0f;
  int id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int bi = 0;
    float bs = sg[0];
#pragma unroll
    for (int i = 1; i < KPER; ++i)
      if (key[i] > best) { best = key[i]; bi = i; bs = sg[i]; }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const int e = (int)__reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)(lane + 32 * bi) : 0xFFFFFFFFu);
    const float s = __shfl_sync(0xFFFFFFFFu, bs, e & 31);
#pragma unroll
    for (int i = 0; i < KPER; ++i)
      if (lane + 32 * i == e) key[i] = 0u;   // taken (below every key of a number or a NaN)
    denom = __fadd_rn(denom, s);
    if (lane == j) { id = e; mine = s; }
  }
  if (lane < k) {
    ids[lane] = id;
    wts[lane] = __fmul_rn(__fdiv_rn(mine, denom), scale);
  }
}

template <int NC>
__global__ void __launch_bounds__(THREADS, 1)
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

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&S.full[s], 2); mbar_init(&S.empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&S.accf[b], 1); mbar_init(&S.acce[b], 4); }
    for (int t = 0; t < TASKS; ++t) { mbar_init(&S.tfull[t], 1); mbar_init(&S.tempty[t], 6); }
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmW13); tma_prefetch_desc(&tmW2);
    if (JS) { tma_prefetch_desc(&tmS13); tma_prefetch_desc(&tmS2); }
  }
  if (warp == 4) { tmem_alloc(&S.tmem, C::TMEM_COLS); tmem_relinquish(); }
  for (int e = threadIdx.x; e < E; e += THREADS) S.mark[e] = 0;
  pdl_wait();   // k_layer_head is done
  pdl_launch_dependents();
  int ticket = 0;
  if (threadIdx.x == 0) ticket = atomicAdd(p.sync, 1);   // in flight while routing runs
  for (int t = warp; t < M; t += THREADS / 32) {
    if (E <= 256) pick<8>(p.key + t * E, p.sig + t * E, E, topk, p.scale, S.ids + t * topk, S.wts + t * topk);
    else pick<kMaxE / 32>(p.key + t * E, p.sig + t * E, E, topk, p.scale, S.ids + t * topk, S.wts + t * topk);
  }
  if (threadIdx.x < M) S.rstd[threadIdx.x] = __ldcg(p.rstd + threadIdx.x);
  __syncthreads();
  for (int q = threadIdx.x; q < M * topk; q += THREADS) {
    S.mark[S.ids[q]] = 1;
    if (blockIdx.x == 0) {
      if (p.ids_out) p.ids_out[q] = S.ids[q];
      if (p.wts_out) p.wts_out[q] = S.wts[q];
    }
  }
  __syncthreads();
  if (warp == 0) {   // the selected experts, ascending
    int n = 0;
    for (int e = lane; e < (E + 31) / 32 * 32; e += 32) {
      const bool on = e < E && S.mark[e];
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
      if (on) S.dlist[n + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(e);
      n += __popc(m);
    }
    if (lane == 0) S.ndist = n;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem, 0);
  const uint64_t deadline = globaltimer() + p.timeout_ns;
  // GEMM1: tile i (a gate and an up tile; the shared expert's first) is chunk i
  // of GEMM2's K.  A unit is 128 K of a GEMM1 tile or two chunks of a GEMM2 tile.
  const int tiles1 = JS + S.ndist * J, CU = (tiles1 + 1) / 2;
  const int64_t U1 = (int64_t)tiles1 * KC, U2 = (int64_t)HT * CU;
  const int G = gridDim.x;
  const int S1 = (int)min((int64_t)G, (U1 + MIN_SHARE - 1) / MIN_SHARE), S2 = (int)min((int64_t)G, (U2 + MIN_SHARE - 1) / MIN_SHARE);
  struct Where { int e, j, iw; bool shared; };
  auto where = [&](int i) -> Where {
    if (i < JS) return {0, i, JS, true};
    const int r = i - JS, slot = r / J;
    return {(int)S.dlist[slot], r - slot * J, J, false};
  };
  auto fail = [&](int site) {
    *abort_flag = 1;
    atomicOr(p.status, ST_TIMEOUT);
    atomicCAS(p.status + 2, 0, (int)(0x80000000u | (9u << 24) | ((unsigned)site << 20) | (blockIdx.x & 0xFFFu)));
  };
  auto drain = [&]() { const uint64_t until = globaltimer() + 2000000ull; while (globaltimer() < until) { } };
  // Ticket -> product (1, 2; 0: no more tasks), its units [u0, u1), units per tile, share, shares.
  struct Task { int gemm, share, shares, len; int64_t total, u0, u1; };
  auto task_of = [&](int t) -> Task {
    Task k;
    if (t < S1) k = {1, S1 - 1 - t, S1, KC, U1, 0, 0};   // a share waits for later ones: they are drawn before it
    else if (t < S1 + S2) k = {2, S2 - 1 - (t - S1), S2, CU, U2, 0, 0};
    else return {0, 0, 1, 1, 0, 0, 0};
    k.u0 = share_begin(k.total, k.shares, k.share);
    k.u1 = share_begin(k.total, k.shares, k.share + 1);
    return k;
  };
  // The other roles take the tasks in the order that the weight stream drew them.
  auto next_task = [&](int n, Task* k) -> bool {   // a whole warp
    if (!mbar_wait(&S.tfull[n % TASKS], (n / TASKS) & 1, deadline, abort_flag)) { fail(1); return false; }
    __syncwarp();
    const int t = S.task[n % TASKS];
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.tempty[n % TASKS]);
    *k = task_of(t);
    return k->gemm != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------ weights and their scales
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!mbar_wait(&S.tempty[n % TASKS], ((n / TASKS) & 1) ^ 1, deadline, abort_flag)) { fail(2); ok = false; break; }
        S.task[n % TASKS] = ticket;
        mbar_arrive(&S.tfull[n % TASKS]);
        const Task k = task_of(ticket);
        if (!k.gemm) break;
        ticket = atomicAdd(p.sync, 1);
        int tile = static_cast<int>(k.u0 / k.len), i = static_cast<int>(k.u0 - (int64_t)tile * k.len);
        Where w = where(k.gemm == 1 ? tile : 0);
        for (int64_t u = k.u0; u < k.u1; ++u) {
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
      if (!ok) drain();
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
      int i = static_cast<int>(k.u0 % k.len);
      bool first = true;
      const int nu = static_cast<int>(k.u1 - k.u0);
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
  } else if (warp == 2) {
    // ------------------------------------------------ operand columns: the tokens', then mid's
    int st = 0;
    uint32_t ph = 0;
    bool ok = true, mid_ready = false;
    Task k;
    fence_proxy_async_global();   // k_layer_head's stores, read by bulk copies
    for (int n = 0; ok && (ok = next_task(n, &k)); ++n) {
      if (k.gemm == 2 && !mid_ready) {
        // every GEMM1 tile's four warps have stored their quarter of mid
        uint32_t spins = 0;
        while (ld_acquire_gpu(p.sync + 1) < 4 * tiles1) {
          if ((++spins & 15u) == 0 && (*abort_flag || globaltimer() > deadline)) { fail(6); ok = false; break; }
        }
        if (!ok) break;
        __syncwarp();
        fence_proxy_async_global();
        mid_ready = true;
      }
      if (lane == 0) {
        int i = static_cast<int>(k.u0 % k.len);
        for (int64_t u = k.u0; u < k.u1; ++u) {
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
  } else if (warp >= 4) {
    // ------------------------------------------------ sums
    const int q = warp - 4, row = 32 * q + lane;   // TMEM lane quarter = warp % 4
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16);
    int seg = 0;
    bool ok = true;
    Task k;
    // adds the later shares' parts [share + 1, c1] of NV values per row, in K order, to v
    auto gather = [&](uint32_t* part, int share, int c1, auto& v, auto nv_const, auto live) -> bool {
      constexpr int NV = decltype(nv_const)::value, CB = 64 / NV;
#pragma unroll 1
      for (int cb = share + 1; cb <= c1; cb += CB) {
        uint32_t w[CB][NV];
        uint32_t spins = 0;
        for (;;) {
          bool all = true;
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            const uint32_t* src = part + (int64_t)min(cb + c, c1) * (NV * 128) + row;
#pragma unroll
            for (int i = 0; i < NV; ++i) w[c][i] = live(i) ? part_peek(src + i * 128) : 1u;
          }
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int i = 0; i < NV; ++i) all &= w[c][i] != 0u;
          if (all) break;
          if ((++spins & 15u) == 0 && (*abort_flag || globaltimer() > deadline)) { fail(8); return false; }
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          if (cb + c > c1) break;
          uint32_t* src = part + (int64_t)(cb + c) * (NV * 128) + row;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            v[i] += part_value(w[c][i]);
            if (live(i)) __stcg(src + i * 128, 0u);   // empty again for the next call
          }
        }
      }
      return true;
    };
    for (int n = 0; ok && next_task(n, &k); ++n) {
      for (int64_t u = k.u0; u < k.u1 && ok; ++seg) {
        const int tile = static_cast<int>(u / k.len);
        const int64_t t0 = (int64_t)tile * k.len, t1 = t0 + k.len, ue = min(t1, k.u1);
        const bool mine = u == t0;   // this share starts the tile and so finishes it
        const int c1 = mine ? share_of(k.total, k.shares, t1 - 1) : k.share;
        const int b = seg & 1;
        if (!mbar_wait(&S.accf[b], (seg >> 1) & 1, deadline, abort_flag)) { fail(9); ok = false; break; }
        __syncwarp();
        tc_fence_after();
        const uint32_t acc = tl + b * 2 * NC;
        // sum over a token's two columns
        auto read = [&](uint32_t col, float* v) {
          float a[16], c[16];
          tmem_ld16(col, a);
          if constexpr (NC == 32) tmem_ld16(col + MT, c);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < MT; ++t) v[t] = a[t] + (NC == 32 ? c[t] : a[(MT + t) & 15]);
        };
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.acce[b]);
        };
        if (k.gemm == 1) {
          float v[2 * MT];   // gate of token t, then up
          read(acc, v);
          read(acc + NC, v + MT);
          release();
          auto live = [&](int i) { return (i & (MT - 1)) < M; };
          if (!mine) {
            uint32_t* dst = p.part1 + (int64_t)k.share * (2 * MT * 128) + row;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
              if (live(i)) part_put(dst + i * 128, v[i]);
          } else {
            if (!gather(p.part1, k.share, c1, v, std::integral_constant<int, 2 * MT>(), live)) { ok = false; break; }
            const Where w = where(tile);
            uint8_t* dst = p.mop + (int64_t)tile * C::B_TILE;
            uint8_t* sf = p.msf + (int64_t)tile * SF_BLOCK;
#pragma unroll
            for (int t = 0; t < MT; t += 2) {
              if (t >= M) break;
              float m[2];
              int s[2];
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                const int tt = t + o;
                float wt = tt < M && w.shared ? 1.0f : 0.0f;
                if (tt < M && !w.shared)
                  for (int j = 0; j < topk; ++j)
                    if (S.ids[tt * topk + j] == w.e) wt = S.wts[tt * topk + j];
                float x = 0.0f;   // a token that did not choose the expert: zero, whatever its sums
                if (tt < M && (w.shared || wt != 0.0f)) {
                  const float r = S.rstd[tt], g = v[tt] * r, h = v[MT + tt] * r;
                  x = wt * (g / (1.0f + expf(-g)) * h);
                }
                const uint32_t am = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
                s[o] = split_exp(__uint_as_float(am));
                m[o] = x * (s[o] == SPLIT_NAN ? __int_as_float(0x7FC00000) : exp2i(-s[o]));
              }
              uint32_t hi, lo;
              split_f16x2(f16x2_of(m[0], m[1], 1.0f), hi, lo);
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                const int tt = t + o;
                if (tt >= M) break;
                dst[tile_byte(tt, row)] = static_cast<uint8_t>(hi >> (8 * o));
                dst[tile_byte(MT + tt, row)] = static_cast<uint8_t>(lo >> (8 * o));
                if (lane == 0) {
                  sf[sf_byte(tt, q)] = static_cast<uint8_t>(split_code_hi(s[o]));
                  sf[sf_byte(MT + tt, q)] = static_cast<uint8_t>(split_code_lo(s[o]));
                }
              }
            }
            __threadfence();
            __syncwarp();
            if (lane == 0 && !(p.test_withhold && tile == 0)) atomicAdd(p.sync + 1, 1);
          }
        } else {
          float v[MT];
          read(acc, v);
          release();
          auto live = [&](int i) { return i < M; };
          if (!mine) {
            uint32_t* dst = p.part2 + (int64_t)k.share * (MT * 128) + row;
#pragma unroll
            for (int i = 0; i < MT; ++i)
              if (live(i)) part_put(dst + i * 128, v[i]);
          } else {
            if (!gather(p.part2, k.share, c1, v, std::integral_constant<int, MT>(), live)) { ok = false; break; }
            const int h = tile * 128 + row;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              if (t >= M) break;
              float y = v[t];
              if (p.residual) y += __uint_as_float((uint32_t)__ldg(p.x + (int64_t)t * p.ldx + h) << 16);
              p.out[(int64_t)t * p.ldo + h] = bf16_bits(y);
            }
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

template <int NC>
static cudaError_t launch_experts(const CUtensorMap* m, const LayerParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may take its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    e = cudaFuncSetAttribute(k_layer_experts<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NC>());
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(grid, THREADS, smem_bytes<NC>(), st, &attr);
  return cudaLaunchKernelEx(&cfg, k_layer_experts<NC>, m[0], m[1], m[2], m[3], p);
}

}  // namespace layer

cudaError_t launch_layer_w4(const CUtensorMap* maps, const LayerParams& p, int sms, cudaStream_t st) {
  using namespace layer;
  const int head = std::max((p.E + 1) / 2, std::min(p.H / 128, sms));
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(head, HEAD_THREADS, 0, st, &attr);
  cudaError_t e;
  if (p.M == 1) e = cudaLaunchKernelEx(&cfg, k_layer_head<1>, p);
  else if (p.M == 2) e = cudaLaunchKernelEx(&cfg, k_layer_head<2>, p);
  else if (p.M <= 4) e = cudaLaunchKernelEx(&cfg, k_layer_head<4>, p);
  else if (p.M <= 8) e = cudaLaunchKernelEx(&cfg, k_layer_head<8>, p);
  else e = cudaLaunchKernelEx(&cfg, k_layer_head<16>, p);
  if (e != cudaSuccess) return e;
  return p.nc == 16 ? launch_experts<16>(maps, p, sms, st) : launch_experts<32>(maps, p, sms, st);
}

}  // namespace moe
