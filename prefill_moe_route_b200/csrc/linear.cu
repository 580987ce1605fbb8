// linear.cu -- y = x W^T (+ bias) for few tokens: MXFP4 weights, bf16
// activations, fp32 sums, one launch (two above 8 tokens, and on large weights above 4).
//
// Bound: the weights' bytes (1 x 40003 x 6144: 24.4 us, 5.4 TB/s, in a burst of 24 calls
// 22.7; 4 x 12288 x 6144: 9.9 us, 4.0 TB/s), behind some 3 us of start, parts and end;
// from about 32 tokens the tiles' way in and out of shared memory.  All times in this
// file are those of calls replayed from a CUDA graph, several matrices in turn; calls
// made one by one take 0.2 to 0.5 us more each, the smallest 4.8 us instead of 2.6 (the
// host).  The product runs on the
// tensor cores with the weights on the MMA's M side straight from their packed
// 4-bit form (no dequantization) and the tokens as 2 columns each (w4.cuh).  The
// K-chunks of all row tiles are one sequence of units (128 rows x 256 K, 17 KB)
// that the CTAs, one per SM, share evenly: every SM streams the same bytes
// whatever the shape.  Where a tile is cut between shares, the share that starts it adds the
// others' parts in K order (so results do not depend on timing); those are the
// first thing that their CTAs finish, and the starting share's last.
//
// Roles: one thread streams tiles (TMA) and their scale blocks (bulk copy), a
// warp for each token splits its K chunks into the operand ring (with two launches
// k_split_x does it before, and the stream brings them), one thread issues the
// MMAs, four warps for every 8 tokens (16 of the largest tile) read the sums out
// of TMEM.
#include "w4.cuh"

namespace moe {
namespace linear {

using namespace w4;

// x and bias are read through L2 (__ldcg): a block can be resident before the
// kernel that writes them has ended.

constexpr int WARP_SPLIT0 = 2;
constexpr int UK = 2;               // K chunks of 128 in a unit
constexpr int SF_SLOTS = 4;         // TMEM scale slots: per chunk 4 columns of weight scales + 4 of token scales

// NC: operand columns, two per token.  SW: warps that split the tokens' K chunks
// in the kernel; 0: k_split_x has done it before.  Measured (us, N = K = 6144, 8
// split warps / 16, a variant that is not kept / before): 4 tokens 6.9 / 7.4 / 8.1, 8 tokens 7.8 / 7.8 / 8.3 (7 x
// 4099 x 2912: 5.2 / 5.6 / 6.1), 16 tokens - / 9.2 / 8.2 (N = 12288: - / 13.4 / 11.4).
template <int NC, int SW>
struct Cfg {
  static constexpr int MT = NC / 2;
  static constexpr bool PRE = SW == 0;
  static constexpr int WARP_EPI0 = WARP_SPLIT0 + (PRE ? 2 : SW);   // the two are idle: TMEM quarters
  // the sums of 8 tokens (of a tile of 64: 16) a group of four warps: one after
  // another their trips through L2 would add up (16 x 6144 x 6144, one group / two:
  // 8.9 / 8.2 us; 32 x 6144 x 6144, two / four: 9.7 / 9.3)
  static constexpr int EG = MT >= 32 ? 4 : MT / 8, ET = MT / EG;
  static constexpr int THREADS = (WARP_EPI0 + 4 * EG) * 32;
  static constexpr int B_TILE = NC * 128;
  static constexpr int A_BYTES = UK * A_TILE, B_BYTES = UK * B_TILE, SF_BYTES = UK * SF_BLOCK;
  static constexpr int STAGE = A_BYTES + B_BYTES + 2 * SF_BYTES;   // weights, tokens, their scales
  static constexpr int STAGES = NC >= 128 ? 3 : NC >= 64 ? 4 : 5;   // as many as fit
  // units of a share sent for L2 before the kernel may read: a round of the ring (more
  // is slower: 8, 12, 16 units of 1 x 6144 x 6144), and where k_split_x comes first
  // and leaves the time, more (us, 8 / 5 / none: 16 x 6144 x 6144 8.9 / 9.2 / 9.8,
  // 32 x 6144 x 12288 13.3 / 13.2 / 13.5)
  static constexpr int AHEAD = NC == 32 ? 8 : 5;
  static constexpr int TMEM_COLS = NC >= 128 ? 512 : 256;
  static constexpr int SF_COL0 = 2 * NC;
};

struct Smem {
  uint64_t full[8], empty[8], accf[2], acce[2];
  uint32_t tmem;
  int abort_flag;
};

template <int NC, int SW>
constexpr int smem_bytes() {
  static_assert(Cfg<NC, SW>::STAGES * Cfg<NC, SW>::STAGE + sizeof(Smem) + 1024 <= 232448, "shared memory");
  return Cfg<NC, SW>::STAGES * Cfg<NC, SW>::STAGE + (int)sizeof(Smem) + 1024;
}

// Limit of one wait.  Its clock starts when the wait has been polled for a while,
// not with the kernel: a large call takes longer than a wait may, and the blocks of
// one can be resident long before the kernel in front of them ends.
struct Limit {
  uint64_t until = 0;
  __device__ __forceinline__ bool over(uint64_t timeout_ns) {
    const uint64_t now = globaltimer();
    if (until == 0) until = now + timeout_ns;
    return now > until;
  }
};
// Bounded wait: false once the limit has passed or another role of the CTA has given up.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
  uint32_t spins = 0;
  Limit limit;
  while (!mbar_try_wait(bar, parity))
    if ((++spins & 255u) == 0 && (*abort_flag || limit.over(timeout_ns))) return false;
  return true;
}

// 8 values of a token's K chunk: 8 bf16 in, 8 bytes of both operand columns (n, n
// + mt) out; four neighbouring lanes hold a block of 32.
__device__ __forceinline__ void split_item(const uint4& u, uint8_t* tile, uint8_t* sf, int n, int mt, int g8) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t am = 0;   // largest magnitudes as bf16 bits
#pragma unroll
  for (int i = 0; i < 4; ++i) am = max_u16x2(am, w[i] & 0x7FFF7FFFu);
  am = max(am & 0xFFFFu, am >> 16);
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  const int s = split_exp(__uint_as_float(am << 16));
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_f16x2(s == SPLIT_NAN ? 0x7E007E00u : f16x2_scaled(w[i], s), hi[i], lo[i]);
  *reinterpret_cast<uint2*>(tile + tile_byte(n, g8 * 8)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
  *reinterpret_cast<uint2*>(tile + tile_byte(mt + n, g8 * 8)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  if ((g8 & 3) == 0) {
    sf[sf_byte(n, g8 >> 2)] = static_cast<uint8_t>(split_code_hi(s));
    sf[sf_byte(mt + n, g8 >> 2)] = static_cast<uint8_t>(split_code_lo(s));
  }
}

// A share's first units start for L2 while the kernel before this call ends (a
// prefetch only: what that kernel writes stays what is read).  1 x 6144 x 6144:
// 7.4 us without, 6.8 with.
__device__ __forceinline__ void prefetch_weights(const LinearParams& p, int share, int ahead) {
  const int u0 = p.shares.begin(share), n = min(p.shares.begin(share + 1) - u0, ahead);
  int tile = u0 / p.KU, ku = u0 - tile * p.KU;
  for (int i = 0; i < n; ++i) {
    const int64_t blk = (int64_t)(tile / p.TT) * p.KC + ku * UK;
    const int nk = min(UK, p.KC - ku * UK);
    prefetch_l2_bulk(p.wcodes + blk * CODE_BLOCK, nk * CODE_BLOCK);
    prefetch_l2_bulk(p.wsf + blk * SF_BLOCK, nk * SF_BLOCK);
    if (++ku == p.KU) { ku = 0; ++tile; }
  }
}

template <int NC, int SW>
__global__ void __launch_bounds__(Cfg<NC, SW>::THREADS, 1)
k_linear_w4(const __grid_constant__ CUtensorMap tmW, const LinearParams p) {
  using C = Cfg<NC, SW>;
  constexpr int MT = C::MT, WARP_EPI0 = C::WARP_EPI0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* abuf = base;                                   // [STAGES][A_BYTES]
  uint8_t* bbuf = abuf + C::STAGES * C::A_BYTES;          // [STAGES][B_BYTES]
  uint8_t* asf = bbuf + C::STAGES * C::B_BYTES;           // [STAGES][SF_BYTES]
  uint8_t* bsf = asf + C::STAGES * C::SF_BYTES;           // [STAGES][SF_BYTES]
  Smem& S = *reinterpret_cast<Smem*>(bsf + C::STAGES * C::SF_BYTES);
  volatile int* abort_flag = &S.abort_flag;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = gridDim.x, share = G - 1 - blockIdx.x;   // a share waits for later ones only, which blocks launched before it hold
  const int KU = p.KU, TT = p.TT;
  const Shares sh = p.shares;
  const int u0 = sh.begin(share), u1 = sh.begin(share + 1), nu = u1 - u0;
  // warps that share one unit's split, one for a token; the groups of them, four at
  // most, must not outnumber the stages (one two rounds ahead of the MMA would read
  // a slot's old phase)
  const int gw = p.M <= 2 ? 2 : p.M <= 4 ? 4 : 8;
  static_assert(C::PRE || SW / 2 <= C::STAGES, "ring depth");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) { mbar_init(&S.full[s], C::PRE ? 1 : 1 + gw); mbar_init(&S.empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&S.accf[b], 1); mbar_init(&S.acce[b], 4 * C::EG); }
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmW);
    prefetch_weights(p, share, C::AHEAD);
  }
  if (warp == WARP_EPI0) { tmem_alloc(&S.tmem, C::TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Nothing above touches global memory but to send it for L2.  Each role works
  // out what it can and then waits for the kernel before this one (0.4 us of the
  // call otherwise); k_split_x waits for the kernel before the call first.
  pdl_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem, 0);
  auto fail = [&](uint32_t site) { wait_ran_out(p.status, abort_flag, 8u << 24 | site << 20); };
  auto drain = [&]() { const uint64_t until = globaltimer() + 2000000ull; while (globaltimer() < until) { } };

  if (warp == 0) {
    // ------------------------------------------------ weights, their scales, ready-made operands
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      const int tile0 = u0 / KU;
      auto next = [&](int& rt, int& tt, int& ku) {
        if (++ku == KU) { ku = 0; if (++tt == TT) { tt = 0; ++rt; } }
      };
      auto weights = [&](int s, int rt, int ku) {
        const int64_t blk = (int64_t)rt * p.KC + ku * UK;
        const int nk = min(UK, p.KC - ku * UK);
        // 4-bit tiles land unpacked.  A box holds UK chunks; a tile's odd last
        // chunk brings its neighbour's first along (zeros past the matrix).
        mbar_arrive_expect_tx(&S.full[s], UK * CODE_BLOCK + nk * (SF_BLOCK + (C::PRE ? C::B_TILE + SF_BLOCK : 0)));
        tma_load_2d(abuf + s * C::A_BYTES, &tmW, &S.full[s], 0, static_cast<int>(blk * 128));
        bulk_load(asf + s * C::SF_BYTES, p.wsf + blk * SF_BLOCK, nk * SF_BLOCK, &S.full[s]);
      };
      auto operand = [&](int s, int tt, int ku) {
        const int64_t blk = (int64_t)tt * p.KC + ku * UK;
        const int nk = min(UK, p.KC - ku * UK);
        bulk_load(bbuf + s * C::B_BYTES, p.xop + blk * C::B_TILE, nk * C::B_TILE, &S.full[s]);
        bulk_load(bsf + s * C::SF_BYTES, p.xsf + blk * SF_BLOCK, nk * SF_BLOCK, &S.full[s]);
      };
      int rt = tile0 / TT, tt = tile0 - rt * TT, ku = u0 - tile0 * KU;
      have(rt); have(tt); have(ku);
      pdl_wait();
      for (int i = 0; i < nu; ++i) {
        if (!bar_wait(&S.empty[st], ph ^ 1, p.timeout_ns, abort_flag)) { fail(1); ok = false; break; }
        weights(st, rt, ku);
        if (C::PRE) operand(st, tt, ku);
        if (++st == C::STAGES) { st = 0; ph ^= 1; }
        next(rt, tt, ku);
      }
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
    int ku = u0 % KU;
    bool first = true;
    pdl_wait();   // nothing to read here, but until the kernel before ends a still ring is no wait of this call
    for (int i = 0; i < nu; ++i) {
      const int b = seg & 1;
      if (first && !bar_wait(&S.acce[b], ((seg >> 1) & 1) ^ 1, p.timeout_ns, abort_flag)) { fail(2); ok = false; break; }
      if (!bar_wait(&S.full[st], ph, p.timeout_ns, abort_flag)) { fail(3); ok = false; break; }
      __syncwarp();
      tc_fence_after();
      const uint32_t d = tmem + b * NC;
      const int nk = min(UK, p.KC - ku * UK);
      const bool last = ku + 1 == KU || i + 1 == nu;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < UK; ++kk) {
          if (kk >= nk) break;
          const uint32_t sfa = tmem + C::SF_COL0 + ((slot + kk) % SF_SLOTS) * 8, sfb = sfa + 4;
          tc_cp_sf(sfa, sdesc_sf(smem_u32(asf + st * C::SF_BYTES + kk * SF_BLOCK)));
          tc_cp_sf(sfb, sdesc_sf(smem_u32(bsf + st * C::SF_BYTES + kk * SF_BLOCK)));
          const uint32_t a0 = smem_u32(abuf + st * C::A_BYTES + kk * A_TILE);
          const uint32_t b0 = smem_u32(bbuf + st * C::B_BYTES + kk * C::B_TILE);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_mxf8f6f4(d, sdesc_sw128(a0 + ks * 32), sdesc_sw128(b0 + ks * 32), idesc_with_sf(IDESC, ks, ks), sfa, sfb,
                         !(first && kk == 0 && ks == 0));
        }
        tc_commit(&S.empty[st]);
        if (last) tc_commit(&S.accf[b]);
      }
      __syncwarp();
      slot = (slot + UK) % SF_SLOTS;
      first = last;
      if (last) ++seg;
      if (++st == C::STAGES) { st = 0; ph ^= 1; }
      if (++ku == KU) ku = 0;
    }
    if (!ok) drain();
    __syncwarp();
  } else if (warp < WARP_EPI0) {
    if constexpr (!C::PRE) {
    // ------------------------------------------------ token operand
    // A lane owns 8 of the unit's 256 K, a warp of the unit's gw one token (all fit one token tile).
    const int sw = warp - WARP_SPLIT0, grp = sw / gw, ngrp = SW / gw, t = sw % gw;
    const int kk = lane >> 4, g8 = lane & 15;
    constexpr int PD = 2;   // a warp's loads in flight (more is more cold code; us, 2 / 4: 7 x 4099 x 2912 5.0 / 5.2,
                            // 1 x 512 x 512 2.7 / 2.8, 8 x 12288 x 6144 11.6 / 11.4)
    int ku = (u0 + grp) % KU;
    auto load = [&]() -> uint4 {   // and on to this group's next unit
      const int k = ku * (UK * 128) + lane * 8;
      ku += ngrp;
      while (ku >= KU) ku -= KU;
      return t < p.M && k < p.K ? __ldcg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ldx + k))
                                : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 buf[PD];
    have(ku);
    pdl_wait();
#pragma unroll
    for (int d = 0; d < PD; ++d) buf[d] = load();
    bool ok = true;
    for (int i0 = grp; i0 < nu && ok; i0 += PD * ngrp) {
#pragma unroll
      for (int d = 0; d < PD; ++d) {
        const int i = i0 + d * ngrp;
        if (i >= nu) break;
        const int st = i % C::STAGES;
        if (!bar_wait(&S.empty[st], ((i / C::STAGES) & 1) ^ 1, p.timeout_ns, abort_flag)) { fail(5); ok = false; break; }
        __syncwarp();
        split_item(buf[d], bbuf + st * C::B_BYTES + kk * C::B_TILE, bsf + st * C::SF_BYTES + kk * SF_BLOCK, t, MT, g8);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.full[st]);
        buf[d] = load();
      }
    }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ sums
    const int q = warp & 3, row = 32 * q + lane;   // TMEM lane quarter = warp % 4
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16);
    constexpr int TB = 8;                   // tokens per step
    // Parts looked for at once.  Two keep the 640 threads of the larger tiles near 64
    // registers, and blocks of the next call's k_split_x start beside this one (us,
    // 4 / 2: 32 x 6144 x 12288 14.4 / 12.9, 64 x 6144 x 6144 13.3 / 12.1; 16 x 6144 x
    // 6144 8.2 / 8.3).
    constexpr int CB = MT >= 32 ? 2 : 4;
    const int g0 = (warp - WARP_EPI0) / 4 * C::ET;   // this group's tokens of the tile
    pdl_wait();
    int seg = 0;
    bool ok = true;
    for (int u = u0; u < u1 && ok; ++seg) {
      const int tile = u / KU, t0 = tile * KU, t1 = t0 + KU, ue = min(t1, u1);
      const int rt = tile / TT, tt = tile - rt * TT;
      const int m = min(min(MT, p.M - tt * MT), g0 + C::ET), n = rt * 128 + row;
      const bool mine = u == t0;                           // this share starts the tile and so finishes it
      const int c1 = mine ? sh.of(t1 - 1) : share;   // shares after this one that hold parts of it
      const int b = seg & 1;
      const float bv = (p.bias && n < p.N) ? __ldcg(p.bias + n) : 0.0f;
      // parts cb .. of tokens tb .. tb + TB - 1
      uint32_t w[CB][TB];
      auto peek = [&](int cb, int tb) {
#pragma unroll
        for (int i = 0; i < CB; ++i) {
          const uint32_t* src = p.part + ((int64_t)(cb + i) * MT + tb) * 128 + row;
#pragma unroll
          for (int t = 0; t < TB; ++t) w[i][t] = cb + i <= c1 && tb + t < m ? part_peek(src + t * 128) : 1u;
        }
      };
      if (g0 < m) peek(share + 1, g0);   // most are there before this share's own sum is
      if (!bar_wait(&S.accf[b], (seg >> 1) & 1, p.timeout_ns, abort_flag)) { fail(7); break; }
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int tb = g0; tb < m && ok; tb += TB) {
        float v[TB];
        {
          float a[8], c[8];
          tmem_ld(tl + b * NC + tb, a);
          tmem_ld(tl + b * NC + MT + tb, c);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < TB; ++t) v[t] = a[t] + c[t];
        }
        if (!mine) {
          uint32_t* dst = p.part + ((int64_t)share * MT + tb) * 128 + row;
#pragma unroll
          for (int t = 0; t < TB; ++t)
            if (tb + t < m && !(p.test_withhold && share == G - 1)) part_put(dst + t * 128, v[t]);
          continue;
        }
        uint32_t spins = 0;
        Limit limit;
#pragma unroll 1
        for (int cb = share + 1; cb <= c1;) {   // the later shares' parts, in K order
          bool all = true;
#pragma unroll
          for (int i = 0; i < CB; ++i)
#pragma unroll
            for (int t = 0; t < TB; ++t) all &= w[i][t] != 0u;
          if (all) {
#pragma unroll
            for (int i = 0; i < CB; ++i) {
              if (cb + i > c1) break;
              uint32_t* src = p.part + ((int64_t)(cb + i) * MT + tb) * 128 + row;
#pragma unroll
              for (int t = 0; t < TB; ++t) {
                v[t] += part_value(w[i][t]);
                if (tb + t < m) __stcg(src + t * 128, 0u);   // empty again for the next call
              }
            }
            cb += CB;
            if (cb > c1) break;
            limit = Limit();
          } else if ((++spins & 15u) == 0 && (*abort_flag || limit.over(p.timeout_ns))) {
            fail(8);
            ok = false;
            break;
          }
          peek(cb, tb);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);   // lanes wait for different words: they give up together
        if (tb + TB < m) peek(share + 1, tb + TB);
        if (n < p.N && ok) {
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            if (tb + t >= m) break;
            const int64_t o = (int64_t)(tt * MT + tb + t) * p.ldo + n;
            if (p.out_f32) reinterpret_cast<float*>(p.out)[o] = v[t] + bv;
            else reinterpret_cast<uint16_t*>(p.out)[o] = bf16_bits(v[t] + bv);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.acce[b]);
      u = ue;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_EPI0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Row-major MXFP4 [N][K/2] + [N][K/32] -> tiles: [N/128][K/128] blocks of 128
// rows x 64 code bytes, then as many 512-byte scale blocks, the rest padded
// with zero codes and unit scales.
__global__ void __launch_bounds__(256) k_pack_w4(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int N, int K,
                                                 int KC, uint8_t* __restrict__ codes, uint8_t* __restrict__ sf) {
  const int64_t blk = blockIdx.x;
  const int rt = static_cast<int>(blk / KC), kc = static_cast<int>(blk % KC);
  for (int i = threadIdx.x; i < 512; i += 256) {   // 512 groups of 32: 16 bytes of codes, one scale
    const int r = i >> 2, g = i & 3, n = rt * 128 + r, k = kc * 128 + g * 32;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint8_t sc = 127;
    if (n < N && k < K) {
      v = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)n * (K / 2) + k / 2));
      sc = __ldg(s + (int64_t)n * (K / 32) + k / 32);
    }
    reinterpret_cast<uint4*>(codes + blk * w4::CODE_BLOCK)[i] = v;
    sf[blk * w4::SF_BLOCK + w4::sf_byte(r, g)] = sc;
  }
}

// The tokens' operand columns and scales, [token tile][K/128] blocks of NC x
// 128 bytes (the tile as the MMA reads it) and of 512 bytes: 16 lanes a chunk of
// one token, 16 tokens a CTA.
template <int NC>
__global__ void __launch_bounds__(256) k_split_x(const LinearParams p) {
  pdl_launch_dependents();   // k_linear_w4 sets up, sends weights for L2 and waits for this kernel's end
  pdl_wait();
  constexpr int MT = NC / 2;
  const int kc = blockIdx.x, t = blockIdx.y * 16 + (threadIdx.x >> 4), g8 = threadIdx.x & 15, k = kc * 128 + g8 * 8;
  const uint4 v = (t < p.M && k < p.K) ? __ldcg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ldx + k))
                                       : make_uint4(0u, 0u, 0u, 0u);
  const int64_t blk = (int64_t)(t / MT) * p.KC + kc;
  if (t / MT < p.TT) split_item(v, p.xop + blk * (NC * 128), p.xsf + blk * SF_BLOCK, t % MT, MT, g8);
}

template <int NC, int SW>
static cudaError_t launch(const CUtensorMap& w, const LinearParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = set_up_kernel(k_linear_w4<NC, SW>, smem_bytes<NC, SW>(), &ready);
  if (e != cudaSuccess) return e;
  // The kernel's set-up may overlap the tail of the call before it.
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg<NC, SW>::THREADS);
  cfg.dynamicSmemBytes = smem_bytes<NC, SW>();
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (Cfg<NC, SW>::PRE) {
    cudaLaunchConfig_t pre = cfg;
    pre.gridDim = dim3(p.KC, (p.M + 15) / 16);
    pre.blockDim = dim3(256);
    pre.dynamicSmemBytes = 0;
    static std::atomic<uint64_t> pre_ready{0};
    if ((e = set_up_kernel(k_split_x<NC>, 0, &pre_ready)) != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&pre, k_split_x<NC>, p)) != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, k_linear_w4<NC, SW>, w, p);
}

}  // namespace linear

cudaError_t launch_linear_w4(const CUtensorMap& w, const LinearParams& p, int nc, int grid, cudaStream_t st) {
  switch (nc) {
    case 16: return linear::launch<16, 8>(w, p, grid, st);
    case 32: return linear::launch<32, 0>(w, p, grid, st);
    case 64: return linear::launch<64, 0>(w, p, grid, st);
    default: return linear::launch<128, 0>(w, p, grid, st);
  }
}

cudaError_t launch_pack_w4(const uint8_t* q, const uint8_t* s, int N, int K, uint8_t* packed, cudaStream_t st) {
  const int RT = (N + 127) / 128, KC = (K + 127) / 128;
  const int64_t blocks = (int64_t)RT * KC;
  linear::k_pack_w4<<<(unsigned)blocks, 256, 0, st>>>(q, s, N, K, KC, packed, packed + blocks * w4::CODE_BLOCK);
  return cudaGetLastError();
}

}  // namespace moe
