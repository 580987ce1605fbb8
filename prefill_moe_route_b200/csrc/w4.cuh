// w4.cuh -- device helpers of the few-token operators (linear.cu, layer.cu):
// MXFP4 weights against bf16 activations on the tensor cores, without rounding
// the activations.
//
// kind::mxf8f6f4 multiplies E2M1 weights (scale per 32 along K) by E4M3
// operands (scale per 32 along K) into fp32.  A bf16 activation has an 8-bit
// significand and an E4M3 value a 4-bit one, so an activation block of 32 is
// written as two operand columns that share the weights:
//   hi = E4M3(v / 2^s),            s = floor(log2 amax) - 7
//   lo = E4M3((v / 2^s - hi) * 32) with scale 2^(s - 5)
// |v| / 2^s < 256, so hi never saturates; the rest is at most 8 and has at most
// 4 significant bits, so hi + lo / 32 is v / 2^s exactly while |v| >= 2^-14
// amax; smaller values of the block keep an absolute error of 2^-21 amax.  s stops
// at -112: in a block whose amax is below 2^-105 the error is up to 2^-126, and
// subnormal bf16 activations (below 2^-126) count as zero.
// An fp32 value (not bf16) passes through f16 (2^-12) and is kept to 2^-9 relative,
// half of what rounding it to bf16 would lose, but no less than 2^-21 amax.  More is a
// third column: half as many MMA columns, operand bytes and hand-over words again, and
// for more than 8 tokens a ring of four stages (16 tokens 86.5 us instead of 83.1 in a
// graph for the stage alone), for an error over all outputs of moe_layer_w4 that goes
// from 1.65e-3 (fp32 everywhere, bf16 out) to 1.8e-3 - 2.0e-3 with two.
// A block that holds an infinity or a NaN becomes NaN in both columns, so only
// its own token's sums become NaN.
#pragma once
#include <atomic>

#include "w4_params.h"
#include "ptx.cuh"
#include "codec.cuh"

namespace moe {
namespace w4 {

// ------------------------------------------------------------ instructions that only these kernels use
// Store to a CTA of the cluster that completes 4 bytes of transaction count on a
// barrier of the same CTA: the value and its arrival in one trip.
__device__ __forceinline__ void st_async_cluster_f32(uint32_t cluster_saddr, float v, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(cluster_saddr), "f"(v),
               "r"(cluster_bar)
               : "memory");
}

__device__ __forceinline__ void red_release_gpu(int32_t* p, int32_t v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int32_t add_acq_rel_gpu(int32_t* p, int32_t v) {   // the value before
  int32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Has a value worked out by this point of the program (before a wait, say).
template <typename T>
__device__ __forceinline__ void have(const T& v) {
  if constexpr (sizeof(T) == 8) asm volatile("" ::"l"(v) : "memory");
  else asm volatile("" ::"r"(v) : "memory");
}

// True in one lane of a converged warp (always the same one).  Tensor-core
// instructions take their descriptors from uniform registers: issued from a
// loop that the whole warp runs under this predicate they cost half of what
// they cost in a loop of one diverged thread (217 against 413 clocks for the
// copies, four N = 16 MMAs and the commit of one 128 x 128 block).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// TMEM -> registers: this warp's 32 lanes, 1, 2, 4 or 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[1]) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  v[0] = __uint_as_float(r);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  v[0] = __uint_as_float(r[0]);
  v[1] = __uint_as_float(r[1]);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------ operands

constexpr int A_TILE = 16384;      // 128 rows x 128 E2M1 in shared memory (8 bytes of codes in each 16)
constexpr int SF_BLOCK = 512;      // scales of 128 rows x 4 groups, in the tensor cores' order
constexpr int CODE_BLOCK = 8192;   // the same tile's codes in global memory

// Scale exponent of a block from its largest magnitude; SPLIT_NAN marks a
// block that is not finite.
constexpr int SPLIT_NAN = -128;
__device__ __forceinline__ int split_exp(float amax) {
  const int ex = static_cast<int>(__float_as_uint(amax) >> 23);   // amax >= 0
  if (ex == 255) return SPLIT_NAN;
  return max(-112, ex - 134);   // floor(log2 amax) - 7, in the range of lo's scale and of f16x2_scaled
}
__device__ __forceinline__ uint32_t split_code_hi(int s) { return s == SPLIT_NAN ? 127u : static_cast<uint32_t>(s + 127); }
__device__ __forceinline__ uint32_t split_code_lo(int s) { return s == SPLIT_NAN ? 127u : static_cast<uint32_t>(s + 122); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two bf16 divided by 2^s as f16, by integer arithmetic on the fields (the
// conversion unit is the scarce one here): magnitudes below 2^-14 after the
// scaling become zero, 2^-21 of the block's largest.
__device__ __forceinline__ uint32_t f16x2_scaled(uint32_t w, int s) {
  const uint32_t off = static_cast<uint32_t>(s + 112) * 0x00800080u;   // exponent fields: e - 127 - s + 15 = e - (s + 112)
  const uint32_t m = max_u16x2(w & 0x7FFF7FFFu, off) - off;
  return (m << 3) | (w & 0x80008000u);
}

// hi and lo codes of two values already divided by 2^s, as f16.
__device__ __forceinline__ void split_f16x2(uint32_t v, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t back, r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(v));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(back));        // exact
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x50005000u));   // times 32
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r));
  hi = h;
  lo = l;
}

// Two fp32 values divided by 2^s (inv = 2^-s) as f16.
__device__ __forceinline__ uint32_t f16x2_of(float a, float b, float inv) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b * inv), "f"(a * inv));
  return r;
}

// Byte of value k (0..127) of operand row n in a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t tile_byte(uint32_t n, uint32_t k) {
  return n * 128u + ((((k >> 4) ^ (n & 7u)) << 4) | (k & 15u));
}
// Byte of row n's scale of group q (0..3) in a 512-byte scale block.
__device__ __forceinline__ uint32_t sf_byte(uint32_t n, uint32_t q) { return 16u * (n & 31u) + 4u * (n >> 5) + q; }

// A wait ran out: recorded in the status words, and the block's other roles are
// told.  A function of its own keeps it out of the roles' code, which every call
// fetches anew.  Word 3 stays until the workspace is zero-filled: what a call that
// gave up leaves there (parts, tickets) is not what the next one starts from.
static __device__ __noinline__ void wait_ran_out(int32_t* status, volatile int* abort_flag, uint32_t where) {
  *abort_flag = 1;
  atomicOr(status, ST_TIMEOUT);
  atomicCAS(status + 2, 0, static_cast<int>(0x80000000u | where | (blockIdx.x & 0xFFFu)));
  atomicOr(status + 3, 1);
}
// One thread of a call: the workspace of a call that gave up, not zero-filled since,
// serves no other.  Reported anew, since moe_get_status clears the status word.
__device__ __forceinline__ void report_used_up(int32_t* status) {
  if (__ldcg(status + 3)) atomicOr(status, ST_TIMEOUT);
}

// a / b for 0 <= a < 2^31, b > 0 and a quotient below 2^21 (then the fp32 quotient
// is at most 2 off): no branches, where integer divisions follow one another in
// a single warp that works out its share.
__device__ __forceinline__ int quick_div(int a, int b) {
  int q = __float2int_rz(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  int r = a - q * b;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = r < 0 ? -1 : r >= b ? 1 : 0;
    q += c;
    r -= c * b;
  }
  return q;
}

// A part of a sum on its way to another CTA: the word is the value's bits
// inverted, so that zero (what the buffer holds between calls) marks a part
// that has not arrived.  Value and arrival are one 4-byte word: no fence, no
// flag, one trip through L2.  The reader puts the zero back.
__device__ __forceinline__ void part_put(uint32_t* p, float v) {
  const uint32_t bits = v == v ? __float_as_uint(v) : 0x7FC00000u;   // any NaN as the one whose inverse is not zero
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(~bits) : "memory");
}
__device__ __forceinline__ uint32_t part_peek(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float part_value(uint32_t word) { return __uint_as_float(~word); }
__device__ __forceinline__ void word_put(uint32_t* p, uint32_t v) {   // v: not all ones
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(~v) : "memory");
}
__device__ __forceinline__ uint4 words_peek(const uint32_t* p) {   // still inverted
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Once per device and kernel: its dynamic shared memory, and the split of the
// SM's memory towards shared memory, without which a small kernel cannot run
// beside one of these large ones (the SM would have to be empty to change it).
template <typename Kernel>
inline cudaError_t set_up_kernel(Kernel* kernel, int smem, std::atomic<uint64_t>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev <= 63 && (ready->load(std::memory_order_relaxed) >> dev & 1u)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && smem) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev <= 63) ready->fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

}  // namespace w4
}  // namespace moe
