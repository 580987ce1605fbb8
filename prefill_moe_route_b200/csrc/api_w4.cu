// api_w4.cu -- the C ABI of the few-token operators on MXFP4 weights with bf16
// activations (include/moe_b200.h): argument checks, workspace plan, tensor
// maps and launches.  Nothing here synchronizes the host.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "host.h"
#include "w4_params.h"

namespace moe {

cudaError_t launch_linear_w4(const CUtensorMap& w, const LinearParams& p, int nc, int grid, cudaStream_t st);
cudaError_t launch_pack_w4(const uint8_t* q, const uint8_t* s, int N, int K, uint8_t* packed, cudaStream_t st);

cudaError_t launch_layer_w4(const CUtensorMap* maps, const LayerParams& p, int sms, cudaStream_t st);

constexpr int kMaxGrid = 148;              // CTAs of these kernels: one per SM of a B200
constexpr size_t kLinearHeader = 256;      // status words

struct LinearPlan {
  int nc, mt;                              // operand columns and tokens per tile
  int RT, TT, KC, KU, grid;
  int64_t units;
  size_t o_xop, o_xsf, total;
};

static int linear_plan(const moe_linear_shape_t& s, int sms, LinearPlan* p) {
  if (s.M < 1 || s.N < 1 || s.K < 32 || s.K % 32) return MOE_ERR_INVALID_ARG;
  if (s.ldx < s.K || s.ldo < s.N || s.ldx % 8) return MOE_ERR_INVALID_ARG;
  if (s.out_type != MOE_OUT_BF16 && s.out_type != MOE_OUT_F32) return MOE_ERR_INVALID_ARG;
  if (s.M > (1 << 19) || s.K > (1 << 20) || s.N > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  p->RT = (s.N + 127) / 128;
  p->KC = (s.K + 127) / 128;
  p->KU = (p->KC + 1) / 2;                 // a unit is two chunks
  if ((int64_t)p->RT * p->KC * 128 > INT_MAX) return MOE_ERR_UNSUPPORTED;   // rows of the packed tensor map
  // Columns of a token tile, 128 at most: more tokens share a tile's weights (us, 128
  // columns / 64: 48 x 6144 x 6144 11.2 / 11.7, 512 x 6144 x 2048 19.3 / 23.3; 64 / 32: 32
  // x 6144 x 6144 9.3 / 11.0).  With 16 the product's kernel splits the tokens itself,
  // above them a kernel before it does; 5 to 8 tokens pay for that kernel from about 8
  // units a CTA (us, 32 / 16: 8 x 40003 x 6144 25.4 / 28.8, 8 x 12288 x 6144 11.0 / 11.8,
  // 8 x 6144 x 6144 7.9 / 7.8, 7 x 4099 x 2912 6.1 / 5.0).
  const bool many = (int64_t)p->RT * p->KU > 8 * kMaxGrid;
  p->nc = s.M <= 4 || (s.M <= 8 && !many) ? 16 : s.M <= 16 ? 32 : s.M <= 32 ? 64 : 128;
  p->mt = p->nc / 2;
  p->TT = (s.M + p->mt - 1) / p->mt;
  p->units = (int64_t)p->RT * p->TT * p->KU;
  if (p->units > INT_MAX) return MOE_ERR_UNSUPPORTED;
  p->grid = (int)std::min<int64_t>(std::min(sms, kMaxGrid), (p->units + 1) / 2);
  // the parts come first and in one place for every shape: they are zero
  // between calls, the operand blocks behind them are not
  p->o_xop = p->total = kLinearHeader + (size_t)kMaxGrid * p->mt * 128 * 4;
  if (p->nc >= 32) {   // made by a kernel of its own
    p->o_xop = p->total = kLinearHeader + (size_t)kMaxGrid * 64 * 128 * 4;
    p->o_xsf = p->o_xop + (size_t)p->TT * p->KC * p->nc * 128;
    p->total = p->o_xsf + (size_t)p->TT * p->KC * 512;
  }
  return MOE_OK;
}

struct LayerPlan {
  size_t o_part1, o_part2, o_sig, o_rstd, o_xop, o_xsf, o_mop, o_msf, total;
};

static int layer_plan(const moe_layer_shape_t& s, LayerPlan* p) {
  if (s.M < 1 || s.E < 1 || s.topk < 1 || s.H < 128 || s.I < 128 || s.shared_I < 0) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(s.routed_scale) || !(s.norm_eps >= 0.0f) || !std::isfinite(s.norm_eps)) return MOE_ERR_INVALID_ARG;
  if (s.ldx < s.H || s.ldo < s.H || s.ldx % 8) return MOE_ERR_INVALID_ARG;
  if (s.M > 16 || s.E > kMaxE || s.topk > kMaxTopk || s.topk > s.E) return MOE_ERR_UNSUPPORTED;
  if (s.H % 128 || s.I % 128 || s.shared_I % 128 || s.H > 65536 || s.I > 65536 || s.shared_I > 65536)
    return MOE_ERR_UNSUPPORTED;
  // One layout for every M.  The parts, sigmoids and norm factors come first, in
  // one place for every shape: they are zero between calls, the rest is written
  // before it is read.
  size_t o = 256;
  auto take = [&](size_t bytes) { size_t r = o; o = align_up(o + bytes, 256); return r; };
  const size_t KC = s.H / 128, tiles = (size_t)std::min(s.E, 16 * s.topk) * (s.I / 128) + s.shared_I / 128;
  p->o_part1 = take((size_t)kMaxGrid * 32 * 128 * 4);
  p->o_part2 = take((size_t)kMaxGrid * 16 * 128 * 4);
  p->o_sig = take((size_t)16 * kMaxE * 4);
  p->o_rstd = take(16 * 4);
  p->o_xop = take(KC * 32 * 128);
  p->o_xsf = take(KC * 512);
  p->o_mop = take(tiles * 32 * 128);
  p->o_msf = take(tiles * 512);
  p->total = o;
  return MOE_OK;
}

// Test knob MOE_TEST_HOLD_ROUTING_US=n: one CTA of every moe_layer_w4 call routes
// n microseconds late (at most a tenth of a second).  Read once per process.
static uint64_t routing_hold_ns() {
  static const uint64_t v = [] {
    const char* e = std::getenv("MOE_TEST_HOLD_ROUTING_US");
    return static_cast<uint64_t>(std::min(std::max(e ? std::atol(e) : 0l, 0l), 100000l)) * 1000;
  }();
  return v;
}

// Tensor map of `batch` 4-bit matrices [rows][K], boxes of 128 x 128 (tiles land unpacked).
static bool mx_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t batch) {
  const uint64_t d[3] = {K, rows, batch}, st[2] = {K / 2, rows * (K / 2)};
  const uint32_t box[3] = {128, 128, 1};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, base, d, st, box);
}

// `rows` rows of `len` bytes, `pitch` bytes apart (rows do not overlap one another).
struct Span {
  uintptr_t at;
  uint64_t rows, len, pitch;
  uintptr_t end() const { return at + (rows - 1) * pitch + len; }
};
static Span span(const void* p, uint64_t bytes) { return {reinterpret_cast<uintptr_t>(p), 1, bytes, bytes}; }
static Span span(const void* p, uint64_t rows, uint64_t len, uint64_t pitch) { return {reinterpret_cast<uintptr_t>(p), rows, len, pitch}; }

// True if a byte lies in both; null and empty spans overlap nothing.  Rows that lie
// between the other's rows (columns of one buffer) are apart.
static bool overlap(const Span& a, const Span& b) {
  if (!a.at || !b.at || !a.len || !b.len || a.at >= b.end() || b.at >= a.end()) return false;
  uint64_t i = 0, j = 0;   // only buffers that lie one inside the other get here: row by row
  if (a.at + a.pitch <= b.at) i = (b.at - a.at) / a.pitch;
  if (b.at + b.pitch <= a.at) j = (a.at - b.at) / b.pitch;
  while (i < a.rows && j < b.rows) {
    const uintptr_t x = a.at + i * a.pitch, y = b.at + j * b.pitch;
    if (x < y + b.len && y < x + a.len) return true;
    if (x + a.len <= y) ++i;
    else ++j;
  }
  return false;
}
// True if a buffer that the call writes overlaps another or one that it only reads.
static bool any_overlap(const Span* out, int nout, const Span* in, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (overlap(out[i], out[j])) return true;
    for (int j = 0; j < nin; ++j)
      if (overlap(out[i], in[j])) return true;
  }
  return false;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_w4_packed_size(int32_t N, int32_t K, size_t* bytes) {
  if (!bytes || N < 1 || K < 32 || K % 32) return fail(MOE_ERR_INVALID_ARG, "moe_w4_packed_size: null pointer, N < 1 or K not a multiple of 32");
  *bytes = (size_t)((N + 127ll) / 128) * ((K + 127ll) / 128) * 8704;
  return MOE_OK;
}

int moe_pack_w4(const uint8_t* q, const uint8_t* scales, int32_t N, int32_t K, uint8_t* packed, void* stream) {
  size_t bytes = 0;
  if (!q || !scales || !packed) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: null pointer argument");
  if (moe_w4_packed_size(N, K, &bytes) != MOE_OK) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: N < 1 or K not a multiple of 32");
  if (bytes / 8704 * 128 > INT_MAX) return fail(MOE_ERR_UNSUPPORTED, "moe_pack_w4: matrix too large");
  if (!aligned(q, 16) || !aligned(packed, 256)) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: q needs 16-byte, packed 256-byte alignment");
  const uintptr_t p0 = reinterpret_cast<uintptr_t>(packed), p1 = p0 + bytes, q0 = reinterpret_cast<uintptr_t>(q),
                  s0 = reinterpret_cast<uintptr_t>(scales), n = N;
  if ((q0 < p1 && p0 < q0 + n * (K / 2)) || (s0 < p1 && p0 < s0 + n * (K / 32)))
    return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: buffers overlap");
  const void* ptrs[3] = {q, scales, packed};
  const int dev = resolve_device(stream, ptrs, 3);
  if (dev < 0) return dev;
  DeviceGuard g(dev);
  const cudaError_t e = launch_pack_w4(q, scales, N, K, packed, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "moe_pack_w4", e);
}

int moe_linear_w4_workspace_size(const moe_linear_shape_t* shape, size_t* bytes) {
  if (!shape || !bytes) return fail(MOE_ERR_INVALID_ARG, "moe_linear_w4_workspace_size: null pointer argument");
  LinearPlan p;
  const int rc = linear_plan(*shape, kMaxGrid, &p);
  if (rc != MOE_OK) return fail(rc, "moe_linear_w4: unsupported shape");
  *bytes = p.total;
  return MOE_OK;
}

int moe_linear_w4(const moe_linear_shape_t* shape, const void* x, const void* w_packed, const float* bias, void* out,
                  void* workspace, size_t ws_bytes, void* stream) {
  if (!shape || !x || !w_packed || !out || !workspace) return fail(MOE_ERR_INVALID_ARG, "moe_linear_w4: null pointer argument");
  if (!aligned(x, 16) || !aligned(w_packed, 256) || !aligned(workspace, 256) || !aligned(bias, 4) ||
      !aligned(out, shape->out_type == MOE_OUT_F32 ? 4 : 2))
    return fail(MOE_ERR_INVALID_ARG, "moe_linear_w4: x needs 16-byte, w_packed and workspace 256-byte, bias and out their type's alignment");
  LinearPlan pl;
  int rc = linear_plan(*shape, kMaxGrid, &pl);
  if (rc != MOE_OK) return fail(rc, "moe_linear_w4: unsupported shape");
  if (ws_bytes < pl.total) return fail(MOE_ERR_WORKSPACE, "moe_linear_w4: workspace smaller than moe_linear_w4_workspace_size");
  const uint64_t M = shape->M, N = shape->N, K = shape->K, esz = shape->out_type == MOE_OUT_F32 ? 4 : 2;
  const Span written[2] = {span(out, M, N * esz, shape->ldo * esz), span(workspace, pl.total)};
  const Span read[3] = {span(x, M, K * 2, shape->ldx * 2), span(w_packed, (uint64_t)pl.RT * pl.KC * 8704), span(bias, N * 4)};
  if (any_overlap(written, 2, read, 3)) return fail(MOE_ERR_INVALID_ARG, "moe_linear_w4: out or workspace overlaps another buffer");
  const void* ptrs[5] = {x, w_packed, bias, out, workspace};
  const int dev = resolve_device(stream, ptrs, 5);
  if (dev < 0) return dev;
  DeviceGuard g(dev);
  rc = linear_plan(*shape, sm_count(dev), &pl);
  if (rc != MOE_OK) return fail(rc, "moe_linear_w4: unsupported shape");
  const uint64_t blocks = (uint64_t)pl.RT * pl.KC;
  CUtensorMap map;
  const uint64_t dims[2] = {128, blocks * 128}, strides[1] = {64};
  const uint32_t box[2] = {128, 256};
  if (!make_map(&map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, w_packed, dims, strides, box))
    return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor map");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LinearParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.bias = bias;
  p.wcodes = static_cast<const uint8_t*>(w_packed);
  p.wsf = p.wcodes + blocks * 8192;
  p.out = out;
  p.part = reinterpret_cast<uint32_t*>(ws + kLinearHeader);
  p.status = reinterpret_cast<int32_t*>(ws);
  p.xop = ws + pl.o_xop;
  p.xsf = ws + pl.o_xsf;
  p.ldx = shape->ldx; p.ldo = shape->ldo; p.shares = w4::Shares((int)pl.units, pl.grid);
  p.M = shape->M; p.N = shape->N; p.K = shape->K; p.KC = pl.KC; p.KU = pl.KU; p.TT = pl.TT;
  p.out_f32 = shape->out_type == MOE_OUT_F32;
  p.test_withhold = take_withhold();
  p.timeout_ns = wait_timeout_ns();
  const cudaError_t e = launch_linear_w4(map, p, pl.nc, pl.grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "moe_linear_w4 kernel launch", e);
}

int moe_layer_w4_workspace_size(const moe_layer_shape_t* shape, size_t* bytes) {
  if (!shape || !bytes) return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4_workspace_size: null pointer argument");
  LayerPlan p;
  const int rc = layer_plan(*shape, &p);
  if (rc != MOE_OK) return fail(rc, "moe_layer_w4: unsupported shape");
  *bytes = p.total;
  return MOE_OK;
}

int moe_layer_w4(const moe_layer_shape_t* shape, const moe_layer_weights_t* w, const void* x, void* out, int32_t* topk_ids,
                 float* topk_w, void* workspace, size_t ws_bytes, void* stream) {
  if (!shape || !w || !x || !out || !workspace || !w->router_w || !w->w13 || !w->w13_scales || !w->w2 || !w->w2_scales)
    return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: null pointer argument");
  LayerPlan pl;
  const int rc = layer_plan(*shape, &pl);
  if (rc != MOE_OK) return fail(rc, "moe_layer_w4: unsupported shape");
  const bool shared = shape->shared_I > 0;
  if (shared && (!w->shared_w13 || !w->shared_w13_scales || !w->shared_w2 || !w->shared_w2_scales))
    return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: null shared expert pointer with shared_I > 0");
  const void* sh[4] = {shared ? w->shared_w13 : nullptr, shared ? w->shared_w13_scales : nullptr,
                       shared ? w->shared_w2 : nullptr, shared ? w->shared_w2_scales : nullptr};
  const void* ptrs[16] = {x, out, workspace, topk_ids, topk_w, w->norm_w, w->router_w, w->bias, w->w13, w->w13_scales,
                          w->w2, w->w2_scales, sh[0], sh[1], sh[2], sh[3]};
  for (int i : {0, 5, 6, 9, 11, 13, 15})
    if (!aligned(ptrs[i], 16)) return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: pointer not 16-byte aligned");
  for (int i : {8, 10, 12, 14})
    if (!aligned(ptrs[i], 32)) return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: weights need 32-byte alignment");
  if (!aligned(workspace, 256) || !aligned(out, 2) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(w->bias, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: workspace needs 256-byte alignment, out, ids, weights and bias their type's");
  if (ws_bytes < pl.total) return fail(MOE_ERR_WORKSPACE, "moe_layer_w4: workspace smaller than moe_layer_w4_workspace_size");
  const uint64_t M = shape->M, H = shape->H, I = shape->I, E = shape->E, S = shape->shared_I, choices = M * shape->topk;
  const Span written[4] = {span(out, M, H * 2, shape->ldo * 2), span(workspace, pl.total), span(topk_ids, choices * 4), span(topk_w, choices * 4)};
  const Span read[12] = {span(x, M, H * 2, shape->ldx * 2), span(w->norm_w, H * 2), span(w->router_w, E * H * 2), span(w->bias, E * 4),
                         span(w->w13, E * I * H), span(w->w13_scales, E * I * H / 16), span(w->w2, E * I * H / 2), span(w->w2_scales, E * I * H / 32),
                         span(sh[0], S * H), span(sh[1], S * H / 16), span(sh[2], S * H / 2), span(sh[3], S * H / 32)};
  if (any_overlap(written, 4, read, 12)) return fail(MOE_ERR_INVALID_ARG, "moe_layer_w4: a buffer that is written overlaps another");
  const int dev = resolve_device(stream, ptrs, 16);
  if (dev < 0) return dev;
  DeviceGuard g(dev);
  CUtensorMap m[4];
  bool ok = mx_map(&m[0], w->w13, H, 2 * I, E) && mx_map(&m[1], w->w2, I, H, E);
  if (shared) ok = ok && mx_map(&m[2], sh[0], H, 2 * S, 1) && mx_map(&m[3], sh[2], S, H, 1);
  else { m[2] = m[0]; m[3] = m[1]; }
  if (!ok) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor map");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LayerParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.norm_w = static_cast<const uint16_t*>(w->norm_w);
  p.router_w = static_cast<const uint16_t*>(w->router_w);
  p.bias = w->bias;
  p.s13 = static_cast<const uint8_t*>(w->w13_scales);
  p.s2 = static_cast<const uint8_t*>(w->w2_scales);
  p.ss13 = static_cast<const uint8_t*>(sh[1]);
  p.ss2 = static_cast<const uint8_t*>(sh[3]);
  p.out = static_cast<uint16_t*>(out);
  p.ids_out = topk_ids;
  p.wts_out = topk_w;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.sync = reinterpret_cast<int32_t*>(ws + 64);
  p.part1 = reinterpret_cast<uint32_t*>(ws + pl.o_part1);
  p.part2 = reinterpret_cast<uint32_t*>(ws + pl.o_part2);
  p.sig = reinterpret_cast<uint32_t*>(ws + pl.o_sig);
  p.rstd = reinterpret_cast<uint32_t*>(ws + pl.o_rstd);
  p.xop = ws + pl.o_xop; p.xsf = ws + pl.o_xsf;
  p.mop = ws + pl.o_mop; p.msf = ws + pl.o_msf;
  p.ldx = shape->ldx; p.ldo = shape->ldo;
  p.M = shape->M; p.H = shape->H; p.I = shape->I; p.S = shape->shared_I; p.E = shape->E; p.topk = shape->topk;
  p.nc = shape->M <= 8 ? 16 : 32;
  p.residual = shape->add_residual != 0;
  p.scale = shape->routed_scale; p.eps = shape->norm_eps;
  p.test_withhold = take_withhold();
  // The kernel's waits end at one time, counted from its start (a clock for each wait
  // is more code of every role, which every call fetches anew: 1 token 16.8 us
  // instead of 16.5, 4 small ones 10.4 instead of 10.1), so the call's own work goes
  // on top: the weights that it may have to read at 0.5 TB/s, a tenth of the usual.
  const uint64_t expert = 3 * H * I, used = std::min<uint64_t>(E, (uint64_t)shape->M * shape->topk);
  p.timeout_ns = wait_timeout_ns() + (used * expert + 3 * H * S) / 2 / 500;
  p.test_hold_ns = routing_hold_ns();
  const cudaError_t e = launch_layer_w4(m, p, std::min(sm_count(dev), kMaxGrid), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "moe_layer_w4 kernel launch", e);
}

}  // extern "C"
