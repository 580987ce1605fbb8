// api_w4.cu -- the C ABI of the few-token operators on MXFP4 weights with bf16
// activations (include/moe_b200.h): argument checks, workspace plan, tensor
// maps and launches.  Nothing here synchronizes the host.
#include <algorithm>
#include <climits>
#include <cstring>

#include "host.h"

namespace moe {

cudaError_t launch_linear_w4(const CUtensorMap& w, const LinearParams& p, int nc, int grid, cudaStream_t st);
cudaError_t launch_pack_w4(const uint8_t* q, const uint8_t* s, int N, int K, uint8_t* packed, cudaStream_t st);

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
  if (s.M > (1 << 20) || s.K > (1 << 20) || s.N > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  p->RT = (s.N + 127) / 128;
  p->KC = (s.K + 127) / 128;
  p->KU = (p->KC + 1) / 2;                 // a unit is two chunks
  if ((int64_t)p->RT * p->KC * 128 > INT_MAX) return MOE_ERR_UNSUPPORTED;   // rows of the packed tensor map
  p->nc = s.M <= 8 ? 16 : s.M <= 16 ? 32 : s.M <= 32 ? 64 : 128;
  p->mt = p->nc / 2;
  p->TT = (s.M + p->mt - 1) / p->mt;
  p->units = (int64_t)p->RT * p->TT * p->KU;
  p->grid = (int)std::min<int64_t>(std::min(sms, kMaxGrid), (p->units + 1) / 2);
  // the parts come first and in one place for every shape: they are zero
  // between calls, the operand blocks behind them are not
  p->o_xop = p->total = kLinearHeader + (size_t)kMaxGrid * p->mt * 128 * 4;
  if (p->nc >= 64) {
    p->o_xop = p->total = kLinearHeader + (size_t)kMaxGrid * 64 * 128 * 4;
    p->o_xsf = p->o_xop + (size_t)p->TT * p->KC * p->nc * 128;
    p->total = p->o_xsf + (size_t)p->TT * p->KC * 512;
  }
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_w4_packed_size(int32_t N, int32_t K, size_t* bytes) {
  if (!bytes || N < 1 || K < 32 || K % 32) return fail(MOE_ERR_INVALID_ARG, "moe_w4_packed_size: null pointer, N < 1 or K not a multiple of 32");
  *bytes = (size_t)((N + 127) / 128) * ((K + 127) / 128) * 8704;
  return MOE_OK;
}

int moe_pack_w4(const uint8_t* q, const uint8_t* scales, int32_t N, int32_t K, uint8_t* packed, void* stream) {
  size_t bytes = 0;
  if (!q || !scales || !packed) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: null pointer argument");
  if (moe_w4_packed_size(N, K, &bytes) != MOE_OK) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: N < 1 or K not a multiple of 32");
  if ((int64_t)(bytes / 8704) * 128 > INT_MAX) return fail(MOE_ERR_UNSUPPORTED, "moe_pack_w4: matrix too large");
  if (!aligned(q, 16) || !aligned(packed, 256)) return fail(MOE_ERR_INVALID_ARG, "moe_pack_w4: q needs 16-byte, packed 256-byte alignment");
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
  if (out == x || out == workspace) return fail(MOE_ERR_INVALID_ARG, "moe_linear_w4: out aliases an input");
  const void* ptrs[5] = {x, w_packed, bias, out, workspace};
  const int dev = resolve_device(stream, ptrs, 5);
  if (dev < 0) return dev;
  DeviceGuard g(dev);
  LinearPlan pl;
  const int rc = linear_plan(*shape, sm_count(dev), &pl);
  if (rc != MOE_OK) return fail(rc, "moe_linear_w4: unsupported shape");
  if (ws_bytes < pl.total) return fail(MOE_ERR_WORKSPACE, "moe_linear_w4: workspace smaller than moe_linear_w4_workspace_size");
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
  p.wsf = static_cast<const uint8_t*>(w_packed) + blocks * 8192;
  p.out = out;
  p.part = reinterpret_cast<uint32_t*>(ws + kLinearHeader);
  p.status = reinterpret_cast<int32_t*>(ws);
  p.xop = ws + pl.o_xop;
  p.xsf = ws + pl.o_xsf;
  p.ldx = shape->ldx; p.ldo = shape->ldo; p.units = pl.units;
  p.M = shape->M; p.N = shape->N; p.K = shape->K; p.KC = pl.KC; p.KU = pl.KU; p.TT = pl.TT;
  p.out_f32 = shape->out_type == MOE_OUT_F32;
  p.test_withhold = take_withhold();
  p.timeout_ns = wait_timeout_ns();
  const cudaError_t e = launch_linear_w4(map, p, pl.nc, pl.grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "moe_linear_w4 kernel launch", e);
}

}  // extern "C"
