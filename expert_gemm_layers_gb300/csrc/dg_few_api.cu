// The C ABI of the few-token operators (include/dg.h): 4-bit weights and
// routed experts.  Argument checks, scratch carving and launches.
#include <cuda_runtime.h>

#include <atomic>

#include "dg_internal.h"

namespace dg {

cudaError_t smem_limit_once(const void* kern, int bytes, int dev) {
  // open addressing on the kernel's address
  struct Slot {
    std::atomic<const void*> kern{nullptr};
    std::atomic<uint64_t> done{0};  // bit per device
  };
  constexpr int kSlots = 128;
  static Slot slots[kSlots];
  size_t at = (reinterpret_cast<uintptr_t>(kern) >> 4) % kSlots;
  for (int i = 0; i < kSlots; ++i, at = (at + 1) % kSlots) {
    const void* k = slots[at].kern.load(std::memory_order_acquire);
    if (k == nullptr) {
      const void* expected = nullptr;
      if (slots[at].kern.compare_exchange_strong(expected, kern)) k = kern;
      else k = expected;
    }
    if (k != kern) continue;
    const uint64_t bit = uint64_t(1) << dev;
    if (slots[at].done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) slots[at].done.fetch_or(bit, std::memory_order_release);
    return e;
  }
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kMaxW4Rows = int64_t(1) << 31;
constexpr int64_t kMaxW4LinearRows = 65535 * 32;
// the router's column index steps by up to 2 * 8 * 256 past the last column in 32 bits
constexpr int64_t kMaxRouteDim = kMaxDim + 1 - 8192;

dg_status check_w4(int64_t rows, int64_t K, int32_t group, const char* what) {
  if (group != 32 && group != 64 && group != 128)
    return fail(DG_ERR_INVALID_ARGUMENT, "%s: group is %d, not 32, 64 or 128", what, group);
  if (rows < 0 || K < 1) return fail(DG_ERR_INVALID_ARGUMENT, "%s: rows must be >= 0 and the row length >= 1", what);
  if (K % group) return fail(DG_ERR_INVALID_ARGUMENT, "%s: the row length is not a multiple of the group", what);
  if (K > kMaxDim || rows > kMaxW4Rows || rows * (K / 8) > (int64_t(1) << 38))
    return fail(DG_ERR_UNSUPPORTED, "%s: rows * row length beyond 2^41, or a size beyond 2^31", what);
  return DG_OK;
}

size_t code_bytes(int64_t rows, int64_t K) { return static_cast<size_t>(rows) * (K / 2); }
size_t scale_bytes(int64_t rows, int64_t K, int32_t group) { return static_cast<size_t>(rows) * (K / group) * 2; }
size_t zero_bytes(int64_t rows, int64_t K, int32_t group) { return static_cast<size_t>(rows) * (K / group); }

dg_status check_moe(const dg_moe_shape* sh, const char* what) {
  if (!sh) return fail(DG_ERR_INVALID_ARGUMENT, "%s: shape is NULL", what);
  if (sh->T < 0 || sh->d < 1 || sh->F < 1 || sh->E < 1 || sh->k < 1)
    return fail(DG_ERR_INVALID_ARGUMENT, "%s: T must be >= 0 and d, F, E, k >= 1", what);
  if (sh->d % 8 || sh->F % 8) return fail(DG_ERR_INVALID_ARGUMENT, "%s: d and F must be multiples of 8", what);
  if (sh->d > (1 << 20) || sh->F > (1 << 20)) return fail(DG_ERR_UNSUPPORTED, "%s: d or F beyond 2^20", what);
  if (sh->E > moe_max_experts())
    return fail(DG_ERR_UNSUPPORTED, "%s: %d experts, more than %d", what, sh->E, moe_max_experts());
  if (sh->k > moe_max_topk())
    return fail(DG_ERR_UNSUPPORTED, "%s: %d choices per token, more than %d", what, sh->k, moe_max_topk());
  if (static_cast<int64_t>(sh->T) * sh->k > moe_max_pairs())
    return fail(DG_ERR_UNSUPPORTED, "%s: T * k = %lld pairs, more than %d (split the batch)", what,
                static_cast<long long>(sh->T) * sh->k, moe_max_pairs());
  return DG_OK;
}

size_t moe_need(const dg_moe_shape& s, int group) {
  return DG_ERROR_BLOCK_BYTES + moe_scratch_bytes(s.T, s.k, s.E, s.d, s.F, group);
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_w4_quantize(int64_t rows, int64_t K, int32_t group, const void* weight, void* codes, void* scales,
                         void* zeros, void* stream) {
  dg_status st = check_w4(rows, K, group, "w4_quantize");
  if (st != DG_OK || rows == 0) return st;
  const Arg args[] = {{"weight", weight, static_cast<size_t>(rows) * K * 2, false, false},
                      {"codes", codes, code_bytes(rows, K), false, true},
                      {"scales", scales, scale_bytes(rows, K, group), false, true},
                      {"zeros", zeros, zero_bytes(rows, K, group), true, true}};
  if ((st = check_args("w4_quantize", args)) != DG_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("w4_quantize", s, 0.0, static_cast<double>(rows) * K * (2.5 + (zeros ? 3.0 : 2.0) / group));
  return launched(launch_w4_quantize(weight, codes, scales, zeros, rows, K, group, s), "w4_quantize");
}

dg_status dg_w4_dequantize(int64_t rows, int64_t K, int32_t group, const void* codes, const void* scales,
                           const void* zeros, void* weight, void* stream) {
  dg_status st = check_w4(rows, K, group, "w4_dequantize");
  if (st != DG_OK || rows == 0) return st;
  const Arg args[] = {{"weight", weight, static_cast<size_t>(rows) * K * 2, false, true},
                      {"codes", codes, code_bytes(rows, K), false, false},
                      {"scales", scales, scale_bytes(rows, K, group), false, false},
                      {"zeros", zeros, zero_bytes(rows, K, group), true, false}};
  if ((st = check_args("w4_dequantize", args)) != DG_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("w4_dequantize", s, 0.0, static_cast<double>(rows) * K * (2.5 + (zeros ? 3.0 : 2.0) / group));
  return launched(launch_w4_dequantize(codes, scales, zeros, weight, rows, K, group, s), "w4_dequantize");
}

size_t dg_w4_linear_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features) {
  (void)out_features;
  if (rows < 0 || in_features < 1 || rows > kMaxW4LinearRows || in_features > kMaxDim / 4) return 0;
  // the finest group takes the most room, staged in the workspace or by the kernel itself
  if (w4_linear_local(rows, in_features, 32)) return DG_ERROR_BLOCK_BYTES;
  return DG_ERROR_BLOCK_BYTES + w4_linear_scratch_bytes(rows, in_features);
}

dg_status dg_w4_linear(int64_t rows, int64_t in_f, int64_t out_f, int32_t group, const void* x, const void* codes,
                       const void* scales, const void* zeros, const void* bias, void* y, void* ws, size_t ws_bytes,
                       void* stream) {
  if (rows < 0 || out_f < 1) return fail(DG_ERR_INVALID_ARGUMENT, "w4_linear: rows must be >= 0, out_features >= 1");
  dg_status st = check_w4(out_f, in_f, group, "w4_linear");
  if (st != DG_OK) return st;
  if (rows > kMaxW4LinearRows)
    return fail(DG_ERR_UNSUPPORTED, "w4_linear: more than %d rows", static_cast<int>(kMaxW4LinearRows));
  if (out_f > kMaxDim - 256 || in_f > kMaxDim / 4)
    return fail(DG_ERR_UNSUPPORTED, "w4_linear: out_features beyond 2^31 - 256, or in_features beyond 2^29");
  if (rows == 0) return DG_OK;
  const size_t need = dg_w4_linear_workspace_bytes(rows, in_f, out_f);
  const Arg args[] = {{"x", x, static_cast<size_t>(rows) * in_f * 2, false, false},
                      {"codes", codes, code_bytes(out_f, in_f), false, false},
                      {"scales", scales, scale_bytes(out_f, in_f, group), false, false},
                      {"zeros", zeros, zero_bytes(out_f, in_f, group), true, false},
                      {"bias", bias, static_cast<size_t>(out_f) * 2, true, false},
                      {"y", y, static_cast<size_t>(rows) * out_f * 2, false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("w4_linear", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "w4_linear")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "w4_linear: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "w4_linear")) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double kn = static_cast<double>(in_f) * out_f;
  TraceScope trace("w4_linear", s, 2.0 * rows * kn,
                   kn * (0.5 + (zeros ? 3.0 : 2.0) / group) + 2.0 * rows * (static_cast<double>(in_f) + out_f));
  return launched(launch_w4_linear(x, codes, scales, zeros, bias, y, static_cast<int>(rows), static_cast<int>(in_f),
                                   static_cast<int>(out_f), group, static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES,
                                   dev, s),
                  "w4_linear");
}

size_t dg_moe_route_workspace_bytes(int64_t T, int64_t d, int32_t E, int32_t k) {
  (void)d;
  (void)k;
  if (T < 0 || E < 1) return 0;
  return DG_ERROR_BLOCK_BYTES + static_cast<size_t>(T) * E * 4;
}

dg_status dg_moe_route(int64_t T, int64_t d, int32_t E, int32_t k, uint32_t flags, float scale, const void* x,
                       const void* w_router, void* idx, void* gates, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || d < 1 || E < 1) return fail(DG_ERR_INVALID_ARGUMENT, "moe_route: T must be >= 0, d and E >= 1");
  if (d % 8) return fail(DG_ERR_INVALID_ARGUMENT, "moe_route: d must be a multiple of 8");
  if (k < 1 || k > E) return fail(DG_ERR_INVALID_ARGUMENT, "moe_route: k must be between 1 and E");
  if (flags & ~(DG_MOE_SIGMOID | DG_MOE_RENORM))
    return fail(DG_ERR_INVALID_ARGUMENT, "moe_route: unknown flags %u", flags);
  if (E > moe_max_experts() || k > moe_max_topk())
    return fail(DG_ERR_UNSUPPORTED, "moe_route: more than %d experts or %d choices per token", moe_max_experts(),
                moe_max_topk());
  if (d > kMaxRouteDim || T > 65535 * 4)
    return fail(DG_ERR_UNSUPPORTED, "moe_route: more than %d tokens, or d beyond 2^31 - 8192", 65535 * 4);
  if (T == 0) return DG_OK;
  const size_t need = dg_moe_route_workspace_bytes(T, d, E, k);
  const Arg args[] = {{"x", x, static_cast<size_t>(T) * d * 2, false, false},
                      {"w_router", w_router, static_cast<size_t>(E) * d * 2, false, false},
                      {"idx", idx, static_cast<size_t>(T) * k * 4, false, true},
                      {"gates", gates, static_cast<size_t>(T) * k * 4, false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  dg_status st = check_args("moe_route", args);
  if (st != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "moe_route")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "moe_route: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "moe_route")) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* logits = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES);
  {
    TraceScope trace("moe_logits", s, 2.0 * T * E * d, 2.0 * d * (static_cast<double>(T) + E));
    st = launched(launch_moe_logits(x, w_router, logits, static_cast<int>(T), static_cast<int>(d), E, dev, s),
                  "moe_route");
    if (st != DG_OK) return st;
  }
  TraceScope trace("moe_topk", s, 0.0, 4.0 * T * E + 8.0 * T * k);
  return launched(launch_moe_topk(logits, idx, gates, static_cast<int>(T), E, k, (flags & DG_MOE_SIGMOID) != 0,
                                  (flags & DG_MOE_RENORM) != 0, scale, dev, s),
                  "moe_route");
}

size_t dg_moe_swiglu_workspace_bytes(const dg_moe_shape* shape, int32_t group) {
  if (check_moe(shape, "moe_swiglu") != DG_OK) return 0;
  if (group != 0 && group != 32 && group != 64 && group != 128) {
    fail(DG_ERR_INVALID_ARGUMENT, "moe_swiglu: group is %d, not 0 (bf16), 32, 64 or 128", group);
    return 0;
  }
  return moe_need(*shape, group);
}

dg_status dg_moe_swiglu(const dg_moe_shape* shape, const void* x, const void* idx, const void* gates,
                        const void* w13, const void* w2, void* y, void* ws, size_t ws_bytes, void* stream) {
  dg_status st = check_moe(shape, "moe_swiglu");
  if (st != DG_OK || shape->T == 0) return st;
  const dg_moe_shape& s = *shape;
  const size_t need = moe_need(s, 0);
  const size_t wn = static_cast<size_t>(s.E) * s.d * s.F * 2, xn = static_cast<size_t>(s.T) * s.d * 2;
  const size_t pn = static_cast<size_t>(s.T) * s.k * 4;
  const Arg args[] = {{"x", x, xn, false, false},        {"idx", idx, pn, false, false},
                      {"gates", gates, pn, false, false}, {"w13", w13, 2 * wn, false, false},
                      {"w2", w2, wn, false, false},       {"y", y, xn, false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("moe_swiglu", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "moe_swiglu")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "moe_swiglu: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "moe_swiglu")) != DG_OK) return st;
  const MoeCall call{x, idx, gates, w13, nullptr, nullptr, w2, nullptr, nullptr, y,
                     static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES, s.T, s.k, s.E, s.d, s.F, 0};
  MoeTrace trace(static_cast<cudaStream_t>(stream));
  return launched(launch_moe_swiglu(call, dev, static_cast<cudaStream_t>(stream), &trace), "moe_swiglu");
}

dg_status dg_moe_swiglu_w4(const dg_moe_shape* shape, int32_t group, const void* x, const void* idx,
                           const void* gates, const void* w13_codes, const void* w13_scales, const void* w13_zeros,
                           const void* w2_codes, const void* w2_scales, const void* w2_zeros, void* y, void* ws,
                           size_t ws_bytes, void* stream) {
  dg_status st = check_moe(shape, "moe_swiglu_w4");
  if (st != DG_OK) return st;
  const dg_moe_shape& s = *shape;
  if (group != 32 && group != 64 && group != 128)
    return fail(DG_ERR_INVALID_ARGUMENT, "moe_swiglu_w4: group is %d, not 32, 64 or 128", group);
  if (s.d % group || s.F % group)
    return fail(DG_ERR_INVALID_ARGUMENT, "moe_swiglu_w4: d and F must be multiples of the group");
  if ((w13_zeros == nullptr) != (w2_zeros == nullptr))
    return fail(DG_ERR_INVALID_ARGUMENT, "moe_swiglu_w4: w13_zeros and w2_zeros must both be given or both be NULL");
  if (s.T == 0) return DG_OK;
  const size_t need = moe_need(s, group);
  const int64_t up_rows = static_cast<int64_t>(s.E) * 2 * s.F, down_rows = static_cast<int64_t>(s.E) * s.d;
  const size_t xn = static_cast<size_t>(s.T) * s.d * 2, pn = static_cast<size_t>(s.T) * s.k * 4;
  const Arg args[] = {{"x", x, xn, false, false},
                      {"idx", idx, pn, false, false},
                      {"gates", gates, pn, false, false},
                      {"w13_codes", w13_codes, code_bytes(up_rows, s.d), false, false},
                      {"w13_scales", w13_scales, scale_bytes(up_rows, s.d, group), false, false},
                      {"w13_zeros", w13_zeros, zero_bytes(up_rows, s.d, group), true, false},
                      {"w2_codes", w2_codes, code_bytes(down_rows, s.F), false, false},
                      {"w2_scales", w2_scales, scale_bytes(down_rows, s.F, group), false, false},
                      {"w2_zeros", w2_zeros, zero_bytes(down_rows, s.F, group), true, false},
                      {"y", y, xn, false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("moe_swiglu_w4", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "moe_swiglu_w4")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "moe_swiglu_w4: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "moe_swiglu_w4")) != DG_OK) return st;
  const MoeCall call{x, idx, gates, w13_codes, w13_scales, w13_zeros, w2_codes, w2_scales, w2_zeros, y,
                     static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES, s.T, s.k, s.E, s.d, s.F, group};
  MoeTrace trace(static_cast<cudaStream_t>(stream));
  return launched(launch_moe_swiglu(call, dev, static_cast<cudaStream_t>(stream), &trace), "moe_swiglu_w4");
}

}  // extern "C"
