// The C ABI of the block-scaled e4m3 operators (include/dg.h): quantiser, linear
// with its gradients, root-mean-square norm.  Argument checks, scratch carving,
// tensor maps and launches.
#include <cuda_runtime.h>

#include "dg_internal.h"
#include "dg_mx.cuh"

namespace dg {

namespace {

constexpr int64_t kMaxDim = 0x7fffffff - 1024;  // tile coordinates step past the last row and column in 32 bits
constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int kMaxNormDim = 32768;
constexpr float kMinEps = 1e-30f;  // squares below binary32's range stay far below it

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }
size_t elements(int64_t a, int64_t b) { return static_cast<size_t>(a) * static_cast<size_t>(b); }
size_t scale_bytes(int64_t rows, int64_t K, int block_rows) {
  return elements(block_rows == 1 ? rows : blocks128(rows), blocks128(K));
}

dg_status check_matrix(int64_t rows, int64_t K, const char* what) {
  if (rows < 0 || K < 1) return fail(DG_ERR_INVALID_ARGUMENT, "%s: rows must be >= 0 and the row length >= 1", what);
  if (K % 16) return fail(DG_ERR_INVALID_ARGUMENT, "%s: the row length must be a multiple of 16", what);
  if (rows > kMaxDim || K > kMaxDim || rows * blocks128(K) > kMaxElements / 128)
    return fail(DG_ERR_UNSUPPORTED, "%s: a size beyond 2^31 - 1025, or more than 2^40 elements", what);
  return DG_OK;
}

dg_status check_format(int64_t rows, int64_t K, int32_t block_rows, const char* what) {
  if (block_rows != 1 && block_rows != 128)
    return fail(DG_ERR_INVALID_ARGUMENT, "%s: block_rows is %d, not 1 or 128", what, block_rows);
  return check_matrix(rows, K, what);
}

dg_status check_linear(int64_t rows, int64_t in_f, int64_t out_f, const char* what) {
  if (rows < 0 || in_f < 1 || out_f < 1)
    return fail(DG_ERR_INVALID_ARGUMENT, "%s: rows must be >= 0, in_features and out_features >= 1", what);
  if (in_f % 16 || out_f % 16)
    return fail(DG_ERR_INVALID_ARGUMENT, "%s: in_features and out_features must be multiples of 16", what);
  dg_status st = check_matrix(rows, in_f, what);
  if (st == DG_OK) st = check_matrix(rows, out_f, what);
  if (st == DG_OK) st = check_matrix(out_f, in_f, what);
  return st;
}

dg_status check_norm(int64_t rows, int64_t d, float eps, const char* what) {
  if (rows < 0 || d < 1) return fail(DG_ERR_INVALID_ARGUMENT, "%s: rows must be >= 0 and d >= 1", what);
  if (d % 8) return fail(DG_ERR_INVALID_ARGUMENT, "%s: d must be a multiple of 8", what);
  if (!(eps >= kMinEps && eps <= 3.4e38f)) return fail(DG_ERR_INVALID_ARGUMENT, "%s: eps must be finite and >= 1e-30", what);
  if (d > kMaxNormDim) return fail(DG_ERR_UNSUPPORTED, "%s: d beyond %d", what, kMaxNormDim);
  if (rows > kMaxDim) return fail(DG_ERR_UNSUPPORTED, "%s: rows beyond 2^31 - 1025", what);
  return DG_OK;
}

// One block-scaled product D [M, N] = A [M, K] B^T (+ bias), B [N, K], or [K, N] where b_mn_major.  sb are the scales of
// B's 128 x 128 blocks, [N][K], or [K][N] where sb_turned.
dg_status run_mx(bool b_mn_major, bool sb_turned, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                 const void* b, const void* sb, const void* bias, void* d, const DeviceInfo& dev, cudaStream_t s,
                 const char* name) {
  CUtensorMap ma, mb, md;
  dg_status st;
  const uint64_t m = M, n = N, k = K;
  if ((st = make_map_3d(&ma, false, a, k, m, 1, k, m * k, 128, 128, 1, "codes")) != DG_OK) return st;
  const int tile_n = mx_tile_n(b_mn_major, M, N, dev);
  st = b_mn_major ? make_map_3d(&mb, false, b, n, k, 1, n, n * k, 128, 128, 1, "weight codes (N-major)")
                  : make_map_3d(&mb, false, b, k, n, 1, k, n * k, 128, tile_n / 2, 1, "weight codes");
  if (st != DG_OK) return st;
  if ((st = make_map_3d_sw(&md, true, d, n, m, 1, 2 * n, 2 * n * m, 32, 32, 1, 64, "output")) != DG_OK) return st;
  MxParams p{};
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.sa = static_cast<const uint8_t*>(sa);
  p.ka = static_cast<int32_t>(blocks128(K));
  p.sb = static_cast<const uint8_t*>(sb);
  p.sb_n = sb_turned ? 1 : p.ka;
  p.sb_k = sb_turned ? static_cast<int32_t>(blocks128(N)) : 1;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.err = dev.err;
  const double w = static_cast<double>(N) * K;
  TraceScope trace(name, s, 2.0 * M * w, static_cast<double>(M) * K + w + 2.0 * M * N);
  return launched(launch_gemm_mx(b_mn_major, tile_n, ma, mb, md, p, dev, s), name);
}

// The product for few rows; sx NULL: x is bf16.
dg_status run_mx_few(const MxFewPlan& plan, int64_t M, int64_t N, int64_t K, const void* x, const void* sx,
                     const void* w, const void* sw, const void* bias, void* y, const DeviceInfo& dev, cudaStream_t s,
                     const char* name) {
  CUtensorMap mw, mx;
  dg_status st;
  const uint64_t m = M, n = N, k = K;
  if ((st = make_map_3d(&mw, false, w, k, n, 1, k, n * k, 128, 128, 1, "weight codes")) != DG_OK) return st;
  if (sx && (st = make_map_3d(&mx, false, x, k, m, 1, k, m * k, 128, plan.nt, 1, "codes")) != DG_OK) return st;
  const double wn = static_cast<double>(N) * K;
  TraceScope trace(name, s, 2.0 * M * wn, static_cast<double>(M) * K + wn + 2.0 * M * N);
  const int Mi = static_cast<int>(M), Ni = static_cast<int>(N), Ki = static_cast<int>(K);
  return launched(sx ? launch_mx_few(plan, mw, mx, sw, sx, bias, y, Mi, Ni, Ki, dev, s)
                     : launch_mx_few_bf16(plan, mw, x, sw, bias, y, Mi, Ni, Ki, dev, s),
                  name);
}

dg_status run_linear(int64_t rows, int64_t in_f, int64_t out_f, const void* x, const void* sx, const void* w,
                     const void* sw, const void* bias, void* y, const DeviceInfo& dev, cudaStream_t s) {
  const MxFewPlan few = mx_few_plan(rows, out_f, in_f, dev);
  if (few.better) return run_mx_few(few, rows, out_f, in_f, x, sx, w, sw, bias, y, dev, s, "fp8_linear_few");
  return run_mx(false, false, rows, out_f, in_f, x, sx, w, sw, bias, y, dev, s, "fp8_linear");
}

// Workspace of the backward: the error block, and what the gradients that are asked for need: for dx dy in 8 bits and the
// weight's codes turned, for d_bias partial column sums, for d_weight x in bf16.
// With many rows the product for dx takes the weight's codes with the contraction along their rows: as they lie, a
// CTA's 112 columns of a 224-column tile begin anywhere in a 128-byte line, and the copies cost 25 of 100 of its time
// (8192 rows, 14336 to 4096: 349 us against 276); turning them costs 2 bytes of traffic a weight, which pays from about
// 2000 rows on.
constexpr int64_t kTurnRows = 2048;
struct BwdLayout {
  size_t dy_codes, dy_scales, sums, w_turned, x, total;
  bool turn;
};
BwdLayout bwd_layout(int64_t rows, int64_t in_f, int64_t out_f, bool dx, bool d_weight, bool d_bias) {
  BwdLayout l;
  size_t at = DG_ERROR_BLOCK_BYTES;
  auto take = [&](bool wanted, size_t bytes) {
    const size_t here = at;
    at = round256(at + (wanted ? bytes : 0));
    return here;
  };
  l.turn = rows >= kTurnRows && out_f <= 65535 * 128;
  l.dy_codes = take(dx, elements(rows, out_f));
  l.dy_scales = take(dx, scale_bytes(rows, out_f, 1));
  l.sums = take(d_bias, 4 * elements(fp8_quantize_sum_parts(rows, static_cast<int>(out_f)), out_f));
  l.w_turned = take(dx && l.turn, elements(out_f, in_f));
  l.x = take(d_weight, 2 * elements(rows, in_f));
  l.total = at;
  return l;
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_fp8_quantize(int64_t rows, int64_t K, int32_t block_rows, const void* x, void* codes, void* scales,
                          void* stream) {
  dg_status st = check_format(rows, K, block_rows, "fp8_quantize");
  if (st != DG_OK || rows == 0) return st;
  const size_t n = elements(rows, K);
  const Arg args[] = {{"x", x, 2 * n, false, false},
                      {"codes", codes, n, false, true},
                      {"scales", scales, scale_bytes(rows, K, block_rows), false, true, true}};
  if ((st = check_args("fp8_quantize", args)) != DG_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("fp8_quantize", s, 0.0, 3.0 * n);
  return launched(launch_fp8_quantize(x, codes, scales, rows, static_cast<int>(K), block_rows, s), "fp8_quantize");
}

dg_status dg_fp8_dequantize(int64_t rows, int64_t K, int32_t block_rows, const void* codes, const void* scales,
                            void* x, void* stream) {
  dg_status st = check_format(rows, K, block_rows, "fp8_dequantize");
  if (st != DG_OK || rows == 0) return st;
  const size_t n = elements(rows, K);
  const Arg args[] = {{"codes", codes, n, false, false},
                      {"scales", scales, scale_bytes(rows, K, block_rows), false, false, true},
                      {"x", x, 2 * n, false, true}};
  if ((st = check_args("fp8_dequantize", args)) != DG_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("fp8_dequantize", s, 0.0, 3.0 * n);
  return launched(launch_fp8_dequantize(codes, scales, x, rows, static_cast<int>(K), block_rows, s), "fp8_dequantize");
}

// Where the activations come in bf16, their codes and scales lie in the workspace behind the error block.
static size_t linear_scales_at(int64_t rows, int64_t in_f) {
  return round256(DG_ERROR_BLOCK_BYTES + elements(rows, in_f));
}

size_t dg_fp8_linear_bf16_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features) {
  if (check_linear(rows, in_features, out_features, "fp8_linear_bf16") != DG_OK) return 0;
  return linear_scales_at(rows, in_features) + round256(scale_bytes(rows, in_features, 1));
}

dg_status dg_fp8_linear_bf16(int64_t rows, int64_t in_f, int64_t out_f, const void* x, const void* w_codes,
                             const void* w_scales, const void* bias, void* y, void* ws, size_t ws_bytes, void* stream) {
  dg_status st = check_linear(rows, in_f, out_f, "fp8_linear_bf16");
  if (st != DG_OK || rows == 0) return st;
  const size_t scales_at = linear_scales_at(rows, in_f), need = scales_at + round256(scale_bytes(rows, in_f, 1));
  const Arg args[] = {{"x", x, 2 * elements(rows, in_f), false, false},
                      {"w_codes", w_codes, elements(out_f, in_f), false, false},
                      {"w_scales", w_scales, scale_bytes(out_f, in_f, 128), false, false, true},
                      {"bias", bias, 2 * static_cast<size_t>(out_f), true, false},
                      {"y", y, 2 * elements(rows, out_f), false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("fp8_linear_bf16", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "fp8_linear_bf16")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "fp8_linear_bf16: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "fp8_linear_bf16")) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const MxFewPlan few = mx_few_plan(rows, out_f, in_f, dev);
  if (rows <= kMxFewBf16Rows)
    return run_mx_few(few, rows, out_f, in_f, x, nullptr, w_codes, w_scales, bias, y, dev, s, "fp8_linear_few_bf16");
  uint8_t* codes = static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES;
  uint8_t* scales = static_cast<uint8_t*>(ws) + scales_at;
  {
    TraceScope trace("fp8_quantize", s, 0.0, 3.0 * elements(rows, in_f));
    st = launched(launch_fp8_quantize(x, codes, scales, rows, static_cast<int>(in_f), 1, s), "fp8_linear_bf16");
    if (st != DG_OK) return st;
  }
  return run_linear(rows, in_f, out_f, codes, scales, w_codes, w_scales, bias, y, dev, s);
}

size_t dg_fp8_linear_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features) {
  if (check_linear(rows, in_features, out_features, "fp8_linear") != DG_OK) return 0;
  return DG_ERROR_BLOCK_BYTES;
}

dg_status dg_fp8_linear(int64_t rows, int64_t in_f, int64_t out_f, const void* x_codes, const void* x_scales,
                        const void* w_codes, const void* w_scales, const void* bias, void* y, void* ws, size_t ws_bytes,
                        void* stream) {
  dg_status st = check_linear(rows, in_f, out_f, "fp8_linear");
  if (st != DG_OK || rows == 0) return st;
  const size_t need = dg_fp8_linear_workspace_bytes(rows, in_f, out_f);
  const Arg args[] = {{"x_codes", x_codes, elements(rows, in_f), false, false},
                      {"x_scales", x_scales, scale_bytes(rows, in_f, 1), false, false, true},
                      {"w_codes", w_codes, elements(out_f, in_f), false, false},
                      {"w_scales", w_scales, scale_bytes(out_f, in_f, 128), false, false, true},
                      {"bias", bias, 2 * static_cast<size_t>(out_f), true, false},
                      {"y", y, 2 * elements(rows, out_f), false, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("fp8_linear", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "fp8_linear")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "fp8_linear: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "fp8_linear")) != DG_OK) return st;
  return run_linear(rows, in_f, out_f, x_codes, x_scales, w_codes, w_scales, bias, y, dev,
                    static_cast<cudaStream_t>(stream));
}

size_t dg_fp8_linear_bwd_workspace_bytes_for(int64_t rows, int64_t in_features, int64_t out_features, int32_t dx,
                                             int32_t d_weight, int32_t d_bias) {
  if (check_linear(rows, in_features, out_features, "fp8_linear_bwd") != DG_OK) return 0;
  return bwd_layout(rows, in_features, out_features, dx != 0, d_weight != 0, d_bias != 0).total;
}

size_t dg_fp8_linear_bwd_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features) {
  return dg_fp8_linear_bwd_workspace_bytes_for(rows, in_features, out_features, 1, 1, 1);
}

dg_status dg_fp8_linear_bwd(int64_t rows, int64_t in_f, int64_t out_f, const void* x_codes, const void* x_scales,
                            const void* w_codes, const void* w_scales, const void* dy, void* dx, void* d_weight,
                            void* d_bias, void* ws, size_t ws_bytes, void* stream) {
  dg_status st = check_linear(rows, in_f, out_f, "fp8_linear_bwd");
  if (st != DG_OK) return st;
  const size_t xn = elements(rows, in_f), wn = elements(out_f, in_f), yn = elements(rows, out_f);
  const BwdLayout l = bwd_layout(rows, in_f, out_f, dx != nullptr, d_weight != nullptr, d_bias != nullptr);
  const bool any = rows > 0;
  const Arg args[] = {{"x_codes", x_codes, xn, !(any && d_weight), false},
                      {"x_scales", x_scales, scale_bytes(rows, in_f, 1), !(any && d_weight), false, true},
                      {"w_codes", w_codes, wn, !(any && dx), false},
                      {"w_scales", w_scales, scale_bytes(out_f, in_f, 128), !(any && dx), false, true},
                      {"dy", dy, 2 * yn, !(any && (dx || d_weight || d_bias)), false},
                      {"dx", dx, 2 * xn, true, true},
                      {"d_weight", d_weight, 2 * wn, true, true},
                      {"d_bias", d_bias, 2 * static_cast<size_t>(out_f), true, true},
                      {"ws", ws, ws ? l.total : 0, true, true}};
  if ((st = check_args("fp8_linear_bwd", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "fp8_linear_bwd")) != DG_OK) return st;
  if (ws_bytes < l.total)
    return fail(DG_ERR_WORKSPACE, "fp8_linear_bwd: workspace has %zu bytes, needs %zu", ws_bytes, l.total);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "fp8_linear_bwd")) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (!any) {
    cudaError_t e = d_weight ? cudaMemsetAsync(d_weight, 0, 2 * wn, s) : cudaSuccess;
    if (e == cudaSuccess && d_bias) e = cudaMemsetAsync(d_bias, 0, 2 * static_cast<size_t>(out_f), s);
    return launched(e, "fp8_linear_bwd");
  }
  if (dx) {
    {
      // the bias's gradient comes along: dy is read once for both
      TraceScope trace("fp8_bwd_quantize_dy", s, 0.0, 3.0 * yn);
      const int K = static_cast<int>(out_f);
      st = launched(d_bias ? launch_fp8_quantize_sum(dy, base + l.dy_codes, base + l.dy_scales, d_bias,
                                                     reinterpret_cast<float*>(base + l.sums), rows, K, dev.err, s)
                           : launch_fp8_quantize(dy, base + l.dy_codes, base + l.dy_scales, rows, K, 1, s),
                    "fp8_linear_bwd");
      if (st != DG_OK) return st;
    }
    const void* b = w_codes;
    if (l.turn) {
      TraceScope trace("fp8_bwd_turn_w", s, 0.0, 2.0 * wn);
      b = base + l.w_turned;
      st = launched(launch_transpose_codes(w_codes, base + l.w_turned, static_cast<int>(out_f), static_cast<int>(in_f), s),
                    "fp8_linear_bwd");
      if (st != DG_OK) return st;
    }
    if ((st = run_mx(!l.turn, true, rows, in_f, out_f, base + l.dy_codes, base + l.dy_scales, b, w_scales, nullptr, dx,
                     dev, s, "fp8_linear_bwd_dx")) != DG_OK)
      return st;
  }
  if (d_weight) {
    // d_weight = dy^T x: the bf16 GEMM with both operands MN-major, x expanded to bf16 (exactly) beforehand
    uint8_t* x = base + l.x;
    {
      TraceScope trace("fp8_bwd_expand_x", s, 0.0, 3.0 * xn);
      st = launched(launch_fp8_dequantize(x_codes, x_scales, x, rows, static_cast<int>(in_f), 1, s), "fp8_linear_bwd");
      if (st != DG_OK) return st;
    }
    const uint64_t R = rows, I = in_f, O = out_f;
    CUtensorMap mdy, mx, mdw;
    GemmParams p{};
    if ((st = make_map_mn(&mdy, dy, O, R, 1, O * 2, R * O * 2, 64, 1, kMnBlocksA, &p.a_mn4, "dy^T")) != DG_OK) return st;
    if ((st = make_map_mn(&mx, x, I, R, 1, I * 2, R * I * 2, 64, 1, kMnBlocksB, &p.b_mn4, "x (N-major)")) != DG_OK)
      return st;
    if ((st = make_map_3d(&mdw, true, d_weight, I, O, 1, I * 2, O * I * 2, 64, 32, 1, "d_weight")) != DG_OK) return st;
    p.G = 1;
    p.M = static_cast<int32_t>(out_f);
    p.N = static_cast<int32_t>(in_f);
    p.K = static_cast<int32_t>(rows);
    p.a_g = p.b_g = p.d_g = G_OUTER;
    if ((st = run_gemm(GV_BF16_MM_STORE, mdy, mx, mdw, mdw, p, dev, s, "fp8_linear_bwd_dw",
                       2.0 * (static_cast<double>(yn) + xn + wn))) != DG_OK)
      return st;
  }
  if (d_bias && !dx) {
    TraceScope trace("fp8_linear_bwd_db", s, 0.0, 2.0 * yn + 2.0 * out_f);
    return launched(launch_fp8_quantize_sum(dy, nullptr, nullptr, d_bias, reinterpret_cast<float*>(base + l.sums), rows,
                                            static_cast<int>(out_f), dev.err, s),
                    "fp8_linear_bwd");
  }
  return DG_OK;
}

dg_status dg_rms_norm(int64_t rows, int64_t d, float eps, const void* x, const void* residual, const void* weight,
                      void* h, void* y, void* codes, void* scales, void* stream) {
  dg_status st = check_norm(rows, d, eps, "rms_norm");
  if (st != DG_OK) return st;
  if ((codes == nullptr) != (scales == nullptr) || (codes == nullptr) == (y == nullptr)) {
    if (rows == 0 && !codes && !scales && !y) return DG_OK;
    return fail(DG_ERR_INVALID_ARGUMENT, "rms_norm: y, or codes and scales, must be given (the others NULL)");
  }
  if (codes && d % 16) return fail(DG_ERR_INVALID_ARGUMENT, "rms_norm: d must be a multiple of 16 for codes");
  if (rows == 0) return DG_OK;
  if ((residual == nullptr) != (h == nullptr))
    return fail(DG_ERR_INVALID_ARGUMENT, "rms_norm: residual and h must both be given or both be NULL");
  const size_t n = elements(rows, d);
  const Arg args[] = {{"x", x, 2 * n, false, false},         {"residual", residual, 2 * n, true, false},
                      {"weight", weight, 2 * static_cast<size_t>(d), false, false},
                      {"h", h, 2 * n, true, true},           {"y", y, 2 * n, true, true},
                      {"codes", codes, n, true, true},       {"scales", scales, scale_bytes(rows, d, 1), true, true, true}};
  if ((st = check_args("rms_norm", args)) != DG_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("rms_norm", s, 0.0, (residual ? 6.0 : 2.0) * n + (codes ? 1.0 : 2.0) * n);
  return launched(launch_rms_norm(x, residual, weight, h, y, codes, scales, rows, static_cast<int>(d), eps, s),
                  "rms_norm");
}

size_t dg_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  if (check_norm(rows, d, 1.0f, "rms_norm_bwd") != DG_OK) return 0;
  return DG_ERROR_BLOCK_BYTES + rms_norm_bwd_scratch_bytes(rows, static_cast<int>(d));
}

dg_status dg_rms_norm_bwd(int64_t rows, int64_t d, float eps, const void* h, const void* weight, const void* dy,
                          const void* dh, void* dx, void* d_weight, void* ws, size_t ws_bytes, void* stream) {
  dg_status st = check_norm(rows, d, eps, "rms_norm_bwd");
  if (st != DG_OK) return st;
  const size_t n = elements(rows, d), need = dg_rms_norm_bwd_workspace_bytes(rows, d);
  const bool any = rows > 0 && (dx || d_weight);
  const Arg args[] = {{"h", h, 2 * n, !any, false},
                      {"weight", weight, 2 * static_cast<size_t>(d), !any, false},
                      {"dy", dy, 2 * n, !any, false},
                      {"dh", dh, 2 * n, true, false},
                      {"dx", dx, 2 * n, true, true},
                      {"d_weight", d_weight, 2 * static_cast<size_t>(d), true, true},
                      {"ws", ws, ws ? need : 0, true, true}};
  if ((st = check_args("rms_norm_bwd", args)) != DG_OK) return st;
  if ((st = check_error_block(ws, ws_bytes, "rms_norm_bwd")) != DG_OK) return st;
  if (ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "rms_norm_bwd: workspace has %zu bytes, needs %zu", ws_bytes, need);
  DeviceInfo dev;
  if ((st = device_info_ws(&dev, ws, ws_bytes, "rms_norm_bwd")) != DG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!any) {
    return d_weight ? launched(cudaMemsetAsync(d_weight, 0, 2 * static_cast<size_t>(d), s), "rms_norm_bwd") : DG_OK;
  }
  TraceScope trace("rms_norm_bwd", s, 0.0, (dh ? 8.0 : 6.0) * n);
  return launched(launch_rms_norm_bwd(h, weight, dy, dh, dx, d_weight,
                                      static_cast<uint8_t*>(ws) + DG_ERROR_BLOCK_BYTES, rows, static_cast<int>(d), eps, dev.err,
                                      s),
                  "rms_norm_bwd");
}

}  // extern "C"
