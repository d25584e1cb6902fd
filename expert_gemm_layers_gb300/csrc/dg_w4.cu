// 4-bit weights with one scale (and optionally one zero point) per group of
// 32, 64 or 128 consecutive columns of a row: quantising, reading back, and
// the product with a few activation rows.
//
//   value[o, k] = (q[o, k] - z[o, g]) * s[o, g],  g = k / group
//
// Codes are two to a byte along k, the even column in the low nibble.
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "dg_w4dot.cuh"

namespace dg {

namespace {

__device__ __forceinline__ bool err_set(const uint32_t* err) { return ld_volatile_u32(err) != 0u; }

constexpr int kVecCols = 8;  // columns a thread handles: 16 bytes of bf16, 4 bytes of codes

// One thread per 8 columns; the GROUP / 8 lanes of a group agree on its scale
// by shuffles.  A group with a NaN or an infinity, or whose range overflows
// binary32, gets a NaN scale.
template <int GROUP, bool ZEROS>
__global__ void w4_quantize_kernel(const uint4* __restrict__ w, uint32_t* __restrict__ codes,
                                   __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ zeros, int64_t vecs) {
  griddep_wait();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  // vecs is a multiple of the GROUP / 8 lanes of a group, so groups are whole;
  // lanes past the end only keep the shuffles convergent
  const bool in = v < vecs;
  const uint4 raw = in ? __ldg(w + v) : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
  float f[8];
  float lo = 0.0f, hi = 0.0f;
  uint32_t top = 0u;  // largest magnitude, as bits: NaN > inf > finite
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(word[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
    lo = fminf(lo, fminf(p.x, p.y));
    hi = fmaxf(hi, fmaxf(p.x, p.y));
    top = max(top, max(word[i] & 0x7fffu, (word[i] >> 16) & 0x7fffu));
  }
#pragma unroll
  for (int o = GROUP / kVecCols / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (!in) return;
  const float quot = ZEROS ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(fmaxf(-lo, hi), 7.0f);
  const bool finite = top < 0x7f80u && isfinite(quot);
  __nv_bfloat16 sb = __float2bfloat16_rn(quot);
  float s = __bfloat162float(sb);
  if (s == 0.0f) s = 1.0f;
  if (!finite) s = __int_as_float(0x7fc00000);
  sb = __float2bfloat16_rn(s);
  float z = 8.0f;
  if (ZEROS && finite) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
  uint32_t code = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = finite ? fminf(fmaxf(rintf(__fdiv_rn(f[i], s)) + z, 0.0f), 15.0f) : z;
    code |= static_cast<uint32_t>(q) << (4 * i);
  }
  codes[v] = code;
  if (v % (GROUP / kVecCols) == 0) {
    const int64_t g = v / (GROUP / kVecCols);
    scales[g] = sb;
    if (ZEROS) zeros[g] = static_cast<uint8_t>(z);
  }
}

// One thread per 8 columns: 4 bytes of codes in, 16 bytes of bf16 out, each
// value rounded once from the exact binary32 product.
template <int GROUP, bool ZEROS>
__global__ void w4_dequantize_kernel(const uint32_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                                     const uint8_t* __restrict__ zeros, uint4* __restrict__ w, int64_t vecs) {
  griddep_wait();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (v >= vecs) return;
  const int64_t g = v / (GROUP / kVecCols);
  const uint32_t code = __ldg(codes + v);
  const float s = __bfloat162float(scales[g]);
  const float z = ZEROS ? static_cast<float>(zeros[g] & 15) : 8.0f;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = static_cast<float>((code >> (8 * i)) & 15u) - z;
    const float b = static_cast<float>((code >> (8 * i + 4)) & 15u) - z;
    out[i] = pack_bf16x2(a * s, b * s);
  }
  w[v] = make_uint4(out[0], out[1], out[2], out[3]);
}

// Activation rows staged once for all CTAs of the product (w4_stage_piece): half
// a warp a (row, step).
template <int GROUP>
__global__ void __launch_bounds__(256)
    w4_stage_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ frag, float2* __restrict__ fx, int rows,
                    int K, const uint32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  const int steps = w4_steps(K), p = threadIdx.x & 15;
  const int64_t total = static_cast<int64_t>(rows) * steps, rb = w4_row_bytes(K);
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 5) * 2; i0 < total;
       i0 += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t i = i0 + ((threadIdx.x >> 4) & 1), row = i / steps;
    const int st = static_cast<int>(i - row * steps), k = st * kW4Step + 8 * p;
    const bool exists = i < total;
    float f[8];
    unpack_piece(exists && k < K ? *reinterpret_cast<const uint4*>(x + row * K + k) : make_uint4(0u, 0u, 0u, 0u), f);
    w4_stage_piece<GROUP>(f, p, st, exists, frag + row * rb, fx + row * w4_fx_stride<GROUP>(K));
  }
}

// y = x W^T (+ bias): a CTA takes 8 / WK blocks of 32 weight rows and up to 8*NT
// activation rows.  LOCAL: it stages those itself, in shared memory (x); else they
// come staged (frag, fx).
template <int GROUP, int NT, bool LOCAL>
__global__ void __launch_bounds__(kRowWarps * 32, NT == 1 ? 3 : NT == 2 ? 2 : 1)
    w4_linear_kernel(const __nv_bfloat16* __restrict__ x, const uint8_t* __restrict__ frag,
                     const float2* __restrict__ fx, const uint8_t* __restrict__ codes,
                     const __nv_bfloat16* __restrict__ scales, const uint8_t* __restrict__ zeros,
                     const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ y, int rows, int K, int N, int WK, const uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t failed = ld_volatile_u32(err);  // looked at before anything is written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk = warp % WK, rg = warp / WK;
  const int r0 = (static_cast<int>(blockIdx.x) * (kRowWarps / WK) + rg) * 16 * kRowTiles;
  const int n0 = static_cast<int>(blockIdx.y) * 8 * NT, count = min(rows - n0, 8 * NT);
  const int64_t rb = w4_row_bytes(K);
  const int fs = w4_fx_stride<GROUP>(K), steps = w4_steps(K);
  uint8_t* joins = smem;
  if constexpr (LOCAL) {
    uint8_t* xs = smem + joins_bytes<NT>(WK);
    float2* xf = reinterpret_cast<float2*>(xs + count * rb);
    const int p = threadIdx.x & 15, hw = threadIdx.x >> 4, total = count * steps;
    for (int i0 = 0; i0 < total; i0 += 16) {
      const int i = i0 + hw, row = i / steps, st = i - row * steps, k = st * kW4Step + 8 * p;
      float f[8];
      unpack_piece(i < total && k < K ? *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(n0 + row) * K + k)
                                      : make_uint4(0u, 0u, 0u, 0u),
                   f);
      w4_stage_piece<GROUP>(f, p, st, i < total, xs + row * rb, xf + row * fs);
    }
    frag = xs;
    fx = xf;
    __syncthreads();
  } else {
    frag += n0 * rb;
    fx += static_cast<int64_t>(n0) * fs;
  }
  RowSums<NT> acc;
  clear<NT>(acc);
  if (r0 < N) {
    // rows past the last one read the last one and store nothing
    const W4Rows r = w4_rows<GROUP>(codes, scales, zeros, K, [&](int i) { return min(r0 + i, N - 1); });
    const W4Cols<NT> cols = w4_cols<GROUP, NT>(frag, fx, K, count, [](int i) { return i; });
    row_dot_w4<GROUP, NT>(r, cols, K, steps * wk / WK, steps * (wk + 1) / WK, acc);
  }
  if (WK > 1) join_slices<NT>(acc, joins, rg, wk, WK);
  if (wk != 0 || r0 >= N || failed != 0u) return;
  w4_unscale<NT>(acc);
#pragma unroll
  for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 16 * m + g + (i >> 1) * 8;
      if (r >= N) continue;
      const float b = bias ? __bfloat162float(bias[r]) : 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = 8 * n + 2 * t + (i & 1);
        if (c < count) y[static_cast<int64_t>(n0 + c) * N + r] = __float2bfloat16_rn(acc[m][n][i] + b);
      }
    }
}

struct W4Weight {
  const uint8_t* codes;
  const __nv_bfloat16* scales;
  const uint8_t* zeros;
};

template <int GROUP, int NT, bool LOCAL>
cudaError_t launch_linear(const void* x, const uint8_t* frag, const float2* fx, const W4Weight& w, const void* bias,
                          void* y, int rows, int K, int N, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int kRows = 16 * kRowTiles;
  const int x_blocks = (rows + 8 * NT - 1) / (8 * NT);
  const int WK = rowdot_split((static_cast<int64_t>(N) + kRows - 1) / kRows, x_blocks, w4_steps(K), 2, kRowWarps,
                              dev.num_sms);
  const int smem = joins_bytes<NT>(WK) + (LOCAL ? static_cast<int>(w4_staged_bytes<GROUP>(rows, K)) : 0);
  auto kern = w4_linear_kernel<GROUP, NT, LOCAL>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), 64 * 1024, dev.device);
  if (e != cudaSuccess) return e;
  const int a_cta = kRowWarps / WK * kRows;
  return launch_pdl(kern, dim3((N + a_cta - 1) / a_cta, x_blocks), dim3(kRowWarps * 32), smem, s,
                    static_cast<const __nv_bfloat16*>(x), frag, fx, w.codes, w.scales, w.zeros,
                    static_cast<const __nv_bfloat16*>(bias),
                    static_cast<__nv_bfloat16*>(y), rows, K, N, WK, static_cast<const uint32_t*>(dev.err));
}

template <int GROUP>
cudaError_t launch_linear_g(const void* x, const W4Weight& w, const void* bias, void* y, int rows, int K, int N,
                            void* scratch, const DeviceInfo& dev, cudaStream_t s) {
  if (w4_linear_local(rows, K, GROUP))
    return launch_linear<GROUP, 1, true>(x, nullptr, nullptr, w, bias, y, rows, K, N, dev, s);
  uint8_t* frag = static_cast<uint8_t*>(scratch);
  float2* fx = reinterpret_cast<float2*>(frag + rows * w4_row_bytes(K));
  const int64_t items = (static_cast<int64_t>(rows) * w4_steps(K) + 15) / 16;
  const int grid = static_cast<int>(items < 8 * dev.num_sms ? items : 8 * dev.num_sms);
  cudaError_t e = launch_pdl(w4_stage_kernel<GROUP>, dim3(grid), dim3(256), 0, s,
                             static_cast<const __nv_bfloat16*>(x), frag, fx, rows, K,
                             static_cast<const uint32_t*>(dev.err));
  if (e != cudaSuccess) return e;
  if (rows <= 8) return launch_linear<GROUP, 1, false>(x, frag, fx, w, bias, y, rows, K, N, dev, s);
  if (rows <= 16) return launch_linear<GROUP, 2, false>(x, frag, fx, w, bias, y, rows, K, N, dev, s);
  return launch_linear<GROUP, 4, false>(x, frag, fx, w, bias, y, rows, K, N, dev, s);
}

template <int GROUP>
cudaError_t launch_quant_g(const void* w, void* codes, void* scales, void* zeros, int64_t vecs, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((vecs + 255) / 256)), block(256);
  auto kern = zeros ? w4_quantize_kernel<GROUP, true> : w4_quantize_kernel<GROUP, false>;
  return launch_pdl(kern, grid, block, 0, s, static_cast<const uint4*>(w), static_cast<uint32_t*>(codes),
                    static_cast<__nv_bfloat16*>(scales), static_cast<uint8_t*>(zeros), vecs);
}

template <int GROUP>
cudaError_t launch_dequant_g(const void* codes, const void* scales, const void* zeros, void* w, int64_t vecs,
                             cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((vecs + 255) / 256)), block(256);
  auto kern = zeros ? w4_dequantize_kernel<GROUP, true> : w4_dequantize_kernel<GROUP, false>;
  return launch_pdl(kern, grid, block, 0, s, static_cast<const uint32_t*>(codes),
                    static_cast<const __nv_bfloat16*>(scales), static_cast<const uint8_t*>(zeros),
                    static_cast<uint4*>(w), vecs);
}

}  // namespace

cudaError_t launch_w4_quantize(const void* w, void* codes, void* scales, void* zeros, int64_t rows, int64_t K,
                               int group, cudaStream_t s) {
  const int64_t vecs = rows * (K / kVecCols);
  if (group == 32) return launch_quant_g<32>(w, codes, scales, zeros, vecs, s);
  if (group == 64) return launch_quant_g<64>(w, codes, scales, zeros, vecs, s);
  return launch_quant_g<128>(w, codes, scales, zeros, vecs, s);
}

cudaError_t launch_w4_dequantize(const void* codes, const void* scales, const void* zeros, void* w, int64_t rows,
                                 int64_t K, int group, cudaStream_t s) {
  const int64_t vecs = rows * (K / kVecCols);
  if (group == 32) return launch_dequant_g<32>(codes, scales, zeros, w, vecs, s);
  if (group == 64) return launch_dequant_g<64>(codes, scales, zeros, w, vecs, s);
  return launch_dequant_g<128>(codes, scales, zeros, w, vecs, s);
}

// Up to 8 rows whose staged form takes no more than 32 KB are staged by every CTA
// itself: reading 1 to 8 short rows costs less than another launch.
bool w4_linear_local(int64_t rows, int64_t K, int group) {
  const int k = static_cast<int>(K);
  return rows <= 8 && K <= 32768 &&
         (group == 32 ? w4_staged_bytes<32>(rows, k) : group == 64 ? w4_staged_bytes<64>(rows, k)
                                                                   : w4_staged_bytes<128>(rows, k)) <= 32 * 1024;
}

size_t w4_linear_scratch_bytes(int64_t rows, int64_t K) {
  // of the finest group; the group is not known to the query
  return static_cast<size_t>(w4_staged_bytes<32>(rows, static_cast<int>(K)));
}

cudaError_t launch_w4_linear(const void* x, const void* codes, const void* scales, const void* zeros,
                             const void* bias, void* y, int rows, int K, int N, int group, void* scratch,
                             const DeviceInfo& dev, cudaStream_t s) {
  const W4Weight w{static_cast<const uint8_t*>(codes), static_cast<const __nv_bfloat16*>(scales),
                   static_cast<const uint8_t*>(zeros)};
  if (group == 32) return launch_linear_g<32>(x, w, bias, y, rows, K, N, scratch, dev, s);
  if (group == 64) return launch_linear_g<64>(x, w, bias, y, rows, K, N, scratch, dev, s);
  return launch_linear_g<128>(x, w, bias, y, rows, K, N, scratch, dev, s);
}

}  // namespace dg
