// 4-bit weights with one scale (and optionally one zero point) per group of
// 32, 64 or 128 consecutive columns of a row: quantising, reading back, and
// the product with a few activation rows.
//
//   value[o, k] = (q[o, k] - z[o, g]) * s[o, g],  g = k / group
//
// Codes are two to a byte along k, the even column in the low nibble.
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "dg_rowdot.cuh"

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

// The one unit of a w4_linear CTA: up to 8*NT activation rows, 8 / WK blocks of
// 32 weight rows.
template <int NT>
struct LinearWork {
  Rows w;
  const __nv_bfloat16* x;
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;
  int nx, K, N;  // activation rows, columns, weight rows
  int r0, n0;    // the CTA's first weight row and activation row

  __device__ int units() const { return 1; }
  __device__ Rows rows(int) const { return w; }
  __device__ int row(int, int rg, int lane, bool& active) const {
    const int r = r0 + rg * 16 * kRowTiles;
    active = r < N;
    return min(r + lane, N - 1);
  }
  __device__ int count(int) const { return min(nx - n0, 8 * NT); }
  __device__ const __nv_bfloat16* xrow(int, int i) const { return x + static_cast<int64_t>(n0 + i) * K; }
  __device__ void finish(int, int rg, const float (&acc)[kRowTiles][NT][4]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 16 * (kRowTiles * rg + m) + g + (i >> 1) * 8;
        if (r >= N) continue;
        const float b = bias ? __bfloat162float(bias[r]) : 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = n0 + 8 * n + 2 * t + (i & 1);
          if (row < nx) y[static_cast<int64_t>(row) * N + r] = __float2bfloat16_rn(acc[m][n][i] + b);
        }
      }
  }
};

template <int GROUP, int NT>
__global__ void __launch_bounds__(kRowWarps * 32, 2)
    w4_linear_kernel(const __nv_bfloat16* __restrict__ x, const uint8_t* __restrict__ codes,
                     const __nv_bfloat16* __restrict__ scales, const uint8_t* __restrict__ zeros,
                     const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ y, int rows, int K, int N,
                     int WK, const uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  const LinearWork<NT> work{Rows{codes, scales, zeros},
                            x,
                            bias,
                            y,
                            rows,
                            K,
                            N,
                            static_cast<int>(blockIdx.x) * (kRowWarps / WK) * 16 * kRowTiles,
                            static_cast<int>(blockIdx.y) * 8 * NT};
  row_stream<GROUP, NT>(work, K, WK, smem);
}

template <int GROUP, int NT>
cudaError_t launch_linear(const void* x, const void* codes, const void* scales, const void* zeros, const void* bias,
                          void* y, int rows, int K, int N, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int kRows = 16 * kRowTiles;
  constexpr int kMostWK = NT == 4 ? 2 : NT == 2 ? 4 : kRowWarps;  // the slices' staged rows have to fit
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(w4_linear_kernel<GROUP, NT>),
                                  rowdot_smem<GROUP, NT>(kMostWK), dev.device);
  if (e != cudaSuccess) return e;
  const int row_blocks = (rows + 8 * NT - 1) / (8 * NT);
  const int steps = (K + rowdot_step<GROUP>() - 1) / rowdot_step<GROUP>();
  const int WK = rowdot_split((static_cast<int64_t>(N) + kRows - 1) / kRows, row_blocks, steps, kMostWK,
                              2 * static_cast<int64_t>(dev.num_sms));
  const int rg = kRowWarps / WK;
  const dim3 grid((N + kRows * rg - 1) / (kRows * rg), row_blocks);
  return launch_pdl(w4_linear_kernel<GROUP, NT>, grid, dim3(kRowWarps * 32), rowdot_smem<GROUP, NT>(WK), s,
                    static_cast<const __nv_bfloat16*>(x), static_cast<const uint8_t*>(codes),
                    static_cast<const __nv_bfloat16*>(scales), static_cast<const uint8_t*>(zeros),
                    static_cast<const __nv_bfloat16*>(bias), static_cast<__nv_bfloat16*>(y), rows, K, N, WK,
                    static_cast<const uint32_t*>(dev.err));
}

template <int GROUP>
cudaError_t launch_linear_g(const void* x, const void* codes, const void* scales, const void* zeros, const void* bias,
                            void* y, int rows, int K, int N, const DeviceInfo& dev, cudaStream_t s) {
  if (rows <= 8) return launch_linear<GROUP, 1>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
  if (rows <= 16) return launch_linear<GROUP, 2>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
  return launch_linear<GROUP, 4>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
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

cudaError_t launch_w4_linear(const void* x, const void* codes, const void* scales, const void* zeros,
                             const void* bias, void* y, int rows, int K, int N, int group, const DeviceInfo& dev,
                             cudaStream_t s) {
  if (group == 32) return launch_linear_g<32>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
  if (group == 64) return launch_linear_g<64>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
  return launch_linear_g<128>(x, codes, scales, zeros, bias, y, rows, K, N, dev, s);
}

}  // namespace dg
