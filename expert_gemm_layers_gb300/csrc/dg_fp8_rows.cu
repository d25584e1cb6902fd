// Row kernels of the block-scaled e4m3 format (include/dg.h): the quantiser and its
// inverse, and the root-mean-square norm (forward, in bf16 or in the format; backward).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dg_fp8.cuh"
#include "dg_internal.h"

namespace dg {

namespace {

// Maximum over the 16 lanes that hold a block.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

constexpr int kThreads = 256;

// A kernel here may begin while the one that makes its input still runs (it then waits), so no load may go through the
// path for data that stays as it is for the whole of a kernel: __ldca, __ldcg and __ldcs, no __ldg.
//
// Kernels that write a call's results look at the error word of its workspace: after a recorded failure they write
// nothing.  It is asked for with the first data and looked at before the first store.  Those that only fill scratch do
// not (read by every warp of 8192 x 14336 it cost 4 of 52 us).
__device__ __forceinline__ uint32_t error_word(const uint32_t* err) { return ld_volatile_u32(err); }

// ------------------------------------------------------------------ quantise, blocks of 1 x 128

// Half a warp takes a block of 128 columns, eight columns a lane, kQuantUnits blocks in flight.
constexpr int kQuantUnits = 4;
template <bool kWhole>  // whole: K is a multiple of 128, blocks lie one after another
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ q,
                                                              uint8_t* __restrict__ scale, int64_t blocks, int K, int nb) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 15;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kQuantUnits * kThreads + threadIdx.x) >> 4;
  uint4 v[kQuantUnits];
  int64_t at[kQuantUnits];
  bool in[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const int64_t b = first + i * (kThreads / 16);
    if (kWhole) {
      at[i] = b * 128 + 8 * sub;
      in[i] = b < blocks;
    } else {
      const int64_t row = b / nb;
      const int c = static_cast<int>(b - row * nb) * 128 + 8 * sub;
      at[i] = row * K + c;
      in[i] = b < blocks && c < K;
    }
    v[i] = in[i] ? __ldcs(reinterpret_cast<const uint4*>(x + at[i])) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const int64_t b = first + i * (kThreads / 16);
    const uint32_t byte = scale_byte(max16(amax_bits8(v[i])) << 16);
    float f[8];
    unpack8(v[i], f);
    if (in[i]) *reinterpret_cast<uint2*>(q + at[i]) = codes8(f, byte);
    if (sub == 0 && b < blocks) scale[b] = static_cast<uint8_t>(byte);
  }
}

// ------------------------------------------------------------------ quantise, blocks of 128 x 128

// One CTA takes kBlocks blocks side by side (256 bytes of each row apiece): 16 lanes across a block, 16 rows at a time,
// all eight reads before the maximum.
template <int kBlocks>
__global__ void __launch_bounds__(256 * kBlocks) quant_tiles_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ q,
                                                                    uint8_t* __restrict__ scale, int64_t rows, int K, int nb) {
  __shared__ uint32_t part[kBlocks][16];
  griddep_wait();
  griddep_launch_dependents();
  const int across = (nb + kBlocks - 1) / kBlocks;
  const int64_t rb = blockIdx.x / across;
  const int kb = kBlocks * static_cast<int>(blockIdx.x - rb * across);
  const int at = threadIdx.x % (16 * kBlocks), row = threadIdx.x / (16 * kBlocks), side = at >> 4;
  const int c = kb * 128 + 8 * at;
  const int64_t r0 = rb * 128 + row;
  uint4 v[8];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    v[i] = r < rows && c < K ? __ldcs(reinterpret_cast<const uint4*>(x + r * K + c)) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, amax_bits8(v[i]));
  m = max16(m);
  if ((threadIdx.x & 15) == 0) part[side][row] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = max(m, part[side][w]);
  const uint32_t byte = scale_byte(m << 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    float f[8];
    unpack8(v[i], f);
    if (r < rows && c < K) *reinterpret_cast<uint2*>(q + r * K + c) = codes8(f, byte);
  }
  if (row == 0 && (at & 15) == 0 && kb + side < nb) scale[rb * nb + kb + side] = static_cast<uint8_t>(byte);
}

// ------------------------------------------------------------------ transpose of codes

// out [K][rows] = in [rows][K], bytes, one 128 x 128 tile a CTA through shared memory (both sizes multiples of 16).  A
// thread turns 4 x 4 bytes; its warp takes 8 such blocks down and 4 across, which with rows of 33 words are 32 banks.
__global__ void __launch_bounds__(kThreads) transpose_codes_kernel(const uint8_t* __restrict__ in, uint8_t* __restrict__ out,
                                                                   int rows, int K) {
  __shared__ uint32_t tile[128][33];
  griddep_wait();
  griddep_launch_dependents();
  const int r0 = blockIdx.y * 128, c0 = blockIdx.x * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (threadIdx.x >> 3) + 32 * i, c = 16 * (threadIdx.x & 7);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < rows && c0 + c < K) v = __ldcg(reinterpret_cast<const uint4*>(in + static_cast<int64_t>(r0 + r) * K + c0 + c));
    uint32_t* t = &tile[r][c / 4];
    t[0] = v.x;
    t[1] = v.y;
    t[2] = v.z;
    t[3] = v.w;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the tile's 32 x 32 blocks as 4 x 8 groups of 8 x 4; a warp takes four of the 32
    const int group = warp * 4 + i, r4 = 8 * (group & 3) + (lane & 7), c4 = 4 * (group >> 2) + (lane >> 3);
    const uint32_t a = tile[4 * r4][c4], b = tile[4 * r4 + 1][c4], c = tile[4 * r4 + 2][c4], d = tile[4 * r4 + 3][c4];
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    const uint32_t o[4] = {__byte_perm(ab0, cd0, 0x5410), __byte_perm(ab0, cd0, 0x7632), __byte_perm(ab1, cd1, 0x5410),
                           __byte_perm(ab1, cd1, 0x7632)};
    if (r0 + 4 * r4 < rows)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c0 + 4 * c4 + k < K)
          *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(c0 + 4 * c4 + k) * rows + r0 + 4 * r4) = o[k];
  }
}

// ------------------------------------------------------------------ dequantise

// A warp takes 256 columns of a row at a time, eight a lane (whole lines in and out), kDeqUnits of them in flight.
constexpr int kDeqUnits = 4;
__global__ void __launch_bounds__(kThreads) dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                           __nv_bfloat16* __restrict__ x, int64_t rows, int K, int nb,
                                                           int row_shift, int spans) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t row = w / spans;
  if (row >= rows) return;
  const int c0 = static_cast<int>(w - row * spans) * (256 * kDeqUnits) + 8 * (threadIdx.x & 31);
  const uint8_t* srow = scale + (row >> row_shift) * nb;
  uint2 v[kDeqUnits];
  float s[kDeqUnits];
#pragma unroll
  for (int i = 0; i < kDeqUnits; ++i) {
    const int c = c0 + 256 * i;
    v[i] = make_uint2(0u, 0u);
    s[i] = 0.0f;
    if (c < K) {
      v[i] = __ldcs(reinterpret_cast<const uint2*>(q + row * K + c));
      s[i] = scale_value(__ldca(srow + (c >> 7)));
    }
  }
#pragma unroll
  for (int i = 0; i < kDeqUnits; ++i) {
    const int c = c0 + 256 * i;
    if (c >= K) break;
    const uint32_t u[2] = {v[i].x, v[i].y};
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(hr));
      o[h] = pack_bf16x2(f.x * s[i], f.y * s[i]);
    }
    *reinterpret_cast<uint4*>(x + row * K + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------ root-mean-square norm

// Sums over the threads of a row: a warp (kWarp) or the whole CTA; all of them get the sums, in one fixed order.
template <bool kWarp, int kSums>
__device__ __forceinline__ void row_sum(float (&v)[kSums], float (*part)[32]) {
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (kWarp) return;
  __syncthreads();  // the previous sums have been read
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < kSums; ++k) part[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += part[k][w];
    v[k] = s;
  }
}

// A row whose mean square and eps together overflow binary32 is summed as (h 2^-64)^2 instead, beside eps 2^-128.
constexpr float kShrink = 5.42101086242752217e-20f;  // 2^-64
__device__ __forceinline__ bool overflows(float mean) { return !(mean < __int_as_float(0x7f800000)); }
__device__ __forceinline__ float shrunk_mean(float sum, float n, float eps) { return sum / n + eps * kShrink * kShrink; }
constexpr int kWarpRows = 8;                          // rows of a CTA where a warp takes one

struct NormArgs {
  const __nv_bfloat16 *x, *res, *w;
  __nv_bfloat16 *h, *y;
  uint8_t *q, *scale;
  int64_t rows;
  int d, nb;
  float eps;
};

// A row a warp (kWarp) or CTA of T threads, C chunks of eight columns a thread, all read at once and kept in registers:
// chunk i of thread t is i * T + t, so that 16 lanes hold a block of 128 columns.  Bound by memory: 8192 x 4096 with a
// residual into 8 bits takes 38 us for 235 MB (6.2 TB/s).
template <bool kWarp, int C, bool kFp8, int kMaxT>
__global__ void __launch_bounds__(kMaxT) rms_norm_kernel(const NormArgs a) {
  __shared__ float part[1][32];
  const int T = kWarp ? 32 : blockDim.x;
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const bool live = row < a.rows;
  const int chunks = a.d / 8;
  griddep_wait();
  griddep_launch_dependents();
  uint4 xv[C], rv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    const bool in = live && c < chunks;
    xv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.x + row * a.d) + c) : make_uint4(0u, 0u, 0u, 0u);
    rv[i] = in && a.res ? __ldcs(reinterpret_cast<const uint4*>(a.res + row * a.d) + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float v[8];
    unpack8(xv[i], v);
    if (a.res) {
      float r[8];
      unpack8(rv[i], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
      xv[i] = pack8(v);  // the sum is a bf16 tensor, and its norm that of what is stored
      if (live && t + i * T < chunks) reinterpret_cast<uint4*>(a.h + row * a.d)[t + i * T] = xv[i];
      unpack8(xv[i], v);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[0] = fmaf(v[e], v[e], sum[0]);
  }
  row_sum<kWarp, 1>(sum, part);
  const float n = static_cast<float>(a.d);
  const float mean = sum[0] / n + a.eps;
  float rstd = 1.0f / sqrtf(mean);
  float pre = 1.0f;
  if (overflows(mean)) {  // the same for all threads of the row
    sum[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
      unpack8(xv[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] = fmaf(v[e] * kShrink, v[e] * kShrink, sum[0]);
    }
    row_sum<kWarp, 1>(sum, part);
    rstd = 1.0f / sqrtf(shrunk_mean(sum[0], n, a.eps));
    pre = kShrink;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    const bool in = live && c < chunks;
    const uint4 wv = c < chunks ? __ldca(reinterpret_cast<const uint4*>(a.w) + c) : make_uint4(0u, 0u, 0u, 0u);
    float v[8], g[8];
    unpack8(xv[i], v);
    unpack8(wv, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * pre * rstd * g[e];
    if (kFp8) {
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
      const uint32_t byte = scale_byte(max16(in ? m : 0u));
      if (in) {
        *reinterpret_cast<uint2*>(a.q + row * a.d + 8 * static_cast<int64_t>(c)) = codes8(v, byte);
        if ((c & 15) == 0) a.scale[row * a.nb + (c >> 4)] = static_cast<uint8_t>(byte);
      }
    } else if (in) {
      reinterpret_cast<uint4*>(a.y + row * a.d)[c] = pack8(v);
    }
  }
}

struct NormBwdArgs {
  const __nv_bfloat16 *h, *w, *dy, *dh;
  __nv_bfloat16* dx;
  float* part;  // [gridDim.x][d], or NULL
  int64_t rows;
  int d;
  float eps;
  const uint32_t* err;
};

// Threads and chunks as in rms_norm_kernel; a CTA takes every gridDim.x-th row (or kWarpRows rows), the next one read
// while this one is worked on.  The weight's gradient stays in registers over a thread's rows and leaves as one partial
// sum a CTA.
template <bool kWarp, int C, int kMaxT>
__global__ void __launch_bounds__(kMaxT, kWarp ? 2 : C == 1 ? 3 : 1) rms_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float part[2][32];
  __shared__ float2 wsum[kWarp ? kWarpRows - 1 : 1][kWarp ? 32 * C * 4 : 1];
  const int T = kWarp ? 32 : blockDim.x;
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int sub = kWarp ? threadIdx.x >> 5 : 0;
  constexpr int kRows = kWarp ? kWarpRows : 1;
  const int chunks = a.d / 8;
  const float n = static_cast<float>(a.d);
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t failed = error_word(a.err);
  uint4 wv[C], hv[C], yv[C], pv[C];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = t + i * T;
      const bool in = row < a.rows && c < chunks;
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      hv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.h + row * a.d) + c) : z;
      yv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.dy + row * a.d) + c) : z;
      pv[i] = in && a.dh ? __ldcs(reinterpret_cast<const uint4*>(a.dh + row * a.d) + c) : z;
    }
  };
#pragma unroll
  for (int i = 0; i < C; ++i)
    wv[i] = t + i * T < chunks ? __ldca(reinterpret_cast<const uint4*>(a.w) + t + i * T) : make_uint4(0u, 0u, 0u, 0u);
  float2 dw[C][4];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[i][e] = make_float2(0.0f, 0.0f);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  fetch(static_cast<int64_t>(blockIdx.x) * kRows + sub);
  if (failed) return;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + sub;
    uint4 hc[C], yc[C], pc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      hc[i] = hv[i];
      yc[i] = yv[i];
      pc[i] = pv[i];
    }
    if (r0 + step < a.rows) fetch(row + step);
    // sum h^2 and sum (dy w) h, or with k = 2^-64 those of h k
    auto sums = [&](float k, float (&s)[2]) {
      float2 q = make_float2(0.0f, 0.0f), r = q;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float2 h[4], y[4], g[4];
        unpack4x2(hc[i], h);
        unpack4x2(yc[i], y);
        unpack4x2(wv[i], g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = mul2(h[e], splat2(k));
          q = fma2(u, u, q);
          r = fma2(mul2(y[e], g[e]), u, r);
        }
      }
      s[0] = q.x + q.y;
      s[1] = r.x + r.y;
      row_sum<kWarp, 2>(s, part);
    };
    float s[2];
    sums(1.0f, s);
    const float square = s[0] / n + a.eps;
    float pre = 1.0f, rstd = 1.0f / sqrtf(square);
    if (overflows(square)) {
      pre = kShrink;
      sums(pre, s);
      rstd = 1.0f / sqrtf(shrunk_mean(s[0], n, a.eps));
    }
    // with n_h = h pre rstd (the normalised row): dx = rstd pre (dy w - n_h mean(dy w n_h)) + dh
    const float2 mean = splat2(-s[1] * rstd / n), out = splat2(rstd * pre);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float2 h[4], y[4], g[4], p[4];
      unpack4x2(hc[i], h);
      unpack4x2(yc[i], y);
      unpack4x2(wv[i], g);
      unpack4x2(pc[i], p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 nh = mul2(h[e], out);
        dw[i][e] = fma2(y[e], nh, dw[i][e]);
        p[e] = fma2(out, fma2(nh, mean, mul2(y[e], g[e])), p[e]);
      }
      if (a.dx && row < a.rows && t + i * T < chunks)
        reinterpret_cast<uint4*>(a.dx + row * a.d)[t + i * T] =
            make_uint4(pack_bf16x2(p[0].x, p[0].y), pack_bf16x2(p[1].x, p[1].y), pack_bf16x2(p[2].x, p[2].y),
                       pack_bf16x2(p[3].x, p[3].y));
    }
  }
  if (!a.part) return;
  if (kWarp) {
    if (sub > 0)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) wsum[sub - 1][(i * 4 + e) * 32 + t] = dw[i][e];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = add2(dw[i][e], wsum[k][(i * 4 + e) * 32 + t]);
  }
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.d;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    if (c >= chunks) continue;
    float4* o = reinterpret_cast<float4*>(out + 8 * c);
    o[0] = make_float4(dw[i][0].x, dw[i][0].y, dw[i][1].x, dw[i][1].y);
    o[1] = make_float4(dw[i][2].x, dw[i][2].y, dw[i][3].x, dw[i][3].y);
  }
}

// The backward in two passes, for rows too long for a CTA's registers.  First, a CTA a row: k = 1 / sqrt(mean h^2 + eps)
// and mean(dy w h) k.
__global__ void __launch_bounds__(256) norm_bwd_rows_kernel(const NormBwdArgs a, float2* __restrict__ coef) {
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const int chunks = a.d / 8;
  const float n = static_cast<float>(a.d);
  griddep_wait();
  griddep_launch_dependents();
  float pre = 1.0f, rstd = 0.0f, s[2];
  for (int pass = 0; pass < 2; ++pass) {
    s[0] = s[1] = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x; c < chunks; c += 256) {
      float h[8], y[8], g[8];
      unpack8(__ldcg(reinterpret_cast<const uint4*>(a.h + row * a.d) + c), h);
      unpack8(__ldcg(reinterpret_cast<const uint4*>(a.dy + row * a.d) + c), y);
      unpack8(__ldca(reinterpret_cast<const uint4*>(a.w) + c), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = h[e] * pre;
        s[0] = fmaf(u, u, s[0]);
        s[1] = fmaf(y[e] * g[e], u, s[1]);
      }
    }
    row_sum<false, 2>(s, part);
    const float square = pre == 1.0f ? s[0] / n + a.eps : shrunk_mean(s[0], n, a.eps);
    rstd = 1.0f / sqrtf(square);
    if (pre != 1.0f || !overflows(square)) break;
    pre = kShrink;
  }
  if (threadIdx.x == 0 && !error_word(a.err)) coef[row] = make_float2(rstd * pre, s[1] * rstd / n);
}

// Then, for 2048 columns a CTA over every gridDim.y-th row: dx, and the weight's gradient in registers.
__global__ void __launch_bounds__(256) norm_bwd_apply_kernel(const NormBwdArgs a, const float2* __restrict__ coef) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (c >= a.d || error_word(a.err)) return;
  float g[8], dw[8] = {};
  unpack8(__ldca(reinterpret_cast<const uint4*>(a.w + c)), g);
  constexpr int kUnits = 4;  // rows in flight
  const int64_t step = gridDim.y;
  for (int64_t r0 = blockIdx.y; r0 < a.rows; r0 += kUnits * step) {
    uint4 hv[kUnits], yv[kUnits], pv[kUnits];
    float2 k[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int64_t r = r0 + i * step;
      const bool in = r < a.rows;
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      hv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.h + r * a.d + c)) : z;
      yv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.dy + r * a.d + c)) : z;
      pv[i] = in && a.dh ? __ldcs(reinterpret_cast<const uint4*>(a.dh + r * a.d + c)) : z;
      k[i] = in ? __ldca(coef + r) : make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int64_t r = r0 + i * step;
      float h[8], y[8], p[8];
      unpack8(hv[i], h);
      unpack8(yv[i], y);
      unpack8(pv[i], p);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nh = h[e] * k[i].x;
        dw[e] = fmaf(y[e], nh, dw[e]);
        p[e] = fmaf(k[i].x, fmaf(-nh, k[i].y, y[e] * g[e]), p[e]);
      }
      if (a.dx && r < a.rows) *reinterpret_cast<uint4*>(a.dx + r * a.d + c) = pack8(p);
    }
  }
  if (!a.part) return;
  float4* o = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.y) * a.d + c);
  o[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
  o[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
}

// out[c] = sum over `parts` partial sums part[k][c], in an order that the sizes fix: 32 columns a CTA, the partial sums
// spread over its 32 warps, four loads in flight each.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* __restrict__ part, __nv_bfloat16* __restrict__ out,
                                                         int parts, int d, const uint32_t* err) {
  __shared__ float s[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t failed = error_word(err);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < d) {
    const float* p = part + c;
    int k = warp;
    for (; k + 96 < parts; k += 128) {
      float u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __ldcs(p + static_cast<int64_t>(k + 32 * i) * d);
      v += (u[0] + u[1]) + (u[2] + u[3]);
    }
    for (; k < parts; k += 32) v += __ldcs(p + static_cast<int64_t>(k) * d);
  }
  s[warp][lane] = v;
  __syncthreads();
  float r = s[lane][warp];  // warp w adds up column w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < d && !failed) out[col] = __float2bfloat16_rn(r);
}

// ------------------------------------------------------------------ quantise a gradient and sum its columns

// Blocks of 1 x 128 as quant_rows_kernel, one CTA taking a column block and every gridDim.y-th group of 16 rows, so that
// the column sums of what it reads stay in registers: part[blockIdx.y][column].  Without kCodes the sums alone, added up
// in the same order.
template <bool kCodes>
__global__ void __launch_bounds__(kThreads) quant_rows_sum_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ q,
                                                                  uint8_t* __restrict__ scale, float* __restrict__ part,
                                                                  int64_t rows, int K, int nb) {
  __shared__ float s[kThreads / 16][128 + 4];
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int c = blockIdx.x * 128 + 8 * sub;
  float sum[8] = {};
  const int64_t step = 16 * static_cast<int64_t>(gridDim.y);
  // kUnits rows a thread in flight; whole groups of 16 rows, so that the lanes of a block stay together
  constexpr int kUnits = 4;
  for (int64_t r0 = 16 * static_cast<int64_t>(blockIdx.y); r0 < rows; r0 += kUnits * step) {
    uint4 v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int64_t r = r0 + i * step + group;
      v[i] = r < rows && c < K ? __ldcs(reinterpret_cast<const uint4*>(x + r * K + c)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int64_t r = r0 + i * step + group;
      float f[8];
      unpack8(v[i], f);
      if (kCodes) {
        const uint32_t byte = scale_byte(max16(amax_bits8(v[i])) << 16);
        if (r < rows && c < K) *reinterpret_cast<uint2*>(q + r * K + c) = codes8(f, byte);
        if (r < rows && sub == 0) scale[r * nb + blockIdx.x] = static_cast<uint8_t>(byte);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s[group][8 * sub + e] = sum[e];
  __syncthreads();
  const int col = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && col < K) {
    float r = 0.0f;
#pragma unroll
    for (int g = 0; g < kThreads / 16; ++g) r += s[g][threadIdx.x];
    part[static_cast<int64_t>(blockIdx.y) * K + col] = r;
  }
}

// Threads of a CTA that takes one row in C chunks a thread, and the instance for a row length: one warp up to 512
// columns, then as few threads as hold the row.
int row_threads(int d, int C) { return ((d / 8 + C - 1) / C + 31) / 32 * 32; }

template <bool kFp8>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t s) {
  const dim3 warp_grid(static_cast<unsigned>((a.rows + kWarpRows - 1) / kWarpRows)), grid(static_cast<unsigned>(a.rows));
  if (a.d <= 256) return launch_pdl(rms_norm_kernel<true, 1, kFp8, 256>, warp_grid, dim3(32 * kWarpRows), 0, s, a);
  if (a.d <= 512) return launch_pdl(rms_norm_kernel<true, 2, kFp8, 256>, warp_grid, dim3(32 * kWarpRows), 0, s, a);
  if (a.d <= 2048) return launch_pdl(rms_norm_kernel<false, 1, kFp8, 256>, grid, dim3(row_threads(a.d, 1)), 0, s, a);
  if (a.d <= 8192) return launch_pdl(rms_norm_kernel<false, 2, kFp8, 512>, grid, dim3(row_threads(a.d, 2)), 0, s, a);
  return launch_pdl(rms_norm_kernel<false, 4, kFp8, 1024>, grid, dim3(row_threads(a.d, 4)), 0, s, a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, void* codes, void* scales, int64_t rows, int K, int block_rows,
                                cudaStream_t s) {
  const int nb = (K + 127) / 128;
  auto* xp = static_cast<const __nv_bfloat16*>(x);
  auto* q = static_cast<uint8_t*>(codes);
  auto* sc = static_cast<uint8_t*>(scales);
  if (block_rows == 1) {
    const int64_t blocks = rows * nb, per = kThreads / 16 * kQuantUnits;
    const dim3 grid(static_cast<unsigned>((blocks + per - 1) / per));
    return K % 128 == 0 ? launch_pdl(quant_rows_kernel<true>, grid, dim3(kThreads), 0, s, xp, q, sc, blocks, K, nb)
                        : launch_pdl(quant_rows_kernel<false>, grid, dim3(kThreads), 0, s, xp, q, sc, blocks, K, nb);
  }
  // Two blocks a CTA where there are many (28672 x 4096, with 7168: 58 us against 62), one where not (1003 x 2064: 2.5
  // us against 3.4; 8192 x 4096, 2048: 16.8 against 18.5).
  const int64_t row_blocks = (rows + 127) / 128;
  if (row_blocks * nb >= 4096)
    return launch_pdl(quant_tiles_kernel<2>, dim3(static_cast<unsigned>(row_blocks * ((nb + 1) / 2))), dim3(512), 0, s, xp, q,
                      sc, rows, K, nb);
  return launch_pdl(quant_tiles_kernel<1>, dim3(static_cast<unsigned>(row_blocks * nb)), dim3(256), 0, s, xp, q, sc, rows, K,
                    nb);
}

cudaError_t launch_fp8_dequantize(const void* codes, const void* scales, void* x, int64_t rows, int K, int block_rows,
                                  cudaStream_t s) {
  const int nb = (K + 127) / 128, spans = (K + 256 * kDeqUnits - 1) / (256 * kDeqUnits);
  const int64_t warps = rows * spans;
  return launch_pdl(dequant_kernel, dim3(static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                    static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), static_cast<__nv_bfloat16*>(x),
                    rows, K, nb, block_rows == 1 ? 0 : 7, spans);
}

cudaError_t launch_transpose_codes(const void* in, void* out, int rows, int K, cudaStream_t s) {
  return launch_pdl(transpose_codes_kernel, dim3((K + 127) / 128, (rows + 127) / 128), dim3(kThreads), 0, s,
                    static_cast<const uint8_t*>(in), static_cast<uint8_t*>(out), rows, K);
}

cudaError_t launch_rms_norm(const void* x, const void* res, const void* w, void* h, void* y, void* codes, void* scales,
                            int64_t rows, int d, float eps, cudaStream_t s) {
  const NormArgs a{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(res),
                   static_cast<const __nv_bfloat16*>(w), static_cast<__nv_bfloat16*>(h), static_cast<__nv_bfloat16*>(y),
                   static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, d, (d + 127) / 128, eps};
  return codes ? norm_launch<true>(a, s) : norm_launch<false>(a, s);
}

namespace {

// SMs that a grid of partial sums is made for.  Written out, so that the order of the sums and the scratch follow from the
// sizes alone.
constexpr int kSms = 152;

// One pass up to 8192 columns; beyond, two (2048 x 16384: 280 us in one with spilled registers, 65 us in two).
bool norm_bwd_one_pass(int d) { return d <= 8192; }

}  // namespace

int rms_norm_bwd_parts(int64_t rows, int d) {
  if (!norm_bwd_one_pass(d)) {
    const int64_t across = (d + 2047) / 2048, want = (kSms * 4 + across - 1) / across;
    return static_cast<int>(rows < want ? rows : want);
  }
  // as many CTAs as run at once: 24 warps of 80 registers a thread with one chunk, 16 of 128 with two
  // (8192 x 1280: 26 us with a part of the CTAs left for a second turn, 16 us)
  const bool warp = d <= 512;
  const int64_t groups = warp ? (rows + kWarpRows - 1) / kWarpRows : rows;
  const int64_t most = kSms * (warp ? 2 : d <= 2048 ? 768 / row_threads(d, 1) : 512 / row_threads(d, 2));
  return static_cast<int>(groups < most ? groups : most);
}

size_t rms_norm_bwd_scratch_bytes(int64_t rows, int d) {
  const size_t coef = norm_bwd_one_pass(d) ? 0 : (static_cast<size_t>(rows) * sizeof(float2) + 255) / 256 * 256;
  return coef + static_cast<size_t>(rms_norm_bwd_parts(rows, d)) * d * sizeof(float);
}

cudaError_t launch_rms_norm_bwd(const void* h, const void* w, const void* dy, const void* dh, void* dx, void* d_weight,
                                void* scratch, int64_t rows, int d, float eps, const uint32_t* err, cudaStream_t s) {
  const int parts = rms_norm_bwd_parts(rows, d);
  const size_t coef_bytes = rms_norm_bwd_scratch_bytes(rows, d) - static_cast<size_t>(parts) * d * sizeof(float);
  float2* coef = static_cast<float2*>(scratch);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + coef_bytes);
  const NormBwdArgs a{static_cast<const __nv_bfloat16*>(h),  static_cast<const __nv_bfloat16*>(w),
                      static_cast<const __nv_bfloat16*>(dy), static_cast<const __nv_bfloat16*>(dh),
                      static_cast<__nv_bfloat16*>(dx),       d_weight ? part : nullptr, rows, d, eps, err};
  cudaError_t e;
  if (!norm_bwd_one_pass(d)) {
    e = launch_pdl(norm_bwd_rows_kernel, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, a, coef);
    if (e != cudaSuccess) return e;
    e = launch_pdl(norm_bwd_apply_kernel, dim3((d + 2047) / 2048, parts), dim3(256), 0, s, a, static_cast<const float2*>(coef));
  } else if (d <= 256)
    e = launch_pdl(rms_norm_bwd_kernel<true, 1, 256>, dim3(parts), dim3(32 * kWarpRows), 0, s, a);
  else if (d <= 512)
    e = launch_pdl(rms_norm_bwd_kernel<true, 2, 256>, dim3(parts), dim3(32 * kWarpRows), 0, s, a);
  else if (d <= 2048)
    e = launch_pdl(rms_norm_bwd_kernel<false, 1, 256>, dim3(parts), dim3(row_threads(d, 1)), 0, s, a);
  else
    e = launch_pdl(rms_norm_bwd_kernel<false, 2, 512>, dim3(parts), dim3(row_threads(d, 2)), 0, s, a);
  if (e != cudaSuccess || !d_weight) return e;
  return launch_pdl(sum_parts_kernel, dim3((d + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(part),
                    static_cast<__nv_bfloat16*>(d_weight), parts, d, err);
}

int fp8_quantize_sum_parts(int64_t rows, int K) {
  const int64_t nb = (K + 127) / 128, groups = (rows + 15) / 16;
  const int64_t want = (kSms * 8 + nb - 1) / nb;  // CTAs that run at once
  return static_cast<int>(groups < want ? groups : want);
}

cudaError_t launch_fp8_quantize_sum(const void* x, void* codes, void* scales, void* sums, float* part, int64_t rows,
                                    int K, const uint32_t* err, cudaStream_t s) {
  const int nb = (K + 127) / 128, parts = fp8_quantize_sum_parts(rows, K);
  const auto kern = codes ? quant_rows_sum_kernel<true> : quant_rows_sum_kernel<false>;
  cudaError_t e = launch_pdl(kern, dim3(nb, parts), dim3(kThreads), 0, s, static_cast<const __nv_bfloat16*>(x),
                             static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), part, rows, K, nb);
  if (e != cudaSuccess) return e;
  return launch_pdl(sum_parts_kernel, dim3((K + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(part),
                    static_cast<__nv_bfloat16*>(sums), parts, K, err);
}

}  // namespace dg
