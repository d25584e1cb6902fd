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

constexpr int kVecCols = 8;  // columns of a piece: 16 bytes of bf16, 4 bytes of codes
constexpr int kQuantPieces = 4;  // pieces a thread has in flight
constexpr int kDequantPieces = 8;

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The codes of a piece: clamp(rne(w / s) + z, 0, 15), the quotient that of binary32
// division, without dividing.  w and s have 8 significant bits, so w / s either is
// n + 1/2 exactly or lies at least 2^-11 from it (|w / s| <= 16).  w * (1 / s) is
// within 2^-18 of w / s.  Adding 768 rounds it to a multiple of 2^-14, which
// restores the exact halves and moves nothing across one; adding 2^23 + 2^22 - 768
// rounds that to an integer, halves to even, in the low bits.
__device__ __forceinline__ uint32_t codes_of(const uint4& v, float inv, float z) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t inv2 = f32x2(inv, inv), snap = f32x2(768.0f, 768.0f);
  const float whole = 12582912.0f - 768.0f;
  const uint64_t whole2 = f32x2(whole, whole);
  const int zi = static_cast<int>(z);
  uint32_t code = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(w[i]);
    const uint64_t n = add2(add2(mul2(f32x2(p.x, p.y), inv2), snap), whole2);
    const int lo = static_cast<int>(static_cast<uint32_t>(n)) - 0x4b400000 + zi;
    const int hi = static_cast<int>(static_cast<uint32_t>(n >> 32)) - 0x4b400000 + zi;
    code |= static_cast<uint32_t>(min(max(lo, 0), 15)) << (8 * i);
    code |= static_cast<uint32_t>(min(max(hi, 0), 15)) << (8 * i + 4);
  }
  return code;
}

// A thread takes pieces of 8 columns; the GROUP / 8 lanes of a group agree on its
// scale by shuffles.  A group with a NaN or an infinity, or whose range overflows
// binary32, gets a NaN scale.
// Reading 2 bytes a weight and writing half a byte should bound it; 28672 x 4096,
// groups of 128: 55 us, 5.4 TB/s, 0.79 of the measured copy rate.  What keeps it from
// that is arithmetic (76% of the issue slots of the busiest pipe): a division a weight
// and one piece at a time took 178 us, codes_of and four pieces 60, scales by four
// lanes 55.  With zero points 76 us, 3.9 TB/s: the smallest and the largest of a group are
// two reductions more, 32-bit ones where a magnitude's is two 16-bit values at a time.
template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(256)
    w4_quantize_kernel(const uint4* __restrict__ w, uint32_t* __restrict__ codes, __nv_bfloat16* __restrict__ scales,
                       uint8_t* __restrict__ zeros, int64_t pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kQuantPieces) + threadIdx.x;
  uint4 raw[kQuantPieces];
  // pieces is a multiple of the GROUP / 8 lanes of a group, so groups are whole;
  // lanes past the end only keep the shuffles convergent
#pragma unroll
  for (int k = 0; k < kQuantPieces; ++k)
    raw[k] = first + 256 * k < pieces ? __ldg(w + first + 256 * k) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t top = 0u;  // largest magnitude, as bf16 bits: NaN > inf > finite
  float lo = 0.0f, hi = 0.0f;
  // The groups of the pieces 0..3 have their scales made by the lanes 0..3 of every
  // four: a division and a reciprocal a thread, not four.
  static_assert(kQuantPieces == 4, "lanes of a group");
  const int mine = threadIdx.x & 3;
#pragma unroll
  for (int k = 0; k < kQuantPieces; ++k) {
    const uint32_t word[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __vmaxu2(t, word[i] & 0x7fff7fffu);
    t = max(t & 0xffffu, t >> 16);
#pragma unroll
    for (int o = GROUP / kVecCols / 2; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
    if (mine == k) top = t;
    if constexpr (ZEROS) {
      float l = 0.0f, h = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack_bf16x2(word[i]);
        l = fminf(l, fminf(p.x, p.y));
        h = fmaxf(h, fmaxf(p.x, p.y));
      }
#pragma unroll
      for (int o = GROUP / kVecCols / 2; o > 0; o >>= 1) {
        l = fminf(l, __shfl_xor_sync(0xffffffffu, l, o));
        h = fmaxf(h, __shfl_xor_sync(0xffffffffu, h, o));
      }
      if (mine == k) {
        lo = l;
        hi = h;
      }
    }
  }
  const float quot = ZEROS ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(__uint_as_float(top << 16), 7.0f);
  float scale = __bfloat162float(__float2bfloat16_rn(quot)), zero = 8.0f;
  if (scale == 0.0f) scale = 1.0f;
  if (top < 0x7f80u && isfinite(quot)) {
    if constexpr (ZEROS) zero = fminf(fmaxf(rintf(__fdiv_rn(-lo, scale)), 0.0f), 15.0f);
  } else {
    scale = __int_as_float(0x7fc00000);
  }
  const float inverse = __frcp_rn(scale);
#pragma unroll
  for (int k = 0; k < kQuantPieces; ++k) {
    const int64_t v = first + 256 * k;
    const int from = (threadIdx.x & 28) | k;
    const float s = __shfl_sync(0xffffffffu, scale, from), inv = __shfl_sync(0xffffffffu, inverse, from);
    const float z = ZEROS ? __shfl_sync(0xffffffffu, zero, from) : 8.0f;
    if (v >= pieces) continue;
    uint32_t code = 0x88888888u;
    if (s >= 7.9e-31f) {  // 2^-100: 1 / s is a normal number
      code = codes_of(raw[k], inv, z);
    } else if (!isnan(s)) {
      const uint32_t word[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      code = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = unpack_bf16x2(word[i / 2]);
        const float q = fminf(fmaxf(rintf(__fdiv_rn(i & 1 ? p.y : p.x, s)) + z, 0.0f), 15.0f);
        code |= static_cast<uint32_t>(q) << (4 * i);
      }
    }
    codes[v] = code;
    if (v % (GROUP / kVecCols) == 0) {
      const int64_t g = v / (GROUP / kVecCols);
      scales[g] = __float2bfloat16_rn(s);
      if (ZEROS) zeros[g] = static_cast<uint8_t>(z);
    }
  }
}

// A piece a thread at a time: 4 bytes of codes in, 16 bytes of bf16 out, each value
// rounded once from the exact binary32 product.  Bound by its writes: 28672 x 4096,
// groups of 128: 43 to 46 us, 6.9 to 6.4 TB/s.  (16 columns a thread, written as two pieces of a
// 32-byte stride, took 55 us: every line was written twice by halves.)
template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(256)
    w4_dequantize_kernel(const uint32_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                         const uint8_t* __restrict__ zeros, uint4* __restrict__ w, int64_t pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kDequantPieces) + threadIdx.x;
  uint32_t raw[kDequantPieces];
  float s[kDequantPieces], z[kDequantPieces];
#pragma unroll
  for (int k = 0; k < kDequantPieces; ++k) {
    const int64_t v = first + 256 * k;
    if (v >= pieces) continue;
    const int64_t g = v / (GROUP / kVecCols);
    raw[k] = __ldg(codes + v);
    s[k] = __bfloat162float(scales[g]);
    z[k] = ZEROS ? static_cast<float>(zeros[g] & 15) : 8.0f;
  }
#pragma unroll
  for (int k = 0; k < kDequantPieces; ++k) {
    const int64_t v = first + 256 * k;
    if (v >= pieces) continue;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // an integer in a binary32 significand, less 2^23 and the zero point: exact
      const float a = __uint_as_float(0x4b000000u | ((raw[k] >> (8 * i)) & 15u)) - (8388608.0f + z[k]);
      const float b = __uint_as_float(0x4b000000u | ((raw[k] >> (8 * i + 4)) & 15u)) - (8388608.0f + z[k]);
      out[i] = pack_bf16x2(a * s[k], b * s[k]);
    }
    w[v] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// Activation rows staged once for all CTAs of the product: a CTA a row, or (STEPS: up
// to 8 rows) 16 steps a CTA, each with a scale of its own.
template <int GROUP, bool STEPS>
__global__ void __launch_bounds__(256)
    w4_stage_kernel(const __nv_bfloat16* __restrict__ x, Staged out, int rows, int K, const uint32_t* err) {
  __shared__ uint32_t top;
  if (!STEPS && threadIdx.x == 0) top = 0u;
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  if constexpr (STEPS) {
    w4_stage_steps<GROUP>(out, rows, K, blockIdx.x, gridDim.x, [&](int i) {
      return reinterpret_cast<const uint8_t*>(x + static_cast<int64_t>(i) * K);
    });
  } else {
    __syncthreads();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
      w4_stage_row<GROUP>(reinterpret_cast<const uint8_t*>(x + r * K), K, out.frag + r * w4_row_bytes(K),
                          out.sums + r * w4_row_sums(K, GROUP), out.factor + r, &top);
  }
}

// Bound by the latency of a warp's instructions more than by bytes: a step is some 250
// of them on 32 rows, and what these shapes allow is 16 to 24 warps an SM.  GPU time,
// floor by the codes' bytes: 1 x 4096 -> 6144, groups of 128, 9.0 us (1.9; an empty
// kernel is seen to take 4.7); 1 x 4096 -> 28672, 18.4 us (8.9); 8 x 14336 -> 4096, 14.2 us
// (4.6); 40 x 1280 -> 15360, groups of 32, 18.6 us (1.8); 64 x 4096 -> 14336, 51 us (4.9,
// and 12 by mma.sync's own rate).  Those are with codes in the L2; from HBM 10.2, 18.9,
// 15.6, 19.2 and 51 us.
// y = x W^T (+ bias): a CTA takes 8 / WK blocks of 32 weight rows and up to 8*NT
// activation rows, or (gridDim.z > 1) its cluster does.  LOCAL: it stages those itself,
// in shared memory; else `in` has them.
template <int GROUP, int NT, bool LOCAL>
__global__ void __launch_bounds__(kRowWarps * 32, LOCAL ? 3 : 2)
    w4_linear_kernel(const __nv_bfloat16* __restrict__ x, Staged in, const uint8_t* __restrict__ codes,
                     const __nv_bfloat16* __restrict__ scales, const uint8_t* __restrict__ zeros,
                     const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ y, int rows, int K, int N,
                     int WK, const uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  const uint32_t failed = ld_volatile_u32(err);  // looked at before anything is written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk = warp % WK, rg = warp / WK;
  const int r0 = (static_cast<int>(blockIdx.x) * (kRowWarps / WK) + rg) * 16 * kRowTiles;
  const int n0 = static_cast<int>(blockIdx.y) * 8 * NT, count = min(rows - n0, 8 * NT);
  const int steps = w4_steps(K);
  const int slice = static_cast<int>(blockIdx.z) * WK + wk, slices = static_cast<int>(gridDim.z) * WK;
  uint8_t* joins = smem + w4_ring_bytes<GROUP, NT>(WK);
  // rows past the last one read the last one and store nothing
  W4Stream<GROUP, NT> stream{w4_rows<GROUP>(codes, scales, zeros, K, [&](int i) { return min(r0 + i, N - 1); }),
                             r0 < N, smem + warp * w4_warp_bytes<GROUP, NT>(), K,
                             steps * slice / slices, steps * (slice + 1) / slices};
  if (r0 < N) stream.start();
  if constexpr (LOCAL) {
    in = w4_staged_at(joins + joins_bytes<NT>(WK), count, K, GROUP);
    w4_stage_local<GROUP>(in, count, K, [&](int i) {
      return reinterpret_cast<const uint8_t*>(x + static_cast<int64_t>(n0 + i) * K);
    });
  } else {
    in.frag += n0 * w4_row_bytes(K);
    in.sums += static_cast<int64_t>(n0) * w4_row_sums(K, GROUP);
    in.factor += n0;
  }
  RowSums<NT> acc;
  clear<NT>(acc);
  auto act = [](int i) { return i; };
  if constexpr (NT > 1) {
    stream.run_wide(in, count, act,
                    smem + kRowWarps * w4_warp_bytes<GROUP, NT>() + wk * w4_xring_bytes<GROUP, NT>(), rg * 32 + lane,
                    32 * (kRowWarps / WK), (steps + slices - 1) / slices, acc);
  } else if (r0 < N) {
    stream.template run<true, !LOCAL>(w4_cols<GROUP, NT>(in, K, count, act), acc);
  }
  griddep_launch_dependents();
  if (WK > 1) join_slices<NT>(acc, joins, rg, wk, WK);
  if (!LOCAL && gridDim.z > 1)
    join_cluster<NT>(acc, joins + joins_bytes<NT>(WK) + rg * join_bytes<NT>(), wk == 0 && r0 < N, gridDim.z);
  if (wk != 0 || r0 >= N || failed != 0u || blockIdx.z != 0) return;
  w4_unscale<NT>(acc, NT == 1 ? nullptr : in.factor, count, act);
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

// Narrow weights on long rows: the CTAs of a cluster take slices of K too.  16 rows,
// K = 14336, N = 4096: 23.1 us with up to 8 CTAs, 25.2 with up to 4, 67 with none.  With a
// join counted as 2 steps, 64 rows of K = 4096, N = 14336 would be split further and take
// 60 us, not 51; as 8 steps, 16 rows of it less far: 23.6 us, not 21.7.
constexpr int kClusterMost = 8, kJoinSteps = 4;

template <int GROUP, int NT, bool LOCAL>
cudaError_t launch_linear(const void* x, const Staged& in, const W4Weight& w, const void* bias, void* y, int rows,
                          int K, int N, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int kRows = 16 * kRowTiles;
  const int x_blocks = (rows + 8 * NT - 1) / (8 * NT);
  const int split = rowdot_split((static_cast<int64_t>(N) + kRows - 1) / kRows, x_blocks, w4_steps(K), LOCAL ? 3 : 2,
                                 w4_most_split<NT>(), dev.num_sms, LOCAL ? 1 : kClusterMost, kJoinSteps);
  const int WK = split < w4_most_split<NT>() ? split : w4_most_split<NT>(), CK = split / WK;
  const int smem = w4_ring_bytes<GROUP, NT>(WK) + joins_bytes<NT>(WK) +
                   (CK > 1 ? kRowWarps / WK * join_bytes<NT>() : 0) +
                   (LOCAL ? static_cast<int>(w4_staged_bytes(rows, K, GROUP, true)) : 0);
  auto kern = w4_linear_kernel<GROUP, NT, LOCAL>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), 160 * 1024, dev.device);
  if (e != cudaSuccess) return e;
  const int a_cta = kRowWarps / WK * kRows;
  const dim3 grid((N + a_cta - 1) / a_cta, x_blocks, CK), block(kRowWarps * 32);
  auto launch = [&](auto how) {
    return how(kern, grid, block, smem, s, static_cast<const __nv_bfloat16*>(x), in, w.codes, w.scales, w.zeros,
               static_cast<const __nv_bfloat16*>(bias), static_cast<__nv_bfloat16*>(y), rows, K, N, WK,
               static_cast<const uint32_t*>(dev.err));
  };
  if (CK > 1) return launch([](auto... a) { return launch_pdl_clusters_z(a...); });
  return launch([](auto... a) { return launch_pdl(a...); });
}

template <int GROUP>
cudaError_t launch_linear_g(const void* x, const W4Weight& w, const void* bias, void* y, int rows, int K, int N,
                            void* scratch, const DeviceInfo& dev, cudaStream_t s) {
  if (w4_linear_local(rows, K, GROUP))
    return launch_linear<GROUP, 1, true>(x, Staged{}, w, bias, y, rows, K, N, dev, s);
  const Staged in = w4_staged_at(static_cast<uint8_t*>(scratch), rows, K, GROUP);
  const int ctas = rows <= 8 ? (rows * w4_steps(K) + 15) / 16 : rows;
  const int grid = ctas < 8 * dev.num_sms ? ctas : 8 * dev.num_sms;
  auto stage = rows <= 8 ? w4_stage_kernel<GROUP, true> : w4_stage_kernel<GROUP, false>;
  cudaError_t e = launch_pdl(stage, dim3(grid), dim3(256), 0, s,
                             static_cast<const __nv_bfloat16*>(x), in, rows, K, static_cast<const uint32_t*>(dev.err));
  if (e != cudaSuccess) return e;
  // blocks of up to four column tiles, as even as it goes
  const int tiles = (rows + 7) / 8, blocks = (tiles + 3) / 4;
  switch ((tiles + blocks - 1) / blocks) {
    case 1: return launch_linear<GROUP, 1, false>(x, in, w, bias, y, rows, K, N, dev, s);
    case 2: return launch_linear<GROUP, 2, false>(x, in, w, bias, y, rows, K, N, dev, s);
    case 3: return launch_linear<GROUP, 3, false>(x, in, w, bias, y, rows, K, N, dev, s);
    default: return launch_linear<GROUP, 4, false>(x, in, w, bias, y, rows, K, N, dev, s);
  }
}

template <int GROUP>
cudaError_t launch_quant_g(const void* w, void* codes, void* scales, void* zeros, int64_t pieces, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((pieces + 256 * kQuantPieces - 1) / (256 * kQuantPieces)));
  auto kern = zeros ? w4_quantize_kernel<GROUP, true> : w4_quantize_kernel<GROUP, false>;
  return launch_pdl(kern, grid, dim3(256), 0, s, static_cast<const uint4*>(w), static_cast<uint32_t*>(codes),
                    static_cast<__nv_bfloat16*>(scales), static_cast<uint8_t*>(zeros), pieces);
}

template <int GROUP>
cudaError_t launch_dequant_g(const void* codes, const void* scales, const void* zeros, void* w, int64_t pieces,
                             cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((pieces + 256 * kDequantPieces - 1) / (256 * kDequantPieces)));
  auto kern = zeros ? w4_dequantize_kernel<GROUP, true> : w4_dequantize_kernel<GROUP, false>;
  return launch_pdl(kern, grid, dim3(256), 0, s, static_cast<const uint32_t*>(codes),
                    static_cast<const __nv_bfloat16*>(scales), static_cast<const uint8_t*>(zeros),
                    static_cast<uint4*>(w), pieces);
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

// Up to 8 rows whose staged form takes no more than 16 KB are staged by every CTA
// itself, which saves a launch: 1 x 2048 -> 4096 takes 5.2 us so, and 5.9 behind a
// staging kernel; 1 x 4096 -> 6144 9.1 and 8.7, with 2 us less for the host.  With more
// the CTAs' own staging costs more than the kernel: 3 x 5120 -> 5120 12.7 and 9.9 us,
// 2 x 4096 -> 4096 8.1 and 7.1, 1 x 14336 -> 4096 14.0 and 12.2.
bool w4_linear_local(int64_t rows, int64_t K, int group) {
  return rows <= 8 && K <= 32768 && w4_staged_bytes(rows, static_cast<int>(K), group, true) <= 16 * 1024;
}

size_t w4_linear_scratch_bytes(int64_t rows, int64_t K) {
  // of the finest group; the group is not known to the query
  return static_cast<size_t>(w4_staged_bytes(rows, static_cast<int>(K), 32, rows <= 8));
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
