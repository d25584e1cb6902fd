// Products of weight rows with a few activation rows, one warp at a time: the
// core of the few-token operators (4-bit linear, routed SwiGLU experts).
//
//   acc[r, n] = sum_k w[r, k] * x[n, k]      16 weight rows, 8*NT activation rows
//
// With few activation rows the weights are the traffic, so each weight is read
// from HBM once, straight into registers, and meets all activation rows there:
// mma.sync m16n8k16 takes the weight fragment from the registers it was loaded
// (or decoded) into, and no shared-memory pass is spent on the stream.
//
// The contraction index of an mma is only a label, the same on both operands,
// so lane (g, t) = (lane / 4, lane % 4) of a warp owns CONSECUTIVE columns of
// weight rows g and g + 8 and of activation row g, loads them as one wide
// vector and feeds them to consecutive mma steps:
//   bf16  : 8 columns, 16 bytes a lane: 32 columns a chunk, two mma steps
//   4 bits: one group a chunk (a quarter of it a lane, 4 to 16 bytes), so an
//           mma never mixes groups; the group's integer sum
//           sum (q - z) * x, exact products in binary32, is scaled once.
// 4-bit codes become bf16 integers by placing them in the mantissa of 128
// (0x4300 | q = 128 + q) and subtracting 128 + z, both exact.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_ptx.cuh"

namespace dg {

// Weight formats: bf16, or 4-bit codes with this group size.
constexpr int kFmtBf16 = 0;

// 16 weight rows seen by one lane: its rows g and g + 8.
struct RowPair {
  const uint8_t* lo;            // row data (bf16 values or codes)
  const uint8_t* hi;
  const __nv_bfloat16* s_lo;    // 4 bits: scales of the row's groups
  const __nv_bfloat16* s_hi;
  const uint8_t* z_lo;          // 4 bits: zero points of the row's groups (NULL: 8)
  const uint8_t* z_hi;
};

template <int FMT>
constexpr int rowdot_chunk() {
  return FMT == kFmtBf16 ? 32 : FMT;
}

// Weights are read once: no L1 line is spent on them.
template <int BYTES>
static __device__ __forceinline__ void ld_weights(const uint8_t* p, uint32_t (&r)[BYTES / 4]) {
  if constexpr (BYTES == 16)
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
  else if constexpr (BYTES == 8)
    asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r[0]) : "l"(p));
}

static __device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Columns (i, i + 4) of a code word as a bf16 pair of q - z, zb = bf16x2 of 128 + z.
static __device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i, uint32_t zb) {
  const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zb));
  return *reinterpret_cast<const uint32_t*>(&d);
}

static __device__ __forceinline__ uint32_t w4_zero_bits(const uint8_t* z, int64_t group) {
  const uint32_t v = z ? static_cast<uint32_t>(z[group]) & 15u : 8u;
  return 0x43004300u | v | (v << 16);
}

// acc += chunks [c0, c1) of the product of the row pair with the activation
// rows xr[n] (this lane's row 8n + g; NULL where there is none).  Thread (g, t)
// ends with acc[n] = (row g, columns 8n + 2t, 8n + 2t + 1; row g + 8, the same).
template <int FMT, int NT>
static __device__ __forceinline__ void row_dot(const RowPair& w, const __nv_bfloat16* const (&xr)[NT], int K, int c0,
                                               int c1, float (&acc)[NT][4]) {
  const int t = threadIdx.x & 3;
  if constexpr (FMT == kFmtBf16) {
    constexpr int U = 4;  // 128 bytes of weights a lane in flight
    for (int c = c0; c < c1; c += U) {
      uint32_t lo[U][4], hi[U][4];
      bool in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (c + u) * 32 + 8 * t;
        in[u] = c + u < c1 && k < K;
        if (in[u]) {
          ld_weights<16>(w.lo + 2 * static_cast<int64_t>(k), lo[u]);
          ld_weights<16>(w.hi + 2 * static_cast<int64_t>(k), hi[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) lo[u][i] = hi[u][i] = 0u;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (c + u) * 32 + 8 * t;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 b = make_uint4(0u, 0u, 0u, 0u);
          if (in[u] && xr[n]) b = *reinterpret_cast<const uint4*>(xr[n] + k);
          mma_bf16(acc[n], lo[u][0], hi[u][0], lo[u][1], hi[u][1], b.x, b.y);
          mma_bf16(acc[n], lo[u][2], hi[u][2], lo[u][3], hi[u][3], b.z, b.w);
        }
      }
    }
  } else {
    constexpr int W = FMT / 32;  // code words of a row a lane takes from a chunk
    constexpr int U = 8 / W > 4 ? 4 : 8 / W;
    for (int c = c0; c < c1; c += U) {
      uint32_t lo[U][W], hi[U][W], zlo[U], zhi[U];
      float slo[U], shi[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u < c1) {
          const int64_t at = static_cast<int64_t>(c + u) * (FMT / 2) + 4 * W * t;
          ld_weights<4 * W>(w.lo + at, lo[u]);
          ld_weights<4 * W>(w.hi + at, hi[u]);
          slo[u] = __bfloat162float(w.s_lo[c + u]);
          shi[u] = __bfloat162float(w.s_hi[c + u]);
          zlo[u] = w4_zero_bits(w.z_lo, c + u);
          zhi[u] = w4_zero_bits(w.z_hi, c + u);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u >= c1) break;
        const int k = (c + u) * FMT + 8 * W * t;
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[n][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          uint32_t a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = w4_pair(lo[u][j], i, zlo[u]);
            b[i] = w4_pair(hi[u][j], i, zhi[u]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (xr[n]) v = *reinterpret_cast<const uint4*>(xr[n] + k + 8 * j);
            // the pairs (0,4) (1,5) | (2,6) (3,7) that the codes come in
            mma_bf16(part[n], a[0], b[0], a[1], b[1], __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
            mma_bf16(part[n], a[2], b[2], a[3], b[3], __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(slo[u], part[n][0], acc[n][0]);
          acc[n][1] = fmaf(slo[u], part[n][1], acc[n][1]);
          acc[n][2] = fmaf(shi[u], part[n][2], acc[n][2]);
          acc[n][3] = fmaf(shi[u], part[n][3], acc[n][3]);
        }
      }
    }
  }
}

// Sums acc over the WK warps that share a row group (warps wk = 0..WK-1 of
// group rg hold slices of K), in a fixed order, into the group's warp 0.
// red: 8 * NT * 128 floats.  Called by all 8 warps of the CTA.
template <int NT>
static __device__ __forceinline__ void join_slices(float (&acc)[NT][4], float* red, int warp, int wk, int WK) {
  if (WK == 1) return;
  const int lane = threadIdx.x & 31;
  __syncthreads();  // the last reader of `red` is done
  if (wk != 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float4*>(red + ((warp * NT + n) * 32 + lane) * 4) =
          make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  }
  __syncthreads();
  if (wk == 0) {
    for (int s = 1; s < WK; ++s) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 v = *reinterpret_cast<const float4*>(red + (((warp + s) * NT + n) * 32 + lane) * 4);
        acc[n][0] += v.x;
        acc[n][1] += v.y;
        acc[n][2] += v.z;
        acc[n][3] += v.w;
      }
    }
  }
}

}  // namespace dg
