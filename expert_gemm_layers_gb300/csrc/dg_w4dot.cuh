// The 4-bit form of the few-token products (dg_rowdot.cuh).
//
//   acc[r, n] = sum_groups s[r, group] * sum_{k in group} (q[r, k] - z[r, group]) * x[n, k]
//
// What bounds it is not the bytes but the instructions that turn codes into
// matrix operands, so they are few:
//  - A code word holds columns 0..7 of a lane.  word & 0x000f000f is the fp16 pair
//    (q0, q4) * 2^-24 as it stands: a fp16 number below 2^-14 is its bits times
//    2^-24, and the tensor cores take such numbers exactly.  word & 0x00f000f0 is
//    (16 q1, 16 q5) * 2^-24.  With word >> 8 that makes 5 operations for 8 codes
//    (inserting an exponent and subtracting the zero point would take 11).
//  - The activations are brought to that form once (w4_stage_piece): each group of
//    a row is scaled by a power of two to magnitudes below 2^15, rounded to fp16,
//    columns 1 3 5 7 divided by 16, in the order the lanes take them.  A bf16
//    number has 8 significant bits, so it fits fp16's 11 exactly unless it is 2^28
//    times smaller than the group's largest; then it is off by at most 2^-40 of
//    that largest, far below one unit of the binary32 sum.
//  - The zero point is taken out of the group's sum at the end:
//    sum (q - z) x = sum q x - z * sum x, the second sum made with the scaling.
//
// A step is 128 columns: 64 bytes of codes a row, loaded straight into registers
// one step ahead.  A lane takes a quarter of each group, so an mma never mixes
// groups.
#pragma once

#include <cuda_fp16.h>

#include "dg_rowdot.cuh"

namespace dg {

constexpr int kW4Step = 128;

// Staged activations: of every row and step 256 bytes of fp16 (pieces of 8
// columns, [piece of a lane][lane t]), and of every row and group {factor, sum}.
// Rows are padded by 64 bytes against bank conflicts in shared memory.
__host__ __device__ inline int w4_steps(int K) { return (K + kW4Step - 1) / kW4Step; }
__host__ __device__ inline int64_t w4_row_bytes(int K) { return 256 * static_cast<int64_t>(w4_steps(K)) + 64; }
template <int GROUP>
__host__ __device__ inline int w4_fx_stride(int K) {  // {factor, sum} pairs of a row
  return w4_steps(K) * (kW4Step / GROUP);
}
template <int GROUP>
__host__ __device__ inline int64_t w4_staged_bytes(int64_t rows, int K) {
  return rows * (w4_row_bytes(K) + 8 * w4_fx_stride<GROUP>(K));
}

// Stages one piece: 8 columns (word: as bf16 pairs, or f as binary32 when IS_F32)
// of step `st` of a row.  The 16 lanes of half a warp hold the 16 pieces of one
// step (p: this lane's); all lanes of the warp call together.  frag, fx: the
// row's; nothing is written where !exists.
template <int GROUP>
static __device__ __forceinline__ void w4_stage_piece(float (&f)[8], int p, int st, bool exists, uint8_t* frag,
                                                      float2* fx) {
  constexpr int W = GROUP / 32;  // code words of a group a lane takes
  // the largest finite magnitude of the group; what is not finite stays so
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
    top = max(top, a < 0x7f800000u ? a : 0u);
  }
#pragma unroll
  for (int o = 2 * W; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  // the factor 2^(14 - E), at most 2^114, so that it and its inverse are normal numbers
  const int E = max(static_cast<int>(top >> 23) - 127, -100);
  const float scale = __int_as_float((127 + 14 - E) << 23), inverse = __int_as_float((127 - 14 + E) << 23);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] *= scale;
    sum += f[i];
  }
#pragma unroll
  for (int o = 2 * W; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // (0,4) (1,5)/16 | (2,6) (3,7)/16
    const float m = i & 1 ? 0.0625f : 1.0f;
    const __half2 h = __floats2half2_rn(f[i] * m, f[i + 4] * m);
    out[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (!exists) return;
  // piece p lies with lane t = p / W % 4, as its piece p / 4W * W + p % W
  *reinterpret_cast<uint4*>(frag + st * 256 + (p / (4 * W) * W + p % W) * 64 + (p / W) % 4 * 16) =
      make_uint4(out[0], out[1], out[2], out[3]);
  if (p % (4 * W) == 0)
    fx[st * (kW4Step / GROUP) + p / (4 * W)] = make_float2(inverse, sum * __int_as_float((127 - 24) << 23));
}

static __device__ __forceinline__ void unpack_piece(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_bf16x2(w[i]);
    f[2 * i] = a.x;
    f[2 * i + 1] = a.y;
  }
}

static __device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from a zero accumulator.
static __device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// A warp's rows of a 4-bit weight.
struct W4Rows {
  const uint8_t* codes;         // the lane's row g of tile 0, and of tile 1
  const uint8_t* codes1;
  uint32_t next0, next1;        // bytes from there to its row g + 8 of the tile
  const __nv_bfloat16* scales;  // [K / GROUP] of row `lane` of the warp's 32
  const uint8_t* zeros;         // the same; NULL: 8
};

// Staged activation rows as a lane reads them: frag[n] is the row of its column
// 8n + g, in 16-byte units from xs; fx[n][i] that of column 8n + 2t + i, in
// {factor, sum} pairs from xf.
template <int NT>
struct W4Cols {
  const uint8_t* xs;
  const float2* xf;
  uint32_t frag[NT], fx[NT][2];
};

// What a lane loads of a step: the code words of its four rows, and scale (high
// half) and zero point (low byte) of the groups of row `lane`.
template <int GROUP>
struct W4Step {
  uint32_t code[kLaneRows][4];
  uint32_t sz[kW4Step / GROUP];
};

template <int GROUP>
static __device__ __forceinline__ void w4_load(const W4Rows& w, int c, int groups, W4Step<GROUP>& v) {
  constexpr int G = kW4Step / GROUP;  // groups a step
  constexpr int W = GROUP / 32;       // code words of a row and group a lane takes
  const int t = threadIdx.x & 3;
  const uint8_t* p0 = w.codes + static_cast<int64_t>(c) * 64 + 4 * W * t;
  const uint8_t* p1 = w.codes1 + static_cast<int64_t>(c) * 64 + 4 * W * t;
  const uint8_t* p[kLaneRows] = {p0, p0 + w.next0, p1, p1 + w.next1};
#pragma unroll
  for (int q = 0; q < G; ++q) {
    if (G == 1 || c * G + q < groups) {  // a group is whole or absent
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        if constexpr (W == 4)
          asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.code[i][0]), "=r"(v.code[i][1]), "=r"(v.code[i][2]), "=r"(v.code[i][3])
                       : "l"(p[i]));
        else if constexpr (W == 2)
          asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                       : "=r"(v.code[i][2 * q]), "=r"(v.code[i][2 * q + 1])
                       : "l"(p[i] + 32 * q));
        else
          asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v.code[i][q]) : "l"(p[i] + 16 * q));
      }
      const uint32_t z = w.zeros ? w.zeros[c * G + q] : 8u;
      v.sz[q] = (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(w.scales + c * G + q)) << 16) | z;
    }
  }
}

template <int GROUP, int NT>
static __device__ __forceinline__ void w4_use(const W4Step<GROUP>& v, const W4Cols<NT>& x, int c, int groups,
                                              RowSums<NT>& acc) {
  constexpr int G = kW4Step / GROUP;
  constexpr int W = GROUP / 32;
  const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    if (G == 1 || c * G + q < groups) {
      RowSums<NT> part;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[n] = *reinterpret_cast<const uint4*>(x.xs + (static_cast<uint64_t>(x.frag[n]) + 16 * c) * 16 +
                                                 (q * W + j) * 64);
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m) {
          const uint32_t l = v.code[2 * m][q * W + j], h = v.code[2 * m + 1][q * W + j];
          const uint32_t l8 = l >> 8, h8 = h >> 8;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (j == 0)
              mma_f16_first(part[m][n], l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u, h & 0x00f000f0u, b[n].x,
                            b[n].y);
            else
              mma_f16(part[m][n], l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u, h & 0x00f000f0u, b[n].x,
                      b[n].y);
            mma_f16(part[m][n], l8 & 0x000f000fu, h8 & 0x000f000fu, l8 & 0x00f000f0u, h8 & 0x00f000f0u, b[n].z,
                    b[n].w);
          }
        }
      }
      float s[kLaneRows], z[kLaneRows];
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        const uint32_t sz = __shfl_sync(0xffffffffu, v.sz[q], 8 * i + g);
        s[i] = __uint_as_float(sz & 0xffff0000u);
        z[i] = 8388608.0f - __uint_as_float(0x4b000000u | (sz & 15u));  // -z, by way of a binary32 significand
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 x0 = x.xf[static_cast<uint64_t>(x.fx[n][0]) + c * G + q];
        const float2 x1 = x.xf[static_cast<uint64_t>(x.fx[n][1]) + c * G + q];
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m) {
          const float sl = s[2 * m], sh = s[2 * m + 1], zl = z[2 * m], zh = z[2 * m + 1];
          acc[m][n][0] = fmaf(sl * x0.x, fmaf(zl, x0.y, part[m][n][0]), acc[m][n][0]);
          acc[m][n][1] = fmaf(sl * x1.x, fmaf(zl, x1.y, part[m][n][1]), acc[m][n][1]);
          acc[m][n][2] = fmaf(sh * x0.x, fmaf(zh, x0.y, part[m][n][2]), acc[m][n][2]);
          acc[m][n][3] = fmaf(sh * x1.x, fmaf(zh, x1.y, part[m][n][3]), acc[m][n][3]);
        }
      }
    }
  }
}

// acc += steps [c0, c1), in units of 2^-24, of the product of a warp's 32 rows
// with up to 8*NT staged activation rows.  Thread (g, t) ends with acc[m][n] =
// (row g of tile m, columns 8n + 2t, 8n + 2t + 1; row g + 8, the same).
template <int GROUP, int NT>
static __device__ __forceinline__ void row_dot_w4(const W4Rows& w, const W4Cols<NT>& x, int K, int c0, int c1,
                                                  RowSums<NT>& acc) {
  const int groups = K / GROUP;
  W4Step<GROUP> a, b;
  if (c0 < c1) w4_load<GROUP>(w, c0, groups, a);
#pragma unroll 1
  for (int c = c0; c < c1; c += 2) {
    if (c + 1 < c1) w4_load<GROUP>(w, c + 1, groups, b);
    w4_use<GROUP, NT>(a, x, c, groups, acc);
    if (c + 1 >= c1) break;
    if (c + 2 < c1) w4_load<GROUP>(w, c + 2, groups, a);
    w4_use<GROUP, NT>(b, x, c + 1, groups, acc);
  }
}

// The rows of a warp, by `row(i)`: index (in `codes`, a matrix of 4-bit rows) of
// row i of the warp's 32, a valid one for every i.
template <int GROUP, typename Row>
static __device__ __forceinline__ W4Rows w4_rows(const uint8_t* codes, const __nv_bfloat16* scales,
                                                 const uint8_t* zeros, int K, Row row) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const int64_t rb = K / 2, at = static_cast<int64_t>(row(lane)) * (K / GROUP);
  return W4Rows{codes + row(g) * rb,
                codes + row(16 + g) * rb,
                static_cast<uint32_t>((row(8 + g) - row(g)) * rb),
                static_cast<uint32_t>((row(24 + g) - row(16 + g)) * rb),
                scales + at,
                zeros ? zeros + at : nullptr};
}

// The columns of a warp, by `act(i)`: index of the staged row of column i, for i < count.
// Columns without a row read the last one and are not used.
template <int GROUP, int NT, typename Act>
static __device__ __forceinline__ W4Cols<NT> w4_cols(const uint8_t* xs, const float2* xf, int K, int count, Act act) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  W4Cols<NT> x;
  x.xs = xs;
  x.xf = xf;
  const uint32_t rb = static_cast<uint32_t>(w4_row_bytes(K) / 16);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    x.frag[n] = static_cast<uint32_t>(act(min(8 * n + g, count - 1))) * rb + t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x.fx[n][i] = static_cast<uint32_t>(act(min(8 * n + 2 * t + i, count - 1))) * w4_fx_stride<GROUP>(K);
  }
  return x;
}

// The sums are in units of 2^-24, those of the codes.
template <int NT>
static __device__ __forceinline__ void w4_unscale(RowSums<NT>& acc) {
#pragma unroll
  for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] *= 16777216.0f;
}

}  // namespace dg
