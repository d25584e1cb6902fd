// The block-scaled e4m3 format (include/dg.h) on values in registers: scale bytes, codes, and bf16 vectors taken apart.
#pragma once

#include "dg_ptx.cuh"

namespace dg {

constexpr uint32_t kScaleNan = 0xffu;
constexpr uint32_t kCodeNan4 = 0x7f7f7f7fu;  // four e4m3 NaN codes
constexpr int kMinExp = -124;                // 2^-124 * 2^-9 = 2^-133: every value is a bf16 number

// e8m0 byte of a block whose largest magnitude has the binary32 bits `a`: 127 + e with
// the least e >= kMinExp for which amax <= 448 * 2^e (448 = 1.75 * 2^8).
static __device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  if (a == 0u) return 127u;
  if (a >= 0x7f800000u) return kScaleNan;
  const int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, kMinExp) + 127);
}
// 2^-(byte - 127) for a byte of scale_byte that is no NaN (3..247).
static __device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^(byte - 127) of any byte.
static __device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == kScaleNan ? 0x7fc00000u : byte << 23);
}

static __device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Eight values in binary32 -> eight codes of a block with the given scale byte.
static __device__ __forceinline__ uint2 codes8(const float (&v)[8], uint32_t byte) {
  if (byte == kScaleNan) return make_uint2(kCodeNan4, kCodeNan4);
  const float k = scale_inverse(byte);
  return make_uint2(e4m3x4(v[0] * k, v[1] * k, v[2] * k, v[3] * k), e4m3x4(v[4] * k, v[5] * k, v[6] * k, v[7] * k));
}

static __device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
static __device__ __forceinline__ void unpack4x2(const uint4& u, float2 (&v)[4]) {
  v[0] = unpack_bf16x2(u.x);
  v[1] = unpack_bf16x2(u.y);
  v[2] = unpack_bf16x2(u.z);
  v[3] = unpack_bf16x2(u.w);
}
static __device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Largest magnitude of eight bf16 values as 16-bit patterns (sign bits cleared; a NaN is the largest).
static __device__ __forceinline__ uint32_t amax_bits8(const uint4& u) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
  return max(a & 0xffffu, a >> 16);
}

}  // namespace dg
