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
//  - The activations are brought to that form once (w4_stage_row, w4_stage_local): a
//    row, or 128 columns of it, is scaled by a power of two so that its largest
//    magnitude lies between 2^14 and 2^15, rounded to fp16, columns 1 3 5 7 of 8
//    divided by 16, in the order the lanes take them.  A bf16 number has 8 significant
//    bits and fp16 numbers come in steps of 2^-24, so all down to 2^-27 of the largest
//    are exact.  Smaller ones are off by at most half a step: 2^-25 of 2^14, that is
//    2^-39 of the largest, and 16 times that, 2^-35, in the odd columns.
//  - The zero point is taken out of the group's sum at the end:
//    sum (q - z) x = sum q x - z * sum x, the second sum made with the scaling.
//
// Inserting exponents took 49 us where this takes 37 (8 experts of 3 x 4096 x 1792, one
// token), and 176 where this takes 101 (128 experts of 3 x 2048 x 768, 48 tokens).
// Tensor-map copies in place of the 16-byte ones below changed nothing: it is not the
// bytes.
//
// A step is 128 columns: 64 bytes of codes a row.  A lane takes a quarter of each
// group, so an mma never mixes groups.
#pragma once

#include <cuda_fp16.h>

#include "dg_rowdot.cuh"

namespace dg {

constexpr int kW4Step = 128;

// Staged activations: of every row and step 256 bytes of fp16 (pieces of 8
// columns, [piece of a lane][lane t]); of every row and group the sum of its scaled
// columns; of every row (or, of up to 8 rows, every step of a row) its factor, a
// power of two.  Rows are padded by 64 bytes against bank conflicts in
// shared memory.
struct Staged {
  uint8_t* frag;
  float* sums;
  float* factor;
};
__host__ __device__ inline int w4_steps(int K) { return (K + kW4Step - 1) / kW4Step; }
__host__ __device__ inline int64_t w4_row_bytes(int K) { return 256 * static_cast<int64_t>(w4_steps(K)) + 64; }
__host__ __device__ inline int w4_row_sums(int K, int group) { return w4_steps(K) * (kW4Step / group); }
__host__ __device__ inline int64_t w4_sums_bytes(int64_t rows, int K, int group) {
  return (4 * rows * w4_row_sums(K, group) + 15) / 16 * 16;
}
__host__ __device__ inline int64_t w4_staged_bytes(int64_t rows, int K, int group, bool step_factors = false) {
  return rows * w4_row_bytes(K) + w4_sums_bytes(rows, K, group) +
         (4 * rows * (step_factors ? w4_steps(K) : 1) + 15) / 16 * 16;
}
__host__ __device__ inline Staged w4_staged_at(uint8_t* p, int64_t rows, int K, int group) {
  float* sums = reinterpret_cast<float*>(p + rows * w4_row_bytes(K));
  return Staged{p, sums, sums + w4_sums_bytes(rows, K, group) / 4};
}

// The largest finite magnitude of a piece of 8 columns, as bits; what is not
// finite stays so and has no part in the scale.
static __device__ __forceinline__ uint32_t w4_top(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
    top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
  }
  return top;
}
// Exponent E of a row's scale 2^(14 - E); at least -100, so that the scale and the factor
// are normal numbers.
static __device__ __forceinline__ int w4_exponent(uint32_t top) { return max(static_cast<int>(top >> 7) - 127, -100); }
// A row's factor: what its products, in units of 2^-24 for the codes and 2^(E - 14) for
// the activations, are multiplied by beside kW4Unit.  It goes to the weights' scales
// before their product with a sum.  The unit is so small that results down to the
// smallest bf16 numbers are held on the way (with 2^24, results below 2^-117 were not),
// and no smaller, so that a scale below 32 is finite beside the largest factor, 2^123.
constexpr float kW4Unit = 16384.0f;
static __device__ __forceinline__ float w4_factor(int E) { return __int_as_float((127 - 4 + E) << 23); }

// Stages pieces p of steps `st` of a row: the 16 lanes of half a warp hold the 16
// pieces of one step; all lanes of the warp call together.  Nothing is written
// where !exists.
template <int GROUP>
static __device__ __forceinline__ void w4_stage_piece(const uint4& v, int E, int p, int st, bool exists,
                                                      uint8_t* frag, float* sums) {
  constexpr int W = GROUP / 32;  // code words of a group a lane takes
  const float scale = __int_as_float((127 + 14 - E) << 23);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_bf16x2(w[i]);
    f[2 * i] = a.x * scale;
    f[2 * i + 1] = a.y * scale;
    sum += f[2 * i] + f[2 * i + 1];
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
  *reinterpret_cast<uint4*>(frag + static_cast<int64_t>(st) * 256 + (p / (4 * W) * W + p % W) * 64 +
                            (p / W) % 4 * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  if (p % (4 * W) == 0) sums[st * (kW4Step / GROUP) + p / (4 * W)] = sum * __int_as_float((127 - 24) << 23);
}

// Stages one row [K] bf16 by the 256 threads of a CTA; `shared_top`: a word that is
// 0 and is left 0.  frag may lie over x: a step's pieces are written by the lanes
// that have read them.  Synchronises the CTA.
template <int GROUP>
static __device__ __forceinline__ void w4_stage_row(const uint8_t* x, int K, uint8_t* frag, float* sums, float* factor,
                                                    uint32_t* shared_top) {
  const int p = threadIdx.x & 15, steps = w4_steps(K);
  auto piece = [&](int st) {
    const int k = st * kW4Step + 8 * p;
    return st < steps && k < K ? *reinterpret_cast<const uint4*>(x + 2 * static_cast<int64_t>(k))
                               : make_uint4(0u, 0u, 0u, 0u);
  };
  uint32_t top = 0u;
  for (int st = threadIdx.x >> 4; st < steps; st += 16) top = max(top, w4_top(piece(st)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) atomicMax(shared_top, top);
  __syncthreads();
  const int E = w4_exponent(*shared_top);
  for (int s0 = 0; s0 < steps; s0 += 16) {
    const int st = s0 + (threadIdx.x >> 4);
    w4_stage_piece<GROUP>(piece(st), E, p, st, st < steps, frag, sums);
  }
  if (threadIdx.x == 0) *factor = w4_factor(E);
  __syncthreads();
  if (threadIdx.x == 0) *shared_top = 0u;
  __syncthreads();
}

// Stages up to 8 rows, every step with a scale of its own (factors[row * steps +
// step]): a row's largest would take another pass and a barrier.  row(i): row i.  The
// 256 threads of a CTA take 16 steps at a time, from the 16th of number `block` on,
// every `blocks`.
template <int GROUP, typename Row>
static __device__ __forceinline__ void w4_stage_steps(const Staged& out, int count, int K, int block, int blocks,
                                                      Row row) {
  const int p = threadIdx.x & 15, hw = threadIdx.x >> 4, steps = w4_steps(K), total = count * steps;
  const int64_t rb = w4_row_bytes(K);
  const int fs = w4_row_sums(K, GROUP);
  for (int i0 = 16 * block; i0 < total; i0 += 16 * blocks) {
    const int i = i0 + hw, r = count == 1 ? 0 : i / steps, st = i - r * steps, k = st * kW4Step + 8 * p;
    const bool exists = i < total;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (exists && k < K) v = *reinterpret_cast<const uint4*>(row(r) + 2 * static_cast<int64_t>(k));
    uint32_t top = w4_top(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int E = w4_exponent(top);
    w4_stage_piece<GROUP>(v, E, p, st, exists, out.frag + r * rb, out.sums + static_cast<int64_t>(r) * fs);
    if (exists && p == 0) out.factor[i] = w4_factor(E);
  }
}
// The same in shared memory, by one CTA, which it synchronises.
template <int GROUP, typename Row>
static __device__ __forceinline__ void w4_stage_local(const Staged& out, int count, int K, Row row) {
  w4_stage_steps<GROUP>(out, count, K, 0, 1, row);
  __syncthreads();
}

// c += a b, or (FIRST) c = a b.
template <bool FIRST>
static __device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// 8n + g, in 16-byte units from xs; sums[n][i] that of column 8n + 2t + i, in
// numbers from xsums.
template <int NT>
struct W4Cols {
  const uint8_t* xs;
  const float* xsums;
  const float* factors;  // of every step of a row, if every step has one
  uint32_t frag[NT], sums[NT][2];
  int frow[2];  // rows of the columns 2t and 2t + 1, in steps from factors
};

// Each warp keeps w4_ring - 1 steps of its rows' codes on the way from HBM in a
// ring of its own, filled by 16-byte asynchronous copies.  A row's 64 bytes of a
// step are swizzled by pieces of 16, so that reads of a piece, half a piece or a
// word a lane all spread over the banks.
template <int NT>
constexpr int w4_ring() {
  return NT > 2 ? 2 : 3;  // two CTAs an SM (40 x 1280 -> 15360 with 3 for NT = 3: 21.9 us, not 18.6)
}
constexpr int kW4StepBytes = kLaneRows * 512;
// Behind the codes: {-zero point, scale} of the warp's 32 rows, [G][32], two steps.
template <int GROUP, int NT>
constexpr int w4_warp_bytes() {
  return w4_ring<NT>() * kW4StepBytes + 2 * 256 * (kW4Step / GROUP);
}
// NT > 1: the staged activations of a slice of K, brought to shared memory once for
// its warps, by steps: fragments in the order the lanes take them, [4][NT][32 lanes]
// of 16 bytes, and the sums, [8*NT][G].
template <int GROUP, int NT>
constexpr int w4_xstep_bytes() {
  return NT * 2048 + 8 * NT * 4 * (kW4Step / GROUP);
}
template <int GROUP, int NT>
constexpr int w4_xring_bytes() {
  return NT > 1 ? w4_ring<NT>() * w4_xstep_bytes<GROUP, NT>() : 0;
}
// The rings of a CTA whose warps split K WK ways.
template <int GROUP, int NT>
constexpr int w4_ring_bytes(int WK) {
  return kRowWarps * w4_warp_bytes<GROUP, NT>() + WK * w4_xring_bytes<GROUP, NT>();
}
// More slices of K would need more room than two CTAs an SM have.
template <int NT>
constexpr int w4_most_split() {
  return NT == 1 ? kRowWarps : 2;
}

// What a lane takes of a step's activations in memory (NT = 1), asked for a step ahead.
template <int GROUP>
struct W4Ahead {
  uint4 b[4];
  float sum[2][kW4Step / GROUP], f[2];
};

// The sums of a row's groups of one step.
template <int G>
static __device__ __forceinline__ void w4_load_sums(float (&to)[G], const float* p) {
  if constexpr (G == 4) *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(p);
  else if constexpr (G == 2) *reinterpret_cast<float2*>(to) = *reinterpret_cast<const float2*>(p);
  else to[0] = *p;
}

template <int GROUP, bool STEP_FACTORS>
static __device__ __forceinline__ void w4_ahead(W4Ahead<GROUP>& a, const W4Cols<1>& x, int c) {
  constexpr int G = kW4Step / GROUP;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a.b[i] = *reinterpret_cast<const uint4*>(x.xs + (static_cast<uint64_t>(x.frag[0]) + 16 * c) * 16 + i * 64);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w4_load_sums<G>(a.sum[i], x.xsums + static_cast<uint64_t>(x.sums[0][i]) + c * G);
    a.f[i] = STEP_FACTORS ? x.factors[x.frow[i] + c] : 1.0f;
  }
}

// One step's product.  slot: its codes; zs: {-zero point, scale} of the warp's rows;
// the step's activations are in shared memory at xstep (NT > 1), or in registers.
// STEP_FACTORS (NT = 1): the activations' factor of the step is applied too.
template <int GROUP, int NT, bool STEP_FACTORS>
static __device__ __forceinline__ void w4_use(const uint8_t* slot, const uint8_t* zs, const W4Ahead<GROUP>* x,
                                              const uint8_t* xstep, int c, int groups, RowSums<NT>& acc) {
  constexpr int G = kW4Step / GROUP;  // groups a step
  constexpr int W = GROUP / 32;       // code words of a row and group a lane takes
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int swz = (g >> 1) & 3;
  const float f0 = STEP_FACTORS ? x->f[0] : 1.0f, f1 = STEP_FACTORS ? x->f[1] : 1.0f;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    if (G == 1 || c * G + q < groups) {  // a group is whole or absent
      // this lane's words of the group: piece and offset within the row's 64 bytes
      const int piece = GROUP == 128 ? t : GROUP == 64 ? 2 * q + (t >> 1) : q;
      const int off = GROUP == 128 ? 0 : GROUP == 64 ? 8 * (t & 1) : 4 * t;
      const uint8_t* from = slot + g * 64 + (piece ^ swz) * 16 + off;
      // one row tile at a time where both would not fit the registers
      constexpr int kTogether = NT > 2 ? 1 : kRowTiles;
#pragma unroll
      for (int m0 = 0; m0 < kRowTiles; m0 += kTogether) {
        float part[kTogether][NT][4];
        uint32_t code[2 * kTogether][W];
#pragma unroll
        for (int i = 0; i < 2 * kTogether; ++i) {
          const uint8_t* p = from + (2 * m0 + i) * 512;
          if constexpr (W == 4) *reinterpret_cast<uint4*>(code[i]) = *reinterpret_cast<const uint4*>(p);
          else if constexpr (W == 2) *reinterpret_cast<uint2*>(code[i]) = *reinterpret_cast<const uint2*>(p);
          else code[i][0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if constexpr (NT > 2 && W == 4) {
              // in order: the compiler would bring four words' fragments forward and
              // spill (64 rows, K = 4096, N = 14336: 51 us this way, 66 us that)
              asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(b[n].x), "=r"(b[n].y), "=r"(b[n].z), "=r"(b[n].w)
                           : "r"(smem_u32(xstep) + ((q * W + j) * NT + n) * 512 + lane * 16));
            } else if constexpr (NT > 1) {
              b[n] = *reinterpret_cast<const uint4*>(xstep + ((q * W + j) * NT + n) * 512 + lane * 16);
            } else {
              b[n] = x->b[q * W + j];
            }
#pragma unroll
          for (int m = 0; m < kTogether; ++m) {
            const uint32_t l = code[2 * m][j], h = code[2 * m + 1][j];
            const uint32_t l8 = l >> 8, h8 = h >> 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (j == 0)
                mma_f16<true>(part[m][n], l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u,
                                        h & 0x00f000f0u, b[n].x, b[n].y);
              else
                mma_f16<false>(part[m][n], l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u,
                                         h & 0x00f000f0u, b[n].x, b[n].y);
              mma_f16<false>(part[m][n], l8 & 0x000f000fu, h8 & 0x000f000fu, l8 & 0x00f000f0u,
                                       h8 & 0x00f000f0u, b[n].z, b[n].w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < kTogether; ++m) {
          const uint8_t* p = zs + q * 256 + (16 * (m0 + m) + g) * 8;
          const float2 l = *reinterpret_cast<const float2*>(p), h = *reinterpret_cast<const float2*>(p + 64);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float(&to)[4] = acc[m0 + m][n];
            // sums of the columns 8n + 2t and 8n + 2t + 1 over the group
            const float* sums = reinterpret_cast<const float*>(xstep + NT * 2048) + (8 * n + 2 * t) * G + q;
            const float x0 = NT > 1 ? sums[0] : x->sum[0][q], x1 = NT > 1 ? sums[G] : x->sum[1][q];
            to[0] = fmaf(STEP_FACTORS ? l.y * f0 : l.y, fmaf(l.x, x0, part[m][n][0]), to[0]);
            to[1] = fmaf(STEP_FACTORS ? l.y * f1 : l.y, fmaf(l.x, x1, part[m][n][1]), to[1]);
            to[2] = fmaf(STEP_FACTORS ? h.y * f0 : h.y, fmaf(h.x, x0, part[m][n][2]), to[2]);
            to[3] = fmaf(STEP_FACTORS ? h.y * f1 : h.y, fmaf(h.x, x1, part[m][n][3]), to[3]);
          }
        }
      }
    }
  }
}

// The codes and scales of steps [c0, c1) of a warp's rows, for up to 8*NT columns.
// start() is apart from run() and run_wide(), so that a kernel can ask for them
// before it has its activations.
template <int GROUP, int NT>
struct W4Stream {
  static constexpr int G = kW4Step / GROUP;
  static constexpr int R = w4_ring<NT>();
  W4Rows w;
  bool active;    // the warp has rows
  uint8_t* ring;  // this warp's w4_warp_bytes
  int K, c0, c1;
  // scales and zero points of row `lane`, of the step after the last one decoded, as they lie in memory
  uint32_t s[2], z;
  uint32_t ones;  // bit q: group q of row `lane` in the step last decoded has scale 1

  __device__ __forceinline__ void fill(int c, int u) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool in = active && c < c1 && c * kW4Step + 32 * t < K;
    const int64_t at = in ? static_cast<int64_t>(c) * 64 + 16 * t : 0;
    const uint32_t dst = smem_u32(ring) + u * kW4StepBytes + g * 64 + (t ^ ((g >> 1) & 3)) * 16;
    cp_async16(dst, w.codes + at, in);
    cp_async16(dst + 512, w.codes + w.next0 + at, in);
    cp_async16(dst + 1024, w.codes1 + at, in);
    cp_async16(dst + 1536, w.codes1 + w.next1 + at, in);
  }
  __device__ __forceinline__ void load_scales(int c) {
    if (!active || c >= c1) return;
    const int64_t at = static_cast<int64_t>(c) * G;
    if (G == 1 || K % kW4Step == 0) {  // every row's scales start on a boundary of the vector
      if constexpr (G == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(w.scales + at);
        s[0] = v.x;
        s[1] = v.y;
        if (w.zeros) z = *reinterpret_cast<const uint32_t*>(w.zeros + at);
      } else if constexpr (G == 2) {
        s[0] = *reinterpret_cast<const uint32_t*>(w.scales + at);
        if (w.zeros) z = *reinterpret_cast<const uint16_t*>(w.zeros + at);
      } else {
        s[0] = *reinterpret_cast<const uint16_t*>(w.scales + at);
        if (w.zeros) z = w.zeros[at];
      }
    } else {
      s[0] = s[1] = z = 0u;
#pragma unroll
      for (int q = 0; q < G; ++q)
        if ((c * G + q) * GROUP < K) {
          s[q / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(w.scales + at + q)) << (16 * (q % 2));
          if (w.zeros) z |= static_cast<uint32_t>(w.zeros[at + q]) << (8 * q);
        }
    }
  }
  __device__ __forceinline__ uint8_t* decoded(int parity) const {
    return ring + R * kW4StepBytes + parity * 256 * G;
  }
  __device__ __forceinline__ void decode(int parity) {
    ones = 0u;
#pragma unroll
    for (int q = 0; q < G; ++q) {
      // -z by way of a binary32 significand
      const float nz = w.zeros ? 8388608.0f - __uint_as_float(0x4b000000u | ((z >> (8 * q)) & 15u)) : -8.0f;
      const uint32_t two = s[q / 2];
      if ((q % 2 ? two >> 16 : two & 0xffffu) == 0x3f80u) ones |= 1u << q;
      *reinterpret_cast<float2*>(decoded(parity) + q * 256 + (threadIdx.x & 31) * 8) =
          make_float2(nz, __uint_as_float(q % 2 ? two & 0xffff0000u : two << 16));
    }
  }
  // A group of zeros is quantised to its zero point with scale 1.  What rounding leaves
  // of sum q x - z * sum x would show there, beside weights that are mostly far below 1:
  // such groups get scale 0, and add exactly nothing.  which: `ones` of the step in
  // `slot`, whose decoded scales are zs.
  __device__ __forceinline__ void drop_zeros(const uint8_t* slot, uint8_t* zs, uint32_t which) const {
    if (!active || !__any_sync(0xffffffffu, which != 0u)) return;
    const int lane = threadIdx.x & 31, g = lane & 7;
    for (int q = 0; q < G; ++q) {
      if (!(which >> q & 1u)) continue;
      float2* p = reinterpret_cast<float2*>(zs + q * 256 + lane * 8);
      const uint32_t zero = static_cast<uint32_t>(static_cast<int>(-p->x)) * 0x11111111u;
      bool all = true;
      for (int i = 0; i < GROUP / 32; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + (lane >> 3) * 512 + g * 64 +
                                                        ((q * (GROUP / 32) + i) ^ ((g >> 1) & 3)) * 16);
        all = all && v.x == zero && v.y == zero && v.z == zero && v.w == zero;
      }
      if (all) p->y = 0.0f;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void start() {
    load_scales(c0);
#pragma unroll
    for (int u = 0; u < R - 1; ++u) fill(c0 + u, u);
  }
  // acc += the product with staged activation rows, in units of w4_unscale.
  // Thread (g, t) ends with acc[m][n] = (row g of tile m, columns 8n + 2t, 8n + 2t + 1;
  // row g + 8, the same).  NT = 1: an active warp by itself, the lanes read `x`, AHEAD:
  // a step before they use it.  STEP_FACTORS: every step of a row has its factor.
  template <bool STEP_FACTORS, bool AHEAD>
  __device__ __forceinline__ void run(const W4Cols<NT>& x, RowSums<NT>& acc) {
    const int groups = K / GROUP;
#pragma unroll
    for (int u = 0; u < R - 1; ++u) cp_async_commit();  // the first holds all of start()'s
    decode(0);
    load_scales(c0 + 1);
    W4Ahead<GROUP> next;
    if (AHEAD && c0 < c1) w4_ahead<GROUP, STEP_FACTORS>(next, x, c0);
    int parity = 0;
#pragma unroll 1
    for (int c = c0; c < c1; c += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (c + u >= c1) break;
        cp_async_wait<R - 2>();
        // the other lanes' copies and scales are in place, and what the step before has read is free
        __syncwarp();
        fill(c + u + R - 1, (u + R - 1) % R);
        cp_async_commit();
        uint8_t* zs = decoded(parity);
        drop_zeros(ring + u * kW4StepBytes, zs, ones);
        parity ^= 1;
        decode(parity);
        load_scales(c + u + 2);
        W4Ahead<GROUP> now;
        if constexpr (AHEAD) {
          now = next;
          if (c + u + 1 < c1) w4_ahead<GROUP, STEP_FACTORS>(next, x, c + u + 1);
        } else {
          w4_ahead<GROUP, STEP_FACTORS>(now, x, c + u);
        }
        w4_use<GROUP, NT, STEP_FACTORS>(ring + u * kW4StepBytes, zs, &now, nullptr, c + u, groups, acc);
      }
    }
    cp_async_wait<0>();
    __syncwarp();
  }
  // The same for NT > 1: all warps of the CTA together, with the same `steps` >=
  // c1 - c0.  xring: the w4_xring_bytes of this warp's slice, filled by its `nx`
  // threads, of which this is number `ix`.  act(i): index of the staged row of column
  // i, for i < count; other columns get the last one and are not used.
  template <typename Act>
  __device__ __forceinline__ void run_wide(const Staged& in, int count, Act act, uint8_t* xring, int ix, int nx,
                                           int steps, RowSums<NT>& acc) {
    constexpr int kX = w4_xstep_bytes<GROUP, NT>();
    const int groups = K / GROUP, tiles = (count + 7) / 8;
    const int64_t rb = w4_row_bytes(K);
    const int fs = w4_row_sums(K, GROUP);
    auto fill_x = [&](int c, int u) {
      if (c < c1) {
        const uint32_t to = smem_u32(xring) + u * kX;
#pragma unroll 1
        for (int i = ix; i < tiles * 128; i += nx) {  // 16 pieces a row, as they lie in the staged row
          const int row = i / 16, p = i % 16;         // p = 4 * (piece of a lane) + t
          cp_async16(to + ((p / 4) * NT + row / 8) * 512 + ((row % 8) * 4 + p % 4) * 16,
                     in.frag + act(min(row, count - 1)) * rb + static_cast<int64_t>(c) * 256 + p * 16, true);
        }
#pragma unroll 1
        for (int row = ix; row < tiles * 8; row += nx) {
          const float* from = in.sums + act(min(row, count - 1)) * static_cast<int64_t>(fs) + c * G;
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + NT * 2048 + row * 4 * G), "l"(from),
                       "n"(4 * G)
                       : "memory");
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < R - 1; ++u) fill_x(c0 + u, u);
    decode(0);
    load_scales(c0 + 1);
    int parity = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < steps; s0 += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (s0 + u >= steps) break;
        const int c = c0 + s0 + u;
        cp_async_wait<R - 2>();
        __syncthreads();  // the step is in place, and what the step before has read is free
        fill(c + R - 1, (u + R - 1) % R);
        fill_x(c + R - 1, (u + R - 1) % R);
        uint8_t* zs = decoded(parity);
        drop_zeros(ring + u * kW4StepBytes, zs, ones);
        parity ^= 1;
        decode(parity);
        load_scales(c + 2);
        if (active && c < c1)
          w4_use<GROUP, NT, false>(ring + u * kW4StepBytes, zs, nullptr, xring + u * kX, c, groups, acc);
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings may be filled again
  }
};

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
static __device__ __forceinline__ W4Cols<NT> w4_cols(const Staged& in, int K, int count, Act act) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  W4Cols<NT> x;
  x.xs = in.frag;
  x.xsums = in.sums;
  x.factors = in.factor;
  for (int i = 0; i < 2; ++i) x.frow[i] = static_cast<int>(act(min(2 * t + i, count - 1))) * w4_steps(K);
  const uint32_t rb = static_cast<uint32_t>(w4_row_bytes(K) / 16);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    x.frag[n] = static_cast<uint32_t>(act(min(8 * n + g, count - 1))) * rb + t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x.sums[n][i] = static_cast<uint32_t>(act(min(8 * n + 2 * t + i, count - 1))) * w4_row_sums(K, GROUP);
  }
  return x;
}

// The sums are in units of 1 / kW4Unit and of their row's factor (NULL: that has been
// applied).  The factor first, as kW4Unit says.
template <int NT, typename Act>
static __device__ __forceinline__ void w4_unscale(RowSums<NT>& acc, const float* factor, int count, Act act) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = factor ? factor[act(min(8 * n + 2 * t + i, count - 1))] : 1.0f;
#pragma unroll
      for (int m = 0; m < kRowTiles; ++m) {
        acc[m][n][i] = acc[m][n][i] * f * kW4Unit;
        acc[m][n][2 + i] = acc[m][n][2 + i] * f * kW4Unit;
      }
    }
}

}  // namespace dg
