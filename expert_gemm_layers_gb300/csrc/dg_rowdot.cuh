// Products of weight rows with a few activation rows, one warp at a time: the
// core of the few-token operators (4-bit linear, routed SwiGLU experts).
//
//   acc[r, n] = sum_k w[r, k] * x[n, k]      16 weight rows, 8*NT activation rows
//
// With few activation rows the weights are the traffic, so each weight is read
// from HBM once and meets all activation rows in the registers of one warp:
// mma.sync m16n8k16 takes the weight fragment as it was loaded (or decoded).
//
// The contraction index of an mma is only a label, the same on both operands,
// so lane (g, t) = (lane / 4, lane % 4) of a warp owns CONSECUTIVE columns of
// weight rows g and g + 8 and of activation row g, loads them as one wide
// vector and feeds them to consecutive mma steps:
//   bf16  : 8 columns, 16 bytes a lane: 32 columns a step, two mma
//   4 bits: a quarter of a group a lane (4 to 16 bytes), so an mma never mixes
//           groups; the group's integer sum sum (q - z) * x, exact products in
//           binary32, is scaled once.
// 4-bit codes become bf16 integers by placing them in the mantissa of 128
// (0x4300 | q = 128 + q) and subtracting 128 + z, both exact.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_ptx.cuh"

namespace dg {

// Activation rows come in two ways.  Up to 8 (NT = 1), the lanes read them
// from global memory, where they stay in L1, and each warp runs by itself.
// More of them (WIDE) are staged in shared memory beside the weights, once for
// all warps of the CTA.
//
// A CTA takes a list of units (row blocks).  Its steps, those of all its units
// one after the other, form one stream: the copies run kRingSteps - 1 steps
// ahead, over the ends of units too, so the stream does not dry up between them.

// Weight formats: bf16, or 4-bit codes with this group size.
constexpr int kFmtBf16 = 0;

constexpr int kRowWarps = 8;  // warps of a CTA
// A warp's 32 weight rows as two 16-row mma tiles; a lane sees rows g and
// g + 8 of each.  Two tiles, because an activation fragment read once then
// serves twice the weights.
constexpr int kRowTiles = 2;

// Weight rows, counted from the base pointers.
struct Rows {
  const uint8_t* data;          // bf16 values or codes
  const __nv_bfloat16* scales;  // 4 bits: scales of the rows' groups
  const uint8_t* zeros;         // 4 bits: zero points of the rows' groups (NULL: 8)
};

// Columns of a pipeline step: 16 bytes of each row a lane, 64 bytes a row.
template <int FMT>
constexpr int rowdot_step() {
  return FMT == kFmtBf16 ? 32 : 128;
}

// Each warp keeps its rows' next steps in a ring of its own (2 KB a step),
// filled by 16-byte asynchronous copies: the copies need no registers, so
// enough bytes are in flight with few warps.  Behind it (4 bits) lie the
// decoded scales and zero points of the warp's 32 rows, two steps of them.
constexpr int kRingSteps = 4;
constexpr int kStepBytes = kRowTiles * 2 * 512;
template <int FMT>
constexpr int scale_slot_bytes() {
  return FMT == kFmtBf16 ? 0 : 256 * (128 / (FMT == kFmtBf16 ? 128 : FMT));
}
template <int FMT>
constexpr int ring_bytes() {
  return kRingSteps * kStepBytes + 2 * scale_slot_bytes<FMT>();
}
// Staged activations of one slice of K (WIDE): 16-byte pieces in the order the
// lanes take them, [kRingSteps][pieces a lane][NT][32 lanes].
template <int FMT, int NT>
constexpr int x_step_bytes() {
  return (FMT == kFmtBf16 ? 1 : 4) * NT * 512;
}
template <int FMT, int NT>
constexpr int x_ring_bytes() {
  return NT > 1 ? kRingSteps * x_step_bytes<FMT, NT>() : 0;
}
// Where the warps of one row block leave their sums to be joined.
template <int NT>
constexpr int join_bytes() {
  return kRowTiles * NT * 512;
}
// Shared memory of a CTA whose warps split K WK ways.
template <int FMT, int NT>
constexpr int rowdot_smem(int WK) {
  return kRowWarps * ring_bytes<FMT>() + WK * x_ring_bytes<FMT, NT>() + (WK > 1 ? kRowWarps * join_bytes<NT>() : 0);
}

static __device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;  // 0: the slot is filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
static __device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
static __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// bf16x2 of 128 + z
static __device__ __forceinline__ uint32_t w4_zero_bits(uint32_t z) {
  const uint32_t v = z & 15u;
  return 0x43004300u | v | (v << 16);
}

// Scales (and zero points) of one row's groups in a step of 128 columns, packed
// as they lie in memory.
struct W4Scales {
  uint2 s;
  uint32_t z;
};

template <int FMT>
static __device__ __forceinline__ W4Scales ld_scales(const __nv_bfloat16* s, const uint8_t* z, int c, int groups) {
  constexpr int G = 128 / FMT;  // groups a step
  const int g0 = c * G;
  W4Scales r{make_uint2(0u, 0u), 0u};
  if (G == 1 || groups % G == 0) {  // every row's scales start on a boundary of the vector
    if constexpr (G == 4) r.s = *reinterpret_cast<const uint2*>(s + g0);
    else if constexpr (G == 2) r.s.x = *reinterpret_cast<const uint32_t*>(s + g0);
    else r.s.x = *reinterpret_cast<const uint16_t*>(s + g0);
    if (z) {
      if constexpr (G == 4) r.z = *reinterpret_cast<const uint32_t*>(z + g0);
      else if constexpr (G == 2) r.z = *reinterpret_cast<const uint16_t*>(z + g0);
      else r.z = z[g0];
    }
  } else {
    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (g0 + i < groups) {
        v[i] = *reinterpret_cast<const uint16_t*>(s + g0 + i);
        if (z) r.z |= static_cast<uint32_t>(z[g0 + i]) << (8 * i);
      }
    r.s = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
  }
  return r;
}

// The products of a CTA's units.  `work` says what they are:
//   int units()                      how many this CTA has
//   Rows rows(u)                     base of the weight rows of unit u
//   int row(u, rg, lane, &active)    index of row `lane` of warp group rg's 32 rows; a valid
//                                    one even where the group has none (active = false)
//   int count(u)                     activation rows, 1 to 8*NT
//   const bf16* xrow(u, i)           activation row i < count(u)
//   void finish(u, rg, acc)          takes the sums: thread (g, t) has acc[m][n] = (row g of
//                                    tile m, columns 8n + 2t, 8n + 2t + 1; row g + 8, the same)
// WK warps share a row block, each with a slice of K.  smem: rowdot_smem.
template <int FMT, int NT, typename Work>
static __device__ __forceinline__ void row_stream(const Work& work, int K, int WK, uint8_t* smem) {
  constexpr bool WIDE = NT > 1;
  constexpr bool W4 = FMT != kFmtBf16;
  constexpr int kStep = rowdot_step<FMT>();
  constexpr int G = W4 ? 128 / (W4 ? FMT : 1) : 1;  // groups a step
  constexpr int W = W4 ? FMT / 32 : 1;              // pieces of 8 columns a lane takes from a group
  constexpr int kPieces = kStep / 8;                // of an activation row in a step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk = warp % WK, rg = warp / WK;
  uint8_t* ring = smem + warp * ring_bytes<FMT>();
  uint8_t* scale_ring = ring + kRingSteps * kStepBytes;
  uint8_t* xring = smem + kRowWarps * ring_bytes<FMT>() + wk * x_ring_bytes<FMT, NT>();
  uint8_t* joins = smem + kRowWarps * ring_bytes<FMT>() + WK * x_ring_bytes<FMT, NT>();
  const int ix = rg * 32 + lane, nx = 32 * (kRowWarps / WK);  // this thread's place among its slice's
  const int units = work.units();
  const int all = (K + kStep - 1) / kStep;
  const int steps = (all + WK - 1) / WK;  // of a slice; some have one less
  const int c0 = all * wk / WK, c1 = all * (wk + 1) / WK;
  // a row's 64 bytes of a step, its 16-byte pieces swizzled by the row so that
  // reads of one piece, half piece or word a lane all spread over the banks
  const int swz = (g >> 1) & 3;
  const uint32_t mine = smem_u32(ring) + g * 64 + ((t ^ swz) * 16);
  const uint32_t stride = W4 ? K / 2u : 2u * K;
  const int groups = W4 ? K / (W4 ? FMT : 1) : 0;

  // the copies' place in the stream
  int fu = 0, fc = c0, fend = c0 + steps, fslot = 0, fcount = 0;
  bool factive = false;
  const uint8_t* src[2 * kRowTiles];
  const __nv_bfloat16* fscale = nullptr;
  const uint8_t* fzero = nullptr;
  W4Scales sc0{make_uint2(0u, 0u), 0u}, sc1 = sc0, sc2 = sc0;  // of the next three steps
  auto fill_unit = [&](int u) {
    const Rows r = work.rows(u);
    const int my_row = work.row(u, rg, lane, factive);
#pragma unroll
    for (int i = 0; i < 2 * kRowTiles; ++i)
      src[i] = r.data + static_cast<uint64_t>(stride) * __shfl_sync(0xffffffffu, my_row, 8 * i + g) + 16 * t +
               static_cast<int64_t>(c0) * 64;
    if constexpr (W4) {
      fscale = r.scales + static_cast<int64_t>(groups) * my_row;
      fzero = r.zeros ? r.zeros + static_cast<int64_t>(groups) * my_row : nullptr;
    }
    if constexpr (WIDE) fcount = work.count(u);
  };
  auto fill = [&]() {
    if (fu < units) {
      const bool in = factive && fc < c1 && fc * kStep + (kStep / 4) * t < K;
      const uint32_t dst = mine + fslot * kStepBytes;
#pragma unroll
      for (int i = 0; i < 2 * kRowTiles; ++i) {
        cp_async16(dst + i * 512, src[i], in);
        src[i] += 64;
      }
      if constexpr (WIDE) {
        const uint32_t xdst = smem_u32(xring) + fslot * x_step_bytes<FMT, NT>();
        const int pieces = (fcount + 7) / 8 * 8 * kPieces;
        for (int i = ix; i < pieces; i += nx) {
          const int row = i / kPieces, p = i % kPieces, k = fc * kStep + 8 * p;
          // where the lane that takes piece p of this row finds it
          const int j = W4 ? (p / (4 * W)) * W + p % W : 0;
          const int to = ((j * NT + row / 8) * 32 + (row % 8) * 4 + (p / W) % 4) * 16;
          const bool xin = fc < c1 && k < K && row < fcount;
          cp_async16(xdst + to, work.xrow(fu, xin ? row : 0) + (xin ? k : 0), xin);
        }
      }
      if constexpr (W4) {
        sc0 = sc1;
        sc1 = sc2;
        if (fc < c1) sc2 = ld_scales<FMT>(fscale, fzero, fc, groups);
        if (!fzero) sc2.z = 0x08080808u;
      }
      if (++fc == fend) {
        fc = c0;
        if (++fu < units) fill_unit(fu);
      }
    } else if constexpr (W4) {
      sc0 = sc1;
      sc1 = sc2;
    }
    cp_async_commit();
    fslot = fslot == kRingSteps - 1 ? 0 : fslot + 1;
  };
  // the order (0,4) (1,5) | (2,6) (3,7) that the codes come in
  auto as_codes = [](uint4 v) {
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
  };

  if (units > 0) fill_unit(0);
#pragma unroll
  for (int i = 0; i < kRingSteps - 1; ++i) fill();

  int slot = 0, parity = 0;
#pragma unroll 1
  for (int u = 0; u < units; ++u) {
    bool active;
    work.row(u, rg, lane, active);
    const int count = work.count(u), nt = (count + 7) >> 3;
    // a lane without an activation row reads the last one: its column is not used
    const __nv_bfloat16* xr = WIDE ? nullptr : work.xrow(u, min(g, count - 1));
    float acc[kRowTiles][NT][4];
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

#pragma unroll 1
    for (int c = c0; c < c0 + steps; ++c) {
      cp_async_wait<kRingSteps - 2>();
      uint8_t* sc = scale_ring + parity * scale_slot_bytes<FMT>();
      parity ^= 1;
      if constexpr (W4) {
        // {bf16x2 of 128 + z, scale} of row `lane`, [G][32]
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const uint32_t two = q < 2 ? sc0.s.x : sc0.s.y;
          const uint32_t sbits = q & 1 ? two & 0xffff0000u : two << 16;
          *reinterpret_cast<uint2*>(sc + (q * 32 + lane) * 8) = make_uint2(w4_zero_bits(sc0.z >> (8 * q)), sbits);
        }
      }
      if constexpr (WIDE) {
        if constexpr (W4) {  // each thread reorders the pieces it copied itself
          uint8_t* xs = xring + slot * x_step_bytes<FMT, NT>();
          for (int i = ix; i < nt * 8 * kPieces; i += nx) {
            const int row = i / kPieces, p = i % kPieces;
            const int j = (p / (4 * W)) * W + p % W;
            uint4* at = reinterpret_cast<uint4*>(xs + ((j * NT + row / 8) * 32 + (row % 8) * 4 + (p / W) % 4) * 16);
            *at = as_codes(*at);
          }
        }
        __syncthreads();
      } else {
        __syncwarp();
      }
      fill();  // into the slot of the step before this one: its readers have passed the barrier
      if (active && c < c1) {
        const uint8_t* rows = ring + slot * kStepBytes + g * 64;
        const uint8_t* xs = xring + slot * x_step_bytes<FMT, NT>() + lane * 16;
        if constexpr (!W4) {
          uint4 b[NT];
          const int k = c * 32 + 8 * t;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (WIDE) {
              if (n < nt) b[n] = *reinterpret_cast<const uint4*>(xs + n * 512);
            } else {
              b[n] = make_uint4(0u, 0u, 0u, 0u);
              if (k < K) b[n] = *reinterpret_cast<const uint4*>(xr + k);
            }
          }
#pragma unroll
          for (int m = 0; m < kRowTiles; ++m) {
            const uint4 lo = *reinterpret_cast<const uint4*>(rows + (t ^ swz) * 16 + m * 1024);
            const uint4 hi = *reinterpret_cast<const uint4*>(rows + (t ^ swz) * 16 + m * 1024 + 512);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (n < nt) {
                mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, b[n].x, b[n].y);
                mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, b[n].z, b[n].w);
              }
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < G; ++q) {
            if (G > 1 && c * 128 + q * FMT >= K) break;  // a group is whole or absent
            const int k0 = c * 128 + q * FMT + 8 * W * t;
            // this lane's words of the group: piece and offset within the row's 64 bytes
            const int piece = FMT == 128 ? t : FMT == 64 ? 2 * q + (t >> 1) : q;
            const int off = FMT == 128 ? 0 : FMT == 64 ? 8 * (t & 1) : 4 * t;
            const uint8_t* at = rows + ((piece ^ swz) * 16) + off;
            // one row tile at a time where both would not fit the registers
            constexpr int kTogether = NT == 4 ? 1 : kRowTiles;
#pragma unroll
            for (int m0 = 0; m0 < kRowTiles; m0 += kTogether) {
              float part[kTogether][NT][4];
              uint32_t code[2 * kTogether][W];
              uint2 zs[2 * kTogether];
#pragma unroll
              for (int i = 0; i < 2 * kTogether; ++i) {
                const uint8_t* from = at + (2 * m0 + i) * 512;
                if constexpr (W == 4) *reinterpret_cast<uint4*>(code[i]) = *reinterpret_cast<const uint4*>(from);
                else if constexpr (W == 2) *reinterpret_cast<uint2*>(code[i]) = *reinterpret_cast<const uint2*>(from);
                else code[i][0] = *reinterpret_cast<const uint32_t*>(from);
                zs[i] = *reinterpret_cast<const uint2*>(sc + (q * 32 + 8 * (2 * m0 + i) + g) * 8);
              }
#pragma unroll
              for (int m = 0; m < kTogether; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int i = 0; i < 4; ++i) part[m][n][i] = 0.0f;
#pragma unroll
              for (int j = 0; j < W; ++j) {
                uint4 b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  if constexpr (WIDE) {
                    if (n < nt) b[n] = *reinterpret_cast<const uint4*>(xs + ((q * W + j) * NT + n) * 512);
                  } else {
                    b[n] = as_codes(*reinterpret_cast<const uint4*>(xr + k0 + 8 * j));
                  }
                }
#pragma unroll
                for (int m = 0; m < kTogether; ++m) {
                  uint32_t al[4], ah[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    al[i] = w4_pair(code[2 * m][j], i, zs[2 * m].x);
                    ah[i] = w4_pair(code[2 * m + 1][j], i, zs[2 * m + 1].x);
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    if (n < nt) {
                      mma_bf16(part[m][n], al[0], ah[0], al[1], ah[1], b[n].x, b[n].y);
                      mma_bf16(part[m][n], al[2], ah[2], al[3], ah[3], b[n].z, b[n].w);
                    }
                  }
                }
              }
#pragma unroll
              for (int m = 0; m < kTogether; ++m) {
                const float sl = __uint_as_float(zs[2 * m].y), sh = __uint_as_float(zs[2 * m + 1].y);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float(&to)[4] = acc[m0 + m][n];
                  to[0] = fmaf(sl, part[m][n][0], to[0]);
                  to[1] = fmaf(sl, part[m][n][1], to[1]);
                  to[2] = fmaf(sh, part[m][n][2], to[2]);
                  to[3] = fmaf(sh, part[m][n][3], to[3]);
                }
              }
            }
          }
        }
      }
      slot = slot == kRingSteps - 1 ? 0 : slot + 1;
    }

    if (WK > 1) {  // join the slices in a fixed order
      uint8_t* mine_j = joins + warp * join_bytes<NT>() + lane * 16;
      __syncthreads();  // the last unit's sums have been read
      if (wk != 0) {
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < nt)
              *reinterpret_cast<float4*>(mine_j + (m * NT + n) * 512) =
                  make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      }
      __syncthreads();
      if (wk == 0) {
        for (int s = 1; s < WK; ++s) {
#pragma unroll
          for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n < nt) {
                const float4 v = *reinterpret_cast<const float4*>(mine_j + s * join_bytes<NT>() + (m * NT + n) * 512);
                acc[m][n][0] += v.x;
                acc[m][n][1] += v.y;
                acc[m][n][2] += v.z;
                acc[m][n][3] += v.w;
              }
        }
      }
    }
    if (wk == 0 && active) work.finish(u, rg, acc);
  }
  cp_async_wait<0>();
}

// How many ways to split K over a CTA's warps: the split with the least time,
// counting a CTA's rounds over its units times the steps of a unit's slice,
// and two steps' worth for ending a unit (three where its slices are joined).
// blocks: 32-row blocks; slots: CTAs that run at a time.
static inline int rowdot_split(int64_t blocks_per_entry, int64_t entries, int steps, int most, int64_t slots) {
  int best = 1;
  int64_t least = 0;
  for (int WK = 1; WK <= most && (WK == 1 || steps >= 2 * WK); WK *= 2) {
    const int64_t units = entries * ((blocks_per_entry * WK + kRowWarps - 1) / kRowWarps);
    const int64_t rounds = (units + slots - 1) / slots;
    const int64_t cost = rounds * ((steps + WK - 1) / WK + (WK == 1 ? 2 : 3));
    if (WK == 1 || cost < least) {
      least = cost;
      best = WK;
    }
  }
  return best;
}

}  // namespace dg
