// Products of weight rows with a few activation rows: the core of the few-token
// operators (4-bit linear, routed SwiGLU experts).
//
//   acc[r, n] = sum_k w[r, k] * x[n, k]      32 weight rows a warp, 8*NT activation rows
//
// With few activation rows the weights are the traffic, so each weight is read
// from HBM once and meets all activation rows in the registers of one warp:
// mma.sync m16n8k16 takes the weight fragment as it was loaded (or decoded).
//
// The contraction index of an mma is only a label, the same on both operands,
// so lane (g, t) = (lane / 4, lane % 4) of a warp owns CONSECUTIVE columns of
// weight rows g and g + 8 and of activation row g, takes them as one wide
// vector and feeds them to consecutive mma steps.
//
// This file: what both weight formats share, and the bf16 form.  dg_w4dot.cuh:
// the 4-bit form.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_ptx.cuh"

namespace dg {

constexpr int kRowWarps = 8;  // warps of a CTA
// A warp's 32 weight rows as two 16-row mma tiles; a lane sees rows g and
// g + 8 of each.  Two tiles, because an activation fragment read once then
// serves twice the weights.  Row 8 * i + g of the 32 is called row i of the lane.
constexpr int kRowTiles = 2;
constexpr int kLaneRows = 2 * kRowTiles;

template <int NT>
using RowSums = float[kRowTiles][NT][4];

// Where the warps of one row block leave their sums to be joined: a warp, and
// all of a CTA whose warps split K WK ways (the first warp of a block keeps its own).
template <int NT>
constexpr int join_bytes() {
  return kRowTiles * NT * 512;
}
template <int NT>
constexpr int joins_bytes(int WK) {
  return (kRowWarps - kRowWarps / WK) * join_bytes<NT>();
}

// Joins the sums of the WK warps that share a row block, in a fixed order, into
// the one with wk = 0.  All warps of the CTA.
template <int NT>
static __device__ __forceinline__ void join_slices(RowSums<NT>& acc, uint8_t* joins, int rg, int wk, int WK) {
  // slice s >= 1 of row block rg
  auto place = [&](int s) { return joins + (rg * (WK - 1) + s - 1) * join_bytes<NT>() + (threadIdx.x & 31) * 16; };
  __syncthreads();  // the last unit's sums have been read
  if (wk != 0) {
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float4*>(place(wk) + (m * NT + n) * 512) =
            make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
  }
  __syncthreads();
  if (wk != 0) return;
  for (int s = 1; s < WK; ++s) {
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 v = *reinterpret_cast<const float4*>(place(s) + (m * NT + n) * 512);
        acc[m][n][0] += v.x;
        acc[m][n][1] += v.y;
        acc[m][n][2] += v.z;
        acc[m][n][3] += v.w;
      }
  }
}

// Joins the sums of a cluster's CTAs, which took slices of K of the same rows, in the
// order of their ranks, into those of rank 0.  place: the warp's join_bytes, the same
// in every CTA; holds: the warp has sums.  All threads of the cluster.
template <int NT>
static __device__ __forceinline__ void join_cluster(RowSums<NT>& acc, uint8_t* place, bool holds, int ctas) {
  const uint32_t at = smem_u32(place) + (threadIdx.x & 31) * 16, rank = cluster_ctarank();
  if (holds && rank != 0) {
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float4*>(place + (threadIdx.x & 31) * 16 + (m * NT + n) * 512) =
            make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
  }
  cluster_sync_all();
  if (holds && rank == 0) {
    for (int r = 1; r < ctas; ++r) {
      const uint32_t from = mapa_shared(at, r);
#pragma unroll
      for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 v = ld_cluster_f32x4(from + (m * NT + n) * 512);
          acc[m][n][0] += v.x;
          acc[m][n][1] += v.y;
          acc[m][n][2] += v.z;
          acc[m][n][3] += v.w;
        }
    }
  }
  cluster_sync_all();  // a CTA's shared memory outlives the reads
}

template <int NT>
static __device__ __forceinline__ void clear(RowSums<NT>& acc) {
#pragma unroll
  for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
}

// How many ways to split K over a CTA's warps (up to `most`), and further over the
// CTAs of a cluster (up to `clusters` of them, whose join costs as much as
// `join_steps` steps): the split with the least time.  It counts the units that fall
// to an SM times the steps of a unit's slice (and one for ending the unit), over the
// rate of an SM with that many CTAs at a time.
// The CTAs of an SM share its pipes, so it is SMs that have to come out even.
static inline int rowdot_split(int64_t blocks_per_entry, int64_t entries, int steps, int ctas, int most,
                               int num_sms, int clusters = 1, int join_steps = 0) {
  // measured on the 4-bit products: of the rate with 24 warps, 8 warps reach about half, 16 about 85%
  constexpr int kRate[4] = {0, 50, 85, 100};
  int best = 1;
  double least = 0.0;
  for (int WK = 1; WK <= most * clusters && (WK == 1 || steps >= 2 * WK); WK *= 2) {
    const int64_t units = entries * ((blocks_per_entry * WK + kRowWarps - 1) / kRowWarps);
    const int64_t rounds = (units + num_sms - 1) / num_sms;
    const int at_a_time = static_cast<int>(rounds < ctas ? rounds : ctas);
    const double cost = static_cast<double>(rounds) * ((steps + WK - 1) / WK + 1 + (WK > most ? join_steps : 0)) /
                        kRate[at_a_time];
    if (WK == 1 || cost < least) {
      least = cost;
      best = WK;
    }
  }
  return best;
}

// ---------------------------------------------------------------- bf16 weights
//
// A step is 32 columns, 8 of them (16 bytes) a lane: two mma a tile.  Each warp
// keeps kBfRing steps of its rows on the way from HBM in a ring of its own (2 KB
// a step), filled by 16-byte asynchronous copies that need no registers; a lane
// reads back what it alone has copied.  Activation rows come in two ways.  Up to
// 8 (NT = 1), the lanes read them from global memory, where they stay in L1, and
// each warp runs by itself.  More of them are staged in shared memory beside the
// weights, once for all warps of the CTA that work on the same slice of K.
//
// Bound by the weights' bytes, which it moves at 0.62 to 0.89 of the measured copy rate:
// the more steps a unit has and the more units an SM, the nearer.  (Weights loaded to
// registers, without the ring: 77.6 us where this takes 67 to 71, one token and 8 experts
// of 3 x 4096 x 1792; 700 where this takes 468 to 504, 128 tokens and 64 experts.)

constexpr int kBfRing = 4;
constexpr int kBfStep = 32;
constexpr int kBfStepBytes = kLaneRows * 512;

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

// Staged activations of one slice of K: 16-byte pieces in the order the lanes
// take them, [kBfRing][NT][32 lanes].
template <int NT>
constexpr int bf_x_bytes() {
  return NT > 1 ? kBfRing * NT * 512 : 0;
}
// Shared memory of a CTA whose warps split K WK ways.
template <int NT>
constexpr int bf_smem(int WK) {
  return kRowWarps * kBfRing * kBfStepBytes + WK * bf_x_bytes<NT>() + joins_bytes<NT>(WK);
}

// acc += steps [c0, c1) of the product of a warp's 32 rows with up to 8*NT
// activation rows.  rows[i]: the lane's row i, plus 16 t bytes.  xrow(i): pointer
// to activation row i, for i < count.  Thread (g, t) ends with acc[m][n] =
// (row g of tile m, columns 8n + 2t, 8n + 2t + 1; row g + 8, the same).
//   ring   this warp's kBfRing * kBfStepBytes
//   xring  NT > 1: the bf_x_bytes of this warp's slice of K, filled by the `nx`
//          threads of the slice, of which this is number `ix`; all warps of the
//          CTA call together with the same `steps` >= c1 - c0, also those without
//          rows (active = false)
template <int NT, typename XRow>
static __device__ __forceinline__ void row_dot_bf16(const uint8_t* const (&rows)[kLaneRows], bool active, XRow xrow,
                                                    int count, int K, int c0, int c1, int steps, RowSums<NT>& acc,
                                                    uint8_t* ring, uint8_t* xring, int ix, int nx) {
  constexpr bool WIDE = NT > 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (!WIDE && !active) return;
  // a lane without an activation row reads the last one: its column is not used
  const __nv_bfloat16* xr = WIDE ? nullptr : xrow(min(g, count - 1)) + 8 * t;
  uint8_t* own = ring + lane * 16;
  auto fill = [&](int c, int slot) {
    const bool in = active && c < c1 && c * kBfStep + 8 * t < K;
    const uint32_t dst = smem_u32(own) + slot * kBfStepBytes;
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) cp_async16(dst + i * 512, rows[i] + (in ? c * 64 : 0), in);
    if constexpr (WIDE) {
      const uint32_t xdst = smem_u32(xring) + slot * NT * 512;
      for (int i = ix; i < 32 * NT; i += nx) {
        const int row = i / 4, k = c * kBfStep + 8 * (i % 4);
        const bool xin = c < c1 && k < K && row < count;
        cp_async16(xdst + i * 16, xrow(xin ? row : 0) + (xin ? k : 0), xin);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int u = 0; u < kBfRing - 1; ++u) fill(c0 + u, u);
  const int end = WIDE ? steps : c1 - c0;
#pragma unroll 1
  for (int s0 = 0; s0 < end; s0 += kBfRing) {
#pragma unroll
    for (int u = 0; u < kBfRing; ++u) {
      const int c = c0 + s0 + u;
      if (s0 + u >= end) break;
      uint4 b[NT];
      if constexpr (!WIDE) {
        b[0] = make_uint4(0u, 0u, 0u, 0u);
        if (c * kBfStep + 8 * t < K) b[0] = *reinterpret_cast<const uint4*>(xr + c * kBfStep);
      }
      cp_async_wait<kBfRing - 2>();
      if constexpr (WIDE) {
        __syncthreads();  // the staged rows are in place; the slot of the step before is free
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[n] = *reinterpret_cast<const uint4*>(xring + (u * NT + n) * 512 + lane * 16);
      }
#pragma unroll
      for (int m = 0; m < kRowTiles; ++m) {
        const uint4 lo = *reinterpret_cast<const uint4*>(own + u * kBfStepBytes + m * 1024);
        const uint4 hi = *reinterpret_cast<const uint4*>(own + u * kBfStepBytes + m * 1024 + 512);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, b[n].x, b[n].y);
          mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, b[n].z, b[n].w);
        }
      }
      // the slot that the step before this one has read
      fill(c + kBfRing - 1, (u + kBfRing - 1) % kBfRing);
    }
  }
  cp_async_wait<0>();
  if constexpr (WIDE) __syncthreads();  // the staged rows may be replaced
}

}  // namespace dg
