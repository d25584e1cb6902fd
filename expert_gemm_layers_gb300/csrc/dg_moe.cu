// Routed experts for few tokens: the router (logits, top-k, gates) and the
// SwiGLU experts' products on bf16 or 4-bit weights.
//
//   e_j = idx[t, j], h_j = silu(w1[e_j] x_t) * (w3[e_j] x_t),
//   y_t = sum_j gates[t, j] * (w2[e_j] h_j)
//
// With few tokens the experts' weights are the traffic: every touched expert's
// rows are read once and meet all of its tokens in registers (dg_rowdot.cuh).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "dg_internal.h"
#include "dg_w4dot.cuh"

namespace dg {

namespace {

__device__ __forceinline__ bool err_set(const uint32_t* err) { return ld_volatile_u32(err) != 0u; }

// ---------------------------------------------------------------- router

// Two binary32 numbers at a time (packed arithmetic: half the instructions).
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) {
  Pair r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// s + p: s becomes the rounded sum, and what that lost, which is found without error
// (Knuth's two-sum), is added to c, which rounds.
__device__ __forceinline__ void two_sum(Pair& s, Pair& c, Pair p) {
  const Pair t = s + p, z = t - s;
  c = c + ((s - (t - z)) + (p - z));
  s = t;
}
__device__ __forceinline__ void two_sum(float& s, float& c, float p) {
  const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
  s = t;
}

constexpr int kLogitWarps = 8;
constexpr int kLogitTokens = 4;
constexpr int kLogitExperts = 2;
constexpr int kLogitSpread = 12;

// logits[t, e]: a warp takes kLogitExperts experts and kLogitTokens tokens, and one
// of KS slices of d (KS > 1 where there are too few of both to fill the GPU).  The
// choice of experts hangs on the order of the logits, so the sums are kept in two
// words (a bf16 product is exact in binary32, two_sum keeps what a sum loses) and rounded
// to binary32 once.  A lane adds d / 64 products to a sum, so its second word is at most
// d / 64 * 2^-24 of sum |x w| and off by at most the square of that.
// Bound by that arithmetic: 8 operations a product, 384 x 4096 on 128 experts: 62 us, 43
// at the FP32 pipes' peak (0.6 by bytes).  2 x 4 products a step, because each operand
// is then unpacked for 2 or 4 of them; asking for a step's columns a step ahead took
// 4 us more (registers).  One token: 2 us beyond an empty kernel's time.
template <int KS>
__global__ void __launch_bounds__(kLogitWarps * 32)
    moe_logits_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wr,
                      float* __restrict__ logits, int T, int d, int E, const uint32_t* err) {
  __shared__ float2 slices[KS > 1 ? kLogitWarps : 1][kLogitExperts * kLogitTokens];
  griddep_wait();
  if (err_set(err)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = (static_cast<int>(blockIdx.x) * (kLogitWarps / KS) + warp / KS) * kLogitExperts;
  const int t0 = static_cast<int>(blockIdx.y) * kLogitTokens;
  Pair s[kLogitExperts][kLogitTokens], c[kLogitExperts][kLogitTokens];
#pragma unroll
  for (int j = 0; j < kLogitExperts; ++j)
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) s[j][i] = c[j][i] = pair_of(0.0f, 0.0f);
  // rows past the last one read the last one and are not stored
  const __nv_bfloat16 *wp[kLogitExperts], *xp[kLogitTokens];
#pragma unroll
  for (int j = 0; j < kLogitExperts; ++j) wp[j] = wr + static_cast<int64_t>(min(e0 + j, E - 1)) * d;
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) xp[i] = x + static_cast<int64_t>(min(t0 + i, T - 1)) * d;
  const int tokens = min(T - t0, kLogitTokens);
  auto products = [&](auto full) {  // without branches where all tokens are there
    constexpr bool kFull = decltype(full)::value;
#pragma unroll 2
    for (int k = 8 * (lane + 32 * (warp % KS)); k < d; k += 256 * KS) {
      uint4 wv[kLogitExperts], xv[kLogitTokens];
#pragma unroll
      for (int j = 0; j < kLogitExperts; ++j) wv[j] = *reinterpret_cast<const uint4*>(wp[j] + k);
#pragma unroll
      for (int i = 0; i < kLogitTokens; ++i)
        if (kFull || i < tokens) xv[i] = *reinterpret_cast<const uint4*>(xp[i] + k);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        auto two = [&](const uint4& v) {
          const uint32_t u = q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
          return pair_of(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        };
        Pair wq[kLogitExperts];
#pragma unroll
        for (int j = 0; j < kLogitExperts; ++j) wq[j] = two(wv[j]);
#pragma unroll
        for (int i = 0; i < kLogitTokens; ++i) {
          if (kFull || i < tokens) {
            const Pair xq = two(xv[i]);
#pragma unroll
            for (int j = 0; j < kLogitExperts; ++j) two_sum(s[j][i], c[j][i], wq[j] * xq);
          }
        }
      }
    }
  };
  if (e0 < E) {
    if (tokens == kLogitTokens) products(std::true_type{});
    else products(std::false_type{});
  }
  griddep_launch_dependents();  // not before: waiting CTAs beside these took up to 10 us more
#pragma unroll
  for (int j = 0; j < kLogitExperts; ++j)
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
      if (i >= tokens) continue;
      const float2 s2 = floats_of(s[j][i]), c2 = floats_of(c[j][i]);
      float sum = s2.x, low = c2.x + c2.y;
      two_sum(sum, low, s2.y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float so = __shfl_xor_sync(0xffffffffu, sum, o), lo = __shfl_xor_sync(0xffffffffu, low, o);
        two_sum(sum, low, so);
        low += lo;
      }
      if constexpr (KS > 1) {
        if (lane == 0) slices[warp][j * kLogitTokens + i] = make_float2(sum, low);
      } else if (lane == 0 && e0 + j < E) {
        // an overflowed or non-finite sum makes its correction NaN: keep the sum itself
        logits[static_cast<int64_t>(t0 + i) * E + e0 + j] = isfinite(sum) ? sum + low : sum;
      }
    }
  if constexpr (KS > 1) {
    __syncthreads();
    const int v = lane, j = v / kLogitTokens, i = v % kLogitTokens;
    if (warp % KS == 0 && v < kLogitExperts * kLogitTokens && e0 + j < E && i < tokens) {
      float sum = slices[warp][v].x, low = slices[warp][v].y;
      for (int k = 1; k < KS; ++k) {
        two_sum(sum, low, slices[warp + k][v].x);
        low += slices[warp + k][v].y;
      }
      logits[static_cast<int64_t>(t0 + i) * E + e0 + j] = isfinite(sum) ? sum + low : sum;
    }
  }
}

// Order of the choice as an unsigned key: larger logit first, NaN behind every
// number; the smaller index wins among equals.
__device__ __forceinline__ uint64_t rank_key(float l, int e) {
  uint32_t u = __float_as_uint(l);
  if (l == 0.0f) u = 0u;  // -0 and +0 are equal
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if (isnan(l)) u = 0u;
  return (static_cast<uint64_t>(u) << 32) | (0xffffffffu - static_cast<uint32_t>(e));
}

constexpr int kTopkWarps = 4;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;

// One warp per token: k times the largest remaining key, then the gates.  384 tokens, 6
// of 128: 2 us beyond an empty kernel's time, the latency of 6 rounds of shuffles.
__global__ void __launch_bounds__(kTopkWarps * 32)
    moe_topk_kernel(const float* __restrict__ logits, int32_t* __restrict__ idx, float* __restrict__ gates, int T,
                    int E, int k, bool sigmoid, bool renorm, float scale, const uint32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * kTopkWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* l = logits + static_cast<int64_t>(t) * E;
  uint64_t last = ~0ull;  // keys below this one are still to be chosen from
  float mine = 0.0f;      // lane j: logit of choice j
  int mine_e = 0;
  float top = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0ull;
    for (int e = lane; e < E; e += 32) {
      const uint64_t key = rank_key(l[e], e);
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      if (other > best) best = other;
    }
    last = best;
    const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    const float v = l[e];
    if (j == 0) top = v;
    if (lane == j) {
      mine = v;
      mine_e = e;
    }
  }
  float bad = 0.0f;  // NaN if some logit is: then the token's gates are
  float all = 0.0f;
  for (int e = lane; e < E; e += 32) {
    const float v = l[e];
    if (isnan(v)) bad = v;
    if (!sigmoid && !renorm) all += expf(v - top);
  }
  float p = 0.0f;
  if (lane < k) {
    // A sigmoid is e^l / (1 + e^l), renormalised times e^-top where all are below 0: gates that
    // are in proportion to each other do not all vanish where 1 / (1 + e^-l) would.
    const float shift = renorm ? fminf(top, 0.0f) : 0.0f;
    if (!sigmoid) p = expf(mine - top);
    else if (mine > 0.0f) p = 1.0f / (1.0f + expf(-mine));
    else p = expf(mine - shift) / (1.0f + expf(mine));
  }
  float sum = renorm ? p : all;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (sigmoid && !renorm) sum = 1.0f;
  if (lane < k) {
    idx[static_cast<int64_t>(t) * k + lane] = mine_e;
    gates[static_cast<int64_t>(t) * k + lane] = p / sum * scale + bad;
  }
}

// ---------------------------------------------------------------- experts

constexpr int kMoeWarps = kRowWarps;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kMaxPairs = 8192;
constexpr int kFmtBf16 = 0;  // weight format: this, or the group size of 4-bit weights

// The work of a call: entries of one expert and up to `cap` of its pairs, which
// stand one after the other in pairs[].  An expert with more pairs has several
// entries.
struct PairMap {
  int* total;  // number of entries
  int* expert;
  int* start;
  int* count;
  int* pairs;
};

__host__ __device__ inline int max_entries(int npairs, int E, int cap) {
  const int active = npairs < E ? npairs : E;
  return active + npairs / cap;
}
// Ints of a PairMap.
__host__ __device__ inline int pair_map_ints(int npairs, int E, int cap) {
  return 4 + 3 * max_entries(npairs, E, cap) + npairs;
}
__host__ __device__ inline PairMap pair_map_at(int* p, int npairs, int E, int cap) {
  const int me = max_entries(npairs, E, cap);
  return PairMap{p, p + 4, p + 4 + me, p + 4 + 2 * me, p + 4 + 3 * me};
}

// Up to 32 pairs: one warp's lanes are the pairs, and every CTA does this itself
// (to the same result: entries in the order of their first pair).
__device__ __forceinline__ void build_small_map(const PairMap& m, const int32_t* idx, int npairs, int E, int cap) {
  const int lane = threadIdx.x & 31;
  int e = lane < npairs ? idx[lane] : -1;
  if (e < 0 || e >= E) e = -1;
  const uint32_t valid = __ballot_sync(0xffffffffu, e >= 0);
  const uint32_t same = __match_any_sync(0xffffffffu, e) & valid, below = (1u << lane) - 1u;
  const int rank = __popc(same & below), n = __popc(same);
  const uint32_t starters = __ballot_sync(0xffffffffu, e >= 0 && rank % cap == 0);
  int before = 0, entry = 0;
  for (uint32_t s = starters; s; s &= s - 1, ++entry) {
    const int l = __ffs(s) - 1;
    const int s_rank = __shfl_sync(0xffffffffu, rank, l), s_n = __shfl_sync(0xffffffffu, n, l);
    const int s_e = __shfl_sync(0xffffffffu, e, l);
    const int size = min(cap, s_n - s_rank);
    if (e == s_e && rank >= s_rank && rank < s_rank + size) m.pairs[before + rank - s_rank] = lane;
    if (lane == 0) {
      m.expert[entry] = s_e;
      m.start[entry] = before;
      m.count[entry] = size;
    }
    before += size;
  }
  if (lane == 0) *m.total = entry;
}

// Any number of pairs, by one CTA, entries in the order of the experts, an
// expert's pairs in theirs (the sort is stable, so that a call repeats bit for
// bit).  Warp w counts and later places the w-th run of pairs: at[w][e] is where
// its next pair of expert e goes.
__device__ __forceinline__ void build_map(const PairMap& m, int* at_all, const int32_t* __restrict__ idx, int npairs,
                                          int E, int cap) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* at = at_all + warp * E;
  const int run = (npairs + kMoeThreads - 1) / kMoeThreads * 32;  // pairs of a warp
  const int p0 = warp * run, p1 = min(p0 + run, npairs);
  for (int e = lane; e < E; e += 32) at[e] = 0;
  __syncwarp();
  for (int p = p0 + lane; p < p1; p += 32) {
    const int e = idx[p];
    if (e >= 0 && e < E) atomicAdd(&at[e], 1);
  }
  __syncthreads();
  if (warp == 0) {  // scans of the pairs and of the entries over the experts
    int pairs_before = 0, entries_before = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < E)
        for (int w = 0; w < kMoeWarps; ++w) n += at_all[w * E + e];
      const int ne = (n + cap - 1) / cap;
      int sn = n, se = ne;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, sn, o);
        const int b = __shfl_up_sync(0xffffffffu, se, o);
        if (lane >= o) {
          sn += a;
          se += b;
        }
      }
      const int start = pairs_before + sn - n;
      if (e < E) {
        int next = start;
        for (int w = 0; w < kMoeWarps; ++w) {
          const int c = at_all[w * E + e];
          at_all[w * E + e] = next;
          next += c;
        }
      }
      for (int i = 0; i < ne; ++i) {
        const int to = entries_before + se - ne + i;
        m.expert[to] = e;
        m.start[to] = start + i * cap;
        m.count[to] = min(cap, n - i * cap);
      }
      pairs_before += __shfl_sync(0xffffffffu, sn, 31);
      entries_before += __shfl_sync(0xffffffffu, se, 31);
    }
    if (lane == 0) *m.total = entries_before;
  }
  __syncthreads();
  for (int q = p0; q < p1; q += 32) {
    const int p = q + lane;
    int e = p < p1 ? idx[p] : -1;
    if (e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1u));
    const int base = e >= 0 ? at[e] : 0;
    __syncwarp();
    if (e >= 0) {
      m.pairs[base + before] = p;
      if (before == 0) at[e] = base + __popc(same);
    }
    __syncwarp();
  }
}

// Rows to stage for 4-bit products, a CTA a row: [n][K] bf16, `stride` bytes apart;
// the staged rows may lie over them.
struct StageArgs {
  const uint8_t* rows;
  Staged out;
  int64_t stride;
  int n, K;
};

template <int GROUP>
__device__ __forceinline__ void stage_rows(const StageArgs& a, int block, int blocks, uint32_t* shared_top) {
  for (int r = block; r < a.n; r += blocks)
    w4_stage_row<GROUP>(a.rows + r * a.stride, a.K, a.out.frag + r * w4_row_bytes(a.K),
                        a.out.sums + static_cast<int64_t>(r) * w4_row_sums(a.K, GROUP), a.out.factor + r, shared_top);
}

// The first launch of a call with more than 32 pairs: CTA 0 builds the map, the
// others stage the tokens (4 bits).
template <int FMT>
__global__ void __launch_bounds__(kMoeThreads)
    moe_plan_kernel(PairMap m, const int32_t* __restrict__ idx, int npairs, int E, int cap, StageArgs x,
                    const uint32_t* err) {
  extern __shared__ __align__(16) int at_all[];
  __shared__ uint32_t top;
  if (threadIdx.x == 0) top = 0u;
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  __syncthreads();
  if (blockIdx.x == 0) {
    build_map(m, at_all, idx, npairs, E, cap);
    return;
  }
  if constexpr (FMT != kFmtBf16)
    stage_rows<FMT>(x, static_cast<int>(blockIdx.x) - 1, static_cast<int>(gridDim.x) - 1, &top);
}

// Stages the hidden rows between the two products (4 bits).
template <int GROUP>
__global__ void __launch_bounds__(kMoeThreads) moe_stage_kernel(StageArgs h, const uint32_t* err) {
  __shared__ uint32_t top;
  if (threadIdx.x == 0) top = 0u;
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  __syncthreads();
  stage_rows<GROUP>(h, blockIdx.x, gridDim.x, &top);
}

// pair / k as a product: kinv = 2^18 / k + 1 is exact for pairs below 2^13 and k up to 2^5.
static_assert(kMaxPairs <= 8192 && kMaxTopk <= 32, "token_of");
inline uint32_t token_factor(int k) { return (1u << 18) / static_cast<uint32_t>(k) + 1u; }
__device__ __forceinline__ int token_of(uint32_t pair, uint32_t kinv) { return static_cast<int>((pair * kinv) >> 18); }

// The operands of one product.  UP: w13 on the tokens, else w2 on the hidden rows.
struct ProductArgs {
  const uint8_t* weights;       // [E, rows, K] bf16, or codes [E, rows, K/2]
  const __nv_bfloat16* scales;  // 4 bits: [E, rows, K/group]
  const uint8_t* zeros;
  const uint8_t* in;    // activation rows, bf16, `in_stride` bytes apart
  Staged staged;        // 4 bits, not LOCAL: the same, staged
  const int32_t* idx;
  const float* gates;
  uint8_t* out;  // UP: h, `out_stride` bytes a pair; else partial rows, binary32
  PairMap map;   // not LOCAL
  int64_t in_stride, out_stride;
  int npairs, E, F, d, cap, WK;
  uint32_t kinv;
};

// A warp's sums to memory.
//   UP    its two row tiles are 16 rows of w1 and the same 16 of w3, so a and b of one
//         (pair, f) meet in one thread: h[pair, f] = bf16(silu(a) * b).  h is rounded
//         to bf16 once: it is the next product's matrix operand.  (In 4 bits, where the
//         operand is scaled fp16, too: the scratch stays 2 bytes a value and the hidden
//         rows are those of the bf16 form, off by 2^-8 of each at most, beside weights of 4 bits.)
//   else  32 rows of w2: part[pair, r] = gate * (w2[e, r] . h[pair])
template <int NT, bool UP>
__device__ __forceinline__ void store_block(const ProductArgs& a, const int* pairs, int count, int b,
                                            const RowSums<NT>& acc) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 8 * n + 2 * t + (i & 1), r = g + (i >> 1) * 8;
      if (c >= count) continue;
      const int64_t p = pairs[c];
      if (UP) {
        const int f = b * 16 + r;
        const float u = acc[0][n][i], v = acc[1][n][i], h = u / (1.0f + expf(-u)) * v;
        if (f < a.F) reinterpret_cast<__nv_bfloat16*>(a.out + p * a.out_stride)[f] = __float2bfloat16_rn(h);
      } else {
        const float gate = a.gates[p];
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m) {
          const int row = b * 32 + 16 * m + r;
          if (row < a.d) reinterpret_cast<float*>(a.out + p * a.out_stride)[row] = gate * acc[m][n][i];
        }
      }
    }
}

// One unit: block `b` (16 rows of F, or 32 of d) of an entry's expert for a warp,
// its `count` pairs as columns.
template <int FMT, int NT, bool UP, bool LOCAL, bool AHEAD>
__device__ __forceinline__ void moe_unit(const ProductArgs& a, int e, const int* pairs, int count, int b, int rg,
                                         int wk, uint8_t* smem, bool failed) {
  const int lane = threadIdx.x & 31, g = lane >> 2, warp = threadIdx.x >> 5;
  const int K = UP ? a.d : a.F, rows = UP ? 2 * a.F : a.d, WK = a.WK;
  const bool active = UP ? b * 16 < a.F : b * 32 < a.d;
  // row i of the warp's 32; rows past the last one read the last one and store nothing
  auto row = [&](int i) {
    if (!UP) return min(b * 32 + i, a.d - 1);
    const int f = min(b * 16 + (i & 15), a.F - 1);
    return i < 16 ? f : a.F + f;
  };
  auto act = [&](int i) -> int64_t { return UP ? token_of(pairs[i], a.kinv) : pairs[i]; };
  RowSums<NT> acc;
  clear<NT>(acc);
  if constexpr (FMT == kFmtBf16) {
    const int steps = (K + kBfStep - 1) / kBfStep;
    const uint8_t* base = a.weights + static_cast<int64_t>(e) * rows * K * 2 + 16 * (lane & 3);
    const uint8_t* rp[kLaneRows];
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) rp[i] = base + static_cast<int64_t>(row(8 * i + g)) * K * 2;
    uint8_t* ring = smem + warp * kBfRing * kBfStepBytes;
    uint8_t* xring = smem + kRowWarps * kBfRing * kBfStepBytes + wk * bf_x_bytes<NT>();
    uint8_t* joins = smem + kRowWarps * kBfRing * kBfStepBytes + WK * bf_x_bytes<NT>();
    auto xrow = [&](int i) { return reinterpret_cast<const __nv_bfloat16*>(a.in + act(i) * a.in_stride); };
    row_dot_bf16<NT>(rp, active, xrow, count, K, steps * wk / WK, steps * (wk + 1) / WK, (steps + WK - 1) / WK, acc,
                     ring, xring, rg * 32 + lane, 32 * (kRowWarps / WK));
    if (WK > 1) join_slices<NT>(acc, joins, rg, wk, WK);
  } else {
    const int steps = w4_steps(K);
    const int64_t first = static_cast<int64_t>(e) * rows, groups = K / FMT;
    uint8_t* joins = smem + w4_ring_bytes<FMT, NT>(WK);
    W4Stream<FMT, NT> stream{w4_rows<FMT>(a.weights + first * (K / 2), a.scales + first * groups,
                                          a.zeros ? a.zeros + first * groups : nullptr, K, row),
                             active, smem + warp * w4_warp_bytes<FMT, NT>(), K, steps * wk / WK,
                             steps * (wk + 1) / WK};
    if (active) stream.start();
    Staged in = a.staged;
    if constexpr (LOCAL) {  // the unit's rows, in shared memory
      in = w4_staged_at(joins + joins_bytes<NT>(WK), count, K, FMT);
      __syncthreads();  // the last unit's rows have been read
      w4_stage_local<FMT>(in, count, K, [&](int i) { return a.in + act(i) * a.in_stride; });
    }
    auto column = [&](int i) { return LOCAL ? i : act(i); };
    if constexpr (NT > 1) {
      stream.run_wide(in, count, column,
                      smem + kRowWarps * w4_warp_bytes<FMT, NT>() + wk * w4_xring_bytes<FMT, NT>(), rg * 32 + lane,
                      32 * (kRowWarps / WK), (steps + WK - 1) / WK, acc);
    } else if (active) {
      stream.template run<LOCAL, AHEAD>(w4_cols<FMT, NT>(in, K, count, column), acc);
    }
    if (active) w4_unscale<NT>(acc, LOCAL ? nullptr : in.factor, count, column);
    if (WK > 1) join_slices<NT>(acc, joins, rg, wk, WK);
  }
  if (wk == 0 && active && !failed) store_block<NT, UP>(a, pairs, count, b, acc);
}

// CTAs an SM holds by registers.
// 4 bits, up to 8 pairs an entry, staged by a kernel in front: two CTAs, whose lanes
// have the registers to ask for activations a step ahead (128 experts of 3 x 2048 x 768,
// 48 tokens: 101 us, with three CTAs and no asking 109).
template <int FMT, int NTMAX, bool LOCAL>
constexpr bool moe_ahead() {
  return FMT != kFmtBf16 && NTMAX == 1 && !LOCAL;
}
template <int FMT, int NTMAX, bool LOCAL>
constexpr int moe_ctas() {
  return NTMAX == 1 && !moe_ahead<FMT, NTMAX, LOCAL>() ? 3 : 2;
}

// Both products walk (entry, row block) units; a CTA takes units blockIdx.x,
// + gridDim.x, ...  LOCAL: up to 32 pairs; every CTA builds the map itself (and
// stages a unit's rows, 4 bits), which saves the 3 to 5 us of a plan kernel in front.
// It lets its successor start only when it ends: CTAs of the next product that wait on
// an SM take the room of this one's (1 to 2% more time).
// GPU time of a whole call and its floor by the touched experts' bytes, 3 x 4096 x 1792
// an expert: bf16, 1 token on 8 experts 67 to 71 us (52), 128 tokens on 64 experts 468 to
// 505 us (416); groups of 128, 1 token 38 us (13), 128 tokens 332 us (107).  bf16,
// 3 x 1288 x 1400, 77 tokens on 60 experts: 143 to 147 us (96).  4 bits, 3 x 2048 x 768 in
// groups of 64, 48 tokens on 128: 101 us (47); 3 x 2048 x 2048, 128 tokens, 4 of 32 experts:
// groups of 128 135 us (31), of 32 182 us (35).  From 9 tokens an expert the 4-bit form is
// bound by its instructions, at 16 warps an SM.
template <int FMT, int NTMAX, bool UP, bool LOCAL>
__global__ void __launch_bounds__(kMoeThreads, moe_ctas<FMT, NTMAX, LOCAL>())
    moe_product_kernel(const __grid_constant__ ProductArgs a, const uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int small_map[LOCAL ? 4 + 3 * 64 + 32 : 1];
  griddep_wait();
  const bool failed = ld_volatile_u32(err) != 0u;  // looked at before anything is written
  PairMap m = a.map;
  if constexpr (LOCAL) {
    m = pair_map_at(small_map, a.npairs, a.E, a.cap);
    if (threadIdx.x < 32) build_small_map(m, a.idx, a.npairs, a.E, a.cap);
    __syncthreads();
  } else if (failed) {
    return;  // there may be no map
  }
  const int warp = threadIdx.x >> 5;
  const int wk = warp % a.WK, rg = warp / a.WK, RG = kMoeWarps / a.WK;
  const int blocks = UP ? (a.F + 16 * RG - 1) / (16 * RG) : (a.d + 32 * RG - 1) / (32 * RG);
  const int units = *m.total * blocks;
  int last = 0;  // NT of the CTA's last unit
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int entry = u / blocks, b = (u - entry * blocks) * RG + rg;
    const int e = m.expert[entry], count = m.count[entry];
    const int* pairs = m.pairs + m.start[entry];
    const int nt = NTMAX >= 4 && count > 24 ? 4 : NTMAX >= 4 && count > 16 ? 3 : NTMAX >= 2 && count > 8 ? 2 : 1;
    if constexpr (NTMAX > 1) {
      // Rings, staged activations and joins lie elsewhere for another NT.  Warps leave a
      // unit one by one (NT = 1 has no barrier, and the first of a row block still reads
      // the joins), so all are through with it before any fills the next one's.
      if (last != 0 && nt != last) __syncthreads();
      last = nt;
    }
    if constexpr (NTMAX >= 4) {
      if (nt == 4) {
        moe_unit<FMT, 4, UP, LOCAL, false>(a, e, pairs, count, b, rg, wk, smem, failed);
        continue;
      }
      if (nt == 3) {
        moe_unit<FMT, 3, UP, LOCAL, false>(a, e, pairs, count, b, rg, wk, smem, failed);
        continue;
      }
    }
    if constexpr (NTMAX >= 2) {
      if (nt == 2) {
        moe_unit<FMT, 2, UP, LOCAL, false>(a, e, pairs, count, b, rg, wk, smem, failed);
        continue;
      }
    }
    moe_unit<FMT, 1, UP, LOCAL, moe_ahead<FMT, NTMAX, LOCAL>()>(a, e, pairs, count, b, rg, wk, smem, failed);
  }
}

// y[t] = the sum of the token's partial rows in the order of its choices;
// choices outside [0, E) have none.
__global__ void moe_combine_kernel(const float* __restrict__ part, const int32_t* __restrict__ idx,
                                   __nv_bfloat16* __restrict__ y, int T, int k, int E, int d, const uint32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  const int d4 = d / 4;
  const int64_t n = static_cast<int64_t>(T) * d4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int t = static_cast<int>(i / d4), c = static_cast<int>(i - static_cast<int64_t>(t) * d4) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < k; ++j) {
      const int p = t * k + j, e = idx[p];
      if (e < 0 || e >= E) continue;
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(p) * d + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(t) * d + c) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// The rings of whichever NT up to NTMAX a unit runs with.
template <int FMT, int NTMAX>
int moe_w4_ring(int WK) {
  int most = w4_ring_bytes<FMT, 1>(WK);
  if constexpr (NTMAX > 1) most = std::max(most, w4_ring_bytes<FMT, 2>(WK));
  if constexpr (NTMAX > 2) most = std::max({most, w4_ring_bytes<FMT, 3>(WK), w4_ring_bytes<FMT, 4>(WK)});
  return most;
}

template <int FMT, int NTMAX, bool UP, bool LOCAL>
cudaError_t launch_product(ProductArgs a, const DeviceInfo& dev, cudaStream_t s) {
  const int K = UP ? a.d : a.F;
  const int blocks = UP ? (a.F + 15) / 16 : (a.d + 31) / 32;
  const int entries = a.npairs < a.E ? a.npairs : a.E;  // active experts, at most
  constexpr bool W4 = FMT != kFmtBf16;
  const int steps = W4 ? w4_steps(K) : (K + kBfStep - 1) / kBfStep;
  a.WK = rowdot_split(blocks, entries, steps, moe_ctas<FMT, NTMAX, LOCAL>(),
                      W4 ? w4_most_split<NTMAX>() : kMoeWarps / NTMAX, dev.num_sms);
  int smem;
  if constexpr (W4)
    smem = moe_w4_ring<FMT, NTMAX>(a.WK) + joins_bytes<NTMAX>(a.WK) +
           (LOCAL ? static_cast<int>(w4_staged_bytes(a.cap, K, FMT, true)) : 0);
  else smem = bf_smem<NTMAX>(a.WK);
  auto kern = moe_product_kernel<FMT, NTMAX, UP, LOCAL>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), 160 * 1024, dev.device);
  if (e != cudaSuccess) return e;
  const int RG = kMoeWarps / a.WK;
  const int64_t units =
      static_cast<int64_t>(max_entries(a.npairs, a.E, a.cap)) * (UP ? (a.F + 16 * RG - 1) / (16 * RG)
                                                                    : (a.d + 32 * RG - 1) / (32 * RG));
  // as many CTAs as the SM's shared memory and registers hold at a time
  int per_sm = 228 * 1024 / (smem + 1024);
  per_sm = per_sm < 1 ? 1 : per_sm > moe_ctas<FMT, NTMAX, LOCAL>() ? moe_ctas<FMT, NTMAX, LOCAL>() : per_sm;
  int64_t grid = static_cast<int64_t>(per_sm) * dev.num_sms;
  if (grid > units) grid = units;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kMoeThreads), smem, s, a,
                    static_cast<const uint32_t*>(dev.err));
}

// Staged rows of a unit, at most, that every CTA makes for itself.  1 token of 4096
// (8.6 KB): 38.0 us so, and 37.5 with two staging kernels, which cost the host 4 us; 4
// tokens of 2048 (16.4 KB), 6 of 64 experts of 768 in groups of 32: 43 and 36 us.
constexpr int64_t kLocalBytes = 10 * 1024;

template <int FMT, bool UP>
cudaError_t launch_product_nt(const ProductArgs& a, bool local, int ntmax, const DeviceInfo& dev, cudaStream_t s) {
  if (local) return launch_product<FMT, 1, UP, true>(a, dev, s);
  if (ntmax == 1) return launch_product<FMT, 1, UP, false>(a, dev, s);
  if (ntmax == 2) return launch_product<FMT, 2, UP, false>(a, dev, s);
  return launch_product<FMT, 4, UP, false>(a, dev, s);
}

// Scratch of a call: the pair map, hidden rows and partial rows of every pair, and
// (4 bits) the staged tokens and the sums and factors of the hidden rows (which are
// staged in place).
struct MoeScratch {
  int64_t map, h, part, x, hsums, hfactor, total;
  int64_t h_stride;
};
MoeScratch moe_scratch(int T, int k, int E, int d, int F, int group) {
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  const int64_t pairs = static_cast<int64_t>(T) * k;
  MoeScratch m{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes);
    return here;
  };
  m.h_stride = group ? w4_row_bytes(F) : 2 * static_cast<int64_t>(F);
  const int cap = T < 8 ? (T < 1 ? 1 : T) : 8;  // the fewest pairs of an entry that a call uses
  m.map = take(4 * static_cast<int64_t>(pair_map_ints(static_cast<int>(pairs), E, cap)));
  m.h = take(pairs * m.h_stride);
  m.part = take(pairs * d * 4);
  if (group) {
    m.x = take(w4_staged_bytes(T, d, group));
    m.hsums = take(w4_sums_bytes(pairs, F, group));
    m.hfactor = take(4 * pairs);
  }
  m.total = at;
  return m;
}

template <int FMT>
cudaError_t moe_launches(const MoeCall& c, const DeviceInfo& dev, cudaStream_t s, MoeTrace* trace) {
  constexpr bool W4 = FMT != kFmtBf16;
  const int npairs = c.T * c.k;
  const MoeScratch sc = moe_scratch(c.T, c.k, c.E, c.d, c.F, FMT);
  uint8_t* base = static_cast<uint8_t*>(c.scratch);
  // an expert gets T*k/E of the pairs on average and at most T distinct ones
  const int typical = (2 * npairs + c.E - 1) / c.E, most = typical < c.T ? typical : c.T;
  int ntmax = most <= 8 ? 1 : most <= 16 ? 2 : 4;
  const int cap = c.T < 8 * ntmax ? c.T : 8 * ntmax;
  bool local = npairs <= 32 && cap <= 8;
  if constexpr (W4)
    local = local && w4_staged_bytes(cap, c.d, FMT, true) <= kLocalBytes &&
            w4_staged_bytes(cap, c.F, FMT, true) <= kLocalBytes;
  if (local) ntmax = 1;
  ProductArgs a{};
  a.idx = static_cast<const int32_t*>(c.idx);
  a.gates = static_cast<const float*>(c.gates);
  a.npairs = npairs;
  a.E = c.E;
  a.F = c.F;
  a.d = c.d;
  a.cap = cap;
  a.kinv = token_factor(c.k);
  a.map = pair_map_at(reinterpret_cast<int*>(base + sc.map), npairs, c.E, cap);
  const uint32_t* err = dev.err;
  Staged staged_x{}, staged_h{};
  if constexpr (W4) {
    staged_x = w4_staged_at(base + sc.x, c.T, c.d, FMT);
    staged_h = Staged{base + sc.h, reinterpret_cast<float*>(base + sc.hsums),
                      reinterpret_cast<float*>(base + sc.hfactor)};
  }
  cudaError_t e;
  if (!local) {
    trace->begin("moe_plan", 0.0, 4.0 * npairs);
    const StageArgs x{static_cast<const uint8_t*>(c.x), staged_x, 2 * static_cast<int64_t>(c.d), W4 ? c.T : 0, c.d};
    const int grid = 1 + (x.n < 4 * dev.num_sms ? x.n : 4 * dev.num_sms);
    e = launch_pdl(moe_plan_kernel<FMT>, dim3(grid), dim3(kMoeThreads), kMoeWarps * c.E * sizeof(int), s, a.map, a.idx,
                   npairs, c.E, cap, x, err);
    trace->end();
    if (e != cudaSuccess) return e;
  }
  const double df = static_cast<double>(c.d) * c.F, n_exp = npairs < c.E ? npairs : c.E;
  const double wb = W4 ? 0.5 + (c.z13 ? 3.0 : 2.0) / (W4 ? FMT : 1) : 2.0;  // bytes of a weight
  // up
  a.weights = static_cast<const uint8_t*>(c.w13);
  a.scales = static_cast<const __nv_bfloat16*>(c.s13);
  a.zeros = static_cast<const uint8_t*>(c.z13);
  a.in = static_cast<const uint8_t*>(c.x);
  a.in_stride = 2 * static_cast<int64_t>(c.d);
  a.staged = staged_x;
  a.out = base + sc.h;
  a.out_stride = sc.h_stride;
  trace->begin("moe_up", 4.0 * npairs * df, n_exp * 2.0 * df * wb + 2.0 * c.T * c.d + 2.0 * npairs * c.F);
  e = launch_product_nt<FMT, true>(a, local, ntmax, dev, s);
  trace->end();
  if (e != cudaSuccess) return e;
  if constexpr (W4) {
    if (!local) {
      trace->begin("moe_stage", 0.0, 4.0 * npairs * c.F);
      const StageArgs h{base + sc.h, staged_h, sc.h_stride, npairs, c.F};
      const int grid = npairs < 8 * dev.num_sms ? npairs : 8 * dev.num_sms;
      e = launch_pdl(moe_stage_kernel<FMT>, dim3(grid), dim3(kMoeThreads), 0, s, h, err);
      trace->end();
      if (e != cudaSuccess) return e;
    }
  }
  // down
  a.weights = static_cast<const uint8_t*>(c.w2);
  a.scales = static_cast<const __nv_bfloat16*>(c.s2);
  a.zeros = static_cast<const uint8_t*>(c.z2);
  a.in = base + sc.h;
  a.in_stride = sc.h_stride;
  a.staged = staged_h;
  a.out = base + sc.part;
  a.out_stride = 4 * static_cast<int64_t>(c.d);
  trace->begin("moe_down", 2.0 * npairs * df, n_exp * df * wb + 2.0 * npairs * c.F + 4.0 * npairs * c.d);
  e = launch_product_nt<FMT, false>(a, local, ntmax, dev, s);
  trace->end();
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(c.T) * (c.d / 4);
  int64_t blocks = (n + 255) / 256;
  if (blocks > 8 * dev.num_sms) blocks = 8 * dev.num_sms;
  trace->begin("moe_combine", 0.0, 4.0 * npairs * c.d + 2.0 * c.T * c.d);
  e = launch_pdl(moe_combine_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                 reinterpret_cast<const float*>(base + sc.part), a.idx, static_cast<__nv_bfloat16*>(c.y), c.T, c.k,
                 c.E, c.d, err);
  trace->end();
  return e;
}

}  // namespace

size_t moe_scratch_bytes(int T, int k, int E, int d, int F, int group) {
  return static_cast<size_t>(moe_scratch(T, k, E, d, F, group).total);
}

cudaError_t launch_moe_swiglu(const MoeCall& c, const DeviceInfo& dev, cudaStream_t s, MoeTrace* trace) {
  switch (c.group) {
    case 0: return moe_launches<kFmtBf16>(c, dev, s, trace);
    case 32: return moe_launches<32>(c, dev, s, trace);
    case 64: return moe_launches<64>(c, dev, s, trace);
    default: return moe_launches<128>(c, dev, s, trace);
  }
}

int moe_max_pairs() { return kMaxPairs; }
int moe_max_experts() { return kMaxExperts; }
int moe_max_topk() { return kMaxTopk; }

cudaError_t launch_moe_logits(const void* x, const void* wr, float* logits, int T, int d, int E, const DeviceInfo& dev,
                              cudaStream_t s) {
  const int pairs = (E + kLogitExperts - 1) / kLogitExperts, blocks = (T + kLogitTokens - 1) / kLogitTokens;
  // a warp for every pair of experts and block of tokens; with fewer than kLogitSpread
  // warps an SM, 2, 4 or 8, to which d is split.  32 x 7168 on 256 experts: 26.7 us, with
  // one warp 29.9; 200 x 4096 on 64: 23.7, 27.8; 16 x 4096 on 128: 10.3 with 8, 10.0 with 4.
  const int64_t warps = static_cast<int64_t>(pairs) * blocks, want = static_cast<int64_t>(kLogitSpread) * dev.num_sms;
  const int KS = warps >= want ? 1 : 2 * warps >= want ? 2 : 4 * warps >= want ? 4 : 8;
  auto kern = KS == 1   ? moe_logits_kernel<1>
              : KS == 2 ? moe_logits_kernel<2>
              : KS == 4 ? moe_logits_kernel<4>
                        : moe_logits_kernel<8>;
  const int a_cta = kLogitWarps / KS;
  return launch_pdl(kern, dim3((pairs + a_cta - 1) / a_cta, blocks), dim3(kLogitWarps * 32), 0, s,
                    static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(wr), logits, T, d, E,
                    static_cast<const uint32_t*>(dev.err));
}

cudaError_t launch_moe_topk(const float* logits, void* idx, void* gates, int T, int E, int k, bool sigmoid,
                            bool renorm, float scale, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pdl(moe_topk_kernel, dim3((T + kTopkWarps - 1) / kTopkWarps), dim3(kTopkWarps * 32), 0, s, logits,
                    static_cast<int32_t*>(idx), static_cast<float*>(gates), T, E, k, sigmoid, renorm, scale,
                    static_cast<const uint32_t*>(dev.err));
}

}  // namespace dg
