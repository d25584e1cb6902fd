// Routed experts for few tokens: the router (logits, top-k, gates) and the
// SwiGLU experts' products on bf16 or 4-bit weights.
//
//   e_j = idx[t, j], h_j = silu(w1[e_j] x_t) * (w3[e_j] x_t),
//   y_t = sum_j gates[t, j] * (w2[e_j] h_j)
//
// With few tokens the experts' weights are the traffic: every touched expert's
// rows are read once and meet all of its tokens in registers (dg_rowdot.cuh).
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "dg_rowdot.cuh"

namespace dg {

namespace {

__device__ __forceinline__ bool err_set(const uint32_t* err) { return ld_volatile_u32(err) != 0u; }

// ---------------------------------------------------------------- router

// s + p without error: s becomes the rounded sum, c collects what was lost
// (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float& s, float& c, float p) {
  const float t = __fadd_rn(s, p);
  const float z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
  s = t;
}

constexpr int kLogitWarps = 8;
constexpr int kLogitTokens = 4;

// logits[t, e]: a warp per expert and kLogitTokens tokens.  The choice of
// experts hangs on the order of the logits, so the sums are kept in two words
// (a bf16 product is exact in binary32, two_sum loses nothing) and rounded to
// binary32 once.
__global__ void __launch_bounds__(kLogitWarps * 32)
    moe_logits_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wr,
                      float* __restrict__ logits, int T, int d, int E, const uint32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;
  const int lane = threadIdx.x & 31;
  const int e = static_cast<int>(blockIdx.x) * kLogitWarps + (threadIdx.x >> 5);
  const int t0 = static_cast<int>(blockIdx.y) * kLogitTokens;
  if (e >= E) return;
  const __nv_bfloat16* w = wr + static_cast<int64_t>(e) * d;
  float s[kLogitTokens], c[kLogitTokens];
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) s[i] = c[i] = 0.0f;
  for (int k = 8 * lane; k < d; k += 256) {
    const uint4 wv = *reinterpret_cast<const uint4*>(w + k);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
      if (t0 + i >= T) break;
      const uint4 xv = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t0 + i) * d + k);
      const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = unpack_bf16x2(ww[j]), b = unpack_bf16x2(xx[j]);
        two_sum(s[i], c[i], __fmul_rn(a.x, b.x));
        two_sum(s[i], c[i], __fmul_rn(a.y, b.y));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float so = __shfl_xor_sync(0xffffffffu, s[i], o);
      const float co = __shfl_xor_sync(0xffffffffu, c[i], o);
      two_sum(s[i], c[i], so);
      c[i] += co;
    }
    // an overflowed or non-finite sum makes its correction NaN: keep the sum itself
    const float sum = s[i] + c[i];
    if (lane == 0 && t0 + i < T)
      logits[static_cast<int64_t>(t0 + i) * E + e] = isfinite(s[i]) ? sum : s[i];
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

// One warp per token: k times the largest remaining key, then the gates.
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
  if (lane < k) p = sigmoid ? 1.0f / (1.0f + expf(-mine)) : expf(mine - top);
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
constexpr int kMoeSmemMax = 227 * 1024;
constexpr size_t kSmSmem = 228 * 1024;

// The work of a call, built by every CTA from idx: entries of one expert and
// up to `cap` of its pairs.  Shared memory: entry_expert[n], entry_start[n],
// entry_count[n] and pairs[] (the pairs sorted by expert).
//
// Every CTA must come to the same order of an expert's pairs, since the units
// of its entries may run on different CTAs: the sort is stable.  Warp w counts
// and later places the w-th run of pairs, so `at[w][e]` is where its next pair
// of expert e goes.
struct PairMap {
  int* at;            // [kMoeWarps][E]
  int* entry_expert;  // [max_entries]
  int* entry_start;
  int* entry_count;
  int* total;       // number of entries
  uint16_t* pairs;  // [npairs]
};

__host__ __device__ inline int max_entries(int npairs, int E, int cap) {
  const int active = npairs < E ? npairs : E;
  return active + npairs / cap;
}

inline size_t pair_map_bytes(int npairs, int E, int cap) {
  return sizeof(int) * (kMoeWarps * static_cast<size_t>(E) + 1 +
                        3 * static_cast<size_t>(max_entries(npairs, E, cap))) +
         (2 * static_cast<size_t>(npairs) + 15) / 16 * 16;
}

__device__ __forceinline__ PairMap build_pair_map(uint8_t* smem, const int32_t* __restrict__ idx, int npairs, int E,
                                                  int cap) {
  PairMap m;
  const int me = max_entries(npairs, E, cap);
  m.at = reinterpret_cast<int*>(smem);
  m.entry_expert = m.at + kMoeWarps * E;
  m.entry_start = m.entry_expert + me;
  m.entry_count = m.entry_start + me;
  m.total = m.entry_count + me;
  m.pairs = reinterpret_cast<uint16_t*>(m.total + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* at = m.at + warp * E;
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
        for (int w = 0; w < kMoeWarps; ++w) n += m.at[w * E + e];
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
          const int c = m.at[w * E + e];
          m.at[w * E + e] = next;
          next += c;
        }
      }
      for (int i = 0; i < ne; ++i) {
        const int to = entries_before + se - ne + i;
        m.entry_expert[to] = e;
        m.entry_start[to] = start + i * cap;
        m.entry_count[to] = min(cap, n - i * cap);
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
      m.pairs[base + before] = static_cast<uint16_t>(p);
      if (before == 0) at[e] = base + __popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  return m;
}

// pair / k as a product: kinv = 2^18 / k + 1 is exact for pairs below 2^13 and k up to 2^5.
static_assert(kMaxPairs <= 8192 && kMaxTopk <= 32, "token_of");
inline uint32_t token_factor(int k) { return (1u << 18) / static_cast<uint32_t>(k) + 1u; }
__device__ __forceinline__ int token_of(uint32_t pair, uint32_t kinv) { return static_cast<int>((pair * kinv) >> 18); }

// One of the two weight tensors of the experts.
struct MoeWeights {
  const uint8_t* data;          // [E, rows, K] bf16, or codes [E, rows, K/2]
  const __nv_bfloat16* scales;  // [E, rows, K/group]
  const uint8_t* zeros;
  int rows, K;
};

template <int FMT>
__device__ __forceinline__ Rows expert_rows(const MoeWeights& w, int e) {
  const int64_t first = static_cast<int64_t>(e) * w.rows;
  if constexpr (FMT == kFmtBf16) return Rows{w.data + first * w.K * 2, nullptr, nullptr};
  const int64_t groups = first * (w.K / (FMT ? FMT : 1));
  return Rows{w.data + first * (w.K / 2), w.scales + groups, w.zeros ? w.zeros + groups : nullptr};
}

// The units of a CTA: (entry, row block) pairs blockIdx.x, + gridDim.x, ... of
// all entries and row blocks.  A row block is 8 / WK warps' worth of rows.
//   UP    a warp's two row tiles are 16 rows of w1 and the same 16 of w3, so a and b
//         of one (pair, f) meet in one thread: h[pair, f] = bf16(silu(a) * b).  h is
//         rounded to bf16 once: it is the next product's matrix operand.
//   else  32 rows of w2: part[pair, r] = gate * (w2[e, r] . h[pair])
template <int FMT, int NT, bool UP>
struct MoeWork {
  const MoeWeights& w;
  const PairMap& m;
  const __nv_bfloat16* in;
  const float* gates;
  void* out;
  uint32_t kinv;
  int F, d, RG, blocks, total;

  __device__ int units() const {
    const int first = blockIdx.x, step = gridDim.x;
    return first < total ? (total - first + step - 1) / step : 0;
  }
  __device__ int entry(int u) const { return static_cast<int>(blockIdx.x + u * gridDim.x) / blocks; }
  __device__ int block(int u) const { return static_cast<int>(blockIdx.x + u * gridDim.x) % blocks; }
  __device__ Rows rows(int u) const { return expert_rows<FMT>(w, m.entry_expert[entry(u)]); }
  __device__ int row(int u, int rg, int lane, bool& active) const {
    const int b = block(u) * RG + rg;
    if (UP) {
      active = b * 16 < F;
      const int f = min(b * 16 + (lane & 15), F - 1);
      return lane < 16 ? f : F + f;
    }
    active = b * 32 < d;
    return min(b * 32 + lane, d - 1);
  }
  __device__ int count(int u) const { return m.entry_count[entry(u)]; }
  __device__ const __nv_bfloat16* xrow(int u, int i) const {
    const int p = m.pairs[m.entry_start[entry(u)] + i];
    return UP ? in + static_cast<int64_t>(token_of(p, kinv)) * d : in + static_cast<int64_t>(p) * F;
  }
  __device__ void finish(int u, int rg, const float (&acc)[kRowTiles][NT][4]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int e = entry(u), n_pairs = m.entry_count[e];
    const uint16_t* pairs = m.pairs + m.entry_start[e];
    const int b = block(u) * RG + rg;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 8 * n + 2 * t + (i & 1), r = g + (i >> 1) * 8;
        if (c >= n_pairs) continue;
        const int64_t p = pairs[c];
        if (UP) {
          const int f = b * 16 + r;
          const float a = acc[0][n][i], v = acc[1][n][i];
          if (f < F) static_cast<__nv_bfloat16*>(out)[p * F + f] = __float2bfloat16_rn(a / (1.0f + expf(-a)) * v);
        } else {
          const float gate = gates[p];
#pragma unroll
          for (int tile = 0; tile < kRowTiles; ++tile) {
            const int row = b * 32 + 16 * tile + r;
            if (row < d) static_cast<float*>(out)[p * d + row] = gate * acc[tile][n][i];
          }
        }
      }
  }
};

// CTAs an SM holds by registers.
template <int FMT, int NT>
constexpr int moe_ctas() {
  return FMT == kFmtBf16 && NT == 1 ? 3 : 2;
}

template <int FMT, int NT, bool UP>
__global__ void __launch_bounds__(kMoeThreads, moe_ctas<FMT, NT>())
    moe_product_kernel(MoeWeights w, const __nv_bfloat16* __restrict__ in, const int32_t* __restrict__ idx,
                       const float* __restrict__ gates, void* __restrict__ out, int npairs, uint32_t kinv, int E,
                       int WK, const uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  if (err_set(err)) return;  // the word changes only between calls: uniform over the CTA
  const PairMap m = build_pair_map(smem + rowdot_smem<FMT, NT>(WK), idx, npairs, E, 8 * NT);
  const int RG = kMoeWarps / WK;
  const int F = UP ? w.rows / 2 : w.K, d = UP ? w.K : w.rows;
  const int blocks = UP ? (F + 16 * RG - 1) / (16 * RG) : (d + 32 * RG - 1) / (32 * RG);
  const MoeWork<FMT, NT, UP> work{w, m, in, gates, out, kinv, F, d, RG, blocks, *m.total * blocks};
  row_stream<FMT, NT>(work, w.K, WK, smem);
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

template <int FMT, int NT, bool UP>
cudaError_t launch_product(const MoeWeights& w, const __nv_bfloat16* in, const int32_t* idx, const float* gates,
                           void* out, int T, int k, int E, const DeviceInfo& dev, cudaStream_t s) {
  const int npairs = T * k;
  const int entries = npairs < E ? npairs : E;  // active experts, at most (more only where one fills several entries)
  const int rows = UP ? w.rows / 2 : w.rows, step = UP ? 16 : 32;
  const int steps = (w.K + rowdot_step<FMT>() - 1) / rowdot_step<FMT>();
  constexpr int kMostWK = NT == 4 ? 2 : NT == 2 ? 4 : kMoeWarps;  // the slices' staged rows have to fit
  const int64_t slots = static_cast<int64_t>(moe_ctas<FMT, NT>()) * dev.num_sms;
  int WK = rowdot_split((rows + step - 1) / step, entries, steps, kMostWK, slots);
  const size_t map = pair_map_bytes(npairs, E, 8 * NT);
  while (WK > 1 && rowdot_smem<FMT, NT>(WK) + map > kMoeSmemMax) WK /= 2;
  const size_t smem = rowdot_smem<FMT, NT>(WK) + map;
  auto kern = moe_product_kernel<FMT, NT, UP>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), kMoeSmemMax, dev.device);
  if (e != cudaSuccess) return e;
  // as many CTAs as the SM's shared memory and registers hold
  int per_sm = static_cast<int>(kSmSmem / (smem + 1024));
  per_sm = per_sm < 1 ? 1 : per_sm > moe_ctas<FMT, NT>() ? moe_ctas<FMT, NT>() : per_sm;
  const int rg = kMoeWarps / WK;
  const int64_t units = static_cast<int64_t>(max_entries(npairs, E, 8 * NT)) * ((rows + step * rg - 1) / (step * rg));
  int64_t grid = static_cast<int64_t>(per_sm) * dev.num_sms;
  if (grid > units) grid = units;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kMoeThreads), smem, s, w, in, idx, gates, out,
                    npairs, token_factor(k), E, WK, static_cast<const uint32_t*>(dev.err));
}

template <int FMT, bool UP>
cudaError_t launch_product_nt(const MoeWeights& w, const __nv_bfloat16* in, const int32_t* idx, const float* gates,
                              void* out, int T, int k, int E, const DeviceInfo& dev, cudaStream_t s) {
  // an expert gets T*k/E of the pairs on average and at most T distinct ones
  const int typical = (2 * T * k + E - 1) / E;
  const int most = typical < T ? typical : T;
  if (most <= 8) return launch_product<FMT, 1, UP>(w, in, idx, gates, out, T, k, E, dev, s);
  if (most <= 16) return launch_product<FMT, 2, UP>(w, in, idx, gates, out, T, k, E, dev, s);
  return launch_product<FMT, 4, UP>(w, in, idx, gates, out, T, k, E, dev, s);
}

template <bool UP>
cudaError_t launch_product_fmt(int fmt, const MoeWeights& w, const __nv_bfloat16* in, const int32_t* idx,
                               const float* gates, void* out, int T, int k, int E, const DeviceInfo& dev,
                               cudaStream_t s) {
  switch (fmt) {
    case kFmtBf16: return launch_product_nt<kFmtBf16, UP>(w, in, idx, gates, out, T, k, E, dev, s);
    case 32: return launch_product_nt<32, UP>(w, in, idx, gates, out, T, k, E, dev, s);
    case 64: return launch_product_nt<64, UP>(w, in, idx, gates, out, T, k, E, dev, s);
    default: return launch_product_nt<128, UP>(w, in, idx, gates, out, T, k, E, dev, s);
  }
}

}  // namespace

int moe_max_pairs() { return kMaxPairs; }
int moe_max_experts() { return kMaxExperts; }
int moe_max_topk() { return kMaxTopk; }

cudaError_t launch_moe_logits(const void* x, const void* wr, float* logits, int T, int d, int E, const DeviceInfo& dev,
                              cudaStream_t s) {
  const dim3 grid((E + kLogitWarps - 1) / kLogitWarps, (T + kLogitTokens - 1) / kLogitTokens);
  return launch_pdl(moe_logits_kernel, grid, dim3(kLogitWarps * 32), 0, s, static_cast<const __nv_bfloat16*>(x),
                    static_cast<const __nv_bfloat16*>(wr), logits, T, d, E, static_cast<const uint32_t*>(dev.err));
}

cudaError_t launch_moe_topk(const float* logits, void* idx, void* gates, int T, int E, int k, bool sigmoid,
                            bool renorm, float scale, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pdl(moe_topk_kernel, dim3((T + kTopkWarps - 1) / kTopkWarps), dim3(kTopkWarps * 32), 0, s, logits,
                    static_cast<int32_t*>(idx), static_cast<float*>(gates), T, E, k, sigmoid, renorm, scale,
                    static_cast<const uint32_t*>(dev.err));
}

cudaError_t launch_moe_up(const MoeSource& w13, const void* x, const void* idx, void* h, int T, int k, int E, int d,
                          int F, const DeviceInfo& dev, cudaStream_t s) {
  const MoeWeights w{static_cast<const uint8_t*>(w13.data), static_cast<const __nv_bfloat16*>(w13.scales),
                     static_cast<const uint8_t*>(w13.zeros), 2 * F, d};
  return launch_product_fmt<true>(w13.group, w, static_cast<const __nv_bfloat16*>(x),
                                  static_cast<const int32_t*>(idx), nullptr, h, T, k, E, dev, s);
}

cudaError_t launch_moe_down(const MoeSource& w2, const void* h, const void* idx, const void* gates, void* part, int T,
                            int k, int E, int d, int F, const DeviceInfo& dev, cudaStream_t s) {
  const MoeWeights w{static_cast<const uint8_t*>(w2.data), static_cast<const __nv_bfloat16*>(w2.scales),
                     static_cast<const uint8_t*>(w2.zeros), d, F};
  return launch_product_fmt<false>(w2.group, w, static_cast<const __nv_bfloat16*>(h),
                                   static_cast<const int32_t*>(idx), static_cast<const float*>(gates), part, T, k, E,
                                   dev, s);
}

cudaError_t launch_moe_combine(const float* part, const void* idx, void* y, int T, int k, int E, int d,
                               const DeviceInfo& dev, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(T) * (d / 4);
  int64_t blocks = (n + 255) / 256;
  if (blocks > 8 * dev.num_sms) blocks = 8 * dev.num_sms;
  return launch_pdl(moe_combine_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, part,
                    static_cast<const int32_t*>(idx), static_cast<__nv_bfloat16*>(y), T, k, E, d,
                    static_cast<const uint32_t*>(dev.err));
}

}  // namespace dg
