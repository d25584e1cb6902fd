// Block-scaled e4m3 linear for few rows (sm_103a): y[t, n] = bias[n] + sum_k x[t, k] w[n, k].
//
// With few rows the product is bound by reading the weight once.  The operands are
// exchanged: 128 rows of the weight fill the MMA's M side (a TMEM lane each) and NT
// = 16 to 128 rows of x its N side, so no part of the tensor core's work is padding
// along the weight.  One CTA takes 128 features and a part of K; the CTAs of a
// cluster share the features and split K, leave their binary32 sums in shared
// memory and add them through distributed shared memory in the order of their ranks
// (the same result every time).  One row, 4096 to 6144: 6.6 us from codes, 7.3 from
// bf16, 25 MB; 4 rows, 4096 to 28672: 22.5 and 24.2 us, 117 MB, 5.2 TB/s.
//
// Warp roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 bring
// the block scales to TMEM (as in dg_mx.cuh) and then do the epilogue.  Where x comes in
// bf16 and has at most four rows, they also quantise it into the stages, every CTA its
// part of K: one launch fewer.  The work grows with the rows that the form provides for; see
// kMxFewBf16Rows for both sides.
#include "dg_fp8.cuh"
#include "dg_internal.h"
#include "dg_mx.cuh"

namespace dg {

namespace {

template <int NT, bool kBf16>
struct FewCfg {
  static constexpr int BM = 128;                 // features a CTA
  static constexpr int STAGES = NT == 16 ? 5 : NT == 64 ? 3 : 4;
  static constexpr int W_BYTES = BM * 128;
  static constexpr int X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int SF_BUFS = 4;
  static constexpr int SF_COLS = 16;             // W words at +0, x words at +8
  static constexpr int SF_BASE = NT < 32 ? 32 : NT;
  static constexpr int X_WORDS = (NT + 31) / 32;
  static constexpr int LOAD_BYTES = W_BYTES + (kBf16 ? 0 : X_BYTES);  // by TMA, a stage
  static constexpr int FULL_COUNT = kBf16 ? 2 : 1;  // arrivals: the producer, and the warp that writes x
  static constexpr int X_ROWS = 4;               // bf16: most rows
  static constexpr uint32_t TMEM_COLS = SF_BASE + SF_BUFS * SF_COLS <= 128 ? 128 : 256;
  static constexpr int MAX_SPLIT = 8;
  // Sums that arrive from the cluster: [rank][feature of this CTA][ROW_F], padded against bank conflicts.
  static constexpr int ROW_F = NT + 4;
  static constexpr int RECV_BYTES = BM * ROW_F * 4;
  static constexpr int FEED_BYTES = 2 * 4 * (NT + 4) * 4;
  // Sums of many rows go to a peer as one bulk copy from the (idle) stages, those of few rows from registers.
  static constexpr bool BULK = NT >= 64;
  static constexpr int NUM_THREADS = 192;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * SF_BUFS + 2;
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + RECV_BYTES + FEED_BYTES + BAR_BYTES;
  static constexpr uint32_t IDESC = ((NT >> 3) << 17) | (1u << 23) | ((BM >> 4) << 24);
  static_assert(NUM_BARS * 8 + 4 <= BAR_BYTES && SMEM_BYTES <= 232448, "shared memory");
  static_assert(!kBf16 || STAGES >= 4, "x is quantised four stages at a time");
};

struct FewParams {
  int32_t M, N, K, kb;         // rows of x, features, columns and K blocks
  const __nv_bfloat16* x;      // [M][K] (kBf16; then no codes and sx)
  const uint8_t *sx, *sw;      // [M][kb], [ceil(N/128)][kb]
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;
  uint32_t* err;
};

// 16 bytes into a cluster CTA's shared memory, counted on an mbarrier of the same CTA.
__device__ __forceinline__ void st_async_v4(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}

// `bytes` of this CTA's shared memory into a cluster CTA's, counted on an mbarrier of that CTA (16-byte units).
__device__ __forceinline__ void dsmem_bulk_copy(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <int NT, bool kBf16>
__global__ void __launch_bounds__(FewCfg<NT, kBf16>::NUM_THREADS)
    mx_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const FewParams p) {
  using Cfg = FewCfg<NT, kBf16>;
  extern __shared__ uint8_t smem_raw[];

  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stage_base = smem_raw + pad;
  float* recv = reinterpret_cast<float*>(stage_base + Cfg::STAGES * Cfg::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(recv) + Cfg::RECV_BYTES + Cfg::FEED_BYTES);
  uint64_t* empty = full + Cfg::STAGES;
  uint64_t* sf_full = empty + Cfg::STAGES;
  uint64_t* sf_empty = sf_full + Cfg::SF_BUFS;
  uint64_t* done = sf_empty + Cfg::SF_BUFS;
  uint64_t* arrived = done + 1;                    // the cluster's sums for this CTA's share of the features
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(arrived + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(gridDim.z);   // the cluster: all CTAs of a (feature, row) tile
  const int rank = static_cast<int>(blockIdx.z);
  const int n0 = static_cast<int>(blockIdx.x) * Cfg::BM;
  const int t0 = static_cast<int>(blockIdx.y) * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / split);
  const int num_kb = kb1 - kb0;
  const int rows = min(NT, p.M - t0);
  const int rows4 = (rows + 3) / 4;                // sums travel four rows at a time
  const int f_count = Cfg::BM / split;             // features whose sums this CTA adds up, from f_first
  const int f_first = rank * f_count;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&full[s], Cfg::FULL_COUNT);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < Cfg::SF_BUFS; ++b) {
      mbar_init(&sf_full[b], 4);
      mbar_init(&sf_empty[b], 1);
    }
    mbar_init(done, 1);
    mbar_init(arrived, 1);
    mbar_arrive_expect_tx(arrived, static_cast<uint32_t>(split * f_count) *
                                       (Cfg::BULK ? static_cast<uint32_t>(Cfg::ROW_F) * 4u : static_cast<uint32_t>(rows4) * 16u));
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    if (!kBf16) tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  cluster_arrive();  // barriers and buffers of this CTA are ready for its peers
  const uint32_t tmem_base = *tmem_holder;
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      for (int i = 0; i < num_kb; ++i) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, SITE_EMPTY)) break;
        uint8_t* sw = stage_base + stage * Cfg::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[stage], Cfg::LOAD_BYTES);
        tma_load_3d(sw, &tmW, &full[stage], (kb0 + i) * 128, n0, 0);
        if (!kBf16) tma_load_3d(sw + Cfg::W_BYTES, &tmX, &full[stage], (kb0 + i) * 128, t0, 0);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == Cfg::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      for (int s = 0; s < Cfg::STAGES; ++s)
        if ((armed & (1u << s)) && !mbar_try_wait(&full[s], (armed_parity >> s) & 1u)) {
          uint32_t dummy = 0;
          mbar_wait_slow(&full[s], (armed_parity >> s) & 1u, &dummy, SITE_DRAIN, kWaitLimitNs);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, sfphase = 0;
      const uint64_t desc0 = smem_desc_sw128(smem_u32(stage_base), 16, 1024);
      for (int i = 0; i < num_kb; i += 4) {
        if (!mbar_wait(&sf_full[buf], sfphase, p.err, SITE_SF_FULL)) break;
        tc_fence_after_sync();
        const uint32_t sf = tmem_base + static_cast<uint32_t>(Cfg::SF_BASE + buf * Cfg::SF_COLS);
        bool ok = true;
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          if (i + static_cast<int>(q) >= num_kb) break;
          ok = ok && mbar_wait(&full[stage], phase, p.err, SITE_FULL);
          if (!ok) break;
          const uint64_t wd = desc0 + static_cast<uint32_t>(stage * (Cfg::STAGE_BYTES / 16));
          constexpr uint32_t kSfId = (1u << 4) | (1u << 29);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_mxf8(tmem_base, wd + 2 * j, wd + Cfg::W_BYTES / 16 + 2 * j, Cfg::IDESC + q * kSfId, sf, sf + 8,
                      (i > 0 || q > 0 || j > 0) ? 1u : 0u);
          tc_commit(&empty[stage]);
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&sf_empty[buf]);
        if (++buf == Cfg::SF_BUFS) {
          buf = 0;
          sfphase ^= 1u;
        }
      }
      tc_commit(done);
      if (!mbar_try_wait(done, 0)) {
        uint32_t dummy = 0;
        mbar_wait_slow(done, 0, &dummy, SITE_DRAIN, kWaitLimitNs);
      }
    }
  } else {
    // ------------------------------------------------------------ scales, then this CTA's sums into shared memory
    const int lg = warp & 3;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * lg) << 16);
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint8_t* sw = p.sw + static_cast<int64_t>(blockIdx.x) * p.kb;  // a tile is one block of the weight's rows
    if (kBf16) {
      // x in bf16: a warp takes one of four K blocks (a scale word), four columns a lane, the next four blocks asked for
      // while these are turned into codes
      const int q = warp - 2;
      uint32_t* words = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(recv) + Cfg::RECV_BYTES);  // [2][NT]
      uint2 v[Cfg::X_ROWS];
      uint32_t ww;
      auto fetch = [&](int kb) {
        const int c = (kb + q) * 128 + 4 * lane;
#pragma unroll
        for (int r = 0; r < Cfg::X_ROWS; ++r)
          v[r] = kb + q < kb1 && c < p.K && r < rows
                     ? __ldca(reinterpret_cast<const uint2*>(p.x + static_cast<int64_t>(t0 + r) * p.K + c))
                     : make_uint2(0u, 0u);
        ww = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ww |= static_cast<uint32_t>(kb + i < kb1 ? __ldcg(sw + kb + i) : 127) << (8 * i);
      };
      fetch(kb0);
      int half = 0;
      for (int kb = kb0; kb < kb1; kb += 4, half ^= 1) {
        const uint32_t a[4] = {ww, ww, ww, ww};
        uint32_t codes[Cfg::X_ROWS];
#pragma unroll
        for (int r = 0; r < Cfg::X_ROWS; ++r) {
          const uint32_t m2 = __vmaxu2(v[r].x & 0x7fff7fffu, v[r].y & 0x7fff7fffu);
          const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16)) << 16);
          const float2 lo = unpack_bf16x2(v[r].x), hi = unpack_bf16x2(v[r].y);
          const float k = scale_inverse(byte);
          codes[r] = byte == kScaleNan ? kCodeNan4 : e4m3x4(lo.x * k, lo.y * k, hi.x * k, hi.y * k);
          if (lane == 0) reinterpret_cast<uint8_t*>(words + half * NT + r)[q] = static_cast<uint8_t>(byte);
        }
        if (kb + 4 < kb1) fetch(kb + 4);
        const int i = kb - kb0 + q;  // the block's place in the ring
        if (i < num_kb) {
          const int stage = i % Cfg::STAGES;
          // after a failed wait the warp only keeps the others company at the barrier below
          ok = ok && warp_wait(&empty[stage], (static_cast<uint32_t>(i / Cfg::STAGES) & 1u) ^ 1u, p.err, SITE_EMPTY);
          uint8_t* xt = stage_base + stage * Cfg::STAGE_BYTES + Cfg::W_BYTES;
#pragma unroll
          for (int r = 0; r < Cfg::X_ROWS; ++r)
            if (ok && r < rows)
              *reinterpret_cast<uint32_t*>(xt + r * 128 + (((lane >> 2) ^ r) << 4) + 4 * (lane & 3)) = codes[r];
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&full[stage]);
        }
        asm volatile("bar.sync 2, 128;" ::: "memory");  // the rows' scale words
        const uint32_t b[4] = {lane < rows ? words[half * NT + lane] : kScaleOnes, kScaleOnes, kScaleOnes, kScaleOnes};
        ok = ok && warp_wait(&sf_empty[buf], phase ^ 1u, p.err, SITE_SF_EMPTY);
        if (!ok) continue;
        tc_fence_after_sync();
        const uint32_t at = lane_addr + static_cast<uint32_t>(Cfg::SF_BASE + buf * Cfg::SF_COLS);
        tmem_st_32x32b_x4(at, a);
        tmem_st_32x32b_x4(at + 8, b);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[buf]);
        if (++buf == Cfg::SF_BUFS) {
          buf = 0;
          phase ^= 1u;
        }
      }
    } else {
      ScaleFeed<NT, 1> feed;
      feed.smem = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(recv) + Cfg::RECV_BYTES);
      feed.sa = p.sx;
      feed.sb = sw;
      feed.sb_n = 0;
      feed.sb_k = 1;
      feed.ka = p.kb;
      feed.rows = p.M;
      feed.blocks = 1;
      feed.tid = static_cast<int>(threadIdx.x) - 64;
      feed.wide = ((p.kb | kb0) & 15) == 0 && (reinterpret_cast<uintptr_t>(p.sx) & 15) == 0;
      feed.fetch(t0, 0, kb0, kb1);
      int half = 0;
      for (int kb = kb0; kb < kb1; kb += 16, half ^= 1) {
        feed.publish(half);
        if (kb + 16 < kb1) feed.fetch(t0, 0, kb + 16, kb1);
        for (int g = 0; g < 4 && kb + 4 * g < kb1; ++g) {
          const uint32_t ww = feed.block(half, g, 0);
          const uint32_t a[4] = {ww, ww, ww, ww};
          uint32_t b[4] = {kScaleOnes, kScaleOnes, kScaleOnes, kScaleOnes};
  #pragma unroll
          for (int j = 0; j < Cfg::X_WORDS; ++j) b[j] = feed.row(half, g, (lane + 32 * j) & (NT - 1));
          // after a failed wait the warp only keeps the others company at the feed's barrier
          ok = ok && warp_wait(&sf_empty[buf], phase ^ 1u, p.err, SITE_SF_EMPTY);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t at = lane_addr + static_cast<uint32_t>(Cfg::SF_BASE + buf * Cfg::SF_COLS);
          tmem_st_32x32b_x4(at, a);
          tmem_st_32x32b_x4(at + 8, b);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_full[buf]);
          if (++buf == Cfg::SF_BUFS) {
            buf = 0;
            phase ^= 1u;
          }
        }
      }
    }
    const bool aborted = ld_volatile_u32(p.err) != 0u;  // a failure of an earlier call: nothing is stored
    ok = ok && warp_wait(done, 0, p.err, SITE_TFULL);
    tc_fence_after_sync();
    cluster_wait();
    if (Cfg::BULK) {
      float* mine = reinterpret_cast<float*>(stage_base) + (32 * lg + lane) * Cfg::ROW_F;
      if (ok) {
#pragma unroll
        for (int c = 0; c < NT; c += 32) {
          if (c >= rows) break;
          uint32_t r[32];
          tmem_ld_32x32b_x32(lane_addr + c, r);
          tmem_ld_wait();
          tmem_regs_after_wait(r);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(mine + c + 4 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
        fence_proxy_async_smem();
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const int to = static_cast<int>(threadIdx.x) - 64;
      if (ok && to < split)
        dsmem_bulk_copy(mapa_shared(smem_u32(recv + f_first * Cfg::ROW_F), to),
                        smem_u32(reinterpret_cast<float*>(stage_base) + to * f_count * Cfg::ROW_F),
                        static_cast<uint32_t>(f_count * Cfg::ROW_F) * 4u, mapa_shared(smem_u32(arrived), to));
    } else if (ok) {
      // thread = feature: its sums go to the CTA that adds this feature up
      const int f = 32 * lg + lane;
      const int to = f / f_count;
      const uint32_t dst = mapa_shared(smem_u32(recv + (f_first + f % f_count) * Cfg::ROW_F), to);
      const uint32_t bar = mapa_shared(smem_u32(arrived), to);
#pragma unroll
      for (int c = 0; c < NT; c += 32) {
        if (c >= rows) break;
        uint32_t r[32];
        tmem_ld_32x32b_x32(lane_addr + c, r);
        tmem_ld_wait();
        tmem_regs_after_wait(r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + 4 * i < rows)
            st_async_v4(dst + static_cast<uint32_t>(c + 4 * i) * 4u, __uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                        __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]), bar);
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    const bool summed = warp_wait(arrived, 0, p.err, SITE_CLOAD);
    if (!summed) __nanosleep(100000);  // failed: let what is still under way land before shared memory goes back
    // Only now: once all CTAs have what they receive, every bulk copy has read its source in the sender's stages too.
    // Its completion is counted at the receiver alone, so an arrival right after sending would let the sender go.
    cluster_arrive();
    if (summed && !aborted) {
      // four rows of two neighbouring features a thread: a warp stores 128 bytes of each row
      const int pairs = f_count / 2;
      for (int u = static_cast<int>(threadIdx.x) - 64; u < rows4 * pairs; u += 128) {
        const int t4 = u / pairs, f = 2 * (u - t4 * pairs);
        const int n = n0 + f_first + f;
        if (n >= p.N) continue;
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
        for (int r = 0; r < split; ++r) {
          const float* at = recv + (r * f_count + f) * Cfg::ROW_F + 4 * t4;
          const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + Cfg::ROW_F);
          v0.x += a.x;
          v0.y += a.y;
          v0.z += a.z;
          v0.w += a.w;
          v1.x += b.x;
          v1.y += b.y;
          v1.z += b.z;
          v1.w += b.w;
        }
        const float2 bias = p.bias ? unpack_bf16x2(__ldca(reinterpret_cast<const uint32_t*>(p.bias + n))) : make_float2(0.f, 0.f);
        const uint32_t o[4] = {pack_bf16x2(v0.x + bias.x, v1.x + bias.y), pack_bf16x2(v0.y + bias.x, v1.y + bias.y),
                               pack_bf16x2(v0.z + bias.x, v1.z + bias.y), pack_bf16x2(v0.w + bias.x, v1.w + bias.y)};
        uint32_t* y = reinterpret_cast<uint32_t*>(p.y + static_cast<int64_t>(t0 + 4 * t4) * p.N + n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * t4 + i < rows) y[static_cast<int64_t>(i) * (p.N / 2)] = o[i];
      }
    }
  }
  if (warp < 2) {
    __syncwarp();
    cluster_wait();
    cluster_arrive();
  }
  cluster_wait();  // no CTA leaves while a peer may still send to it or copy out of it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

int few_tile(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

template <int NT, bool kBf16 = false>
cudaError_t few_launch(const CUtensorMap& w, const CUtensorMap& x, const FewParams& p, int split, const DeviceInfo& dev,
                       cudaStream_t s) {
  using Cfg = FewCfg<NT, kBf16>;
  auto kern = mx_few_kernel<NT, kBf16>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), Cfg::SMEM_BYTES, dev.device);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters_z(kern, dim3((p.N + Cfg::BM - 1) / Cfg::BM, (p.M + NT - 1) / NT, split), dim3(Cfg::NUM_THREADS),
                               Cfg::SMEM_BYTES, s, w, x, p);
}

}  // namespace

MxFewPlan mx_few_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  MxFewPlan plan;
  plan.nt = few_tile(M);
  const int64_t kb = (K + 127) / 128;
  // CTAs that run at once: two an SM, one with tiles of 128 rows
  const int64_t places = static_cast<int64_t>(dev.num_sms) * (plan.nt == 128 ? 1 : 2);
  const int64_t tiles = (N + 127) / 128 * ((M + plan.nt - 1) / plan.nt);
  // K is split while the CTAs keep to 85 of 100 places (clusters do not fit into all of them: 48 clusters of 6 took
  // 12.8 us where 48 of 5 took 10.3) and have two K blocks each; eight ways for long K only (4096 to 4096, one row:
  // 7.6 us four ways, 8.2 eight; 14336 to 4096, 24 rows: 16.4 and 16.6).
  plan.split = 1;
  for (int c = 2; c <= FewCfg<16, false>::MAX_SPLIT; c *= 2)
    if (tiles * c * 100 <= places * 85 && kb >= (c == 8 ? 64 : 2 * c)) plan.split = c;
  // Above 64 rows the tiles of dg_mx.cuh may take less time.  Both sides measured at 11, 32 and 112 K blocks and 96 to 512
  // rows: here about 11 us and 0.3 us a K block of a CTA, there 7.3 us and a turn's K blocks at 0.2 us (tiles of 128
  // columns) or 0.245 us (192 rows: 16.8 against 13.4 us for 4096 to 4096, 27.6 against 30.5 us for 14336 to 4096).
  int64_t turns;
  const int unit = mx_tile_n(false, M, N, dev, &turns) == 128 ? 16 : 20;
  const int64_t waves = (tiles * plan.split + places - 1) / places, blocks = (kb + plan.split - 1) / plan.split;
  plan.better = M <= 64 || (M <= 512 && 300 + 25 * waves * blocks < unit * turns * kb);
  return plan;
}

cudaError_t launch_mx_few(const MxFewPlan& plan, const CUtensorMap& w, const CUtensorMap& x, const void* sw,
                          const void* sx, const void* bias, void* y, int M, int N, int K, const DeviceInfo& dev,
                          cudaStream_t s) {
  const FewParams p{M, N, K, (K + 127) / 128, nullptr, static_cast<const uint8_t*>(sx),
                    static_cast<const uint8_t*>(sw), static_cast<const __nv_bfloat16*>(bias),
                    static_cast<__nv_bfloat16*>(y), dev.err};
  switch (plan.nt) {
    case 16: return few_launch<16>(w, x, p, plan.split, dev, s);
    case 32: return few_launch<32>(w, x, p, plan.split, dev, s);
    case 64: return few_launch<64>(w, x, p, plan.split, dev, s);
    default: return few_launch<128>(w, x, p, plan.split, dev, s);
  }
}

cudaError_t launch_mx_few_bf16(const MxFewPlan& plan, const CUtensorMap& w, const void* x, const void* sw,
                               const void* bias, void* y, int M, int N, int K, const DeviceInfo& dev, cudaStream_t s) {
  const FewParams p{M, N, K, (K + 127) / 128, static_cast<const __nv_bfloat16*>(x), nullptr,
                    static_cast<const uint8_t*>(sw), static_cast<const __nv_bfloat16*>(bias),
                    static_cast<__nv_bfloat16*>(y), dev.err};
  return few_launch<16, true>(w, w, p, plan.split, dev, s);
}

}  // namespace dg
