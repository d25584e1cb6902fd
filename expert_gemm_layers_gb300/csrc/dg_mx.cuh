// Persistent tcgen05 GEMM on e4m3 operands with power-of-two block scales
// (sm_103a, CTA pairs): D[m, n] = bias[n] + sum_k a[m, k] b[n, k] with
//   a = A code * 2^(sa[m, k/128] - 127),  b = B code * 2^(sb[n/128, k/128] - 127).
//
// The scales are applied by the tensor core itself: tcgen05.mma with
// .kind::mxf8f6f4.block_scale reads one e8m0 byte per row and 32 values of K from
// TMEM, so the accumulator needs no promotion in registers at block borders.  The
// operands' blocks are 128 long, so the four K steps of a stage read the same byte;
// a 32-bit TMEM word holds the bytes of four K blocks and the instruction
// descriptor's scale index picks one.  Scales therefore move once every 512 K.
//
// Warp roles (320 threads a CTA):
//   warp 0      TMA producer: ring of (A, B) K blocks of 128 bytes a row
//   warp 1      MMA issuer (pair leader, one lane)
//   warps 2-5   epilogue: TMEM -> + bias -> bf16 -> swizzled staging -> TMA store
//   warps 6-9   scales: global bytes -> shared memory -> tcgen05.st into one of four
//               TMEM buffers (every warp writes its own lane quarter: the layout
//               wants row r's word in lane r % 32 of all quarters, column r / 32)
// TMEM: two accumulators of BN columns (224 or 128) and, in the last 64, the scale
// buffers; 224 is what two accumulators can have beside them.  Bound by the tensor
// core: 8192 x 14336 to 4096 in 272 to 280 us, 3430 to 3530 TFLOP/s.
//
// B is K-major ([N][K], the forward) or MN-major ([K][N], the input gradient, whose
// contraction runs over the weight's rows): the weight's codes are held once.
#pragma once

#include "dg_gemm.cuh"

namespace dg {

struct MxParams {
  int32_t M, N;
  int32_t tiles_m, tiles_n, n_fastest;
  const uint8_t* sa;         // [M][ka]: e8m0 bytes of A's rows
  int32_t ka;                // K blocks = ceil(K / 128)
  const uint8_t* sb;         // byte of column block nb and K block kb at sb[nb * sb_n + kb * sb_k]
  int32_t sb_n, sb_k;
  const __nv_bfloat16* bias; // [N] or NULL
  uint32_t* err;
};

enum MxSite : uint32_t { SITE_SF_EMPTY = 8, SITE_SF_FULL = 9 };

template <bool kBMN, int kBN>
struct MxCfg {
  static constexpr int CTAS = 2;
  static constexpr int BM = 128;
  static constexpr int UMMA_M = 256;
  static constexpr int BN = kBN;
  static constexpr int B_ROWS = BN / CTAS;
  static constexpr int BK = 128;
  static constexpr int K_STEPS = 4;
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = BM * 128;
  // MN-major: 128 K rows of 128 bytes, of which the MMA reads B_ROWS columns
  static constexpr int B_BYTES = kBMN ? 128 * 128 : B_ROWS * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int EPI_WARPS = 4;
  static constexpr int CHUNK = 32;                     // output columns per staging buffer
  static constexpr int EPI_BUF_BYTES = 32 * CHUNK * 2;
  static constexpr int EPI_BUFS = 2;                   // staging buffers a warp (four: no change)
  static constexpr int EPI_BYTES = EPI_WARPS * EPI_BUFS * EPI_BUF_BYTES;
  static constexpr int SF_WARPS = 4;
  static constexpr int SF_BUFS = 4;
  static constexpr int SF_COLS = 16;                   // A words at +0, B words at +8
  static constexpr int SF_BASE = 512 - SF_BUFS * SF_COLS;
  static constexpr int NB_WORDS = BN / 32;
  static constexpr int NB_BLOCKS = (BN + 127 + 127) / 128;  // 128-column blocks that a tile can touch
  static constexpr int NUM_THREADS = 64 + 32 * (EPI_WARPS + SF_WARPS);
  static constexpr int NUM_BARS = 2 * STAGES + 4 + 2 * SF_BUFS + 1;
  static constexpr int BAR_BYTES = 256;
  static constexpr int FEED_BYTES = (2 * 4 * (BM + 4) * 4 + 15) / 16 * 16;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + FEED_BYTES + BAR_BYTES;
  // kind::mxf8f6f4 instruction descriptor: e4m3 x e4m3, majorness, N, e8m0 scales (bit 23),
  // M; bits 4-5 and 29-30 (scale index of B and A) are filled in per K block
  static constexpr uint32_t IDESC = (static_cast<uint32_t>(kBMN) << 16) | ((BN >> 3) << 17) | (1u << 23) |
                                    ((UMMA_M >> 4) << 24);
  static_assert(NUM_BARS * 8 + 4 <= BAR_BYTES, "barrier area");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(2 * BN <= SF_BASE && BN % 32 == 0 && NB_WORDS <= 8, "tensor memory");
  static_assert(STAGE_BYTES % 1024 == 0 && A_BYTES % 1024 == 0, "swizzled tiles");
  static_assert(!kBMN || B_ROWS <= 128, "one 128-byte MN block a CTA");
};

// D(tmem of both CTAs) (+)= (A x scales) (B x scales), e4m3, one e8m0 scale per 32 K.
static __device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                      uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

static __device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Thread i of the warp writes lane (base + i), columns col..col+N-1.
static __device__ __forceinline__ void tmem_st_32x32b_x4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
static __device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
static __device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Arrive once on an mbarrier given by its shared::cluster address, with the default release at CTA scope: what it
// orders here are tcgen05 accesses that have completed (wait::ld, wait::st) and been fenced.  A release at cluster
// scope waits for the thread's memory accesses to reach that scope, up to a microsecond.
static __device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Cluster barrier in two halves: every thread of the cluster arrives, and waits later.  The arrival is relaxed, for
// where no memory is passed on (barriers' initialisation has a fence of its own) and none of the thread's accesses to
// a peer can still be under way: a releasing one first waits for the thread's accesses, 2000 cycles in a prologue that
// has just asked for memory.
static __device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
static __device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// mbar_wait by a whole warp: all lanes go on or none does.
static __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, site));
}

// One lane of a converged warp, the same one every time.  Under `if (elect_one())` the compiler knows that a single
// lane issues the copies and MMAs: a stage's four MMAs took 115 cycles to issue and its two copies 290, against 350
// and 400 under `lane == 0` (clock64).
static __device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(v)
      :
      : "memory");
  return v != 0u;
}

constexpr uint32_t kScaleOnes = 0x7f7f7f7fu;  // four scales of 1

// How 128 threads bring block scales to the words that tcgen05.st writes, 16 K blocks at a time: the bytes of kRows
// rows (K blocks next to one another) and of up to kBlocks 128-blocks of the other operand go through registers
// (fetch, a batch ahead) into shared memory (publish), each byte once.  Fetched word by word in every warp and waited
// for at once they came every 2400 cycles per 512 K, five times slower than the tensor core uses them; rows whose
// length is no multiple of 16 blocks cost 32 sectors an instruction.
template <int kRows, int kBlocks>
struct ScaleFeed {
  static constexpr int PER = kRows / 8;  // narrow: two rows an instruction and warp
  uint32_t* smem;                        // [2][4 groups][kRows + 4]: rows, then blocks
  const uint8_t *sa, *sb;
  int64_t sb_n, sb_k;
  int ka, rows, blocks;                  // bytes of a row; rows and blocks that exist
  int tid;
  bool wide;                             // rows can be read in 16 bytes
  uint32_t v[PER < 4 ? 4 : PER], w;

  __device__ __forceinline__ void fetch(int row0, int block0, int kb, int kend) {
    const int warp = tid >> 5, lane = tid & 31;
    if (wide) {
      uint4 q = make_uint4(kScaleOnes, kScaleOnes, kScaleOnes, kScaleOnes);
      if (tid < kRows && row0 + tid < rows)
        q = __ldcg(reinterpret_cast<const uint4*>(sa + static_cast<int64_t>(row0 + tid) * ka + kb));
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
      v[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int r = row0 + warp * (kRows / 4) + 2 * i + (lane >> 4), k = kb + (lane & 15);
        v[i] = r < rows && k < kend ? __ldcg(sa + static_cast<int64_t>(r) * ka + k) : 127u;
      }
    }
    const int k = kb + lane;
    w = warp < kBlocks && lane < 16 && block0 + warp < blocks && k < kend ? __ldcg(sb + (block0 + warp) * sb_n + k * sb_k)
                                                                         : 127u;
  }
  __device__ __forceinline__ void publish(int half) {
    const int warp = tid >> 5, lane = tid & 31;
    uint32_t* at = smem + half * 4 * (kRows + 4);
    if (wide) {
      if (tid < kRows)
#pragma unroll
        for (int g = 0; g < 4; ++g) at[g * (kRows + 4) + tid] = v[g];
    } else {
      uint8_t* bytes = reinterpret_cast<uint8_t*>(at + ((lane & 15) >> 2) * (kRows + 4)) + (lane & 3);
#pragma unroll
      for (int i = 0; i < PER; ++i) bytes[4 * (warp * (kRows / 4) + 2 * i + (lane >> 4))] = static_cast<uint8_t>(v[i]);
    }
    if (warp < kBlocks && lane < 16)
      reinterpret_cast<uint8_t*>(at + (lane >> 2) * (kRows + 4) + kRows + warp)[lane & 3] = static_cast<uint8_t>(w);
    asm volatile("bar.sync 2, 128;" ::: "memory");
  }
  __device__ __forceinline__ uint32_t row(int half, int g, int r) const { return smem[(half * 4 + g) * (kRows + 4) + r]; }
  __device__ __forceinline__ uint32_t block(int half, int g, int b) const {
    return smem[(half * 4 + g) * (kRows + 4) + kRows + b];
  }
};

template <bool kBMN, int kBN>
__global__ void __launch_bounds__(MxCfg<kBMN, kBN>::NUM_THREADS, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmD, const MxParams p) {
  using Cfg = MxCfg<kBMN, kBN>;
  extern __shared__ uint8_t smem_raw[];

  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stage_base = smem_raw + pad;
  uint8_t* epi_base = stage_base + Cfg::STAGES * Cfg::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi_base + Cfg::EPI_BYTES + Cfg::FEED_BYTES);
  uint64_t* empty = full + Cfg::STAGES;
  uint64_t* tfull = empty + Cfg::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* sf_full = tempty + 2;
  uint64_t* sf_empty = sf_full + Cfg::SF_BUFS;
  uint64_t* drain = sf_empty + Cfg::SF_BUFS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0u;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], Cfg::EPI_WARPS * Cfg::CTAS);
    }
    for (int b = 0; b < Cfg::SF_BUFS; ++b) {
      mbar_init(&sf_full[b], Cfg::SF_WARPS * Cfg::CTAS);
      mbar_init(&sf_empty[b], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmD);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  griddep_wait();
  tc_fence_before_sync();
  cluster_arrive();
  cluster_wait();
  __syncthreads();  // the TMEM address in shared memory
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;

  const int total_tiles = p.tiles_m * p.tiles_n;
  const int num_kb = p.ka;
  const int unit = static_cast<int>(blockIdx.x) / Cfg::CTAS;
  const int num_units = static_cast<int>(gridDim.x) / Cfg::CTAS;
  auto coords = [&](int tile, int& mt, int& nt) {
    if (p.n_fastest) {
      mt = tile / p.tiles_n;
      nt = tile - mt * p.tiles_n;
    } else {
      nt = tile / p.tiles_m;
      mt = tile - nt * p.tiles_m;
    }
  };

  // After a failure recorded earlier the pipeline still runs (or gives up at its first long wait, which looks
  // at the error word) but nothing is stored: that way no CTA waits for the word before its first copy.
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += num_units) {
        int mt, nt;
        coords(tile, mt, nt);
        const int m0 = mt * Cfg::UMMA_M + static_cast<int>(rank) * Cfg::BM;
        const int n0 = nt * Cfg::BN + static_cast<int>(rank) * Cfg::B_ROWS;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, SITE_EMPTY)) {
            ok = false;
            break;
          }
          // the pair's copies all complete on the leader's barrier
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          uint8_t* sa = stage_base + stage * Cfg::STAGE_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES * Cfg::CTAS);
          tma_load_3d_pair(sa, &tmA, bar, kb * Cfg::BK, m0, 0);
          if (kBMN)
            tma_load_3d_pair(sa + Cfg::A_BYTES, &tmB, bar, n0, kb * Cfg::BK, 0);
          else
            tma_load_3d_pair(sa + Cfg::A_BYTES, &tmB, bar, kb * Cfg::BK, n0, 0);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every load issued must land before the CTA exits
      for (int s = 0; s < Cfg::STAGES; ++s)
        if (leader && (armed & (1u << s)) && !mbar_try_wait(&full[s], (armed_parity >> s) & 1u)) {
          uint32_t dummy = 0;
          mbar_wait_slow(&full[s], (armed_parity >> s) & 1u, &dummy, SITE_DRAIN, kWaitLimitNs);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (pair leader)
    if (leader && elect_one()) {
      int stage = 0, sfb = 0;
      uint32_t phase = 0, tphase = 0, sfphase = 0;
      bool ok = true;
      int local = 0;
      // K-major: 32 bytes on in the swizzle row per K step.  MN-major: 32 K rows of 128 bytes on;
      // groups of 8 K rows lie 1024 bytes apart.
      const uint64_t a0 = smem_desc_sw128(smem_u32(stage_base), 16, 1024);
      const uint64_t b0 = smem_desc_sw128(smem_u32(stage_base) + Cfg::A_BYTES, kBMN ? 128 * 128 : 16, 1024);
      for (int tile = unit; tile < total_tiles && ok; tile += num_units, ++local) {
        const int acc = local & 1;
        if (!mbar_wait(&tempty[acc], ((tphase >> acc) & 1u) ^ 1u, p.err, SITE_TEMPTY)) break;
        tphase ^= 1u << acc;
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Cfg::BN);
        // four K blocks a turn, straight through: what lies between one block's MMAs and the next one's leaves the
        // tensor core without work
        for (int kb = 0; kb < num_kb && ok; kb += 4) {
          if (!mbar_wait(&sf_full[sfb], sfphase, p.err, SITE_SF_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sf = tmem_base + static_cast<uint32_t>(Cfg::SF_BASE + sfb * Cfg::SF_COLS);
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            if (kb + static_cast<int>(q) >= num_kb) break;
            ok = ok && mbar_wait(&full[stage], phase, p.err, SITE_FULL);
            if (!ok) break;
            const uint64_t ad = a0 + static_cast<uint32_t>(stage * (Cfg::STAGE_BYTES / 16));
            const uint64_t bd = b0 + static_cast<uint32_t>(stage * (Cfg::STAGE_BYTES / 16));
            constexpr uint32_t kScaleId = (1u << 4) | (1u << 29);
#pragma unroll
            for (int j = 0; j < Cfg::K_STEPS; ++j)
              umma_mxf8_pair(d_tmem, ad + 2 * j, bd + (kBMN ? 256 : 2) * j, Cfg::IDESC + q * kScaleId, sf, sf + 8,
                             (kb > 0 || q > 0 || j > 0) ? 1u : 0u);
            tc_commit_pair_mc(&empty[stage], 0x3);
            if (++stage == Cfg::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit_pair_mc(&sf_empty[sfb], 0x3);
          if (++sfb == Cfg::SF_BUFS) {
            sfb = 0;
            sfphase ^= 1u;
          }
        }
        if (ok) tc_commit_pair_mc(&tfull[acc], 0x3);
      }
      // every MMA issued must complete before TMEM is released
      tc_commit_pair_mc(drain, 0x1);
      if (!mbar_try_wait(drain, 0)) {
        uint32_t dummy = 0;
        mbar_wait_slow(drain, 0, &dummy, SITE_DRAIN, kWaitLimitNs);
      }
    }
  } else if (warp < 2 + Cfg::EPI_WARPS) {
    // ------------------------------------------------------------ epilogue
    const int lg = warp & 3;
    uint8_t* stg = epi_base + (warp - 2) * Cfg::EPI_BUFS * Cfg::EPI_BUF_BYTES;
    uint32_t tphase = 0, ctr = 0;
    const bool aborted = ld_volatile_u32(p.err) != 0u;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * lg) << 16);
    int local = 0;
    for (int tile = unit; tile < total_tiles; tile += num_units, ++local) {
      int mt, nt;
      coords(tile, mt, nt);
      const int row0 = mt * Cfg::UMMA_M + static_cast<int>(rank) * Cfg::BM + 32 * lg;
      const int n0 = nt * Cfg::BN;
      const int acc = local & 1;
      int nchunks = (min(p.N - n0, Cfg::BN) + Cfg::CHUNK - 1) / Cfg::CHUNK;
      if (row0 >= p.M) nchunks = 0;
      if (!warp_wait(&tfull[acc], (tphase >> acc) & 1u, p.err, SITE_TFULL)) break;
      tphase ^= 1u << acc;
      tc_fence_after_sync();
      auto release_acc = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(mapa_shared(smem_u32(&tempty[acc]), 0));
      };
      if (nchunks == 0) release_acc();
      auto store_chunk = [&](const uint32_t (&r)[32], int c0) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
        if (p.bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (c0 + 8 * q < p.N) {
              const uint4 bv = __ldca(reinterpret_cast<const uint4*>(p.bias + c0 + 8 * q));
              const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 b2 = unpack_bf16x2(bw[e]);
                v[8 * q + 2 * e] += b2.x;
                v[8 * q + 2 * e + 1] += b2.y;
              }
            }
          }
        }
        uint8_t* sbuf = stg + (ctr & (Cfg::EPI_BUFS - 1)) * Cfg::EPI_BUF_BYTES;
        ++ctr;
        // the store that last read this buffer must be done
        if (lane == 0) bulk_wait_group_read<Cfg::EPI_BUFS - 1>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(sbuf + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                         pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !aborted) {
          tma_store_3d(&tmD, sbuf, c0, row0, 0);
          bulk_commit_group();
        }
      };
      const uint32_t acc_addr = lane_addr + static_cast<uint32_t>(acc * Cfg::BN);
      for (int j = 0; j < nchunks; j += 2) {
        uint32_t r0[32], r1[32];
        const bool two = j + 1 < nchunks;
        tmem_ld_32x32b_x32(acc_addr + static_cast<uint32_t>(Cfg::CHUNK * j), r0);
        if (two) tmem_ld_32x32b_x32(acc_addr + static_cast<uint32_t>(Cfg::CHUNK * (j + 1)), r1);
        tmem_ld_wait();
        tmem_regs_after_wait(r0);
        tmem_regs_after_wait(r1);
        if (j + 2 >= nchunks) release_acc();
        store_chunk(r0, n0 + Cfg::CHUNK * j);
        if (two) store_chunk(r1, n0 + Cfg::CHUNK * (j + 1));
      }
    }
    if (lane == 0) bulk_wait_group_read<0>();  // the staging buffers have been read
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scales
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    ScaleFeed<Cfg::BM, Cfg::NB_BLOCKS> feed;
    feed.smem = reinterpret_cast<uint32_t*>(epi_base + Cfg::EPI_BYTES);
    feed.sa = p.sa;
    feed.sb = p.sb;
    feed.sb_n = p.sb_n;
    feed.sb_k = p.sb_k;
    feed.ka = p.ka;
    feed.rows = p.M;
    feed.blocks = (p.N + 127) / 128;
    feed.tid = static_cast<int>(threadIdx.x) - (Cfg::NUM_THREADS - 128);
    feed.wide = (p.ka & 15) == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15) == 0;
    auto fetch = [&](int tile, int kb) {
      int mt, nt;
      coords(tile, mt, nt);
      feed.fetch(mt * Cfg::UMMA_M + static_cast<int>(rank) * Cfg::BM, (nt * Cfg::BN) >> 7, kb, num_kb);
    };
    int buf = 0, half = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (unit < total_tiles) fetch(unit, 0);
    for (int tile = unit; tile < total_tiles; tile += num_units) {
      int mt, nt;
      coords(tile, mt, nt);
      const int n0 = nt * Cfg::BN;
      for (int kb = 0; kb < num_kb; kb += 16, half ^= 1) {
        feed.publish(half);
        if (kb + 16 < num_kb)
          fetch(tile, kb + 16);
        else if (tile + num_units < total_tiles)
          fetch(tile + num_units, 0);
        for (int g = 0; g < 4 && kb + 4 * g < num_kb; ++g) {
          uint32_t a[4], b[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = feed.row(half, g, lane + 32 * j);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            b[j] = j < Cfg::NB_WORDS ? feed.block(half, g, ((n0 + lane + 32 * j) >> 7) - (n0 >> 7)) : kScaleOnes;
          // after a failed wait the warp only keeps the others company at the feed's barrier
          ok = ok && warp_wait(&sf_empty[buf], phase ^ 1u, p.err, SITE_SF_EMPTY);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t at = lane_addr + static_cast<uint32_t>(Cfg::SF_BASE + buf * Cfg::SF_COLS);
          tmem_st_32x32b_x4(at, a);
          tmem_st_32x32b_x8(at + 8, b);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(mapa_shared(smem_u32(&sf_full[buf]), 0));
          if (++buf == Cfg::SF_BUFS) {
            buf = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  }

  // The last arrivals on the leader's `tempty` have no reader; this barrier, whose arrival releases, is what keeps the
  // leader's shared memory until they have landed.
  griddep_launch_dependents();
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace dg
