// Instantiations of the block-scaled e4m3 GEMM and its launcher.
#include "dg_internal.h"
#include "dg_mx.cuh"

namespace dg {

namespace {

template <bool kBMN, int kBN>
cudaError_t launch_mx(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d, MxParams p,
                      const DeviceInfo& dev, cudaStream_t s) {
  using Cfg = MxCfg<kBMN, kBN>;
  auto kern = gemm_mx_kernel<kBMN, kBN>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), Cfg::SMEM_BYTES, dev.device);
  if (e != cudaSuccess) return e;
  p.tiles_m = (p.M + Cfg::UMMA_M - 1) / Cfg::UMMA_M;
  p.tiles_n = (p.N + Cfg::BN - 1) / Cfg::BN;
  // along the longer side fastest, as the bf16 GEMM's order
  p.n_fastest = p.tiles_n < p.tiles_m ? 1 : 0;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x7fffffff - dev.num_sms) return cudaErrorInvalidValue;
  const int64_t pairs = dev.num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(Cfg::NUM_THREADS);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kern, a, b, d, p);
}

}  // namespace

// Tiles of 128 columns take about 0.8 of the time of those of 224 (a K block 0.2 us against 0.245 us), so they are taken
// where they need no more turns of the CTA pairs (512 rows, 4096 to 4096: 13.5 us against 15.2; 1024 rows, where they
// need two turns: 19.6 against 16.7; 8192 rows, 14336 to 4096, 14 against 8 turns: 393 against 277).  As they lie
// (MN-major) the weight's codes come in boxes of 128 columns a CTA, of which such a tile would use half.
int mx_tile_n(bool b_mn_major, int64_t M, int64_t N, const DeviceInfo& dev, int64_t* turns) {
  const int64_t pairs = dev.num_sms / 2, rows = (M + 255) / 256;
  const int64_t wide = (rows * ((N + kMxTileN - 1) / kMxTileN) + pairs - 1) / pairs;
  const int64_t narrow = (rows * ((N + 127) / 128) + pairs - 1) / pairs;
  const bool take = !b_mn_major && 4 * narrow < 5 * wide;
  if (turns) *turns = take ? narrow : wide;
  return take ? 128 : kMxTileN;
}

cudaError_t launch_gemm_mx(bool b_mn_major, int tile_n, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d,
                           const MxParams& p, const DeviceInfo& dev, cudaStream_t s) {
  if (b_mn_major) return launch_mx<true, kMxTileN>(a, b, d, p, dev, s);
  return tile_n == 128 ? launch_mx<false, 128>(a, b, d, p, dev, s) : launch_mx<false, kMxTileN>(a, b, d, p, dev, s);
}

}  // namespace dg
