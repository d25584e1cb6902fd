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

cudaError_t launch_gemm_mx(bool b_mn_major, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d,
                           const MxParams& p, const DeviceInfo& dev, cudaStream_t s) {
  return b_mn_major ? launch_mx<true, kMxTileN>(a, b, d, p, dev, s) : launch_mx<false, kMxTileN>(a, b, d, p, dev, s);
}

}  // namespace dg
