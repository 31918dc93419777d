// Instantiation unit of the grouped tensor-memory kernel (GU_OP, GU_FP8,
// GU_ROWM, GU_MT, GU_CHAIN, GU_ANY set by the including file).
#include "grouped_umma.cuh"

namespace moe {

namespace {
const auto gu_kernel = grouped_umma_kernel<GU_OP, GU_FP8, GU_ROWM, GU_MT, GU_CHAIN, GU_ANY>;

cudaLaunchConfig_t gu_config(int pairs, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(gu_threads(GU_ANY));
  cfg.dynamicSmemBytes = gu_smem();
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}
}  // namespace

template <>
bool gu_launch<GU_OP, GU_FP8, GU_ROWM, GU_MT, GU_CHAIN, GU_ANY>(const GuParams& p, int pairs, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gu_config(pairs, s, attr);
  return cudaLaunchKernelEx(&cfg, gu_kernel, static_cast<const GuKernelParams<GU_FP8, GU_ANY>&>(p)) == cudaSuccess;
}

template <>
int gu_pairs<GU_OP, GU_FP8, GU_ROWM, GU_MT, GU_CHAIN, GU_ANY>() {
  if (cudaFuncSetAttribute(gu_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)gu_smem()) != cudaSuccess)
    return GU_QUERY_FAILED;
  // The register hand-over of these kernels counts on what the block starts
  // with: with fewer its epilogue would wait for ever (the build checks it too).
  cudaFuncAttributes fa;
  if (GU_ANY || gu_hand_over(GU_MT, GU_CHAIN)) {
    if (cudaFuncGetAttributes(&fa, gu_kernel) != cudaSuccess) return GU_QUERY_FAILED;
    if ((fa.numRegs + 7) / 8 * 8 != gu_launch_regs(GU_ANY)) return GU_REGISTERS;
  }
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gu_config(1, nullptr, attr);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gu_kernel, &cfg) != cudaSuccess) return GU_QUERY_FAILED;
  return n < kGuPairsMax ? n : kGuPairsMax;
}

}  // namespace moe
