// Launchers of the RMS norm and int8 kernels (not part of the ABI). Each
// returns the cudaError_t of its launches.
#pragma once

#include "qlora_internal.h"
#include "qlora_i8.h"

namespace qlora {

// Lets a kernel use up to 220 KB (or `most`) of dynamic shared memory. Always the
// same number for a kernel: host threads that launch it at the same time set
// the attribute under each other's feet.
template <class... P>
cudaError_t allow_smem(void (*kernel)(P...), int most = 220 * 1024) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Launches a kernel that reads and writes nothing before grid_dep_wait, so that its
// launch and set-up overlap the end of the work ahead of it on the stream. It saves
// 0.4 to 1.4 us a call in a graph (norm 8 x 4096 1.6 and 2.2 us, one token of
// 14336 x 4096 12.3 and 13.5; norm gradient 8192 x 1024 18.0 and 17.9: nothing) and
// 0.3 to 5.6 us a call launched among others (4096 x 4096 norm 21.7 and 24.4 us, its
// gradient's two launches 27.3 and 32.8). cluster: CTAs of a cluster.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, int cluster,
                             const A &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

cudaError_t launch_i8_quantize(const void *X, bool f32, int64_t M, int64_t K, const float *col_scale, int8_t *codes,
                               float *scale, cudaStream_t st);
cudaError_t launch_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                 cudaStream_t st);

// hf, wf: the stream / the weight is fp32 (else bf16).
cudaError_t launch_rmsnorm_fwd(const uint16_t *X, const void *R, bool hf, const void *w, bool wf, float eps, int64_t M,
                               int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale, cudaStream_t st);
size_t rmsnorm_bwd_ws_bytes(int64_t M, int64_t K);
cudaError_t launch_rmsnorm_bwd(const uint16_t *dY, const void *H, bool hf, const void *w, bool wf, float eps,
                               const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW, void *ws,
                               cudaStream_t st);

}  // namespace qlora
