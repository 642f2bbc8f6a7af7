// Launches of the tiled block-scaled FP8 products (fp8_gemm_kernel.h).
#include "fp8_gemm_kernel.h"

namespace moe {

hipError_t launch_fp8_gemm(const Fp8Args& g, int tile_rows, bool f32, int grid, hipStream_t s) {
  auto go = [&](auto kernel) { kernel<<<grid, kFp8Threads, 0, s>>>(g); };
  switch (tile_rows) {
    case 64: f32 ? go(fp8_gemm_kernel<1, false, true>) : go(fp8_gemm_kernel<1, false, false>); break;
    case 128: f32 ? go(fp8_gemm_kernel<2, false, true>) : go(fp8_gemm_kernel<2, false, false>); break;
    default: go(fp8_gemm_kernel<4, false, false>); break;   // bf16 outputs only
  }
  return hipGetLastError();
}

}  // namespace moe
