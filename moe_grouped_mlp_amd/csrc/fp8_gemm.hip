// Launch of the tiled block-scaled FP8 product (fp8_gemm_kernel.h).
#include "fp8_gemm_kernel.h"

namespace moe {
namespace {

template <int JMAX, bool F32, bool WIDE>
hipError_t launch(const Fp8Args& g, hipStream_t s) {
  fp8_gemm_kernel<JMAX, false, F32, WIDE><<<g.grid, kFp8Threads, 0, s>>>(g);
  if (hipError_t e = hipGetLastError()) return e;
  if (g.part) fp8_join_kernel<JMAX, F32><<<g.grid, kFp8Threads, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Args& g, bool f32, bool wide, int groups, hipStream_t s) {
  if (f32) return groups == 1 ? launch<1, true, true>(g, s) : launch<2, true, true>(g, s);
  if (wide) return groups == 1 ? launch<1, false, true>(g, s) : launch<2, false, true>(g, s);
  if (groups == 1) return launch<1, false, false>(g, s);
  return groups == 2 ? launch<2, false, false>(g, s) : launch<4, false, false>(g, s);
}

}  // namespace moe
