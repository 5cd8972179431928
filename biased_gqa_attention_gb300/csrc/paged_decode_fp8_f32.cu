// paged_decode_fp8_f32.cu -- the decode over 8-bit pages for fp32 q and y: q and the
// weights as two fp16 parts each.  A part times a code is exact and summed in fp32; the parts hold
// q to 2^-23 of its row's largest element, and a weight to 2^-22 of it or 2^-35 of the largest.
#include "paged_decode_fp8.cuh"

namespace extkv {

cudaError_t launch_paged_fp8_f32(const void* params, int* cluster, int variant, cudaStream_t s) {
  PagedParams p = *static_cast<const PagedParams*>(params);
  const bool two = p.rows == 16;
  cudaError_t e;
  if (p.D == 64) e = two ? launch_fp8_d<float, 64, 2, 32, 8, 12>(p, variant, s) : launch_fp8_d<float, 64, 1, 32, 8, 12>(p, variant, s);
  else if (p.D == 128) e = two ? launch_fp8_d<float, 128, 2, 32, 6, 8>(p, variant, s) : launch_fp8_d<float, 128, 1, 32, 4, 12>(p, variant, s);
  else e = launch_fp8_d<float, 256, 1, 32, 4, 6>(p, variant, s);
  *cluster = p.cluster;
  return e;
}

}  // namespace extkv
