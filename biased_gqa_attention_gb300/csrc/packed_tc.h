// packed_tc.h -- the tensor-core packed prefill (host side).
#pragma once

#include "packed_plan.cuh"

namespace extkv {

bool packed_tc_supported(int64_t D, int dtype);
// query rows of a work item: two M = 128 tiles
constexpr int kPackedTcRows = 256;
cudaError_t launch_packed_tc(PackedParams& p, uint32_t wait_limit_plus1, cudaStream_t s, const char** name);
cudaError_t launch_packed_tc_d256(const PackedParams& p, cudaStream_t s);

}  // namespace extkv
