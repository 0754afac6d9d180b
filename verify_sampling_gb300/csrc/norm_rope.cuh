// Launchers of the head norms with rotary positions and of the packed cache's read-back (norm_rope.cu).
#pragma once

#include "common.cuh"

namespace spec {

constexpr int kNormRopeMaxDim = 512;

cudaError_t launch_norm_rope(const spec_norm_rope_args& a, cudaStream_t stream);
cudaError_t launch_cache_read(const spec_cache_read_packed_args& a, cudaStream_t stream);

}  // namespace spec
