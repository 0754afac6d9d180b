// Launcher of the rotary-position kernel (rope.cu).
#pragma once

#include "common.cuh"

namespace spec {

constexpr int kRopeMaxDim = 512;

cudaError_t launch_rope_cache(const spec_rope_cache_args& a, cudaStream_t stream);

}  // namespace spec
