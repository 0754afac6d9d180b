// Launcher of the logit-adjustment kernel (logits.cu).
#pragma once

#include "common.cuh"

namespace spec {

cudaError_t launch_adjust_logits(const spec_logits_args& a, cudaStream_t stream);

}  // namespace spec
