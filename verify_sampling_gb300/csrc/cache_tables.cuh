// Launchers of the paged-cache bookkeeping kernels (cache_tables.cu).
#pragma once

#include "common.cuh"

namespace spec {

cudaError_t launch_cache_reserve(const spec_cache_reserve_args& a, cudaStream_t stream);
cudaError_t launch_cache_commit(const spec_cache_commit_args& a, cudaStream_t stream);

}  // namespace spec
