// Attention over a cache in 4 bits: launchers and sizes.
#pragma once

#include "attention.cuh"

namespace spec {

namespace attn {

constexpr int kNarrowRows = 16;    // query rows of the narrow kernel's largest item
constexpr int kNarrowBlocks = 3;   // blocks an SM, at most

}  // namespace attn

// Partial rows and layout of the narrow kernel beside the wide one's.
inline size_t attn_narrow_rows(int rows, int Hq) {
  return 2 * (size_t)std::min(rows, attn_window_rows(Hq)) * Hq + (size_t)attn::kMaxCtas * attn::kNarrowBlocks * attn::kNarrowRows;
}

// What a call over a packed cache works with: both kernels' pieces.
struct PackedWork {
  float *part, *narrow_part;
  float2 *stat, *narrow_stat;
  int64_t *plan, *narrow_plan;
};

// The tensor-core kernel of attention_tc.cu over a packed cache: the segments of more than `narrow`
// query rows of the packed rows [lo, hi).
cudaError_t launch_attention_wide(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, int lo, int hi, int narrow,
                                  const PackedWork& work, cudaStream_t stream);
bool attn_packed_ok(const spec_prefix_attention_args& a, const q4::Cache& packed, int* sms);
cudaError_t launch_attention_packed(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, const PackedWork& work,
                                    cudaStream_t stream);

}  // namespace spec
