// Shared-prefix attention: what its kernels share, and their launchers.
#pragma once

#include <algorithm>

#include "common.cuh"

namespace spec {

constexpr int kAttnMaxDim = 256;

namespace attn {

constexpr int kMaxCtas = 256;   // blocks of the tensor-core kernel (one an SM)
constexpr int kItemRows = 256;  // query rows of one of its work items
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The packed rows of request r, or none (with a status bit) where its offsets
// leave [0, rows] or descend.
struct Rows {
  int row0, n;
};
__device__ __forceinline__ Rows rows_between(const spec_prefix_attention_args& a, int lo, int hi,
                                             uint32_t* bad) {
  const int row0 = a.row_off[lo], row1 = a.row_off[hi];
  if (row0 < 0 || row1 < row0 || row1 > a.rows) {
    *bad |= SPEC_STATUS_BAD_LEN;
    return Rows{0, 0};
  }
  return Rows{row0, row1 - row0};
}
// Own keys of request r, cut to its page table.
__device__ __forceinline__ int own_keys(const spec_prefix_attention_args& a, int r, uint32_t* bad) {
  const int kv = a.kv_len[r];
  const int64_t most = (int64_t)a.max_pages * a.page_size;
  if (kv < 0 || kv > most) {
    *bad |= SPEC_STATUS_BAD_LEN;
    return kv < 0 ? 0 : (int)most;
  }
  return kv;
}
__device__ __forceinline__ int prefix_keys(const spec_prefix_attention_args& a, int g, uint32_t* bad) {
  const int len = a.prefix_len[g];
  const int64_t most = (int64_t)a.max_prefix_pages * a.page_size;
  if (len < 0 || len > most) {
    *bad |= SPEC_STATUS_BAD_LEN;
    return len < 0 ? 0 : (int)most;
  }
  return len;
}
// Requests [lo, hi) of group g, or none where its offsets leave [0, R] or descend.
__device__ __forceinline__ int2 group_requests(const spec_prefix_attention_args& a, int g, uint32_t* bad) {
  const int lo = a.group_off[g], hi = a.group_off[g + 1];
  if (lo < 0 || hi < lo || hi > a.R) {
    *bad |= SPEC_STATUS_BAD_LEN;
    return make_int2(0, 0);
  }
  return make_int2(lo, hi);
}
__device__ __forceinline__ int page_of(const spec_prefix_attention_args& a, const int32_t* table, int i,
                                       uint32_t* bad) {
  const int page = table[i];
  if (page < 0 || page >= a.n_pages) {
    *bad |= SPEC_STATUS_BAD_PAGE;
    return 0;
  }
  return page;
}
// Last i in [0, n) with off[i] <= v (0 if there is none): the request of a row, the group of a request.
__device__ __forceinline__ int last_at_or_below(const int32_t* off, int n, int v) {
  int lo = 0, hi = n;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace attn

// The tensor-core kernels take packed rows in windows of up to 2^20 query rows (rows x
// heads), one after the other, so that their workspace is bounded: 1.1 GB at heads of 128,
// where 2^25 query rows in one would leave 34 GB of pieces.  A window is thousands of items.
inline int attn_window_rows(int Hq) { return std::max(1, (1 << 20) / Hq); }
// Partial rows (D fp32 values, a maximum and a sum each) that a workspace has room for.
inline size_t attn_partial_rows(int rows, int Hq) {
  return 2 * (size_t)std::min(rows, attn_window_rows(Hq)) * Hq + (size_t)attn::kMaxCtas * attn::kItemRows;
}
// Bytes of the work positions that the tensor-core kernel leaves for its join.
inline size_t attn_plan_bytes(int R) { return (size_t)(2 * (size_t)R + 2) * 8; }

bool attn_tc_ok(const spec_prefix_attention_args& a, int* sms);
cudaError_t launch_attention_tc(const spec_prefix_attention_args& a, int sms, float* part, float2* stat,
                                int64_t* plan, cudaStream_t stream);
cudaError_t launch_attention_generic(const spec_prefix_attention_args& a, float* part, float2* stat,
                                     cudaStream_t stream);

}  // namespace spec
