// C-ABI entry points of the operators around the target model's forward pass:
// argument validation and launches.  Every check happens on the host before
// anything is launched; no call synchronises the host or allocates memory.
#include "attention.cuh"
#include "cache_tables.cuh"
#include "checks.cuh"
#include "logits.cuh"
#include "rope.cuh"

namespace {

using namespace spec;

constexpr int kMaxRequests = 65535;

// R, the page size, the page count and the table width of a paged cache.
bool cache_sizes_ok(int R, int page_size, int n_pages, int max_pages) {
  return R >= 0 && R <= kMaxRequests && page_size >= 1 && n_pages >= 1 && max_pages >= 1 &&
         (int64_t)n_pages * page_size < ((int64_t)1 << 31);
}

bool attention_sizes_ok(int rows, int R, int Hq, int D) {
  return rows >= 0 && R >= 0 && R <= kMaxRequests && Hq >= 1 && Hq <= 1024 && D >= 1 &&
         D <= kAttnMaxDim && (int64_t)rows * Hq < ((int64_t)1 << 31);
}

// Workspace parts: partial rows, their maxima and sums, the work positions.
size_t attention_part_bytes(int rows, int Hq, int D) {
  return align256(attn_partial_rows(rows, Hq) * D * sizeof(float));
}
size_t attention_stat_bytes(int rows, int Hq) {
  return align256(attn_partial_rows(rows, Hq) * sizeof(float2));
}

int status_of(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace

extern "C" {

int spec_cache_reserve(const spec_cache_reserve_args* args, spec_stream_t stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_cache_reserve_args& a = *args;
  if (!cache_sizes_ok(a.R, a.page_size, a.n_pages, a.max_pages) || a.rows < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!a.ring || !a.ring_pos || !a.ring_out || a.ring_out == a.ring_pos) return SPEC_ERR_INVALID_ARG;
  if (a.R > 0 && (!a.kv_len || !a.row_off || !a.block_table || !a.new_len ||
                  a.new_len == a.kv_len || a.new_len == a.row_off || a.new_len == a.pos_base))
    return SPEC_ERR_INVALID_ARG;
  if (a.rows > 0 && (!a.position || !a.request || !a.slot)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(a.kv_len, 4) || !aligned(a.row_off, 4) || !aligned(a.pos_base, 4) ||
      !aligned(a.block_table, 4) || !aligned(a.ring, 4) || !aligned(a.ring_pos, 8) ||
      !aligned(a.ring_out, 8) || !aligned(a.new_len, 4) || !aligned(a.position, 4) ||
      !aligned(a.request, 4) || !aligned(a.slot, 4) || !aligned(a.status, 4))
    return SPEC_ERR_ALIGNMENT;
  return status_of(launch_cache_reserve(a, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_cache_commit(const spec_cache_commit_args* args, spec_stream_t stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_cache_commit_args& a = *args;
  if (!cache_sizes_ok(a.R, a.page_size, a.n_pages, a.max_pages)) return SPEC_ERR_INVALID_ARG;
  if (!a.ring || !a.ring_pos || !a.ring_out || a.ring_out == a.ring_pos) return SPEC_ERR_INVALID_ARG;
  if (a.R > 0 && (!a.kv_len || !a.new_len || !a.keep || !a.block_table || !a.kv_out ||
                  a.kv_out == a.kv_len || a.kv_out == a.new_len || a.kv_out == a.keep))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(a.kv_len, 4) || !aligned(a.new_len, 4) || !aligned(a.keep, 4) ||
      !aligned(a.block_table, 4) || !aligned(a.ring, 4) || !aligned(a.ring_pos, 8) ||
      !aligned(a.ring_out, 8) || !aligned(a.kv_out, 4) || !aligned(a.status, 4))
    return SPEC_ERR_ALIGNMENT;
  return status_of(launch_cache_commit(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_attention_workspace_bytes(int rows, int R, int Hq, int D) {
  if (!attention_sizes_ok(rows, R, Hq, D)) return 0;
  return attention_part_bytes(rows, Hq, D) + attention_stat_bytes(rows, Hq) + align256(attn_plan_bytes(R));
}

int spec_prefix_attention(const spec_prefix_attention_args* args, spec_stream_t stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  spec_prefix_attention_args a = *args;
  if (!cache_sizes_ok(a.R, a.page_size, a.n_pages, a.max_pages) || a.rows < 0 || !valid_dtype(a.dtype) ||
      a.Hq < 1 || a.Hq > 1024 || a.Hk < 1 || a.Hq % a.Hk != 0 || a.D < 1 || a.G < 0 || a.G > a.R ||
      (int64_t)a.rows * a.Hq >= ((int64_t)1 << 31) || !(a.scale > 0.f) || !(a.scale < 1e30f))
    return SPEC_ERR_INVALID_ARG;
  if (a.D > kAttnMaxDim) return SPEC_ERR_UNSUPPORTED;
  if (a.R == 0 || a.rows == 0) return SPEC_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.row_off || !a.kv_len || !a.block_table || !a.out)
    return SPEC_ERR_INVALID_ARG;
  if (a.G > 0 && (!a.group_off || !a.prefix_len || !a.prefix_table || a.max_prefix_pages < 1))
    return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype_size(a.dtype);
  if (!aligned(a.q, es) || !aligned(a.k_cache, es) || !aligned(a.v_cache, es) || !aligned(a.out, es) ||
      !aligned(a.row_off, 4) || !aligned(a.kv_len, 4) || !aligned(a.block_table, 4) ||
      !aligned(a.lse, 4) || !aligned(a.status, 4) ||
      (a.G > 0 && (!aligned(a.group_off, 4) || !aligned(a.prefix_len, 4) || !aligned(a.prefix_table, 4))))
    return SPEC_ERR_ALIGNMENT;
  const int rc = check_workspace(a.workspace, a.workspace_bytes,
                                 spec_attention_workspace_bytes(a.rows, a.R, a.Hq, a.D));
  if (rc != SPEC_OK) return rc;
  char* ws = static_cast<char*>(a.workspace);
  float* part = reinterpret_cast<float*>(ws);
  float2* stat = reinterpret_cast<float2*>(ws + attention_part_bytes(a.rows, a.Hq, a.D));
  int64_t* plan = reinterpret_cast<int64_t*>(ws + attention_part_bytes(a.rows, a.Hq, a.D) +
                                             attention_stat_bytes(a.rows, a.Hq));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  return status_of(attn_tc_ok(a, &sms) ? launch_attention_tc(a, sms, part, stat, plan, s)
                                       : launch_attention_generic(a, part, stat, s));
}

int spec_rope_cache(const spec_rope_cache_args* args, spec_stream_t stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  spec_rope_cache_args a = *args;
  if (a.rows < 0 || a.Hq < 0 || a.Hq > 1024 || a.Hk < 0 || a.Hk > 1024 || a.D < 1 || a.rot < 0 ||
      a.rot > a.D || a.rot % 2 != 0 || !valid_dtype(a.dtype) ||
      (a.layout != SPEC_ROPE_HALF && a.layout != SPEC_ROPE_INTERLEAVED))
    return SPEC_ERR_INVALID_ARG;
  if (a.D > kRopeMaxDim) return SPEC_ERR_UNSUPPORTED;
  if (a.Hk == 0) {
    a.k = a.v = nullptr;
    a.k_cache = a.v_cache = nullptr;
    a.slot = nullptr;
    a.k_row = a.k_head = a.v_row = a.v_head = 0;
  }
  if (a.Hq == 0) {
    a.q = nullptr;
    a.q_out = nullptr;
    a.q_row = a.q_head = a.q_out_row = a.q_out_head = 0;
  }
  if (a.rows > 0) {
    if (!a.position || (a.rot > 0 && !a.freq)) return SPEC_ERR_INVALID_ARG;
    if (a.Hq > 0 && (!a.q || !a.q_out)) return SPEC_ERR_INVALID_ARG;
    // in place: every element where it was, or one row's results would be another's input
    if (a.Hq > 0 && a.q == a.q_out && ((a.rows > 1 && a.q_row != a.q_out_row) || (a.Hq > 1 && a.q_head != a.q_out_head)))
      return SPEC_ERR_INVALID_ARG;
    if (a.Hk > 0 && (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.slot || a.n_slots < 1))
      return SPEC_ERR_INVALID_ARG;
  }
  const size_t es = dtype_size(a.dtype);
  if (!aligned(a.q, es) || !aligned(a.k, es) || !aligned(a.v, es) || !aligned(a.q_out, es) ||
      !aligned(a.k_cache, es) || !aligned(a.v_cache, es) || !aligned(a.freq, 8) ||
      !aligned(a.position, 4) || !aligned(a.slot, 4) || !aligned(a.status, 4))
    return SPEC_ERR_ALIGNMENT;
  return status_of(launch_rope_cache(a, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_adjust_logits(const spec_logits_args* args, spec_stream_t stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_logits_args& a = *args;
  if (a.R < 0 || a.R > kMaxRequests || a.V < 1 || a.V >= (1 << 30) || a.rows < 0 ||
      !valid_dtype(a.dtype))
    return SPEC_ERR_INVALID_ARG;
  if (a.R == 0 || a.rows == 0) return SPEC_OK;
  if (!a.logits || !a.out || a.ld < a.V || a.out_ld < a.V || a.ld >= ((int64_t)1 << 31) ||
      a.out_ld >= ((int64_t)1 << 31))
    return SPEC_ERR_INVALID_ARG;
  if (a.out == a.logits && a.out_ld != a.ld) return SPEC_ERR_INVALID_ARG;
  if (!a.row_off && (a.rows_per_request < 0 || (int64_t)a.R * a.rows_per_request > a.rows))
    return SPEC_ERR_INVALID_ARG;
  if ((a.repetition || a.frequency || a.presence) && (a.tokens_cols < 0 || a.tokens_ld < a.tokens_cols || (a.tokens_cols > 0 && !a.tokens) || !a.length))
    return SPEC_ERR_INVALID_ARG;
  if (a.x && (a.x_cols < 0 || a.x_cols > 64 || a.x_ld < a.x_cols)) return SPEC_ERR_INVALID_ARG;
  if ((a.bias_off != nullptr) != (a.bias_tok != nullptr) ||
      (a.bias_off != nullptr) != (a.bias_val != nullptr) || (a.bias_off && a.n_bias < 0))
    return SPEC_ERR_INVALID_ARG;
  if (a.mask && (a.n_masks < 1 || a.mask_ld < (a.V + 31) / 32)) return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype_size(a.dtype);
  if (!aligned(a.logits, es) || !aligned(a.out, es) || !aligned(a.row_off, 4) ||
      !aligned(a.tokens, 4) || !aligned(a.prompt_len, 4) || !aligned(a.length, 4) ||
      !aligned(a.x, 4) || !aligned(a.repetition, 4) || !aligned(a.frequency, 4) ||
      !aligned(a.presence, 4) || !aligned(a.bias_off, 4) || !aligned(a.bias_tok, 4) ||
      !aligned(a.bias_val, 4) || !aligned(a.mask, 4) || !aligned(a.mask_row, 4) ||
      !aligned(a.status, 4))
    return SPEC_ERR_ALIGNMENT;
  return status_of(launch_adjust_logits(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
