// Penalties for repeated tokens, biases and grammar masks on packed rows of logits.
//
// Mathematics (all in fp32, rounded once): with c = how often v is among the
// request's generated tokens and the row's drafted ones, and seen = c > 0 or v in
// the prompt,
//   z <- z > 0 ? z / repetition : z * repetition   where seen
//   z <- z - frequency * c - presence * [c > 0]
//   z <- z + bias[v],   z <- -inf where the row's mask bit is 0.
//
// Layout: a block takes a slice of the vocabulary of one request for all its
// rows.  Half of its warps read the request's tokens, count those of the slice in
// shared memory and list each token that a rule names once; the others stream the
// rows through as 16-byte vectors that only the mask can change, a warp at a time
// taking the next piece, and the first half joins them when its tables stand.  Then
// the listed entries are computed from the inputs and written over, one thread
// each.  (With the rules applied inside the stream a warp met a named entry in two
// of three vectors and the round case took 1390 us; with the tables built
// before the stream, 622 us.)
// The history costs 4 bytes a token and slice from L2, where a table of counts
// over the vocabulary would cost 4 bytes an entry and request from HBM, and has to
// be kept up between rounds.  It is half of the time from about 3000 tokens on where a
// request has one row (V = 129280, fp32: one request 2.9 us without a history, 6.4 after 4000
// tokens, 31 after 32000; 64 requests 12.7, 29.6 and 133), from about 15000 with 4.7 rows a
// request (49 us, 57 and 170).  Rows share the counts: a row's drafted tokens are
// compared at listed entries only.
// Bound by memory: each logit is read and written once (the round case, 512 requests of
// up to 9 rows of 129280 in fp32: 461 us, 5.7 TB/s).
#include "logits.cuh"

#include <algorithm>

namespace spec {

namespace {

constexpr int kThreads = 256;
// A slice of any alignment meets slice / VEC + 1 vectors: just under whole pieces of 128.
// 31 KB of tables; registers (48) allow five blocks an SM.  At the round case 461 us,
// slices of 4096 545, six blocks (42 registers) 500, seven 662.
constexpr int kMaxSlice = 3040;
constexpr int kMinSlice = 992;
constexpr int kUnroll = 4;
constexpr int kBuilders = kThreads / 2;  // threads that build the tables
constexpr int kMaxDraft = 64;
constexpr uint32_t kPrompt = 0x80000000u;

template <typename T, int VEC>
struct RawVec;
template <>
struct RawVec<float, 4> {
  using type = uint4;
};
template <>
struct RawVec<__nv_bfloat16, 8> {
  using type = uint4;
};
template <>
struct RawVec<float, 1> {
  using type = uint32_t;
};
template <>
struct RawVec<__nv_bfloat16, 1> {
  using type = uint16_t;
};

template <typename T, int VEC>
union Vec {
  typename RawVec<T, VEC>::type raw;
  T e[VEC];
  __device__ Vec() {}
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

// Bits [at, at + n) of a bitmap, n <= 8, without touching a word they do not reach.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int at, int n) {
  const int i = at >> 5, sh = at & 31;
  uint32_t b = w[i] >> sh;
  if (sh + n > 32) b |= w[i + 1] << (32 - sh);
  return b & ((1u << n) - 1u);
}

__device__ __forceinline__ void hide(float& e) { e = -CUDART_INF_F; }
__device__ __forceinline__ void hide(__nv_bfloat16& e) { e = __ushort_as_bfloat16(0xff80); }

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) adjust_kernel(spec_logits_args p, int slice) {
  // tables of the slice: output tokens (kPrompt where the prompt has it), bias entry + 1, and the
  // named tokens, each once
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* count = smem;
  int32_t* bias = reinterpret_cast<int32_t*>(smem + slice);
  uint16_t* named = reinterpret_cast<uint16_t*>(smem + 2 * slice);
  uint32_t* seen = smem + 2 * slice + slice / 2;  // bitmap of the named tokens
  __shared__ int32_t draft_s[kMaxDraft];
  __shared__ int n_named, n_taken;
  const int tid = threadIdx.x, r = blockIdx.y;
  const int s0 = blockIdx.x * slice, s1 = min(s0 + slice, p.V);
  const bool counts = p.repetition || p.frequency || p.presence;
  uint32_t bad = 0;

  int row0 = p.row_off ? p.row_off[r] : r * p.rows_per_request;
  int row1 = p.row_off ? p.row_off[r + 1] : row0 + p.rows_per_request;
  if (row0 < 0 || row1 < row0 || row1 > p.rows) {
    bad |= SPEC_STATUS_BAD_LEN;
    row0 = min(max(row0, 0), p.rows);
    row1 = min(max(row1, row0), p.rows);
  }
  const int n = row1 - row0;
  const int per = (n + gridDim.z - 1) / gridDim.z;  // rows of this block
  const int j0 = min((int)blockIdx.z * per, n), j1 = min(j0 + per, n);
  const int n_draft = counts && p.x ? min(max(j1 - 1, 0), p.x_cols) : 0;

  if (j0 < j1) {
    uint4* clear = reinterpret_cast<uint4*>(smem);
    for (int i = tid; i < (2 * slice) / 4; i += kThreads) clear[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < slice / 32; i += kThreads) seen[i] = 0u;
    if (tid == 0) n_named = n_taken = 0;
    __syncthreads();
    auto name = [&](int d) {
      const uint32_t bit = 1u << (d & 31);
      if (!(atomicOr(&seen[d >> 5], bit) & bit)) named[atomicAdd(&n_named, 1)] = (uint16_t)d;
    };
    auto inside = [&](int t) { return t >= s0 && t < s1; };
    if (tid < kBuilders) {
      if (counts) {
        const int32_t* tok = p.tokens + (size_t)r * p.tokens_ld;
        int len = p.length[r];
        if (len < 0 || len > p.tokens_cols) {
          bad |= SPEC_STATUS_BAD_LEN;
          len = min(max(len, 0), p.tokens_cols);
        }
        const int prompt = p.prompt_len ? p.prompt_len[r] : 0;
        constexpr int kDeep = 8;
        for (int i = tid; i < len; i += kBuilders * kDeep) {
          int t[kDeep];
#pragma unroll
          for (int k = 0; k < kDeep; ++k) t[k] = i + k * kBuilders < len ? tok[i + k * kBuilders] : 0;
#pragma unroll
          for (int k = 0; k < kDeep; ++k) {
            const int at = i + k * kBuilders;
            if (at >= len) break;
            if ((unsigned)t[k] >= (unsigned)p.V) bad |= SPEC_STATUS_BAD_TOKEN;
            if (inside(t[k])) {
              const int d = t[k] - s0;
              if (at < prompt) atomicOr(&count[d], kPrompt);
              else atomicAdd(&count[d], 1u);
              name(d);
            }
          }
        }
        for (int i = tid; i < n_draft; i += kBuilders) {
          const int t = p.x[(size_t)r * p.x_ld + i];
          draft_s[i] = t;
          if ((unsigned)t >= (unsigned)p.V) bad |= SPEC_STATUS_BAD_TOKEN;
          if (inside(t)) name(t - s0);
        }
      }
      if (p.bias_off) {
        int b0 = p.bias_off[r], b1 = p.bias_off[r + 1];
        if (b0 < 0 || b1 < b0 || b1 > p.n_bias) {
          bad |= SPEC_STATUS_BAD_LEN;
          b0 = min(max(b0, 0), p.n_bias);
          b1 = min(max(b1, b0), p.n_bias);
        }
        for (int i = b0 + tid; i < b1; i += kBuilders) {
          const int t = p.bias_tok[i];
          if ((unsigned)t >= (unsigned)p.V) bad |= SPEC_STATUS_BAD_TOKEN;
          if (inside(t)) {
            atomicMax(&bias[t - s0], i + 1);  // a token's last entry counts
            name(t - s0);
          }
        }
      }
    }

    const bool same = p.out == p.logits && p.out_ld == p.ld;
    auto mask_of = [&](size_t b) -> const uint32_t* {
      if (!p.mask) return nullptr;
      const int m = p.mask_row ? p.mask_row[b] : (int)b;
      if (m >= p.n_masks) bad |= SPEC_STATUS_BAD_ROW;
      return m < 0 || m >= p.n_masks ? nullptr
                                     : reinterpret_cast<const uint32_t*>(p.mask) + (size_t)m * p.mask_ld;
    };
    using V = Vec<T, VEC>;
    using R = decltype(V().raw);
    // Pieces of 32 x kUnroll vectors.  Vectors lie on 16 bytes of memory: vector i
    // of a row starts at entry i * VEC - lead, so a slice meets one more of them
    // than it is long.  One that reaches past the slice is taken entry by entry, so
    // that no entry is written by two blocks.
    constexpr uint32_t kAll = (1u << VEC) - 1u;
    const int pieces = (slice / VEC + 1 + 32 * kUnroll - 1) / (32 * kUnroll);
    while (!same || p.mask) {
      int u = 0;
      if ((tid & 31) == 0) u = atomicAdd(&n_taken, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      const int j = j0 + u / pieces;
      if (j >= j1) break;
      const size_t b = (size_t)(row0 + j);
      const T* in = (const T*)p.logits + b * p.ld;
      T* out = (T*)p.out + b * p.out_ld;
      const int lead = VEC == 1 ? 0 : (int)(((uintptr_t)in / sizeof(T)) & (VEC - 1));
      const int i0 = (s0 + lead) / VEC + (u % pieces) * 32 * kUnroll + (tid & 31);
      const int i_end = (s1 + lead + VEC - 1) / VEC;
      V x[kUnroll];
      uint32_t al[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int v = (i0 + k * 32) * VEC - lead;
        if (v >= s0 && v + VEC <= s1) x[k].raw = *reinterpret_cast<const R*>(in + v);
      }
      const uint32_t* mask = mask_of(b);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int v = (i0 + k * 32) * VEC - lead;
        al[k] = kAll;
        if (mask && v >= s0 && v + VEC <= s1) al[k] = bits_at(mask, v, VEC);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (i0 + k * 32 >= i_end) break;
        const int v = (i0 + k * 32) * VEC - lead;
        if (v >= s0 && v + VEC <= s1) {
          if (al[k] != kAll) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              if (!(al[k] >> e & 1u)) hide(x[k].e[e]);
          }
          if (!same || al[k] != kAll) *reinterpret_cast<R*>(out + v) = x[k].raw;
        } else {
          for (int e = 0; e < VEC; ++e) {
            const int w = v + e;
            if (w < s0 || w >= s1) continue;
            T z = in[w];
            if (mask && !bits_at(mask, w, 1)) hide(z);
            out[w] = z;
          }
        }
      }
    }
    __syncthreads();  // the stream is written, the lists are whole

    const float rep = p.repetition ? p.repetition[r] : 1.f, freq = p.frequency ? p.frequency[r] : 0.f,
                pres = p.presence ? p.presence[r] : 0.f;
    const int listed = n_named;
    // a row's listed entries side by side; several rows where the list is short
    const int wide = listed == 0 ? 0 : min(listed, kThreads), tall = wide == 0 ? 0 : kThreads / wide;
    const int jt = wide == 0 ? 0 : tid / wide;
    for (int j = j0 + jt; jt < tall && j < j1; j += tall) {
      const size_t b = (size_t)(row0 + j);
      const T* in = (const T*)p.logits + b * p.ld;
      T* out = (T*)p.out + b * p.out_ld;
      const uint32_t* mask = mask_of(b);
      const int upto = min(j, n_draft);
      for (int i = tid - jt * wide; i < listed; i += wide) {
        const int d = named[i], v = s0 + d;
        const float z0 = to_f(in[v]);
        if (mask && !bits_at(mask, v, 1)) continue;
        const uint32_t w = count[d];
        const int bi = bias[d];
        uint32_t c = w & ~kPrompt;
        for (int k = 0; k < upto; ++k) c += draft_s[k] == v;
        if (c == 0 && w == 0 && bi == 0) continue;  // drafted for a later row only
        float z = z0;
        if (c > 0 || w != 0) z = z > 0.f ? z / rep : z * rep;
        if (c > 0) z = z - freq * (float)c - pres;
        if (bi > 0) z += p.bias_val[bi - 1];
        from_f(z, out + v);
      }
    }
  }
  if (bad) set_status(p.status, bad);
}

template <typename T, int VEC>
cudaError_t launch(const spec_logits_args& a, cudaStream_t stream) {
  // Few rows: small slices, so that one row of a large vocabulary spreads over the SMs
  // (one row of 129280: 4.8 us, 5.6 with large ones); otherwise the largest, whose blocks
  // read the history least often (10 requests of up to 4 rows: 9.4 us, 11.7 with small ones).
  const long long blocks = (long long)a.R * ((a.V + kMaxSlice - 1) / kMaxSlice);
  const int slice = blocks < 304 ? kMinSlice : kMaxSlice;
  // A request with many rows is split over blocks of about 8: each builds the tables
  // again, but reads the rows beside the others (bf16, up to 64 rows each: 8 requests of
  // 129280 entries 65 us with 16 a block, 35 with 8 or 4; 64 of 50257 114, 104 and 112;
  // with 2 a block the round case would take 542).
  const int parts = (int)std::min<long long>(64, std::max<long long>(1, (long long)a.rows / (8ll * a.R)));
  const size_t smem = (size_t)(2 * slice + slice / 2 + slice / 32) * 4;
  const dim3 grid((a.V + slice - 1) / slice, a.R, parts);
  adjust_kernel<T, VEC><<<grid, kThreads, smem, stream>>>(a, slice);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adjust_logits(const spec_logits_args& a, cudaStream_t stream) {
  if (a.R == 0 || a.rows == 0) return cudaSuccess;
  const size_t es = a.dtype == SPEC_F32 ? 4 : 2;
  // 16-byte vectors wherever a row lies on the same offset from 16 bytes in both arrays
  const bool wide = ((uintptr_t)a.logits - (uintptr_t)a.out) % 16 == 0 &&
                    ((a.ld - a.out_ld) * (int64_t)es) % 16 == 0;
  if (a.dtype == SPEC_F32) return wide ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
  return wide ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
}

}  // namespace spec
