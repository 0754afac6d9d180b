// Shared-prefix attention for the sizes the tensor-core kernel does not take:
// fp32, head sizes other than 64 and 128, pages that do not tile 128 keys.
//
// Mathematics: softmax with a running maximum and sum, out = sum p v / sum p.
// Layout: a warp takes one row and query head over a share of its keys, 8 lanes
// to a key, four keys at a time, each group of 8 with its own running state until
// the end.  Shares of a row's keys (few rows, long contexts) are joined by a
// second kernel.  Bound by the load latency of a key; the sizes that serving
// models have go to attention_tc.cu.
#include "attention.cuh"

#include <algorithm>

namespace spec {

namespace {

using namespace attn;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplits = 64;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T e[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

// Elements d = (i * 8 + lane of the group) * VEC + e of a head, i < PER / VEC.
template <typename T, int VEC, int PER>
__global__ void __launch_bounds__(kThreads) attention_kernel(spec_prefix_attention_args a, int splits,
                                                             float* part, float2* stat) {
  constexpr int NI = PER / VEC;
  using P = Pack<T, VEC>;
  const int lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.rows * a.Hq) return;
  const int b = (int)(unit / a.Hq), hq = (int)(unit % a.Hq), h = hq / (a.Hq / a.Hk);
  uint32_t bad = 0;
  const int r = last_at_or_below(a.row_off, a.R, b);
  const Rows rows = rows_between(a, r, r + 1, &bad);
  if (b < rows.row0 || b >= rows.row0 + rows.n) {  // no request's row
    if (bad) set_status(a.status, bad);
    return;
  }
  const int kv = own_keys(a, r, &bad);
  const int own = min(kv, max(0, kv - rows.n + (b - rows.row0) + 1));
  int shared = 0;
  const int32_t* ptable = nullptr;
  if (a.G > 0) {
    const int g = last_at_or_below(a.group_off, a.G, r);
    const int2 in = group_requests(a, g, &bad);
    if (r >= in.x && r < in.y) {
      shared = prefix_keys(a, g, &bad);
      ptable = a.prefix_table + (size_t)g * a.max_prefix_pages;
    }
  }
  const int32_t* table = a.block_table + (size_t)r * a.max_pages;
  const int total = shared + own, share = (total + splits - 1) / splits;
  const int t0 = min((int)blockIdx.y * share, total), t1 = min(t0 + share, total);

  const T* q = (const T*)a.q + (size_t)b * a.q_row + (size_t)hq * a.q_head;
  const int nv = a.D / VEC;
  float qv[PER], acc[PER];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int w = i * 8 + sub;
    P x;
    if (w < nv) x = *reinterpret_cast<const P*>(q + w * VEC);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      qv[i * VEC + e] = w < nv ? to_f(x.e[e]) : 0.f;
      acc[i * VEC + e] = 0.f;
    }
  }
  const float sl = a.scale * kLog2e;
  float m = -CUDART_INF_F, l = 0.f;
  for (int t = t0 + grp; t - grp < t1; t += 4) {
    const bool live = t < t1;
    float dot = 0.f;
    P kx[NI], vx[NI];
    if (live) {
      const bool pre = t < shared;
      const int at = pre ? t : t - shared;
      const int pi = at / a.page_size;
      const int page = page_of(a, pre ? ptable : table, pi, &bad);
      const size_t o = (((size_t)page * a.page_size + (at - pi * a.page_size)) * a.Hk + h) * a.D;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (i * 8 + sub < nv) {
          kx[i] = *reinterpret_cast<const P*>((const T*)a.k_cache + o + (i * 8 + sub) * VEC);
          vx[i] = *reinterpret_cast<const P*>((const T*)a.v_cache + o + (i * 8 + sub) * VEC);
        }
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (i * 8 + sub < nv) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) dot = fmaf(qv[i * VEC + e], to_f(kx[i].e[e]), dot);
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (!live) continue;
    const float z = dot * sl;
    if (z > m) {
      const float c = exp2f(m - z);  // 0 at the first key
      l *= c;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= c;
      m = z;
    }
    const float w = z == -CUDART_INF_F ? 0.f : exp2f(z - m);
    l += w;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i * 8 + sub < nv) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[i * VEC + e] = fmaf(w, to_f(vx[i].e[e]), acc[i * VEC + e]);
      }
  }
  // the four groups' states
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), top = fmaxf(m, mo);
    const float c = m == -CUDART_INF_F ? 0.f : exp2f(m - top);
    l *= c;
    l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      acc[i] *= c;
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    m = top;
  }
  if (splits > 1) {
    const size_t slot = ((size_t)blockIdx.y * a.rows + b) * a.Hq + hq;
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (i * 8 + sub < nv) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) part[slot * a.D + (i * 8 + sub) * VEC + e] = acc[i * VEC + e];
        }
      if (sub == 0) stat[slot] = make_float2(m, l);
    }
  } else if (grp == 0) {
    T* out = (T*)a.out + (size_t)b * a.out_row + (size_t)hq * a.out_head;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a row without keys: zeros
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i * 8 + sub < nv) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) put(out + (i * 8 + sub) * VEC + e, acc[i * VEC + e] * inv);
      }
    if (a.lse && sub == 0)
      a.lse[(size_t)b * a.Hq + hq] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
  }
  if (bad) set_status(a.status, bad);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(spec_prefix_attention_args a, int splits,
                                                        const float* part, const float2* stat) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.rows * a.Hq) return;
  const int b = (int)(unit / a.Hq), hq = (int)(unit % a.Hq);
  uint32_t bad = 0;
  const int r = last_at_or_below(a.row_off, a.R, b);
  const Rows rows = rows_between(a, r, r + 1, &bad);
  if (b < rows.row0 || b >= rows.row0 + rows.n) return;
  const size_t step = (size_t)a.rows * a.Hq;
  float m = -CUDART_INF_F, l = 0.f;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, stat[unit + s * step].x);
  for (int s = 0; s < splits; ++s) {
    const float2 t = stat[unit + s * step];
    if (t.y != 0.f) l += t.y * exp2f(t.x - m);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = (T*)a.out + (size_t)b * a.out_row + (size_t)hq * a.out_head;
  for (int d = lane; d < a.D; d += 32) {
    float o = 0.f;
    for (int s = 0; s < splits; ++s) {
      const float2 t = stat[unit + s * step];
      if (t.y != 0.f) o = fmaf(part[(unit + s * step) * a.D + d], exp2f(t.x - m), o);
    }
    put(out + d, o * inv);
  }
  if (a.lse && lane == 0) a.lse[unit] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

template <typename T, int VEC>
cudaError_t launch(const spec_prefix_attention_args& a, float* part, float2* stat, cudaStream_t stream) {
  const long long units = (long long)a.rows * a.Hq;
  // Shares of at least 64 keys, until there are about eight warps an SM for 152
  // SMs, within the workspace's partial rows.
  const long long keys = ((long long)a.max_pages + (a.G > 0 ? a.max_prefix_pages : 0)) * a.page_size;
  const long long want = std::min<long long>({kMaxSplits, (152 * 8 + units - 1) / units, (keys + 63) / 64,
                                              (long long)(attn_partial_rows(a.rows, a.Hq) / units)});
  const int splits = (int)std::max(1ll, want);
  const dim3 grid((unsigned)((units + kWarps - 1) / kWarps), splits);
  if (a.D <= 128) attention_kernel<T, VEC, 16><<<grid, kThreads, 0, stream>>>(a, splits, part, stat);
  else attention_kernel<T, VEC, 32><<<grid, kThreads, 0, stream>>>(a, splits, part, stat);
  if (splits > 1) join_kernel<T><<<grid.x, kThreads, 0, stream>>>(a, splits, part, stat);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_generic(const spec_prefix_attention_args& a, float* part, float2* stat,
                                     cudaStream_t stream) {
  auto on = [&](const void* p) { return ((uintptr_t)p % 16) == 0; };
  const int vec = a.dtype == SPEC_F32 ? 4 : 8;
  const bool wide = a.D % vec == 0 && a.q_row % vec == 0 && a.q_head % vec == 0 && on(a.q) &&
                    on(a.k_cache) && on(a.v_cache);
  if (a.dtype == SPEC_F32)
    return wide ? launch<float, 4>(a, part, stat, stream) : launch<float, 1>(a, part, stat, stream);
  return wide ? launch<__nv_bfloat16, 8>(a, part, stat, stream)
              : launch<__nv_bfloat16, 1>(a, part, stat, stream);
}

}  // namespace spec
