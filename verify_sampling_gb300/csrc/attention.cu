// Shared-prefix attention for the sizes the tensor-core kernels do not take:
// fp32, head sizes other than 64 and 128, pages that do not tile 128 keys; over caches of
// the queries' type or of 4 bits.
//
// Mathematics: softmax with a running maximum and sum, out = sum p v / sum p, all in
// fp32 FMAs on tiles converted to fp32 in shared memory.
// Layout: a block takes 32 query rows (packed rows x the query heads of one key head)
// of a request over a share of its keys, prefix and own in turn, 32 keys at a time;
// all of its threads fetch a tile, and a warp has 8 of the rows.  A thread scores four
// rows against two keys (6 shared loads for 32 FMAs), 16 lanes share a row's maximum,
// the weights go through shared memory as one float4 pair a key, and each lane adds
// up four columns (eight for heads over 128) of the warp's eight rows.  Shares of a
// row's keys (few rows, long contexts) are joined by a second kernel.
// Bound by FMA issue where a request has 8 rows x heads or more, else by the fetches.
// (A warp a row and query head, 8 lanes to a key, fetched every key once for each of
// them and spent most of its instructions on reductions: 390 us for 40 requests of up to 6
// rows, 16 heads of 80 on 2 key heads, fp32, behind a prefix of 1500 tokens, 151 us now.)
#include "attention.cuh"

#include <algorithm>

namespace spec {

namespace {

using namespace attn;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplits = 64;  // two a lane of the join
constexpr int kRows = 32, kKeys = 32;  // of a tile
constexpr int kWarpRows = kRows / kWarps;
constexpr int kFetch = 2;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T e[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

// Row strides in shared memory: heads padded to four floats; keys by four more, so that
// the same four columns of 8 keys lie on different banks.
__host__ __device__ inline int padded(int D) { return (D + 3) & ~3; }
inline size_t tile_bytes(int D) {
  return (size_t)(kRows * padded(D) + kKeys * (padded(D) + 4) + kKeys * padded(D)) * sizeof(float);
}

template <typename T, int VEC, int SETS, bool PACKED>  // SETS: 128 columns each
__global__ void __launch_bounds__(kThreads) attention_kernel(spec_prefix_attention_args a, q4::Cache packed, int splits,
                                                             float* part, float2* stat) {
  extern __shared__ __align__(16) float smem[];
  __shared__ __align__(16) float p_s[kWarps][kKeys][kWarpRows];
  __shared__ float row_s[kWarps][kWarpRows];
  __shared__ int64_t key_s[kKeys];  // first element (4 bits: byte) of each key of the tile, -1: none
  __shared__ int64_t scale_s[PACKED ? kKeys : 1];
  using P = Pack<T, VEC>;
  const int D = a.D, Dp = padded(D), per_head = a.Hq / a.Hk;
  float* q_s = smem;
  float* k_s = q_s + kRows * Dp;
  float* v_s = k_s + kKeys * (Dp + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int packs = (D + VEC - 1) / VEC;
  const int r = blockIdx.x, h = blockIdx.y, split = blockIdx.z % splits;
  uint32_t bad = 0;
  const Rows rows = rows_between(a, r, r + 1, &bad);
  const int kv = own_keys(a, r, &bad);
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
  const int m_all = rows.n * per_head;

  for (int m0 = blockIdx.z / splits * kRows; m0 < m_all; m0 += gridDim.z / splits * kRows) {
    const int m_n = min(kRows, m_all - m0);
    auto limit_of = [&](int m) {  // keys of query row m: the prefix's and its own
      return shared + min(kv, max(0, kv - rows.n + (m0 + m) / per_head + 1));
    };
    const int total = limit_of(m_n - 1);  // of the tile's last row
    const int share = ((total + splits - 1) / splits + kKeys - 1) / kKeys * kKeys;
    const int t0 = min(split * share, total), t1 = min(t0 + share, total);

    __syncthreads();  // the last rows' readers of q_s are done
    for (int i = tid; i < kRows * (Dp / 4); i += kThreads) {
      const int m = i / (Dp / 4), c = (i - m * (Dp / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m < m_n) {
        const int j = (m0 + m) / per_head, hq = h * per_head + (m0 + m - j * per_head);
        const T* q = (const T*)a.q + (size_t)(rows.row0 + j) * a.q_row + (size_t)hq * a.q_head + c;
        const float s = a.scale * kLog2e;  // scores in log2 units
        x.x = to_f(q[0]) * s;
        if (c + 1 < D) x.y = to_f(q[1]) * s;
        if (c + 2 < D) x.z = to_f(q[2]) * s;
        if (c + 3 < D) x.w = to_f(q[3]) * s;
      }
      *reinterpret_cast<float4*>(q_s + m * Dp + c) = x;
    }
    const int tq = lane >> 4, tk = lane & 15;  // four rows and two keys of the warp's
    const int w0 = warp * kWarpRows;           // the warp's first row
    const bool busy = w0 < m_n;
    int limit[4];
    float m[4], l[4], acc[SETS][kWarpRows][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      limit[i] = limit_of(w0 + tq * 4 + i);
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < SETS; ++x)
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[x][i][e] = 0.f;

    for (int t = t0; t < t1; t += kKeys) {
      if (tid < kKeys) {
        const int at = t + tid;
        int64_t o = -1;
        if (at < t1) {
          const bool pre = at < shared;
          const int own = pre ? at : at - shared, pi = own / a.page_size;
          const int page = page_of(a, pre ? ptable : table, pi, &bad);
          const int tok = own - pi * a.page_size;
          if (PACKED) {
            o = q4::data_at(page, h, tok, a.Hk, D / q4::kGroup, a.page_size);
            scale_s[tid] = q4::scale_at(page, h, tok, a.Hk, D / q4::kGroup, a.page_size);
          } else {
            o = (((int64_t)page * a.page_size + tok) * a.Hk + h) * D;
          }
        }
        key_s[tid] = o;
      }
      __syncthreads();  // the keys' places; the last tile's readers are done too
      // kFetch packs of keys and of values a thread are on their way together
      if (PACKED) {
        const int words = D / 8;  // of 8 elements
        for (int i = tid; i < kKeys * words; i += kThreads * kFetch) {
          uint32_t x[kFetch], y[kFetch];
          float sx[kFetch], sy[kFetch];
#pragma unroll
          for (int f = 0; f < kFetch; ++f) {
            const int j = i + f * kThreads, key = j / words, w = j - key * words;
            x[f] = y[f] = 0x88888888u;  // zeros
            sx[f] = sy[f] = 0.f;
            if (j >= kKeys * words || key_s[key] < 0) continue;
            const int64_t o = key_s[key] + (int64_t)(w >> 2) * 16 * a.page_size + (w & 3) * 4, so = scale_s[key] + (w >> 2);
            x[f] = *reinterpret_cast<const uint32_t*>(packed.k + o);
            y[f] = *reinterpret_cast<const uint32_t*>(packed.v + o);
            sx[f] = q4::scale_of(packed.k_scale[so]);
            sy[f] = q4::scale_of(packed.v_scale[so]);
          }
#pragma unroll
          for (int f = 0; f < kFetch; ++f) {
            const int j = i + f * kThreads, key = j / words, c = (j - key * words) * 8;
            if (j >= kKeys * words) continue;
            float* ks = k_s + key * (Dp + 4) + c;
            float* vs = v_s + key * Dp + c;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ks[e] = (float)((int)(x[f] >> 4 * e & 15u) - 8) * sx[f];
              vs[e] = (float)((int)(y[f] >> 4 * e & 15u) - 8) * sy[f];
            }
          }
        }
      } else {
        for (int i = tid; i < kKeys * packs; i += kThreads * kFetch) {
          P x[kFetch], y[kFetch];
          int at[kFetch];
#pragma unroll
          for (int f = 0; f < kFetch; ++f) {
            const int j = i + f * kThreads, key = j / packs, c = (j - key * packs) * VEC;
            at[f] = -1;
            if (j >= kKeys * packs) continue;
            at[f] = key << 16 | c;
            const int64_t o = key_s[key];
            if (o >= 0) {
              x[f] = *reinterpret_cast<const P*>((const T*)a.k_cache + o + c);
              y[f] = *reinterpret_cast<const P*>((const T*)a.v_cache + o + c);
            } else {
#pragma unroll
              for (int e = 0; e < VEC; ++e) put(&x[f].e[e], 0.f), put(&y[f].e[e], 0.f);
            }
          }
#pragma unroll
          for (int f = 0; f < kFetch; ++f) {
            if (at[f] < 0) continue;
            const int key = at[f] >> 16, c = at[f] & 0xffff;
            float* ks = k_s + key * (Dp + 4) + c;
            float* vs = v_s + key * Dp + c;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              ks[e] = to_f(x[f].e[e]);
              vs[e] = to_f(y[f].e[e]);
            }
          }
        }
      }
      if (Dp > D && tid < kKeys)
        for (int c = D; c < Dp; ++c) k_s[tid * (Dp + 4) + c] = v_s[tid * Dp + c] = 0.f;
      __syncthreads();
      if (!busy) continue;

      float s[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
      const float* qr = q_s + (w0 + tq * 4) * Dp;
      const float* kr = k_s + tk * (Dp + 4);
      for (int c = 0; c < Dp; c += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(kr + c);
        const float4 k1 = *reinterpret_cast<const float4*>(kr + 16 * (Dp + 4) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(qr + i * Dp + c);
          s[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[i][0]))));
          s[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[i][1]))));
        }
      }
      float c4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t + tk >= min(limit[i], t1)) s[i][0] = -CUDART_INF_F;
        if (t + tk + 16 >= min(limit[i], t1)) s[i][1] = -CUDART_INF_F;
        float top = fmaxf(s[i][0], s[i][1]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m[i]);
        const float sub = top == -CUDART_INF_F ? 0.f : top;
        c4[i] = exp2f(m[i] - sub);  // 0 from -inf
        m[i] = top;
        s[i][0] = exp2f(s[i][0] - sub);
        s[i][1] = exp2f(s[i][1] - sub);
        l[i] = fmaf(l[i], c4[i], s[i][0] + s[i][1]);  // this lane's keys
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<float4*>(&p_s[warp][tk + 16 * x][tq * 4]) = make_float4(s[0][x], s[1][x], s[2][x], s[3][x]);
      if (tk == 0) *reinterpret_cast<float4*>(&row_s[warp][tq * 4]) = make_float4(c4[0], c4[1], c4[2], c4[3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) {
        const float c = row_s[warp][i];
#pragma unroll
        for (int x = 0; x < SETS; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[x][i][e] *= c;
      }
#pragma unroll 4
      for (int key = 0; key < kKeys; ++key) {
        const float4 pa = *reinterpret_cast<const float4*>(&p_s[warp][key][0]);
        const float4 pb = *reinterpret_cast<const float4*>(&p_s[warp][key][4]);
        const float pv[kWarpRows] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
          const int c = x * 128 + lane * 4;
          if (c < Dp) {
            const float4 v = *reinterpret_cast<const float4*>(v_s + key * Dp + c);
#pragma unroll
            for (int i = 0; i < kWarpRows; ++i) {
              acc[x][i][0] = fmaf(pv[i], v.x, acc[x][i][0]);
              acc[x][i][1] = fmaf(pv[i], v.y, acc[x][i][1]);
              acc[x][i][2] = fmaf(pv[i], v.z, acc[x][i][2]);
              acc[x][i][3] = fmaf(pv[i], v.w, acc[x][i][3]);
            }
          }
        }
      }
      __syncwarp();  // p_s and row_s are read before the next tile's take their place
    }
    if (!busy) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      const int row = w0 + tq * 4 + i;
      if (tk != 0 || row >= m_n) continue;
      const int j = (m0 + row) / per_head, b = rows.row0 + j, hq = h * per_head + (m0 + row - j * per_head);
      if (splits > 1) stat[((size_t)split * a.rows + b) * a.Hq + hq] = make_float2(m[i], l[i]);
      else if (a.lse) a.lse[(size_t)b * a.Hq + hq] = l[i] == 0.f ? -CUDART_INF_F : (m[i] + log2f(l[i])) * kLn2;
    }
    if (tk == 0) *reinterpret_cast<float4*>(&row_s[warp][tq * 4]) = make_float4(l[0], l[1], l[2], l[3]);
    __syncwarp();
    for (int i = 0; i < kWarpRows && w0 + i < m_n; ++i) {
      const int j = (m0 + w0 + i) / per_head, b = rows.row0 + j, hq = h * per_head + (m0 + w0 + i - j * per_head);
      const float sum = row_s[warp][i], inv = sum == 0.f ? 0.f : 1.f / sum;  // a row without keys: zeros
#pragma unroll
      for (int x = 0; x < SETS; ++x) {
        const int c = x * 128 + lane * 4;
        float o[4];
#pragma unroll
        for (int z = 0; z < kWarpRows; ++z)
          if (z == i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = acc[x][z][e];
          }
        if (splits > 1) {
          float* to = part + (((size_t)split * a.rows + b) * a.Hq + hq) * D + c;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < D) to[e] = o[e];
        } else {
          T* to = (T*)a.out + (size_t)b * a.out_row + (size_t)hq * a.out_head + c;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < D) put(to + e, o[e] * inv);
        }
      }
    }
    __syncwarp();
  }
  if (bad) set_status(a.status, bad);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(spec_prefix_attention_args a, int splits,
                                                        const float* part, const float2* stat) {
  const int lane = threadIdx.x & 31, d = blockIdx.y * 32 + lane;  // 32 columns of a row and head a warp
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.rows * a.Hq) return;
  const int b = (int)(unit / a.Hq), hq = (int)(unit % a.Hq);
  uint32_t bad = 0;
  const int r = last_at_or_below(a.row_off, a.R, b);
  const Rows rows = rows_between(a, r, r + 1, &bad);
  if (b < rows.row0 || b >= rows.row0 + rows.n) return;
  const size_t step = (size_t)a.rows * a.Hq;
  // a lane a share (two where there are more than 32): its weight against the largest maximum
  float2 st[2];
  float m = -CUDART_INF_F, l = 0.f, w[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    st[x] = make_float2(-CUDART_INF_F, 0.f);
    if (x * 32 + lane < splits) st[x] = stat[unit + (x * 32 + lane) * step];
    m = fmaxf(m, st[x].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    w[x] = st[x].x == -CUDART_INF_F ? 0.f : exp2f(st[x].x - m);
    l = fmaf(st[x].y, w[x], l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row without keys: zeros
  T* out = (T*)a.out + (size_t)b * a.out_row + (size_t)hq * a.out_head;
  float o = 0.f;
#pragma unroll 16
  for (int s = 0; s < splits; ++s) {
    const float ws = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
    o = fmaf(part[(unit + s * step) * a.D + min(d, a.D - 1)], ws, o);
  }
  if (d < a.D) put(out + d, o * inv);
  if (a.lse && d == 0) a.lse[unit] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

template <typename T, int VEC, int SETS, bool PACKED>
cudaError_t launch(const spec_prefix_attention_args& a, const q4::Cache& packed, float* part, float2* stat, cudaStream_t stream) {
  const long long units = (long long)a.rows * a.Hq;
  // Blocks for the mean request's rows (a longer one's loop), and shares of at least
  // 64 keys, until there are about eight blocks an SM for 152 SMs, within the
  // workspace's partial rows.  (The 40 requests above 151 us, 159 with four blocks an SM, 147
  // with sixteen; without their prefix 57.7, 60.0 and 57.9; 9 requests of 12 heads of 80 behind
  // prefixes of 500 tokens 25.4 us, 32.8 with shares of 128 keys.)
  const long long keys = ((long long)a.max_pages + (a.G > 0 ? a.max_prefix_pages : 0)) * a.page_size;
  const long long per_head = a.Hq / a.Hk;
  const long long tiles = std::min<long long>(512, (a.rows * per_head + (long long)kRows * a.R - 1) / ((long long)kRows * a.R));
  const long long blocks = (long long)a.R * a.Hk * tiles;
  const int splits = (int)std::max(1ll, std::min<long long>({kMaxSplits, (152 * 8 + blocks - 1) / blocks, (keys + 63) / 64,
                                                             (long long)(attn_partial_rows(a.rows, a.Hq) / units)}));
  const size_t smem = tile_bytes(a.D);
  auto kernel = attention_kernel<T, VEC, SETS, PACKED>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  kernel<<<dim3(a.R, a.Hk, (unsigned)(tiles * splits)), kThreads, smem, stream>>>(a, packed, splits, part, stat);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  if (splits > 1)
    join_kernel<T><<<dim3((unsigned)((units + kWarps - 1) / kWarps), (a.D + 31) / 32), kThreads, 0, stream>>>(a, splits, part, stat);
  return cudaGetLastError();
}

template <typename T, int VEC, bool PACKED = false>
cudaError_t launch(const spec_prefix_attention_args& a, float* part, float2* stat, cudaStream_t stream,
                   const q4::Cache& packed = q4::Cache{}) {
  return a.D <= 128 ? launch<T, VEC, 1, PACKED>(a, packed, part, stat, stream)
                    : launch<T, VEC, 2, PACKED>(a, packed, part, stat, stream);
}

}  // namespace

cudaError_t launch_attention_generic(const spec_prefix_attention_args& a, float* part, float2* stat,
                                     cudaStream_t stream) {
  auto on = [&](const void* p) { return ((uintptr_t)p % 16) == 0; };
  const int vec = a.dtype == SPEC_F32 ? 4 : 8;
  const bool wide = a.D % vec == 0 && on(a.k_cache) && on(a.v_cache);
  if (a.dtype == SPEC_F32)
    return wide ? launch<float, 4>(a, part, stat, stream) : launch<float, 1>(a, part, stat, stream);
  return wide ? launch<__nv_bfloat16, 8>(a, part, stat, stream)
              : launch<__nv_bfloat16, 1>(a, part, stat, stream);
}

cudaError_t launch_attention_packed_generic(const spec_prefix_attention_args& a, const q4::Cache& packed, float* part,
                                          float2* stat, cudaStream_t stream) {
  return a.dtype == SPEC_F32 ? launch<float, 1, true>(a, part, stat, stream, packed)
                             : launch<__nv_bfloat16, 1, true>(a, part, stat, stream, packed);
}

}  // namespace spec
