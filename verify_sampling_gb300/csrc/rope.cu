// Rotary positions on queries and keys, with the keys and values written to
// their slots of the paged cache: one pass over the projection's output.
//
// Mathematics: pair i of a head turns by the angle position * freq[i]:
//   (x, y) -> scale * (x cos - y sin, y cos + x sin).
// The angle is reduced in turns, not radians: with f = freq / (2 pi) kept as an
// fp32 pair hi + lo and the position p < 2^24 exact in fp32, p * hi = t + e with
// one product and one fma (e exact), t - rint(t) is exact, and the fraction
// (t - rint(t)) + (e + p * lo) is off by a few 2^-26 turns at any position, where
// an fp32 product of radians would be off by p * 2^-24.  sincospif takes it from
// there.  It costs two fmas an angle, where 64-bit products would hold up the
// heads of small models (the fp64 pipe is 1/64 of the fp32 one).
//
// Layout: a block takes kRopeTokens or fewer tokens (or a part of one), computes
// their cosines and sines once into shared memory for all heads, and moves units
// of two 16-byte vectors: the two halves of a pair in the half layout, two
// vectors next to each other otherwise.  Four units a thread are loaded before
// the first is used.  Bound by memory: every element is read and written once.
#include "rope.cuh"

#include <algorithm>

namespace spec {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kRopeTokens = 8;

template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  using type = uint4;
};
template <>
struct Raw<4> {
  using type = uint32_t;
};
template <>
struct Raw<2> {
  using type = uint16_t;
};

template <typename T, int VEC>
union Vec {
  typename Raw<sizeof(T) * VEC>::type raw;
  T e[VEC];
  __device__ Vec() {}
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float* o) { *o = v; }
// one rounding to the stored type, after the sum of both products in fp32
__device__ __forceinline__ void from_f(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ void turn(T& x, T& y, float2 cs) {
  const float a = to_f(x), b = to_f(y);
  from_f(a * cs.x - b * cs.y, &x);
  from_f(b * cs.x + a * cs.y, &y);
}

// The two vectors of a unit: element offsets in the head (-1: none) and how they turn.
struct Unit {
  int a, b;
  int kind;  // 0: copied, 1: a and b turn together, 2: pairs inside each vector
};

template <int VEC, bool INTER>
__device__ __forceinline__ Unit unit_of(int u, int D, int rot, bool rotated) {
  const int half = rot >> 1;
  if (rotated && (VEC == 1 || !INTER)) {
    const int pairs = half / VEC;
    if (u < pairs) return INTER ? Unit{2 * u, 2 * u + 1, 1} : Unit{u * VEC, half + u * VEC, 1};
    const int a = rot + 2 * (u - pairs) * VEC;  // the part of the head that does not turn
    return Unit{a < D ? a : -1, a + VEC < D ? a + VEC : -1, 0};
  }
  const int a = 2 * u * VEC;
  return Unit{a < D ? a : -1, a + VEC < D ? a + VEC : -1, rotated ? 2 : 0};
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(spec_rope_cache_args p, int tokens, int units,
                                                        int per_block) {
  extern __shared__ float2 cs_s[];  // [tokens][rot / 2]
  __shared__ int slot_s[kRopeTokens];
  __shared__ bool live_s[kRopeTokens];
  using V = Vec<T, VEC>;
  const int half = p.rot >> 1, heads = p.Hq + 2 * p.Hk;
  const int row0 = blockIdx.x * tokens, nrow = min(tokens, p.rows - row0);
  const int begin = blockIdx.y * per_block, end = min(begin + per_block, nrow * heads * units);

  uint32_t bad = 0;
  for (int i = threadIdx.x; i < nrow * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const int pos = min(max(p.position[row0 + t], 0), (1 << 24) - 1);
    const double turns = p.freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
    const float hi = (float)turns, lo = (float)(turns - (double)hi), x = (float)pos;
    const float m = x * hi, e = fmaf(x, hi, -m);
    const float frac = (m - rintf(m)) + fmaf(x, lo, e);
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs_s[i] = make_float2(c * p.scale, s * p.scale);
  }
  if (threadIdx.x < nrow) {
    const int pos = p.position[row0 + threadIdx.x];
    int slot = p.slot ? p.slot[row0 + threadIdx.x] : -1;
    if (pos >= (1 << 24)) bad |= SPEC_STATUS_BAD_POSITION;
    if (slot >= p.n_slots) {
      bad |= SPEC_STATUS_BAD_PAGE;
      slot = -1;
    }
    slot_s[threadIdx.x] = slot;
    live_s[threadIdx.x] = pos >= 0;
  }
  if (bad) set_status(p.status, bad);
  __syncthreads();

  for (int i0 = begin + threadIdx.x; i0 < end; i0 += kThreads * kUnroll) {
    V va[kUnroll], vb[kUnroll];
    Unit un[kUnroll];
    T* to[kUnroll];
    int tok[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * kThreads;
      to[k] = nullptr;
      if (i >= end) continue;
      const int hh = i / units, u = i - hh * units, t = hh / heads, h = hh - t * heads;
      if (!live_s[t]) continue;
      const size_t row = (size_t)(row0 + t);
      const T* from;
      if (h < p.Hq) {
        from = (const T*)p.q + row * p.q_row + (size_t)h * p.q_head;
        to[k] = (T*)p.q_out + row * p.q_out_row + (size_t)h * p.q_out_head;
      } else {
        const int s = slot_s[t];
        if (s < 0) continue;
        const bool key = h < p.Hq + p.Hk;
        const int hk = h - p.Hq - (key ? 0 : p.Hk);
        from = key ? (const T*)p.k + row * p.k_row + (size_t)hk * p.k_head
                   : (const T*)p.v + row * p.v_row + (size_t)hk * p.v_head;
        to[k] = (T*)(key ? p.k_cache : p.v_cache) + ((size_t)s * p.Hk + hk) * p.D;
      }
      un[k] = unit_of<VEC, INTER>(u, p.D, p.rot, h < p.Hq + p.Hk);
      tok[k] = t;
      using R = decltype(va[k].raw);
      if (un[k].a >= 0) va[k].raw = *reinterpret_cast<const R*>(from + un[k].a);
      if (un[k].b >= 0) vb[k].raw = *reinterpret_cast<const R*>(from + un[k].b);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (!to[k]) continue;
      const float2* cs = cs_s + tok[k] * half;
      if (un[k].kind == 1) {
        const int f = INTER ? un[k].a >> 1 : un[k].a;
#pragma unroll
        for (int j = 0; j < VEC; ++j) turn(va[k].e[j], vb[k].e[j], cs[f + j]);
      } else if constexpr (VEC > 1 && INTER) {
        if (un[k].kind == 2) {
#pragma unroll
          for (int j = 0; j < VEC; j += 2) {
            if (un[k].a < p.rot) turn(va[k].e[j], va[k].e[j + 1], cs[(un[k].a + j) >> 1]);
            if (un[k].b >= 0 && un[k].b < p.rot)
              turn(vb[k].e[j], vb[k].e[j + 1], cs[(un[k].b + j) >> 1]);
          }
        }
      }
      using R = decltype(va[k].raw);
      if (un[k].a >= 0) *reinterpret_cast<R*>(to[k] + un[k].a) = va[k].raw;
      if (un[k].b >= 0) *reinterpret_cast<R*>(to[k] + un[k].b) = vb[k].raw;
    }
  }
}

template <typename T, int VEC>
cudaError_t launch(const spec_rope_cache_args& a, cudaStream_t stream) {
  const bool inter = a.layout == SPEC_ROPE_INTERLEAVED;
  const int half = a.rot / 2, heads = a.Hq + 2 * a.Hk;
  const int copied = (a.D + 2 * VEC - 1) / (2 * VEC);
  const int turned = (VEC == 1 || !inter) ? half / VEC + (a.D - a.rot + 2 * VEC - 1) / (2 * VEC) : copied;
  const int units = std::max(copied, turned);
  // Enough tokens for four units a thread, or a part of one token where it has
  // more than that; with few rows one unit a thread, over more blocks.
  const long long per_token = (long long)heads * units;
  const int deep = kThreads * kUnroll;
  const int tokens = (int)std::min<long long>(std::min(kRopeTokens, std::max(1, a.rows / 304)),
                                              std::max(1ll, deep / std::max(1ll, per_token)));
  const int per_block = a.rows < 304 ? kThreads : tokens == 1 ? deep : (int)(tokens * per_token);
  const int parts = (int)((tokens * per_token + per_block - 1) / per_block);
  const dim3 grid((a.rows + tokens - 1) / tokens, std::max(1, parts));
  const size_t smem = (size_t)tokens * half * sizeof(float2);
  if (inter) rope_kernel<T, VEC, true><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  else rope_kernel<T, VEC, false><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_cache(const spec_rope_cache_args& a, cudaStream_t stream) {
  if (a.rows == 0 || a.Hq + a.Hk == 0) return cudaSuccess;
  // 16-byte vectors where every row, head, half and remainder starts on one
  const int vec = a.dtype == SPEC_F32 ? 4 : 8;
  const int turn_step = a.layout == SPEC_ROPE_HALF ? a.rot / 2 : a.rot;
  auto on = [&](const void* p) { return ((uintptr_t)p % 16) == 0; };
  const bool wide =
      a.D % vec == 0 && turn_step % vec == 0 && a.rot % vec == 0 && a.q_row % vec == 0 &&
      a.q_head % vec == 0 && a.q_out_row % vec == 0 && a.q_out_head % vec == 0 && a.k_row % vec == 0 &&
      a.k_head % vec == 0 && a.v_row % vec == 0 && a.v_head % vec == 0 && on(a.q) && on(a.k) &&
      on(a.v) && on(a.q_out) && on(a.k_cache) && on(a.v_cache);
  if (a.dtype == SPEC_F32) return wide ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
  return wide ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
}

}  // namespace spec
