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
// vectors next to each other otherwise.  Either way unit u of a head takes the
// frequencies [u VEC, (u + 1) VEC), which lie in shared memory as one float4 column
// a unit, so that the units of a head read without bank conflicts.  Four units a
// thread are loaded before the first is used.  Bound by memory: every element is
// read and written once.
#include "rope.cuh"

#include <algorithm>

namespace spec {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kRopeTokens = 8;

template <typename T, int VEC>
union Vec {
  uint4 raw;
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
  // spelled out, so that every kernel rounds alike
  from_f(fmaf(a, cs.x, -__fmul_rn(b, cs.y)), &x);
  from_f(fmaf(b, cs.x, __fmul_rn(a, cs.y)), &y);
}

// cos and sin, times the scale, of position x times the frequency (radians).
__device__ __forceinline__ float2 cos_sin(float x, double freq, float scale) {
  const double turns = freq * 0.15915494309189533577;  // 1 / (2 pi)
  const float hi = (float)turns, lo = (float)(turns - (double)hi);
  const float m = x * hi, e = fmaf(x, hi, -m);
  const float frac = (m - rintf(m)) + fmaf(x, lo, e);
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * scale, s * scale);
}

// Where a unit is read and written.
template <typename T>
struct Move {
  const T* from;
  T* to;  // null: nothing to do
};

template <typename T>
__device__ __forceinline__ Move<T> head_of(const spec_rope_cache_args& p, size_t row, int h, int slot) {
  if (h < p.Hq)
    return Move<T>{(const T*)p.q + row * p.q_row + (size_t)h * p.q_head,
                   (T*)p.q_out + row * p.q_out_row + (size_t)h * p.q_out_head};
  if (slot < 0) return Move<T>{nullptr, nullptr};
  const bool key = h < p.Hq + p.Hk;
  const int hk = h - p.Hq - (key ? 0 : p.Hk);
  return Move<T>{key ? (const T*)p.k + row * p.k_row + (size_t)hk * p.k_head
                     : (const T*)p.v + row * p.v_row + (size_t)hk * p.v_head,
                 (T*)(key ? p.k_cache : p.v_cache) + ((size_t)slot * p.Hk + hk) * p.D};
}

// Slot of each of the block's rows; -2 where the row is left out.
__device__ __forceinline__ void read_slots(const spec_rope_cache_args& p, int row0, int nrow, int* slot_s) {
  if ((int)threadIdx.x >= nrow) return;
  const int pos = p.position[row0 + threadIdx.x];
  int slot = p.slot ? max(p.slot[row0 + threadIdx.x], -1) : -1;
  uint32_t bad = 0;
  if (pos >= (1 << 24)) bad |= SPEC_STATUS_BAD_POSITION;
  if (slot >= p.n_slots) {
    bad |= SPEC_STATUS_BAD_PAGE;
    slot = -1;
  }
  slot_s[threadIdx.x] = pos < 0 ? -2 : slot;
  if (bad) set_status(p.status, bad);
}
__device__ __forceinline__ float position_of(const spec_rope_cache_args& p, int row) {
  return (float)min(max(p.position[row], 0), (1 << 24) - 1);
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(spec_rope_cache_args p, int tokens, int units,
                                                        int per_block) {
  static_assert(VEC == 16 / (int)sizeof(T), "16-byte vectors");
  constexpr int kCol = VEC / 4;  // float4s of a unit's cosines
  extern __shared__ __align__(16) float4 cs_s[];  // a token: cosines [kCol][turning], then sines
  __shared__ int slot_s[kRopeTokens];
  using V = Vec<T, VEC>;
  const int half = p.rot >> 1, heads = p.Hq + 2 * p.Hk, turned = p.Hq + p.Hk;
  const int turning = (half + VEC - 1) / VEC;  // units that turn
  const int row0 = blockIdx.x * tokens, nrow = min(tokens, p.rows - row0);
  const int begin = blockIdx.y * per_block, end = min(begin + per_block, nrow * heads * units);

  for (int i = threadIdx.x; i < nrow * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const float2 cs = cos_sin(position_of(p, row0 + t), p.freq[f], p.scale);
    const int u = f / VEC, e = f % VEC;
    float* col = reinterpret_cast<float*>(cs_s + (size_t)t * 2 * kCol * turning + (e / 4) * turning + u) + e % 4;
    col[0] = cs.x;
    col[4 * kCol * turning] = cs.y;
  }
  read_slots(p, row0, nrow, slot_s);
  __syncthreads();

  // (token, head, unit) of the thread's next unit, stepped by the block's threads
  int i = begin + threadIdx.x;
  int h = i / units, u = i - h * units, t = h / heads;
  h -= t * heads;
  const int dh = kThreads / units, du = kThreads - dh * units;
  while (i < end) {
    V va[kUnroll], vb[kUnroll];
    Move<T> mv[kUnroll];
    int tu[kUnroll], ea[kUnroll], eb[kUnroll];  // token and unit; element offsets, -1: none
    bool rot[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      mv[k].to = nullptr;
      if (i < end) {
        const int slot = slot_s[t];
        if (slot > -2) mv[k] = head_of<T>(p, (size_t)(row0 + t), h, slot);
        rot[k] = h < turned;
        tu[k] = t * 2 * kCol * turning + u;
        if (!INTER && rot[k] && u < turning) {
          ea[k] = u * VEC;
          eb[k] = half + u * VEC;
        } else {  // two vectors next to each other, past the turning part where there is one
          ea[k] = !INTER && rot[k] ? p.rot + 2 * (u - turning) * VEC : 2 * u * VEC;
          eb[k] = ea[k] + VEC;
          if (!INTER) rot[k] = false;
        }
        if (mv[k].to && ea[k] < p.D) va[k].raw = *reinterpret_cast<const uint4*>(mv[k].from + ea[k]);
        if (mv[k].to && eb[k] < p.D) vb[k].raw = *reinterpret_cast<const uint4*>(mv[k].from + eb[k]);
      }
      i += kThreads;
      u += du;
      h += dh;
      if (u >= units) {
        u -= units;
        ++h;
      }
      while (h >= heads && i < end) {
        h -= heads;
        ++t;
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (!mv[k].to) continue;
      if (rot[k]) {
        float4 c[kCol], s[kCol];
        if (!INTER || ea[k] < p.rot) {
#pragma unroll
          for (int j = 0; j < kCol; ++j) {
            c[j] = cs_s[tu[k] + j * turning];
            s[j] = cs_s[tu[k] + (kCol + j) * turning];
          }
        }
        const float* cf = reinterpret_cast<const float*>(c);
        const float* sf = reinterpret_cast<const float*>(s);
        if (!INTER) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) turn(va[k].e[e], vb[k].e[e], make_float2(cf[e], sf[e]));
        } else {
          if (ea[k] < p.rot) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) turn(va[k].e[e], va[k].e[e + 1], make_float2(cf[e / 2], sf[e / 2]));
          }
          if (eb[k] < p.rot) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2)
              turn(vb[k].e[e], vb[k].e[e + 1], make_float2(cf[VEC / 2 + e / 2], sf[VEC / 2 + e / 2]));
          }
        }
      }
      if (ea[k] < p.D) *reinterpret_cast<uint4*>(mv[k].to + ea[k]) = va[k].raw;
      if (eb[k] < p.D) *reinterpret_cast<uint4*>(mv[k].to + eb[k]) = vb[k].raw;
    }
  }
}

// The same, element by element: sizes, strides or addresses that are off 16 bytes.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(spec_rope_cache_args p, int tokens, int units,
                                                               int per_block) {
  extern __shared__ __align__(16) float2 cs2_s[];  // [tokens][rot / 2]
  __shared__ int slot_s[kRopeTokens];
  const int half = p.rot >> 1, heads = p.Hq + 2 * p.Hk;
  const int row0 = blockIdx.x * tokens, nrow = min(tokens, p.rows - row0);
  const int begin = blockIdx.y * per_block, end = min(begin + per_block, nrow * heads * units);
  for (int i = threadIdx.x; i < nrow * half; i += kThreads) {
    const int t = i / half;
    cs2_s[i] = cos_sin(position_of(p, row0 + t), p.freq[i - t * half], p.scale);
  }
  read_slots(p, row0, nrow, slot_s);
  __syncthreads();
  for (int i = begin + threadIdx.x; i < end; i += kThreads) {
    const int hh = i / units, u = i - hh * units, t = hh / heads, h = hh - t * heads;
    if (slot_s[t] < -1) continue;
    const Move<T> mv = head_of<T>(p, (size_t)(row0 + t), h, slot_s[t]);
    if (!mv.to) continue;
    if (h < p.Hq + p.Hk && u < half) {
      const int a = INTER ? 2 * u : u, b = INTER ? a + 1 : half + u;
      T x = mv.from[a], y = mv.from[b];
      turn(x, y, cs2_s[t * half + u]);
      mv.to[a] = x;
      mv.to[b] = y;
    } else {
      const int a = h < p.Hq + p.Hk ? p.rot + 2 * (u - half) : 2 * u;
      if (a < p.D) mv.to[a] = mv.from[a];
      if (a + 1 < p.D) mv.to[a + 1] = mv.from[a + 1];
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
  if constexpr (VEC == 1) {
    const size_t smem = (size_t)tokens * half * sizeof(float2);
    if (inter) rope_scalar_kernel<T, true><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
    else rope_scalar_kernel<T, false><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  } else {
    const size_t smem = (size_t)tokens * 2 * ((half + VEC - 1) / VEC) * VEC * sizeof(float);
    if (inter) rope_kernel<T, VEC, true><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
    else rope_kernel<T, VEC, false><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  }
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
