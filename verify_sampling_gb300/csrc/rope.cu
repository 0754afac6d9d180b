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
// Layout: a unit is two 16-byte vectors of a head: the two halves of its pairs in
// the half layout, two vectors next to each other otherwise; either way unit u
// takes the frequencies [u VEC, (u + 1) VEC).  A thread keeps one unit of one token
// and steps over the heads, queries, keys and values in turn, and then over a few
// more tokens, the next step's loads ahead of this step's products: its cosines and
// sines are read from shared memory once a token (one float4 column a unit, free of bank
// conflicts) and stay in registers, and a step is two loads, the products and two
// stores.  A thread's first loads go out before the cosines are computed.
// Bound by memory: every element is read and written once (2560 rows of 64 + 2 * 8
// heads of 128, bf16: 26.1 us, 4.0 TB/s; 40001 rows of 32 + 2 * 4 heads: 165 us, 5.0
// TB/s).  With units dealt out to threads one by one, each with its own addresses and
// cosines, the first took 40 us.
#include "rope.cuh"

#include <algorithm>
#include <climits>

namespace spec {

namespace {

constexpr int kThreads = 256;     // of the element-wise kernel
constexpr int kMaxThreads = 320;  // of the other: two blocks an SM at 96 registers (three spill: 98 us for 26)
constexpr int kUnroll = 2;
constexpr int kRopeTokens = 8;  // of a block
constexpr int kReps = 4;        // of a thread, one after the other

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

// Where head h of a row (queries, keys, values in turn) is read and written (null:
// nowhere).  A row that is left out is read all the same: its rows exist.
template <typename T>
__device__ __forceinline__ const T* source_of(const spec_rope_cache_args& p, size_t row, int h) {
  if (h < p.Hq) return (const T*)p.q + row * p.q_row + (size_t)h * p.q_head;
  if (h < p.Hq + p.Hk) return (const T*)p.k + row * p.k_row + (size_t)(h - p.Hq) * p.k_head;
  return (const T*)p.v + row * p.v_row + (size_t)(h - p.Hq - p.Hk) * p.v_head;
}
template <typename T>
__device__ __forceinline__ T* target_of(const spec_rope_cache_args& p, size_t row, int h, int slot) {
  if (slot < -1) return nullptr;
  if (h < p.Hq) return (T*)p.q_out + row * p.q_out_row + (size_t)h * p.q_out_head;
  if (slot < 0) return nullptr;
  const bool key = h < p.Hq + p.Hk;
  return (T*)(key ? p.k_cache : p.v_cache) +
         ((size_t)slot * p.Hk + (h - p.Hq - (key ? 0 : p.Hk))) * p.D;
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

// `group` threads take a token at a time: `heads_at_once` heads of `units` units, in
// `chunks` steps of kUnroll times that many heads.  `groups` of them share a block,
// and each takes `reps` tokens one after the other.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kMaxThreads, 2) rope_kernel(spec_rope_cache_args p, int groups, int reps, int units,
                                                              int heads_at_once, int chunks) {
  constexpr int VEC = 16 / (int)sizeof(T);
  constexpr int kCol = VEC / 4;  // float4s of a unit's cosines
  extern __shared__ __align__(16) float4 cs_s[];  // a token: cosines [kCol][turning], then sines
  struct Step {
    Vec<T, VEC> a[kUnroll], b[kUnroll];
  };
  const int half = p.rot >> 1, heads = p.Hq + 2 * p.Hk, turned = p.Hq + p.Hk;
  const int turning = (half + VEC - 1) / VEC;  // units that turn
  const int group = units * heads_at_once;
  const int row0 = blockIdx.x * groups * reps, nrow = min(groups * reps, p.rows - row0);
  const int g = threadIdx.x / group, in_group = threadIdx.x - g * group;
  const int h0 = in_group / units, u = in_group - h0 * units;

  // the unit's elements in a head that turns and in a value head; past the head: none
  const bool turns = INTER || u < turning;
  const int ra = INTER ? 2 * u * VEC : turns ? u * VEC : p.rot + 2 * (u - turning) * VEC;
  const int rb = !INTER && turns ? half + u * VEC : ra + VEC;
  const int va = 2 * u * VEC, vb = va + VEC;
  const int q_head = (int)p.q_head, k_head = (int)p.k_head, v_head = (int)p.v_head, o_head = (int)p.q_out_head;
  const int steps = reps * chunks;

  // (a row that is left out is read all the same: no load waits for a position)
  auto load = [&](int step, Step& x) {
    const int rep = step / chunks, t = rep * groups + g;
    if (t >= nrow) return;
    const size_t row = (size_t)(row0 + t);
    const int hb = h0 + (step - rep * chunks) * kUnroll * heads_at_once;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = hb + i * heads_at_once;
      if (h >= heads) break;
      const T* from = h < p.Hq     ? (const T*)p.q + row * p.q_row + (int64_t)h * q_head
                      : h < turned ? (const T*)p.k + row * p.k_row + (int64_t)(h - p.Hq) * k_head
                                   : (const T*)p.v + row * p.v_row + (int64_t)(h - turned) * v_head;
      const int a = h < turned ? ra : va, b = h < turned ? rb : vb;
      if (a < p.D) x.a[i].raw = *reinterpret_cast<const uint4*>(from + a);
      if (b < p.D) x.b[i].raw = *reinterpret_cast<const uint4*>(from + b);
    }
  };
  float c[VEC], s[VEC];
  int pos = -1, slot = -1;
  auto store = [&](int step, Step& x) {
    const int rep = step / chunks, t = rep * groups + g;
    if (t >= nrow) return;
    const size_t row = (size_t)(row0 + t);
    if (step == rep * chunks) {  // the token's first step
      pos = p.position[row];
      slot = p.slot ? p.slot[row] : -1;
      if (in_group == 0) {
        const uint32_t bad = (pos >= (1 << 24) ? SPEC_STATUS_BAD_POSITION : 0u) |
                             (slot >= p.n_slots ? SPEC_STATUS_BAD_PAGE : 0u);
        if (bad) set_status(p.status, bad);
      }
      if (slot >= p.n_slots) slot = -1;
      if (u < turning) {
        const float4* col = cs_s + (size_t)t * 2 * kCol * turning + u;
#pragma unroll
        for (int j = 0; j < kCol; ++j) {
          const float4 m = col[j * turning], n = col[(kCol + j) * turning];
          c[4 * j] = m.x, c[4 * j + 1] = m.y, c[4 * j + 2] = m.z, c[4 * j + 3] = m.w;
          s[4 * j] = n.x, s[4 * j + 1] = n.y, s[4 * j + 2] = n.z, s[4 * j + 3] = n.w;
        }
      }
    }
    if (pos < 0) return;
    const int hb = h0 + (step - rep * chunks) * kUnroll * heads_at_once;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = hb + i * heads_at_once;
      if (h >= heads) break;
      if (h < turned) {
        if (INTER) {
          if (ra < p.rot) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) turn(x.a[i].e[e], x.a[i].e[e + 1], make_float2(c[e / 2], s[e / 2]));
          }
          if (rb < p.rot) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2)
              turn(x.b[i].e[e], x.b[i].e[e + 1], make_float2(c[VEC / 2 + e / 2], s[VEC / 2 + e / 2]));
          }
        } else if (turns) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) turn(x.a[i].e[e], x.b[i].e[e], make_float2(c[e], s[e]));
        }
      }
      if (h >= p.Hq && slot < 0) continue;
      T* to = h < p.Hq     ? (T*)p.q_out + row * p.q_out_row + (int64_t)h * o_head
              : h < turned ? (T*)p.k_cache + ((size_t)slot * p.Hk + (h - p.Hq)) * p.D
                           : (T*)p.v_cache + ((size_t)slot * p.Hk + (h - turned)) * p.D;
      const int a = h < turned ? ra : va, b = h < turned ? rb : vb;
      if (a < p.D) *reinterpret_cast<uint4*>(to + a) = x.a[i].raw;
      if (b < p.D) *reinterpret_cast<uint4*>(to + b) = x.b[i].raw;
    }
  };

  Step x, y;
  load(0, x);
  // the first step's data is on its way: now the cosines it waits for, of all the block's tokens
  for (int i = threadIdx.x; i < nrow * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    const float2 cs = cos_sin(position_of(p, row0 + t), p.freq[f], p.scale);
    const int uf = f / VEC, e = f % VEC;
    float* to = reinterpret_cast<float*>(cs_s + (size_t)t * 2 * kCol * turning + (e / 4) * turning + uf) + e % 4;
    to[0] = cs.x;
    to[4 * kCol * turning] = cs.y;
  }
  __syncthreads();
  for (int step = 0; step < steps; step += 2) {
    if (step + 1 < steps) load(step + 1, y);
    store(step, x);
    if (step + 1 >= steps) break;
    if (step + 2 < steps) load(step + 2, x);
    store(step + 1, y);
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
    const T* from = source_of<T>(p, (size_t)(row0 + t), h);
    T* to = target_of<T>(p, (size_t)(row0 + t), h, slot_s[t]);
    if (!to) continue;
    if (h < p.Hq + p.Hk && u < half) {
      const int a = INTER ? 2 * u : u, b = INTER ? a + 1 : half + u;
      T x = from[a], y = from[b];
      turn(x, y, cs2_s[t * half + u]);
      to[a] = x;
      to[b] = y;
    } else {
      const int a = h < p.Hq + p.Hk ? p.rot + 2 * (u - half) : 2 * u;
      if (a < p.D) to[a] = from[a];
      if (a + 1 < p.D) to[a + 1] = from[a + 1];
    }
  }
}

template <typename T>
cudaError_t launch_wide(const spec_rope_cache_args& a, cudaStream_t stream) {
  constexpr int VEC = 16 / (int)sizeof(T);
  const bool inter = a.layout == SPEC_ROPE_INTERLEAVED;
  const int half = a.rot / 2, heads = a.Hq + 2 * a.Hk;
  const int copied = (a.D + 2 * VEC - 1) / (2 * VEC);
  const int turned = inter ? copied : half / VEC + (a.D - a.rot + 2 * VEC - 1) / (2 * VEC);
  const int units = std::max(copied, turned);
  // Heads at once: a token's heads over a group of threads, kUnroll a thread
  // where there are rows enough; with few rows one, so that a token is one step.
  const int share = a.rows >= 304 ? kUnroll : 1;
  const int most = std::max(1, kMaxThreads / units);
  const int at_once = std::min(most, (heads + share - 1) / share);
  const int chunks = (heads + kUnroll * at_once - 1) / (kUnroll * at_once);
  const int group = units * at_once;
  const int groups = std::max(1, std::min({kRopeTokens, kMaxThreads / group, std::max(1, a.rows / 304)}));
  // As many tokens a thread as fill whole rounds of blocks best; a block's start costs
  // about two tokens (2560 rows of 80 heads: 25.9 us with three, 29.5 with four in 2.1
  // rounds, 31.2 with one).
  const int slots = 152 * std::max(1, 2 * kMaxThreads / (group * groups));
  int reps = 1, best = INT_MAX;
  for (int r = std::min(kReps, kRopeTokens / groups); r >= 1; --r) {
    const int blocks = (a.rows + groups * r - 1) / (groups * r), cost = (blocks + slots - 1) / slots * (r + 2);
    if (cost < best) {
      best = cost;
      reps = r;
    }
  }
  const size_t smem = (size_t)groups * reps * 2 * ((half + VEC - 1) / VEC) * VEC * sizeof(float);
  const dim3 grid((a.rows + groups * reps - 1) / (groups * reps));
  if (inter) rope_kernel<T, true><<<grid, group * groups, smem, stream>>>(a, groups, reps, units, at_once, chunks);
  else rope_kernel<T, false><<<grid, group * groups, smem, stream>>>(a, groups, reps, units, at_once, chunks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scalar(const spec_rope_cache_args& a, cudaStream_t stream) {
  const int half = a.rot / 2, heads = a.Hq + 2 * a.Hk;
  const int units = std::max((a.D + 1) / 2, half + (a.D - a.rot + 1) / 2);
  const long long per_token = (long long)heads * units;
  const int tokens = (int)std::min<long long>(std::min(kRopeTokens, std::max(1, a.rows / 304)),
                                              std::max(1ll, 1024 / std::max(1ll, per_token)));
  const int per_block = a.rows < 304 ? kThreads : tokens == 1 ? 1024 : (int)(tokens * per_token);
  const int parts = (int)((tokens * per_token + per_block - 1) / per_block);
  const dim3 grid((a.rows + tokens - 1) / tokens, std::max(1, parts));
  const size_t smem = (size_t)tokens * half * sizeof(float2);
  if (a.layout == SPEC_ROPE_INTERLEAVED)
    rope_scalar_kernel<T, true><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  else
    rope_scalar_kernel<T, false><<<grid, kThreads, smem, stream>>>(a, tokens, units, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_cache(const spec_rope_cache_args& a, cudaStream_t stream) {
  if (a.rows == 0 || a.Hq + a.Hk == 0) return cudaSuccess;
  // 16-byte vectors where every row, head, half and remainder starts on one
  const int vec = a.dtype == SPEC_F32 ? 4 : 8;
  const int turn_step = a.layout == SPEC_ROPE_HALF ? a.rot / 2 : a.rot;
  auto on = [&](const void* p) { return ((uintptr_t)p % 16) == 0; };
  auto small = [](int64_t stride) { return stride >= 0 && stride < ((int64_t)1 << 31); };
  const bool wide =
      a.D % vec == 0 && turn_step % vec == 0 && a.rot % vec == 0 && a.q_row % vec == 0 &&
      a.q_head % vec == 0 && a.q_out_row % vec == 0 && a.q_out_head % vec == 0 && a.k_row % vec == 0 &&
      a.k_head % vec == 0 && a.v_row % vec == 0 && a.v_head % vec == 0 && on(a.q) && on(a.k) &&
      on(a.v) && on(a.q_out) && on(a.k_cache) && on(a.v_cache) && small(a.q_head) && small(a.k_head) &&
      small(a.v_head) && small(a.q_out_head);
  if (a.dtype == SPEC_F32) return wide ? launch_wide<float>(a, stream) : launch_scalar<float>(a, stream);
  return wide ? launch_wide<__nv_bfloat16>(a, stream) : launch_scalar<__nv_bfloat16>(a, stream);
}

}  // namespace spec
