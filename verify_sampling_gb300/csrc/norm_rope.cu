// Norms of query and key heads with rotary positions, keys and values written to a paged
// cache of the inputs' type or of 4 bits; and the read-back of such a cache.
//
// Mathematics: y = x w rsqrt(mean x^2 + eps), then pair i of a head turns by the angle
// position * freq[i] (rotary.cuh), all in fp32 from one read of the head, rounded once at
// the end: to the stored type, or to the nearest of a group's 15 values (packed.cuh).
// A head whose mean square + eps is outside [2^-90, 2^90] is computed again, times a power of two
// (norm_turn).  Asking for that costs every head a comparison and a vote, 1 to 3.5%: 2560 rows of 80 heads
// 25.3 and 25.8 us, 40001 rows of 40 heads 133.8 and 138.2.  (A pass over all of a token's heads, and
// another where one was not in range: 26.4 and 136, and 31.5 us for 30.8 at 2560 rows into 4 bits.)
//
// Layout: a head lies over a group of lanes, a 16-byte vector each, in the order of its
// elements, so that a load, a store, a group of 32 elements to code and a head's sum of
// squares are each a few lanes side by side.  A pair's other half comes from its lane by a shuffle, and
// what a lane's elements are taken times (weights, cosines, sines) stays in its registers over
// a token's heads.
//
// Heads that lie side by side (norm_rope_bulk_kernel): bulk copies through a ring of tokens in
// shared memory.  Strided heads and small batches of small rows (norm_rope_kernel): a warp takes a
// part of a token's heads, four steps' loads together.  Pairs that are not whole vectors,
// larger heads and odd strides (norm_rope_general_kernel): other halves from shared memory.
// The first two give a row the same bits.
// Figures are of launches one after another over 400 MB of inputs.  Bound by memory in long batches: 40001
// rows of 40 heads of 128 in bf16, half of a head turned, 138 us (5.9 TB/s; this ring without arithmetic 126), 2560 rows of
// 80 heads 25.8 (21; the rotary kernel's ring, two blocks an SM of four stages, moves and turns them in 18.5), where the second
// kernel takes 274 and 55.  Rows of 20 KB: one row 4.9 and 5.6 us, 456 rows 8.3 and 13.5; rows of 5 KB: 76
// rows 3.8 and 5.7, 2432 rows 11.6 and 18.6; rows of 1.2 KB: 2432 rows 8.4 and 7.8, 4864 rows 12.4
// and 13.9, hence kBulkRow and kBulkBytes.  fp32: 2560 rows of 48 heads 27.8 us (36.4; at the copy rate 18.5), 40001 of 24
// 152 (209; 145).  Three blocks an SM for two: 24.9 and 26.5 us at 2560 rows.  Into 4 bits the arithmetic
// of the coding counts as well (0.6 instructions a clock and scheduler): 2560 rows 30 us (the second kernel 55), 9000 rows of
// 48 heads 63 (94).  Three blocks of 64 registers took 37 us for 37.7 and, with smaller stages, 88 for 82 (both with the
// read-back), so these have two.  The third kernel serves what is rare: 2560 rows of 40 heads of 80, 74 of them turned,
// 56 us (4.8 at the copy rate), of 24 heads of 512 180 (18.5), of 32 heads of 256 in fp32 65 (24.7).
#include "norm_rope.cuh"

#include <algorithm>
#include <type_traits>

#include "packed.cuh"
#include "rotary.cuh"
#include "tc.cuh"

namespace spec {

namespace {

using rotary::cos_sin;
using rotary::in_turns;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSteps = 4;  // loads of a lane on their way together

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T e[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

// A lane's 16 bytes of a head, normed and turned.  What an element and the other half of its pair
// are taken times (the weight's part of it, cosine or signed sine) is the same for all heads of
// a token and kind: mine[e] and others[e]; the head's 1 / rms comes last.
template <typename T>
struct Lane {
  static constexpr int VEC = 16 / (int)sizeof(T);
  uint64_t mine[VEC / 2], others[VEC / 2];
  bool turning;  // the lane's elements are below rot
};
__device__ __forceinline__ void unpack(const uint4& v, uint64_t (&x)[4], __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = tc::pair(w[e] << 16, w[e] & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const uint4& v, uint64_t (&x)[2], float) {
  x[0] = tc::pair(v.x, v.y);
  x[1] = tc::pair(v.z, v.w);
}
__device__ __forceinline__ uint4 packed_up(const uint64_t (&y)[4], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = tc::halves(y[e]);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(v.y), "f"(v.x));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 packed_up(const uint64_t (&y)[2], float) {
  const float2 a = tc::halves(y[0]), b = tc::halves(y[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}
// The lane's factors from cosines and signed sines (co, si; read where `turning`) and the head's weight.
template <typename T, bool INTER>
__device__ __forceinline__ void factors(Lane<T>& f, const float* co, const float* si, const float* weight, int first, int half) {
  constexpr int VEC = Lane<T>::VEC;
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    float m[2], o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = first + e + k, at = INTER ? d ^ 1 : d < half ? d + half : d - half;
      m[k] = f.turning ? co[e + k] : 1.f;
      o[k] = f.turning ? si[e + k] : 0.f;
      if (weight) {
        m[k] *= weight[d];
        if (f.turning) o[k] *= weight[at];
      }
    }
    f.mine[e / 2] = tc::pair(m[0], m[1]);
    f.others[e / 2] = tc::pair(o[0], o[1]);
  }
}
// 1 / sqrt(x) of a normal number, 0 or infinity.
__device__ __forceinline__ float rsqrt_of(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A mean square + eps in the middle of fp32's range: squares that vanished beside it do no harm, nor do its elements'
// products with weights to 2^77.
__device__ __forceinline__ bool in_range(float square) {
  constexpr uint32_t kLeast = (127u - 90) << 23, kMost = (127u + 90) << 23;
  return __float_as_uint(square) - kLeast <= kMost - kLeast;  // (a NaN's bits lie past them)
}
// The power of two that brings the larger of a head's largest magnitude (its bits) and sqrt(eps) to [1/4, 1/2): the head
// times it has the same norm, with eps times its square, and squares, sums and products of ordinary size.
__device__ __forceinline__ float unit_of(uint32_t most, float eps) {
  const int f = 252 - (int)min(max(most, __float_as_uint(sqrtf(eps))) >> 23, 254u);
  return __uint_as_float(f > 0 ? (uint32_t)f << 23 : 0x400000u >> -f);
}
// All lanes of a warp call it; a head is `lanes` of them, `other` the lane of the other halves (half layout).
// `load(again)` gives the lane's elements; a head out of range asks for them again (kept, they would take registers of all).
template <typename T, bool INTER, class Load>
__device__ __forceinline__ void norm_turn(Load load, uint64_t (&y)[Lane<T>::VEC / 2], const Lane<T>& f, bool norm, int lanes, int other,
                                          float inv_d, float eps) {
  constexpr int N = Lane<T>::VEC / 2;
  uint64_t x[N], z[N];
  auto elements = [&](auto again) {
    const uint4 v = load(again);
    unpack(v, x, T());
    if (INTER) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 t = tc::halves(x[e]);
        z[e] = tc::pair(t.y, t.x);
      }
    } else {
      uint4 w;
      w.x = __shfl_sync(0xffffffffu, v.x, other), w.y = __shfl_sync(0xffffffffu, v.y, other);
      w.z = __shfl_sync(0xffffffffu, v.z, other), w.w = __shfl_sync(0xffffffffu, v.w, other);
      unpack(w, z, T());
    }
    if (!f.turning) {
#pragma unroll
      for (int e = 0; e < N; ++e) z[e] = 0;  // (what is not its pair may be NaN)
    }
  };
  auto turned = [&] {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = tc::fma2(x[e], f.mine[e], tc::mul2(z[e], f.others[e]));
  };
  auto squares = [&] {
    uint64_t sum2 = tc::mul2(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < N; ++e) sum2 = tc::fma2(x[e], x[e], sum2);
    const float2 s = tc::halves(sum2);
    float sum = s.x + s.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o < lanes) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
  };
  elements(std::false_type{});
  turned();
  if (!norm) {
    if (!f.turning) {
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = x[e];  // (its sign, where it is zero)
    }
    return;
  }
  float square = fmaf(squares(), inv_d, eps);
  if (!__all_sync(0xffffffffu, in_range(square))) {
    elements(std::true_type{});
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float2 t = tc::halves(x[e]);
      most = max(most, max(__float_as_uint(fabsf(t.x)), __float_as_uint(fabsf(t.y))));
    }
    for (int o = 1; o < lanes; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float unit = in_range(square) ? 1.f : unit_of(most, eps);  // each head by itself: its bits do not depend on its neighbours
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e] = tc::mul2(x[e], tc::pair(unit, unit));
      z[e] = tc::mul2(z[e], tc::pair(unit, unit));
    }
    turned();
    square = fmaf(squares(), inv_d, eps * unit * unit);
  }
  const float r = rsqrt_of(square);
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = tc::mul2(y[e], tc::pair(r, r));
}
template <int N>
__device__ __forceinline__ void spread(const uint64_t (&y)[N], float (&to)[2 * N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float2 v = tc::halves(y[e]);
    to[2 * e] = v.x;
    to[2 * e + 1] = v.y;
  }
}

// The larger magnitude, NaN where either is one.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ float larger(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// Codes of M groups' scales and a lane's VEC elements of each as nibbles, for all lanes of the
// warp; side by side, as each is a chain of dependent steps.
template <int VEC, int M>
__device__ __forceinline__ void code_groups(float (&y)[M][VEC], uint32_t (&w)[M], uint32_t (&code)[M]) {
  auto codes = [&] {
    float most[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      most[m] = fabsf(y[m][0]);
#pragma unroll
      for (int e = 1; e + 1 < VEC; e += 2) most[m] = larger(most[m], y[m][e], y[m][e + 1]);
      if (VEC % 2 == 0) most[m] = larger(most[m], y[m][VEC - 1]);
    }
#pragma unroll
    for (int o = 1; o < q4::kGroup / VEC; o <<= 1)
#pragma unroll
      for (int m = 0; m < M; ++m) most[m] = larger(most[m], __shfl_xor_sync(0xffffffffu, most[m], o));
    uint32_t largest = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) largest = max(largest, code[m] = q4::code_of(most[m]));
    return largest;
  };
  if (__any_sync(0xffffffffu, codes() == 255)) {  // NaN is stored as 0, what is past the largest scale as 7 of it
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (y[m][e] != y[m][e]) y[m][e] = 0.f;
    codes();
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[m][e] = fminf(fmaxf(y[m][e], -7.f * q4::scale_of(code[m])), 7.f * q4::scale_of(code[m]));
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float s = q4::scale_of(code[m]);
    w[m] = q4::nibbles_of(y[m], s, q4::reciprocal(s));
  }
}

// Codes a lane's VEC elements of each chunk and writes them to the token's head in the cache.
// All lanes of the warp call it; `on`: this one's head is written.
template <int VEC, int CH>
__device__ __forceinline__ void store_packed(const float (&from)[CH * VEC], int first, int step, int D, bool on, uint8_t* data,
                                             uint8_t* scale, int P) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int d = first + c * step;  // this lane's first element
    float y[1][VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[0][e] = from[c * VEC + e];
    uint32_t words[1], code[1];
    code_groups<VEC, 1>(y, words, code);
    uint32_t w = words[0];
    if (VEC < 8) w <<= 4 * (d & 7);
#pragma unroll
    for (int o = 1; o < 8 / VEC; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
    if (!on || d >= D) continue;
    const int g = d / q4::kGroup, in_g = d % q4::kGroup;
    if (in_g % 8 == 0) *reinterpret_cast<uint32_t*>(data + (size_t)g * 16 * P + in_g / 2) = w;
    if (in_g == 0) scale[g] = (uint8_t)code[0];
  }
}

// Whole vectors that turn or do not: a head over `lanes` lanes (a power of two).
template <typename T, bool INTER, bool PACKED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(spec_norm_rope_args p, int parts, int lanes) {
  constexpr int VEC = Lane<T>::VEC, N = VEC / 2;
  extern __shared__ __align__(16) float2 smem[];
  const int half = p.rot >> 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* turns = smem;                    // [half]
  float2* cs = smem + half + warp * half;  // [half] of the warp's token
  for (int f = tid; f < half; f += kThreads) turns[f] = in_turns(p.freq[f]);
  __syncthreads();

  const int at_once = 32 / lanes, sub = lane / lanes, first = (lane % lanes) * VEC;
  const int q_steps = (p.Hq + at_once - 1) / at_once, k_steps = (p.Hk + at_once - 1) / at_once;
  const int steps = q_steps + 2 * k_steps, per = (steps + parts - 1) / parts;
  const float inv_d = 1.f / (float)p.D;
  const bool live = first < p.D;
  const int other = (lane + (first < half ? half : -half) / VEC) & 31;  // half layout: where the other halves lie
  const int64_t units = (int64_t)p.rows * parts;
  auto kind_of = [&](int st) { return st < q_steps ? 0 : st < q_steps + k_steps ? 1 : 2; };  // queries, keys, values
  auto head_of = [&](int st, int kind) { return (st - (kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + k_steps)) * at_once + sub; };

  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units; unit += (int64_t)gridDim.x * kWarps) {
    const int row = (int)(unit / parts), part = (int)(unit - (int64_t)row * parts);
    const int begin = part * per, end = min(begin + per, steps);
    uint4 x[kSteps];
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int st = s0 + i;
        if (st >= end) break;
        const int kind = kind_of(st), h = head_of(st, kind);
        const T* from = kind == 0   ? (const T*)p.q + (int64_t)row * p.q_row + h * p.q_head
                        : kind == 1 ? (const T*)p.k + (int64_t)row * p.k_row + h * p.k_head
                                    : (const T*)p.v + (int64_t)row * p.v_row + h * p.v_head;
        x[i] = make_uint4(0, 0, 0, 0);
        if (h < (kind == 0 ? p.Hq : p.Hk) && live) x[i] = *reinterpret_cast<const uint4*>(from + first);
      }
    };
    load(begin);  // a row that is left out is read all the same: no load waits for a position
    const int pos = p.position[row];
    int slot = p.slot ? p.slot[row] : -1;
    if (part == 0 && lane == 0) {
      const uint32_t bad = (pos >= (1 << 24) ? SPEC_STATUS_BAD_POSITION : 0u) | (slot >= p.n_slots ? SPEC_STATUS_BAD_PAGE : 0u);
      if (bad) set_status(p.status, bad);
    }
    if (pos < 0) continue;
    if (slot >= p.n_slots) slot = -1;
    const float at = (float)min(pos, (1 << 24) - 1);
    __syncwarp();
    for (int f = lane; f < half; f += 32) cs[f] = cos_sin(at, turns[f], p.scale);
    __syncwarp();
    Lane<T> lf;
    lf.turning = first < p.rot;
    float co[VEC], si[VEC];
    if (lf.turning) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 t = cs[INTER ? (first + e) / 2 : first < half ? first + e : first + e - half];
        co[e] = t.x;
        si[e] = (INTER ? e % 2 == 0 : first < half) ? -t.y : t.y;
      }
    }
    int have = -1;  // kind whose factors these are
    const int64_t page = PACKED && slot >= 0 ? slot / p.page_size : 0;
    const int tok = PACKED && slot >= 0 ? (int)(slot - page * p.page_size) : 0, groups = p.D / q4::kGroup;

    for (int s0 = begin; s0 < end; s0 += kSteps) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int st = s0 + i;
        if (st >= end) break;
        const int kind = kind_of(st), h = head_of(st, kind);
        const bool on = h < (kind == 0 ? p.Hq : p.Hk) && (kind == 0 || slot >= 0);
        uint64_t y[N];
        if (kind == 2) {
          unpack(x[i], y, T());
        } else {
          const float* weight = kind == 0 ? p.q_weight : p.k_weight;
          if (kind != have) {
            factors<T, INTER>(lf, co, si, live ? weight : nullptr, first, half);
            have = kind;
          }
          norm_turn<T, INTER>([&](auto) { return x[i]; }, y, lf, weight != nullptr, lanes, other, inv_d, p.eps);
        }
        if (PACKED && kind > 0) {
          float yf[VEC];
          spread(y, yf);
          const int head = on ? h : 0;
          store_packed<VEC, 1>(yf, first, 32 * VEC, p.D, on,
                               (uint8_t*)(kind == 1 ? p.k_cache : p.v_cache) + q4::data_at(page, head, tok, p.Hk, groups, p.page_size),
                               (kind == 1 ? p.k_scale : p.v_scale) + q4::scale_at(page, head, tok, p.Hk, groups, p.page_size), p.page_size);
          continue;
        }
        if (!on || !live) continue;
        T* to = kind == 0 ? (T*)p.q_out + (int64_t)row * p.q_out_row + h * p.q_out_head
                          : (T*)(kind == 1 ? p.k_cache : p.v_cache) + ((int64_t)slot * p.Hk + h) * p.D;
        *reinterpret_cast<uint4*>(to + first) = kind == 2 ? x[i] : packed_up(y, T());
      }
      if (s0 + kSteps < end) load(s0 + kSteps);
    }
  }
}

// Any sizes: a head over `lanes` lanes (a power of two), or over the whole warp in CH chunks of 32 VEC
// elements; the other halves of pairs come from shared memory.
template <typename T, int VEC, int CH, bool PACKED>
__global__ void __launch_bounds__(kThreads) norm_rope_general_kernel(spec_norm_rope_args p, int parts, int lanes) {
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) float2 smem[];
  const int half = p.rot >> 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* turns = smem;                         // [half]
  float2* cs = smem + half + warp * half;       // [half] of the warp's token
  float* buf = reinterpret_cast<float*>(smem + half * (1 + kWarps)) + warp * 32 * VEC * CH;  // its heads
  for (int f = tid; f < half; f += kThreads) turns[f] = in_turns(p.freq[f]);
  __syncthreads();

  const int at_once = CH == 1 ? 32 / lanes : 1;
  const int sub = CH == 1 ? lane / lanes : 0, l = CH == 1 ? lane % lanes : lane;
  const int first = l * VEC, step = 32 * VEC;  // element e of chunk c is first + c * step + e
  const bool inter = p.layout == SPEC_ROPE_INTERLEAVED;
  const int q_steps = (p.Hq + at_once - 1) / at_once, k_steps = (p.Hk + at_once - 1) / at_once;
  const int steps = q_steps + 2 * k_steps, per = (steps + parts - 1) / parts;
  const float inv_d = 1.f / (float)p.D;
  const int64_t units = (int64_t)p.rows * parts;

  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units; unit += (int64_t)gridDim.x * kWarps) {
    const int row = (int)(unit / parts), part = (int)(unit - (int64_t)row * parts);
    const int begin = part * per, end = min(begin + per, steps);
    P x[kSteps][CH];
    // kind 0: queries, 1: keys, 2: values
    auto kind_of = [&](int st) { return st < q_steps ? 0 : st < q_steps + k_steps ? 1 : 2; };
    auto head_of = [&](int st, int kind) { return (st - (kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + k_steps)) * at_once + sub; };
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int st = s0 + i;
        if (st >= end) break;
        const int kind = kind_of(st), h = head_of(st, kind);
        const T* from = kind == 0   ? (const T*)p.q + (int64_t)row * p.q_row + h * p.q_head
                        : kind == 1 ? (const T*)p.k + (int64_t)row * p.k_row + h * p.k_head
                                    : (const T*)p.v + (int64_t)row * p.v_row + h * p.v_head;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (h < (kind == 0 ? p.Hq : p.Hk) && first + c * step < p.D) x[i][c] = *reinterpret_cast<const P*>(from + first + c * step);
      }
    };
    load(begin);  // a row that is left out is read all the same: no load waits for a position
    const int pos = p.position[row];
    int slot = p.slot ? p.slot[row] : -1;
    if (part == 0 && lane == 0) {
      const uint32_t bad = (pos >= (1 << 24) ? SPEC_STATUS_BAD_POSITION : 0u) | (slot >= p.n_slots ? SPEC_STATUS_BAD_PAGE : 0u);
      if (bad) set_status(p.status, bad);
    }
    if (pos < 0) continue;
    if (slot >= p.n_slots) slot = -1;
    const float at = (float)min(pos, (1 << 24) - 1);
    __syncwarp();
    for (int f = lane; f < half; f += 32) cs[f] = cos_sin(at, turns[f], p.scale);
    __syncwarp();
    for (int s0 = begin; s0 < end; s0 += kSteps) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int st = s0 + i;
        if (st >= end) break;
        const int kind = kind_of(st), h = head_of(st, kind);
        const bool on = h < (kind == 0 ? p.Hq : p.Hk) && (kind == 0 || slot >= 0);
        if (kind == 2 && !PACKED) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (on && first + c * step < p.D)
              *reinterpret_cast<P*>((T*)p.v_cache + ((int64_t)slot * p.Hk + h) * p.D + first + c * step) = x[i][c];
          continue;
        }
        float y[CH * VEC];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < VEC; ++e) y[c * VEC + e] = first + c * step < p.D ? to_f(x[i][c].e[e]) : 0.f;
        const float* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
        if (weight) {
          auto squares = [&] {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < CH * VEC; ++e) sum = fmaf(y[e], y[e], sum);
            for (int o = 1; o < (CH == 1 ? lanes : 32); o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            return sum;
          };
          float square = fmaf(squares(), inv_d, p.eps);
          if (!__all_sync(0xffffffffu, in_range(square))) {  // as norm_turn
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < CH * VEC; ++e) most = max(most, __float_as_uint(fabsf(y[e])));
            for (int o = 1; o < (CH == 1 ? lanes : 32); o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float unit = in_range(square) ? 1.f : unit_of(most, p.eps);
#pragma unroll
            for (int e = 0; e < CH * VEC; ++e) y[e] *= unit;
            square = fmaf(squares(), inv_d, p.eps * unit * unit);
          }
          const float r = rsqrt_of(square);
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (first + c * step < p.D)
#pragma unroll
              for (int e = 0; e < VEC; ++e) y[c * VEC + e] *= r * weight[first + c * step + e];
        }
        if (kind < 2 && half > 0) {
          float* mine = buf + sub * lanes * VEC;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) mine[first + c * step + e] = y[c * VEC + e];
          __syncwarp();
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const int d = first + c * step + e;
              if (d >= p.rot) continue;
              const bool low = inter ? d % 2 == 0 : d < half;
              const float2 t = cs[inter ? d / 2 : low ? d : d - half];
              const float z = mine[inter ? d ^ 1 : low ? d + half : d - half];
              y[c * VEC + e] = fmaf(y[c * VEC + e], t.x, __fmul_rn(z, low ? -t.y : t.y));
            }
        }
        if (PACKED && kind > 0) {
          const int64_t page = on ? slot / p.page_size : 0;
          const int tok = on ? (int)(slot - page * p.page_size) : 0, groups = p.D / q4::kGroup, head = on ? h : 0;
          store_packed<VEC, CH>(y, first, step, p.D, on,
                              (uint8_t*)(kind == 1 ? p.k_cache : p.v_cache) + q4::data_at(page, head, tok, p.Hk, groups, p.page_size),
                              (kind == 1 ? p.k_scale : p.v_scale) + q4::scale_at(page, head, tok, p.Hk, groups, p.page_size),
                              p.page_size);
          continue;
        }
        if (!on) continue;
        T* to = kind == 0 ? (T*)p.q_out + (int64_t)row * p.q_out_row + h * p.q_out_head
                          : (T*)p.k_cache + ((int64_t)slot * p.Hk + h) * p.D;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          P o;
#pragma unroll
          for (int e = 0; e < VEC; ++e) put(&o.e[e], y[c * VEC + e]);
          if (first + c * step < p.D) *reinterpret_cast<P*>(to + first + c * step) = o;
        }
      }
      if (s0 + kSteps < end) load(s0 + kSteps);
    }
  }
}

// ---------------------------------------------------------------- bulk rows --
// Rows whose heads lie side by side, by bulk copies through a ring of stages in shared
// memory, a few tokens each: one warp issues loads and stores, one computes the
// cosines of the stages ahead, the others take heads as above, in place where a bulk store
// takes them on (queries, and the keys of a cache of the inputs' type).  Every wait is bounded: on
// a timeout the block sets SPEC_STATUS_TIMEOUT, waits for its copies in flight and returns.
constexpr int kBulkThreads = kThreads + 64;
constexpr int bulk_blocks(bool packed) { return packed ? 2 : 3; }  // an SM
constexpr int kMaxStages = 4;
constexpr uint64_t kWaitNs = 2000000000ull;

template <bool PACKED>
struct Ring {
  uint64_t full[kMaxStages], done[kMaxStages], freed[kMaxStages];
  int2 at[kMaxStages][kWarps];  // position (-1: left out) and slot (-1: none) of a stage's tokens
  longlong2 packed_at[PACKED ? kMaxStages : 1][kWarps];  // first bytes of the slots' data and scales in a cache of 4 bits
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t phase) {
  return tc::mbar_try_wait(bar, phase & 1u) || tc::mbar_wait(bar, phase & 1u, kWaitNs);
}

// Stage i of the block holds tokens (blockIdx.x + i * gridDim.x) * tokens and on; `tokens`
// divides the warps.
template <typename T, bool INTER, bool PACKED>
__global__ void __launch_bounds__(kBulkThreads, bulk_blocks(PACKED))
    norm_rope_bulk_kernel(spec_norm_rope_args p, int tokens, int stages, int lanes) {
  constexpr int VEC = Lane<T>::VEC, N = VEC / 2;
  extern __shared__ __align__(128) uint8_t bulk_s[];
  const int half = p.rot >> 1, turned = p.Hq + p.Hk;
  const uint32_t head_bytes = p.D * (uint32_t)sizeof(T), row_bytes = (turned + p.Hk) * head_bytes;
  const uint32_t stage_bytes = tokens * row_bytes;
  Ring<PACKED>& ring = *reinterpret_cast<Ring<PACKED>*>(bulk_s + stages * stage_bytes);
  float2* turns = reinterpret_cast<float2*>(&ring + 1);
  float* weight_s = reinterpret_cast<float*>(turns + ((half + 1) & ~1));  // [queries, keys][D]
  // what a lane's elements and the others of their pairs are taken times:
  // [stage][token][queries, keys][mine, others][VEC / 4][lane] float4
  float* factor_s = weight_s + 2 * p.D;
  const int head_lanes = p.D / VEC;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (p.rows + tokens - 1) / tokens;
  const int n = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  auto first_row = [&](int i) { return ((int)blockIdx.x + i * (int)gridDim.x) * tokens; };
  constexpr int kLoader = kWarps, kCosines = kWarps + 1;

  auto load = [&](int i) {  // queries, keys and values of a stage's tokens
    const int row0 = first_row(i), count = min(tokens, p.rows - row0), st = i % stages;
    if (lane == 0) tc::mbar_expect_tx(&ring.full[st], count * row_bytes);
    __syncwarp();
    if (lane < 3 * count) {
      const int t = lane / 3, part = lane - 3 * t;
      const size_t row = (size_t)(row0 + t);
      const T* from = part == 0   ? (const T*)p.q + row * p.q_row
                      : part == 1 ? (const T*)p.k + row * p.k_row
                                  : (const T*)p.v + row * p.v_row;
      const uint32_t bytes = (part == 0 ? p.Hq : p.Hk) * head_bytes;
      const uint32_t to = part == 0 ? 0 : part == 1 ? p.Hq * head_bytes : turned * head_bytes;
      if (bytes) tc::bulk_load(bulk_s + st * stage_bytes + t * row_bytes + to, from, bytes, &ring.full[st]);
    }
  };

  if (warp == kLoader) {
    if (lane < stages) {
      tc::mbar_init(&ring.full[lane], 2);
      tc::mbar_init(&ring.done[lane], kWarps);
      tc::mbar_init(&ring.freed[lane], 1);
    }
    tc::fence_barrier_init();
    __syncwarp();
    for (int i = 0; i < min(stages, n); ++i) load(i);  // nobody waits for one before the barrier below
  } else {
    for (int f = tid; f < half; f += kThreads) turns[f] = in_turns(p.freq[f]);
    for (int d = tid; d < 2 * p.D; d += kThreads) {
      const float* w = d < p.D ? p.q_weight : p.k_weight;
      weight_s[d] = w ? w[d < p.D ? d : d - p.D] : 1.f;
    }
  }
  __syncthreads();

  if (warp == kLoader) {
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int st = i % stages;
      ok = __all_sync(0xffffffffu, wait_for(&ring.done[st], i / stages));
      if (!ok) break;
      const int row0 = first_row(i), count = min(tokens, p.rows - row0);
      if (lane < 3 * count) {
        const int t = lane / 3, part = lane - 3 * t;
        const int2 at = ring.at[st][t];
        const uint8_t* from = bulk_s + st * stage_bytes + t * row_bytes;
        const size_t slot = (size_t)at.y * p.Hk * p.D;
        if (part == 0 && p.Hq && at.x >= 0)
          tc::bulk_store((T*)p.q_out + (size_t)(row0 + t) * p.q_out_row, from, p.Hq * head_bytes);
        if (!PACKED && part == 1 && p.Hk && at.x >= 0 && at.y >= 0)
          tc::bulk_store((T*)p.k_cache + slot, from + p.Hq * head_bytes, p.Hk * head_bytes);
        if (!PACKED && part == 2 && p.Hk && at.x >= 0 && at.y >= 0)
          tc::bulk_store((T*)p.v_cache + slot, from + turned * head_bytes, p.Hk * head_bytes);
      }
      tc::bulk_commit();
      if (i > 0 && i - 1 + stages < n) {  // the stage before this one has been read: its next tokens
        tc::bulk_wait_read<1>();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ring.freed[(i - 1) % stages]);
        load(i - 1 + stages);
      }
    }
    if (!ok) {  // the loads in flight land before the block's memory goes
      if (lane == 0) set_status(p.status, SPEC_STATUS_TIMEOUT);
      for (int st = 0; st < stages; ++st) {
        // the last load of a stage: the phase its barrier is in, or the one before
        wait_for(&ring.full[st], 0);
        wait_for(&ring.full[st], 1);
      }
    }
    tc::bulk_wait();
  } else if (warp == kCosines) {
    auto read = [&](int i) {  // position and slot of token `lane` of stage i
      const int row = first_row(i) + lane;
      if (i >= n || lane >= tokens || row >= p.rows) return make_int2(0, -1);
      return make_int2(p.position[row], p.slot ? p.slot[row] : -1);
    };
    auto place = [&](int d) { return ((d % VEC >> 2) * head_lanes + d / VEC) * 4 + (d & 3); };
    for (int d = p.rot + lane; d < p.D; d += 32)  // what does not turn: the same for all
      for (int x = 0; x < 2 * stages * tokens; ++x) {
        float* to = factor_s + (size_t)x * 2 * p.D + place(d);
        to[0] = weight_s[(x & 1) * p.D + d];
        to[p.D] = 0.f;
      }
    int2 next = read(0);
    uint32_t bad = 0;
    for (int i = 0; i < n; ++i) {
      const int st = i % stages;
      int2 at = next;
      next = read(i + 1);
      if (at.x >= (1 << 24)) bad |= SPEC_STATUS_BAD_POSITION;
      if (at.y >= p.n_slots) bad |= SPEC_STATUS_BAD_PAGE, at.y = -1;
      const float x = (float)min(max(at.x, 0), (1 << 24) - 1);
      if (i >= stages && !__all_sync(0xffffffffu, wait_for(&ring.freed[st], i / stages - 1))) break;
      if (lane < tokens) {
        ring.at[st][lane] = at;
        if (PACKED && at.y >= 0) {
          const int page = at.y / p.page_size, tok = at.y - page * p.page_size, groups_of = p.D / q4::kGroup;
          ring.packed_at[st][lane] = make_longlong2(q4::data_at(page, 0, tok, p.Hk, groups_of, p.page_size),
                                                    q4::scale_at(page, 0, tok, p.Hk, groups_of, p.page_size));
        }
      }
      for (int j0 = 0, t = 0, f = lane; j0 < tokens * half; j0 += 32, f += 32) {  // pair f of token t
        while (f >= half) f -= half, ++t;
        const float pos = __shfl_sync(0xffffffffu, x, t & (kWarps - 1));
        if (t >= tokens) continue;
        float* of = factor_s + (size_t)(st * tokens + t) * 4 * p.D;
        const float2 v = cos_sin(pos, turns[f], p.scale);
        const int d0 = INTER ? 2 * f : f, d1 = INTER ? d0 + 1 : f + half, p0 = place(d0), p1 = place(d1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float w0 = weight_s[k * p.D + d0], w1 = weight_s[k * p.D + d1];
          float* to = of + k * 2 * p.D;
          to[p0] = v.x * w0;
          to[p1] = v.x * w1;
          to[p.D + p0] = -v.y * w1;
          to[p.D + p1] = v.y * w0;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ring.full[st]);
    }
    if (bad) set_status(p.status, bad);
  } else {
    const int each = kWarps / tokens, t = warp / each, in_t = warp - t * each;  // a token's warps
    const int at_once = 32 / lanes, sub = lane / lanes, l = lane % lanes, first = l * VEC;
    const bool live = first < p.D;
    const float inv_d = 1.f / (float)p.D;
    const int other = (lane + (first < half ? half : -half) / VEC) & 31;  // half layout: where the other halves lie
    const uint32_t hop = each * at_once * head_bytes, head_codes = p.D / q4::kGroup * p.page_size;
    const int group = first / q4::kGroup;  // the lane's, and its bytes from a head's first
    const int64_t in_group = (int64_t)group * 16 * p.page_size + first % q4::kGroup / 2;
    uint32_t phase = 0;
    for (int i = 0, st = 0; i < n; ++i, st = st + 1 < stages ? st + 1 : (phase ^= 1u, 0)) {
      if (!__all_sync(0xffffffffu, wait_for(&ring.full[st], phase))) break;
      const int2 at = ring.at[st][t];
      if (first_row(i) + t < p.rows && at.x >= 0) {
        Lane<T> lf;
        lf.turning = first < p.rot;
        auto factors_of = [&](int kind) {
          const float4* f4 = reinterpret_cast<const float4*>(factor_s + (size_t)((st * tokens + t) * 2 + kind) * 2 * p.D) + (live ? l : 0);
#pragma unroll
          for (int j = 0; j < VEC / 4; ++j) {
            const float4 m = f4[j * head_lanes], o = f4[p.D / 4 + j * head_lanes];
            lf.mine[2 * j] = tc::pair(m.x, m.y), lf.mine[2 * j + 1] = tc::pair(m.z, m.w);
            lf.others[2 * j] = tc::pair(o.x, o.y), lf.others[2 * j + 1] = tc::pair(o.z, o.w);
          }
        };
        uint8_t* token = bulk_s + st * stage_bytes + t * row_bytes + first * sizeof(T);
        auto elements = [](const uint8_t* from, bool on, auto again) {  // from shared memory
          uint4 v = make_uint4(0, 0, 0, 0);
          if (on) v = again.value ? tc::lds128(from) : *reinterpret_cast<const uint4*>(from);
          return v;
        };
        auto heads = [&](int kind, int begin, int count, const float* weight) {  // in place
          factors_of(kind);
          uint8_t* from = token + (uint32_t)(begin + in_t * at_once + sub) * head_bytes;
          for (int h0 = in_t * at_once; h0 < count; h0 += each * at_once, from += hop) {
            const bool on = h0 + sub < count && live;
            uint64_t y[N];
            norm_turn<T, INTER>([&](auto again) { return elements(from, on, again); }, y, lf, weight != nullptr, lanes, other, inv_d, p.eps);
            if (on) *reinterpret_cast<uint4*>(from) = packed_up(y, T());
          }
        };
        heads(0, 0, p.Hq, p.q_weight);
        if (!PACKED) {
          heads(1, p.Hq, p.Hk, p.k_weight);
        } else {  // a head of keys and its values together
          factors_of(1);
          const longlong2 to = at.y >= 0 ? ring.packed_at[st][t] : make_longlong2(0, 0);
          const uint8_t* from = token + (uint32_t)(p.Hq + in_t * at_once + sub) * head_bytes;
          const int64_t data_at = to.x + in_group, scale_at = to.y + group;
          for (int h0 = in_t * at_once; h0 < p.Hk; h0 += each * at_once, from += hop) {
            const bool on = h0 + sub < p.Hk && live;
            const uint4 v = elements(from + p.Hk * head_bytes, on, std::false_type{});
            uint64_t y[N];
            float both[2][VEC];
            norm_turn<T, INTER>([&](auto again) { return elements(from, on, again); }, y, lf, p.k_weight != nullptr, lanes, other, inv_d, p.eps);
            spread(y, both[0]);
            unpack(v, y, T());
            spread(y, both[1]);
            uint32_t w[2], code[2];
            code_groups<VEC, 2>(both, w, code);
#pragma unroll
            for (int m = 0; m < 2 && VEC < 8; ++m) {
              w[m] <<= 4 * (first & 7);
              w[m] |= __shfl_xor_sync(0xffffffffu, w[m], 1);
            }
            if (!on || at.y < 0) continue;
            const uint32_t head = (h0 + sub) * head_codes;  // (a page's bytes are below 2^31)
            const int64_t d_at = data_at + head * (size_t)16, s_at = scale_at + head;
            if (first % 8 == 0) {
              *reinterpret_cast<uint32_t*>((uint8_t*)p.k_cache + d_at) = w[0];
              *reinterpret_cast<uint32_t*>((uint8_t*)p.v_cache + d_at) = w[1];
            }
            if (first % q4::kGroup == 0) p.k_scale[s_at] = (uint8_t)code[0], p.v_scale[s_at] = (uint8_t)code[1];
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ring.done[st]);
    }
  }
}

// Rows of 4 KB or more, or batches of 4 MB (measured at the top).
constexpr size_t kBulkRow = 4096, kBulkBytes = 4000000;

// Shared memory of a block with `stages` stages.
template <typename T, bool PACKED>
size_t bulk_bytes(const spec_norm_rope_args& a, int tokens, int stages) {
  const size_t half = a.rot / 2, row = (size_t)(a.Hq + 2 * a.Hk) * a.D * sizeof(T);
  return stages * tokens * row + sizeof(Ring<PACKED>) + (half + 1) / 2 * 16 + (size_t)(2 + stages * tokens * 4) * a.D * sizeof(float);
}
constexpr size_t kBulkMemory = 222 * 1024, kStageBytes = 20 * 1024;
template <typename T, bool PACKED>
bool launch_bulk(const spec_norm_rope_args& a, int lanes, cudaStream_t stream, cudaError_t* err) {
  const size_t row = (size_t)(a.Hq + 2 * a.Hk) * a.D * sizeof(T);
  auto dense = [&](int n, int64_t head) { return n < 2 || head == a.D; };  // heads side by side
  if (!dense(a.Hq, a.q_head) || !dense(a.Hq, a.q_out_head) || !dense(a.Hk, a.k_head) || !dense(a.Hk, a.v_head)) return false;
  if (row < kBulkRow && a.rows * row < kBulkBytes) return false;
  // Stages of up to 20 KB, one token each until every block has one; three stages at least, with fewer tokens or
  // blocks an SM where they do not fit.
  int tokens = 0, stages = 0, blocks = bulk_blocks(PACKED);
  for (;; --blocks) {
    if (blocks == 0) return false;
    tokens = std::max(1, std::min({kWarps, a.rows / (152 * blocks), (int)(kStageBytes / row)}));
    while (tokens & (tokens - 1)) tokens &= tokens - 1;
    auto fit = [&] {
      for (stages = kMaxStages; stages > 0 && bulk_bytes<T, PACKED>(a, tokens, stages) > kBulkMemory / blocks;) --stages;
      return stages >= 3;
    };
    while (!fit() && tokens > 1) tokens /= 2;
    if (stages >= 3) break;
  }
  auto kernel = a.layout == SPEC_ROPE_INTERLEAVED ? norm_rope_bulk_kernel<T, true, PACKED> : norm_rope_bulk_kernel<T, false, PACKED>;
  *err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBulkMemory);
  if (*err != cudaSuccess) return true;
  const int groups = (a.rows + tokens - 1) / tokens;
  kernel<<<std::min(groups, blocks * 152), kBulkThreads, bulk_bytes<T, PACKED>(a, tokens, stages), stream>>>(a, tokens, stages, lanes);
  *err = cudaGetLastError();
  return true;
}

// Lanes of a head, heads of a warp at a time and what a launch of warps of single heads takes.
struct Shape {
  int lanes, parts;
  unsigned blocks;
};
Shape shape_of(const spec_norm_rope_args& a, int vec, bool packed, bool chunks = false) {
  Shape s;
  for (s.lanes = chunks ? 32 : 1; s.lanes * vec < a.D && s.lanes < 32;) s.lanes *= 2;
  if (packed) s.lanes = std::max(s.lanes, q4::kGroup / vec);
  const int at_once = 32 / s.lanes;
  const int steps = (a.Hq + at_once - 1) / at_once + 2 * ((a.Hk + at_once - 1) / at_once);
  // warps for eight blocks an SM, as far as a warp keeps four steps
  const int64_t warps = 152 * 8 * kWarps;
  s.parts = (int)std::max<int64_t>(1, std::min<int64_t>((steps + kSteps - 1) / kSteps, warps / std::max(a.rows, 1)));
  s.blocks = (unsigned)std::min<int64_t>(((int64_t)a.rows * s.parts + kWarps - 1) / kWarps, 152 * 8);
  return s;
}

template <typename T, int VEC, int CH, bool PACKED>
cudaError_t launch_general(const spec_norm_rope_args& a, cudaStream_t stream) {
  const Shape s = shape_of(a, VEC, PACKED, CH > 1);
  const size_t smem = (size_t)(a.rot / 2) * (1 + kWarps) * sizeof(float2) + (size_t)kWarps * 32 * VEC * CH * sizeof(float);
  norm_rope_general_kernel<T, VEC, CH, PACKED><<<s.blocks, kThreads, smem, stream>>>(a, s.parts, s.lanes);
  return cudaGetLastError();
}

template <typename T, bool PACKED>
cudaError_t launch(const spec_norm_rope_args& a, bool wide, cudaStream_t stream) {
  constexpr int VEC = 16 / (int)sizeof(T);
  if (!wide) return a.D <= 128 ? launch_general<T, 1, 4, PACKED>(a, stream) : launch_general<T, 1, 16, PACKED>(a, stream);
  if (a.D > 64 * VEC) return launch_general<T, VEC, VEC == 8 ? 2 : 4, PACKED>(a, stream);
  if (a.D > 32 * VEC) return launch_general<T, VEC, 2, PACKED>(a, stream);
  const bool inter = a.layout == SPEC_ROPE_INTERLEAVED;
  if ((inter ? a.rot : a.rot / 2) % VEC != 0) return launch_general<T, VEC, 1, PACKED>(a, stream);
  const Shape s = shape_of(a, VEC, PACKED);
  cudaError_t err;
  if (launch_bulk<T, PACKED>(a, s.lanes, stream, &err)) return err;
  const size_t smem = (size_t)(a.rot / 2) * (1 + kWarps) * sizeof(float2);
  if (inter) norm_rope_kernel<T, true, PACKED><<<s.blocks, kThreads, smem, stream>>>(a, s.parts, s.lanes);
  else norm_rope_kernel<T, false, PACKED><<<s.blocks, kThreads, smem, stream>>>(a, s.parts, s.lanes);
  return cudaGetLastError();
}

// ------------------------------------------------------------- read-back ---
// A thread turns 4 bytes into 8 elements, 4 threads side by side a group; it keeps its word of a row
// and steps over rows.  `shift`: the page size's logarithm, or -1.
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(spec_cache_read_packed_args p, int at_once, int shift) {
  const int groups = p.D / q4::kGroup, words = p.Hk * groups * 4, wide = min(words, kThreads);
  const int which = blockIdx.y, r0 = threadIdx.x / wide;
  T* out = (T*)(which ? p.v : p.k);
  if (!out || r0 >= at_once) return;
  const uint8_t* data = (const uint8_t*)(which ? p.v_cache : p.k_cache);
  const uint8_t* scales = which ? p.v_scale : p.k_scale;
  for (int w = threadIdx.x - r0 * wide; w < words; w += wide) {
    const int h = w / (4 * groups), g = w / 4 - h * groups;
    const uint8_t* word = data + q4::data_at(0, h, 0, p.Hk, groups, p.page_size) + (size_t)g * 16 * p.page_size + (w & 3) * 4;
    const uint8_t* code = scales + q4::scale_at(0, h, 0, p.Hk, groups, p.page_size) + g;
    const uint32_t page_bytes = (uint32_t)q4::data_at(1, 0, 0, p.Hk, groups, p.page_size), page_codes = page_bytes / 16;  // (below 2^31)
    const int64_t step = (int64_t)gridDim.x * at_once;
    uint4* to = reinterpret_cast<uint4*>(out + ((blockIdx.x * (int64_t)at_once + r0) * words + w) * 8);
#pragma unroll 4
    for (int64_t row = (int64_t)blockIdx.x * at_once + r0; row < p.rows; row += step, to += step * words * (int)sizeof(T) / 2) {
      const int slot = p.slot[row];
      uint32_t v = 0x88888888u, b = 0;  // zeros
      if (slot >= p.n_slots) set_status(p.status, SPEC_STATUS_BAD_PAGE);
      if (slot >= 0 && slot < p.n_slots) {
        const uint32_t page = shift >= 0 ? (uint32_t)slot >> shift : (uint32_t)slot / (uint32_t)p.page_size;
        const uint32_t tok = slot - page * p.page_size;
        v = *reinterpret_cast<const uint32_t*>(word + (size_t)page * page_bytes + tok * 16);
        b = code[(size_t)page * page_codes + tok * groups];
      }
      const q4::Scale s = q4::scale_pair(b * 0x10001u);
      const uint32_t p0 = q4::element_pair<0>(v, s), p1 = q4::element_pair<1>(v, s), p2 = q4::element_pair<2>(v, s), p3 = q4::element_pair<3>(v, s);
      const uint32_t x[4] = {__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410), __byte_perm(p0, p1, 0x7632), __byte_perm(p2, p3, 0x7632)};
      if (sizeof(T) == 2) {
        *to = make_uint4(x[0], x[1], x[2], x[3]);
      } else {
        to[0] = make_uint4(x[0] << 16, x[0] & 0xffff0000u, x[1] << 16, x[1] & 0xffff0000u);
        to[1] = make_uint4(x[2] << 16, x[2] & 0xffff0000u, x[3] << 16, x[3] & 0xffff0000u);
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const spec_norm_rope_args& a, cudaStream_t stream) {
  if (a.rows == 0 || a.Hq + a.Hk == 0) return cudaSuccess;
  const int vec = a.dtype == SPEC_F32 ? 4 : 8;
  auto on = [&](const void* p) { return ((uintptr_t)p % 16) == 0; };
  bool wide = a.D % vec == 0 && a.q_row % vec == 0 && a.q_head % vec == 0 && a.q_out_row % vec == 0 && a.q_out_head % vec == 0 &&
              a.k_row % vec == 0 && a.k_head % vec == 0 && a.v_row % vec == 0 && a.v_head % vec == 0 && on(a.q) && on(a.k) &&
              on(a.v) && on(a.q_out) && on(a.k_cache) && on(a.v_cache);
  const bool packed = a.cache == SPEC_CACHE_PACKED && a.Hk > 0;
  if (a.dtype == SPEC_F32) return packed ? launch<float, true>(a, wide, stream) : launch<float, false>(a, wide, stream);
  return packed ? launch<__nv_bfloat16, true>(a, wide, stream) : launch<__nv_bfloat16, false>(a, wide, stream);
}

cudaError_t launch_cache_read(const spec_cache_read_packed_args& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int words = a.Hk * (a.D / 8), at_once = std::max(1, kThreads / words);
  int shift = 0;  // of a page size that is a power of two, or -1
  while ((1 << shift) < a.page_size && shift < 30) ++shift;
  if (1 << shift != a.page_size) shift = -1;
  // Two blocks an SM and kind, and four: 128k words 4.2 and 4.7 us, 328k (2560 rows of 8 heads of 128) 6.6 and 6.5, 640k 10.3 and
  // 9.7, 1.02M 14.8 and 13.4, 1.9M (30011 rows of 8 heads of 64) 25.9 and 23.6; over rows that lie in L2 328k 8.2 and 8.5 and 1.9M
  // 23.3 and 21.3.  (Three: 4.2, 5.6, 8.3, 11.5 and 21.0.)
  const int blocks = 152 * ((int64_t)a.rows * words < (1 << 20) ? 2 : 4);
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)a.rows + at_once - 1) / at_once, blocks), 2);
  if (a.dtype == SPEC_F32) cache_read_kernel<float><<<grid, kThreads, 0, stream>>>(a, at_once, shift);
  else cache_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a, at_once, shift);
  return cudaGetLastError();
}

}  // namespace spec
