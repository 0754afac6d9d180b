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
// Layout, small batches and strided heads (rope_kernel): a unit is two 16-byte vectors
// of a head: the two halves of its pairs in the half layout, two vectors next to each
// other otherwise; either way unit u takes the frequencies [u VEC, (u + 1) VEC).  A thread
// keeps one unit of one token and steps over the heads, queries, keys and values in turn,
// and then over a few more tokens, the next step's loads ahead of this step's products:
// its cosines and sines are read from shared memory once a token (one float4 column a
// unit, free of bank conflicts) and stay in registers, and a step is two loads, the
// products and two stores.  A thread's first loads go out before the cosines are computed.
//
// Long batches (rope_bulk_kernel): bulk copies through a ring in shared memory, described
// there.  What bounds both is memory, every element read and written once; a thread's
// registers hold too few bytes in flight for it: 2560 rows of 64 + 2 * 8 heads of 128 in
// bf16 took 26.0 us (4.0 TB/s) by the first kernel, 19.7 (5.3 TB/s) by the second, 40001
// rows of 32 + 2 * 4 heads 164 us and 122 (6.7 TB/s).
#include "rope.cuh"
#include "tc.cuh"

#include <algorithm>
#include <climits>

namespace spec {

namespace {

constexpr int kThreads = 256;     // of the element-wise kernel
constexpr int kMaxThreads = 320;  // of rope_kernel: two blocks an SM at 96 registers (three spill: 98 us for 26)
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

// A frequency (radians) in turns, hi + lo.
__device__ __forceinline__ float2 in_turns(double freq) {
  const double turns = freq * 0.15915494309189533577;  // 1 / (2 pi)
  const float hi = (float)turns;
  return make_float2(hi, (float)(turns - (double)hi));
}
// cos and sin, times the scale, of position x times the frequency.
__device__ __forceinline__ float2 cos_sin(float x, float2 turns, float scale) {
  const float m = x * turns.x, e = fmaf(x, turns.x, -m);
  const float frac = (m - rintf(m)) + fmaf(x, turns.y, e);
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * scale, s * scale);
}
__device__ __forceinline__ float2 cos_sin(float x, double freq, float scale) {
  return cos_sin(x, in_turns(freq), scale);
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

// ------------------------------------------------------------ long batches --
// Rows whose heads lie side by side, by bulk copies through a ring of stages in
// shared memory: a stage is a few tokens, turned in place.  One warp issues the loads
// and, when a stage is turned, its stores (values are not touched in between); one
// computes the cosines of the stages ahead; the others turn queries and keys.  Every wait
// is bounded: on a timeout the block sets SPEC_STATUS_TIMEOUT, waits for its copies in
// flight and returns.
constexpr int kWorkers = 256, kBulkThreads = kWorkers + 64;
constexpr int kMaxStages = 4, kMaxTokens = 16;
constexpr uint64_t kWaitNs = 2000000000ull;

struct Ring {
  uint64_t full[kMaxStages], done[kMaxStages], freed[kMaxStages];
  int2 at[kMaxStages][kMaxTokens];  // position (-1: left out) and slot (-1: none) of a stage's tokens
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t phase) {
  return tc::mbar_try_wait(bar, phase & 1u) || tc::mbar_wait(bar, phase & 1u, kWaitNs);
}

// Stage i of the block holds tokens (blockIdx.x + i * gridDim.x) * tokens and on; `tokens`
// divides the workers.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kBulkThreads, 3) rope_bulk_kernel(spec_rope_cache_args p, int tokens, int stages) {
  constexpr int VEC = 16 / (int)sizeof(T);
  constexpr int kPairs = INTER ? VEC / 2 : VEC;  // of a unit: a vector, or a vector of each half
  constexpr int kCol = kPairs / 2;               // float4s of its cosines and sines
  extern __shared__ __align__(128) uint8_t bulk_s[];
  const int half = p.rot >> 1, units = half / kPairs, turned = p.Hq + p.Hk;
  const uint32_t head_bytes = p.D * (uint32_t)sizeof(T), row_bytes = (turned + p.Hk) * head_bytes;
  const uint32_t stage_bytes = tokens * row_bytes;
  Ring& ring = *reinterpret_cast<Ring*>(bulk_s + stages * stage_bytes);
  float2* freq_s = reinterpret_cast<float2*>(&ring + 1);
  float4* cs_s = reinterpret_cast<float4*>(freq_s + ((half + 1) & ~1));  // [stage][token][kCol][units]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (p.rows + tokens - 1) / tokens;
  const int n = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  auto first_row = [&](int i) { return ((int)blockIdx.x + i * (int)gridDim.x) * tokens; };
  constexpr int kLoader = kWorkers / 32, kCosines = kLoader + 1;

  // the copies of a token: queries, keys, values
  auto load = [&](int i) {
    const int row0 = first_row(i), count = min(tokens, p.rows - row0), st = i % stages;
    if (lane == 0) tc::mbar_expect_tx(&ring.full[st], count * row_bytes);
    __syncwarp();
    for (int c = lane; c < 3 * count; c += 32) {
      const int t = c / 3, part = c - 3 * t;
      const size_t row = (size_t)(row0 + t);
      const T* from = part == 0 ? (const T*)p.q + row * p.q_row
                      : part == 1 ? (const T*)p.k + row * p.k_row : (const T*)p.v + row * p.v_row;
      const uint32_t bytes = (part == 0 ? p.Hq : p.Hk) * head_bytes;
      const uint32_t to = part == 0 ? 0 : part == 1 ? p.Hq * head_bytes : turned * head_bytes;
      if (bytes) tc::bulk_load(bulk_s + st * stage_bytes + t * row_bytes + to, from, bytes, &ring.full[st]);
    }
  };

  if (warp == kLoader) {
    if (lane < stages) {
      tc::mbar_init(&ring.full[lane], 2);
      tc::mbar_init(&ring.done[lane], kWorkers / 32);
      tc::mbar_init(&ring.freed[lane], 1);
    }
    tc::fence_barrier_init();
    __syncwarp();
    for (int i = 0; i < min(stages, n); ++i) load(i);  // nobody waits for one before the barrier below
  } else {
    for (int f = tid; f < half; f += kWorkers) freq_s[f] = in_turns(p.freq[f]);
  }
  __syncthreads();

  if (warp == kLoader) {
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int st = i % stages;
      ok = __all_sync(0xffffffffu, wait_for(&ring.done[st], i / stages));
      if (!ok) break;
      const int row0 = first_row(i), count = min(tokens, p.rows - row0);
      for (int c = lane; c < 3 * count; c += 32) {
        const int t = c / 3, part = c - 3 * t;
        const int2 at = ring.at[st][t];
        const uint8_t* from = bulk_s + st * stage_bytes + t * row_bytes;
        const size_t slot = (size_t)at.y * p.Hk * p.D;
        if (part == 0 && p.Hq && at.x >= 0)
          tc::bulk_store((T*)p.q_out + (size_t)(row0 + t) * p.q_out_row, from, p.Hq * head_bytes);
        if (part == 1 && p.Hk && at.x >= 0 && at.y >= 0)
          tc::bulk_store((T*)p.k_cache + slot, from + p.Hq * head_bytes, p.Hk * head_bytes);
        if (part == 2 && p.Hk && at.x >= 0 && at.y >= 0)
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
      if (lane < tokens) ring.at[st][lane] = at;
      for (int t = 0; t < tokens; ++t) {
        const float pos = __shfl_sync(0xffffffffu, x, t);
        float2* cs = reinterpret_cast<float2*>(cs_s + (size_t)(st * tokens + t) * kCol * units);
        for (int f = lane; f < half; f += 32) {
          const int u = f / kPairs, e = f % kPairs;
          cs[((e >> 1) * units + u) * 2 + (e & 1)] = cos_sin(pos, freq_s[f], p.scale);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ring.full[st]);
    }
    if (bad) set_status(p.status, bad);
  } else {
    const int share = kWorkers / tokens, t = tid / share, in_t = tid - t * share;  // a token's threads
    const int at_once = units > 0 ? share / units : 0, h0 = units > 0 ? in_t / units : 0, u = in_t - h0 * units;
    for (int i = 0; i < n; ++i) {
      const int st = i % stages;
      if (!__all_sync(0xffffffffu, wait_for(&ring.full[st], i / stages))) break;
      if (h0 < at_once && first_row(i) + t < p.rows) {
        const float4* col = cs_s + (size_t)(st * tokens + t) * kCol * units + u;
        float4 cs[kCol];
#pragma unroll
        for (int j = 0; j < kCol; ++j) cs[j] = col[j * units];
        uint8_t* at = bulk_s + st * stage_bytes + t * row_bytes + u * 16;
#pragma unroll 3
        for (int h = h0; h < turned; h += at_once) {
          uint4* a = reinterpret_cast<uint4*>(at + h * head_bytes);
          Vec<T, VEC> x, y;
          x.raw = a[0];
          if (INTER) {
#pragma unroll
            for (int j = 0; j < kCol; ++j) {
              turn(x.e[4 * j], x.e[4 * j + 1], make_float2(cs[j].x, cs[j].y));
              turn(x.e[4 * j + 2], x.e[4 * j + 3], make_float2(cs[j].z, cs[j].w));
            }
          } else {
            y.raw = a[units];
#pragma unroll
            for (int j = 0; j < kCol; ++j) {
              turn(x.e[2 * j], y.e[2 * j], make_float2(cs[j].x, cs[j].y));
              turn(x.e[2 * j + 1], y.e[2 * j + 1], make_float2(cs[j].z, cs[j].w));
            }
            a[units] = y.raw;
          }
          a[0] = x.raw;
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ring.done[st]);
    }
  }
}

// Shared memory of a block with `stages` stages.
template <typename T>
size_t bulk_bytes(const spec_rope_cache_args& a, int tokens, int stages) {
  const size_t half = a.rot / 2, row = (size_t)(a.Hq + 2 * a.Hk) * a.D * sizeof(T);
  return stages * tokens * row + sizeof(Ring) + (half + 1) / 2 * 16 + stages * tokens * half * sizeof(float2);
}
// Three blocks an SM where four stages fit (40001 rows of 10 KB: 122 us, 125 with two
// blocks and stages of 20 KB, 152 with one block), else two (9000 rows of 20 KB: 57.5 us,
// 64 with three blocks of three stages).
constexpr size_t kBulkMemory = 222 * 1024, kStageBytes = 17 * 1024;
// From 12 MB on: below, the first round of stages is most of the work (3.7 MB: 6.9 us
// against 5.5 of the kernel above, 12.5 MB that lie in L2 6.2 both).  Inputs that do not lie
// in L2: 12.3 MB in 750 rows, most blocks with one or two stages, 6.9 us against 8.3; 12.5 MB
// in 610 rows 7.2 against 8.4; 26.6 MB 11.5 against 16.0.  kBulkRows is four tokens an SM.
constexpr size_t kBulkBytes = 12000000;
constexpr int kBulkRows = 608;
bool bulk_ok(const spec_rope_cache_args& a, size_t row_bytes) {
  auto dense = [&](int n, int64_t head) { return n < 2 || head == a.D; };  // heads side by side
  return a.rows >= kBulkRows && a.rows * row_bytes >= kBulkBytes && dense(a.Hq, a.q_head) &&
         dense(a.Hq, a.q_out_head) && dense(a.Hk, a.k_head) && dense(a.Hk, a.v_head);
}

template <typename T>
cudaError_t launch_bulk(const spec_rope_cache_args& a, int tokens, int stages, int blocks, cudaStream_t stream) {
  const int groups = (a.rows + tokens - 1) / tokens, grid = std::min(groups, blocks * 152);
  const size_t smem = bulk_bytes<T>(a, tokens, stages);
  auto kernel = a.layout == SPEC_ROPE_INTERLEAVED ? rope_bulk_kernel<T, true> : rope_bulk_kernel<T, false>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBulkMemory / 2);
  if (err != cudaSuccess) return err;
  kernel<<<grid, kBulkThreads, smem, stream>>>(a, tokens, stages);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_wide(const spec_rope_cache_args& a, cudaStream_t stream) {
  constexpr int VEC = 16 / (int)sizeof(T);
  const bool inter = a.layout == SPEC_ROPE_INTERLEAVED;
  const int half = a.rot / 2, heads = a.Hq + 2 * a.Hk;
  if (bulk_ok(a, (size_t)heads * a.D * sizeof(T))) {
    const size_t row = (size_t)heads * a.D * sizeof(T);
    const int units = half / (inter ? VEC / 2 : VEC);  // no more of a token than its threads: 128 at most of 256
    int tokens = std::min({kMaxTokens, kWorkers / std::max(1, units), a.rows / kBulkRows,
                           std::max(1, (int)(kStageBytes / row))});
    // a power of two shares the threads out evenly (40000 rows of 1.5 KB: 8 tokens 36 us, 11 43)
    while (tokens & (tokens - 1)) tokens &= tokens - 1;
    for (int blocks = 3; blocks >= 2; --blocks)
      for (int stages = kMaxStages; stages >= (blocks == 3 ? kMaxStages : 3); --stages)
        if (bulk_bytes<T>(a, tokens, stages) <= kBulkMemory / blocks)
          return launch_bulk<T>(a, tokens, stages, blocks, stream);
  }
  const int copied = (a.D + 2 * VEC - 1) / (2 * VEC);
  const int turned = inter ? copied : half / VEC + (a.D - a.rot + 2 * VEC - 1) / (2 * VEC);
  const int units = std::max(copied, turned);
  // Heads at once: a token's heads over a group of threads, kUnroll a thread.
  const int most = std::max(1, kMaxThreads / units);
  const int at_once = std::min(most, (heads + kUnroll - 1) / kUnroll);
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
