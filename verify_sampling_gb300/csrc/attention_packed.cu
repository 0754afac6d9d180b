// Attention over a cache in 4 bits for few query rows a key head (decoding, short drafts).
//
// Mathematics: the pieces of attention_tc.cu (a reference m that follows the running maximum
// in steps of 8, l = sum 2^(z - m), O = sum 2^(z - m) v), over elements made in bf16 (packed.cuh).
//
// Few rows mean that the bytes of the cache bound it, 17 KB a tile of 128 keys, 390 ns of an
// SM's share of memory: the tensor cores have to be busy for little more than the rows that are
// there, and what turns 32768 nibbles into operands is most of the work.  So keys lie along
// the products' M: S^T = K Q^T and O^T = V^T P^T by mma.m16n8k16, 8 rows a product, whose A
// fragments are made in registers and never stored: ldmatrix on the packed bytes gives a thread 8
// dimensions of its key (K), or, transposed, 4 dimensions of two keys side by side (V), and the
// order of dimensions and of rows within a product is free as long as both operands agree.
// P^T is S^T's accumulator, rounded to bf16 and transposed by movmatrix.  (tcgen05 takes its
// operands from shared memory or TMEM: the nibbles would go there and back, at M = 128 with
// 128 rows for 8.  The wide kernel does that where rows are many.)
//
// Instruction issue bounds it before memory does: 256 requests of one row over 4096 keys each, 8
// key heads of 128 (1.2 GB), take 250 us (4.8 TB/s, 71% of the copy rate), about 620 instructions
// a warp for 32 keys.  Shifts and masks run at half an instruction a clock, so K's nibbles become
// whole numbers n - 8 in fp16 (one shift a word where bf16 takes three), and a group's scale
// goes on its part of the score, in fp32.  The queries in fp16 are exact: a row is taken times a
// power of two that brings its largest element to 2^13, and what falls below 2^-24 then is 2^-37
// of that.  Values keep bf16: fp16 has not the scales' range.
//
// Block: a producer warp walks the block's items (attention_plan.cuh) and loads query rows,
// pages and scales by bulk copies into a ring of tiles; four warps take 32 keys of each tile, with
// a maximum, sums and results of their own, and join at an item's end.  Three blocks an SM hide
// one's item changes behind the others' tiles.
//
// Every wait is bounded: on a timeout the block sets SPEC_STATUS_TIMEOUT, waits for its copies
// in flight and returns.
#include "attention_packed.cuh"

#include <cfloat>
#include <climits>

#include "attention_plan.cuh"

namespace spec {

namespace {

using q4::element_pair;
using q4::number_pair;
using q4::Scale;

constexpr int kWarps = 4, kThreads = 32 * (kWarps + 1);
constexpr int kItemSlots = 2;
constexpr int kNarrowMost = 16;  // query rows of a segment that is the narrow kernel's where both run
constexpr float kSlack = 8.f;  // log2 units the maximum may grow by before O is rescaled

// NB: blocks of 8 query rows of an item.  An item's start and end cost a little over two tiles: with 0, 5, 9 and 14
// quarters of a tile 256 requests of one row take 73, 64.7, 61.7 and 62.9 us (500 keys in the mean), 268.8, 256.6,
// 254.4 and 258.5 us (4096 keys).  Heads of 64 with 4, 6, 9 and 14: 101 requests of up to 4 rows (16 rows an item) 52.2, 50.0, 45.7 and
// 46.5 us, 256 of one row (8) over 500 keys 46.1, 45.3, 46.4 and 47.9; heads of 128 and 100 requests of 2 rows (16) 81, 74.5, 69.0 and 69.3.
template <int NB>
struct NarrowCosts {
  static constexpr int kItemRows = 8 * NB, kLeast = 4;
  static constexpr bool kShared = true, kWide = false;
  __device__ static __forceinline__ int tile(int) { return 4; }
  __device__ static __forceinline__ int start(int) { return 9; }
  __device__ static __forceinline__ int tiles_before(int x, int) { return (x + 3) >> 2; }
};

// Blocks an SM: as many as hold the results of two row blocks of 128 dimensions in registers, or of less.
constexpr int narrow_blocks(int D, int NB) { return D * NB == 256 ? 2 : kNarrowBlocks; }

template <int D, int NB>
struct Sizes {
  static constexpr int kGroups = D / q4::kGroup;
  static constexpr int kData = kTile * D / 2, kScales = kTile * kGroups;  // of a tile's keys (or values)
  static constexpr int kStageBytes = 2 * (kData + kScales);
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kQuery = NB * 8 * D * 2;  // an item's query rows
  static constexpr int kJoin = 2 * NB * 8 * D * 4;
};

struct Bars {
  uint64_t full[8], empty[8], item_full[kItemSlots], item_empty[kItemSlots], meet;
  Item items[kItemSlots];
  Layout lay;
  int64_t warp_sum[kThreads / 32];
  volatile int abort_flag;
};

template <int D, int NB>
struct Smem {
  using S = Sizes<D, NB>;
  static constexpr int kQ = S::kStages * S::kStageBytes;
  static constexpr int kJoin = kQ + kItemSlots * S::kQuery;
  static constexpr int kStat = kJoin + S::kJoin;  // [kWarps][NB * 8] float2
  static constexpr int kBars = kStat + kWarps * NB * 8 * 8;
  static constexpr int kBytes = kBars + (int)sizeof(Bars);
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// fp16x2 with `lo` in the low half
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// fp16 operands: d += a b, and d = a b.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int D, int NB>
__global__ void __launch_bounds__(kThreads, narrow_blocks(D, NB))
    attention_narrow_kernel(const spec_prefix_attention_args a, const q4::Cache packed, const Window w, float* part, float2* stat,
                            int64_t* plan) {
  using S = Sizes<D, NB>;
  using M = Smem<D, NB>;
  using C = NarrowCosts<NB>;
  constexpr int G = S::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + M::kBars);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per_head = a.Hq / a.Hk;
  lay_out<C, kThreads>(a, w, &bars.lay, bars.warp_sum, plan, [&] {
    if (tid == 0) {
      bars.abort_flag = 0;
      for (int i = 0; i < S::kStages; ++i) {
        tc::mbar_init(&bars.full[i], 1);
        tc::mbar_init(&bars.empty[i], kWarps);
      }
      for (int i = 0; i < kItemSlots; ++i) {
        tc::mbar_init(&bars.item_full[i], 1);
        tc::mbar_init(&bars.item_empty[i], kWarps);
      }
      tc::mbar_init(&bars.meet, kWarps);
      tc::fence_barrier_init();
    }
  });
  __syncthreads();
  auto warp_wait = [&](uint64_t* bar, uint32_t phase) {  // all of a warp's lanes go on, or all give up
    bool got = tc::mbar_try_wait(bar, phase & 1u);
    if (!__all_sync(0xffffffffu, got)) {
      got = slow_wait(bar, phase, &bars.abort_flag, a.status);
      got = __all_sync(0xffffffffu, got);
    }
    return got;
  };
  const int Pe = min(a.page_size, kTile);  // keys of a page within a tile

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer --
    Walker<C> walk(a, w, bars.lay);
    Item it;
    uint32_t bad = 0, seq = 0, n_item = 0;
    bool ok = true;
    // A tile's copies, two a lane at most: keys' and values' data (a page's head in one, or a
    // copy a group where pages are longer than a tile) and scales.  What is the same for every
    // tile is worked out here: the producer's instructions are all one scheduler's.
    const int groups_in = a.page_size > kTile ? 1 : G, parts = 2 * (G / groups_in + 1);  // copies of a page
    const uint32_t page_bytes = (uint32_t)(Pe * (16 * G + G)) * 2;                      // of a page within a tile
    struct Copy {
      const uint8_t* from;   // of page 0, head 0
      uint32_t page, head, tok;  // bytes to the next one's
      uint32_t to, bytes;
      int x;  // page of the tile
    };
    auto copy_of = [&](int c) {
      const int x = c / parts, rest = c - x * parts, kv = rest & 1, piece = rest >> 1;
      const bool data = piece < G / groups_in;
      const uint32_t unit = data ? 16 : 1;  // bytes of a group
      Copy r;
      r.from = (data ? (kv ? packed.v : packed.k) : (kv ? packed.v_scale : packed.k_scale)) + (data ? (size_t)piece * 16 * a.page_size : 0);
      r.head = unit * G * a.page_size;
      r.page = r.head * a.Hk;
      r.tok = data ? 16 : G;
      r.to = kv * (S::kData + S::kScales) + (data ? (x * G + piece) * Pe * 16 : S::kData + x * Pe * G);
      r.bytes = unit * Pe * (data ? groups_in : G);
      r.x = x;
      return r;
    };
    const Copy first_copy = copy_of(lane), second_copy = copy_of(lane + 32);
    const int tiles_a_page = max(a.page_size / kTile, 1), pages_a_tile = kTile / Pe;
    for (;; ++n_item) {
      const bool more = walk.next(it);
      if (!more) it.rows = 0;  // the end
      const uint32_t slot = n_item % kItemSlots;
      ok = warp_wait(&bars.item_empty[slot], (n_item / kItemSlots) ^ 1u);
      if (!ok) break;
      if (lane == 0) {
        bars.items[slot] = it;
        if (it.rows > 0) tc::mbar_expect_tx(&bars.item_full[slot], (uint32_t)(it.rows * D * 2));
        else tc::mbar_arrive(&bars.item_full[slot]);
      }
      if (it.rows == 0) break;
      __syncwarp();
      if (lane < it.rows) {
        const int m = it.m0 + lane, j = m / per_head;
        tc::bulk_load(smem + M::kQ + slot * S::kQuery + lane * D * 2,
                      (const __nv_bfloat16*)a.q + (int64_t)(it.row0 + j) * a.q_row + (int64_t)(it.h * per_head + (m - j * per_head)) * a.q_head,
                      D * 2, &bars.item_full[slot]);
      }
      // page ids, 32 at a time, the next 32 on their way
      const int pages = (it.keys + a.page_size - 1) / a.page_size;
      int first = it.lo * pages_a_tile, in_page = 0;  // the tile's first page, and its tile of a longer one
      if (tiles_a_page > 1) {
        first = it.lo / tiles_a_page;
        in_page = it.lo - first * tiles_a_page;
      }
      int base = first;
      auto fetch = [&](int from) { return from + lane < pages ? page_of(a, it.table, from + lane, &bad) : 0; };
      int cur = fetch(base), nxt = fetch(base + 32);
      const uint8_t* head1 = first_copy.from + (size_t)first_copy.head * it.h;
      const uint8_t* head2 = second_copy.from + (size_t)second_copy.head * it.h;
      for (int i = it.lo; i < it.hi; ++i, ++seq) {
        if (first >= base + 32) {
          cur = nxt;
          base += 32;
          nxt = fetch(base + 32);
        }
        const int used = min(pages_a_tile, pages - first);  // pages with keys
        const uint32_t st = seq % S::kStages;
        ok = warp_wait(&bars.empty[st], (seq / S::kStages) ^ 1u);
        if (!ok) break;
        if (lane == 0) tc::mbar_expect_tx(&bars.full[st], used * page_bytes);
        __syncwarp();
        uint8_t* to = smem + st * S::kStageBytes;
        const uint32_t skip = in_page * kTile;
        const int page = __shfl_sync(0xffffffffu, cur, (first - base + first_copy.x) & 31);
        if (lane < used * parts)
          tc::bulk_load(to + first_copy.to, head1 + (size_t)first_copy.page * (uint32_t)page + skip * first_copy.tok, first_copy.bytes, &bars.full[st]);
        if (used * parts > 32) {
          const int page2 = __shfl_sync(0xffffffffu, cur, (first - base + second_copy.x) & 31);
          if (lane + 32 < used * parts)
            tc::bulk_load(to + second_copy.to, head2 + (size_t)second_copy.page * (uint32_t)page2 + skip * second_copy.tok, second_copy.bytes,
                          &bars.full[st]);
        }
        if (tiles_a_page == 1) {
          first += pages_a_tile;
        } else if (++in_page == tiles_a_page) {
          in_page = 0;
          ++first;
        }
      }
      if (!ok) break;
    }
    if (bad) set_status(a.status, bad);
    if (!ok) {  // the copies in flight land before the block's memory goes
      const uint32_t from = seq > (uint32_t)S::kStages ? seq - S::kStages : 0u;
      for (uint32_t s = from; s < seq; ++s) tc::mbar_wait(&bars.full[s % S::kStages], (s / S::kStages) & 1u, kWaitNs);
      for (uint32_t s = n_item > kItemSlots ? n_item - kItemSlots : 0u; s <= n_item; ++s)
        tc::mbar_wait(&bars.item_full[s % kItemSlots], (s / kItemSlots) & 1u, kWaitNs / 100);
    }
  } else {
    // ----------------------------------------------------------- consumers --
    const int g = lane >> 2, t = lane & 3;
    const float sl = a.scale * kLog2e;
    const uint32_t sbase = tc::smem_u32(smem);
    // ldmatrix rows of this lane: blocks of 8 keys 4 warp + 2 b + (lane >> 3 & 1), group (lane >> 4) and then two on
    uint32_t row_at[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int key = (warp * 4 + 2 * b + (lane >> 3 & 1)) * 8, page = key / Pe;
      row_at[b] = (uint32_t)((page * G + (lane >> 4)) * Pe * 16 + (key - page * Pe + (lane & 7)) * 16);
    }
    const uint32_t two_groups = 2 * Pe * 16;
    const bool wide_out = ((uintptr_t)a.out & 7) == 0 && a.out_row % 4 == 0 && a.out_head % 4 == 0;
    float* join = reinterpret_cast<float*>(smem + M::kJoin);
    float2* row_stat = reinterpret_cast<float2*>(smem + M::kStat);
    uint32_t st = 0, st_phase = 0, met = 0;
    bool ok = true;
    auto meet = [&] {  // the four warps (a named barrier's wait would have no limit)
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.meet);
      ok = warp_wait(&bars.meet, met++);
      return ok;
    };
    for (uint32_t n_item = 0;; ++n_item) {
      const uint32_t slot = n_item % kItemSlots;
      ok = warp_wait(&bars.item_full[slot], n_item / kItemSlots);
      if (!ok) break;
      const Item it = bars.items[slot];
      if (it.rows == 0) break;
      // query fragments in fp16: dimensions 32 c + 8 t + (i, i + 4) of row g, times a power of two
      uint32_t q[NB][G][4];
      float row_sl[NB][2];  // scores of rows 2 t, 2 t + 1 to log2 units
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint8_t* qs = smem + M::kQ + slot * S::kQuery + (nb * 8 + g) * D * 2 + t * 16;
        uint4 v[G];
        uint32_t most = 0;  // magnitudes' fp32 bits
#pragma unroll
        for (int c = 0; c < G; ++c) {
          v[c] = tc::lds128(qs + c * 64);
          const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = max(most, max(x[e] << 16 & 0x7fff0000u, x[e] & 0x7fff0000u));
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const uint32_t e = most >> 23, up = e == 255u ? 127u : min(267u - e, 253u);  // exponent fields (a row with infinities: as it is)
        const float f = __uint_as_float(up << 23), back = __uint_as_float((254u - up) << 23);
        auto low = [&](uint32_t x) { return __uint_as_float(x << 16) * f; };
        auto high = [&](uint32_t x) { return __uint_as_float(x & 0xffff0000u) * f; };
#pragma unroll
        for (int c = 0; c < G; ++c) {
          q[nb][c][0] = pack_f16(low(v[c].x), low(v[c].z));
          q[nb][c][1] = pack_f16(high(v[c].x), high(v[c].z));
          q[nb][c][2] = pack_f16(low(v[c].y), low(v[c].w));
          q[nb][c][3] = pack_f16(high(v[c].y), high(v[c].w));
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)  // (not 0, which would make NaN of a masked score)
          row_sl[nb][x] = fmaxf(sl * __shfl_sync(0xffffffffu, back, (2 * t + x) * 4), FLT_MIN);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.item_empty[slot]);
      int limit[NB][2];  // keys of rows 2 t, 2 t + 1 of each block (rows past the item's: any)
      float ref[NB][2], l[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = min(nb * 8 + 2 * t + e, it.rows - 1);
          limit[nb][e] = it.prefix ? it.keys : min(it.keys, it.first_own + (it.m0 + m) / per_head);
          ref[nb][e] = -CUDART_INF_F;
          l[nb][e] = 0.f;
        }
      const int least = it.prefix ? it.keys : min(it.keys, it.first_own + it.m0 / per_head);  // of the first row
      float o[G][2][NB][4];
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][x][nb][e] = 0.f;

      for (int i = it.lo; i < it.hi; ++i) {
        ok = warp_wait(&bars.full[st], st_phase);
        if (!ok) break;
        const uint32_t ks = sbase + st * S::kStageBytes, vs = ks + S::kData + S::kScales;
        const uint8_t* k_code = smem + st * S::kStageBytes + S::kData + (warp * 32 + g) * G;
        const uint8_t* v_code = smem + st * S::kStageBytes + 2 * S::kData + S::kScales + (warp * 32 + 2 * t) * G;
        uint64_t s2[2][NB][2];  // scores of keys g and g + 8 of 16, rows 2 t and 2 t + 1
#pragma unroll
        for (int c = 0; c < G; c += 2) {
          uint32_t r[2][4];  // [pair of blocks][block, block + 1 of group c, then of c + 1]
#pragma unroll
          for (int b = 0; b < 2; ++b) ldmatrix4(r[b], ks + row_at[b] + (c >> 1) * two_groups);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t w0 = r[b][2 * cc], w1 = r[b][2 * cc + 1], h0 = w0 >> 8, h1 = w1 >> 8;
              const float z0 = q4::scale_of(k_code[(16 * b) * G + c + cc]), z1 = q4::scale_of(k_code[(16 * b + 8) * G + c + cc]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                float d[4];
                const uint32_t* qq = q[nb][c + cc];
                mma_f16_first(d, number_pair<0>(w0, h0), number_pair<0>(w1, h1), number_pair<1>(w0, h0), number_pair<1>(w1, h1), qq[0], qq[1]);
                mma_f16(d, number_pair<2>(w0, h0), number_pair<2>(w1, h1), number_pair<3>(w0, h0), number_pair<3>(w1, h1), qq[2], qq[3]);
                const uint64_t lo = tc::pair(d[0], d[1]), hi = tc::pair(d[2], d[3]);
                uint64_t* sp = s2[b][nb];
                sp[0] = c + cc == 0 ? tc::mul2(lo, tc::pair(z0, z0)) : tc::fma2(lo, tc::pair(z0, z0), sp[0]);
                sp[1] = c + cc == 0 ? tc::mul2(hi, tc::pair(z1, z1)) : tc::fma2(hi, tc::pair(z1, z1), sp[1]);
              }
            }
        }
        float s[2][NB][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 v = tc::halves(s2[b][nb][x]);
              s[b][nb][2 * x] = v.x;
              s[b][nb][2 * x + 1] = v.y;
            }
        // keys behind a row's last
        const int key0 = i * kTile + warp * 32 + g;
        if (i * kTile + kTile > least) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * b + 8 * (e >> 1) >= limit[nb][e & 1]) s[b][nb][e] = -CUDART_INF_F;
        }
        bool grown = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = fmaxf(fmaxf(s[0][nb][e], s[0][nb][e + 2]), fmaxf(s[1][nb][e], s[1][nb][e + 2]));
            grown |= top * row_sl[nb][e] > ref[nb][e] + kSlack;
          }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(fmaxf(s[0][nb][e], s[0][nb][e + 2]), fmaxf(s[1][nb][e], s[1][nb][e + 2])) * row_sl[nb][e];
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              // each row by its own scores alone: its bits do not depend on its neighbours
              const float to = top > ref[nb][e] + kSlack ? top : ref[nb][e];
              const float f = to == ref[nb][e] ? 1.f : tc::ex2(ref[nb][e] - to);  // 0 from -inf
              ref[nb][e] = to;
              l[nb][e] *= f;
#pragma unroll
              for (int c = 0; c < G; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  o[c][x][nb][e] *= f;
                  o[c][x][nb][e + 2] *= f;
                }
            }
        }
        uint32_t p[2][NB][2];  // weights of keys 2 t, 2 t + 1 (and + 8) of each 16, row g
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float sub0 = ref[nb][0] == -CUDART_INF_F ? 0.f : ref[nb][0], sub1 = ref[nb][1] == -CUDART_INF_F ? 0.f : ref[nb][1];
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float p0 = tc::ex2(fmaf(s[b][nb][2 * x], row_sl[nb][0], -sub0));
              const float p1 = tc::ex2(fmaf(s[b][nb][2 * x + 1], row_sl[nb][1], -sub1));
              l[nb][0] += p0;
              l[nb][1] += p1;
              // rounded to bf16: 8 bits of a weight are 8 bits of its share of the result
              p[b][nb][x] = transposed(pack_bf16(p0, p1));
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int c = 0; c < G; c += 2) {
            uint32_t r[4];
            ldmatrix4_trans(r, vs + row_at[b] + (c >> 1) * two_groups);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              Scale z[2];  // of keys 2 t and 2 t + 1 of both blocks
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint8_t* at = v_code + (16 * b + 8 * x) * G + c + cc;
                z[x] = q4::scale_two(at[0], at[G]);
              }
              const uint32_t v0 = r[2 * cc], v1 = r[2 * cc + 1];
              const uint32_t f0 = element_pair<0>(v0, z[0]), f1 = element_pair<1>(v0, z[0]), f2 = element_pair<0>(v1, z[1]),
                             f3 = element_pair<1>(v1, z[1]);
              const uint32_t h0 = element_pair<2>(v0, z[0]), h1 = element_pair<3>(v0, z[0]), h2 = element_pair<2>(v1, z[1]),
                             h3 = element_pair<3>(v1, z[1]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma(o[c + cc][0][nb], f0, f1, f2, f3, p[b][nb][0], p[b][nb][1]);
                mma(o[c + cc][1][nb], h0, h1, h2, h3, p[b][nb][0], p[b][nb][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.empty[st]);
        if (++st == S::kStages) {
          st = 0;
          st_phase ^= 1u;
        }
      }
      if (!ok) break;
      // ---- the warps' results: maxima and sums of all, results pairwise
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], x);
          if (g == 0) row_stat[warp * NB * 8 + nb * 8 + 2 * t + e] = make_float2(ref[nb][e], l[nb][e]);
        }
      if (!meet()) break;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 v[kWarps];
          float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll
          for (int x = 0; x < kWarps; ++x) {
            v[x] = row_stat[x * NB * 8 + nb * 8 + 2 * t + e];
            top = fmaxf(top, v[x].x);
          }
          const float sub = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll
          for (int x = 0; x < kWarps; ++x) sum = fmaf(v[x].y, tc::ex2(v[x].x - sub), sum);
          const float f = tc::ex2(ref[nb][e] - sub);  // 0 from -inf
          ref[nb][e] = top;
          l[nb][e] = sum;
#pragma unroll
          for (int c = 0; c < G; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              o[c][x][nb][e] *= f;
              o[c][x][nb][e + 2] *= f;
            }
        }
      auto give = [&](float* to) {
#pragma unroll
        for (int c = 0; c < G; ++c)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              *reinterpret_cast<float4*>(to + (((c * 2 + x) * NB + nb) * 32 + lane) * 4) =
                  make_float4(o[c][x][nb][0], o[c][x][nb][1], o[c][x][nb][2], o[c][x][nb][3]);
      };
      auto take = [&](const float* from) {
#pragma unroll
        for (int c = 0; c < G; ++c)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const float4 v = *reinterpret_cast<const float4*>(from + (((c * 2 + x) * NB + nb) * 32 + lane) * 4);
              o[c][x][nb][0] += v.x, o[c][x][nb][1] += v.y, o[c][x][nb][2] += v.z, o[c][x][nb][3] += v.w;
            }
      };
      float* mine = join + (warp & 1) * NB * 8 * D;
      if (warp >= 2) give(mine);
      if (!meet()) break;
      if (warp < 2) take(mine);
      if (warp == 1) give(mine);
      if (!meet()) break;
      if (warp > 0) continue;
      take(join + NB * 8 * D);
      // row 2 t + e: dimensions 32 c + 4 g .. + 3
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = nb * 8 + 2 * t + e;
          if (m >= it.rows) continue;
          const float sum = l[nb][e];
          const int j = (it.m0 + m) / per_head, row = it.row0 + j, hq = it.h * per_head + (it.m0 + m - j * per_head);
          if (!it.direct) {
            const size_t at = it.slot + m;
#pragma unroll
            for (int c = 0; c < G; ++c)
              *reinterpret_cast<float4*>(part + at * D + 32 * c + 4 * g) =
                  make_float4(o[c][0][nb][e], o[c][0][nb][e + 2], o[c][1][nb][e], o[c][1][nb][e + 2]);
            if (g == 0) stat[at] = make_float2(ref[nb][e], sum);
            continue;
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row without keys: zeros
          __nv_bfloat16* out = (__nv_bfloat16*)a.out + (int64_t)row * a.out_row + (int64_t)hq * a.out_head + 4 * g;
#pragma unroll
          for (int c = 0; c < G; ++c) {
            const uint2 v = make_uint2(pack_bf16(o[c][0][nb][e] * inv, o[c][0][nb][e + 2] * inv),
                                       pack_bf16(o[c][1][nb][e] * inv, o[c][1][nb][e + 2] * inv));
            if (wide_out) {
              *reinterpret_cast<uint2*>(out + 32 * c) = v;
            } else {
              *reinterpret_cast<uint32_t*>(out + 32 * c) = v.x;
              *reinterpret_cast<uint32_t*>(out + 32 * c + 2) = v.y;
            }
          }
          if (a.lse && g == 0) a.lse[(size_t)row * a.Hq + hq] = sum == 0.f ? -CUDART_INF_F : (ref[nb][e] + log2f(sum)) * kLn2;
        }
    }
  }
  tc::grid_dep_launch();
}

template <int D, int NB>
cudaError_t launch(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, const PackedWork& work, bool both,
                   cudaStream_t stream) {
  using C = NarrowCosts<NB>;
  constexpr int kBytes = Smem<D, NB>::kBytes;
  auto kernel = attention_narrow_kernel<D, NB>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err != cudaSuccess) return err;
  const int blocks = std::min(narrow_blocks(D, NB), 227 * 1024 / (kBytes + 1024));
  const int most_rows = attn_window_rows(a.Hq), windows = (int)(((int64_t)a.rows + most_rows - 1) / most_rows);
  const int step = (int)(((int64_t)a.rows + windows - 1) / windows);
  const Pieces narrow{work.narrow_part, work.narrow_stat, work.narrow_plan}, wide{work.part, work.stat, work.plan};
  for (int64_t lo = 0; lo < a.rows; lo += step) {
    const Window w{(int)lo, (int)std::min<int64_t>(lo + step, a.rows), both ? kNarrowMost : INT_MAX};
    if (both && (err = launch_attention_wide(a, packed, sms, w.lo, w.hi, w.narrow, work, stream)) != cudaSuccess) return err;
    kernel<<<sms * blocks, kThreads, kBytes, stream>>>(a, packed, w, work.narrow_part, work.narrow_stat, work.narrow_plan);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    err = launch_join<D, WideCosts<true>, C>(a, w, windows, wide, narrow, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t launch(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, const PackedWork& work, cudaStream_t stream) {
  const int64_t m = (int64_t)a.rows * (a.Hq / a.Hk), R = a.R;  // query rows of a key head
  // The narrow kernel alone where no segment has more than kNarrowMost query rows, or where requests without
  // a prefix have few; otherwise the wide one takes the segments of more before it.  (256 requests of
  // 1024 keys, 8 heads a key head: 1 or 2 rows a request 162 us by the narrow kernel alone, 170 by
  // both; 1 to 4 rows 246 and 224; 1 to 12 rows 541 and 253, with 32 rows for 16 as the border 261.)  The
  // mean knows nothing of one long request among single rows: 255 rows and a request of 256 over 8000 keys, 8 heads a key head,
  // 859 us by the narrow kernel alone and 711 by both, 255 and 700 at 4 heads 1074 and 821, 2000 and 4000 19.4 ms and 3.9; but 31 rows and
  // a request of 30 over 8000 keys 125 us and 206.
  const bool both = m > kNarrowMost && (a.G > 0 || m > kNarrowMost * R);
  // 16 rows an item cost 1.45 times 8 (D = 128: 256 requests of 4096 keys 461 us and 318) or 1.22 times (D = 64: 101
  // requests of 1500 keys 54 us and 44), but read the keys of a request of 9 to 16 rows once: where a
  // request has several rows, some have more than the mean.  250 requests of up to 1500 keys, 8 rows an item and 16: heads of 64, a
  // mean of 4.4 rows 58 and 67 us, 5.9 55 and 64, 6.0 (some of 9) 71 and 68, 7.5 76 and 66, 10 76 and 66; heads of 128, 7.5 98 and
  // 110, and past 8 neither is ahead everywhere: 8.3 95 and 114, 9.2 110 and 114, 101 requests of up to 3000 keys 9.4 80 and 77.
  const int64_t most = D == 64 && a.rows > a.R ? 6 : 8;
  if (m <= most * R) return launch<D, 1>(a, packed, sms, work, both, stream);
  return launch<D, 2>(a, packed, sms, work, both, stream);
}

}  // namespace

// bf16 heads of 64 or 128, pages that tile 128 keys, rows, data and scales on 16 bytes.
bool attn_packed_ok(const spec_prefix_attention_args& a, const q4::Cache& packed, int* sms) {
  if (((uintptr_t)packed.k_scale | (uintptr_t)packed.v_scale) % 16 != 0) return false;
  return attn_tc_ok(a, sms);
}

cudaError_t launch_attention_packed(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, const PackedWork& work,
                                    cudaStream_t stream) {
  return a.D == 128 ? launch<128>(a, packed, sms, work, stream) : launch<64>(a, packed, sms, work, stream);
}

}  // namespace spec
