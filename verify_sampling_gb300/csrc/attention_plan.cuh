// What the tensor-core attention kernels share: the work layout that every block computes from
// the lengths, and the join of a row's pieces.
//
// An item is up to C::kItemRows query rows (packed rows x the query heads of one key head) of
// a segment, a group over its prefix or a request over its own keys.  The items' tiles of 128
// keys, laid end to end with a fixed cost an item, are cut into equal lengths, one per block: blocks
// finish together whatever the mix of one long prefix, many short requests or one request
// alone.  An item cut between blocks leaves several pieces; the join adds up every row's.
//
// C says what an item and a tile cost.  Two kernels may share a call's segments: the
// narrow one takes those of up to Window::narrow query rows, the wide one the others.
#pragma once

#include <cstddef>

#include "attention.cuh"
#include "tc.cuh"

namespace spec {

namespace {

using namespace attn;

constexpr int kTile = 128;  // keys of a tile
constexpr uint64_t kWaitNs = 2000000000ull;

// ------------------------------------------------------------ work layout --
// Costs, in units of 0.1 us, measured: a tile of an item of both softmax groups (bound
// by the products), a tile of a smaller one (bound by its 64 KB where all blocks stream,
// otherwise by its chain of product, softmax and product), and an item's start and end.
// Over a packed cache (SHARED: a narrow kernel takes the segments of few rows) both kinds of tile cost
// what their unpacking does, 2 us: with the other kernel's costs the round of 256 requests behind a
// prefix took 911 us, with these 839.
template <bool SHARED>
struct WideCosts {
  static constexpr int kItemRows = attn::kItemRows;
  static constexpr bool kShared = SHARED, kWide = true;
  static constexpr int kPair = SHARED ? 20 : 17, kSingle = SHARED ? 20 : 15, kLeast = kPair;
  __device__ static __forceinline__ int tile(int rows) { return rows > kTile ? kPair : kSingle; }
  __device__ static __forceinline__ int start(int rows) { return rows > kTile ? (SHARED ? 30 : 57) : (SHARED ? 20 : 21); }
  // Tiles whose costs begin before `x` units of an item's tiles.
  __device__ static __forceinline__ int tiles_before(int x, int rows) {
    return rows > kTile ? (unsigned)(x + kPair - 1) / kPair : (unsigned)(x + kSingle - 1) / kSingle;
  }
};

struct Window {  // the packed rows of a launch: [lo, hi)
  int lo, hi;
  int narrow;  // where two kernels share the segments: query rows of the largest that the narrow one takes
};
__device__ __forceinline__ Rows inside(const Rows& rows, const Window& w) {
  const int lo = max(rows.row0, w.lo), hi = min(rows.row0 + rows.n, w.hi);
  return Rows{lo, max(hi - lo, 0)};
}

struct Segment {  // a group's prefix or a request's own keys
  int row0, n;    // packed rows in the window
  int keys;
  int first_own;  // own index of row 0's last key + 1 (prefix: keys)
  const int32_t* table;
  bool prefix;
};

struct Item {
  int row0, m0, rows;  // query rows m0 .. m0 + rows of the segment's n * heads-per-key-head
  int h, lo, hi;       // key head, tiles
  int keys;            // keys the item reads
  int first_own;
  bool prefix;
  bool direct;  // the whole of its rows' keys: the result itself is written
  const int32_t* table;
  size_t slot;  // partial row of its row m0
};

struct Layout {
  int64_t per;  // cost of a block
  int64_t x0, x1;
  int k0;        // first segment and its position
  int64_t s0;
};

__device__ __forceinline__ Segment segment(const spec_prefix_attention_args& a, const Window& w, int k, uint32_t* bad) {
  Segment s;
  if (k < a.G) {
    const int2 in = group_requests(a, k, bad);
    const Rows rows = inside(rows_between(a, in.x, in.y, bad), w);
    s = Segment{rows.row0, rows.n, prefix_keys(a, k, bad), 0,
                a.prefix_table + (size_t)k * a.max_prefix_pages, true};
    s.first_own = s.keys;
  } else {
    const int r = k - a.G;
    const Rows all = rows_between(a, r, r + 1, bad), rows = inside(all, w);
    const int kv = own_keys(a, r, bad);
    s = Segment{rows.row0, rows.n, kv, kv - all.n + 1 + (rows.row0 - all.row0),
                a.block_table + (size_t)r * a.max_pages, false};
  }
  return s;
}
// The group that request r is in, or -1, and the keys of its prefix.
__device__ __forceinline__ int group_of(const spec_prefix_attention_args& a, int r, uint32_t* bad) {
  if (a.G == 0) return -1;
  const int g = last_at_or_below(a.group_off, a.G, r);
  const int2 in = group_requests(a, g, bad);
  return r >= in.x && r < in.y ? g : -1;
}
__device__ __forceinline__ int shared_keys(const spec_prefix_attention_args& a, int r, uint32_t* bad) {
  const int g = group_of(a, r, bad);
  return g < 0 ? 0 : prefix_keys(a, g, bad);
}
// Keys that the item of query rows [C::kItemRows i, ..) needs: its last row's.
template <class C>
__device__ __forceinline__ int item_keys(const Segment& s, int i, int per_head) {
  if (s.prefix) return s.keys;
  const int j = min(s.n - 1, (i * C::kItemRows + C::kItemRows - 1) / per_head);
  return max(0, min(s.keys, s.first_own + j));
}
template <class C>
__device__ __forceinline__ int item_count(const Segment& s, int per_head, const Window& w) {
  const unsigned m = (unsigned)s.n * (unsigned)per_head;  // rows * Hq < 2^31
  if (C::kShared && ((int)m > w.narrow) != C::kWide) return 0;
  return (int)((m + C::kItemRows - 1) / C::kItemRows);
}
// Cost of an item of `rows` query rows (or more: C::kItemRows are its own).
template <class C>
__device__ __forceinline__ int item_cost(int keys, int rows) {
  const int tiles = (keys + kTile - 1) / kTile;
  return tiles ? C::start(rows) + tiles * C::tile(rows) : 0;
}
template <class C>
__device__ __forceinline__ int64_t head_cost(const Segment& s, int per_head, const Window& w) {
  const int n = item_count<C>(s, per_head, w);
  if (n == 0) return 0;
  int64_t c = item_cost<C>(item_keys<C>(s, n - 1, per_head), s.n * per_head - (n - 1) * C::kItemRows);
  if (s.prefix) return c + (int64_t)(n - 1) * item_cost<C>(s.keys, C::kItemRows);
#pragma unroll 1
  for (int i = 0; i < n - 1; ++i) c += item_cost<C>(item_keys<C>(s, i, per_head), C::kItemRows);
  return c;
}
// x / y rounded up or a little more, by one 32-bit division: the code of a 64-bit one
// is a good part of what a block with little work has to fetch before it starts.
__device__ __forceinline__ int64_t share_of(int64_t x, unsigned y) {
  const int drop = max(0, 32 - __clzll(x));
  return (int64_t)((unsigned)(x >> drop) / y + 1) << drop;
}

// The block's items in order.  (One copy of each step: a block's first item waits for
// this code to be fetched.)
template <class C>
struct Walker {
  const spec_prefix_attention_args& a;
  const Window& w;
  int64_t pos, x0, x1;
  int k, h, i, per_head, count;
  Segment seg;
  bool alone;  // a request without a prefix
  uint32_t bad;

  __device__ Walker(const spec_prefix_attention_args& args, const Window& window, const Layout& lay)
      : a(args), w(window), pos(lay.s0), x0(lay.x0), x1(lay.x1), k(lay.k0 - 1), h(0), i(0),
        per_head(args.Hq / args.Hk), count(0), alone(false), bad(0) {}
  __device__ __forceinline__ bool next(Item& it) {
#pragma unroll 1
    while (pos < x1) {
      if (i >= count) {  // next head, or next segment
        i = 0;
        if (count == 0 || ++h >= a.Hk) {
          h = 0;
          if (++k >= a.G + a.R) return false;
          seg = segment(a, w, k, &bad);
          count = item_count<C>(seg, per_head, w);
          alone = k >= a.G && (a.G == 0 || shared_keys(a, k - a.G, &bad) == 0);
          if (count > 0 && pos < x0) {  // the layout starts in this segment: whole heads before it
            const int64_t c = head_cost<C>(seg, per_head, w);
#pragma unroll 1
            for (; pos + c <= x0 && h + 1 < a.Hk; ++h) pos += c;
          }
        }
        continue;
      }
      const int keys = item_keys<C>(seg, i, per_head), m = seg.n * per_head;
      it.m0 = i * C::kItemRows;
      ++i;
      const int left = m - it.m0;
      const int cost = item_cost<C>(keys, left), tiles = (keys + kTile - 1) / kTile;
      const int64_t at = pos + C::start(left);
      pos += cost;
      if (cost == 0 || pos <= x0) continue;
      it.lo = x0 <= at ? 0 : C::tiles_before((int)(x0 - at), left);  // x0 - at < cost
      it.hi = x1 <= at ? 0 : x1 >= pos ? tiles : C::tiles_before((int)(x1 - at), left);
      if (it.lo >= it.hi) continue;
      it.row0 = seg.row0;
      it.rows = min(C::kItemRows, left);
      it.h = h;
      it.keys = keys;
      it.first_own = seg.first_own;
      it.prefix = seg.prefix;
      it.direct = alone && it.lo == 0 && it.hi == tiles;
      it.table = seg.table;
      it.slot = (seg.prefix ? 0 : (size_t)(w.hi - w.lo) * a.Hq) + (size_t)(seg.row0 - w.lo) * a.Hq + (size_t)h * m +
                it.m0 + (size_t)C::kItemRows * blockIdx.x;
      return true;
    }
    return false;
  }
};

// The block's part of the layout, to *lay; every thread a run of segments, one scan.  `setup` is
// done before a barrier of the block; another has to follow before *lay is read.  Block 0 leaves the
// segments' positions in `plan`, for the join.
template <class C, int kThreads, class Setup>
__device__ __forceinline__ void lay_out(const spec_prefix_attention_args& a, const Window& w, Layout* lay,
                                        int64_t* warp_sum, int64_t* plan, Setup setup) {
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per_head = a.Hq / a.Hk;
  const int n_seg = a.G + a.R, run = (n_seg + kThreads - 1) / kThreads;
  const int k0 = min(tid * run, n_seg), k1 = min(k0 + run, n_seg);
  uint32_t bad = 0;
  auto cost_of = [&](int k) { return a.Hk * head_cost<C>(segment(a, w, k, &bad), per_head, w); };
  int64_t mine = 0;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) mine += cost_of(k);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  setup();
  if (tid == 0) *lay = Layout{0, 0, 0, 0, 0};
  __syncthreads();
  int64_t sum = lane < kThreads / 32 ? warp_sum[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  const int64_t total = __shfl_sync(0xffffffffu, sum, 31);
  const int64_t upto = __shfl_sync(0xffffffffu, sum, warp);
  int64_t at = upto - __shfl_sync(0xffffffffu, inc, 31) + inc - mine;  // the thread's first segment
  // at least one tile a block, so that every block of an item's range has one
  const int64_t per = max(share_of(total, gridDim.x), (int64_t)C::kLeast);
  const int64_t x0 = per * blockIdx.x, x1 = min(x0 + per, total);
  const bool here = x0 < x1 && at <= x0 && x0 < at + mine;
  if (here || blockIdx.x == 0) {
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      const int64_t c = run == 1 ? mine : cost_of(k);
      if (blockIdx.x == 0) plan[1 + k] = at;
      if (here && at <= x0 && x0 < at + c) *lay = Layout{per, x0, x1, k, at};
      at += c;
    }
  }
  if (blockIdx.x == 0 && tid == 0) plan[0] = per;
  if (bad && blockIdx.x == 0) set_status(a.status, bad);
}

// The rest of a wait whose first look failed.  Gives up when the time limit passes or
// another warp has given up.
__device__ __forceinline__ bool slow_wait_here(uint64_t* bar, uint32_t phase, volatile int* abort_flag, uint32_t* status) {
  const uint64_t t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait_suspend(bar, phase & 1u, 1000000u)) {
    if (*abort_flag) return false;
    if (tc::globaltimer_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      set_status(status, SPEC_STATUS_TIMEOUT);
      return false;
    }
  }
  return true;
}
// (Out of line: the code of a role that a short item runs once has to fit the instruction
// cache beside the others'.)
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t phase, volatile int* abort_flag, uint32_t* status) {
  return slow_wait_here(bar, phase, abort_flag, status);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// bf16x2 with `lo` in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ----------------------------------------------------------------- join ----
constexpr int kJoinThreads = 128;
constexpr int kFewRows = 152 * 8;  // query rows of a call whose join has a block for each
constexpr int kJoinBlocks = 152 * 16;
constexpr int kJoinRows = 64;  // query rows (packed rows x heads of a key head) of a block at a time

constexpr int kJoinLanes = 16;  // threads of a row
constexpr int join_rows(int share) { return share > 1 ? 1 : kJoinRows; }  // of a block at a time

// Cost of a head's items before item `upto`, and of all of them; a row's threads add them up.
template <class C>
__device__ __forceinline__ void costs_of(const Segment& s, const Window& w, int per_head, int upto, int64_t* before, int64_t* all) {
  const int n = item_count<C>(s, per_head, w), lane = threadIdx.x % kJoinLanes;
  const uint32_t lanes = (uint32_t)((1ull << kJoinLanes) - 1) << (threadIdx.x & 31 & ~(kJoinLanes - 1));
  int64_t x = 0, y = 0;
  for (int i = lane; i < n; i += kJoinLanes) {
    const int64_t c = item_cost<C>(item_keys<C>(s, i, per_head), s.n * per_head - i * C::kItemRows);
    y += c;
    if (i < upto) x += c;
  }
#pragma unroll
  for (int o = kJoinLanes / 2; o > 0; o >>= 1) {
    x += __shfl_xor_sync(lanes, x, o);
    y += __shfl_xor_sync(lanes, y, o);
  }
  *before = x;
  *all = y;
}

// Joins the pieces of every row that has more than one.  A block takes a request's
// rows, tiles of 64 of one key head after the other: what says where their pieces are
// is a chain of dependent loads, paid once a block.  Half a warp a row: twice the rows in
// flight (the round of 256 requests behind a prefix 779 us in all, 790 with a warp a row, both in
// short runs: after half a second the power limit's clock makes it 828).
struct Pieces {  // what a kernel leaves
  const float* part;
  const float2* stat;
  const int64_t* plan;
};
// kShare: half-warps that share a row's pieces (all of a block's or one).
template <int D, int kShare, class C, class N>
__device__ __forceinline__ void join_request(const spec_prefix_attention_args& a, const Window& w, int r, const Pieces& wide,
                                             const Pieces& narrow) {
  constexpr int kPer = D / kJoinLanes, kBatch = 4, kHalves = kJoinThreads / kJoinLanes;
  constexpr int kTileRows = join_rows(kShare);
  static_assert(kShare == 1 || kShare == kHalves, "a block's half-warps");
  const int lane = threadIdx.x % kJoinLanes, per_head = a.Hq / a.Hk;
  const int share = kShare > 1 ? threadIdx.x / kJoinLanes : 0;
  uint32_t bad = 0;
  const Segment own = segment(a, w, a.G + r, &bad);
  int g = group_of(a, r, &bad);
  Segment pre{0, 0, 0, 0, nullptr, true};
  if (g >= 0) pre = segment(a, w, g, &bad);
  if (own.row0 < pre.row0 || own.row0 + own.n > pre.row0 + pre.n) g = -1;  // rows out of order
  const int m_own = own.n * per_head;
  const int m_off = (own.row0 - pre.row0) * per_head;  // the request's first row among the group's
  tc::grid_dep_wait();  // all of the above is the caller's; the pieces and their layout are ready now
  // the kernel that took the segment, and the query rows of its items
  const bool own_n = C::kShared && m_own <= w.narrow, pre_n = C::kShared && pre.n * per_head <= w.narrow;
  const Pieces& from_own = own_n ? narrow : wide;
  const Pieces& from_pre = pre_n ? narrow : wide;
  const int own_rows = own_n ? N::kItemRows : C::kItemRows, pre_rows = pre_n ? N::kItemRows : C::kItemRows;
  const int64_t own_per = from_own.plan[0], pre_per = from_pre.plan[0];
  const int64_t own_at = from_own.plan[1 + a.G + r], pre_at = g >= 0 ? from_pre.plan[1 + g] : 0;

  const int tiles = (m_own + kTileRows - 1) / kTileRows, all_tiles = tiles * a.Hk;
  int item[2] = {-1, -1}, head = -1;  // own and prefix item, and key head, whose pieces are known
  int64_t before[2] = {0, 0}, all[2] = {0, 0};
  int first[2] = {0, 0}, count[2] = {0, 0};
  auto pieces = [&](auto costs, int k, const Segment& s, int64_t at, int64_t per, int h, int i) {  // blocks that have pieces of item i
    using X = decltype(costs);
    if (i == item[k] && h == head) return;
    const int tiles = (item_keys<X>(s, i, per_head) + kTile - 1) / kTile;
    count[k] = 0;
    if (i != item[k]) costs_of<X>(s, w, per_head, i, &before[k], &all[k]);
    item[k] = i;
    if (tiles == 0) return;
    const int rows = s.n * per_head - i * X::kItemRows;
    at += h * all[k] + before[k] + X::start(rows);
    first[k] = (int)(at / per);
    count[k] = (int)((at + (int64_t)(tiles - 1) * X::tile(rows)) / per) - first[k] + 1;
  };
  auto find = [&](bool n, int k, const Segment& s, int64_t at, int64_t per, int h, int m) {
    if (C::kShared && n) pieces(N{}, k, s, at, per, h, m / N::kItemRows);
    else pieces(C{}, k, s, at, per, h, m / C::kItemRows);
  };

  const bool wide_out = ((uintptr_t)a.out & 7) == 0 && a.out_row % 4 == 0 && a.out_head % 4 == 0;

#pragma unroll 1
  for (int x = blockIdx.y; x < all_tiles; x += gridDim.y) {
    const int h = x / tiles, m0 = (x - h * tiles) * kTileRows;
    const size_t own_slot = ((size_t)(w.hi - w.lo) + (own.row0 - w.lo)) * a.Hq + (size_t)h * m_own;
    const size_t pre_slot = (size_t)(pre.row0 - w.lo) * a.Hq + (size_t)h * pre.n * per_head + m_off;
    for (int m = m0 + (kShare > 1 ? 0 : threadIdx.x / kJoinLanes); m < min(m0 + kTileRows, m_own); m += kHalves / kShare) {
      find(own_n, 0, own, own_at, own_per, h, m);
      if (g >= 0) find(pre_n, 1, pre, pre_at, pre_per, h, m_off + m);
      head = h;
      const int c0 = count[0], n = c0 + count[1];
      if (count[1] == 0 && n == 1) continue;  // written by its block
      // piece p lies at one of two places plus p steps of an item's rows
      const size_t own_at_row = own_slot + m + (size_t)own_rows * first[0];
      const size_t pre_at_row = pre_slot + m + (size_t)pre_rows * first[1] - (size_t)pre_rows * c0;
      const float* own_part = from_own.part + own_at_row * D + lane * kPer;
      const float* pre_part = from_pre.part + (ptrdiff_t)pre_at_row * D + lane * kPer;
      float top = -CUDART_INF_F, sum = 0.f, o[kPer];
#pragma unroll
      for (int d = 0; d < kPer; ++d) o[d] = 0.f;
#pragma unroll 1
      for (int p0 = share * kBatch; p0 < n; p0 += kShare * kBatch) {
        float2 st[kBatch];
        float v[kBatch][kPer];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int p = p0 + i;
          st[i] = make_float2(-CUDART_INF_F, 0.f);
          if (p < n) {
            const size_t step = (size_t)p * (p < c0 ? own_rows : pre_rows);
            st[i] = (p < c0 ? from_own.stat + own_at_row : from_pre.stat + (ptrdiff_t)pre_at_row)[step];
            const float* src = (p < c0 ? own_part : pre_part) + step * D;
#pragma unroll
            for (int d = 0; d < kPer; d += 4) {
              const float4 y = *reinterpret_cast<const float4*>(src + d);
              v[i][d] = y.x, v[i][d + 1] = y.y, v[i][d + 2] = y.z, v[i][d + 3] = y.w;
            }
          }
        }
        const float m_new = fmaxf(max3(st[0].x, st[1].x, st[2].x), fmaxf(st[3].x, top));
        const float c = top == -CUDART_INF_F ? 0.f : tc::ex2(top - m_new);
        sum *= c;
#pragma unroll
        for (int d = 0; d < kPer; ++d) o[d] *= c;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (p0 + i >= n) break;
          const float w = st[i].x == -CUDART_INF_F ? 0.f : tc::ex2(st[i].x - m_new);
          sum = fmaf(st[i].y, w, sum);
#pragma unroll
          for (int d = 0; d < kPer; ++d) o[d] = fmaf(v[i][d], w, o[d]);
        }
        top = m_new;
      }
      if (kShare > 1) {  // the half-warps' sums, by the first of them
        __shared__ __align__(16) float o_s[kHalves][D];
        __shared__ float2 stat_s[kHalves];
        __syncthreads();  // the last row's are read
#pragma unroll
        for (int d = 0; d < kPer; ++d) o_s[share][lane * kPer + d] = o[d];
        if (lane == 0) stat_s[share] = make_float2(top, sum);
        __syncthreads();
        if (share > 0) continue;
        float m_all = top;
#pragma unroll
        for (int x = 1; x < kHalves; ++x) m_all = fmaxf(m_all, stat_s[x].x);
        const float c = top == -CUDART_INF_F ? 0.f : tc::ex2(top - m_all);
        sum *= c;
#pragma unroll
        for (int d = 0; d < kPer; ++d) o[d] *= c;
#pragma unroll
        for (int x = 1; x < kHalves; ++x) {
          const float w = stat_s[x].x == -CUDART_INF_F ? 0.f : tc::ex2(stat_s[x].x - m_all);
          sum = fmaf(stat_s[x].y, w, sum);
#pragma unroll
          for (int d = 0; d < kPer; ++d) o[d] = fmaf(o_s[x][lane * kPer + d], w, o[d]);
        }
        top = m_all;
      }
      const int j = m / per_head, b = own.row0 + j, hq = h * per_head + (m - j * per_head);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row without keys: zeros
      __nv_bfloat16* out = (__nv_bfloat16*)a.out + (size_t)b * a.out_row + (size_t)hq * a.out_head + lane * kPer;
      uint32_t r2[kPer / 2];
#pragma unroll
      for (int d = 0; d < kPer; d += 2) r2[d / 2] = pack_bf16(o[d] * inv, o[d + 1] * inv);
      if (wide_out) {
#pragma unroll
        for (int d = 0; d < kPer / 2; d += 2) *reinterpret_cast<uint2*>(out + 2 * d) = make_uint2(r2[d], r2[d + 1]);
      } else {
#pragma unroll
        for (int d = 0; d < kPer / 2; ++d) *reinterpret_cast<uint32_t*>(out + 2 * d) = r2[d];
      }
      if (a.lse && lane == 0)
        a.lse[(size_t)b * a.Hq + hq] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
    }
  }
}

// Where the window is a part of the rows (kPart), the blocks share out its requests, from
// the first to the last that has rows in it; otherwise there is a block for each.
template <int D, bool kPart, int kShare, class C, class N>
__global__ void __launch_bounds__(kJoinThreads, 4)
    join_pieces_kernel(const spec_prefix_attention_args a, const Window w, const Pieces wide, const Pieces narrow) {
  int r = blockIdx.x;
  if (!kPart) {
    join_request<D, kShare, C, N>(a, w, r, wide, narrow);
    return;
  }
  __shared__ int first_s, last_s;
  if (threadIdx.x == 0) first_s = a.R, last_s = -1;
  __syncthreads();
  int first = a.R, last = -1;
#pragma unroll 8
  for (int i = threadIdx.x; i < a.R; i += kJoinThreads) {
    const int row0 = a.row_off[i], row1 = a.row_off[i + 1];
    if (row0 < row1 && row0 < w.hi && row1 > w.lo) first = min(first, i), last = max(last, i);
  }
  if (last >= 0) {
    atomicMin(&first_s, first);
    atomicMax(&last_s, last);
  }
  __syncthreads();
  for (r += first_s; r <= last_s; r += gridDim.x) join_request<D, kShare, C, N>(a, w, r, wide, narrow);
  tc::grid_dep_wait();  // a block without requests, too, ends after the pieces' kernel
}

// Blocks of the join for a call's rows in `windows` windows.
inline dim3 join_grid(const spec_prefix_attention_args& a, int windows, int tile_rows) {
  // a block a tile of the mean request, until there are kJoinBlocks of them
  const int per_head = a.Hq / a.Hk;
  const int64_t tiles = (((int64_t)a.rows * per_head + (int64_t)tile_rows * a.R - 1) / ((int64_t)tile_rows * a.R)) * a.Hk;
  const int at_once = std::min(a.R, (a.R + windows - 1) / windows + (windows > 1));  // requests of a window
  const int64_t most = (kJoinBlocks + at_once - 1) / at_once;
  return dim3(at_once, (unsigned)(tiles < most ? tiles : most));
}

template <int D, class C, class N>
cudaError_t launch_join(const spec_prefix_attention_args& a, const Window& w, int windows, const Pieces& wide, const Pieces& narrow,
                        cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  // Few rows over a packed cache have many pieces each: a block shares them (one row of 20001 keys, 32 heads on 8:
  // 57 pieces a row, 21.4 us with a row a half-warp, 15.8 with a row a block).
  const bool few = C::kShared && windows == 1 && (int64_t)a.rows * a.Hq <= kFewRows;
  constexpr int kHalves = C::kShared ? kJoinThreads / kJoinLanes : 1;
  cfg.gridDim = join_grid(a, windows, join_rows(few ? kHalves : 1));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg,
                            windows > 1 ? join_pieces_kernel<D, true, 1, C, N>
                            : few       ? join_pieces_kernel<D, false, kHalves, C, N>
                                        : join_pieces_kernel<D, false, 1, C, N>,
                            a, w, wide, narrow);
}

}  // namespace

}  // namespace spec
