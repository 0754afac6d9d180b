// Shared-prefix attention on the tensor cores (bf16, heads of 64 or 128): a
// round's packed rows against the prefix pages that their group shares and each
// request's own pages, every key read once for all the rows that need it.
//
// Mathematics: for a row with scaled scores z (log2 units) over a piece of its
// keys, the piece keeps a reference m, l = sum 2^(z - m) and O = sum 2^(z - m) v;
// pieces join as out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  m follows the
// running maximum only when it has grown by more than 8, so O is rescaled a few
// times a row instead of once a tile; a weight is then at most 2^8 and fp32 sums
// lose nothing by it.  Weights are rounded to bf16 for the second product (8 bits
// of a weight are 8 bits of its share of the result); l adds them unrounded.
//
// Work: an item is up to 256 query rows (packed rows x the query heads of one
// key head) of a group over its prefix, or of a request over its own keys.  The
// items' tiles of 128 keys, laid end to end with a fixed cost an item, are cut
// into equal lengths, one per block and one block per SM: blocks finish together
// whatever the mix of one long prefix, many short requests or one request alone.
// Lengths are device data, so each block computes the layout itself (one scan).
// An item cut between blocks leaves several pieces; a second kernel joins every
// row's pieces.
//
// Block: planner warp (walks the block's items and posts them in shared memory),
// producer warp (TMA of key and value tiles, 64 x page boxes, into one ring), loader
// warp (query rows: TMA where the heads of a key head divide a box, else 16-byte
// copies into the swizzled places), MMA warp (S = Q K^T into TMEM, O += P V with P
// read from TMEM), and two softmax groups of 128 rows.  A row has two threads of a
// warp, each half of its columns, that meet in a shuffle for the maximum: with one
// thread a row the time from scores to weights (1870 clocks) was most of the 3860 of a
// tile, and the tensor pipe waited for it.  An item of more than 128 rows uses both groups on
// the same key tile, one's softmax under the other's products; smaller items
// alternate between them, and the next item's first product is issued before the
// current one's last weights are ready.
//
// Every wait is bounded; on a timeout the block sets SPEC_STATUS_TIMEOUT, waits
// for its copies and products in flight and frees its TMEM.
#include <cuda.h>

#include <cstddef>

#include "attention.cuh"
#include "fused_tc.cuh"
#include "tc.cuh"

namespace spec {

namespace {

using namespace attn;

constexpr int kTile = 128;  // keys of a tile, rows of a softmax group
// Softmax warps: group t (rows 128 t ..) is warps 8 t .. 8 t + 7; warps w and w + 4 of it
// share 32 rows (TMEM lanes go by the warp's number mod 4), 16 each, and a row has
// threads i and i + 16 of its warp, each half of its columns.
constexpr int kSoftWarps = 16, kProducer = 16, kMma = 17, kPlanner = 18, kLoader = 19;
constexpr int kThreads = 640;
constexpr int kItemSlots = 4, kItemReaders = 3 + kSoftWarps;  // producer, MMA, loader, softmax warps
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kSlack = 8.f;  // log2 units the maximum may grow by before O is rescaled
// Costs, in units of 0.1 us, measured: a tile of an item of both softmax groups (bound
// by the products), a tile of a smaller one (bound by its 64 KB where all blocks stream,
// otherwise by its chain of product, softmax and product), and an item's start and end.
constexpr int kCostPair = 17, kCostSingle = 15, kCostStartPair = 57, kCostStartSingle = 21;

// ------------------------------------------------------------ work layout --
struct Window {  // the packed rows of a launch: [lo, hi)
  int lo, hi;
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
// Keys that the item of query rows [256 i, ..) needs: its last row's.
__device__ __forceinline__ int item_keys(const Segment& s, int i, int per_head) {
  if (s.prefix) return s.keys;
  const int j = min(s.n - 1, (i * kItemRows + kItemRows - 1) / per_head);
  return max(0, min(s.keys, s.first_own + j));
}
__device__ __forceinline__ int item_count(const Segment& s, int per_head) {
  return (int)(((unsigned)s.n * (unsigned)per_head + kItemRows - 1) / kItemRows);  // rows * Hq < 2^31
}
__device__ __forceinline__ int tile_cost(int rows) { return rows > kTile ? kCostPair : kCostSingle; }
__device__ __forceinline__ int start_cost(int rows) { return rows > kTile ? kCostStartPair : kCostStartSingle; }
// Cost of an item of `rows` query rows (or more: 256 are its own).
__device__ __forceinline__ int item_cost(int keys, int rows) {
  const int tiles = (keys + kTile - 1) / kTile;
  return tiles ? start_cost(rows) + tiles * tile_cost(rows) : 0;
}
__device__ __forceinline__ int64_t head_cost(const Segment& s, int per_head) {
  const int n = item_count(s, per_head);
  if (n == 0) return 0;
  int64_t c = item_cost(item_keys(s, n - 1, per_head), s.n * per_head - (n - 1) * kItemRows);
  if (s.prefix) return c + (int64_t)(n - 1) * item_cost(s.keys, kItemRows);
#pragma unroll 1
  for (int i = 0; i < n - 1; ++i) c += item_cost(item_keys(s, i, per_head), kItemRows);
  return c;
}
// x / y rounded up or a little more, by one 32-bit division: the code of a 64-bit one
// is a good part of what a block with little work has to fetch before it starts.
__device__ __forceinline__ int64_t share_of(int64_t x, unsigned y) {
  const int drop = max(0, 32 - __clzll(x));
  return (int64_t)((unsigned)(x >> drop) / y + 1) << drop;
}

// Tiles whose costs begin before `x` units of an item's tiles.
__device__ __forceinline__ int tiles_before(int x, int rows) {
  return rows > kTile ? (unsigned)(x + kCostPair - 1) / kCostPair : (unsigned)(x + kCostSingle - 1) / kCostSingle;
}

// The block's items in order.  (One copy of each step: a block's first item waits for
// this code to be fetched.)
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
          count = item_count(seg, per_head);
          alone = k >= a.G && (a.G == 0 || shared_keys(a, k - a.G, &bad) == 0);
          if (count > 0 && pos < x0) {  // the layout starts in this segment: whole heads before it
            const int64_t c = head_cost(seg, per_head);
#pragma unroll 1
            for (; pos + c <= x0 && h + 1 < a.Hk; ++h) pos += c;
          }
        }
        continue;
      }
      const int keys = item_keys(seg, i, per_head), m = seg.n * per_head;
      it.m0 = i * kItemRows;
      ++i;
      const int left = m - it.m0;
      const int cost = item_cost(keys, left), tiles = (keys + kTile - 1) / kTile;
      const int64_t at = pos + start_cost(left);
      pos += cost;
      if (cost == 0 || pos <= x0) continue;
      it.lo = x0 <= at ? 0 : tiles_before((int)(x0 - at), left);  // x0 - at < cost
      it.hi = x1 <= at ? 0 : x1 >= pos ? tiles : tiles_before((int)(x1 - at), left);
      if (it.lo >= it.hi) continue;
      it.row0 = seg.row0;
      it.rows = min(kItemRows, left);
      it.h = h;
      it.keys = keys;
      it.first_own = seg.first_own;
      it.prefix = seg.prefix;
      it.direct = alone && it.lo == 0 && it.hi == tiles;
      it.table = seg.table;
      it.slot = (seg.prefix ? 0 : (size_t)(w.hi - w.lo) * a.Hq) + (size_t)(seg.row0 - w.lo) * a.Hq + (size_t)h * m +
                it.m0 + (size_t)kItemRows * blockIdx.x;
      return true;
    }
    return false;
  }
};

// ------------------------------------------------------------- tcgen05 -----
// Descriptors of the 128-byte swizzle layout (8-row groups 1024 bytes apart) differ
// in their low words alone.  The products are issued by one lane through a predicate,
// not inside a branch: the warp's control flow and addresses stay uniform, so they
// live in uniform registers, which the instruction takes.  Issued from a one-lane
// branch, the moves into them held the tensor pipe to 54% of its rate.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, swizzle
// K-major operand at a shared address
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
// MN-major operand: rows of 64 elements, the next 64 elements `lead` bytes on
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t lead) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi), "r"(lead)
      : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          tc::smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// 1 in one lane of the warp.
__device__ __forceinline__ uint32_t elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// Columns [0, 16) of 16 TMEM lanes to threads 0-15, the 16 from `SPLIT` on of the same
// lanes to threads 16-31: a row's two halves in one warp.
template <int SPLIT>
__device__ __forceinline__ void tmem_ld16h(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "n"(SPLIT)
      : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_ld32h(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(SPLIT)
      : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_ld64h(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,"
      "%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64], %65;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "n"(SPLIT)
      : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16h(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17};" ::"r"(taddr), "n"(SPLIT),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 16 bytes to a shared address, without registers in between.
__device__ __forceinline__ void copy16(uint32_t saddr, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// 32 bytes to a 32-byte address: one whole sector.
__device__ __forceinline__ void store32(float* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// bf16x2 with `lo` in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The rest of a wait whose first look failed.  Gives up when the time limit passes or
// another warp has given up.  (Out of line: the code of a role that a short item
// runs once has to fit the instruction cache beside the others'.)
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t phase, volatile int* abort_flag, uint32_t* status) {
  for (int i = 0; i < 2000; ++i) {
    if (tc::mbar_wait(bar, phase & 1u, kWaitNs / 2000)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, SPEC_STATUS_TIMEOUT);
  return false;
}

// Everything shared beside the tiles.
struct Shared {
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], drain;
  Item items[kItemSlots];
  Layout lay;
  int64_t warp_sum[kThreads / 32];
  uint32_t tmem;
  volatile int abort_flag;
};

template <int D>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kRing = 2 * kTileBytes;  // after the two query tiles
  static constexpr int kShared = kRing + kStages * kTileBytes;
  static constexpr int kBytes = kShared + (int)sizeof(Shared);
  static_assert(kBytes <= 227 * 1024, "shared memory of a block");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ CUtensorMap q_map, const int q_box,
                        const spec_prefix_attention_args a, const Window w, float* part, float2* stat, int64_t* plan) {
  using S = Smem<D>;
  constexpr int kHalves = D / 64;
  constexpr int kHalfBytes = kTile * 128;  // 64 elements of 128 keys
  // The tiles' swizzle needs 1024 bytes' alignment.  All shared memory is this one
  // array, so it starts where the block's window does.
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared& bars = *reinterpret_cast<Shared*>(smem + S::kShared);
  Item* items = bars.items;
  Layout& lay = bars.lay;
  int64_t* warp_sum = bars.warp_sum;
  volatile int& abort_flag = bars.abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be uniform
  const int per_head = a.Hq / a.Hk;

  // ---- the work layout: every thread a run of segments, one scan
  {
    const int n_seg = a.G + a.R, run = (n_seg + kThreads - 1) / kThreads;
    const int k0 = min(tid * run, n_seg), k1 = min(k0 + run, n_seg);
    uint32_t bad = 0;
    auto cost_of = [&](int k) { return a.Hk * head_cost(segment(a, w, k, &bad), per_head); };
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
    if (warp == kMma) tc::tmem_alloc(&bars.tmem, 512);
    if (warp == kLoader) {
      // arrivals of each barrier, in the order they lie in
      constexpr int kP = 2 * kItemSlots + 20 + 6, kEnd = kP + 7;
      static_assert(offsetof(Shared, p_half) == 8 * kP && offsetof(Shared, drain) == 8 * (kEnd - 1), "order");
      uint64_t* bar = bars.item_full;
      for (int i = lane; i < kEnd; i += 32)
        tc::mbar_init(bar + i, i >= kItemSlots && i < 2 * kItemSlots ? kItemReaders
                               : i >= kP && i < kP + 4               ? 8
                                                                     : 1);
      tc::fence_barrier_init();
    }
    if (warp == kProducer && lane == 0) {
      abort_flag = 0;
      lay = Layout{0, 0, 0, 0, 0};
      tc::tma_prefetch_desc(&k_map);
      tc::tma_prefetch_desc(&v_map);
      if (q_box > 0) tc::tma_prefetch_desc(&q_map);
    }
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
    const int64_t per = max(share_of(total, gridDim.x), (int64_t)max(kCostPair, kCostSingle));
    const int64_t x0 = per * blockIdx.x, x1 = min(x0 + per, total);
    const bool here = x0 < x1 && at <= x0 && x0 < at + mine;
    if (here || blockIdx.x == 0) {
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        const int64_t c = run == 1 ? mine : cost_of(k);
        if (blockIdx.x == 0) plan[1 + k] = at;
        if (here && at <= x0 && x0 < at + c) lay = Layout{per, x0, x1, k, at};
        at += c;
      }
    }
    if (blockIdx.x == 0 && tid == 0) plan[0] = per;
    if (bad && blockIdx.x == 0) set_status(a.status, bad);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  }
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  // A wait of a whole warp: all of its lanes go on, or all give up.
  auto warp_wait = [&](uint64_t* bar, uint32_t phase) {
    bool got = tc::mbar_try_wait(bar, phase & 1u);
    if (!__all_sync(0xffffffffu, got)) {
      got = slow_wait(bar, phase, &abort_flag, a.status);
      got = __all_sync(0xffffffffu, got);
    }
    return got;
  };
  if (warp == kProducer) {
    // ------------------------------------------------------------ producer --
    uint32_t seq = 0;  // ring positions used: keys and values in turn
    uint32_t bad = 0, ph = 0;
    int st = 0;
    bool ok = true;
    const int box = min(a.page_size, kTile), boxes = kTile / box;  // keys of a box, boxes of a tile
    for (uint32_t n_item = 0;; ++n_item) {
      const Item& posted = items[n_item % kItemSlots];
      ok = warp_wait(&bars.item_full[n_item % kItemSlots], n_item / kItemSlots);
      if (!ok || posted.rows == 0) break;
      const Item it = posted;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.item_empty[n_item % kItemSlots]);
      for (int i = it.lo; ok && i < it.hi; ++i) {
        const int live = min(kTile, it.keys - i * kTile);
        const int used = (live + box - 1) / box;  // pages (or parts of one) that have keys
        int row = 0;
        const int which = lane / kHalves;
        if (which < used) {
          const int key = i * kTile + which * box, pi = key / a.page_size;
          row = page_of(a, it.table, pi, &bad) * a.page_size + (key - pi * a.page_size);
        }
        for (int kv = 0; kv < 2; ++kv, ++seq) {
          ok = warp_wait(&bars.empty[st], ph ^ 1u);
          if (!ok) break;
          if (lane == 0) tc::mbar_expect_tx(&bars.full[st], (uint32_t)(used * box * D * 2));
          __syncwarp();
          if (which < used && which < boxes) {
            const int half = lane % kHalves;
            tc::tma_load_3d(smem + S::kRing + st * S::kTileBytes + half * kHalfBytes + which * box * 128,
                            kv ? &v_map : &k_map, &bars.full[st], half * 64, it.h, row);
          }
          if (++st == S::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) break;
    }
    if (bad) set_status(a.status, bad);
    if (!ok) {  // the copies in flight land before the block's memory goes
      const uint32_t from = seq > (uint32_t)S::kStages ? seq - S::kStages : 0u;
      for (uint32_t s = from; s < seq; ++s)
        tc::mbar_wait(&bars.full[s % S::kStages], (s / S::kStages) & 1u, kWaitNs);
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ products --
    {
      const uint32_t lead = elected();
      int rows = 0, tiles = 0, n_rows = 0, n_tiles = 0;  // of the current and the next item
      uint32_t n_item = 0;
      uint32_t q_n[2] = {0, 0}, p_n[2] = {0, 0};
      int turn = 0;  // softmax group of the next small item
      bool ok = true;
      constexpr uint32_t kDescS = tc::bf16_idesc(128, kTile);
      constexpr uint32_t kDescO = tc::bf16_idesc(128, D) | (1u << 16);  // values: keys down, head across
      const uint32_t q_lo = desc_k(tc::smem_u32(smem));
      const uint32_t k_lo = desc_k(tc::smem_u32(smem + S::kRing));
      const uint32_t v_lo = desc_mn(tc::smem_u32(smem + S::kRing), kHalfBytes);
      struct Place {  // a ring position: its stage and the parity of its barriers
        uint32_t stage, phase;
        __device__ __forceinline__ Place next() const {
          return stage + 1 == S::kStages ? Place{0, phase ^ 1u} : Place{stage + 1, phase};
        }
      };
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (ok) ok = warp_wait(bar, phase);
      };
      auto scores = [&](int t, const Place& k, bool last) {  // S_t = Q_t K^T
        const uint32_t kb = k_lo + k.stage * (S::kTileBytes >> 4), qb = q_lo + t * (S::kTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          constexpr uint32_t kStep = 32 >> 4;
          const uint32_t off = (c >> 2) * (kHalfBytes >> 4) + (c & 3) * kStep;
          mma_ss(lead, tmem + t * kTile, qb + off, kb + off, kDescS, c > 0);
        }
        commit_if(lead, &bars.s_full[t]);
        if (last) commit_if(lead, &bars.q_empty[t]);
      };
      // O_t (+)= P_t V, the keys of one half of each thread's weights at a time: keys 0-31
      // and 64-95 of the tile, then the others
      auto values = [&](int t, const Place& v, bool first, int part) {
        const uint32_t vb = v_lo + v.stage * (S::kTileBytes >> 4);
#pragma unroll
        for (int x = 0; x < kTile / 32; ++x) {
          const int c = (x >> 1) * 4 + part * 2 + (x & 1);
          mma_ts(lead, tmem + 2 * kTile + t * kTile, tmem + t * kTile + c * 8, vb + c * (2048 >> 4), kDescO,
                 x > 0 || part > 0 || !first);
        }
      };
      auto begin = [&](int l0, int l1, const Place& k, int tiles) {  // an item's first scores
        wait(&bars.full[k.stage], k.phase);
        for (int t = l0; t <= l1 && ok; ++t) {
          wait(&bars.q_full[t], q_n[t]++);
          if (!ok) break;
          tc::fence_after_sync();
          scores(t, k, tiles == 1);
        }
        if (ok) commit_if(lead, &bars.empty[k.stage]);
      };
      auto next = [&](int& r, int& n) {  // the next item's rows and tiles; false after the last
        const uint32_t slot = n_item % kItemSlots;
        wait(&bars.item_full[slot], n_item / kItemSlots);
        ++n_item;
        if (!ok) return false;
        // (from one lane, so that what follows is uniform)
        r = __shfl_sync(0xffffffffu, items[slot].rows, 0);
        n = __shfl_sync(0xffffffffu, items[slot].hi - items[slot].lo, 0);
        if (r == 0) return false;
        if (lane == 0) tc::mbar_arrive(&bars.item_empty[slot]);
        return true;
      };
      auto lanes = [&](int r, int& p, int& q) {  // the softmax groups of an item
        if (r > kTile) {
          p = 0;
          q = 1;
        } else {
          p = q = turn;
          turn ^= 1;
        }
      };
      int l0 = 0, l1 = 0;
      Place key{0, 0};  // the current tile's keys; its values follow
      bool more = next(rows, tiles);
      if (more) {
        lanes(rows, l0, l1);
        begin(l0, l1, key, tiles);
      }
      while (more && ok) {
        bool more_next = false, early = false;
        int n0 = 0, n1 = 0;
        for (int i = 0; i < tiles && ok; ++i) {
          const bool last = i + 1 == tiles;
          const Place val = key.next(), then = val.next();
          if (last) {
            more_next = next(n_rows, n_tiles);
            if (more_next) {
              lanes(n_rows, n0, n1);
              // ahead of the current item's last values, if all is there: the other
              // group may still be busy with the item before
              early = l0 == l1 && n0 == n1 && n0 != l0 &&
                      __all_sync(0xffffffffu, tc::mbar_try_wait(&bars.q_full[n0], q_n[n0] & 1u) &&
                                                  tc::mbar_try_wait(&bars.full[then.stage], then.phase));
              if (early) begin(n0, n1, then, n_tiles);
            }
          }
          wait(&bars.full[val.stage], val.phase);
          if (!last) wait(&bars.full[then.stage], then.phase);
          for (int t = l0; t <= l1 && ok; ++t) {
            wait(&bars.p_half[t], p_n[t]);
            if (!ok) break;
            tc::fence_after_sync();
            values(t, val, i == 0, 0);
            wait(&bars.p_full[t], p_n[t]++);
            if (!ok) break;
            tc::fence_after_sync();
            values(t, val, i == 0, 1);
            if (last) commit_if(lead, &bars.o_full[t]);
            else scores(t, then, i + 2 == tiles);
          }
          if (!ok) break;
          commit_if(lead, &bars.empty[val.stage]);
          if (!last) commit_if(lead, &bars.empty[then.stage]);
          key = then;
        }
        if (!ok) break;
        more = more_next;
        rows = n_rows;
        tiles = n_tiles;
        l0 = n0;
        l1 = n1;
        if (more && !early) begin(l0, l1, key, tiles);
      }
      if (!ok) {  // the products in flight end before TMEM is freed
        commit_if(lead, &bars.drain);
        tc::mbar_wait(&bars.drain, 0, kWaitNs);
      }
    }
    __syncwarp();
  } else if (warp == kPlanner) {
    // ------------------------------------------------------------- planner --
    Walker walk(a, w, lay);
    Item it;
    for (uint32_t n_item = 0;; ++n_item) {
      if (!walk.next(it)) it.rows = 0;  // the end
      const uint32_t slot = n_item % kItemSlots;
      if (!warp_wait(&bars.item_empty[slot], (n_item / kItemSlots) ^ 1u)) break;
      if (lane == 0) {
        items[slot] = it;
        tc::mbar_arrive(&bars.item_full[slot]);
      }
      if (it.rows == 0) break;
    }
  } else if (warp == kLoader) {
    // -------------------------------------------------------------- loader --
    uint32_t n[2] = {0, 0};  // query tiles taken
    int turn = 0;
    bool ok = true;
    for (uint32_t n_item = 0; ok; ++n_item) {
      const Item& posted = items[n_item % kItemSlots];
      ok = warp_wait(&bars.item_full[n_item % kItemSlots], n_item / kItemSlots);
      if (!ok || posted.rows == 0) break;
      const int row0 = posted.row0, m0 = posted.m0, rows = posted.rows, h = posted.h;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.item_empty[n_item % kItemSlots]);
      const bool both = rows > kTile;
      const int t0 = both ? 0 : turn, t1 = both ? 1 : turn;
      if (!both) turn ^= 1;
      for (int t = t0; ok && t <= t1; ++t) {
        ok = warp_wait(&bars.q_empty[t], n[t] ^ 1u);
        if (!ok) break;
        ++n[t];
        // rows past the item's keep what was there: their results are not read
        const int first = both ? t * kTile : 0, live = min(kTile, rows - first);
        if (q_box > 0) {  // boxes of q_box query rows: whole packed rows of one key head
          const int boxes = (live + q_box - 1) / q_box;
          if (lane == 0) tc::mbar_expect_tx(&bars.q_full[t], (uint32_t)(boxes * q_box * D * 2));
          __syncwarp();
          const int half = lane % kHalves, x = lane / kHalves;
          if (x < boxes)
            tc::tma_load_3d(smem + t * S::kTileBytes + half * kHalfBytes + x * q_box * 128, &q_map,
                            &bars.q_full[t], half * 64, h * per_head, row0 + (m0 + first + x * q_box) / per_head);
          continue;
        }
        const uint32_t to = tc::smem_u32(smem) + t * S::kTileBytes;
        constexpr int kChunks = D / 8;  // 16-byte pieces of a row
        const int c = lane % kChunks;
        for (int r = lane / kChunks; r < live; r += 32 / kChunks) {
          const int qrow = m0 + first + r, j = qrow / per_head;
          const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + (size_t)(row0 + j) * a.q_row +
                                   (size_t)(h * per_head + (qrow - j * per_head)) * a.q_head + c * 8;
          copy16(to + r * 128 + (c >> 3) * kHalfBytes + (((c & 7) ^ (r & 7)) << 4), q);
        }
      }
      if (q_box > 0) continue;
      copies_wait();
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0 && ok)
        for (int t = t0; t <= t1; ++t) tc::mbar_arrive(&bars.q_full[t]);
    }
    if (abort_flag && q_box > 0)
      for (int t = 0; t < 2; ++t)
        if (n[t] > 0) tc::mbar_wait(&bars.q_full[t], (n[t] - 1u) & 1u, kWaitNs);
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax --
    constexpr int kCols = kTile / 2, kDims = D / 2;  // scores and result columns of a thread
    const int t = warp >> 3, half = lane >> 4;
    const int row16 = (warp & 3) * 32 + (warp >> 2 & 1) * 16, in_t = row16 + (lane & 15);
    const uint32_t lane_base = (uint32_t)row16 << 16;  // TMEM lanes in the high half
    const uint32_t s_addr = tmem + lane_base + t * kTile, o_addr = s_addr + 2 * kTile;
    const float sl = a.scale * kLog2e;
    const bool wide_out = ((uintptr_t)a.out & 15) == 0 && a.out_row % 8 == 0 && a.out_head % 8 == 0;
    uint32_t seq = 0, n_item = 0, s_n = 0, o_n = 0;  // ring position, items seen, waits done
    int turn = 0;
    bool ok = true;
    auto other = [](float v) { return __shfl_xor_sync(0xffffffffu, v, 16); };  // the row's other thread's
    // This softmax group's next item and its ring position.
    auto next = [&](Item& it, uint32_t& seq0) {
      while (true) {
        const Item& posted = items[n_item % kItemSlots];
        ok = warp_wait(&bars.item_full[n_item % kItemSlots], n_item / kItemSlots);
        if (!ok || posted.rows == 0) return false;
        it = posted;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.item_empty[n_item % kItemSlots]);
        ++n_item;
        const bool pair_item = it.rows > kTile;
        const int mine = pair_item ? t : turn;
        if (!pair_item) turn ^= 1;
        seq0 = seq;
        seq += 2u * (uint32_t)(it.hi - it.lo);
        if (mine == t) return true;
      }
    };
    Item it;
    uint32_t seq0 = 0;
    bool more = next(it, seq0);
    while (more) {
      const bool pair_item = it.rows > kTile;
      const int m = (pair_item ? t * kTile : 0) + in_t;
      const bool valid = m < it.rows;
      const int qrow = it.m0 + m, j = qrow / per_head;
      const int limit = it.prefix ? it.keys : min(it.keys, it.first_own + j);  // keys of this row
      float ref = -CUDART_INF_F, l = 0.f;
      for (int i = it.lo; i < it.hi; ++i) {
        ok = warp_wait(&bars.s_full[t], s_n++);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t s[kCols];
        tmem_ld64h<kCols>(s_addr, s);
        tc::tmem_ld_wait();
        const int lim = limit - i * kTile - half * kCols;
        if (__any_sync(0xffffffffu, lim < kCols)) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c >= lim) s[c] = 0xff800000u;  // -inf
        }
        float m0 = -CUDART_INF_F, m1 = m0, m2 = m0, m3 = m0;
#pragma unroll
        for (int e = 0; e < kCols; e += 8) {
          m0 = max3(m0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          m1 = max3(m1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          m2 = max3(m2, __uint_as_float(s[e + 4]), __uint_as_float(s[e + 5]));
          m3 = max3(m3, __uint_as_float(s[e + 6]), __uint_as_float(s[e + 7]));
        }
        float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sl;
        top = fmaxf(top, other(top));
        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
          // each row by its own scores alone: its bits do not depend on its neighbours
          const float to = top > ref + kSlack ? top : ref;
          const float c = to == ref ? 1.f : tc::ex2(ref - to);  // 0 from -inf
          ref = to;
          l *= c;
          if (i > it.lo) {
#pragma unroll 1
            for (int d = 0; d < kDims; d += 16) {
              uint32_t o[16];
              tmem_ld16h<kDims>(o_addr + d, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
              tmem_st16h<kDims>(o_addr + d, o);
            }
          }
        }
        const float sub = ref == -CUDART_INF_F ? 0.f : ref;
        const uint64_t sl2 = pair(sl, sl), sub2 = pair(-sub, -sub);
        // Values past the item's keys may be anything, NaN among them: zeros instead.
        // (The first softmax group of two does it, whose product is issued first.)
        const int live = it.keys - i * kTile;
        if (live < kTile && (!pair_item || t == 0)) {
          const uint32_t sv = seq0 + 2u * (uint32_t)(i - it.lo) + 1u;
          ok = warp_wait(&bars.full[sv % S::kStages], sv / S::kStages);
          if (!ok) break;
          if (in_t >= live) {
            uint8_t* to = smem + S::kRing + (sv % S::kStages) * S::kTileBytes + in_t * 128;
#pragma unroll 1
            for (int c = half; c < D / 8; c += 2)
              *reinterpret_cast<uint4*>(to + (c >> 3) * kHalfBytes + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async();
        }
        // The first half of the weights goes to the products while the second is
        // computed: over the scores, which the warp has read.
        uint64_t a0 = 0, a1 = 0;
        uint32_t p[kCols / 2];
        auto weights = [&](int from, int to) {
#pragma unroll
          for (int e = from; e < to; e += 4) {
            const float2 z0 = halves(fma2(pair(s[e], s[e + 1]), sl2, sub2));
            const float2 z1 = halves(fma2(pair(s[e + 2], s[e + 3]), sl2, sub2));
            const float p0 = tc::ex2(z0.x), p1 = tc::ex2(z0.y), p2 = tc::ex2(z1.x), p3 = tc::ex2(z1.y);
            a0 = add2(a0, pair(p0, p1));
            a1 = add2(a1, pair(p2, p3));
            p[e / 2] = pack_bf16(p0, p1);
            p[e / 2 + 1] = pack_bf16(p2, p3);
          }
        };
        weights(0, kCols / 2);
        tmem_st16h<kCols / 2>(s_addr, p);
        weights(kCols / 2, kCols * 3 / 4);
        tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.p_half[t]);
        weights(kCols * 3 / 4, kCols);
        tmem_st16h<kCols / 2>(s_addr + kCols / 4, p + kCols / 4);
        const float2 sum = halves(add2(a0, a1));
        l += sum.x + sum.y;
        tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.p_full[t]);
      }
      if (!ok) break;
      const size_t slot = it.slot + m;
      const bool direct = it.direct;
      const int row = it.row0 + j, hq = it.h * per_head + (qrow - j * per_head);
      ok = warp_wait(&bars.o_full[t], o_n++);
      if (!ok) break;
      tc::fence_after_sync();
      l += other(l);
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row without keys: zeros
#pragma unroll 1
      for (int d = 0; d < kDims; d += 32) {
        uint32_t o[32];
        tmem_ld32h<kDims>(o_addr + d, o);
        tc::tmem_ld_wait();
        if (!valid) continue;
        if (!direct) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) store32(part + slot * D + half * kDims + d + e, o + e);
          continue;
        }
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          p[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        __nv_bfloat16* out =
            (__nv_bfloat16*)a.out + (size_t)row * a.out_row + (size_t)hq * a.out_head + half * kDims + d;
        if (wide_out) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(out + 2 * e) = make_uint4(p[e], p[e + 1], p[e + 2], p[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) *reinterpret_cast<uint32_t*>(out + 2 * e) = p[e];
        }
      }
      tc::fence_before_sync();
      if (valid && half == 0) {
        if (!direct) stat[slot] = make_float2(ref, l);
        else if (a.lse) a.lse[(size_t)row * a.Hq + hq] = l == 0.f ? -CUDART_INF_F : (ref + log2f(l)) * kLn2;
      }
      more = next(it, seq0);
    }
  }
  tc::grid_dep_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMma) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------- join ----
constexpr int kJoinThreads = 128;
constexpr int kJoinBlocks = 152 * 16;
constexpr int kJoinRows = 64;  // query rows (packed rows x heads of a key head) of a block at a time

constexpr int kJoinLanes = 16;  // threads of a row

// Cost of a head's items before item `upto`, and of all of them; a row's threads add them up.
__device__ __forceinline__ void costs_of(const Segment& s, int per_head, int upto, int64_t* before, int64_t* all) {
  const int n = item_count(s, per_head), lane = threadIdx.x % kJoinLanes;
  const uint32_t lanes = (uint32_t)((1ull << kJoinLanes) - 1) << (threadIdx.x & 31 & ~(kJoinLanes - 1));
  int64_t x = 0, y = 0;
  for (int i = lane; i < n; i += kJoinLanes) {
    const int64_t c = item_cost(item_keys(s, i, per_head), s.n * per_head - i * kItemRows);
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
template <int D>
__device__ __forceinline__ void join_request(const spec_prefix_attention_args& a, const Window& w, int r,
                                             const float* part, const float2* stat, const int64_t* plan) {
  constexpr int kPer = D / kJoinLanes, kBatch = 4;
  const int lane = threadIdx.x % kJoinLanes, per_head = a.Hq / a.Hk;
  uint32_t bad = 0;
  const Segment own = segment(a, w, a.G + r, &bad);
  int g = group_of(a, r, &bad);
  Segment pre{0, 0, 0, 0, nullptr, true};
  if (g >= 0) pre = segment(a, w, g, &bad);
  if (own.row0 < pre.row0 || own.row0 + own.n > pre.row0 + pre.n) g = -1;  // rows out of order
  const int m_own = own.n * per_head;
  const int m_off = (own.row0 - pre.row0) * per_head;  // the request's first row among the group's
  tc::grid_dep_wait();  // all of the above is the caller's; the pieces and their layout are ready now
  const int64_t per = plan[0];
  const int64_t own_at = plan[1 + a.G + r], pre_at = g >= 0 ? plan[1 + g] : 0;

  const int tiles = (m_own + kJoinRows - 1) / kJoinRows, all_tiles = tiles * a.Hk;
  int item[2] = {-1, -1}, head = -1;  // own and prefix item, and key head, whose pieces are known
  int64_t before[2] = {0, 0}, all[2] = {0, 0};
  int first[2] = {0, 0}, count[2] = {0, 0};
  auto pieces = [&](int k, const Segment& s, int64_t at, int h, int i) {  // blocks that have pieces of item i
    if (i == item[k] && h == head) return;
    const int tiles = (item_keys(s, i, per_head) + kTile - 1) / kTile;
    count[k] = 0;
    if (i != item[k]) costs_of(s, per_head, i, &before[k], &all[k]);
    item[k] = i;
    if (tiles == 0) return;
    const int rows = s.n * per_head - i * kItemRows;
    at += h * all[k] + before[k] + start_cost(rows);
    first[k] = (int)(at / per);
    count[k] = (int)((at + (int64_t)(tiles - 1) * tile_cost(rows)) / per) - first[k] + 1;
  };

  const bool wide_out = ((uintptr_t)a.out & 7) == 0 && a.out_row % 4 == 0 && a.out_head % 4 == 0;

#pragma unroll 1
  for (int x = blockIdx.y; x < all_tiles; x += gridDim.y) {
    const int h = x / tiles, m0 = (x - h * tiles) * kJoinRows;
    const size_t own_slot = ((size_t)(w.hi - w.lo) + (own.row0 - w.lo)) * a.Hq + (size_t)h * m_own;
    const size_t pre_slot = (size_t)(pre.row0 - w.lo) * a.Hq + (size_t)h * pre.n * per_head + m_off;
    for (int m = m0 + threadIdx.x / kJoinLanes; m < min(m0 + kJoinRows, m_own); m += kJoinThreads / kJoinLanes) {
      pieces(0, own, own_at, h, m / kItemRows);
      if (g >= 0) pieces(1, pre, pre_at, h, (m_off + m) / kItemRows);
      head = h;
      const int c0 = count[0], n = c0 + count[1];
      if (count[1] == 0 && n == 1) continue;  // written by its block
      // piece p lies at one of two places plus p steps of 256 rows
      const size_t own_at_row = own_slot + m + (size_t)kItemRows * first[0];
      const size_t pre_at_row = pre_slot + m + (size_t)kItemRows * first[1] - (size_t)kItemRows * c0;
      const float* own_part = part + own_at_row * D + lane * kPer;
      const float* pre_part = part + (ptrdiff_t)pre_at_row * D + lane * kPer;
      float top = -CUDART_INF_F, sum = 0.f, o[kPer];
#pragma unroll
      for (int d = 0; d < kPer; ++d) o[d] = 0.f;
#pragma unroll 1
      for (int p0 = 0; p0 < n; p0 += kBatch) {
        float2 st[kBatch];
        float v[kBatch][kPer];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int p = p0 + i;
          st[i] = make_float2(-CUDART_INF_F, 0.f);
          if (p < n) {
            st[i] = stat[(p < c0 ? own_at_row : pre_at_row) + (size_t)(p * kItemRows)];
            const float* src = (p < c0 ? own_part : pre_part) + (size_t)p * (kItemRows * D);
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
template <int D, bool kPart>
__global__ void __launch_bounds__(kJoinThreads, 4)
    join_tc_kernel(const spec_prefix_attention_args a, const Window w, const float* part, const float2* stat,
                   const int64_t* plan) {
  int r = blockIdx.x;
  if (!kPart) {
    join_request<D>(a, w, r, part, stat, plan);
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
  for (r += first_s; r <= last_s; r += gridDim.x) join_request<D>(a, w, r, part, stat, plan);
  tc::grid_dep_wait();  // a block without requests, too, ends after the pieces' kernel
}

template <int D>
cudaError_t launch(const spec_prefix_attention_args& a, int sms, float* part, float2* stat, int64_t* plan,
                   cudaStream_t stream) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hk, (uint64_t)a.n_pages * a.page_size};
  const uint32_t box[3] = {64, 1, (uint32_t)(a.page_size < kTile ? a.page_size : kTile)};
  CUtensorMap km, vm;
  if (!fused::encode_tiled(&km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.k_cache, 3, dims, box) ||
      !fused::encode_tiled(&vm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.v_cache, 3, dims, box))
    return cudaErrorInvalidValue;
  // query boxes of 32 rows (a small item loads few), or of one packed row's heads
  const int per_head = a.Hq / a.Hk;
  int q_box = per_head > 32 ? per_head : 32;
  CUtensorMap qm = km;
  {
    const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.rows};
    const uint64_t qstrides[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_row * 2};
    const uint32_t qbox[3] = {64, (uint32_t)per_head, (uint32_t)(q_box / per_head)};
    if (kTile % per_head != 0 || q_box % per_head != 0 || a.q_head < D || a.q_row < D ||
        !fused::encode_tiled_strided(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qdims, qstrides, qbox))
      q_box = 0;
  }
  cudaError_t err = cudaFuncSetAttribute(attention_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<D>::kBytes);
  if (err != cudaSuccess) return err;
  // windows of equal size
  const int most_rows = attn_window_rows(a.Hq), windows = (int)(((int64_t)a.rows + most_rows - 1) / most_rows);
  const int step = (int)(((int64_t)a.rows + windows - 1) / windows);
  // a block of the join a tile of the mean request, until there are kJoinBlocks of them
  const int64_t tiles = (((int64_t)a.rows * per_head + (int64_t)kJoinRows * a.R - 1) / ((int64_t)kJoinRows * a.R)) * a.Hk;
  const int at_once = std::min(a.R, (a.R + windows - 1) / windows + (windows > 1));  // requests of a window
  const int64_t most = (kJoinBlocks + at_once - 1) / at_once;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(at_once, (unsigned)(tiles < most ? tiles : most));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (int64_t lo = 0; lo < a.rows; lo += step) {
    const Window w{(int)lo, (int)std::min<int64_t>(lo + step, a.rows)};
    attention_tc_kernel<D><<<sms, kThreads, Smem<D>::kBytes, stream>>>(km, vm, qm, q_box, a, w, part, stat, plan);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    err = cudaLaunchKernelEx(&cfg, windows > 1 ? join_tc_kernel<D, true> : join_tc_kernel<D, false>, a, w,
                             (const float*)part, (const float2*)stat, (const int64_t*)plan);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace

// bf16 heads of 64 or 128, pages that tile 128 keys in boxes of 8 rows or more,
// 16-byte rows, an sm_100-family GPU.
bool attn_tc_ok(const spec_prefix_attention_args& a, int* sms) {
  if (a.dtype != SPEC_BF16 || (a.D != 64 && a.D != 128)) return false;
  const int P = a.page_size;
  if (P < 128 ? (P < 8 || 128 % P != 0) : P % 128 != 0) return false;
  auto on = [](const void* p, size_t n) { return ((uintptr_t)p % n) == 0; };
  if (!on(a.q, 16) || a.q_row % 8 != 0 || a.q_head % 8 != 0 || !on(a.k_cache, 16) || !on(a.v_cache, 16) ||
      !on(a.out, 4) || a.out_row % 2 != 0 || a.out_head % 2 != 0)
    return false;
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  return major == 10 && *sms >= 1 && *sms <= kMaxCtas;
}

cudaError_t launch_attention_tc(const spec_prefix_attention_args& a, int sms, float* part, float2* stat,
                                int64_t* plan, cudaStream_t stream) {
  return a.D == 128 ? launch<128>(a, sms, part, stat, plan, stream)
                    : launch<64>(a, sms, part, stat, plan, stream);
}

}  // namespace spec
