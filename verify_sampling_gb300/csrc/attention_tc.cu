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
#include <type_traits>

#include "attention_packed.cuh"
#include "attention_plan.cuh"
#include "fused_tc.cuh"
#include "tc.cuh"

namespace spec {

namespace {

using namespace attn;
using tc::add2;
using tc::fma2;
using tc::halves;
using tc::pair;

// (kTile: keys of a tile, and rows of a softmax group)
// Softmax warps: group t (rows 128 t ..) is warps 8 t .. 8 t + 7; warps w and w + 4 of it
// share 32 rows (TMEM lanes go by the warp's number mod 4), 16 each, and a row has
// threads i and i + 16 of its warp, each half of its columns.
constexpr int kSoftWarps = 16, kProducer = 16, kMma = 17, kPlanner = 18, kLoader = 19, kUnpack = 20;
constexpr int kItemSlots = 4;
constexpr int kUnpackWarps = 8;  // a packed cache's: half of a key's groups each thread
template <bool kPacked>
struct Roles {
  static constexpr int kThreads = 640 + (kPacked ? 32 * kUnpackWarps : 0);
  // producer, MMA, loader, softmax and unpacking warps
  static constexpr int kItemReaders = 3 + kSoftWarps + (kPacked ? kUnpackWarps : 0);
};
constexpr float kSlack = 8.f;  // log2 units the maximum may grow by before O is rescaled


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
// Everything shared beside the tiles.
struct Shared {
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], drain;
  uint64_t packed_full[6], packed_empty[6];
  Item items[kItemSlots];
  Layout lay;
  int64_t warp_sum[Roles<true>::kThreads / 32];
  uint32_t tmem;
  volatile int abort_flag;
};

template <int D, bool kPacked>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = (kPacked ? 4 : 5) * (128 / D);
  static constexpr int kRing = 2 * kTileBytes;  // after the two query tiles
  // a packed cache's tiles: data and scales of 128 keys or values
  static constexpr int kGroups = D / q4::kGroup, kPackedData = kTile * D / 2, kPackedBytes = kPackedData + kTile * kGroups;
  static constexpr int kPackedStages = kPacked ? (D == 128 ? 3 : 6) : 0;
  static constexpr int kPackedRing = kRing + kStages * kTileBytes;
  static constexpr int kShared = kPackedRing + kPackedStages * kPackedBytes;
  static constexpr int kBytes = kShared + (int)sizeof(Shared);
  static_assert(kBytes <= 227 * 1024, "shared memory of a block");
};

template <int D, bool kPacked>
__global__ void __launch_bounds__(Roles<kPacked>::kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ CUtensorMap q_map, const int q_box, const q4::Cache packed,
                        const spec_prefix_attention_args a, const Window w, float* part, float2* stat, int64_t* plan) {
  using S = Smem<D, kPacked>;
  using R = Roles<kPacked>;
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

  lay_out<WideCosts<kPacked>, R::kThreads>(a, w, &lay, warp_sum, plan, [&] {
    if (warp == kMma) tc::tmem_alloc(&bars.tmem, 512);
    if (warp == kLoader) {
      // arrivals of each barrier, in the order they lie in
      constexpr int kP = 2 * kItemSlots + 20 + 6, kEnd = kP + 7 + (kPacked ? 12 : 0);
      static_assert(offsetof(Shared, full) == 16 * kItemSlots && offsetof(Shared, p_half) == 8 * kP &&
                        offsetof(Shared, packed_empty) == 8 * (kP + 13),
                    "order");
      uint64_t* bar = bars.item_full;
      for (int i = lane; i < kEnd; i += 32)
        tc::mbar_init(bar + i, i >= kItemSlots && i < 2 * kItemSlots                  ? R::kItemReaders
                               : i >= kP && i < kP + 4                                ? 8
                               : kPacked && i >= 2 * kItemSlots && i < 2 * kItemSlots + 10 ? kUnpackWarps
                               : kPacked && i >= kP + 13                              ? kUnpackWarps
                                                                                      : 1);
      tc::fence_barrier_init();
    }
    if (warp == kProducer && lane == 0) {
      abort_flag = 0;
      if (!kPacked) {
        tc::tma_prefetch_desc(&k_map);
        tc::tma_prefetch_desc(&v_map);
      }
      if (q_box > 0) tc::tma_prefetch_desc(&q_map);
    }
  });
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  // A wait of a whole warp: all of its lanes go on, or all give up.
  auto warp_wait = [&](uint64_t* bar, uint32_t phase) {
    bool got = tc::mbar_try_wait(bar, phase & 1u);
    if (!__all_sync(0xffffffffu, got)) {
      // (a kernel that calls a function cannot move registers)
      got = kPacked ? slow_wait_here(bar, phase, &abort_flag, a.status) : slow_wait(bar, phase, &abort_flag, a.status);
      got = __all_sync(0xffffffffu, got);
    }
    return got;
  };
  auto producer = [&] {
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
      if (kPacked) {  // pages' heads and their scales, by bulk copies
        constexpr int G = S::kGroups;
        const int pieces = a.page_size > kTile ? G : 1;  // copies of a page's data within a tile
        for (int i = it.lo; ok && i < it.hi; ++i) {
          const int live = min(kTile, it.keys - i * kTile);
          const int used = (live + box - 1) / box, copies = used * (pieces + 1);
          const int x = lane / (pieces + 1), piece = lane - x * (pieces + 1);
          int page = 0, tok = 0;
          if (lane < copies) {
            const int key = i * kTile + x * box, pi = key / a.page_size;
            page = page_of(a, it.table, pi, &bad);
            tok = key - pi * a.page_size;
          }
          for (int kv = 0; kv < 2; ++kv, ++seq) {
            ok = warp_wait(&bars.packed_empty[st], ph ^ 1u);
            if (!ok) break;
            if (lane == 0) tc::mbar_expect_tx(&bars.packed_full[st], (uint32_t)(used * box * (D / 2 + G)));
            __syncwarp();
            if (lane < copies) {
              uint8_t* to = smem + S::kPackedRing + st * S::kPackedBytes;
              if (piece < pieces)
                tc::bulk_load(to + (x * G + piece) * box * 16,
                              (kv ? packed.v : packed.k) + q4::data_at(page, it.h, tok, a.Hk, G, a.page_size) +
                                  (int64_t)piece * 16 * a.page_size,
                              (uint32_t)(box * 16 * (G / pieces)), &bars.packed_full[st]);
              else
                tc::bulk_load(to + S::kPackedData + x * box * G,
                              (kv ? packed.v_scale : packed.k_scale) + q4::scale_at(page, it.h, tok, a.Hk, G, a.page_size),
                              (uint32_t)(box * G), &bars.packed_full[st]);
            }
            if (++st == S::kPackedStages) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
      } else {
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
      }
      if (!ok) break;
    }
    if (bad) set_status(a.status, bad);
    if (!ok) {  // the copies in flight land before the block's memory goes
      constexpr uint32_t kLoaded = kPacked ? S::kPackedStages : S::kStages;
      uint64_t* loaded = kPacked ? bars.packed_full : bars.full;
      const uint32_t from = seq > kLoaded ? seq - kLoaded : 0u;
      for (uint32_t s = from; s < seq; ++s) tc::mbar_wait(&loaded[s % kLoaded], (s / kLoaded) & 1u, kWaitNs);
    }
  };
  auto products = [&] {
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
  };
  auto planner = [&] {
    // ------------------------------------------------------------- planner --
    Walker<WideCosts<kPacked>> walk(a, w, lay);
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
  };
  auto loader = [&] {
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
  };
  auto unpack = [&] {
    // -------------------------------------------------------------- unpack --
    // Half of a key's (or value's) groups from the packed ring to their row of the operand tile, a thread.
    constexpr int G = S::kGroups, kMine = G / 2;
    const int at = (warp - kUnpack) * 32 + lane, key = at % kTile, c0 = at / kTile * kMine;
    const int box = min(a.page_size, kTile), page = key / box;
    const uint8_t* from = smem + S::kPackedRing + (page * G + c0) * box * 16 + (key - page * box) * 16;
    uint8_t* to = smem + S::kRing + key * 128;
    const uint32_t turn = (key & 7) << 4;
    uint32_t st = 0, ph = 0, pst = 0, pph = 0;
    bool ok = true;
    for (uint32_t n_item = 0; ok; ++n_item) {
      const Item& posted = items[n_item % kItemSlots];
      ok = warp_wait(&bars.item_full[n_item % kItemSlots], n_item / kItemSlots);
      if (!ok || posted.rows == 0) break;
      const int tiles = 2 * (posted.hi - posted.lo);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.item_empty[n_item % kItemSlots]);
      for (int i = 0; i < tiles; ++i) {
        ok = warp_wait(&bars.packed_full[pst], pph) && warp_wait(&bars.empty[st], ph ^ 1u);
        if (!ok) break;
        const uint8_t* src = from + pst * S::kPackedBytes;
        const uint8_t* sp = smem + S::kPackedRing + pst * S::kPackedBytes + S::kPackedData + key * G + c0;
        const uint32_t scales = G == 4 ? *reinterpret_cast<const uint16_t*>(sp) : *sp;
        uint4 v[kMine];
#pragma unroll
        for (int c = 0; c < kMine; ++c) v[c] = tc::lds128(src + c * box * 16);
        uint8_t* dst = to + st * S::kTileBytes;
        auto words = [&](auto is_key) {
#pragma unroll
          for (int c = 0; c < kMine; ++c) {
            const q4::Scale z = q4::scale_pair(__byte_perm(scales, 0, 0x4040 | c * 0x0101));
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t p0 = q4::element_pair<0>(w[x], z), p1 = q4::element_pair<1>(w[x], z);
              const uint32_t p2 = q4::element_pair<2>(w[x], z), p3 = q4::element_pair<3>(w[x], z);
              // keys in the queries' order; values' columns as they come (8 elements e lie at
              // 2 (e mod 4) + e / 4), for which the results' columns are put in order
              const uint4 o = decltype(is_key)::value
                                  ? make_uint4(__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410), __byte_perm(p0, p1, 0x7632),
                                               __byte_perm(p2, p3, 0x7632))
                                  : make_uint4(p0, p1, p2, p3);
              const int chunk = (c0 + c) * 4 + x;
              *reinterpret_cast<uint4*>(dst + (chunk >> 3) * kHalfBytes + (((chunk & 7) << 4) ^ turn)) = o;
            }
          }
        };
        if (i % 2 == 0) words(std::true_type{});
        else words(std::false_type{});
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&bars.full[st]);
          tc::mbar_arrive(&bars.packed_empty[pst]);
        }
        if (++st == S::kStages) {
          st = 0;
          ph ^= 1u;
        }
        if (++pst == S::kPackedStages) {
          pst = 0;
          pph ^= 1u;
        }
      }
    }
  };
  auto softmax = [&] {
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
        if (kPacked) {  // (one load of 64 asks for more registers than the block starts with)
          tmem_ld32h<kCols>(s_addr, s);
          tmem_ld32h<kCols>(s_addr + 32, s + 32);
        } else {
          tmem_ld64h<kCols>(s_addr, s);
        }
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
        // A packed cache's elements are numbers, whatever its bytes.
        if (!kPacked && live < kTile && (!pair_item || t == 0)) {
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
        if (kPacked) {  // the values' columns in order
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const uint32_t x1 = o[e + 1], x2 = o[e + 2], x3 = o[e + 3], x4 = o[e + 4], x5 = o[e + 5], x6 = o[e + 6];
            o[e + 4] = x1, o[e + 1] = x2, o[e + 5] = x3, o[e + 2] = x4, o[e + 6] = x5, o[e + 3] = x6;
          }
        }
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
  };

  if (kPacked) {
    // Softmax threads need more registers than an 896th of the file: the other three warpgroups
    // give theirs, 512 x 96 + 384 x 40 of the 896 x 72 that the block starts with.
    if (warp >= kSoftWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
      if (warp == kProducer) producer();
      else if (warp == kMma) products();
      else if (warp == kPlanner) planner();
      else if (warp == kLoader) loader();
      else unpack();
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
      softmax();
    }
  } else {  // (in this order: with the softmax warps' branch first the round of 256 requests took 816 us for 795)
    if (warp == kProducer) producer();
    else if (warp == kMma) products();
    else if (warp == kPlanner) planner();
    else if (warp == kLoader) loader();
    else softmax();
  }
  tc::grid_dep_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMma) tc::tmem_dealloc(tmem, 512);
}

// The map of the query rows; *q_box: query rows of a box, of 32 rows (a small item loads few) or of one packed
// row's heads; 0: none.
CUtensorMap query_map(const spec_prefix_attention_args& a, int* q_box) {
  const int per_head = a.Hq / a.Hk;
  CUtensorMap qm{};
  *q_box = per_head > 32 ? per_head : 32;
  const uint64_t qdims[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.rows};
  const uint64_t qstrides[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_row * 2};
  const uint32_t qbox[3] = {64, (uint32_t)per_head, (uint32_t)(*q_box / per_head)};
  if (kTile % per_head != 0 || *q_box % per_head != 0 || a.q_head < a.D || a.q_row < a.D ||
      !fused::encode_tiled_strided(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qdims, qstrides, qbox))
    *q_box = 0;
  return qm;
}

template <int D>
cudaError_t launch(const spec_prefix_attention_args& a, int sms, float* part, float2* stat, int64_t* plan,
                   cudaStream_t stream) {
  using S = Smem<D, false>;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hk, (uint64_t)a.n_pages * a.page_size};
  const uint32_t box[3] = {64, 1, (uint32_t)(a.page_size < kTile ? a.page_size : kTile)};
  CUtensorMap km, vm;
  if (!fused::encode_tiled(&km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.k_cache, 3, dims, box) ||
      !fused::encode_tiled(&vm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.v_cache, 3, dims, box))
    return cudaErrorInvalidValue;
  int q_box;
  const CUtensorMap qm = query_map(a, &q_box);
  auto kernel = attention_tc_kernel<D, false>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (err != cudaSuccess) return err;
  // windows of equal size
  const int most_rows = attn_window_rows(a.Hq), windows = (int)(((int64_t)a.rows + most_rows - 1) / most_rows);
  const int step = (int)(((int64_t)a.rows + windows - 1) / windows);
  for (int64_t lo = 0; lo < a.rows; lo += step) {
    const Window w{(int)lo, (int)std::min<int64_t>(lo + step, a.rows), 0};
    kernel<<<sms, Roles<false>::kThreads, S::kBytes, stream>>>(km, vm, qm, q_box, q4::Cache{}, a, w, part, stat, plan);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    const Pieces pieces{part, stat, plan};
    err = launch_join<D, WideCosts<false>, WideCosts<false>>(a, w, windows, pieces, pieces, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t launch_packed(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, const Window& w, const PackedWork& work,
                          cudaStream_t stream) {
  using S = Smem<D, true>;
  int q_box;
  const CUtensorMap qm = query_map(a, &q_box);
  auto kernel = attention_tc_kernel<D, true>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (err != cudaSuccess) return err;
  kernel<<<sms, Roles<true>::kThreads, S::kBytes, stream>>>(qm, qm, qm, q_box, packed, a, w, work.part, work.stat, work.plan);
  return cudaGetLastError();
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

cudaError_t launch_attention_wide(const spec_prefix_attention_args& a, const q4::Cache& packed, int sms, int lo, int hi, int narrow,
                                  const PackedWork& work, cudaStream_t stream) {
  const Window w{lo, hi, narrow};
  return a.D == 128 ? launch_packed<128>(a, packed, sms, w, work, stream) : launch_packed<64>(a, packed, sms, w, work, stream);
}

}  // namespace spec
