// Paged-cache bookkeeping of a round: the rows' positions, requests and slots
// from the requests' lengths, pages taken from the ring of free ones, and pages
// given back after the verification.
//
// Mathematics: an exclusive scan over the requests of the pages each needs (or
// gives back); everything else is one division per row.
//
// Layout: no block waits for another.  Every block scans the lengths of all
// requests itself (8 bytes a request, from L2 after the first block) and keeps
// the part it needs: reserve the requests whose rows meet its kChunk packed rows,
// commit the kOwn requests whose pages it returns (and a look at the ids of those before).  One launch each, where a
// scan kernel followed by a map kernel would be two.  Rows are dealt out, not
// requests, so one prompt of thousands of tokens spreads over the GPU like
// thousands of requests of one token.
#include "cache_tables.cuh"

#include <algorithm>
#include <climits>

namespace spec {

namespace {

constexpr int kChunk = 1024;  // packed rows of a reserve block
constexpr int kOwn = 128;     // requests of a commit block

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b > 0); }

// Exclusive prefix of `v` over the block; `total` is the block's sum.
template <int kThreads>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long* warp_sum,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();  // the previous round's readers of warp_sum are done
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long sum = lane < kThreads / 32 ? warp_sum[lane] : 0ull;  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  const unsigned long long all = __shfl_sync(0xffffffffu, sum, 31);
  const unsigned long long upto = __shfl_sync(0xffffffffu, sum, warp > 0 ? warp - 1 : 0);
  const unsigned long long before = warp > 0 ? upto : 0ull;
  *total = all;
  return before + inc - v;
}

// One request that has rows in the block's chunk.
struct Entry {
  int r, row0, n, kv, have, base;
  unsigned off;  // its first page's place in the ring, counted from the head
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads) reserve_kernel(spec_cache_reserve_args a) {
  __shared__ Entry list[kChunk];
  __shared__ unsigned long long warp_sum[kThreads / 32];
  __shared__ unsigned taken_s;
  const int tid = threadIdx.x, P = a.page_size;
  // (no sum of these passes a.rows, which may be any int)
  const int b0 = blockIdx.x * kChunk, n_rows = min(kChunk, a.rows - b0), b1 = b0 + n_rows;
  const bool first = blockIdx.x == 0;
  const long long head = a.ring_pos[0], tail = a.ring_pos[1];
  const long long avail = min(max(tail - head, 0ll), (long long)a.n_pages);
  long long hm = head % a.n_pages;
  if (hm < 0) hm += a.n_pages;
  uint32_t bad = (tail - head != avail) ? SPEC_STATUS_BAD_LEN : 0u;
  if (tid == 0) taken_s = 0u;

  // scan of the needs (high word) and of the requests met here (low word)
  unsigned long long carry = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + tid;
    int kv = 0, row0 = 0, n = 0, have = 0, need = 0;
    bool ok = false;
    if (r < a.R) {
      kv = a.kv_len[r];
      row0 = a.row_off[r];
      const int row1 = a.row_off[r + 1];
      ok = kv >= 0 && row0 >= 0 && row1 >= row0 && row1 <= a.rows && kv <= INT_MAX - (row1 - row0);
      if (!ok) bad |= SPEC_STATUS_BAD_LEN;
      if (ok) {
        n = row1 - row0;
        have = ceil_div(kv, P);
        const int want = ceil_div(kv + n, P);
        need = want - have;
        if (want > a.max_pages) {
          bad |= SPEC_STATUS_NO_PAGES;
          ok = false;
          need = 0;
        }
      }
    }
    const bool met = ok && n > 0 && row0 < b1 && row0 + n > b0;
    unsigned long long all;
    const unsigned long long at =
        carry + block_scan<kThreads>(((unsigned long long)need << 32) | (met ? 1u : 0u), warp_sum, &all);
    carry += all;
    const unsigned off = (unsigned)(at >> 32), place = (unsigned)at;
    const bool granted = ok && (need == 0 || (long long)off + need <= avail);
    if (ok && !granted) bad |= SPEC_STATUS_NO_PAGES;
    if (met && place < kChunk)
      list[place] = Entry{r, row0, granted ? n : 0, kv, have,
                          a.pos_base ? a.pos_base[r] : 0, off};
    if (first && r < a.R) {
      a.new_len[r] = granted ? kv + n : max(kv, 0);
      if (granted && need > 0) atomicMax(&taken_s, off + (unsigned)need);
    }
  }
  __syncthreads();
  if (first && tid == 0) {
    a.ring_out[0] = head + taken_s;
    a.ring_out[1] = tail;
  }

  const int n_list = min((int)(unsigned)carry, kChunk);
  for (int i = tid; i < n_rows; i += kThreads) {
    const int b = b0 + i;
    int lo = 0, hi = n_list;  // the last entry that starts at or before row b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (list[mid].row0 <= b) lo = mid;
      else hi = mid;
    }
    int position = -1, request = -1, slot = -1;
    if (n_list > 0) {
      const Entry e = list[lo];
      const int j = b - e.row0;
      if (j >= 0 && j < e.n) {
        const int p = e.kv + j, pi = p / P, in = p - pi * P;
        int32_t* entry = a.block_table + (size_t)e.r * a.max_pages + pi;
        int page;
        if (pi < e.have) {
          page = *entry;
        } else {
          long long q = hm + e.off + (pi - e.have);
          if (q >= a.n_pages) q -= a.n_pages;
          page = a.ring[q];
          if (in == 0) *entry = page;  // the page's first row: the one writer of the entry
        }
        request = e.r;
        position = e.base + p;
        if (page >= 0 && page < a.n_pages) slot = page * P + in;
        else bad |= SPEC_STATUS_BAD_PAGE;
      }
    }
    a.position[b] = position;
    a.request[b] = request;
    a.slot[b] = slot;
  }
  if (bad) set_status(a.status, bad);
}

// A page id outside the cache gets no place in the ring: the ids after it close up.  So
// a block looks at the ids of the requests before its own too, kPages a thread at a time
// and in order; where none is strange (one barrier tells) a page's place is its number,
// otherwise the strange ones are scanned.  The request of a page is the last one that
// starts at or before it: starts are marked in shared memory and a maximum runs over the
// marks (a binary search a page spent 4 us of 11 on bank conflicts with 2000 requests).
constexpr int kPages = 4;

template <int kThreads>
__global__ void __launch_bounds__(kThreads) commit_kernel(spec_cache_commit_args a) {
  constexpr int kRound = kThreads * kPages;
  __shared__ unsigned long long warp_sum[kThreads / 32];
  __shared__ unsigned long long at_s[kThreads];  // of a scan's requests: number of the first page given back,
  __shared__ int stay_s[kThreads];               // and its table entry
  __shared__ __align__(8) uint16_t mark_s[kRound];  // 1 + the request that starts at a page, 0: none
  __shared__ int warp_top[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = a.page_size;
  const int own0 = blockIdx.x * kOwn, own1 = min(own0 + kOwn, a.R);
  const long long head = a.ring_pos[0], tail = a.ring_pos[1];
  // the ring has room for n_pages ids: more than that can only come from bad lengths
  const unsigned long long room = (unsigned long long)max(0ll, a.n_pages - max(tail - head, 0ll));
  long long tm = tail % a.n_pages;
  if (tm < 0) tm += a.n_pages;
  uint32_t bad = 0;

  unsigned long long carry = 0;  // pages that have got a place
  int kv = 0, len = 0, keep = 0;
  auto lengths = [&](int r) {
    if (r < own1) kv = a.kv_len[r], len = a.new_len[r], keep = a.keep[r];
  };
  lengths(tid);
  for (int r0 = 0; r0 < own1; r0 += kThreads) {
    const int r = r0 + tid;
    int stay = 0, back = 0;
    if (r < own1) {
      int kept;
      if (kv >= 0 && len >= kv && ceil_div(len, P) <= a.max_pages) {
        kept = keep < 0 ? 0 : (keep < len - kv ? kv + keep : len);
        stay = ceil_div(kept, P);
        back = ceil_div(len, P) - stay;
      } else {
        bad |= SPEC_STATUS_BAD_LEN;
        kept = max(kv, 0);
      }
      if (r >= own0) a.kv_out[r] = kept;
    }
    lengths(r + kThreads);  // the next scan's, on their way during this one's pages
    unsigned long long all;
    const unsigned long long at = block_scan<kThreads>((unsigned long long)back, warp_sum, &all);
    at_s[tid] = at;
    stay_s[tid] = stay;
    for (unsigned long long i0 = 0; i0 < all; i0 += kRound) {
      reinterpret_cast<uint2*>(mark_s)[tid] = make_uint2(0u, 0u);
      __syncthreads();
      if (back > 0 && at < i0 + kRound && at + back > i0) mark_s[at > i0 ? at - i0 : 0] = (uint16_t)(tid + 1);
      __syncthreads();
      const uint2 m = reinterpret_cast<const uint2*>(mark_s)[tid];
      int owner[kPages] = {(int)(m.x & 0xffffu), (int)(m.x >> 16), (int)(m.y & 0xffffu), (int)(m.y >> 16)};
#pragma unroll
      for (int u = 1; u < kPages; ++u) owner[u] = max(owner[u], owner[u - 1]);
      int top = owner[kPages - 1];  // of the warp's threads up to this one
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, t);
      }
      if (lane == 31) warp_top[warp] = top;
      __syncthreads();
      const int before_warp = __reduce_max_sync(0xffffffffu, lane < warp ? warp_top[lane] : 0);
      const int up = __shfl_up_sync(0xffffffffu, top, 1), before = max(before_warp, lane > 0 ? up : 0);
      int page[kPages];
      bool here[kPages], strange[kPages], found = false;  // here: a page of an own request
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        const unsigned long long i = i0 + tid * kPages + u;
        here[u] = false;
        page[u] = 0;
        if (i >= all) continue;
        const int lo = max(owner[u], before) - 1;
        here[u] = r0 + lo >= own0;
        page[u] = a.block_table[(size_t)(r0 + lo) * a.max_pages + stay_s[lo] + (i - at_s[lo])];
      }
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        strange[u] = page[u] < 0 || page[u] >= a.n_pages;
        found |= strange[u];
      }
      unsigned long long gone = 0, misses = 0;
      if (__syncthreads_or(found)) {
        bad |= SPEC_STATUS_BAD_PAGE;
        unsigned long long mine = 0;
#pragma unroll
        for (int u = 0; u < kPages; ++u) mine += strange[u];
        gone = block_scan<kThreads>(mine, warp_sum, &misses);
      }
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        const unsigned long long place = carry + (i0 + tid * kPages + u) - gone;
        if (here[u] && !strange[u] && place < room) {
          const long long q = tm + (long long)place;
          a.ring[q < a.n_pages ? q : q - a.n_pages] = page[u];
        }
        gone += strange[u];
      }
      carry -= misses;  // (the pages' numbers count from this scan's first)
    }
    carry += all;
  }
  if (blockIdx.x == gridDim.x - 1 && tid == 0) {  // the block that has seen every request
    if (carry > room) bad |= SPEC_STATUS_BAD_LEN;
    a.ring_out[0] = head;
    a.ring_out[1] = tail + (long long)min(carry, room);
  }
  if (bad) set_status(a.status, bad);
}

}  // namespace

// Reserve: blocks of 256 threads where the scan is one round of a few warps (1 request 2.7 us,
// 3.3 with 1024 threads; 32 requests 3.7 and 3.9; 64 4.5 and 4.1; 512 7.0 and 4.5), and where
// there are more blocks than two an SM (250 prompts in 486 blocks: 6.2 us, 9.2 with 1024).
constexpr int kFew = 32;

cudaError_t launch_cache_reserve(const spec_cache_reserve_args& a, cudaStream_t stream) {
  const int blocks = std::max(1, (int)(((long long)a.rows + kChunk - 1) / kChunk));
  if (a.R <= kFew || (a.R <= 256 && blocks > 2 * 152)) reserve_kernel<256><<<blocks, 256, 0, stream>>>(a);
  else reserve_kernel<1024><<<blocks, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_commit(const spec_cache_commit_args& a, cudaStream_t stream) {
  const int blocks = std::max(1, (a.R + kOwn - 1) / kOwn);
  // 256 threads where one block has all requests (32 requests 3.1 us, 4.3 with 1024 threads; 128
  // 3.4 and 4.6); more requests bring more pages (512 requests 5.8 and 4.7, 250 prompts 5.2 and
  // 4.7; 256 requests that give back few 3.5 and 4.7).
  if (a.R <= kOwn) commit_kernel<256><<<blocks, 256, 0, stream>>>(a);
  else commit_kernel<1024><<<blocks, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace spec
