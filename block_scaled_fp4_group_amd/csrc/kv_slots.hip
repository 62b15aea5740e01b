// Block tables and cache slots of a step's new tokens, from the request lengths.
//
// Request b holds c_b cached tokens in ceil(c_b / p) pages of p tokens and
// brings n_b new ones; the pages it still needs are the next entries of the
// free list, in request order:
//   need_b  = ceil((c_b + n_b) / p) - ceil(c_b / p)
//   first_b = need_0 + .. + need_{b-1}
//   table[b, ceil(c_b / p) + i] = free_pages[first_b + i]          i < need_b
//   token i of request b: position c_b + i, slot table[b, pos / p] * p + pos % p
//
// One launch: every workgroup scans the (short) length lists itself in LDS and
// then fills its slice of the tokens and of the new pages, so no workgroup
// waits for another.  A new page is looked up in the free list, never read back
// from the table, and the table's old entries are never written, so the update
// in place needs no order between workgroups.
//
// Bound by latency: 64 requests of one token take 3.5 us, 1500 requests with
// 140792 new tokens 7.7 us (1.2 MB written), launch after launch in a graph; an empty
// launch takes about 2.
#include "common.h"

namespace moe {

constexpr int kSlotThreads = 256;
constexpr int kSlotMaxRequests = 4096;
constexpr int kSlotPerThread = kSlotMaxRequests / kSlotThreads;

struct SlotArgs {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;
  int64_t table_stride;
  int32_t* slots;
  int32_t* positions;
  int32_t* cu_new;
  int32_t* counts;
  int64_t max_new, max_pages;
  int32_t num_requests, max_blocks, page_shift, position_base;
  int64_t num_free;
};

// last b with pref[b] <= x (pref ascending, pref[0] = 0)
__device__ __forceinline__ int last_at_most(const int64_t* pref, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct SlotRequest {
  int64_t cached;   // tokens in the cache, at most what the table holds
  int64_t fresh;    // new tokens (also those without room in the table)
  int64_t held, need;
};

__device__ __forceinline__ SlotRequest slot_request(const SlotArgs& a, int b) {
  const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
  const int64_t up = ((int64_t)1 << a.page_shift) - 1;
  SlotRequest r;
  r.cached = min((int64_t)max(a.cached[b], 0), cap);
  r.fresh = max(a.fresh[b], 0);
  r.held = (r.cached + up) >> a.page_shift;
  r.need = ((min(r.cached + r.fresh, cap) + up) >> a.page_shift) - r.held;
  return r;
}

// The last workgroup writes the offsets and the counts, the others the pages and the
// tokens: what it reads for the counts is not waited for by theirs.
__global__ __launch_bounds__(kSlotThreads) void kv_slots_kernel(SlotArgs a) {
  __shared__ int64_t tok[kSlotMaxRequests + 1], page[kSlotMaxRequests + 1];   // exclusive prefix sums
  __shared__ int64_t part[3][kSlotThreads / 64];
  const int B = a.num_requests, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const bool counts = blockIdx.x == gridDim.x - 1;
  // each thread sums its run of consecutive requests, the 256 sums are scanned
  // (each wave its own, then the waves' totals), and the runs are written out from
  // their starts
  const int per = (B + kSlotThreads - 1) / kSlotThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  int64_t nt = 0, np = 0, lost = 0;
  if (counts) {
    // Tokens that go into a page entered as -1 before: only the last page held has room
    // for any.  (Without room some entry is read and not used.)  Eight requests' loads
    // are under way at once.
    for (int first = tid; first < B; first += 8 * kSlotThreads) {
      SlotRequest r[8];
      int32_t pg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = slot_request(a, min(first + i * kSlotThreads, B - 1));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        pg[i] = a.table[min(first + i * kSlotThreads, B - 1) * a.table_stride + max(r[i].held - 1, (int64_t)0)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + i * kSlotThreads < B && !(pg[i] >= 0 && pg[i] < a.max_pages))
          lost += min(r[i].fresh, (r[i].held << a.page_shift) - r[i].cached);
    }
  }
  for (int b = b0; b < b1; ++b) {
    const SlotRequest r = slot_request(a, b);
    nt += r.fresh;
    np += r.need;
  }
  int64_t st = nt, sp = np;                                         // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t x = __shfl_up(st, d), y = __shfl_up(sp, d);
    if (lane >= d) {
      st += x;
      sp += y;
    }
  }
  if (lane == 63) {
    part[0][wv] = st;
    part[1][wv] = sp;
  }
  __syncthreads();
  int64_t t0 = st - nt, p0 = sp - np, total = 0, pages = 0;
#pragma unroll
  for (int w = 0; w < kSlotThreads / 64; ++w) {
    if (w < wv) {
      t0 += part[0][w];
      p0 += part[1][w];
    }
    total += part[0][w];
    pages += part[1][w];
  }
  for (int b = b0; b < b1; ++b) {
    const SlotRequest r = slot_request(a, b);
    tok[b] = t0;
    page[b] = p0;
    // tokens that get a slot: up to the end of the last page the free list still had
    const int64_t got = min(max(a.num_free - p0, (int64_t)0), r.need);
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
    const int64_t end = min(min(r.cached + r.fresh, cap), got == r.need ? cap : (r.held + got) << a.page_shift);
    lost += r.fresh - max(end - r.cached, (int64_t)0);
    t0 += r.fresh;
    p0 += r.need;
  }
  if (tid == 0) {
    tok[B] = total;
    page[B] = pages;
  }
  if (counts) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) lost += __shfl_xor(lost, d);
    if (lane == 0) part[2][wv] = lost;
  }
  __syncthreads();
  if (counts) {
    for (int b = tid; b <= B; b += kSlotThreads) a.cu_new[b] = (int32_t)min(tok[b], (int64_t)0x7fffffff);
    if (tid == 0) {
      lost = 0;
#pragma unroll
      for (int w = 0; w < kSlotThreads / 64; ++w) lost += part[2][w];
      a.counts[0] = (int32_t)min(min(pages, a.num_free), (int64_t)0x7fffffff);
      a.counts[1] = (int32_t)min(pages, (int64_t)0x7fffffff);
      a.counts[2] = (int32_t)min(lost, (int64_t)0x7fffffff);
    }
    return;
  }
  const int64_t step = (int64_t)(gridDim.x - 1) * kSlotThreads, at = (int64_t)blockIdx.x * kSlotThreads + tid;
  for (int64_t j = at; j < pages; j += step) {
    const int b = last_at_most(page, B, j);
    const int64_t block = slot_request(a, b).held + j - page[b];
    a.table[b * a.table_stride + block] = j < a.num_free ? a.free_pages[j] : -1;
  }
  for (int64_t t = at; t < a.max_new; t += step) {
    int32_t slot = -1, pos32 = 0;
    if (t < total) {
      const int b = last_at_most(tok, B, t);
      const SlotRequest r = slot_request(a, b);
      const int64_t pos = r.cached + t - tok[b], block = pos >> a.page_shift;
      pos32 = (int32_t)min(pos + a.position_base, (int64_t)0x7fffffff);
      if (block < a.max_blocks) {
        const int64_t j = page[b] + block - r.held;
        const int32_t pg = block < r.held ? a.table[b * a.table_stride + block] : (j < a.num_free ? a.free_pages[j] : -1);
        if (pg >= 0 && pg < a.max_pages)
          slot = (int32_t)(((int64_t)pg << a.page_shift) + (pos & (((int64_t)1 << a.page_shift) - 1)));
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos32;
  }
}

int kv_slots_max_requests() { return kSlotMaxRequests; }

moe_status launch_kv_slots(const int32_t* cached, const int32_t* fresh, int B, const int32_t* free_pages,
                           int64_t num_free, int page_shift, int32_t* table, int64_t table_stride, int max_blocks,
                           int position_base, int64_t max_new, int32_t* slots, int32_t* positions, int32_t* cu_new,
                           int32_t* counts, hipStream_t stream) {
  SlotArgs a;
  a.cached = cached;
  a.fresh = fresh;
  a.free_pages = free_pages;
  a.table = table;
  a.table_stride = table_stride;
  a.slots = slots;
  a.positions = positions;
  a.cu_new = cu_new;
  a.counts = counts;
  a.max_new = max_new;
  a.max_pages = (int64_t)0x7fffffff >> page_shift;    // pages whose slots fit in 31 bits
  a.num_requests = B;
  a.max_blocks = max_blocks;
  a.page_shift = page_shift;
  a.position_base = position_base;
  a.num_free = num_free;
  const int64_t blocks = (max_new + kSlotThreads - 1) / kSlotThreads;
  // two workgroups of 64 KB of LDS fit a CU: 512 run at once (one more: 7.8 -> 10.9 us)
  const uint32_t grid = 1 + (uint32_t)(blocks < 1 ? 1 : (blocks > 511 ? 511 : blocks));
  hipLaunchKernelGGL(kv_slots_kernel, dim3(grid), dim3(kSlotThreads), 0, stream, a);
  return launch_status("moe_kv_slots");
}

}  // namespace moe
