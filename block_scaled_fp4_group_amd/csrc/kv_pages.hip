// Pages of a paged cache: requests that go on as several (fork), the pages that no
// request holds (free), live pages moved to the front of the pool (compact).
//
// There are no reference counts: a page is live while the table's rows reach it, and
// the calls that need to know mark the pages that they reach in a bitmap, so a page
// that several requests share counts once, and nothing has to be kept between calls.
//
// What bounds them: forks and moves copy pages (32 forks of 8 parents' last pages, 16.8 MB
// read and written: 5.6 us; 538 moves of 72 KB, 79 MB: 16 us, 4.9 TB/s where a large copy reaches
// 5.1, behind a plan of 5 us by one workgroup); the rest are launches that wait for each other.
//
// A page's content is bytes here: up to eight buffers (keys and values, bf16 or codes
// and scales), page p of each at p * page_bytes.
#include <algorithm>

#include "common.h"

namespace moe {

constexpr int kForkThreads = 256;
constexpr int kMarkThreads = 1024;
constexpr int kMarkPages = 1 << 20;                 // 128 KB of LDS
constexpr int kCopyChunk = 16384;                   // bytes of a page per workgroup and step

struct PageBuffers {
  uint8_t* data[MOE_PAGE_BUFFERS];
  int64_t bytes[MOE_PAGE_BUFFERS];
  int32_t count;
};

struct TableArgs {
  const int32_t* table;
  int64_t stride;
  const int32_t* lens;
  int32_t rows, max_blocks, page_shift;
  int64_t num_pages;
};

__device__ __forceinline__ int held_pages(const TableArgs& t, int row) {
  const int64_t up = ((int64_t)1 << t.page_shift) - 1;
  return (int)min(((int64_t)max(t.lens[row], 0) + up) >> t.page_shift, (int64_t)t.max_blocks);
}

// Bytes [from, to) of page src to page dst of every buffer, the buffers' pages taken
// as one behind the other; 16 bytes per thread and load, four loads under way.
__device__ __forceinline__ void copy_page(const PageBuffers& b, int64_t dst, int64_t src, int64_t from, int64_t to) {
  int64_t begin = 0;
  for (int i = 0; i < b.count; ++i) {
    const int64_t lo = max(from - begin, (int64_t)0), hi = min(to - begin, b.bytes[i]);
    begin += b.bytes[i];
    const uint8_t* s = b.data[i] + src * b.bytes[i];
    uint8_t* d = b.data[i] + dst * b.bytes[i];
    const int64_t step = (int64_t)blockDim.x * 16;
    for (int64_t at = lo + threadIdx.x * 16; at < hi; at += 4 * step) {
      u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at + u * step < hi) v[u] = *(const u32x4*)(s + at + u * step);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at + u * step < hi) *(u32x4*)(d + at + u * step) = v[u];
    }
  }
}

// ------------------------------------------------------------------- fork
struct ForkArgs {
  TableArgs t;
  int32_t* table;
  int32_t* lens;
  const int32_t* parents;
  const int32_t* children;
  const int32_t* free_pages;
  int64_t num_free;
  int32_t* counts;
  PageBuffers buffers;
  int32_t num_forks, slices;
  int64_t page_bytes;                               // of all buffers
};

// Workgroup (fork, slice): whether fork i needs a page, and how many before it do, is
// counted by every workgroup itself (of a last page that is whole only by slice 0), which writes
// the child's row as slice 0 and copies its slice of the last page.  Pages of 16 KB, one slice: 512
// forks 7 us, 4096 20, 16384 0.32 ms, 65536 7.8 ms.  Pages of 1 MB: 32 forks in 64 slices 10 us,
// 512 in 8 98 us (1 GB), 4096 in one, 512 of them with a page left, 0.19 ms; in 64 slices, which all
// count, 0.85 ms, and 16384 20 ms for 0.48.
__global__ __launch_bounds__(kForkThreads) void kv_fork_kernel(ForkArgs a) {
  __shared__ int part[kForkThreads / 64];
  const int fork = blockIdx.x / (uint32_t)a.slices, slice = blockIdx.x % (uint32_t)a.slices;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  auto valid = [&](int i, int& p, int& c) {
    p = a.parents[i];
    c = a.children[i];
    return p >= 0 && p < a.t.rows && c >= 0 && c < a.t.rows && p != c;
  };
  const int64_t mask = ((int64_t)1 << a.t.page_shift) - 1, cap = (int64_t)a.t.max_blocks << a.t.page_shift;
  auto length = [&](int row) { return min((int64_t)max(a.t.lens[row], 0), cap); };
  if (slice > 0) {                                                  // only the page's copy: is there one?
    int p, c;
    if (!valid(fork, p, c) || (length(p) & mask) == 0) return;
  }
  const bool last = fork == max(a.num_forks, 1) - 1 && slice == 0;
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < (last ? a.num_forks : fork); i += kForkThreads) {
    int p, c;
    const int need = valid(i, p, c) && (length(p) & mask) != 0;
    before += i < fork ? need : 0;
    all += need;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    before += __shfl_xor(before, d);
    all += __shfl_xor(all, d);
  }
  if (lane == 0) part[wv] = before;
  __syncthreads();
  before = part[0] + part[1] + part[2] + part[3];
  auto free_page = [&](int i) {                                     // -1: none left
    const int64_t p = i < a.num_free ? a.free_pages[i] : -1;
    return p < a.t.num_pages ? p : -1;
  };
  if (last) {
    auto sum = [&](int x) {
      __syncthreads();
      if (lane == 0) part[wv] = x;
      __syncthreads();
      return part[0] + part[1] + part[2] + part[3];
    };
    all = sum(all);
    int taken = 0;
    for (int i = threadIdx.x; i < all; i += kForkThreads) taken += free_page(i) >= 0;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) taken += __shfl_xor(taken, d);
    taken = sum(taken);
    if (threadIdx.x == 0) {
      a.counts[0] = taken;
      a.counts[1] = all;
    }
  }
  if (a.num_forks == 0) return;
  int p, c;
  if (!valid(fork, p, c)) return;
  const int64_t len = length(p), whole = len >> a.t.page_shift;
  const bool cut = (len & mask) != 0;
  const int32_t* from = a.t.table + p * a.t.stride;
  const int64_t fresh = cut ? free_page(before) : -1;
  if (slice == 0) {
    int32_t* to = a.table + c * a.t.stride;
    for (int64_t i = threadIdx.x; i < whole; i += kForkThreads) to[i] = from[i];
    if (threadIdx.x == 0) {
      if (cut) to[whole] = fresh < 0 ? -1 : (int32_t)fresh;
      a.lens[c] = (int32_t)(cut && fresh < 0 ? whole << a.t.page_shift : len);
    }
  }
  if (!cut) return;
  const int64_t old = from[whole];
  if (fresh < 0 || old < 0 || old >= a.t.num_pages) return;
  const int64_t each = ((a.page_bytes + a.slices - 1) / a.slices + 15) & ~(int64_t)15;
  copy_page(a.buffers, fresh, old, slice * each, min(a.page_bytes, (slice + 1) * each));
}

// ------------------------------------------------------------- live pages
// Four times 64 entries, lanes side by side on rows of fewer than 64 (so many lanes to a row as
// the power of two that holds it), under way at once behind their rows' lengths: bits of the
// pages set by `set`.  wave of `waves`.  (Rows in 64 bits: all waves' together may be 16 times as
// many as the table has.)
template <class Set>
__device__ __forceinline__ void mark_rows(const TableArgs& t, int wave, int waves, Set set) {
  const int shift = t.max_blocks > 32 ? 6 : (t.max_blocks <= 1 ? 0 : 32 - __builtin_clz(t.max_blocks - 1));
  const int lane = threadIdx.x & 63, sub = lane >> shift, per = 64 >> shift, step = 1 << shift;
  for (int64_t first = (int64_t)(4 * per) * wave; first < t.rows; first += (int64_t)(4 * per) * waves) {
    int n[4], most = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) n[u] = held_pages(t, (int)min(first + u * per + sub, (int64_t)t.rows - 1));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      n[u] = first + u * per + sub < t.rows ? n[u] : 0;
      most = max(most, n[u]);
    }
    for (int i = lane & (step - 1); i < most; i += step) {
      int32_t p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = i < n[u] ? t.table[(first + u * per + sub) * t.stride + i] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p[u] >= 0 && p[u] < t.num_pages) set(p[u]);
    }
  }
}

// Of a large table or pool the marks are made in memory, a byte for each page, by all
// workgroups (cleared by one launch, set by the next; plain stores of the same value need no
// atomics), of a small one in LDS, a bit for each page, by the workgroup that uses them.
// Entries 1500 x 256 of a pool of 190000 pages: 80 us by one workgroup, 12 us so (17 with a
// bit for each page, set by atomics).  By one workgroup / by all, us: 64 x 64 of 4000 pages
// freed 4.5 / 7.4, 256 x 64 of 16000 9.0 / 8.7, 100 x 160 of 60000 18 / 10 (its workgroup
// sweeps all pages), 512 x 64 of 30000 15 / 9; 100 x 160 of 60000 compacted 22 / 24, 512 x 64 of 30000
// 24 / 21.
constexpr int64_t kMarkAlone = 16384;               // entries
constexpr int64_t kSweepAlone = 16384, kPlanAlone = 65536;   // pages
static bool marks_alone(int64_t rows, int64_t max_blocks, int64_t num_pages, int64_t pages) {
  return rows * max_blocks <= kMarkAlone && num_pages <= pages;
}
static int64_t mark_bytes(int64_t num_pages) { return (num_pages + 127) / 128 * 128; }
// (list, if there is one: -1 everywhere, of which the sweep then overwrites the front)
__global__ __launch_bounds__(256) void kv_clear_kernel(uint8_t* marks, int64_t bytes, int32_t* list, int pages) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
  if (i < bytes) *(u32x4*)(marks + i) = u32x4{0u, 0u, 0u, 0u};
  if (!list) return;
  const int base = blockIdx.x * 4096;
  for (int j = base + threadIdx.x; j < min(base + 4096, pages); j += 256) list[j] = -1;
}
__global__ __launch_bounds__(256) void kv_mark_kernel(TableArgs t, uint8_t* marks) {
  mark_rows(t, blockIdx.x * 4 + (threadIdx.x >> 6), gridDim.x * 4, [&](int p) { marks[p] = 1; });
}
// Marks of pages 32 w .. 32 w + 31 as bits: four bytes of 0 or 1 meet in a product's top
// bits, each in one place.
__device__ __forceinline__ uint32_t mark_word(const uint8_t* marks, int w) {
  uint32_t bits = 0u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32x4 x = *(const u32x4*)(marks + 32 * (int64_t)w + 16 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) bits |= (x[j] * 0x10204080u) >> 28 << (16 * i + 4 * j);
  }
  return bits;
}

// Those of pages 32 w + 8 q .. 32 w + 8 q + 7.
__device__ __forceinline__ uint32_t mark_byte(const uint8_t* marks, int w, int q) {
  const u32x2 x = *(const u32x2*)(marks + 32 * (int64_t)w + 8 * q);
  return (x[0] * 0x10204080u) >> 28 | (x[1] * 0x10204080u) >> 28 << 4;
}

// All marks as bits in LDS, by the whole workgroup: read, or made here.  Ends with a barrier.
__device__ __forceinline__ void load_pages(const TableArgs& t, const uint8_t* marks, uint32_t* bits, int words) {
  if (marks) {
    for (int i = threadIdx.x; i < words; i += kMarkThreads) bits[i] = mark_word(marks, i);
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < words; i += kMarkThreads) bits[i] = 0u;
  __syncthreads();
  mark_rows(t, threadIdx.x >> 6, kMarkThreads / 64, [&](int p) { atomicOr(&bits[p >> 5], 1u << (p & 31)); });
  __syncthreads();
}

// Exclusive prefix sum of x over the workgroup's threads; all: its sum.  Ends with a barrier.
__device__ __forceinline__ int scan_block(int x, int* all, int* part) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int sum = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 63) part[wv] = sum;
  __syncthreads();
  int before = 0;
  *all = 0;
#pragma unroll
  for (int w = 0; w < kMarkThreads / 64; ++w) {
    before += w < wv ? part[w] : 0;
    *all += part[w];
  }
  __syncthreads();
  return before + sum - x;
}

struct FreeArgs {
  TableArgs t;
  const uint8_t* marks;                             // null: made by the one workgroup
  int32_t* free_pages;
  int32_t* counts;
};

// Workgroup i sweeps words kSweepWords i .. of the marks' bits (the only one: all); what it
// finds free follows what there is before, which it counts itself.
constexpr int kSweepWords = kMarkThreads / 4;       // 8 pages to a thread

__global__ __launch_bounds__(kMarkThreads) void kv_sweep_kernel(FreeArgs a) {
  __shared__ uint32_t bits[kSweepAlone / 32];
  __shared__ int32_t out[32 * kSweepWords];
  __shared__ int part[kMarkThreads / 64];
  const int P = (int)a.t.num_pages, words = (P + 31) / 32;
  int w0 = 0, w1 = words, before = 0;                               // held pages before w0
  if (a.marks) {
    w0 = blockIdx.x * kSweepWords;
    w1 = min(w0 + kSweepWords, words);
    uint32_t x = 0u;                                                // (marks are 0 or 1)
    for (int i = 16 * (int)threadIdx.x; i < 32 * w0; i += 8 * 16 * kMarkThreads) {
      u32x4 v[8];                                                   // 16 pages each, 8 loads under way
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = i + u * 16 * kMarkThreads;
        v[u] = at < 32 * w0 ? *(const u32x4*)(a.marks + at) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) x = __builtin_amdgcn_sad_u8(v[u][j], 0u, x);
    }
    scan_block((int)x, &before, part);
  } else {
    load_pages(a.t, nullptr, bits, words);
  }
  before = 32 * w0 - before;                                        // from here on: free ones
  // the list of kSweepWords words at a time through LDS, so that it is stored in whole lines
  for (int base = w0; base < w1; base += kSweepWords) {
    const int w = base + (threadIdx.x >> 2), q = threadIdx.x & 3;
    uint32_t f = 0u;                                                // 8 pages to a thread
    if (w < w1) {
      f = ~(a.marks ? mark_byte(a.marks, w, q) : bits[w] >> (8 * q)) & 255u;
      const int pages = P - (32 * w + 8 * q);
      if (pages < 8) f &= (1u << max(pages, 0)) - 1u;
    }
    int n;
    int at = scan_block(__popc(f), &n, part);
    for (; f; f &= f - 1) out[at++] = 32 * w + 8 * q + __builtin_ctz(f);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kMarkThreads) a.free_pages[before + i] = out[i];
    before += n;
    __syncthreads();
  }
  if (w1 < words) return;
  // the last workgroup knows how many there are
  if (threadIdx.x == 0) {
    a.counts[0] = before;
    a.counts[1] = P - before;
  }
  if (!a.marks)                                                     // (else done by the first launch)
    for (int i = before + threadIdx.x; i < P; i += kMarkThreads) a.free_pages[i] = -1;
}

// ---------------------------------------------------------------- compact
// Workspace: the number of live pages, the number of moves, and for each page at or
// behind that number where it goes (-1: nowhere); then the moves' sources and targets.
struct CompactArgs {
  TableArgs t;
  const uint8_t* marks;                             // null: made by the planning workgroup
  int32_t* out;
  int64_t out_stride;
  int32_t* counts;
  int32_t* ws;
  PageBuffers buffers;
  int64_t page_bytes;
};
__device__ __forceinline__ int32_t* move_to(const CompactArgs& a) { return a.ws + 4; }                      // [num_pages]
__device__ __forceinline__ int32_t* move_src(const CompactArgs& a) { return a.ws + 4 + a.t.num_pages; }     // [num_pages / 2]
__device__ __forceinline__ int32_t* move_dst(const CompactArgs& a) { return move_src(a) + a.t.num_pages / 2; }

// The i-th live page at or behind the live ones' number n goes to the i-th hole before it.
__global__ __launch_bounds__(kMarkThreads) void kv_compact_plan_kernel(CompactArgs a) {
  __shared__ uint32_t bits[kMarkPages / 32];
  __shared__ int part[kMarkThreads / 64];
  const int P = (int)a.t.num_pages, words = (P + 31) / 32;
  load_pages(a.t, a.marks, bits, words);
  int x = 0, n, moves = 0;
  for (int w = threadIdx.x; w < words; w += kMarkThreads) x += __popc(bits[w]);
  scan_block(x, &n, part);
  // 8 pages to a thread; holes before page n and held pages from it on counted in the halves
  // of one number (at most 8192 in a step)
  int holes = 0;
  for (int base = 0; base < words; base += kMarkThreads / 4) {
    const int w = base + (threadIdx.x >> 2), p = 32 * w + 8 * (int)(threadIdx.x & 3);
    const uint32_t held = w < words ? bits[w] >> (8 * (threadIdx.x & 3)) & 255u : 0u;
    const uint32_t front = p + 8 <= n ? 255u : (p >= n ? 0u : (1u << (n - p)) - 1u);   // pages before n
    uint32_t f = ~held & front, g = held & ~front;
    int all;
    const int at = scan_block(__popc(f) | __popc(g) << 16, &all, part);
    int at_hole = holes + (at & 0xffff), at_far = moves + (at >> 16);
    for (; f; f &= f - 1) move_dst(a)[at_hole++] = p + __builtin_ctz(f);
    for (; g; g &= g - 1) move_src(a)[at_far++] = p + __builtin_ctz(g);
    holes += all & 0xffff;
    moves += all >> 16;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kMarkThreads) move_to(a)[move_src(a)[i]] = move_dst(a)[i];
  if (threadIdx.x == 0) {
    a.ws[0] = n;
    a.ws[1] = moves;
    a.counts[0] = n;
    a.counts[1] = moves;
  }
}

// Rows of the table, and pages in chunks, by all workgroups.
__global__ __launch_bounds__(256) void kv_compact_move_kernel(CompactArgs a) {
  const int n = a.ws[0], moves = a.ws[1];
  for (int64_t row = blockIdx.x; row < a.t.rows; row += gridDim.x) {
    const int held = held_pages(a.t, (int)row);
    const int32_t* e = a.t.table + row * a.t.stride;
    int32_t* o = a.out + row * a.out_stride;
    for (int i = threadIdx.x; i < a.t.max_blocks; i += 256) {
      int32_t p = i < held ? e[i] : -1;
      if (p >= n && p < a.t.num_pages) p = move_to(a)[p];
      o[i] = p < 0 || p >= a.t.num_pages ? -1 : p;
    }
  }
  const int64_t chunks = (a.page_bytes + kCopyChunk - 1) / kCopyChunk, all = moves * chunks;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int64_t m = i / chunks, from = (i % chunks) * kCopyChunk;
    copy_page(a.buffers, move_dst(a)[m], move_src(a)[m], from, min(from + kCopyChunk, a.page_bytes));
  }
}

// ------------------------------------------------------------------- host
static TableArgs table_args(const int32_t* table, int64_t stride, int rows, int max_blocks, const int32_t* lens,
                            int page_shift, int64_t num_pages) {
  TableArgs t;
  t.table = table;
  t.stride = stride;
  t.lens = lens;
  t.rows = rows;
  t.max_blocks = max_blocks;
  t.page_shift = page_shift;
  t.num_pages = num_pages;
  return t;
}

static PageBuffers page_buffers(const moe_page_buffers& b, int64_t* all) {
  PageBuffers p = {};
  *all = 0;
  p.count = b.count;
  for (int i = 0; i < b.count; ++i) {
    p.data[i] = (uint8_t*)b.data[i];
    p.bytes[i] = b.page_bytes[i];
    *all += b.page_bytes[i];
  }
  return p;
}

int64_t kv_pages_most() { return kMarkPages; }
size_t kv_free_ws_bytes(int64_t rows, int64_t max_blocks, int64_t num_pages) {
  return marks_alone(rows, max_blocks, num_pages, kSweepAlone) ? 0 : (size_t)mark_bytes(num_pages);
}
// (the marks first: 16-byte aligned)
size_t kv_compact_ws_bytes(int64_t num_pages) {
  return (size_t)mark_bytes(num_pages) + (size_t)(4 + num_pages + 2 * (num_pages / 2)) * 4;
}

// The marks in memory, if they are made there.
static uint8_t* launch_marks(const TableArgs& t, int64_t alone, void* ws, int32_t* list, hipStream_t stream) {
  if (marks_alone(t.rows, t.max_blocks, t.num_pages, alone)) return nullptr;
  uint8_t* marks = (uint8_t*)ws;
  const int64_t bytes = mark_bytes(t.num_pages);
  hipLaunchKernelGGL(kv_clear_kernel, dim3((uint32_t)((bytes + 4095) / 4096)), dim3(256), 0, stream, marks, bytes, list,
                     (int)t.num_pages);
  const int64_t wgs = ((int64_t)t.rows + 15) / 16;                   // (they go on where there are more rows)
  if (t.rows > 0) hipLaunchKernelGGL(kv_mark_kernel, dim3((uint32_t)(wgs < 65536 ? wgs : 65536)), dim3(256), 0, stream, t, marks);
  return marks;
}

moe_status launch_kv_fork(int32_t* table, int64_t stride, int rows, int max_blocks, int32_t* lens, const int32_t* parents,
                          const int32_t* children, int num_forks, const int32_t* free_pages, int64_t num_free,
                          int page_shift, const moe_page_buffers& buffers, int64_t num_pages, int32_t* counts,
                          hipStream_t stream) {
  ForkArgs a;
  a.t = table_args(table, stride, rows, max_blocks, lens, page_shift, num_pages);
  a.table = table;
  a.lens = lens;
  a.parents = parents;
  a.children = children;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.counts = counts;
  a.num_forks = num_forks;
  a.buffers = page_buffers(buffers, &a.page_bytes);
  const int64_t slices = (a.page_bytes + kCopyChunk - 1) / kCopyChunk;
  // (a page's copy by so many workgroups, as long as all forks' are not more than the chip holds
  // twice over: each of them counts)
  const int64_t most = std::min<int64_t>(64, std::max<int64_t>(1, 4096 / std::max(num_forks, 1)));
  a.slices = (int)std::max<int64_t>(1, std::min(slices, most));
  const uint32_t grid = num_forks == 0 ? 1u : (uint32_t)num_forks * (uint32_t)a.slices;
  hipLaunchKernelGGL(kv_fork_kernel, dim3(grid), dim3(kForkThreads), 0, stream, a);
  return launch_status("moe_kv_fork");
}

moe_status launch_kv_free_pages(const int32_t* table, int64_t stride, int rows, int max_blocks, const int32_t* lens,
                                int page_shift, int64_t num_pages, int32_t* free_pages, int32_t* counts, void* ws,
                                hipStream_t stream) {
  FreeArgs a;
  a.t = table_args(table, stride, rows, max_blocks, lens, page_shift, num_pages);
  a.free_pages = free_pages;
  a.counts = counts;
  a.marks = launch_marks(a.t, kSweepAlone, ws, free_pages, stream);
  const int64_t words = (num_pages + 31) / 32;
  const uint32_t grid = a.marks ? (uint32_t)((words + kSweepWords - 1) / kSweepWords) : 1u;
  hipLaunchKernelGGL(kv_sweep_kernel, dim3(grid), dim3(kMarkThreads), 0, stream, a);
  return launch_status("moe_kv_free_pages");
}

moe_status launch_kv_compact(const int32_t* table, int64_t stride, int rows, int max_blocks, const int32_t* lens,
                             int page_shift, const moe_page_buffers& buffers, int64_t num_pages, int32_t* out,
                             int64_t out_stride, int32_t* counts, void* ws, hipStream_t stream) {
  CompactArgs a;
  a.t = table_args(table, stride, rows, max_blocks, lens, page_shift, num_pages);
  a.out = out;
  a.out_stride = out_stride;
  a.counts = counts;
  a.ws = (int32_t*)((uint8_t*)ws + mark_bytes(num_pages));
  a.buffers = page_buffers(buffers, &a.page_bytes);
  a.marks = launch_marks(a.t, kPlanAlone, ws, nullptr, stream);
  hipLaunchKernelGGL(kv_compact_plan_kernel, dim3(1), dim3(kMarkThreads), 0, stream, a);
  moe_status st = launch_status("moe_kv_compact");
  if (st != MOE_OK) return st;
  hipLaunchKernelGGL(kv_compact_move_kernel, dim3(2048), dim3(256), 0, stream, a);
  return launch_status("moe_kv_compact");
}

}  // namespace moe
