// Pages of a paged cache: requests that go on as several (fork), the pages that no
// request holds (free), live pages moved to the front of the pool (compact).
//
// There are no reference counts: a page is live while the table's rows reach it, and
// the calls that need to know mark the pages that they reach in a bitmap, so a page
// that several requests share counts once, and nothing has to be kept between calls.
//
// A page's content is bytes here: up to eight buffers (keys and values, bf16 or codes
// and scales), page p of each at p * page_bytes.
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
// counted by every workgroup itself.  Slice 0 writes the child's row.
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
  if (last) {
    __syncthreads();
    if (lane == 0) part[wv] = all;
    __syncthreads();
    all = part[0] + part[1] + part[2] + part[3];
    if (threadIdx.x == 0) {
      a.counts[0] = (int32_t)min((int64_t)all, a.num_free);
      a.counts[1] = all;
    }
  }
  if (a.num_forks == 0) return;
  int p, c;
  if (!valid(fork, p, c)) return;
  const int64_t len = length(p), whole = len >> a.t.page_shift;
  const bool cut = (len & mask) != 0;
  const int32_t* from = a.t.table + p * a.t.stride;
  const int64_t fresh = cut && before < a.num_free ? a.free_pages[before] : -1;
  if (slice == 0) {
    int32_t* to = a.table + c * a.t.stride;
    for (int64_t i = threadIdx.x; i < whole; i += kForkThreads) to[i] = from[i];
    if (threadIdx.x == 0) {
      if (cut) to[whole] = (int32_t)fresh;
      a.lens[c] = (int32_t)(cut && fresh < 0 ? whole << a.t.page_shift : len);
    }
  }
  if (!cut) return;
  const int64_t old = from[whole];
  if (fresh < 0 || fresh >= a.t.num_pages || old < 0 || old >= a.t.num_pages) return;
  const int64_t each = ((a.page_bytes + a.slices - 1) / a.slices + 15) & ~(int64_t)15;
  copy_page(a.buffers, fresh, old, slice * each, min(a.page_bytes, (slice + 1) * each));
}

// ------------------------------------------------------------- live pages
// The bitmap of live pages in LDS, by the whole workgroup; ends with a barrier.
__device__ __forceinline__ void mark_pages(const TableArgs& t, uint32_t* bits, int words) {
  for (int i = threadIdx.x; i < words; i += kMarkThreads) bits[i] = 0u;
  __syncthreads();
  // a wave per row, 64 entries at a time
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int row = wv; row < t.rows; row += kMarkThreads / 64) {
    const int n = held_pages(t, row);
    const int32_t* e = t.table + row * t.stride;
    for (int i = lane; i < n; i += 64) {
      const int32_t p = e[i];
      if (p >= 0 && p < t.num_pages) atomicOr(&bits[p >> 5], 1u << (p & 31));
    }
  }
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
  int32_t* free_pages;
  int32_t* counts;
};

// One workgroup marks and sweeps.
__global__ __launch_bounds__(kMarkThreads) void kv_free_kernel(FreeArgs a) {
  __shared__ uint32_t bits[kMarkPages / 32];
  __shared__ int part[kMarkThreads / 64];
  const int P = (int)a.t.num_pages, words = (P + 31) / 32;
  mark_pages(a.t, bits, words);
  // each thread sweeps a run of words: what it finds free follows what those before it found
  const int per = (words + kMarkThreads - 1) / kMarkThreads;
  const int w0 = min((int)threadIdx.x * per, words), w1 = min(w0 + per, words);
  auto free_of = [&](int w) { return ~bits[w] & (w == words - 1 && (P & 31) ? (1u << (P & 31)) - 1u : ~0u); };
  int n = 0, all;
  for (int w = w0; w < w1; ++w) n += __popc(free_of(w));
  int at = scan_block(n, &all, part);
  for (int w = w0; w < w1; ++w)
    for (uint32_t f = free_of(w); f; f &= f - 1) a.free_pages[at++] = 32 * w + __builtin_ctz(f);
  for (int i = all + threadIdx.x; i < P; i += kMarkThreads) a.free_pages[i] = -1;
  if (threadIdx.x == 0) {
    a.counts[0] = all;
    a.counts[1] = P - all;
  }
}

// ---------------------------------------------------------------- compact
// Workspace: the number of live pages, the number of moves, and for each page at or
// behind that number where it goes (-1: nowhere); then the moves' sources and targets.
struct CompactArgs {
  TableArgs t;
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
  mark_pages(a.t, bits, words);
  const int per = (words + kMarkThreads - 1) / kMarkThreads;
  const int w0 = min((int)threadIdx.x * per, words), w1 = min(w0 + per, words);
  int x = 0, n, moves;
  for (int w = w0; w < w1; ++w) x += __popc(bits[w]);
  scan_block(x, &n, part);
  auto below = [&](int w) { return w < n >> 5 ? ~0u : (w == n >> 5 ? (1u << (n & 31)) - 1u : 0u); };   // pages of word w before n
  int holes = 0, far = 0;
  for (int w = w0; w < w1; ++w) {
    holes += __popc(~bits[w] & below(w));
    far += __popc(bits[w] & ~below(w));
  }
  int at_hole = scan_block(holes, &moves, part), at_far = scan_block(far, &moves, part);
  for (int w = w0; w < w1; ++w)
    for (uint32_t f = ~bits[w] & below(w); f; f &= f - 1) move_dst(a)[at_hole++] = 32 * w + __builtin_ctz(f);
  __syncthreads();
  for (int w = w0; w < w1; ++w)
    for (uint32_t f = bits[w] & ~below(w); f; f &= f - 1) {
      const int p = 32 * w + __builtin_ctz(f);
      move_to(a)[p] = move_dst(a)[at_far];
      move_src(a)[at_far++] = p;
    }
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
  for (int row = blockIdx.x; row < a.t.rows; row += gridDim.x) {
    const int held = held_pages(a.t, row);
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
size_t kv_compact_ws_bytes(int64_t num_pages) { return (size_t)(4 + num_pages + 2 * (num_pages / 2)) * 4; }

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
  a.slices = (int)(slices < 1 ? 1 : (slices > 64 ? 64 : slices));
  const uint32_t grid = num_forks == 0 ? 1u : (uint32_t)num_forks * (uint32_t)a.slices;
  hipLaunchKernelGGL(kv_fork_kernel, dim3(grid), dim3(kForkThreads), 0, stream, a);
  return launch_status("moe_kv_fork");
}

moe_status launch_kv_free_pages(const int32_t* table, int64_t stride, int rows, int max_blocks, const int32_t* lens,
                                int page_shift, int64_t num_pages, int32_t* free_pages, int32_t* counts, hipStream_t stream) {
  FreeArgs a;
  a.t = table_args(table, stride, rows, max_blocks, lens, page_shift, num_pages);
  a.free_pages = free_pages;
  a.counts = counts;
  hipLaunchKernelGGL(kv_free_kernel, dim3(1), dim3(kMarkThreads), 0, stream, a);
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
  a.ws = (int32_t*)ws;
  a.buffers = page_buffers(buffers, &a.page_bytes);
  hipLaunchKernelGGL(kv_compact_plan_kernel, dim3(1), dim3(kMarkThreads), 0, stream, a);
  moe_status st = launch_status("moe_kv_compact");
  if (st != MOE_OK) return st;
  hipLaunchKernelGGL(kv_compact_move_kernel, dim3(2048), dim3(256), 0, stream, a);
  return launch_status("moe_kv_compact");
}

}  // namespace moe
