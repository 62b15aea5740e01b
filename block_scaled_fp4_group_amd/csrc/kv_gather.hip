// Cached keys and values as contiguous rows, as attn_prompt takes them: row
// cu_k[b] + i of the outputs is key i of sequence b -- the shared prefix's keys first,
// then the request's own.  From a bf16 cache a copy, from one held in 4 bits the values
// that the codes stand for, code x scale x global, which bf16 holds exactly.
//
// Memory traffic is all there is.  A workgroup takes 32 rows of one head's keys or values:
// it finds their places, then its threads take 16 values each.  (With all heads of the rows
// to a workgroup 364 rows x 8 x 128 took 13 us, 11 times one after the other.)  9751 rows of 4 heads of
// 192 + 128: from 4 bits 13.5 us (32 MB, 2.4 TB/s), from bf16 11.4 us (50 MB, 4.4 TB/s), where a large copy
// reaches 5.1: a workgroup's search, table entry and rows follow one another, and a thread's two
// stores each fill half of the lines that they touch.
#include "common.h"

namespace moe {

constexpr int kGatherThreads = 256, kGatherRows = 32;

struct GatherArgs {
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_scale;                           // 4 bits: else null
  const uint8_t* v_scale;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* prefix_table;
  const int32_t* cu;
  int64_t prefix_len, total, num_pages;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t ko_ts, ko_hs, vo_ts, vo_hs;
  int32_t num_seqs, max_blocks, kv_heads, k_dim, v_dim, page_shift;
  float k_global, v_global;
};

// 16 codes times a scale (with its global) as 16 bf16
__device__ __forceinline__ void store_fp4(uint16_t* dst, u32x2 codes, float s) {
  const u32x2 a = nvfp4_dequant4(codes[0] & 0xFFFFu, s), b = nvfp4_dequant4(codes[0] >> 16, s);
  const u32x2 c = nvfp4_dequant4(codes[1] & 0xFFFFu, s), d = nvfp4_dequant4(codes[1] >> 16, s);
  *(u32x4*)dst = u32x4{a[0], a[1], b[0], b[1]};
  *(u32x4*)(dst + 8) = u32x4{c[0], c[1], d[0], d[1]};
}

template <bool FP4>
__global__ __launch_bounds__(kGatherThreads) void kv_gather_kernel(GatherArgs a) {
  __shared__ int64_t slots[kGatherRows];                            // page << page_shift | row in it; or:
  constexpr int64_t kNoPage = -1, kNoSequence = -2;
  const int kind = blockIdx.x & 1, h = (int)((blockIdx.x >> 1) % (uint32_t)a.kv_heads);
  const int64_t row0 = (int64_t)((blockIdx.x >> 1) / (uint32_t)a.kv_heads) * kGatherRows;
  const int64_t page_mask = ((int64_t)1 << a.page_shift) - 1;
  if (threadIdx.x < kGatherRows) {
    const int64_t row = row0 + threadIdx.x;
    int64_t slot = kNoSequence;
    // the last sequence that begins at or before the row (offsets are clamped, not descending)
    if (row < a.total && row >= a.cu[0] && row < a.cu[a.num_seqs]) {
      int lo = 0, hi = a.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= row) lo = mid;
        else hi = mid;
      }
      const int64_t i = row - a.cu[lo], key = i - a.prefix_len;
      const int64_t block = (key < 0 ? i : key) >> a.page_shift;
      int64_t page = -1;
      slot = kNoPage;
      if (key < 0) page = a.prefix_table[block];
      else if (block < a.max_blocks) page = a.table[lo * a.table_stride + block];
      if (page >= 0 && page < a.num_pages) slot = (page << a.page_shift) | ((key < 0 ? i : key) & page_mask);
    }
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
  const int rows = (int)min((int64_t)kGatherRows, a.total - row0);
  const int blocks = (kind == 0 ? a.k_dim : a.v_dim) / 16, dim = 16 * blocks;
  const uint8_t* from = kind == 0 ? a.k : a.v;
  uint16_t* to = kind == 0 ? a.k_out + row0 * a.ko_ts + h * a.ko_hs : a.v_out + row0 * a.vo_ts + h * a.vo_hs;
  const int64_t ts = kind == 0 ? a.ko_ts : a.vo_ts;
  for (int f = threadIdx.x; f < rows * blocks; f += kGatherThreads) {
    const int b = f % blocks, r = f / blocks;
    const int64_t slot = slots[r];
    uint16_t* dst = to + r * ts + 16 * b;
    if (slot == kNoSequence) continue;                              // the row is left as it was
    if (slot == kNoPage) {
      *(u32x4*)dst = *(u32x4*)(dst + 8) = u32x4{0u, 0u, 0u, 0u};   // not one of the cache's pages
    } else if (FP4) {
      const int64_t page = slot >> a.page_shift, in = slot & page_mask, head = page * a.kv_heads + h;
      const int64_t at = (head << a.page_shift) + in;
      const u32x2 codes = *(const u32x2*)(from + at * (dim / 2) + 8 * b);
      const uint8_t* s = kind == 0 ? a.k_scale + at * blocks + b : a.v_scale + ((head * blocks + b) << a.page_shift) + in;
      store_fp4(dst, codes, e4m3_to_f32(*s) * (kind == 0 ? a.k_global : a.v_global));
    } else {
      const uint16_t* src = (const uint16_t*)from + (slot * a.kv_heads + h) * dim + 16 * b;
      const u32x4 x = *(const u32x4*)src, y = *(const u32x4*)(src + 8);
      *(u32x4*)dst = x;
      *(u32x4*)(dst + 8) = y;
    }
  }
}

// workgroups (host: in 31 bits)
int64_t kv_gather_grid(int64_t total, int kv_heads) { return (total + kGatherRows - 1) / kGatherRows * kv_heads * 2; }

static GatherArgs gather_args(int kv_heads, int k_dim, int v_dim, const int32_t* table, int64_t table_stride, int max_blocks,
                              const int32_t* prefix_table, int64_t prefix_len, const int32_t* cu, int num_seqs,
                              int64_t total, const moe_heads& k_out, const moe_heads& v_out) {
  GatherArgs a = {};
  a.table = table;
  a.table_stride = table_stride;
  a.prefix_table = prefix_table;
  a.cu = cu;
  a.prefix_len = prefix_len;
  a.total = total;
  a.k_out = (uint16_t*)k_out.data;
  a.ko_ts = k_out.token_stride;
  a.ko_hs = k_out.head_stride;
  a.v_out = (uint16_t*)v_out.data;
  a.vo_ts = v_out.token_stride;
  a.vo_hs = v_out.head_stride;
  a.num_seqs = num_seqs;
  a.max_blocks = max_blocks;
  a.kv_heads = kv_heads;
  a.k_dim = k_dim;
  a.v_dim = v_dim;
  return a;
}

moe_status launch_kv_gather(const moe_kv_cache& c, int kv_heads, int k_dim, int v_dim, const int32_t* table,
                            int64_t table_stride, int max_blocks, const int32_t* prefix_table, int64_t prefix_len,
                            const int32_t* cu, int num_seqs, int64_t total, const moe_heads& k_out, const moe_heads& v_out,
                            hipStream_t stream) {
  GatherArgs a = gather_args(kv_heads, k_dim, v_dim, table, table_stride, max_blocks, prefix_table, prefix_len, cu, num_seqs,
                             total, k_out, v_out);
  a.k = (const uint8_t*)c.k;
  a.v = (const uint8_t*)c.v;
  a.num_pages = c.num_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  hipLaunchKernelGGL(kv_gather_kernel<false>, dim3((uint32_t)kv_gather_grid(total, kv_heads)), dim3(kGatherThreads), 0, stream, a);
  return launch_status("moe_kv_gather");
}

moe_status launch_kv_gather_fp4(const moe_kv_cache_fp4& c, int kv_heads, int k_dim, int v_dim, const int32_t* table,
                                int64_t table_stride, int max_blocks, const int32_t* prefix_table, int64_t prefix_len,
                                const int32_t* cu, int num_seqs, int64_t total, const moe_heads& k_out,
                                const moe_heads& v_out, hipStream_t stream) {
  GatherArgs a = gather_args(kv_heads, k_dim, v_dim, table, table_stride, max_blocks, prefix_table, prefix_len, cu, num_seqs,
                             total, k_out, v_out);
  a.k = (const uint8_t*)c.k;
  a.v = (const uint8_t*)c.v;
  a.k_scale = (const uint8_t*)c.k_scale;
  a.v_scale = (const uint8_t*)c.v_scale;
  a.num_pages = c.num_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.k_global = c.k_global;
  a.v_global = c.v_global;
  hipLaunchKernelGGL(kv_gather_kernel<true>, dim3((uint32_t)kv_gather_grid(total, kv_heads)), dim3(kGatherThreads), 0, stream, a);
  return launch_status("moe_kv_gather_fp4");
}

}  // namespace moe
