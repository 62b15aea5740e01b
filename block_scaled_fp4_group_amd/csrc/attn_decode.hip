// Attention of one new token per request over a paged cache, with a prefix that
// all requests share.
//
//   out[b, h] = sum_j p_j v_j over the prefix's keys and request b's own keys,
//   p = softmax of q[b, h] . k_j * scale over both together.
//
// Split over the keys: the prefix's keys meet the query rows of every request
// (B * G rows per key head, G query heads each) in one product, the own keys of
// a request only its G rows.  Each part leaves its unnormalised sum, maximum and
// weight sum in float; a second kernel joins the parts of a row:
//   M = max m_i,  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// With a single part the first kernel writes the result itself.
//
// A workgroup's four waves take every fourth tile of 32 keys for the same 32
// query rows, each from its own LDS, and join their sums at the end.
#include "attn_common.h"

namespace moe {

constexpr int kDecWaves = 4;
constexpr int kDecThreads = kDecWaves * 64;
constexpr int kDecKeys = 32;                        // per wave and tile
constexpr int kDecStep = kDecWaves * kDecKeys;      // per workgroup and round

struct DecodePlan {
  int64_t chunk_p, chunk_s;                         // keys per part
  int32_t parts_p, parts_s;                         // parts of the prefix, of a request's own keys
  int32_t blocks_p, blocks_s;                       // 32-row blocks of B * G rows, of G rows
};

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* prefix_table;
  int64_t prefix_len, max_len;
  uint16_t* out;
  float* lse;
  float* part_o;                                    // [parts][B * Hq][DV]
  float2* part_ml;                                  // [parts][B * Hq]: maximum (base 2), weight sum
  int32_t num_requests, q_heads, kv_heads, num_pages, page_shift;
  float c;
  DecodePlan plan;
};

__device__ __forceinline__ int64_t own_len(const DecodeArgs& a, int b) {
  return min(max((int64_t)a.lens[b], (int64_t)0), a.max_len);
}

template <int DQ, int DV>
__global__ __launch_bounds__(kDecThreads) void attn_decode_kernel(DecodeArgs a) {
  using W = AttnWave<DQ, DV, 1>;
  constexpr int kTile = W::kKeyBytes + W::kValBytes;
  static_assert(kTile >= 32 * DV * 4, "a wave's tile memory holds its sums");
  __shared__ __attribute__((aligned(16))) uint8_t mem[kDecWaves][kTile];
  __shared__ float2 ml[kDecWaves][32];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, h = lane >> 5, r = lane & 31;
  const int G = a.q_heads / a.kv_heads;
  const int kvh = blockIdx.x % a.kv_heads;
  int64_t item = blockIdx.x / a.kv_heads;
  const int64_t prefix_items = (int64_t)a.plan.parts_p * a.plan.blocks_p;
  // this workgroup's rows (request row / G, head row % G from row0 on), keys and part
  const int32_t* table;
  int64_t key0, key1, rows, row0;
  int b0, part;
  if (item < prefix_items) {
    part = (int)(item / a.plan.blocks_p);
    row0 = (item % a.plan.blocks_p) * 32;
    rows = (int64_t)a.num_requests * G;
    b0 = 0;
    table = a.prefix_table;
    key0 = part * a.plan.chunk_p;
    key1 = min(key0 + a.plan.chunk_p, a.prefix_len);
  } else {
    item -= prefix_items;
    const int s = (int)(item % a.plan.parts_s);
    item /= a.plan.parts_s;
    row0 = (item % a.plan.blocks_s) * 32;
    b0 = (int)(item / a.plan.blocks_s);
    rows = G;
    part = a.plan.parts_p + s;
    table = a.table + b0 * a.table_stride;
    key0 = s * a.plan.chunk_s;
    key1 = min(key0 + a.plan.chunk_s, own_len(a, b0));
    // nothing here: the joining kernel skips the part (a single part of a request
    // without keys still writes its empty row)
    if (key1 <= key0 && a.part_o) return;
  }
  const int64_t row = min(row0 + r, rows - 1);
  const int b = b0 + (int)(row / G), hq = kvh * G + (int)(row % G);
  W w;
  w.init(a.q + b * a.q_ts + hq * a.q_hs, lane);
  uint8_t* ks = mem[wv];
  uint8_t* vs = mem[wv] + W::kKeyBytes;
  for (int64_t t0 = key0 + wv * kDecKeys; t0 < key1; t0 += kDecStep) {
    // the row of the cache that holds key t0 + r (keys past the end: the last)
    const int64_t key = min(t0 + r, key1 - 1);
    const int page = min(max(table[key >> a.page_shift], 0), a.num_pages - 1);
    const int slot = (int)(((int64_t)page << a.page_shift) + (key & (((int64_t)1 << a.page_shift) - 1)));
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < W::kKeyBytes / 1024; ++i) {
      constexpr int C = DQ / 8;
      const int f = i * 64 + lane, kr = f / C, ch = f % C;
      const int64_t at = ((int64_t)__shfl(slot, kr) * a.kv_heads + kvh) * DQ + ch * 8;
      *(u32x4*)(ks + kr * (DQ * 2) + (ch ^ at_swz<DQ>(kr)) * 16) = *(const u32x4*)(a.k_cache + at);
    }
#pragma unroll
    for (int i = 0; i < W::kValBytes / 1024; ++i) {
      constexpr int C = DV / 8;
      const int f = i * 64 + lane, kr = f / C, ch = f % C;
      const int64_t at = ((int64_t)__shfl(slot, kr) * a.kv_heads + kvh) * DV + ch * 8;
      *(u32x4*)(vs + kr * (DV * 2) + (ch ^ at_swz<DV>(kr)) * 16) = *(const u32x4*)(a.v_cache + at);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (t0 + kDecKeys <= key1) w.tile(ks, vs, a.c);
    else w.tile_masked(ks, vs, lane, a.c, (int)(key1 - 1 - t0));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // join the four waves: 4 floats of a row at a time, chunks spread over the banks
  constexpr int kChunks = DV / 4;
  auto at = [](int rr, int ch) { return rr * kChunks + (ch ^ (rr & (kChunks - 1))); };
  f32x4* mine = (f32x4*)mem[wv];
#pragma unroll
  for (int ob = 0; ob < W::OB; ++ob)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mine[at(r, 8 * ob + 2 * i + h)] = f32x4{w.o[ob][4 * i], w.o[ob][4 * i + 1], w.o[ob][4 * i + 2], w.o[ob][4 * i + 3]};
  if (h == 0) ml[wv][r] = float2{w.m, w.l};
  __syncthreads();
  const int64_t Hall = (int64_t)a.num_requests * a.q_heads;
  for (int f = threadIdx.x; f < 32 * kChunks; f += kDecThreads) {
    const int rr = f / kChunks, ch = f % kChunks;
    if (row0 + rr >= rows) continue;
    float M = neg_inf();
#pragma unroll
    for (int i = 0; i < kDecWaves; ++i) M = fmaxf(M, ml[i][rr].x);
    const float base = M == neg_inf() ? 0.0f : M;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float L = 0.0f;
#pragma unroll
    for (int i = 0; i < kDecWaves; ++i) {
      // a wave without keys for the row has m = -inf, weight 0 and sums of 0
      const float e = __builtin_amdgcn_exp2f(ml[i][rr].x - base);
      L = fmaf(e, ml[i][rr].y, L);
      const f32x4 x = ((const f32x4*)mem[i])[at(rr, ch)];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(e, x[j], o[j]);
    }
    const int bb = b0 + (int)((row0 + rr) / G), hh = kvh * G + (int)((row0 + rr) % G);
    const int64_t at_row = (int64_t)bb * a.q_heads + hh;
    if (a.part_o) {
      *(f32x4*)(a.part_o + (part * Hall + at_row) * DV + ch * 4) = o;
      if (ch == 0) a.part_ml[part * Hall + at_row] = float2{M, L};
    } else {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      *(u32x2*)(a.out + bb * a.o_ts + hh * a.o_hs + ch * 4) =
          u32x2{cvt_bf16x2(o[0] * inv, o[1] * inv), cvt_bf16x2(o[2] * inv, o[3] * inv)};
      if (a.lse && ch == 0) a.lse[at_row] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
    }
  }
}

// One workgroup per output row: its four waves take every fourth part.
template <int DV>
__global__ __launch_bounds__(kDecThreads) void attn_join_kernel(DecodeArgs a) {
  __shared__ float red[kDecWaves][DV];
  __shared__ float2 ml[kDecWaves];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t Hall = (int64_t)a.num_requests * a.q_heads, at_row = blockIdx.x;
  const int b = (int)(at_row / a.q_heads), hq = (int)(at_row % a.q_heads);
  const int64_t len = own_len(a, b);
  const int n = a.plan.parts_p + (int)((len + a.plan.chunk_s - 1) / a.plan.chunk_s);
  float M = neg_inf(), L = 0.0f, o[DV / 64];
#pragma unroll
  for (int j = 0; j < DV / 64; ++j) o[j] = 0.0f;
  for (int p = wv; p < n; p += kDecWaves) {
    const float2 x = a.part_ml[p * Hall + at_row];
    const float M1 = fmaxf(M, x.x), base = M1 == neg_inf() ? 0.0f : M1;
    const float e0 = __builtin_amdgcn_exp2f(M - base), e1 = __builtin_amdgcn_exp2f(x.x - base);
    L = fmaf(L, e0, x.y * e1);
    const float* src = a.part_o + (p * Hall + at_row) * DV + lane * (DV / 64);
#pragma unroll
    for (int j = 0; j < DV / 64; ++j) o[j] = fmaf(o[j], e0, src[j] * e1);
    M = M1;
  }
#pragma unroll
  for (int j = 0; j < DV / 64; ++j) red[wv][lane * (DV / 64) + j] = o[j];
  if (lane == 0) ml[wv] = float2{M, L};
  __syncthreads();
  if (threadIdx.x >= DV / 2) return;
  float M1 = neg_inf(), L1 = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
  for (int i = 0; i < kDecWaves; ++i) M1 = fmaxf(M1, ml[i].x);
  const float base = M1 == neg_inf() ? 0.0f : M1;
#pragma unroll
  for (int i = 0; i < kDecWaves; ++i) {
    const float e = __builtin_amdgcn_exp2f(ml[i].x - base);
    L1 = fmaf(e, ml[i].y, L1);
    x0 = fmaf(e, red[i][2 * threadIdx.x], x0);
    x1 = fmaf(e, red[i][2 * threadIdx.x + 1], x1);
  }
  const float inv = L1 == 0.0f ? 0.0f : 1.0f / L1;
  *(uint32_t*)(a.out + b * a.o_ts + hq * a.o_hs + 2 * threadIdx.x) = cvt_bf16x2(x0 * inv, x1 * inv);
  if (a.lse && threadIdx.x == 0) a.lse[at_row] = L1 == 0.0f ? neg_inf() : (M1 + __builtin_amdgcn_logf(L1)) * kLn2;
}

static DecodePlan decode_plan(int64_t B, int q_heads, int kv_heads, int64_t prefix_len, int64_t max_len) {
  DecodePlan p;
  const int G = q_heads / kv_heads;
  p.blocks_p = (int32_t)((B * G + 31) / 32);
  p.blocks_s = (G + 31) / 32;
  // keys per workgroup so that about 1024 workgroups share the work
  const int64_t work = kv_heads * (prefix_len * p.blocks_p + B * max_len * p.blocks_s);
  int64_t chunk = (work / 1024 + kDecStep - 1) / kDecStep * kDecStep;
  if (chunk < 2 * kDecStep) chunk = 2 * kDecStep;
  p.chunk_p = p.chunk_s = chunk;
  p.parts_p = (int32_t)((prefix_len + chunk - 1) / chunk);
  p.parts_s = (int32_t)((max_len + chunk - 1) / chunk);
  if (p.parts_p + p.parts_s == 0) p.parts_s = 1;      // no key anywhere: the single part writes the empty rows
  return p;
}

size_t attn_decode_ws_bytes(int64_t B, int q_heads, int kv_heads, int v_dim, int64_t prefix_len, int64_t max_len) {
  const DecodePlan p = decode_plan(B, q_heads, kv_heads, prefix_len, max_len);
  const size_t parts = (size_t)p.parts_p + (size_t)p.parts_s;
  return parts <= 1 ? 0 : parts * (size_t)B * (size_t)q_heads * ((size_t)v_dim * 4 + 8);
}

static int64_t plan_grid(const DecodePlan& p, int64_t B, int kv_heads) {
  return ((int64_t)p.parts_p * p.blocks_p + B * p.blocks_s * p.parts_s) * kv_heads;
}

int64_t attn_decode_grid(int64_t B, int q_heads, int kv_heads, int64_t prefix_len, int64_t max_len) {
  return plan_grid(decode_plan(B, q_heads, kv_heads, prefix_len, max_len), B, kv_heads);
}

template <int DQ, int DV>
static void launch_decode(const DecodeArgs& a, hipStream_t stream) {
  const uint32_t grid = (uint32_t)plan_grid(a.plan, a.num_requests, a.kv_heads);
  hipLaunchKernelGGL((attn_decode_kernel<DQ, DV>), dim3(grid), dim3(kDecThreads), 0, stream, a);
  if (a.part_o)
    hipLaunchKernelGGL((attn_join_kernel<DV>), dim3((uint32_t)(a.num_requests * a.q_heads)), dim3(kDecThreads), 0,
                       stream, a);
}

moe_status launch_attn_decode(const moe_heads& q, const moe_kv_cache& cache, const int32_t* table,
                              int64_t table_stride, const int32_t* lens, int64_t B, int64_t max_len,
                              const int32_t* prefix_table, int64_t prefix_len, const moe_attn_params& p,
                              const moe_heads& out, float* lse, void* ws, hipStream_t stream) {
  DecodeArgs a;
  a.q = (const uint16_t*)q.data;
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.out = (uint16_t*)out.data;
  a.o_ts = out.token_stride;
  a.o_hs = out.head_stride;
  a.k_cache = (const uint16_t*)cache.k;
  a.v_cache = (const uint16_t*)cache.v;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.max_len = max_len;
  a.lse = lse;
  a.num_requests = (int32_t)B;
  a.q_heads = p.q_heads;
  a.kv_heads = p.kv_heads;
  a.num_pages = (int32_t)cache.num_pages;
  a.page_shift = __builtin_ctz((unsigned)cache.page_size);
  a.c = p.scale * kLog2e;
  a.plan = decode_plan(B, p.q_heads, p.kv_heads, prefix_len, max_len);
  const int64_t parts = (int64_t)a.plan.parts_p + a.plan.parts_s;
  // (the sums first: they keep their 16-byte alignment)
  a.part_o = parts > 1 ? (float*)ws : nullptr;
  a.part_ml = parts > 1 ? (float2*)(a.part_o + parts * B * p.q_heads * p.v_dim) : nullptr;
  if (p.k_dim == 64) launch_decode<64, 64>(a, stream);
  else if (p.k_dim == 128) launch_decode<128, 128>(a, stream);
  else launch_decode<192, 128>(a, stream);
  return launch_status("moe_attn_decode");
}

}  // namespace moe
