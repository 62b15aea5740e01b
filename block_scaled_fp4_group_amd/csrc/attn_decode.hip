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
// Workgroups of four waves walk the keys in tiles through LDS stages that all
// waves fill (direct loads; every lane finds its rows through the block table)
// while another is computed on:
//   wide   (prefix, many rows): 128 rows, 32 per wave; the prefix is read once
//          per 128 rows.  Bound by the matrix cores.
//   narrow (own keys, and a prefix with few rows): 64 rows, two waves per 32.
//          Bound by reading the cache.
// Both kinds run in one launch, their workgroups interleaved, so that the one's
// matrix work and the other's reads share the chip.
#include <algorithm>

#include "attn_common.h"

namespace moe {

constexpr int kDecThreads = 256;
constexpr int kDecKeys = 64;

struct DecodePlan {
  int32_t wide;                                     // prefix workgroups are wide
  int32_t chunk_p, chunk_s;                         // tiles per part
  int32_t parts_p, parts_s;                         // parts of the prefix, of a request's own keys
  int32_t blocks_p, blocks_s;                       // row blocks of B * G rows, of G rows
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

// One workgroup's share: rows row0 .. of `rows` (row r is request b0 + r / G, its
// head r % G of key head kvh) against keys key0 .. key1 - 1 of `table`.
struct DecodeItem {
  const int32_t* table;
  int64_t key0, key1, row0, rows;
  int b0, kvh, part;
};

// The row of the cache that key `key` of an item sits in; e: its table entry.
__device__ __forceinline__ int cache_row(const DecodeArgs& a, int e, int64_t key) {
  return (int)(((int64_t)min(max(e, 0), a.num_pages - 1) << a.page_shift) +
               (key & (((int64_t)1 << a.page_shift) - 1)));
}

// A wave's 32 rows finished: its part, or the result itself.
template <class W, int DV>
__device__ __forceinline__ void store_rows(const DecodeArgs& a, const DecodeItem& it, const W& w, int b, int hq, int h) {
  const int64_t at_row = (int64_t)b * a.q_heads + hq;
  if (a.part_o) {
    const int64_t at = (int64_t)it.part * a.num_requests * a.q_heads + at_row;
    float* po = a.part_o + at * DV + 4 * h;
#pragma unroll
    for (int x = 0; x < W::OB; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(f32x4*)(po + 32 * x + 8 * i) = f32x4{w.o[x][4 * i], w.o[x][4 * i + 1], w.o[x][4 * i + 2], w.o[x][4 * i + 3]};
    if (h == 0) a.part_ml[at] = float2{w.m, w.l};
  } else {
    const float inv = w.l == 0.0f ? 0.0f : 1.0f / w.l;
    uint16_t* op = a.out + b * a.o_ts + hq * a.o_hs + 4 * h;
#pragma unroll
    for (int x = 0; x < W::OB; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(u32x2*)(op + 32 * x + 8 * i) = u32x2{cvt_bf16x2(w.o[x][4 * i] * inv, w.o[x][4 * i + 1] * inv),
                                               cvt_bf16x2(w.o[x][4 * i + 2] * inv, w.o[x][4 * i + 3] * inv)};
    if (a.lse && h == 0) a.lse[at_row] = w.l == 0.0f ? neg_inf() : (w.m + __builtin_amdgcn_logf(w.l)) * kLn2;
  }
}

// 128 rows, 32 per wave; tiles of 64 keys in two stages.
template <int DQ, int DV>
__device__ __forceinline__ void decode_wide(const DecodeArgs& a, const DecodeItem& it, uint8_t* mem) {
  using W = AttnWave<DQ, DV, 2>;
  constexpr int kKeys = 64;
  uint8_t* ks = mem;
  uint8_t* vs = mem + 2 * W::kKeyBytes;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  const int64_t wrow = it.row0 + wv * 32;                           // this wave's first row
  const bool active = wrow < it.rows;
  const int64_t row = min(wrow + (lane & 31), it.rows - 1);
  const int b = it.b0 + (int)(row / G), hq = it.kvh * G + (int)(row % G);
  W w;
  w.init(a.q + b * a.q_ts + hq * a.q_hs, lane);
  // Lane l looks up the cache row of key l of a tile (past the end: the last
  // key), one tile ahead of the loads that use it: the table entry of tile t + 2
  // is read when the loads of tile t + 1 go out.
  const int64_t n_keys = it.key1 - it.key0;
  const int n_tiles = (int)((n_keys + kKeys - 1) / kKeys), n_whole = (int)(n_keys / kKeys);
  auto key_of = [&](int t) { return min(it.key0 + (int64_t)t * kKeys + lane, it.key1 - 1); };
  auto entry = [&](int t) { return it.table[key_of(t) >> a.page_shift]; };
  const uint32_t k_lds = at_lds_addr(ks) + (uint32_t)wv * 1024u, v_lds = at_lds_addr(vs) + (uint32_t)wv * 1024u;
  const uint8_t* kc = (const uint8_t*)(a.k_cache + (int64_t)it.kvh * DQ);
  const uint8_t* vc = (const uint8_t*)(a.v_cache + (int64_t)it.kvh * DV);
  const int64_t k_row = (int64_t)a.kv_heads * DQ * 2, v_row = (int64_t)a.kv_heads * DV * 2;
  auto load = [&](int slot, int st) {
#pragma unroll
    for (int i = 0; i < W::kKeyBytes / 16 / kDecThreads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DQ / 8);
      at_load_lds(k_lds + (uint32_t)(st * W::kKeyBytes + i * kDecThreads * 16),
                  kc + (int64_t)__shfl(slot, r) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < W::kValBytes / 16 / kDecThreads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DV / 8);
      at_load_lds(v_lds + (uint32_t)(st * W::kValBytes + i * kDecThreads * 16),
                  vc + (int64_t)__shfl(slot, r) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16);
    }
  };
  load(cache_row(a, entry(0), key_of(0)), 0);
  int next = entry(1);
  auto step = [&](auto stage, auto whole, int t) {
    constexpr int st = decltype(stage)::value;
    const uint8_t* k = ks + st * W::kKeyBytes;
    const uint8_t* v = vs + st * W::kValBytes;
    // tile t has landed; everyone is done with tile t - 1, whose stage the next loads refill
    at_wait_barrier<0>();
    if (t + 1 < n_tiles) {
      load(cache_row(a, next, key_of(t + 1)), st ^ 1);
      next = entry(t + 2);
    }
    if (!active) return;
    if (decltype(whole)::value) w.tile(k, v, a.c);
    else w.tile_masked(k, v, lane, a.c, (int)min(n_keys - 1 - (int64_t)t * kKeys, (int64_t)kKeys));
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  int t = 0;
  for (; t + 1 < n_whole; t += 2) {
    step(S0(), std::true_type(), t);
    step(S1(), std::true_type(), t + 1);
  }
  for (; t < n_tiles; t += 2) {
    step(S0(), std::false_type(), t);
    if (t + 1 < n_tiles) step(S1(), std::false_type(), t + 1);
  }
  if (wrow + (lane & 31) < it.rows) store_rows<W, DV>(a, it, w, b, hq, h);
}

// 64 rows: waves 0, 1 the first 32, waves 2, 3 the others; even waves compute
// the even tiles of 32 keys, odd waves the odd ones, and the two sums are joined
// at the end.  The reads are what counts: NS stages, so that while one tile is
// computed on NS - 1 are under way (at two workgroups per CU 96 KB: with 64 KB a
// CU the reads of one 131072-key request ran at 5.6 TB/s).
//
// Loads in order of issue, per wave: D(t), the rows of tile t, L of them; E(t),
// the table entries of tile t, one load, into a ring in LDS.  Step t waits for
// D(t) and E(t + NS - 1), issues D(t + NS - 1) and E(t + 2 NS - 2): the waited-for
// pair went out together in step t - NS + 1, so the NS - 2 pairs issued since may
// be in flight.  Near the end fewer are.
template <int DQ, int DV, int NS>
__device__ __forceinline__ void decode_narrow(const DecodeArgs& a, const DecodeItem& it, uint8_t* mem) {
  using W = AttnWave<DQ, DV, 1>;
  constexpr int kKeys = 32, kRing = 2 * NS;                         // entries live 2 NS - 2 steps
  constexpr int kKeyLoads = W::kKeyBytes / 16 / kDecThreads, kValLoads = W::kValBytes / 16 / kDecThreads;
  constexpr int L = kKeyLoads + kValLoads + 1;
  uint8_t* ks = mem;
  uint8_t* vs = ks + NS * W::kKeyBytes;
  const int* ring = (const int*)(vs + NS * W::kValBytes);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int rb = wv >> 1, odd = wv & 1;
  const int G = a.q_heads / a.kv_heads;
  const int64_t wrow = it.row0 + rb * 32;                           // this wave's first row
  const bool active = wrow < it.rows;
  const int64_t row = min(wrow + (lane & 31), it.rows - 1);
  const int b = it.b0 + (int)(row / G), hq = it.kvh * G + (int)(row % G);
  const int64_t n_keys = it.key1 - it.key0;
  const int n_tiles = (int)((n_keys + kKeys - 1) / kKeys);
  const uint32_t k_lds = at_lds_addr(ks) + (uint32_t)wv * 1024u, v_lds = at_lds_addr(vs) + (uint32_t)wv * 1024u;
  const uint8_t* kc = (const uint8_t*)(a.k_cache + (int64_t)it.kvh * DQ);
  const uint8_t* vc = (const uint8_t*)(a.v_cache + (int64_t)it.kvh * DV);
  const int64_t k_row = (int64_t)a.kv_heads * DQ * 2, v_row = (int64_t)a.kv_heads * DV * 2;
  auto key_of = [&](int t, int r) { return min(it.key0 + (int64_t)t * kKeys + r, it.key1 - 1); };   // past the end: the last
  // (every wave fetches all entries itself: it then need not wait for another's)
  auto fetch = [&](int t) {
    at_load_lds4(at_lds_addr(ring) + (uint32_t)(t % kRing) * 256u, it.table + (key_of(t, lane & 31) >> a.page_shift));
  };
  auto load = [&](int t) {
    const int st = t % NS;
    const int* e = ring + (t % kRing) * 64;
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DQ / 8);
      at_load_lds(k_lds + (uint32_t)(st * W::kKeyBytes + i * kDecThreads * 16),
                  kc + cache_row(a, e[r], key_of(t, r)) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DV / 8);
      at_load_lds(v_lds + (uint32_t)(st * W::kValBytes + i * kDecThreads * 16),
                  vc + cache_row(a, e[r], key_of(t, r)) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16);
    }
  };
  W w;
  if (n_tiles > 0)
    for (int t = 0; t < NS - 1; ++t) fetch(t);
  w.init(a.q + b * a.q_ts + hq * a.q_hs, lane);                     // (waits for the first entries too)
  if (n_tiles > 0) {
    at_wait<0>();
    for (int t = 0; t < NS - 1; ++t) {
      if (t < n_tiles) load(t);
      fetch(t + NS - 1);
    }
  }
  static_assert(NS == 3 || NS == 4, "the waits below");
  auto arrive = [&](int t) {
    // pairs issued after tile t's: NS - 2, at the end as many as tiles are left
    const int after = min(n_tiles - 1 - t, NS - 2);
    if (after == 0) at_wait_barrier<0>();
    else if (after == 1) at_wait_barrier<L>();
    else at_wait_barrier<2 * L>();
    if (t + NS - 1 < n_tiles) {
      load(t + NS - 1);
      fetch(t + 2 * NS - 2);
    }
  };
  const int n_whole = (int)(n_keys / kKeys);
  for (int t = 0; t < n_whole; ++t) {
    arrive(t);
    if (active && (t & 1) == odd) w.tile(ks + (t % NS) * W::kKeyBytes, vs + (t % NS) * W::kValBytes, a.c);
  }
  if (n_tiles > n_whole) {                                          // the last one, cut
    const int t = n_whole;
    arrive(t);
    if (active && (t & 1) == odd)
      w.tile_masked(ks + (t % NS) * W::kKeyBytes, vs + (t % NS) * W::kValBytes, lane, a.c,
                    (int)(n_keys - 1 - (int64_t)t * kKeys));
  }
  // The odd waves' sums reach the even ones through the tiles' memory (same rows
  // and columns in the same lanes).
  at_wait_barrier<0>();
  f32x4* box = (f32x4*)(mem + rb * (W::OB * 4 + 1) * 1024);
  if (odd) {
#pragma unroll
    for (int x = 0; x < W::OB; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        box[(4 * x + i) * 64 + lane] = f32x4{w.o[x][4 * i], w.o[x][4 * i + 1], w.o[x][4 * i + 2], w.o[x][4 * i + 3]};
    box[W::OB * 4 * 64 + lane] = f32x4{w.m, w.l, 0.0f, 0.0f};
  }
  at_wait_barrier<0>();
  if (odd) return;
  const f32x4 ml = box[W::OB * 4 * 64 + lane];
  const float M = fmaxf(w.m, ml[0]), base = M == neg_inf() ? 0.0f : M;
  const float e0 = __builtin_amdgcn_exp2f(w.m - base), e1 = __builtin_amdgcn_exp2f(ml[0] - base);
  w.m = M;
  w.l = w.l * e0 + ml[1] * e1;
#pragma unroll
  for (int x = 0; x < W::OB; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 y = box[(4 * x + i) * 64 + lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) w.o[x][4 * i + j] = w.o[x][4 * i + j] * e0 + y[j] * e1;
    }
  if (wrow + (lane & 31) < it.rows) store_rows<W, DV>(a, it, w, b, hq, h);
}

template <int DQ, int DV>
__global__ __launch_bounds__(kDecThreads, 2) void attn_decode_kernel(DecodeArgs a) {
  // stages of 32 keys and the ring of table entries; two workgroups fit a CU's 160 KB
  constexpr int kTile = 32 * (DQ + DV) * 2, NS = 4 * kTile + 2048 <= 80 * 1024 ? 4 : 3;
  constexpr int kNarrow = NS * kTile + 2 * NS * 256, kWide = 4 * kTile;
  __shared__ __attribute__((aligned(16))) uint8_t mem[kNarrow > kWide ? kNarrow : kWide];
  const DecodePlan& p = a.plan;
  DecodeItem it;
  it.kvh = blockIdx.x % a.kv_heads;
  const int64_t i = blockIdx.x / (uint32_t)a.kv_heads;
  const int64_t np = (int64_t)p.parts_p * p.blocks_p, n = np + (int64_t)a.num_requests * p.blocks_s * p.parts_s;
  const int64_t ip = i * np / n;                                    // prefix items spread evenly over the launch
  if ((i + 1) * np / n != ip) {
    // row blocks of one part side by side: they share the part's keys in L2
    it.part = (int)(ip / p.blocks_p);
    it.row0 = (ip % p.blocks_p) * (p.wide ? 128 : 64);
    it.rows = (int64_t)a.num_requests * (a.q_heads / a.kv_heads);
    it.b0 = 0;
    it.table = a.prefix_table;
    it.key0 = (int64_t)it.part * p.chunk_p * kDecKeys;
    it.key1 = min(it.key0 + (int64_t)p.chunk_p * kDecKeys, a.prefix_len);
    if (p.wide) return decode_wide<DQ, DV>(a, it, mem);
  } else {
    // first parts of all requests first: later ones may not exist
    int64_t is = i - ip;
    const int s = (int)(is / ((int64_t)a.num_requests * p.blocks_s));
    is %= (int64_t)a.num_requests * p.blocks_s;
    it.row0 = (is % p.blocks_s) * 64;
    it.b0 = (int)(is / p.blocks_s);
    it.rows = a.q_heads / a.kv_heads;
    it.part = p.parts_p + s;
    it.table = a.table + it.b0 * a.table_stride;
    it.key0 = (int64_t)s * p.chunk_s * kDecKeys;
    it.key1 = min(it.key0 + (int64_t)p.chunk_s * kDecKeys, own_len(a, it.b0));
    // nothing here: the joining kernel skips the part (a single part of a request
    // without keys still writes its empty row)
    if (it.key1 <= it.key0) {
      if (a.part_o) return;
      it.key1 = it.key0;
    }
  }
  decode_narrow<DQ, DV, NS>(a, it, mem);
}

// The parts of an output row joined: WPR waves per row take every WPR-th part.
// Each wave first finds its parts' maximum (64 parts at a time, one per lane), so
// the sums' loads follow without waiting for one another.
template <int DV, int WPR>
__global__ __launch_bounds__(WPR <= 4 ? 256 : WPR * 64) void attn_join_kernel(DecodeArgs a) {
  constexpr int kWaves = WPR <= 4 ? 4 : WPR, kRows = kWaves / WPR;
  __shared__ float2 red[kWaves][64];
  __shared__ float2 ml[kWaves];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = wv % WPR;
  const int64_t Hall = (int64_t)a.num_requests * a.q_heads;
  const int64_t at_row = (int64_t)blockIdx.x * kRows + wv / WPR;
  const bool live = at_row < Hall;                                  // whole waves; a row's waves agree
  constexpr int E = DV / 64;                                        // values per lane
  float M = neg_inf(), L = 0.0f, o[2] = {0.0f, 0.0f};
  if (live) {
    const int b = (int)(at_row / a.q_heads);
    const int64_t chunk = (int64_t)a.plan.chunk_s * kDecKeys;
    const int n = a.plan.parts_p + (int)((own_len(a, b) + chunk - 1) / chunk);
    const int mine = (n - sub + WPR - 1) / WPR;                     // parts sub, sub + WPR, ...
    for (int base = 0; base < mine; base += 64) {
      const int cnt = min(64, mine - base);
      float2 x = float2{neg_inf(), 0.0f};
      if (lane < cnt) x = a.part_ml[(int64_t)(sub + (base + lane) * WPR) * Hall + at_row];
      float mx = x.x;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
      const float M1 = fmaxf(M, mx), ref = M1 == neg_inf() ? 0.0f : M1;
      const float e = __builtin_amdgcn_exp2f(x.x - ref), e0 = __builtin_amdgcn_exp2f(M - ref);
      float l = x.y * e;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) l += __shfl_xor(l, d);
      L = L * e0 + l;
      M = M1;
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] *= e0;
      for (int p = 0; p < cnt; p += 8) {                            // 8 loads in flight
        float y[8][2];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int q = min(p + u, cnt - 1);
          const float* src = a.part_o + ((int64_t)(sub + (base + q) * WPR) * Hall + at_row) * DV + lane * E;
          y[u][0] = src[0];
          if (E == 2) y[u][1] = src[1];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (p + u >= cnt) break;
          const float ep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), p + u));
          o[0] = fmaf(ep, y[u][0], o[0]);
          if (E == 2) o[1] = fmaf(ep, y[u][1], o[1]);
        }
      }
    }
  }
  if (WPR > 1) {
    red[wv][lane] = float2{o[0], o[1]};
    if (lane == 0) ml[wv] = float2{M, L};
    __syncthreads();
    if (sub != 0) return;
    float M1 = M;
#pragma unroll
    for (int i = 1; i < WPR; ++i) M1 = fmaxf(M1, ml[wv + i].x);
    const float ref = M1 == neg_inf() ? 0.0f : M1;
    float e = __builtin_amdgcn_exp2f(M - ref);
    L *= e;
    o[0] *= e;
    o[1] *= e;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      e = __builtin_amdgcn_exp2f(ml[wv + i].x - ref);
      const float2 y = red[wv + i][lane];
      L = fmaf(e, ml[wv + i].y, L);
      o[0] = fmaf(e, y.x, o[0]);
      o[1] = fmaf(e, y.y, o[1]);
    }
    M = M1;
  }
  if (!live) return;
  const int b = (int)(at_row / a.q_heads), hq = (int)(at_row % a.q_heads);
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* dst = a.out + b * a.o_ts + hq * a.o_hs + lane * E;
  if (E == 2) *(uint32_t*)dst = cvt_bf16x2(o[0] * inv, o[1] * inv);
  else *dst = (uint16_t)f32_to_bf16_bits(o[0] * inv);
  if (a.lse && lane == 0) a.lse[at_row] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

static DecodePlan decode_plan(int64_t B, int q_heads, int kv_heads, int64_t prefix_len, int64_t max_len) {
  DecodePlan p;
  const int64_t G = q_heads / kv_heads, rows = B * G;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  p.wide = rows > 64;
  p.blocks_p = (int32_t)up(rows, p.wide ? 128 : 64);
  p.blocks_s = (int32_t)up(G, 64);
  // Two workgroups run on each of the 256 CUs, and a tile takes about as long in
  // either kind (2.1 us of matrix work, 2.6 us of its share of the reads): parts
  // of tiles / 512 tiles each fill the chip once.  Own keys go in finer parts
  // (their lengths differ; max_len is only a bound), at least 2 tiles.
  const int64_t tiles_p = up(prefix_len, kDecKeys), tiles_s = up(max_len, kDecKeys);
  const int64_t work = kv_heads * (tiles_p * p.blocks_p + tiles_s * B * p.blocks_s);
  const int64_t fill = std::max<int64_t>(2, up(work, 512));
  p.parts_p = (int32_t)up(tiles_p, fill);
  p.chunk_p = (int32_t)std::max<int64_t>(1, up(tiles_p, std::max(p.parts_p, 1)));
  p.chunk_s = (int32_t)std::max<int64_t>(2, up(fill, 2));
  p.parts_s = (int32_t)up(tiles_s, p.chunk_s);
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
  if (!a.part_o) return;
  const uint32_t rows = (uint32_t)(a.num_requests * a.q_heads);
  // waves per row: as many as leave each 8 parts or so, one round of loads
  const int parts = a.plan.parts_p + a.plan.parts_s;
  if (parts <= 16) hipLaunchKernelGGL((attn_join_kernel<DV, 1>), dim3((rows + 3) / 4), dim3(256), 0, stream, a);
  else if (parts <= 48) hipLaunchKernelGGL((attn_join_kernel<DV, 4>), dim3(rows), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((attn_join_kernel<DV, 16>), dim3(rows), dim3(1024), 0, stream, a);
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
