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
//
// With few keys one workgroup per request and key head does it all instead
// (attn_decode_small_kernel below).
//
// Workgroups of four waves walk the keys in tiles through LDS stages that all
// waves fill (direct loads; every lane finds its rows through the block table)
// while another is computed on:
//   wide   (prefix, many rows): 128 rows, 32 per wave; the prefix is read once
//          per 128 rows.  Bound by the matrix cores.
//   narrow (own keys, and a prefix with few rows): 32 or 64 rows.
//          Bound by reading the cache.
// The own keys of all requests are one list of tiles, which the narrow workgroups
// of a key head share out evenly, whatever the lengths: each takes one run of the
// list, across as many requests as it covers, without emptying its load pipeline
// at more than the requests' ends.  All workgroups of a launch fit the chip at
// once, so the wide ones' matrix work and the narrow ones' reads run side by side
// (decode_plan says when there are more).
//
// Measured: one request with 131072 own keys x 32/8 heads x 128: 83 us and 6 for the
// join, 6.5 TB/s of the 6.9 that contiguous reads reach; 96 requests behind 32768
// keys x 64/4 x 192: 145 to 150 us in all, 0.88 PFLOP/s; 64 behind 8192 with 69511
// own keys x 64/8 x 128: 71 to 73 us, 318 MB at 4.4 TB/s beside 17 GFLOP of prefix.
#include <algorithm>

#include "attn_common.h"

namespace moe {

constexpr int kDecThreads = 256;
constexpr int kDecSlots = 512;                      // two workgroups on each of 256 CUs
constexpr int kWideKeys = 64, kNarrowKeys = 32;     // per tile

// Where the waves of a CU's two workgroups could both go on, the older's would go
// first and its workgroup end 20% before the other, which then runs alone.  So
// they take turns by tiles, two to the younger's one (blocks are handed out in
// order: the second half are the younger ones); and a narrow workgroup's few
// instructions, which keep its reads going, come before a wide one's.  64 requests
// behind 8192 tokens 78.5 -> 71.2 us (turns alone 75.0, the wide ones first 78.1),
// 96 behind 32768 150 -> 145 us, one with 131072 tokens 98 -> 95 us.
template <int LOW>
__device__ __forceinline__ void take_turns(int t) {
  const bool younger = blockIdx.x >= kDecSlots / 2;
  if ((t % 3 != 0) == younger) __builtin_amdgcn_s_setprio(LOW + 1);
  else __builtin_amdgcn_s_setprio(LOW);
}

struct DecodePlan {
  int32_t small;                                    // no parts, the rest is 0
  int32_t wide;                                     // prefix workgroups are wide
  int32_t parts_p, chunk_p;                         // parts of the prefix, keys in each
  int32_t blocks_p;                                 // row blocks of B * G rows (wide 128, narrow 32 rb)
  int32_t rb;                                       // narrow workgroups take 32 rb rows
  int32_t blocks_s, rows_s;                         // row blocks of G rows, rows in each
  int32_t runs;                                     // narrow workgroups per key head and row block
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
  // Workspace.  Prefix: part x (two per narrow workgroup, one for each of its wave
  // pairs) of row b * Hq + h is entry x * B * Hq + row.  Own keys: run w's share of
  // request b -- (w + b, as the runs and the requests are walked in one order, is
  // each pair's own) -- entry own + (((head * blocks + block) * (runs + B) + w + b)
  // * 2 + pair) * rows_s + row.
  float* part_o;                                    // [entries][DV]
  float2* part_ml;                                  // [entries]: maximum (base 2), weight sum
  int32_t* first;                                   // [B + 1]: tiles of the requests before
  int64_t own;
  int32_t num_requests, q_heads, kv_heads, num_pages, page_shift;
  float c;
  DecodePlan plan;
};

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int len) { return (int)min((int64_t)max(len, 0), a.max_len); }
__device__ __forceinline__ int len_at(const DecodeArgs& a, int b) {   // b uniform: a scalar load
  return clamp_len(a, *(const __attribute__((address_space(4))) int32_t*)(a.lens + b));
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kNarrowKeys - 1) / kNarrowKeys; }

// The row of the cache that key `key` sits in; e: its table entry.
__device__ __forceinline__ int cache_row(const DecodeArgs& a, int e, int key) {
  return (min(max(e, 0), a.num_pages - 1) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}

// This lane's row of a finished part.
template <class W, int DV>
__device__ __forceinline__ void store_part(const DecodeArgs& a, const W& w, int64_t entry, int h) {
  float* po = a.part_o + entry * DV + 4 * h;
#pragma unroll
  for (int x = 0; x < W::OB; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f32x4*)(po + 32 * x + 8 * i) = f32x4{w.o[x][4 * i], w.o[x][4 * i + 1], w.o[x][4 * i + 2], w.o[x][4 * i + 3]};
  if (h == 0) a.part_ml[entry] = float2{w.m, w.l};
}

// Values of keys past the end (they repeat the last) become zeros in their stage:
// their weights are 0, and 0 times an infinity would not be.
template <int DV, int ROWS>
__device__ __forceinline__ void clear_values(uint8_t* vs, int valid) {
#pragma unroll
  for (int i = 0; i < ROWS * DV * 2 / 16 / kDecThreads; ++i) {
    const int f = i * kDecThreads + threadIdx.x;
    if (f / (DV / 8) >= valid) *(u32x4*)(vs + f * 16) = u32x4{0u, 0u, 0u, 0u};
  }
  at_wait_barrier<63>();                                            // (no load is waited for)
}

// Prefix part `part`, 128 rows from row0, 32 per wave; tiles of 64 keys in two stages.
// PAGED: pages hold 64 rows or more, so a tile's rows follow one another (rows past
// the end are the page's own and masked); a lane's offsets in a tile are constant
// then.  Otherwise each lane finds its rows.
template <int DQ, int DV, bool PAGED>
__device__ __forceinline__ void decode_wide(const DecodeArgs& a, int kvh, int part, int row0, uint8_t* mem) {
  using W = AttnWave<DQ, DV, kWideKeys / 32>;
  uint8_t* ks = mem;
  uint8_t* vs = mem + 2 * W::kKeyBytes;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int G = a.q_heads / a.kv_heads, rows = a.num_requests * G;
  const int wrow = row0 + wv * 32;                                  // this wave's first row
  const int row = min(wrow + (lane & 31), rows - 1);
  const int b = row / G, hq = kvh * G + row % G;
  W w;
  w.init(a.q + b * a.q_ts + hq * a.q_hs, lane);
  // Lane l looks up the cache row of key l of a tile (past the end: the last
  // key), one tile ahead of the loads that use it: the table entry of tile t + 2
  // is read when the loads of tile t + 1 go out.
  const int key0 = part * a.plan.chunk_p, n_keys = (int)min((int64_t)a.plan.chunk_p, a.prefix_len - key0);
  const int n_tiles = (n_keys + kWideKeys - 1) / kWideKeys, n_whole = n_keys / kWideKeys;
  auto key_of = [&](int t) { return key0 + min(t * kWideKeys + (PAGED ? 0 : lane), n_keys - 1); };
  auto entry = [&](int t) { return a.prefix_table[key_of(t) >> a.page_shift]; };
  const uint32_t k_lds = at_lds_addr(ks) + (uint32_t)wv * 1024u, v_lds = at_lds_addr(vs) + (uint32_t)wv * 1024u;
  const uint8_t* kc = (const uint8_t*)(a.k_cache + (int64_t)kvh * DQ);
  const uint8_t* vc = (const uint8_t*)(a.v_cache + (int64_t)kvh * DV);
  const uint32_t k_row = (uint32_t)a.kv_heads * DQ * 2, v_row = (uint32_t)a.kv_heads * DV * 2;
  constexpr int kKeyLoads = W::kKeyBytes / 16 / kDecThreads, kValLoads = W::kValBytes / 16 / kDecThreads;
  uint32_t koff[PAGED ? kKeyLoads : 1], voff[PAGED ? kValLoads : 1];
  if (PAGED) {
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DQ / 8);
      koff[i] = (uint32_t)r * k_row + (uint32_t)((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16u;   // < 2^31: 63 rows of 65536 heads
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DV / 8);
      voff[i] = (uint32_t)r * v_row + (uint32_t)((f % (DV / 8)) ^ at_swz<DV>(r)) * 16u;
    }
  }
  auto load = [&](int slot, int st) {
    const uint32_t kt = k_lds + (uint32_t)(st * W::kKeyBytes), vt = v_lds + (uint32_t)(st * W::kValBytes);
    if (PAGED) {
      const uint32_t row = (uint32_t)__builtin_amdgcn_readfirstlane(slot);
      const at_rsrc kr = at_make_rsrc(kc + (uint64_t)row * k_row), vr = at_make_rsrc(vc + (uint64_t)row * v_row);
#pragma unroll
      for (int i = 0; i < kKeyLoads; ++i) at_load_lds(kt + i * kDecThreads * 16, kr, koff[i], 0);
#pragma unroll
      for (int i = 0; i < kValLoads; ++i) at_load_lds(vt + i * kDecThreads * 16, vr, voff[i], 0);
      return;
    }
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DQ / 8);
      at_load_lds<false>(kt + i * kDecThreads * 16,
                         kc + (uint64_t)(uint32_t)__shfl(slot, r) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DV / 8);
      at_load_lds<false>(vt + i * kDecThreads * 16,
                         vc + (uint64_t)(uint32_t)__shfl(slot, r) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16);
    }
  };
  load(cache_row(a, entry(0), key_of(0)), 0);
  int next = entry(1);
  auto step = [&](auto stage, int t) {
    constexpr int st = decltype(stage)::value;
    // tile t has landed; everyone is done with tile t - 1, whose stage the next loads refill
    at_wait_barrier<0>();
    take_turns<0>(t);
    if (t + 1 < n_tiles) {
      load(cache_row(a, next, key_of(t + 1)), st ^ 1);
      next = entry(t + 2);
    }
    const bool cut = t >= n_whole;
    if (cut) clear_values<DV, kWideKeys>(vs + st * W::kValBytes, n_keys - t * kWideKeys);
    if (wrow >= rows) return;
    w.scores(ks + st * W::kKeyBytes);
    if (cut) w.mask(lane, n_keys - 1 - t * kWideKeys);
    w.weights(a.c);
    w.values(vs + st * W::kValBytes);
  };
  for (int t = 0; t < n_tiles; t += 2) {
    step(std::integral_constant<int, 0>(), t);
    if (t + 1 < n_tiles) step(std::integral_constant<int, 1>(), t + 1);
  }
  if (wrow + (lane & 31) < rows)
    store_part<W, DV>(a, w, (int64_t)part * a.num_requests * a.q_heads + (int64_t)b * a.q_heads + hq, h);
}

// Where a narrow workgroup is in its run of tiles: tile `tile` of request b, which
// has len keys from key0 on.  PREFIX: one request, the prefix's part.
template <bool PREFIX>
struct Cursor {
  int b, tile, tiles, len, key0;
  const int32_t* table;
  __device__ __forceinline__ void next(const DecodeArgs& a) {
    if (++tile < tiles || PREFIX) return;
    do {
      ++b;
      len = len_at(a, b);
    } while (len == 0);
    tiles = tiles_of(len);
    tile = 0;
    table = a.table + b * a.table_stride;
  }
  __device__ __forceinline__ int key(int r) const { return key0 + min(tile * kNarrowKeys + r, len - 1); }   // past the end: the last
};

// n_tiles tiles from `at` on for 32 RB rows: waves 0, 1 the first 16 RB, waves 2, 3
// the others; even waves compute every other tile, odd waves those between, and the
// two leave parts of their own.  The reads are what counts: NS stages, so that
// while one tile is computed on NS - 1 are under way.
//
// Loads in order of issue, per wave: D(t), the rows of tile t, and E(t), the table
// entries of tile t, one load, into a ring in LDS; L loads in a pair.  Step t waits
// for D(t) and E(t + NS - 1), issues D(t + NS - 1) and E(t + 2 NS - 2): the
// waited-for pair went out together in step t - NS + 1, so the NS - 2 pairs issued
// since may be in flight.  Near the end fewer are.
template <int DQ, int DV, int NS, int RB, bool PREFIX>
__device__ __forceinline__ void decode_narrow(const DecodeArgs& a, int kvh, Cursor<PREFIX> at, int n_tiles, int row0, int rows,
                                              int64_t entry0, uint8_t* mem) {
  using W = AttnWave16<DQ, DV, RB>;
  constexpr int kRing = 2 * NS;                                     // entries live 2 NS - 2 steps
  constexpr int kKeyLoads = W::kKeyBytes / 16 / kDecThreads, kValLoads = W::kValBytes / 16 / kDecThreads;
  constexpr int L = kKeyLoads + kValLoads + 1;
  static_assert(NS == 3 || NS == 4, "the waits below");
  uint8_t* ks = mem;
  uint8_t* vs = ks + NS * W::kKeyBytes;
  const int* ring = (const int*)(vs + NS * W::kValBytes);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int odd = wv & 1, G = a.q_heads / a.kv_heads;
  const int wrow = row0 + (wv >> 1) * 16 * RB;                      // this wave's first row
  const uint32_t k_lds = at_lds_addr(ks) + (uint32_t)wv * 1024u, v_lds = at_lds_addr(vs) + (uint32_t)wv * 1024u;
  const uint8_t* kc = (const uint8_t*)(a.k_cache + (int64_t)kvh * DQ);
  const uint8_t* vc = (const uint8_t*)(a.v_cache + (int64_t)kvh * DV);
  const uint32_t k_row = (uint32_t)a.kv_heads * DQ * 2, v_row = (uint32_t)a.kv_heads * DV * 2;
  Cursor<PREFIX> ahead = at, behind = at;                           // of the entries; of the computation (`at`: of the rows)
  int fetched = 0, loaded = 0;                                      // tiles, also their places in ring and stages
  // (every wave fetches all entries itself: it then need not wait for another's;
  // past the run's end it fetches the last again, unread)
  auto fetch = [&]() {
    at_load_lds4(at_lds_addr(ring) + (uint32_t)(fetched % kRing) * 256u, ahead.table + (ahead.key(lane & 31) >> a.page_shift));
    if (++fetched < n_tiles) ahead.next(a);
  };
  auto load = [&]() {
    const int st = loaded % NS;
    const int* e = ring + (loaded % kRing) * 64;
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DQ / 8);
      at_load_lds<!PREFIX>(k_lds + (uint32_t)(st * W::kKeyBytes + i * kDecThreads * 16),
                  kc + (uint64_t)(uint32_t)cache_row(a, e[r], at.key(r)) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int f = i * kDecThreads + threadIdx.x, r = f / (DV / 8);
      at_load_lds<!PREFIX>(v_lds + (uint32_t)(st * W::kValBytes + i * kDecThreads * 16),
                  vc + (uint64_t)(uint32_t)cache_row(a, e[r], at.key(r)) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16);
    }
    if (++loaded < n_tiles) at.next(a);
  };
  W w;
  w.offsets(lane);
  auto begin = [&]() {                                              // the rows of the computation's request
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = min(wrow + 16 * rb + (lane & 15), rows - 1);
      const int b = PREFIX ? row / G : behind.b, hq = kvh * G + (PREFIX ? row % G : row);
      w.init(rb, a.q + b * a.q_ts + hq * a.q_hs, lane);
    }
    w.settle();
    at_wait<0>();                                                   // nothing of before is counted below
  };
  for (int t = 0; t < NS - 1; ++t) fetch();
  begin();
  for (int t = 0; t < NS - 1; ++t) {
    if (t < n_tiles) load();
    fetch();
  }
  for (int t = 0; t < n_tiles; ++t) {
    // pairs issued after tile t's: NS - 2, at the end as many as tiles are left
    take_turns<2>(t);
    const int after = min(n_tiles - 1 - t, NS - 2);
    if (after == 0) at_wait_barrier<0>();
    else if (after == 1) at_wait_barrier<L>();
    else at_wait_barrier<2 * L>();
    if (t + NS - 1 < n_tiles) {
      load();
      fetch();
    }
    const int last = behind.len - 1 - behind.tile * kNarrowKeys;
    const uint8_t* k = ks + (t % NS) * W::kKeyBytes;
    uint8_t* v = vs + (t % NS) * W::kValBytes;
    if (last < kNarrowKeys - 1) clear_values<DV, kNarrowKeys>(v, last + 1);
    if (wrow < rows && (t & 1) == odd) {
      w.scores(k);
      if (last < kNarrowKeys - 1) w.mask(lane, last);
      w.weights(a.c);
      w.values(v);
    }
    const bool end = t + 1 == n_tiles;
    if (end || behind.tile + 1 == behind.tiles) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const int row = wrow + 16 * rb + (lane & 15);
        if (row >= rows) continue;
        const int64_t entry = PREFIX ? entry0 + ((int64_t)odd * a.num_requests + row / G) * a.q_heads + kvh * G + row % G
                                     : entry0 + ((int64_t)behind.b * 2 + odd) * a.plan.rows_s + row - row0;
#pragma unroll
        for (int x = 0; x < W::OB; ++x) *(f32x4*)(a.part_o + entry * DV + 16 * x + 4 * (lane >> 4)) = w.o[rb][x];
        if (lane < 16) a.part_ml[entry] = float2{w.m[rb], w.l[rb]};
      }
      if (end) break;
      behind.next(a);
      begin();
    } else {
      behind.next(a);
    }
  }
}

template <int DQ, int DV, int RB>
__global__ __launch_bounds__(kDecThreads, 2) void attn_decode_kernel(DecodeArgs a) {
  // narrow: stages of 32 keys and the ring of table entries; two workgroups fit a CU's 160 KB
  constexpr int kTile = kNarrowKeys * (DQ + DV) * 2, NS = 4 * kTile + 2048 <= 80 * 1024 ? 4 : 3;
  constexpr int kNarrow = NS * kTile + 2 * NS * 256, kWide = 2 * kWideKeys * (DQ + DV) * 2;
  __shared__ __attribute__((aligned(16))) uint8_t mem[kNarrow > kWide ? kNarrow : kWide];
  const DecodePlan& p = a.plan;
  const int kvh = blockIdx.x % a.kv_heads, lane = threadIdx.x & 63;
  int item = blockIdx.x / (uint32_t)a.kv_heads;
  if (item < p.parts_p * p.blocks_p) {
    // row blocks of one part side by side: they share the part's keys in L2
    const int part = item / p.blocks_p, block = item % p.blocks_p;
    if (p.wide && a.page_shift >= 6) return decode_wide<DQ, DV, true>(a, kvh, part, block * 128, mem);
    if (p.wide) return decode_wide<DQ, DV, false>(a, kvh, part, block * 128, mem);
    Cursor<true> at;
    at.b = at.tile = 0;
    at.key0 = part * p.chunk_p;
    at.len = (int)min((int64_t)p.chunk_p, a.prefix_len - at.key0);
    at.tiles = tiles_of(at.len);
    at.table = a.prefix_table;
    return decode_narrow<DQ, DV, NS, RB, true>(a, kvh, at, at.tiles, block * 32 * RB, a.num_requests * (a.q_heads / a.kv_heads),
                                           (int64_t)part * 2 * a.num_requests * a.q_heads, mem);
  }
  item -= p.parts_p * p.blocks_p;
  const int run = item / p.blocks_s, block = item % p.blocks_s;
  // tiles of all requests; the first workgroup writes down where each request's begin
  const int B = a.num_requests;
  int total = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int n = b0 + lane < B ? tiles_of(clamp_len(a, a.lens[b0 + lane])) : 0;
    int sum = n;                                                    // inclusive over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    if (blockIdx.x == (uint32_t)(p.parts_p * p.blocks_p * a.kv_heads) && threadIdx.x < 64 && b0 + lane < B)
      a.first[b0 + lane] = total + sum - n;
    total += __builtin_amdgcn_readlane(sum, 63);
  }
  if (blockIdx.x == (uint32_t)(p.parts_p * p.blocks_p * a.kv_heads) && threadIdx.x == 0) a.first[B] = total;
  const int each = (total + p.runs - 1) / p.runs, begin = run * each, end = min(begin + each, total);
  if (begin >= end) return;
  // the request that tile `begin` belongs to: the last whose tiles begin at or before it
  Cursor<false> at;
  int before = 0, b = 0;
  for (int b0 = 0, sofar = 0; b0 < B; b0 += 64) {
    const int n = b0 + lane < B ? tiles_of(clamp_len(a, a.lens[b0 + lane])) : 0;
    int sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t le = __ballot(sofar + sum - n <= begin && n > 0);
    if (le) {
      const int l = 63 - __builtin_clzll(le);
      b = b0 + l;
      before = sofar + __builtin_amdgcn_readlane(sum - n, l);
    }
    sofar += __builtin_amdgcn_readlane(sum, 63);
    if (sofar > begin) break;
  }
  at.b = b;
  at.tile = begin - before;
  at.len = len_at(a, at.b);
  at.tiles = tiles_of(at.len);
  at.key0 = 0;
  at.table = a.table + at.b * a.table_stride;
  const int row0 = block * p.rows_s, rows = min(row0 + p.rows_s, a.q_heads / a.kv_heads);
  const int64_t entry0 = a.own + ((int64_t)(kvh * p.blocks_s + block) * (p.runs + B) + run) * 2 * p.rows_s;
  decode_narrow<DQ, DV, NS, RB, false>(a, kvh, at, end - begin, row0, rows, entry0, mem);
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
  const int Hall = a.num_requests * a.q_heads;
  const int at_row = blockIdx.x * kRows + wv / WPR;
  const bool live = at_row < Hall;                                  // whole waves; a row's waves agree
  const int b = min(at_row, Hall - 1) / a.q_heads, hq = min(at_row, Hall - 1) % a.q_heads;
  constexpr int E = DV / 64;                                        // values per lane
  float M = neg_inf(), L = 0.0f, o[2] = {0.0f, 0.0f};
  if (live) {
    const DecodePlan& p = a.plan;
    // own parts: two for each run that the request's tiles lie in
    const int np = p.parts_p * (p.wide ? 1 : 2);
    int n = np, run0 = 0;
    if (p.runs > 0) {
      const int t0 = a.first[b], t1 = a.first[b + 1], each = (a.first[a.num_requests] + p.runs - 1) / p.runs;
      if (t1 > t0) {
        run0 = t0 / each;
        n += 2 * ((t1 - 1) / each - run0 + 1);
      }
    }
    const int G = a.q_heads / a.kv_heads, kvh = hq / G, g = hq % G, block = g / p.rows_s;
    const int64_t own = a.own + ((int64_t)(kvh * p.blocks_s + block) * (p.runs + a.num_requests) + run0 + b) * 2 * p.rows_s +
                        g - block * p.rows_s;
    auto entry = [&](int x) { return x < np ? (int64_t)x * Hall + at_row : own + (int64_t)(x - np) * p.rows_s; };
    const int mine = (n - sub + WPR - 1) / WPR;                     // parts sub, sub + WPR, ...
    for (int base = 0; base < mine; base += 64) {
      const int cnt = min(64, mine - base);
      float2 x = float2{neg_inf(), 0.0f};
      if (lane < cnt) x = a.part_ml[entry(sub + (base + lane) * WPR)];
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
      for (int q0 = 0; q0 < cnt; q0 += 8) {                         // 8 loads in flight
        float y[8][2];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float* src = a.part_o + entry(sub + (base + min(q0 + u, cnt - 1)) * WPR) * DV + lane * E;
          y[u][0] = src[0];
          if (E == 2) y[u][1] = src[1];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (q0 + u >= cnt) break;
          const float ep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), q0 + u));
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
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* dst = a.out + b * a.o_ts + hq * a.o_hs + lane * E;
  if (E == 2) *(uint32_t*)dst = cvt_bf16x2(o[0] * inv, o[1] * inv);
  else *dst = (uint16_t)f32_to_bf16_bits(o[0] * inv);
  if (a.lse && lane == 0) a.lse[at_row] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// Few keys: a workgroup per request and key head answers alone, without parts and
// a second launch.  Its eight waves take every eighth tile of 32 keys, prefix first,
// each through registers into its own LDS, the next tile's loads under way while
// one is computed on; then the waves' sums are joined.  Every request reads the
// prefix for itself (from L2 after the first).  At most 16 heads of a key head.
// PAGED: pages hold 8 rows or more, so the whole rows of one load (4 of 128 columns,
// 8 of 64) follow one another: one row is looked up for all lanes (8 requests behind
// 777 tokens 10.8 -> 10.4 us; keys of 192 columns do not come in whole rows and gain
// nothing).
constexpr int kSmallWaves = 8;

template <int DQ, int DV, bool PAGED>
__global__ __launch_bounds__(kSmallWaves * 64) void attn_decode_small_kernel(DecodeArgs a) {
  using W = AttnWave16<DQ, DV, 1>;
  constexpr int kRegion = W::kKeyBytes + W::kValBytes, kOut = DV + 4;             // floats of a row of sums (padded: banks)
  constexpr int kKeyLoads = W::kKeyBytes / 1024, kValLoads = W::kValBytes / 1024;  // 16 bytes per lane
  static_assert(16 * kOut * 4 + 16 * 8 <= kRegion, "a wave's sums fit its region");
  __shared__ __attribute__((aligned(16))) uint8_t mem[kSmallWaves * kRegion];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kvh = blockIdx.x % (uint32_t)a.kv_heads, b = blockIdx.x / (uint32_t)a.kv_heads, G = a.q_heads / a.kv_heads;
  const int len = len_at(a, b), prefix = (int)a.prefix_len;
  const int tiles_p = tiles_of(prefix), n_tiles = tiles_p + tiles_of(len);
  const int32_t* own = a.table + b * a.table_stride;
  auto base_of = [&](int t) { return (t < tiles_p ? t : t - tiles_p) * kNarrowKeys; };
  auto end_of = [&](int t) { return t < tiles_p ? prefix : len; };
  // lane's row of tile t (past the end: the last key's)
  auto slot_of = [&](int t) {
    const int key = min(base_of(t) + (lane & 31), end_of(t) - 1);
    return cache_row(a, (t < tiles_p ? a.prefix_table : own)[key >> a.page_shift], key);
  };
  const uint8_t* kc = (const uint8_t*)(a.k_cache + (int64_t)kvh * DQ);
  const uint8_t* vc = (const uint8_t*)(a.v_cache + (int64_t)kvh * DV);
  const uint32_t k_row = (uint32_t)a.kv_heads * DQ * 2, v_row = (uint32_t)a.kv_heads * DV * 2;
  u32x4 kr[kKeyLoads], vr[kValLoads];
  static_assert(!PAGED || DQ != 192, "");
  constexpr int kRowsK = 512 / DQ, kRowsV = 512 / DV;               // whole rows of a load
  auto load = [&](int slot) {
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) {
      const int f = i * 64 + lane, r = f / (DQ / 8);
      if (PAGED) {
        // (rows past the end: those of the last key's group, its page's own)
        const uint32_t row = (uint32_t)__builtin_amdgcn_readlane(slot, i * kRowsK) & ~(uint32_t)(kRowsK - 1);
        kr[i] = *(const u32x4*)(kc + (uint64_t)row * k_row + ((uint32_t)(r - i * kRowsK) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16u));
        continue;
      }
      kr[i] = *(const u32x4*)(kc + (uint64_t)(uint32_t)__shfl(slot, r) * k_row + ((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int f = i * 64 + lane, r = f / (DV / 8);
      if (PAGED) {
        const uint32_t row = (uint32_t)__builtin_amdgcn_readlane(slot, i * kRowsV) & ~(uint32_t)(kRowsV - 1);
        vr[i] = *(const u32x4*)(vc + (uint64_t)row * v_row + ((uint32_t)(r - i * kRowsV) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16u));
        continue;
      }
      vr[i] = *(const u32x4*)(vc + (uint64_t)(uint32_t)__shfl(slot, r) * v_row + ((f % (DV / 8)) ^ at_swz<DV>(r)) * 16);
    }
  };
  uint8_t* ks = mem + wv * kRegion;
  uint8_t* vs = ks + W::kKeyBytes;
  int t = wv, next = 0;
  W w;
  w.init(0, a.q + b * a.q_ts + (int64_t)(kvh * G + min(lane & 15, G - 1)) * a.q_hs, lane);
  if (t < n_tiles) {
    const int slot = slot_of(t);
    if (t + kSmallWaves < n_tiles) next = slot_of(t + kSmallWaves);
    load(slot);
  }
  w.offsets(lane);
  for (; t < n_tiles; t += kSmallWaves) {
    const int last = end_of(t) - 1 - base_of(t);
#pragma unroll
    for (int i = 0; i < kKeyLoads; ++i) *(u32x4*)(ks + (i * 64 + lane) * 16) = kr[i];
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      // (a weight of 0 times an infinity past the end would not be 0)
      const bool there = (i * 64 + lane) / (DV / 8) <= last;
      *(u32x4*)(vs + (i * 64 + lane) * 16) = there ? vr[i] : u32x4{0u, 0u, 0u, 0u};
    }
    asm volatile("" ::: "memory");                                  // (a wave's own LDS accesses stay in order)
    if (t + kSmallWaves < n_tiles) {
      load(next);
      if (t + 2 * kSmallWaves < n_tiles) next = slot_of(t + 2 * kSmallWaves);
    }
    w.scores(ks);
    if (last < kNarrowKeys - 1) w.mask(lane, last);
    w.weights(a.c);
    w.values(vs);
    asm volatile("" ::: "memory");
  }
  // each wave's sums, maxima and weight sums into its region; joined by 4 columns per thread
  float* po = (float*)ks;
#pragma unroll
  for (int x = 0; x < W::OB; ++x) *(f32x4*)(po + (lane & 15) * kOut + 16 * x + 4 * (lane >> 4)) = w.o[0][x];
  if (lane < 16) ((float2*)(po + 16 * kOut))[lane] = float2{w.m[0], w.l[0]};
  __syncthreads();
  const int row = threadIdx.x / (DV / 4), col = threadIdx.x % (DV / 4) * 4;
  if (row >= G) return;
  float2 ml[kSmallWaves];
  float M = neg_inf(), L = 0.0f;
#pragma unroll
  for (int i = 0; i < kSmallWaves; ++i) {
    ml[i] = ((const float2*)((const float*)(mem + i * kRegion) + 16 * kOut))[row];
    M = fmaxf(M, ml[i].x);
  }
  const float ref = M == neg_inf() ? 0.0f : M;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kSmallWaves; ++i) {
    const float e = __builtin_amdgcn_exp2f(ml[i].x - ref);
    const f32x4 o = *(const f32x4*)((const float*)(mem + i * kRegion) + row * kOut + col);
    L = fmaf(e, ml[i].y, L);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fmaf(e, o[j], sum[j]);
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int hq = kvh * G + row;
  *(u32x2*)(a.out + b * a.o_ts + hq * a.o_hs + col) =
      u32x2{cvt_bf16x2(sum[0] * inv, sum[1] * inv), cvt_bf16x2(sum[2] * inv, sum[3] * inv)};
  if (a.lse && col == 0) a.lse[(int64_t)b * a.q_heads + hq] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// Whether one workgroup per request and key head is sooner done than parts and
// their join, in nanoseconds as measured (128-wide heads; others by their bytes).
// Small: 3500, and 220 for each tile of 32 keys of the longest request, prefix
// included, in as many rounds as the chip needs at a workgroup per CU; or the
// reading of the own keys (half of the bound) at a little under the parts' rate.
// Parts: 10000 for two launches, and the reading of all keys once.
// 32/8 heads x 128: 32 requests with up to 700 own keys 13.7 us alone, 18.4 in parts; one
// with 2048 behind a prefix of 2000 27.8 and 12.7.  Within 5% of the better one at 338 of 360 sizes tried,
// 1 to 96 requests with up to 16 to 2048 own keys behind 0 to 2000, all head sizes
// (of 64-wide ones' workgroups a CU holds two: 88 of 90).  The others are for the most
// part batches of 33 to 64 rows behind 2000 keys, up to 1.5 times slower in parts.
static bool small_is_sooner(int64_t B, int64_t G, int64_t kv_heads, int64_t prefix_len, int64_t max_len, int64_t dims) {
  if (G > 16) return false;
  const int64_t tiles_p = (prefix_len + 31) / 32, tiles_s = (max_len + 31) / 32, rounds = (B * kv_heads + 255) / 256;
  if (tiles_p + tiles_s > 1024) return false;                       // (the products below stay small)
  const int64_t own = 3 * kv_heads * B * tiles_s / 2 * dims / 256, prefix = 3 * kv_heads * tiles_p * dims / 256;
  const int64_t small = 3500 + std::max(220 * (tiles_p + tiles_s) * rounds * dims / 256, own + own / 7);
  return small < 10000 + own + prefix;
}

static DecodePlan decode_plan(int64_t B, int q_heads, int kv_heads, int64_t prefix_len, int64_t max_len, int dims) {
  DecodePlan p = {};
  const int64_t G = q_heads / kv_heads, rows = B * G;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  p.small = small_is_sooner(B, G, kv_heads, prefix_len, max_len, dims);
  if (p.small) return p;
  p.wide = rows > 64;
  p.rb = G > 32 || (!p.wide && rows > 32) ? 2 : 1;
  p.blocks_p = (int32_t)up(rows, p.wide ? 128 : 32 * p.rb);
  p.blocks_s = (int32_t)up(G, 32 * p.rb);
  p.rows_s = (int32_t)std::min<int64_t>(G, 32 * p.rb);
  // The workgroups that the chip holds at once are shared by the two kinds so that
  // both end at about the same time.  64 keys of a prefix take a wide workgroup 6
  // units, a narrow one 7, and own keys a narrow one 10 (1.5 us of matrix work for 128
  // rows, 2.7 us of its share of the reads; 128-wide heads).  The own lengths are not
  // known here: one is counted at the bound, the others at half, and each request once
  // more for starting on it.  (One request with 7647 keys behind 12490, 32/8 heads: 31
  // us with half of the bound and equal units for the narrow ones, 24 us so.  Over 80
  // sizes own keys at 7 or 14 units take 3% longer on average, all own lengths at half 1%,
  // equal units for the narrow ones 1%.)
  // (64 requests behind 8192 tokens: 79 us with shares by keys alone, of which the
  // prefix's workgroups worked 39.)
  const int64_t tiles_p = up(prefix_len, 64), tiles_s = max_len == 0 ? 0 : up((B + 1) * up(max_len, 64), 2) + B;
  const int64_t cost_p = p.wide ? 6 : 7, cost_s = 10;
  const int64_t per_part = kv_heads * p.blocks_p, per_run = kv_heads * p.blocks_s;
  const int64_t work_p = per_part * tiles_p * cost_p, work_s = per_run * tiles_s * cost_s;
  int64_t parts = 0;
  if (tiles_p > 0) {
    // parts of the prefix, at least two tiles in each: the share rounded down or up
    const int64_t most = up(tiles_p, 2), room = max_len == 0 ? kDecSlots : kDecSlots - per_run;
    parts = std::max<int64_t>(1, std::min(most, kDecSlots * work_p / (work_p + work_s) / per_part));
    auto time = [&](int64_t n) { return std::max(up(tiles_p, n) * cost_p, work_s / std::max<int64_t>(1, kDecSlots - n * per_part)); };
    if (parts < most && (parts + 1) * per_part <= room && time(parts + 1) < time(parts)) ++parts;
  }
  p.chunk_p = tiles_p == 0 ? 0 : (int32_t)(up(tiles_p, parts) * 64);
  p.parts_p = tiles_p == 0 ? 0 : (int32_t)up(prefix_len, p.chunk_p);
  // Runs of the own keys, at least two narrow tiles in each: the rest of the chip.  Many
  // rows on few prefix keys (one part) leave little of it or nothing, but end early: then
  // as many runs as the whole chip holds, the last of which start when those are done,
  // if that is sooner.  (512 requests x 64/8 x 128 behind 100 tokens, up to 2048 own keys:
  // 576 -> 462 us; 1000 requests, whose prefix leaves room for one run: 33.6 -> 0.91 ms.)
  int64_t places = kDecSlots - p.parts_p * per_part;
  if (p.parts_p == 1 && max_len > 0) {
    const int64_t prefix = up(per_part, kDecSlots) * (p.chunk_p / 64) * cost_p;
    if (places < per_run || prefix + work_s / kDecSlots < work_s / places) places = kDecSlots;
  }
  const int64_t left = places / per_run;
  p.runs = max_len == 0 ? 0 : (int32_t)std::max<int64_t>(1, std::min(left, up(B * up(max_len, kNarrowKeys), 2)));
  return p;
}

// entries of the two kinds of parts; the workspace holds their sums, their maxima
// and weight sums, and the requests' first tiles
static int64_t prefix_entries(const DecodePlan& p, int64_t B, int q_heads) {
  return p.parts_p * (p.wide ? 1 : 2) * B * q_heads;
}
static int64_t plan_entries(const DecodePlan& p, int64_t B, int q_heads, int kv_heads) {
  return prefix_entries(p, B, q_heads) +
         (p.runs > 0 ? (int64_t)kv_heads * p.blocks_s * (p.runs + B) * 2 * p.rows_s : 0);
}

size_t attn_decode_ws_bytes(int64_t B, int q_heads, int kv_heads, int k_dim, int v_dim, int64_t prefix_len, int64_t max_len) {
  const DecodePlan p = decode_plan(B, q_heads, kv_heads, prefix_len, max_len, k_dim + v_dim);
  const int64_t entries = plan_entries(p, B, q_heads, kv_heads);
  return entries == 0 ? 0 : (size_t)entries * ((size_t)v_dim * 4 + 8) + ((size_t)B + 1) * 4;
}

static int64_t plan_grid(const DecodePlan& p, int kv_heads) {
  return ((int64_t)p.parts_p * p.blocks_p + (int64_t)p.runs * p.blocks_s) * kv_heads;
}

int64_t attn_decode_grid(int64_t B, int q_heads, int kv_heads, int k_dim, int v_dim, int64_t prefix_len, int64_t max_len) {
  const DecodePlan p = decode_plan(B, q_heads, kv_heads, prefix_len, max_len, k_dim + v_dim);
  return p.small ? B * kv_heads : plan_grid(p, kv_heads);
}

template <int DQ, int DV>
static void launch_decode(const DecodeArgs& a, hipStream_t stream) {
  if (a.plan.small) {
    const dim3 grid((uint32_t)(a.num_requests * a.kv_heads)), threads(kSmallWaves * 64);
    constexpr bool kWhole = DQ != 192;
    if (kWhole && a.page_shift >= 3) hipLaunchKernelGGL((attn_decode_small_kernel<DQ, DV, kWhole>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_small_kernel<DQ, DV, false>), grid, threads, 0, stream, a);
    return;
  }
  const uint32_t grid = (uint32_t)plan_grid(a.plan, a.kv_heads);
  if (grid > 0) {
    if (a.plan.rb == 1) hipLaunchKernelGGL((attn_decode_kernel<DQ, DV, 1>), dim3(grid), dim3(kDecThreads), 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_kernel<DQ, DV, 2>), dim3(grid), dim3(kDecThreads), 0, stream, a);
  }
  const uint32_t rows = (uint32_t)(a.num_requests * a.q_heads);
  // waves per row: as many as leave each 8 parts or so, one round of loads (a
  // request's own parts: two per run it lies in, on average runs / B of them)
  const int parts = a.plan.parts_p * (a.plan.wide ? 1 : 2) + 2 * (1 + a.plan.runs / a.num_requests);
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
  a.plan = decode_plan(B, p.q_heads, p.kv_heads, prefix_len, max_len, p.k_dim + p.v_dim);
  const int64_t entries = plan_entries(a.plan, B, p.q_heads, p.kv_heads);
  a.part_o = (float*)ws;                            // (the sums first: they need 16-byte alignment)
  a.part_ml = (float2*)(a.part_o + entries * p.v_dim);
  a.first = (int32_t*)(a.part_ml + entries);
  a.own = prefix_entries(a.plan, B, p.q_heads);
  if (p.k_dim == 64) launch_decode<64, 64>(a, stream);
  else if (p.k_dim == 128) launch_decode<128, 128>(a, stream);
  else launch_decode<192, 128>(a, stream);
  return launch_status("moe_attn_decode");
}

}  // namespace moe
