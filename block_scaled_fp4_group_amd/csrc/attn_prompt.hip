// Causal attention over whole prompts: packed sequences, grouped heads.
//
//   out[i, h] = sum_j p_ij v[j, h / G],  p_i = softmax over the keys row i sees
// of q_i . k_j * scale.  Row i of a sequence with Lq queries and Lk keys sees
// keys 0 .. i + Lk - Lq (the last query sees every key; with Lk < Lq the first
// rows see none and give 0).
//
// The G query heads of a key head see the same keys, so a sequence's rows are
// taken token by token with the G heads of each token side by side: row m is head
// m % G of token m / G.  A workgroup takes 128 such rows, 32 per wave
// (attn_common.h), and walks the keys in tiles of 64 through LDS.  Its rows span
// only 128 / G tokens: all waves end at about the same key, and little is computed
// beyond the diagonal (against 128 tokens of one head: 32 prompts of 21 to 2048 tokens
// 195 -> 188 us, 3 of up to 3500 with context 448 -> 425 us).
//
// Bound by the matrix cores' power budget where the keys are many: 16384 tokens x
// 32/4 heads x 128 take 1.83 to 1.95 ms = 1.13 to 1.2 PFLOP/s by the box, matrix
// units busy 70% of the cycles at the 1.64 GHz that the chip then runs at (a library's
// 8192^3 product reaches 1.25 PFLOP/s).  Where the keys are few a
// workgroup costs 7 us beside its tiles (1 us each alone on a CU, 1.7 beside
// another): 0.7 to find its rows, 3 until the first tile is there, 1.7 to store, 2
// until the next one starts, which the others on its CU hide in part: the 32 prompts
// above take 156 to 163 us, 790 TFLOP/s.
//
// Few rows with many keys (a short addition to a long context) would leave most of
// the chip idle: their keys are split over several workgroups, whose float sums,
// maxima and weight sums a second launch joins (prompt_splits).
#include <algorithm>

#include "attn_common.h"

namespace moe {

constexpr int kPromptThreads = 256;
constexpr int kPromptRows = kPromptThreads / 64 * 32;
constexpr int kPromptKeys = 64;

// What a CU holds at once.  128-wide heads: three workgroups, by keeping a wave at
// 168 registers and the values in one LDS stage (48 KB), loaded while their tile's
// weights are formed -- against two with two stages, on two boxes: 16384 tokens x 32/4
// 2.01 -> 1.95 and 1.96 -> 1.85 ms, the 32 prompts above 171 -> 163 and 168 -> 160 us,
// 4096 x 32/8 150 -> 138 us, and 2% slower where a workgroup has a CU to itself.  64-wide heads fit four with two
// stages (one: 64 us for 60 at 4096 x 16/16); 192-wide ones fit two either way.
template <int DQ>
constexpr int kPromptPerSimd = DQ == 64 ? 4 : (DQ == 128 ? 3 : 2);
template <int DQ>
constexpr int kPromptValStages = DQ == 128 ? 1 : 2;

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int32_t total_q, total_k;
  int32_t num_seqs, q_heads, kv_heads;
  uint32_t g_mul;     // n / G = n * g_mul >> 32 + g_shift, see div_g
  int32_t g_shift;
  float c;            // scale * log2(e)
  // SPLIT: part s of row r (token * q_heads + head) is entry r * splits + s
  float* part_o;      // [entries][DV]
  float2* part_ml;    // [entries]: maximum (base 2), weight sum
  int32_t splits;
};

// n / G for 0 <= n < 2^31: with 2^(s - 1) < G <= 2^s and p = 31 + s, g_mul =
// ceil(2^p / G) = (2^p + e) / G, 0 <= e < G, so n * g_mul / 2^p = n / G + n e / (G 2^p),
// and n e < 2^p: less than 1 / G too much, which never reaches the next whole number.
__device__ __forceinline__ int div_g(const PromptArgs& a, int n) {
  return a.g_shift < 0 ? n : (int)(__umulhi((uint32_t)n, a.g_mul) >> a.g_shift);
}

struct PromptTile {
  int q0, k0;         // the sequence's first query and key
  int lq, lk;         // its lengths
  int row0, rows;     // the tile's first row, the sequence's rows (lq * G)
};

// Row tiles without a plan made beforehand: sequence b owns the virtual tiles
// from cu_q[b] * G / 128 + b on, at least as many as it needs, so a tile's
// sequence is found by searching cu_q itself (64 probes at a time), and
// total_q * G / 128 + num_seqs workgroups per key head cover any lengths.  Tiles
// past a sequence's end have row0 >= rows.  Within a sequence the last tile (the
// one that sees most keys) comes first.
// (total_q * G < 2^31, checked on the host.)
__device__ __forceinline__ PromptTile prompt_tile(const PromptArgs& a, int vt, int G, int lane) {
  auto cu = [&](const int32_t* p, int i, int total) { return min(max(p[i], 0), total); };
  PromptTile t;
  int b;
  if (a.num_seqs <= 64) {
    // lane b holds sequence b: one round of loads
    const int at = min(lane, a.num_seqs - 1);
    const int q0 = cu(a.cu_q, at, a.total_q), q1 = cu(a.cu_q, at + 1, a.total_q);
    const int k0 = cu(a.cu_k, at, a.total_k), k1 = cu(a.cu_k, at + 1, a.total_k);
    const uint64_t mask = __ballot(lane < a.num_seqs && q0 * G / kPromptRows + lane <= vt) | 1;
    b = 63 - __builtin_clzll(mask);
    t.q0 = __builtin_amdgcn_readlane(q0, b);
    t.lq = __builtin_amdgcn_readlane(q1, b) - t.q0;
    t.k0 = __builtin_amdgcn_readlane(k0, b);
    t.lk = __builtin_amdgcn_readlane(k1, b) - t.k0;
  } else {
    int lo = 0, n = a.num_seqs;
    while (n > 1) {
      const int stride = (n + 63) >> 6, off = lane * stride;
      const bool le = off < n && cu(a.cu_q, lo + off, a.total_q) * G / kPromptRows + lo + off <= vt;
      const int seg = (63 - __builtin_clzll(__ballot(le) | 1)) * stride;
      lo += seg;
      n = min(stride, n - seg);
    }
    b = __builtin_amdgcn_readfirstlane(lo);
    t.q0 = cu(a.cu_q, b, a.total_q);
    t.lq = cu(a.cu_q, b + 1, a.total_q) - t.q0;
    t.k0 = cu(a.cu_k, b, a.total_k);
    t.lk = cu(a.cu_k, b + 1, a.total_k) - t.k0;
  }
  t.lq = max(t.lq, 0);
  t.lk = max(t.lk, 0);
  t.rows = t.lq * G;
  const int idx = vt - (t.q0 * G / kPromptRows + b), need = (t.rows + kPromptRows - 1) / kPromptRows;
  t.row0 = idx < 0 || idx >= need ? t.rows : (need - 1 - idx) * kPromptRows;
  return t;
}

// The wave's results from the accumulators to memory, or as a part to the workspace.
// Whether some of the workgroup's is not finite (never with CAREFUL).
template <int DQ, int DV, bool CAREFUL, bool SPLIT, class W, class Row>
__device__ __forceinline__ bool prompt_store(const PromptArgs& a, const W& w, uint32_t thread, int wrow, int wv, int part,
                                             const PromptTile& T, const Row& row_of, uint8_t* ks) {
  asm volatile("" : "+v"(thread));                                  // (nothing of this is held in registers before)
  const int lane = thread & 63, h = lane >> 5;
  int row, hq;
  row_of(lane, row, hq);
  at_wait_barrier<0>();                                             // everyone is done with the stages
  // The results go through LDS, so that stores write whole rows (2.6 us of a
  // workgroup's time as 8-byte pieces, 1.6 us so): 16-byte chunk c of row r lies at
  // chunk c ^ r of the keys' stages, a quarter per wave.
  constexpr int CH = DV / 8;
  static_assert(4 * 32 * DV * 2 <= 2 * W::kKeyBytes, "");
  uint8_t* rows = ks + wv * (32 * DV * 2);
  float odd = 0.0f;                                                 // NaN once some result is not finite
  if (SPLIT) {
    if (wrow + (lane & 31) < T.rows) {
      const int64_t entry = ((int64_t)(T.q0 + row) * a.q_heads + hq) * a.splits + part;
      float* po = a.part_o + entry * DV + 4 * h;
#pragma unroll
      for (int b = 0; b < W::OB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(f32x4*)(po + 32 * b + 8 * i) = f32x4{w.o[b][4 * i], w.o[b][4 * i + 1], w.o[b][4 * i + 2], w.o[b][4 * i + 3]};
      if (h == 0) a.part_ml[entry] = float2{w.m, w.l};
    }
    if (!CAREFUL) {
#pragma unroll
      for (int b = 0; b < W::OB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) odd = fmaf(w.o[b][i], 0.0f, odd);
    }
  } else {
    const float inv = w.l == 0.0f ? 0.0f : 1.0f / w.l;
#pragma unroll
    for (int b = 0; b < W::OB; ++b)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = w.o[b][4 * i + j] * inv;
          if (!CAREFUL) odd = fmaf(y[j], 0.0f, odd);
        }
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          // the halves of the wave hold 4 columns each of groups i and i + 1 of 8; each gets one group
          const auto x = __builtin_amdgcn_permlane32_swap(cvt_bf16x2(y[j], y[j + 1]), cvt_bf16x2(y[4 + j], y[5 + j]), false, false);
          v[j / 2] = x[0];
          v[2 + j / 2] = x[1];
        }
        const int r = lane & 31, c = 4 * b + i + h;
        *(u32x4*)(rows + r * (DV * 2) + ((c ^ (r & (CH - 1))) * 16)) = v;
      }
    asm volatile("" ::: "memory");                                    // (a wave's own LDS accesses stay in order)
    const int64_t at = (int64_t)(T.q0 + row) * a.o_ts + hq * a.o_hs;
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; ++i) {
      const int r = (i * 64 + lane) / CH, c = lane % CH;
      const u32x4 v = *(const u32x4*)(rows + r * (DV * 2) + ((c ^ (r & (CH - 1))) * 16));
      const int64_t to = (int64_t)__shfl((long long)at, r);
      if (wrow + r < T.rows) *(u32x4*)(a.out + to + c * 8) = v;
    }
    if (a.lse && h == 0 && wrow + (lane & 31) < T.rows)
      a.lse[(int64_t)(T.q0 + row) * a.q_heads + hq] = w.l == 0.0f ? neg_inf() : (w.m + __builtin_amdgcn_logf(w.l)) * kLn2;
  }
  if (CAREFUL) return false;
  // each wave's word, in its quarter
  if (lane == 0) *(int*)rows = 0;
  if (odd != odd) *(int*)rows = 1;
  at_wait_barrier<63>();                                            // (the stores are not waited for)
  int any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= *(const int*)(ks + i * (32 * DV * 2));
  return any != 0;
}

// The rows of workgroup `block`, this is its thread `thread`.  Whether some result
// is not finite; in that case the workgroup's rows have to be done again,
// CAREFUL: a value that is infinite or NaN reaches the rows that see it only.
// (Testing the values of each masked tile beforehand took half as long as the tile.)
// SPLIT: one of `splits` workgroups for the same rows, an equal run of their tiles
// of keys each.
template <int DQ, int DV, bool CAREFUL, bool SPLIT>
__device__ __forceinline__ bool prompt_rows(const PromptArgs& a, uint32_t block, uint32_t thread, uint8_t* ks, uint8_t* vs) {
  using W = AttnWave<DQ, DV, kPromptKeys / 32>;
  constexpr int kThreads = kPromptThreads;
  constexpr int VS = kPromptValStages<DQ>;
  const int lane = thread & 63, wv = __builtin_amdgcn_readfirstlane(thread >> 6);
  // the key head varies fastest: workgroups go to the XCDs in turn, so one key
  // head's workgroups meet in few L2s
  const int G = a.q_heads / a.kv_heads;
  const int kvh = block % (uint32_t)a.kv_heads;
  const uint32_t item = block / (uint32_t)a.kv_heads;
  const int part = SPLIT ? (int)(item % (uint32_t)a.splits) : 0;
  const PromptTile T = prompt_tile(a, (int)(SPLIT ? item / (uint32_t)a.splits : item), G, lane);
  if (T.row0 >= T.rows) return false;
  const int wrow = T.row0 + wv * 32;
  // this lane's row: its token and head (rows past the end repeat the last)
  auto row_of = [&](int l, int& row, int& hq) {
    const int m = min(wrow + (l & 31), T.rows - 1);
    row = div_g(a, m);
    hq = kvh * G + m - row * G;
  };
  int row, hq;
  row_of(lane, row, hq);
  const int pos = row + T.lk - T.lq;                                // last key this row sees
  // the last key that a row of the workgroup sees, and one of this wave; keys that
  // all its rows see
  auto key_of = [&](int r) { return div_g(a, min(r, T.rows - 1)) + T.lk - T.lq; };
  const int n_keys = max(0, key_of(T.row0 + kPromptRows - 1) + 1);
  const int wave_last = key_of(wrow + 31), all_see = key_of(T.row0) + 1;
  const uint16_t* kp = a.k + (int64_t)T.k0 * a.k_ts + kvh * a.k_hs;
  const uint16_t* vp = a.v + (int64_t)T.k0 * a.v_ts + kvh * a.v_hs;
  // Each lane's share of a tile: 16-byte chunk i * threads + thread of the
  // swizzled tile, i.e. of row r the chunk that belongs there; its offset from
  // the tile's first row in memory.  Rows past the last key repeat it.
  constexpr int kKeyLoads = W::kKeyBytes / 16 / kThreads, kValLoads = W::kValBytes / 16 / kThreads;
  const uint32_t k_row = (uint32_t)(a.k_ts * 2), v_row = (uint32_t)(a.v_ts * 2);   // bytes; a tile spans < 2 GiB (host)
  auto k_off = [&](int i, int end, uint32_t th) {
    const int f = i * kThreads + (int)th, r = f / (DQ / 8);
    return (uint32_t)min(r, end) * k_row + (uint32_t)((f % (DQ / 8)) ^ at_swz<DQ>(r)) * 16u;
  };
  auto v_off = [&](int i, int end, uint32_t th) {
    const int f = i * kThreads + (int)th, r = f / (DV / 8);
    return (uint32_t)min(r, end) * v_row + (uint32_t)((f % (DV / 8)) ^ at_swz<DV>(r)) * 16u;
  };
  // Where a tile's share is whole rows, load i is load 0 further on by a uniform
  // number of rows (a multiple of 16, after which the swizzle repeats).
  constexpr bool kUniK = kThreads % (DQ / 8) == 0;
  static_assert(kThreads % (DV / 8) == 0, "");
  const uint32_t k_step = kThreads / (DQ / 8) * k_row, v_step = kThreads / (DV / 8) * v_row;
  uint32_t koff[kUniK ? 1 : kKeyLoads], voff = v_off(0, kPromptKeys - 1, thread);
  asm volatile("" : "+v"(voff));                                    // (kept as 32 bits, not as the product it came from)
#pragma unroll
  for (int i = 0; i < (kUniK ? 1 : kKeyLoads); ++i) {
    koff[i] = k_off(i, kPromptKeys - 1, thread);
    asm volatile("" : "+v"(koff[i]));
  }
  const uint32_t k_lds = at_lds_addr(ks) + (uint32_t)wv * 1024u, v_lds = at_lds_addr(vs) + (uint32_t)wv * 1024u;
  // (the last tile's own offsets are formed where they are used, from an opaque copy
  // of the thread's number: nothing of them is held in registers meanwhile)
  auto load_k = [&](int t, int st) {
    const int key0 = t * kPromptKeys, end = T.lk - 1 - key0;
    const at_rsrc kr = at_make_rsrc(kp + key0 * a.k_ts);
    const uint32_t kt = k_lds + (uint32_t)(st * W::kKeyBytes);
    if (end >= kPromptKeys - 1) {
#pragma unroll
      for (int i = 0; i < kKeyLoads; ++i) at_load_lds(kt + i * kThreads * 16, kr, koff[kUniK ? 0 : i], kUniK ? i * k_step : 0);
    } else {
      uint32_t th = thread;
      asm volatile("" : "+v"(th));
#pragma unroll
      for (int i = 0; i < kKeyLoads; ++i) at_load_lds(kt + i * kThreads * 16, kr, k_off(i, end, th), 0);
    }
  };
  auto load_v = [&](int t, int st) {
    const int key0 = t * kPromptKeys, end = T.lk - 1 - key0;
    const at_rsrc vr = at_make_rsrc(vp + key0 * a.v_ts);
    const uint32_t vt = v_lds + (uint32_t)(st * W::kValBytes);
    if (end >= kPromptKeys - 1) {
#pragma unroll
      for (int i = 0; i < kValLoads; ++i) at_load_lds(vt + i * kThreads * 16, vr, voff, i * v_step);
    } else {
      uint32_t th = thread;
      asm volatile("" : "+v"(th));
#pragma unroll
      for (int i = 0; i < kValLoads; ++i) at_load_lds(vt + i * kThreads * 16, vr, v_off(i, end, th), 0);
    }
  };
  const int all_tiles = (n_keys + kPromptKeys - 1) / kPromptKeys;
  const int run = SPLIT ? (all_tiles + a.splits - 1) / a.splits : all_tiles;
  const int t0 = SPLIT ? min(part * run, all_tiles) : 0, n_tiles = SPLIT ? min(t0 + run, all_tiles) : all_tiles;
  // tiles that every row of the workgroup sees whole come first; for the others
  // (around the diagonal) each wave looks whether it sees any of it at all
  const int n_whole = max(0, min(n_tiles, all_see / kPromptKeys));
  auto seen = [&](int t) { return t * kPromptKeys <= wave_last; };
  if (n_tiles > t0) {                                               // under way while the queries are read
    load_k(t0, 0);
    if (VS == 2) load_v(t0, 0);
  }
  W w;
  w.init(a.q + (int64_t)(T.q0 + row) * a.q_ts + hq * a.q_hs, lane);
  // Keys of tile t (with two stages its values too) have landed, and everyone is
  // done with tile t - 1, whose stages the next loads refill.
  auto begin = [&](int t, int st) {
    at_wait_barrier<0>();
    if (VS == 1) load_v(t, 0);
    if (t + 1 < n_tiles) {
      load_k(t + 1, st ^ 1);
      if (VS == 2) load_v(t + 1, st ^ 1);
    }
  };
  // before the values are used: with one stage they are still under way, and the
  // next tile's keys behind them
  auto landed = [&](int t) {
    if (VS == 2) return;
    if (t + 1 < n_tiles) at_wait_barrier<kKeyLoads>();
    else at_wait_barrier<0>();
  };
  const bool real = wrow < T.rows;                                  // some row of this wave is
  int t = t0;
  if (!CAREFUL) {
    auto step = [&](auto stage, int tile) {
      constexpr int st = decltype(stage)::value;
      begin(tile, st);
      if (real) {
        w.scores(ks + st * W::kKeyBytes);
        w.weights(a.c);
      }
      landed(tile);
      if (real) w.values(vs + (VS == 2 ? st : 0) * W::kValBytes);
    };
    for (; t + 1 < n_whole; t += 2) {
      step(std::integral_constant<int, 0>(), t);
      step(std::integral_constant<int, 1>(), t + 1);
    }
  }
  // (a last odd whole tile goes with the others)
#pragma unroll 1
  for (; t < n_tiles; ++t) {
    const int st = (t - t0) & 1;
    begin(t, st);
    const bool now = real && seen(t);
    if (now) {
      w.scores(ks + st * W::kKeyBytes);
      w.mask(lane, pos - t * kPromptKeys);
      w.weights(a.c);
    }
    landed(t);
    if (!now) continue;
    // A value that a row does not see has weight 0; an infinity or a NaN among them
    // makes the row's result NaN all the same, which the end notices.
    const uint8_t* v = vs + (VS == 2 ? st : 0) * W::kValBytes;
    if (CAREFUL) w.values_careful(v, lane, pos - t * kPromptKeys);
    else w.values(v);
  }
  return prompt_store<DQ, DV, CAREFUL, SPLIT>(a, w, thread, wrow, wv, part, T, row_of, ks);
}

template <int DQ, int DV, bool SPLIT>
__global__ __launch_bounds__(kPromptThreads, kPromptPerSimd<DQ>) void attn_prompt_kernel(PromptArgs a) {
  using W = AttnWave<DQ, DV, kPromptKeys / 32>;
  __shared__ __attribute__((aligned(16))) uint8_t ks[2 * W::kKeyBytes];
  __shared__ __attribute__((aligned(16))) uint8_t vs[kPromptValStages<DQ> * W::kValBytes];
  uint32_t block = blockIdx.x, thread = threadIdx.x;
  if (!prompt_rows<DQ, DV, false, SPLIT>(a, block, thread, ks, vs)) return;
  // (opaque copies: nothing of the first run is kept in registers for this one)
  asm volatile("" : "+s"(block));
  asm volatile("" : "+v"(thread));
  at_wait_barrier<0>();                                             // everyone has read the words; the stages are refilled
  prompt_rows<DQ, DV, true, SPLIT>(a, block, thread, ks, vs);
}

// The parts of the rows joined, a wave per row: M = max m_s, then
// out = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s.  At most 64 parts, lane s weighs
// part s.  Rows outside the sequences are left alone.
template <int DV>
__global__ __launch_bounds__(256) void attn_prompt_join_kernel(PromptArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = r / a.q_heads;
  const int hq = (int)(r % a.q_heads);
  if (token < min(max(a.cu_q[0], 0), a.total_q) || token >= min(max(a.cu_q[a.num_seqs], 0), a.total_q)) return;
  constexpr int E = DV / 64;                                        // values per lane
  float2 x = float2{neg_inf(), 0.0f};
  if (lane < a.splits) x = a.part_ml[r * a.splits + lane];
  float M = x.x;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor(M, d));
  const float e = __builtin_amdgcn_exp2f(x.x - (M == neg_inf() ? 0.0f : M));
  float L = x.y * e, o[2] = {0.0f, 0.0f};
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) L += __shfl_xor(L, d);
  const float* src = a.part_o + r * a.splits * DV + lane * E;
  for (int s0 = 0; s0 < a.splits; s0 += 8) {                        // 8 loads in flight
    float y[8][2];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float* p = src + (int64_t)min(s0 + u, a.splits - 1) * DV;
      y[u][0] = p[0];
      if (E == 2) y[u][1] = p[1];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (s0 + u >= a.splits) break;
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), s0 + u));
      o[0] = fmaf(w, y[u][0], o[0]);
      if (E == 2) o[1] = fmaf(w, y[u][1], o[1]);
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* dst = a.out + token * a.o_ts + hq * a.o_hs + lane * E;
  if (E == 2) *(uint32_t*)dst = cvt_bf16x2(o[0] * inv, o[1] * inv);
  else *dst = (uint16_t)f32_to_bf16_bits(o[0] * inv);
  if (a.lse && lane == 0) a.lse[r] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

static int64_t prompt_tiles(int64_t total_q, int64_t G, int64_t num_seqs) { return total_q * G / kPromptRows + num_seqs; }

// Workgroups that share a tile of rows.  The lengths are not known here: the average
// number of keys counts, in tiles.  A tile takes 1.0 us (128-wide heads) while there
// is a workgroup per CU at most, 1.7 with two, 2.3 with three; parts cost 6 us for the second
// launch and their floats written and read at 4 TB/s.  16 tokens on 4096 keys x 32/8
// x 128: 14 us for 71 unsplit; 128 on 8192: 39 for 135; 512 on 8192: 88 for 140.
// Never with less than 512 keys on average, which the callers may rely on.
static int prompt_splits(int64_t total_q, int64_t total_k, int64_t num_seqs, int64_t q_heads, int64_t kv_heads, int64_t k_dim,
                         int64_t v_dim) {
  if (num_seqs <= 0 || total_q <= 0 || total_k < 512 * num_seqs) return 1;
  const int64_t groups = prompt_tiles(total_q, q_heads / kv_heads, num_seqs) * kv_heads;
  if (groups > 256) return 1;
  const int64_t n = (total_k / num_seqs + kPromptKeys - 1) / kPromptKeys, unit = (k_dim + v_dim) * 1000 / 256;   // ns
  const int64_t part = total_q * q_heads * (v_dim * 4 + 8) / 2000;   // ns
  int best = 1;
  int64_t least = unit * n;
  const int64_t per_cu = k_dim == 64 ? kPromptPerSimd<64> : (k_dim == 128 ? kPromptPerSimd<128> : kPromptPerSimd<192>);
  const int64_t most = std::min<int64_t>(std::min<int64_t>(64, 256 * per_cu / groups), n / 2);
  const int64_t slower[4] = {10, 17, 23, 30};                       // by workgroups on a CU, tenths
  for (int64_t s = 2; s <= most; ++s) {
    const int64_t time = unit * slower[(groups * s - 1) / 256] / 10 * ((n + s - 1) / s) + 6000 + s * part;
    if (time < least) {
      least = time;
      best = (int)s;
    }
  }
  return best;
}

size_t attn_prompt_ws_bytes(int64_t total_q, int64_t total_k, int64_t num_seqs, const moe_attn_params& p) {
  const int s = prompt_splits(total_q, total_k, num_seqs, p.q_heads, p.kv_heads, p.k_dim, p.v_dim);
  return s == 1 ? 0 : (size_t)(total_q * p.q_heads * s) * ((size_t)p.v_dim * 4 + 8);
}

template <int DQ, int DV>
static void launch_prompt(const PromptArgs& a, hipStream_t stream) {
  const int64_t groups = prompt_tiles(a.total_q, a.q_heads / a.kv_heads, a.num_seqs) * a.kv_heads;
  if (a.splits == 1) {
    hipLaunchKernelGGL((attn_prompt_kernel<DQ, DV, false>), dim3((uint32_t)groups), dim3(kPromptThreads), 0, stream, a);
    return;
  }
  hipLaunchKernelGGL((attn_prompt_kernel<DQ, DV, true>), dim3((uint32_t)(groups * a.splits)), dim3(kPromptThreads), 0, stream, a);
  hipLaunchKernelGGL((attn_prompt_join_kernel<DV>), dim3((uint32_t)(((int64_t)a.total_q * a.q_heads + 3) / 4)), dim3(256), 0,
                     stream, a);
}

moe_status launch_attn_prompt(const moe_heads& q, const moe_heads& k, const moe_heads& v, const int32_t* cu_q,
                              const int32_t* cu_k, int num_seqs, int64_t total_q, int64_t total_k,
                              const moe_attn_params& p, const moe_heads& out, float* lse, void* ws, hipStream_t stream) {
  PromptArgs a;
  a.splits = prompt_splits(total_q, total_k, num_seqs, p.q_heads, p.kv_heads, p.k_dim, p.v_dim);
  a.part_o = (float*)ws;
  a.part_ml = (float2*)(a.part_o + total_q * p.q_heads * a.splits * p.v_dim);
  a.q = (const uint16_t*)q.data;
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.k = (const uint16_t*)k.data;
  a.k_ts = k.token_stride;
  a.k_hs = k.head_stride;
  a.v = (const uint16_t*)v.data;
  a.v_ts = v.token_stride;
  a.v_hs = v.head_stride;
  a.out = (uint16_t*)out.data;
  a.o_ts = out.token_stride;
  a.o_hs = out.head_stride;
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.num_seqs = num_seqs;
  a.total_q = (int32_t)total_q;
  a.total_k = (int32_t)total_k;
  a.q_heads = p.q_heads;
  a.kv_heads = p.kv_heads;
  const uint32_t G = (uint32_t)(p.q_heads / p.kv_heads);
  const int bits = G == 1 ? 0 : 32 - __builtin_clz(G - 1);          // 2^(bits - 1) < G <= 2^bits
  a.g_shift = bits - 1;
  a.g_mul = G == 1 ? 0 : (uint32_t)((((uint64_t)1 << (31 + bits)) + G - 1) / G);
  a.c = p.scale * kLog2e;
  if (p.k_dim == 64) launch_prompt<64, 64>(a, stream);
  else if (p.k_dim == 128) launch_prompt<128, 128>(a, stream);
  else launch_prompt<192, 128>(a, stream);
  return launch_status("moe_attn_prompt");
}

}  // namespace moe
