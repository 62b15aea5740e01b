// Attention of one new token per request over a paged cache held in 4 bits (NVFP4: E2M1
// codes, an E4M3 scale for 16 values, a power-of-two scale for all keys and all
// values), with a prefix that all requests share.
//
//   out[b, h] = sum_j p_j v_j over the prefix's keys and request b's own keys,
//   p = softmax of q[b, h] . k_j * scale over both together.
//
// Split over the keys and joined as for a bf16 cache (attn_decode.hip).  What differs is
// the way from memory to the matrix cores.  Codes times scales are f16 values exactly, so
// the products run on f16 operands, keys' and values' alike; queries are f16 times a power
// of two of their row.  A quarter of the bytes comes from memory, and vector work takes
// their place: 8 codes need 4 converts and 4 packed multiplications.
//
// narrow (own keys, and a prefix with few rows): every wave takes tiles of 64 keys by
//   itself.  Keys go from memory into the registers where the product wants them, in 16-byte
//   pieces of a row: the product's k index is enumerated as the pieces hold it.  Values go
//   through the wave's own LDS as codes and come back transposed (ds_read_b64_tr_b4: 16
//   lanes read 16 rows of 16 codes, each receives one column's), 16 keys of one column to a
//   lane; the scores' accumulators give the weights of just these keys.  The next tile's
//   loads are under way while one is computed on; no barrier but at a request's end, where
//   the workgroup's waves join their sums in LDS.
// wide (prefix, many rows): a workgroup's 128 rows meet 64 keys at a time, which its
//   threads have turned into f16 rows in LDS; from there on it is the bf16 form's.
// alone (few keys): a workgroup's waves share all tiles of a request and key head, join their
//   sums in LDS and write the result: one launch.
//
// What bounds it.  Own keys: reads.  1 request of 131072 keys (32 / 8 heads of 128 + 128, 151 MB)
// takes 29.5 us in the kernel and 5.5 in the join; each further key costs what 6.3 TB/s give
// (contiguous reads reach 6.9), the rest are a few dependent trips at the start (lengths, table,
// codes: 4 us), the waves' unequal ends and the join's launch.  48 requests of up to
// 16384 keys (64 / 4 heads of 192 + 128, 268 MB): 54 + 5 us; their lists of unequal requests
// end unevenly, a CU's older workgroups 10 us before its younger ones -- turns by wave
// priority moved that by nothing.  Prefix: 96 requests behind 32768 keys (64 / 4 heads of 192 +
// 128) 155 + 8 us, 0.83 PFLOP/s; matrix cores 39% busy, vector work (conversions, exponentials)
// 45%, LDS 40%, on two waves for each SIMD, whose registers (232 to 255) leave no room for a
// third.  64 behind 8192 (64 / 8 of 128 + 128) 38 + 7 us, 0.45 PFLOP/s, 17%, 27%, 18%: a workgroup
// has few tiles to its fill, its parts (29 MB in all) and the join.  8 requests behind 777 keys,
// alone: 9.3 us, 64 workgroups on 256 CUs, whose waves take up to three tiles one after the other
// (of one tile 6.4 us, of two 8.6, of four 12.8, of eight 21.4: 2.1 each).
#include <algorithm>
#include <cmath>

#include "attn_common.h"
#include "attn_join.h"

namespace moe {

constexpr int kF4Keys = 64;                         // per tile
constexpr int kF4Waves = 4;                         // of a workgroup that leaves parts

struct Fp4Plan {
  int32_t small;                                    // waves of a workgroup that answers alone: no parts, the rest is 0
  int32_t wide;                                     // prefix workgroups are wide
  int32_t parts_p, chunk_p;                         // parts of the prefix, keys in each
  int32_t blocks_p;                                 // row blocks of B * G rows (wide 128, narrow 16 rb)
  int32_t rb;                                       // narrow workgroups take 16 rb rows
  int32_t blocks_s, rows_s;                         // row blocks of G rows, rows in each
  int32_t runs;                                     // narrow workgroups per key head and row block
};

struct Fp4Args {
  const uint16_t* q;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const uint8_t* k;
  const uint8_t* ks;
  const uint8_t* v;
  const uint8_t* vs;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* prefix_table;
  int64_t prefix_len, max_len;
  uint16_t* out;
  float* lse;
  float* part_o;                                    // as JoinArgs says, one part per workgroup
  float2* part_ml;
  int32_t* first;
  int64_t own;
  int32_t num_requests, q_heads, kv_heads, num_pages, page_shift;
  float c, v_scale;
  int32_t c_exp;                                    // scale times log2(e) times the keys' global is c 2^c_exp
  Fp4Plan plan;
};

// What a row's scores are multiplied by, its queries being f16 times 2^-e.  Multiplied by zero
// or infinity a score of -inf (a key that is not there) or 0 would be NaN.  Scores are below
// 2^34, so with the smallest normal number they are all next to zero, as with any below it; where
// the factor passes 2^127, those whose row's largest query value counts pass float's range.
__device__ __forceinline__ float score_factor(const Fp4Args& a, int e) {
  return fminf(fmaxf(ldexpf(a.c, a.c_exp + e), 0x1p-126f), 0x1p127f);
}

__device__ __forceinline__ int f4_clamp_len(const Fp4Args& a, int len) { return (int)min((int64_t)max(len, 0), a.max_len); }
__device__ __forceinline__ int f4_len_at(const Fp4Args& a, int b) {   // b uniform: a scalar load
  return f4_clamp_len(a, *(const __attribute__((address_space(4))) int32_t*)(a.lens + b));
}
__device__ __forceinline__ int f4_tiles(int keys) { return (keys + kF4Keys - 1) / kF4Keys; }

// Inclusive sum over the wave's lanes: within rows of 16, then their last lanes on.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return x;
}

__device__ __forceinline__ f16x2 f16_pair(uint32_t w) { return __builtin_bit_cast(f16x2, w); }

// Two E4M3 bytes (word SEL of w) as f16: exact.
template <bool SEL>
__device__ __forceinline__ f16x2 scale_pair(uint32_t w) { return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, SEL); }

// 8 codes times their scales: s0 .. s3 for the pairs.
__device__ __forceinline__ f16x8 fp4x8_f16(uint32_t w, f16x2 s0, f16x2 s1, f16x2 s2, f16x2 s3) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s0;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s1;
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s2;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s3;
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ f16x8 fp4x8_f16(uint32_t w, _Float16 s) {
  const f16x2 p = {s, s};
  return fp4x8_f16(w, p, p, p, p);
}

// Rows of one group of 16 keys: a buffer from their uniform address on, so that a load takes
// the lane's 32-bit offset as it is.  (Of 64-bit addresses base and lane offset are added up
// ahead of the loop, two registers for every load of a tile.)
__device__ __forceinline__ rsrc_t group_rsrc(const uint8_t* p) { return make_rsrc(p, 0x7fffffffu); }

typedef int f4_i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) f4_i32x2 f4_lds_i32x2;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16_f16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// One wave's tile of 64 keys against 16 RB query rows.  Lane l, r = l % 16, g = l / 16:
// scores s[rb][t][i] of row r and key 16 t + 4 g + i; sums o[rb][b][i] of row r and value
// column 16 b + 4 g + i.
template <int DQ, int DV, int RB>
struct Fp4Wave {
  static constexpr int KS = DQ / 32, OB = DV / 16;
  static constexpr int kCodes = kF4Keys * DV / 2;                   // bytes of LDS: codes, then scales as f16
  static constexpr int kStage = kCodes + OB * kF4Keys * 2;
  static constexpr int kOut = DV + 4;                               // floats of a row of sums (padded: banks)
  static constexpr int kRegion = kStage > 16 * kOut * 4 + 128 ? kStage : 16 * kOut * 4 + 128;
  static constexpr int kEntryKeys = DV == 128 ? 8 : 4;              // keys that a lane's piece of the values' scales covers
  f16x8 q[RB][KS];
  f32x4 o[RB][OB], s[RB][4];
  f16x8 p[RB][2];
  float m[RB], l[RB], c[RB];
  // a tile on its way
  uint32_t kc[4][KS], kscale[4], kscale2[DQ == 192 ? 4 : 1];
  u32x4 vc[DV / 32];
  uint32_t vscale[DV / 64];
  uint32_t tr;                                                      // this lane's offset of the transposing reads

  __device__ __forceinline__ void setup(int lane) {
    const int g = lane >> 4, t = (lane >> 2) & 3, i = lane & 3;
    if (DV == 128) tr = (uint32_t)((16 * t + 4 * g + i) * 64 + t * 16);
    else tr = (uint32_t)((t >> 1) * 1024 + (8 * g + 4 * (t & 1) + i) * 32 + (t >> 1) * 16);
  }
  // first column of this lane's k index in step s
  __device__ __forceinline__ static int column(int g, int s) {
    if (DQ == 64) return 16 * g + 8 * s;
    return s < 4 ? 32 * g + 8 * s : 128 + 16 * g + 8 * (s - 4);
  }
  // row: this lane's query row of block rb
  __device__ __forceinline__ void load_query(int rb, const uint16_t* row, int lane) {
#pragma unroll
    for (int k = 0; k < KS; ++k) q[rb][k] = __builtin_bit_cast(f16x8, *(const u32x4*)(row + column(lane >> 4, k)));
  }
  __device__ __forceinline__ void init(int rb, const Fp4Args& a) {
    u32x4 x[KS];
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) x[k] = __builtin_bit_cast(u32x4, q[rb][k]);
#pragma unroll
    for (int k = 0; k < KS; ++k) most = query_most(x[k], most);
    const int e = query_exponent(quarter_max(most));
#pragma unroll
    for (int k = 0; k < KS; ++k) q[rb][k] = query_f16(x[k], e);
    c[rb] = score_factor(a, e);
#pragma unroll
    for (int b = 0; b < OB; ++b) o[rb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[rb] = neg_inf();
    l[rb] = 0.0f;
  }
  // The tile's loads: keys of 16 at a time, and all values.  ONCE: nothing reads them again
  // (non-temporal: 131072 own keys 33.2 -> 30.5 us).  slot: lane's cache row (page << shift |
  // row) of the tile's key kEntryKeys * (lane % (64 / kEntryKeys)), the last group of 16 keys
  // for those behind it.
  // (rows of a head before a cache row: page * heads + head pages of them, and the row)
  __device__ __forceinline__ static uint64_t rows_at(const Fp4Args& a, int kvh, uint32_t slot) {
    return ((uint64_t)((int64_t)(slot >> a.page_shift) * a.kv_heads + kvh) << a.page_shift) + (slot & ((1u << a.page_shift) - 1u));
  }
  __device__ __forceinline__ static uint64_t group_at(const Fp4Args& a, int kvh, int slot, int t) {
    return rows_at(a, kvh, (uint32_t)__builtin_amdgcn_readlane(slot, t * (16 / kEntryKeys)));
  }
  template <bool ONCE>
  __device__ __forceinline__ void load_keys(const Fp4Args& a, int kvh, int slot, int lane, int t) {
    const int g = lane >> 4, r = lane & 15;
    const uint64_t at = group_at(a, kvh, slot, t);
    const rsrc_t kp = group_rsrc(a.k + at * (DQ / 2)), sp = group_rsrc(a.ks + at * (DQ / 16));
    if (DQ == 64) {
      const u32x2 x = ONCE ? bload64_nt(kp, r * 32 + 8 * g, 0) : bload64(kp, r * 32 + 8 * g, 0);
      kc[t][0] = x[0];
      kc[t][1] = x[1];
      kscale[t] = bload8(sp, r * 4 + g, 0);
    } else {
      const int at16 = r * (DQ / 2) + 16 * g;
      const u32x4 x = ONCE ? bload128_nt(kp, at16, 0) : bload128(kp, at16, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) kc[t][k] = x[k];
      kscale[t] = bload16(sp, r * (DQ / 16) + 2 * g, 0);
      if (DQ == 192) {
        const int at8 = r * 96 + 64 + 8 * g;
        const u32x2 y = ONCE ? bload64_nt(kp, at8, 0) : bload64(kp, at8, 0);
        kc[t][KS - 2] = y[0];
        kc[t][KS - 1] = y[1];
        kscale2[t] = bload8(sp, r * 12 + 8 + g, 0);
      }
    }
  }
  template <bool ONCE>
  __device__ __forceinline__ void load_values(const Fp4Args& a, int kvh, int slot, int lane) {
    if (DV == 128) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const rsrc_t vp = group_rsrc(a.v + group_at(a, kvh, slot, t) * 64);
        const int at = (lane >> 2) * 64 + ((lane & 3) ^ t) * 16;
        vc[t % (DV / 32)] = ONCE ? bload128_nt(vp, at, 0) : bload128(vp, at, 0);
      }
    } else {
      // two groups of 16 keys to a load: row 4 g' + i of group 2 h + t'
      const int p2 = lane >> 1, tt = (p2 >> 2) & 1, key = 4 * (p2 >> 3) + (p2 & 3);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t lo = group_at(a, kvh, slot, 2 * h), hi = group_at(a, kvh, slot, 2 * h + 1);
        vc[h] = *(const u32x4*)(a.v + ((tt ? hi : lo) + key) * 32 + ((lane & 1) ^ h) * 16);
      }
    }
    const int block = lane / (kF4Keys / kEntryKeys);
    const uint64_t page = (uint64_t)((uint32_t)slot >> a.page_shift) * a.kv_heads + kvh;
    const uint8_t* vp = a.vs + ((page * OB + block) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    if (DV == 128) {
      const u32x2 x = *(const u32x2*)vp;
      vscale[0] = x[0];
      vscale[DV / 64 - 1] = x[1];
    } else {
      vscale[0] = *(const uint32_t*)vp;
    }
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(const Fp4Args& a, int kvh, int slot, int lane) {
    load_values<ONCE>(a, kvh, slot, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) load_keys<ONCE>(a, kvh, slot, lane, t);
  }
  // Values' codes and scales of the tile that has come, into the wave's stage; those of keys
  // past `last` count as zero whatever lies there.
  __device__ __forceinline__ void store(uint8_t* mem, int lane, int last) {
#pragma unroll
    for (int i = 0; i < DV / 32; ++i) *(u32x4*)(mem + i * 1024 + lane * 16) = vc[i];
    const int x = lane % (kF4Keys / kEntryKeys), block = lane / (kF4Keys / kEntryKeys);
    if (last < kF4Keys - 1) {
#pragma unroll
      for (int w = 0; w < DV / 64; ++w) {
        const int there = last + 1 - (kEntryKeys * x + 4 * w);      // bytes that count
        vscale[w] = there >= 4 ? vscale[w] : (there <= 0 ? 0u : vscale[w] & ((1u << (8 * there)) - 1u));
      }
    }
#pragma unroll
    for (int w = 0; w < DV / 64; ++w) {
      const int first = kEntryKeys * x + 4 * w, t = first >> 4, g = (first >> 2) & 3;
      const f16x2 lo = scale_pair<false>(vscale[w]), hi = scale_pair<true>(vscale[w]);
      *(f16x4*)(mem + kCodes + block * (kF4Keys * 2) + g * 32 + t * 8) = f16x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
  // The tile's scores; MORE: the next tile's loads follow as soon as the registers they go to
  // are free (values' codes are in LDS by now).
  template <bool MORE, bool ONCE>
  __device__ __forceinline__ void scores(const Fp4Args& a, int kvh, int slot, int lane) {
    if (MORE) {
      __builtin_amdgcn_sched_barrier(0);                            // (not earlier, into registers of their own)
      load_values<ONCE>(a, kvh, slot, lane);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) s[rb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const f16x2 s01 = scale_pair<false>(kscale[t]), s2 = scale_pair<false>(kscale2[DQ == 192 ? t : 0]);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const f16x8 kf = fp4x8_f16(kc[t][k], k < 2 ? s01[0] : (k < 4 ? s01[1] : s2[0]));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb][t] = mfma16_f16(kf, q[rb][k], s[rb][t]);
      }
      if (MORE) {
        __builtin_amdgcn_sched_barrier(0);
        load_keys<ONCE>(a, kvh, slot, lane, t);
      }
    }
  }
  // keys past `last` are not there
  __device__ __forceinline__ void mask(int lane, int last) {
    const int seen = last - 4 * (lane >> 4);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[rb][t][i] = 16 * t + i <= seen ? s[rb][t][i] : neg_inf();
  }
  // as AttnWave::weights
  __device__ __forceinline__ void weights() {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      float mx = neg_inf();
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[rb][t][i]);
      mx = mul_rounded(quarter_max(mx), c[rb]) - AttnF16::kLift;
      const bool grown = has_grown<AttnF16>(mx, m[rb]);
      if (__any(grown)) {
        const float alpha = grown ? __builtin_amdgcn_exp2f(m[rb] - mx) : 1.0f;
        m[rb] = grown ? mx : m[rb];
        l[rb] *= alpha;
#pragma unroll
        for (int b = 0; b < OB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[rb][b][i] *= alpha;
      }
      const float base = m[rb] == neg_inf() ? 0.0f : m[rb];
      const float2 f = split_scale(base, c[rb]);
      if (__any(f.y == 1.0f)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[rb][t][i] = mul_rounded(s[rb][t][i], f.x);
      }
      float sum = 0.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] = __builtin_amdgcn_exp2f(fmaf(s[rb][2 * u + j / 4][j % 4], f.y, -base));
          sum += w[j];
        }
        p[rb][u] = __builtin_bit_cast(f16x8, u32x4{AttnF16::pair(w[0], w[1]), AttnF16::pair(w[2], w[3]),
                                                   AttnF16::pair(w[4], w[5]), AttnF16::pair(w[6], w[7])});
      }
      l[rb] += quarter_sum(sum);
    }
  }
  // (LDS is read one block of columns ahead of the products; left to itself the compiler reads
  // all of them at once, into registers that the loads under way need)
  __device__ __forceinline__ void values(const uint8_t* mem, int lane) {
    const uint8_t* sc = mem + kCodes + (lane >> 4) * 32;
    f4_i32x2 w[2];
    u32x4 sa[2], sb[2];
    auto read = [&](int b) {
      w[b & 1] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((f4_lds_i32x2*)(mem + (tr ^ ((b >> 1) * 16)) + (b & 1) * 8));
      sa[b & 1] = *(const u32x4*)(sc + b * (kF4Keys * 2));
      sb[b & 1] = *(const u32x4*)(sc + b * (kF4Keys * 2) + 16);
    };
    read(0);
#pragma unroll
    for (int b = 0; b < OB; ++b) {
      if (b + 1 < OB) read(b + 1);
      const u32x4 s0 = sa[b & 1], s1 = sb[b & 1];
      const f16x8 v0 = fp4x8_f16((uint32_t)w[b & 1][0], f16_pair(s0[0]), f16_pair(s0[1]), f16_pair(s0[2]), f16_pair(s0[3]));
      const f16x8 v1 = fp4x8_f16((uint32_t)w[b & 1][1], f16_pair(s1[0]), f16_pair(s1[1]), f16_pair(s1[2]), f16_pair(s1[3]));
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        o[rb][b] = mfma16_f16(v0, p[rb][0], o[rb][b]);
        o[rb][b] = mfma16_f16(v1, p[rb][1], o[rb][b]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // this wave's sums of block rb, maxima and weight sums into its region
  __device__ __forceinline__ void leave(uint8_t* mem, int rb, int lane) const {
    float* po = (float*)mem;
#pragma unroll
    for (int x = 0; x < OB; ++x) *(f32x4*)(po + (lane & 15) * kOut + 16 * x + 4 * (lane >> 4)) = o[rb][x];
    if (lane < 16) ((float2*)(po + 16 * kOut))[lane] = float2{m[rb], l[rb]};
  }
};

// The waves' sums of row `row`, columns col .. col + 3, joined.
template <int DV, int WAVES, int REGION>
__device__ __forceinline__ f32x4 join_waves(const uint8_t* mem, int row, int col, float* M, float* L) {
  constexpr int kOut = DV + 4;
  float2 ml[WAVES];
  *M = neg_inf();
  *L = 0.0f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    ml[i] = ((const float2*)((const float*)(mem + i * REGION) + 16 * kOut))[row];
    *M = fmaxf(*M, ml[i].x);
  }
  const float ref = *M == neg_inf() ? 0.0f : *M;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    const float e = __builtin_amdgcn_exp2f(ml[i].x - ref);
    const f32x4 o = *(const f32x4*)((const float*)(mem + i * REGION) + row * kOut + col);
    *L = fmaf(e, ml[i].y, *L);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fmaf(e, o[j], sum[j]);
  }
  return sum;
}

// Lane's part in finding a tile's rows: its key -- of the tile that begins at key `base` (of
// `len`), key KEYS * (lane % (64 / KEYS)), or in the last group of 16 where that is past the
// end -- and the table's entry for it.  The entry is loaded before the loads of the tile
// before, so that it is there without a wait for those.
struct Fp4Entry {
  int at, page;
  __device__ __forceinline__ int slot(const Fp4Args& a) const {
    return (min(max(page, 0), a.num_pages - 1) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
  }
};
template <int KEYS>
__device__ __forceinline__ Fp4Entry f4_entry(const Fp4Args& a, const int32_t* table, int base, int len, int lane) {
  const int key = base + KEYS * (lane % (kF4Keys / KEYS));
  Fp4Entry e;
  e.at = key < len ? key : ((len - 1) & ~15) + (key & 15);
  e.page = table[e.at >> a.page_shift];
  return e;
}

// A wave's place in a list of tiles that its workgroup's waves share out in turn: tile
// `tile` of request b, which has `len` keys; `left` tiles of the list from here on.
// PREFIX: one request, the prefix's part, whose keys begin at key0.
template <bool PREFIX>
struct Fp4Cursor {
  int b, tile, tiles, len, left, key0;
  const int32_t* table;
  __device__ __forceinline__ void forward(const Fp4Args& a, int n) {
    left -= n;
    if (left <= 0) return;
    tile += n;
    while (!PREFIX && tile >= tiles) {
      tile -= tiles;
      do {
        ++b;
        len = f4_len_at(a, b);
      } while (len == 0);
      tiles = f4_tiles(len);
      table = a.table + b * a.table_stride;
    }
  }
};

// The tiles from `at` on, for 16 RB rows of each request's `rows` from row0 on.
template <int DQ, int DV, int RB, bool PREFIX>
__device__ __forceinline__ void fp4_narrow(const Fp4Args& a, int kvh, Fp4Cursor<PREFIX> at, int row0, int rows, int64_t entry0,
                                           uint8_t* mem) {
  using W = Fp4Wave<DQ, DV, RB>;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.q_heads / a.kv_heads;
  uint8_t* mine = mem + wv * W::kRegion;
  auto entry_of = [&](const Fp4Cursor<PREFIX>& x) {
    // (the prefix's part begins at a whole tile of the prefix)
    return f4_entry<W::kEntryKeys>(a, x.table, x.key0 + x.tile * kF4Keys, x.key0 + x.len, lane);
  };
  W w;
  w.setup(lane);
  // The tile that is computed on, the one whose loads are under way by then, the one whose
  // entries are (past the end: those of the one before once more).
  Fp4Cursor<PREFIX> now = at;
  now.forward(a, wv);
  Fp4Cursor<PREFIX> next = now;
  next.forward(a, kF4Waves);
  Fp4Cursor<PREFIX> far = next;
  auto load_queries = [&](int b) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = min(row0 + 16 * rb + (lane & 15), rows - 1);
      const int rq = PREFIX ? row / G : b, hq = kvh * G + (PREFIX ? row % G : row);
      w.load_query(rb, a.q + rq * a.q_ts + hq * a.q_hs, lane);
    }
  };
  Fp4Entry entry = {0, 0};
  load_queries(at.b);
  if (now.left > 0) {
    const int slot = entry_of(now).slot(a);
    entry = entry_of(next);
    w.template load<!PREFIX>(a, kvh, slot, lane);
    far.forward(a, kF4Waves);
  }
  auto step = [&](auto more) {
    const int last = now.len - 1 - now.tile * kF4Keys;
    w.store(mine, lane, last);
    if constexpr (decltype(more)::value) {
      const int slot = entry.slot(a);
      entry = entry_of(far);
      w.template scores<true, !PREFIX>(a, kvh, slot, lane);
    } else {
      w.template scores<false, !PREFIX>(a, kvh, 0, lane);
    }
    if (last < kF4Keys - 1) w.mask(lane, last);
    w.weights();
    asm volatile("" ::: "memory");                                  // (a wave's own LDS accesses stay in order)
    w.values(mine, lane);
    asm volatile("" ::: "memory");
    now = next;
    next = far;
    far.forward(a, kF4Waves);
  };
  // the requests of the list one after the other
  for (int b = at.b, rest = at.left, tile = at.tile, tiles = at.tiles;;) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) w.init(rb, a);
    // (with and without a next tile apart: loads that may or may not have gone out would be
    // waited for with the ones before them)
    while (next.left > 0 && now.b == b) step(std::true_type());
    if (now.left > 0 && now.b == b) step(std::false_type());
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      w.leave(mine, rb, lane);
      __syncthreads();
      for (int f = threadIdx.x; f < 16 * (DV / 4); f += kF4Waves * 64) {
        const int r = f / (DV / 4), col = f % (DV / 4) * 4, row = row0 + 16 * rb + r;
        if (row >= rows) continue;
        float M, L;
        const f32x4 sum = join_waves<DV, kF4Waves, W::kRegion>(mem, r, col, &M, &L);
        const int64_t entry = PREFIX ? entry0 + (int64_t)(row / G) * a.q_heads + kvh * G + row % G
                                     : entry0 + (int64_t)b * a.plan.rows_s + row - row0;
        *(f32x4*)(a.part_o + entry * DV + col) = sum;
        if (col == 0) a.part_ml[entry] = float2{M, L};
      }
      __syncthreads();
    }
    // on to the next request with keys, if the list goes that far
    rest -= tiles - tile;
    if (PREFIX || rest <= 0) break;
    do ++b;
    while (f4_len_at(a, b) == 0);
    tiles = f4_tiles(f4_len_at(a, b));
    tile = 0;
    load_queries(b);
  }
}

// Prefix part `part`, 128 rows from row0, 32 per wave; tiles of 64 keys in two stages.
// A thread takes blocks of 16 values from memory to f16 rows in LDS, a tile ahead of the
// products, their loads another tile ahead; half a block goes out behind every other product of
// the scores, whose wave has no vector work of its own (96 requests behind 32768 keys of 192 + 128 165 ->
// 157 us; behind the values' products 165, and a block's addresses must be one register and
// constants, or registers spill).  All three of matrix cores, vector units and LDS reads (each
// wave reads all of a tile for its 32 rows) are busy 40 to 50% of the time.  PAGED: pages hold 64 rows or more, so a tile's
// blocks follow one another; otherwise those of 16 keys do (96 requests behind 32768 keys of 64
// / 4 heads of 192 + 128: 158 us, 171 in pages of 16).  Rows past the end are the page's own,
// or the last 16's; their values' scales count as 0.
template <int DQ, int DV, bool PAGED>
__device__ __forceinline__ void fp4_wide(const Fp4Args& a, int kvh, int part, int row0, uint8_t* mem) {
  using W = AttnWave<DQ, DV, kF4Keys / 32, AttnF16>;
  uint8_t* ks = mem;
  uint8_t* vs = mem + 2 * W::kKeyBytes;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int G = a.q_heads / a.kv_heads, rows = a.num_requests * G;
  const int wrow = row0 + wv * 32;                                  // this wave's first row
  const int row = min(wrow + (lane & 31), rows - 1);
  const int b = row / G, hq = kvh * G + row % G;
  const int key0 = part * a.plan.chunk_p, n_keys = (int)min((int64_t)a.plan.chunk_p, a.prefix_len - key0);
  const int n_tiles = f4_tiles(n_keys);
  const int mask = (1 << a.page_shift) - 1;
  // cache row of a tile's first key, or lane by lane of the first key of its 16 (past the end:
  // the last 16's)
  auto slot_of = [&](int t) {
    const int key = key0 + (PAGED ? min(t, n_tiles - 1) * kF4Keys : min(t * kF4Keys + (lane & ~15), (n_keys - 1) & ~15));
    const int e = a.prefix_table[key >> a.page_shift];
    return (min(max(e, 0), a.num_pages - 1) << a.page_shift) + (key & mask);
  };
  constexpr int KI = DQ / 64, VI = DV / 64, KB = DQ / 16, VB = DV / 16;   // blocks per thread; per row
  u32x2 kc[KI], vc[VI];
  uint32_t ksc[KI], vsc[VI];
  // Buffers from a uniform cache row on (64-bit base, the lanes' 32-bit offsets): of the tile,
  // or of the 16 keys that all lanes of a wave take blocks of (16 rows are 16, 8 or 12 x 16
  // blocks: whole waves).
  // This thread's blocks: of keys of 4 or 8 blocks, block kblk of rows krow, krow + kRows, ...; of
  // 12, blocks kblk, kblk + 4 and kblk + 8 of row krow; of values as of keys.  So their places
  // differ by constants (the swizzle repeats every 16 rows, and keeps chunks of 8 together).
  constexpr int kRows = KB == 12 ? 0 : 256 / KB, kBlocks = KB == 12 ? 4 : 0, vRows = 256 / VB;
  const int krow = threadIdx.x / (KB == 12 ? 4 : KB), kblk = threadIdx.x % (KB == 12 ? 4 : KB);
  const int vrow = threadIdx.x / VB, vblk = threadIdx.x % VB;
  // the first block's 16 keys (one group for a wave's lanes), rows within them or the tile
  const int kgroup = KB == 12 ? wv : 4 * wv / KB, vgroup = 4 * wv / VB;
  const int kin = (PAGED ? krow : krow - 16 * kgroup) * KB + kblk, vin = PAGED ? vrow : vrow - 16 * vgroup;
  const uint32_t kto = (uint32_t)(krow * (DQ * 2) + ((2 * kblk) ^ at_swz<DQ>(krow)) * 16);
  const uint32_t vto = (uint32_t)(vrow * (DV * 2) + ((2 * vblk) ^ at_swz<DV>(vrow)) * 16);
  const uint32_t vsin = ((uint32_t)vblk << a.page_shift) + vin;
  auto rows_at = [&](int slot, int group, uint64_t* head) {          // (head: of the page's values' scales)
    const uint32_t sl = (uint32_t)__builtin_amdgcn_readlane(slot, PAGED ? 0 : group * 16);
    *head = (uint64_t)(sl >> a.page_shift) * a.kv_heads + kvh;
    return (*head << a.page_shift) + (sl & mask);
  };
  auto load = [&](int slot, int i) {                                // block i of KI + VI
    uint64_t head;
    if (i < KI) {
      const uint64_t at = rows_at(slot, kgroup + i * (kRows / 16), &head);
      const int more = i * ((PAGED ? kRows * KB : 0) + kBlocks);
      kc[i] = bload64(make_rsrc(a.k + at * (DQ / 2), 0x7fffffffu), kin * 8, more * 8);
      ksc[i] = bload8(make_rsrc(a.ks + at * KB, 0x7fffffffu), kin, more);
    } else {
      i -= KI;
      const uint64_t at = rows_at(slot, vgroup + i * (vRows / 16), &head);
      const int more = PAGED ? i * vRows : 0;
      vc[i] = bload64(make_rsrc(a.v + at * (DV / 2), 0x7fffffffu), (vin * VB + vblk) * 8, more * VB * 8);
      vsc[i] = bload8(make_rsrc(a.vs + ((head * VB) << a.page_shift) + (at - (head << a.page_shift)), 0x7fffffffu), vsin, more);
    }
  };
  auto put = [&](int st, int valid, int j) {                        // half j of 2 (KI + VI); valid: keys that are there
    int i = j >> 1;
    const uint32_t x = (j & 1) * 16;
    if (i < KI) {
      const _Float16 s = scale_pair<false>(ksc[i])[0];
      *(f16x8*)(ks + (kto ^ x) + st * W::kKeyBytes + i * (kRows * DQ * 2 + kBlocks * 32)) = fp4x8_f16(kc[i][j & 1], s);
    } else {
      i -= KI;
      const _Float16 s = scale_pair<false>(vrow + i * vRows >= valid ? 0u : vsc[i])[0];
      *(f16x8*)(vs + (vto ^ x) + st * W::kValBytes + i * (vRows * DV * 2)) = fp4x8_f16(vc[i][j & 1], s);
    }
  };
  constexpr int kHalves = 2 * (KI + VI);
  int slot = slot_of(0);
#pragma unroll
  for (int i = 0; i < KI + VI; ++i) load(slot, i);
  slot = slot_of(1);
  W w;
  const float c = score_factor(a, w.init(a.q + b * a.q_ts + hq * a.q_hs, lane));
#pragma unroll
  for (int j = 0; j < kHalves; ++j) {
    put(0, n_keys, j);
    if (j & 1) load(slot, j >> 1);
  }
  slot = slot_of(2);
  auto step = [&](auto stage, int t) {
    constexpr int st = decltype(stage)::value;
    // tile t is in its stage; everyone is done with tile t - 1, whose stage is refilled (at the
    // end with the last tile once more, which nothing reads)
    at_wait_barrier<63>();
    take_turns<0>(t);
    const int valid = n_keys - (t + 1) * kF4Keys, far = slot_of(t + 3);
    auto refill = [&](int j) {
      put(st ^ 1, valid, j);
      if (j & 1) load(slot, j >> 1);
    };
    if (wrow >= rows) {
#pragma unroll
      for (int j = 0; j < kHalves; ++j) refill(j);
      slot = far;
      return;
    }
    w.scores(ks + st * W::kKeyBytes, [&](int i) {
#pragma unroll
      for (int j = 0; j < kHalves; ++j)
        if (i == j * W::kScoreOps / kHalves) refill(j);
    });
    slot = far;
    if (t == n_tiles - 1) w.mask(lane, n_keys - 1 - t * kF4Keys);
    w.weights(c);
    w.values(vs + st * W::kValBytes);
  };
  for (int t = 0; t < n_tiles; t += 2) {
    step(std::integral_constant<int, 0>(), t);
    if (t + 1 < n_tiles) step(std::integral_constant<int, 1>(), t + 1);
  }
  if (wrow + (lane & 31) < rows) {
    const int64_t entry = (int64_t)part * a.num_requests * a.q_heads + (int64_t)b * a.q_heads + hq;
    float* po = a.part_o + entry * DV + 4 * h;
#pragma unroll
    for (int x = 0; x < W::OB; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(f32x4*)(po + 32 * x + 8 * i) = f32x4{w.o[x][4 * i], w.o[x][4 * i + 1], w.o[x][4 * i + 2], w.o[x][4 * i + 3]};
    if (h == 0) a.part_ml[entry] = float2{w.m, w.l};
  }
}

// Workgroups that a CU holds at once.  Two keep as many reads under way as memory takes, and
// more lists of tiles begin and end more often; a third, for which 128-wide keys leave the
// registers, took 36.0 us for 34.5 (1 request of 131072 keys), 21.7 for 19.1 (of 16 / 2 heads) and the same
// for many requests.  64-wide keys need four to have as much under way (100 requests of up to 6000: two
// 44.9 us, four 39.6).
constexpr int fp4_small_per_cu(int k_dim, int waves) { return (k_dim == 64 ? 16 : 12) / waves; }
constexpr int fp4_per_cu(int k_dim, int rb, bool wide) { return k_dim == 64 && rb == 1 && !wide ? 4 : 2; }

template <int DQ, int DV, int RB, bool WIDE>
__global__ __launch_bounds__(kF4Waves * 64, fp4_per_cu(DQ, RB, WIDE)) void attn_decode_fp4_kernel(Fp4Args a) {
  constexpr int kNarrow = kF4Waves * Fp4Wave<DQ, DV, RB>::kRegion, kWide = WIDE ? 2 * kF4Keys * (DQ + DV) * 2 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t mem[kNarrow > kWide ? kNarrow : kWide];
  const Fp4Plan& p = a.plan;
  const int kvh = blockIdx.x % a.kv_heads, lane = threadIdx.x & 63;
  int item = blockIdx.x / (uint32_t)a.kv_heads;
  if (item < p.parts_p * p.blocks_p) {
    // row blocks of one part side by side: they share the part's keys in L2
    const int part = item / p.blocks_p, block = item % p.blocks_p;
    if (WIDE && a.page_shift >= 6) return fp4_wide<DQ, DV, true>(a, kvh, part, block * 128, mem);
    if (WIDE) return fp4_wide<DQ, DV, false>(a, kvh, part, block * 128, mem);
    Fp4Cursor<true> at;
    at.b = at.tile = 0;
    at.key0 = part * p.chunk_p;
    at.len = (int)min((int64_t)p.chunk_p, a.prefix_len - at.key0);
    at.tiles = at.left = f4_tiles(at.len);
    at.table = a.prefix_table;
    return fp4_narrow<DQ, DV, RB, true>(a, kvh, at, block * 16 * RB, a.num_requests * (a.q_heads / a.kv_heads),
                                        (int64_t)part * a.num_requests * a.q_heads, mem);
  }
  item -= p.parts_p * p.blocks_p;
  const int run = item / p.blocks_s, block = item % p.blocks_s;
  // Tiles of all requests, 64 requests at a time; the first workgroup writes down where each
  // request's begin.  Then the request that tile `begin` belongs to: the last whose tiles
  // begin at or before it.
  const int B = a.num_requests;
  const bool writes = blockIdx.x == (uint32_t)(p.parts_p * p.blocks_p * a.kv_heads) && threadIdx.x < 64;
  auto len_of = [&](int b0) { return b0 + lane < B ? f4_clamp_len(a, a.lens[b0 + lane]) : 0; };
  int len = 0, n = 0, sum = 0, total = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    len = len_of(b0);
    n = f4_tiles(len);
    sum = wave_scan(n);
    if (writes && b0 + lane < B) a.first[b0 + lane] = total + sum - n;
    total += __builtin_amdgcn_readlane(sum, 63);
  }
  if (writes && lane == 0) a.first[B] = total;
  const int each = (total + p.runs - 1) / p.runs, begin = run * each, end = min(begin + each, total);
  if (begin >= end) return;
  Fp4Cursor<false> at;
  at.b = at.tile = at.len = 0;
  for (int b0 = 0, sofar = 0; b0 < B; b0 += 64) {
    if (B > 64) {                                                   // (else as above)
      len = len_of(b0);
      n = f4_tiles(len);
      sum = wave_scan(n);
    }
    const uint64_t le = __ballot(sofar + sum - n <= begin && n > 0);
    if (le) {
      const int l = 63 - __builtin_clzll(le);
      at.b = b0 + l;
      at.tile = begin - sofar - __builtin_amdgcn_readlane(sum - n, l);
      at.len = __builtin_amdgcn_readlane(len, l);
    }
    sofar += __builtin_amdgcn_readlane(sum, 63);
    if (sofar > begin) break;
  }
  at.tiles = f4_tiles(at.len);
  at.left = end - begin;
  at.key0 = 0;
  at.table = a.table + at.b * a.table_stride;
  const int row0 = block * p.rows_s, rows = min(row0 + p.rows_s, a.q_heads / a.kv_heads);
  const int64_t entry0 = a.own + ((int64_t)(kvh * p.blocks_s + block) * (p.runs + B) + run) * p.rows_s;
  fp4_narrow<DQ, DV, RB, false>(a, kvh, at, row0, rows, entry0, mem);
}

// Few keys: a workgroup per request and key head answers alone, without parts and a
// second launch.  Its WAVES waves take every WAVES-th tile, the prefix's first.  At most 16
// heads of a key head.
template <int DQ, int DV, int WAVES>
__global__ __launch_bounds__(WAVES * 64, fp4_small_per_cu(DQ, WAVES)) void attn_decode_fp4_small_kernel(Fp4Args a) {
  using W = Fp4Wave<DQ, DV, 1>;
  __shared__ __attribute__((aligned(16))) uint8_t mem[WAVES * W::kRegion];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kvh = blockIdx.x % (uint32_t)a.kv_heads, b = blockIdx.x / (uint32_t)a.kv_heads, G = a.q_heads / a.kv_heads;
  const int len = f4_len_at(a, b), prefix = (int)a.prefix_len;
  const int tiles_p = f4_tiles(prefix), n_tiles = tiles_p + f4_tiles(len);
  const int32_t* own = a.table + b * a.table_stride;
  uint8_t* mine = mem + wv * W::kRegion;
  auto entry_of = [&](int t) {
    const bool front = t < tiles_p;
    return f4_entry<W::kEntryKeys>(a, front ? a.prefix_table : own, (front ? t : t - tiles_p) * kF4Keys, front ? prefix : len, lane);
  };
  int t = wv;
  W w;
  w.setup(lane);
  Fp4Entry entry = {0, 0};
  w.load_query(0, a.q + b * a.q_ts + (int64_t)(kvh * G + min(lane & 15, G - 1)) * a.q_hs, lane);
  if (t < n_tiles) {
    const int slot = entry_of(t).slot(a);
    entry = entry_of(min(t + WAVES, n_tiles - 1));
    w.template load<false>(a, kvh, slot, lane);
  }
  w.init(0, a);
  auto step = [&](auto more) {
    const int last = t < tiles_p ? prefix - 1 - t * kF4Keys : len - 1 - (t - tiles_p) * kF4Keys;
    w.store(mine, lane, last);
    if constexpr (decltype(more)::value) {
      const int slot = entry.slot(a);
      entry = entry_of(min(t + 2 * WAVES, n_tiles - 1));
      w.template scores<true, false>(a, kvh, slot, lane);
    } else {
      w.template scores<false, false>(a, kvh, 0, lane);
    }
    if (last < kF4Keys - 1) w.mask(lane, last);
    w.weights();
    asm volatile("" ::: "memory");                                  // (a wave's own LDS accesses stay in order)
    w.values(mine, lane);
    asm volatile("" ::: "memory");
  };
  for (; t + WAVES < n_tiles; t += WAVES) step(std::true_type());
  if (t < n_tiles) step(std::false_type());
  w.leave(mine, 0, lane);
  __syncthreads();
  for (int f = threadIdx.x; f < G * (DV / 4); f += WAVES * 64) {
    const int row = f / (DV / 4), col = f % (DV / 4) * 4;
    float M, L;
    const f32x4 sum = join_waves<DV, WAVES, W::kRegion>(mem, row, col, &M, &L);
    const float inv = L == 0.0f ? 0.0f : a.v_scale / L;
    const int hq = kvh * G + row;
    *(u32x2*)(a.out + b * a.o_ts + hq * a.o_hs + col) =
        u32x2{cvt_bf16x2(sum[0] * inv, sum[1] * inv), cvt_bf16x2(sum[2] * inv, sum[3] * inv)};
    if (a.lse && col == 0) a.lse[(int64_t)b * a.q_heads + hq] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
  }
}

// Waves of a workgroup that answers a request's heads of one key head alone; 0: parts are
// sooner.  Such a workgroup has no parts to write and no second launch, but its time grows
// with its tiles, and it reads the prefix for its request only, with the matrix cores' 16
// rows as full as the heads make them.  Measured, us, alone / in parts (8 key heads of 128 +
// 128, 4 query heads each): 1 request of 1024 keys 8.5 / 9.0, of 2048 12.7 / 9.1; 8 of 2048
// 13.0 / 13.3; 16 of 2048 13.5 / 16.0, of 4096 22.1 / 20.1; 256 of 1024 40 / 55, of 4096 128 /
// 120; 64 behind 1024 with up to 1024 of their own 23 / 27, 256 66 / 59.  (4 key heads of 192
// + 128, 16 query heads each: 64 of 4096 28 / 35, 256 behind 2048 with 64 51 / 64; 8 of 64 + 64,
// one each: 256 behind 1024 with 64 29 / 21.)  Within 5% of the better at 140 of 150 sizes.
// Where they all run at once, 8 waves divide a request's tiles better (1 of 1024 8.5 us, 9.6
// with 4); else three workgroups of 4 on a CU leave less time idle than one of 8 (256 of 1024
// 40 us, 59 with 8).
static int fp4_small_waves(int64_t B, int64_t G, int64_t kv_heads, int64_t prefix_len, int64_t max_len, int64_t k_dim) {
  const int64_t tiles_p = (prefix_len + 63) / 64, tiles = tiles_p + (max_len + 63) / 64, items = B * kv_heads;
  if (G > 16 || tiles > std::min<int64_t>(64, 16 + items / 4) || tiles_p * items > 8192 + 2048 * G) return 0;
  return items <= 256 * fp4_small_per_cu(k_dim, 8) ? 8 : 4;
}

static Fp4Plan fp4_plan(int64_t B, const moe_attn_params& a, int64_t prefix_len, int64_t max_len) {
  const int q_heads = a.q_heads, kv_heads = a.kv_heads, dims = a.k_dim + a.v_dim;
  Fp4Plan p = {};
  const int64_t G = q_heads / kv_heads, rows = B * G;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  p.small = fp4_small_waves(B, G, kv_heads, prefix_len, max_len, a.k_dim);
  if (p.small) return p;
  // Wide workgroups meet a tile with 128 rows and a quarter of the conversions, but each needs
  // several tiles to fill its stages, and leaves the own keys fewer places the longer the
  // prefix is to them; long own keys want the places that narrow ones with their more parts
  // would take.  Measured, us, wide / narrow (8 key heads of 128 + 128): 128 rows behind 8192
  // with 16 own keys 30 / 26, with 1024 32 / 32; 64 rows behind 32768 with 1024 36 / 33,
  // behind 2048 17 / 18.5; 768 rows behind 8192 with 16 58 / 64, behind 32768 137 / 194; 16 rows
  // behind 32768 27 / 19.  Within 5% of the better at 546 of 605 sizes, 25% or more behind it at
  // 15, with few own keys: 192 rows behind 32768 with 300 55 / 79 (narrow taken), 256 of one query
  // head behind 8192 with 16 38 / 58 (narrow), 768 of 4 key heads of 192 + 128 behind 32768 with 16
  // 129 / 100 (wide).
  p.wide = prefix_len > 0 && (rows >= 384 || (rows >= 32 && max_len * 32768 >= G * prefix_len * dims));
  p.rb = G > 16 || (prefix_len > 0 && !p.wide && rows > 16) ? 2 : 1;
  p.blocks_p = (int32_t)up(rows, p.wide ? 128 : 16 * p.rb);
  p.blocks_s = (int32_t)up(G, 16 * p.rb);
  p.rows_s = (int32_t)std::min<int64_t>(G, 16 * p.rb);
  // as the bf16 form's plan: units of work per 64 keys, the own lengths unknown (one at the
  // bound, the others at half).  5 for a wide tile to 3 for a narrow one: over 24 sizes 2%
  // sooner on average than 6, 1% than 4, 4% than 8.
  const int64_t slots = 256 * fp4_per_cu(a.k_dim, p.rb, p.wide);
  const int64_t tiles_p = up(prefix_len, 64), tiles_s = max_len == 0 ? 0 : up((B + 1) * up(max_len, 64), 2) + B;
  const int64_t cost_p = p.wide ? 5 : 3, cost_s = 3;
  const int64_t per_part = kv_heads * p.blocks_p, per_run = kv_heads * p.blocks_s;
  const int64_t work_p = per_part * tiles_p * cost_p, work_s = per_run * tiles_s * cost_s;
  int64_t parts = 0;
  if (tiles_p > 0) {
    const int64_t most = up(tiles_p, p.wide ? 2 : 4), room = max_len == 0 ? slots : slots - per_run;
    parts = std::max<int64_t>(1, std::min(most, slots * work_p / (work_p + work_s) / per_part));
    auto time = [&](int64_t n) { return std::max(up(tiles_p, n) * cost_p, work_s / std::max<int64_t>(1, slots - n * per_part)); };
    if (parts < most && (parts + 1) * per_part <= room && time(parts + 1) < time(parts)) ++parts;
  }
  p.chunk_p = tiles_p == 0 ? 0 : (int32_t)(up(tiles_p, parts) * 64);
  p.parts_p = tiles_p == 0 ? 0 : (int32_t)up(prefix_len, p.chunk_p);
  int64_t places = slots - p.parts_p * per_part;
  if (p.parts_p <= 1 && max_len > 0) {
    const int64_t prefix = p.parts_p == 0 ? 0 : up(per_part, slots) * (p.chunk_p / 64) * cost_p;
    if (places < per_run || prefix + work_s / slots < work_s / places) places = slots;
  }
  const int64_t left = places / per_run;
  // (a run that holds several short requests takes them one after the other, so there are
  // as many as keep each request's 4 tiles at a time apart: 32 requests of 64 keys 16.5 ->
  // 9.2 us in parts, 8 behind 1024 + 16 20.5 -> 14.2)
  p.runs = max_len == 0 ? 0 : (int32_t)std::max<int64_t>(1, std::min(left, B * up(max_len, kF4Keys * kF4Waves)));
  return p;
}

static int64_t fp4_prefix_entries(const Fp4Plan& p, int64_t B, int q_heads) { return (int64_t)p.parts_p * B * q_heads; }
static int64_t fp4_entries(const Fp4Plan& p, int64_t B, int q_heads, int kv_heads) {
  return fp4_prefix_entries(p, B, q_heads) + (p.runs > 0 ? (int64_t)kv_heads * p.blocks_s * (p.runs + B) * p.rows_s : 0);
}

size_t attn_decode_fp4_ws_bytes(int64_t B, const moe_attn_params& p, int64_t prefix_len, int64_t max_len) {
  const Fp4Plan plan = fp4_plan(B, p, prefix_len, max_len);
  const int64_t entries = fp4_entries(plan, B, p.q_heads, p.kv_heads);
  return entries == 0 ? 0 : (size_t)entries * ((size_t)p.v_dim * 4 + 8) + ((size_t)B + 1) * 4;
}

static int64_t fp4_grid(const Fp4Plan& p, int kv_heads) {
  return ((int64_t)p.parts_p * p.blocks_p + (int64_t)p.runs * p.blocks_s) * kv_heads;
}

// Threads of the larger of both launches.
int64_t attn_decode_fp4_threads(int64_t B, const moe_attn_params& p, int64_t prefix_len, int64_t max_len) {
  const Fp4Plan plan = fp4_plan(B, p, prefix_len, max_len);
  if (plan.small) return B * p.kv_heads * plan.small * 64;
  return std::max(fp4_grid(plan, p.kv_heads) * kF4Waves * 64,
                  (B * p.q_heads + 3) * 64 * join_waves(plan.parts_p, 1, plan.runs, (int)B));
}

template <int DQ, int DV>
static void launch_fp4(const Fp4Args& a, hipStream_t stream) {
  if (a.plan.small) {
    const dim3 grid((uint32_t)(a.num_requests * a.kv_heads)), threads(a.plan.small * 64);
    if (a.plan.small == 8) hipLaunchKernelGGL((attn_decode_fp4_small_kernel<DQ, DV, 8>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_fp4_small_kernel<DQ, DV, 4>), grid, threads, 0, stream, a);
    return;
  }
  const uint32_t grid = (uint32_t)fp4_grid(a.plan, a.kv_heads);
  const dim3 threads(kF4Waves * 64);
  if (grid > 0) {
    if (a.plan.rb == 1 && !a.plan.wide) hipLaunchKernelGGL((attn_decode_fp4_kernel<DQ, DV, 1, false>), dim3(grid), threads, 0, stream, a);
    else if (a.plan.rb == 1) hipLaunchKernelGGL((attn_decode_fp4_kernel<DQ, DV, 1, true>), dim3(grid), threads, 0, stream, a);
    else if (!a.plan.wide) hipLaunchKernelGGL((attn_decode_fp4_kernel<DQ, DV, 2, false>), dim3(grid), threads, 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_fp4_kernel<DQ, DV, 2, true>), dim3(grid), threads, 0, stream, a);
  }
  JoinArgs j;
  j.out = a.out;
  j.o_ts = a.o_ts;
  j.o_hs = a.o_hs;
  j.lse = a.lse;
  j.part_o = a.part_o;
  j.part_ml = a.part_ml;
  j.first = a.first;
  j.own = a.own;
  j.num_requests = a.num_requests;
  j.q_heads = a.q_heads;
  j.kv_heads = a.kv_heads;
  j.prefix_parts = a.plan.parts_p;
  j.run_parts = 1;
  j.runs = a.plan.runs;
  j.blocks_s = a.plan.blocks_s;
  j.rows_s = a.plan.rows_s;
  j.v_scale = a.v_scale;
  launch_join<DV>(j, stream);
}

moe_status launch_attn_decode_fp4(const moe_heads& q, const moe_kv_cache_fp4& cache, const int32_t* table,
                                  int64_t table_stride, const int32_t* lens, int64_t B, int64_t max_len,
                                  const int32_t* prefix_table, int64_t prefix_len, const moe_attn_params& p,
                                  const moe_heads& out, float* lse, void* ws, hipStream_t stream) {
  Fp4Args a;
  a.q = (const uint16_t*)q.data;
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.out = (uint16_t*)out.data;
  a.o_ts = out.token_stride;
  a.o_hs = out.head_stride;
  a.k = (const uint8_t*)cache.k;
  a.ks = (const uint8_t*)cache.k_scale;
  a.v = (const uint8_t*)cache.v;
  a.vs = (const uint8_t*)cache.v_scale;
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
  a.c = std::frexp(p.scale, &a.c_exp) * kLog2e;
  a.c_exp += std::ilogb(cache.k_global);
  a.v_scale = cache.v_global;
  a.plan = fp4_plan(B, p, prefix_len, max_len);
  const int64_t entries = fp4_entries(a.plan, B, p.q_heads, p.kv_heads);
  a.part_o = (float*)ws;                            // (the sums first: they need 16-byte alignment)
  a.part_ml = (float2*)(a.part_o + entries * p.v_dim);
  a.first = (int32_t*)(a.part_ml + entries);
  a.own = fp4_prefix_entries(a.plan, B, p.q_heads);
  if (p.k_dim == 64) launch_fp4<64, 64>(a, stream);
  else if (p.k_dim == 128) launch_fp4<128, 128>(a, stream);
  else launch_fp4<192, 128>(a, stream);
  return launch_status("moe_attn_decode_fp4");
}

}  // namespace moe
