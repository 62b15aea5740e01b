// One wave's part of attention on gfx950's bf16 matrix cores, shared by the
// prompt and the decode kernel: 32 query rows against a tile of keys in LDS.
//
// The scores are formed transposed, S^T = K Q^T (32x32x16 MFMA, K rows as the
// first operand), so lane l holds the scores of ONE query row, l % 32, against
// half of the tile's keys; lane l ^ 32 holds the other half.  Row maximum and
// sum are then in-lane except for one exchange between the lane's halves, and
// the running scale factors need no broadcast.  The weights P^T come out of the
// score accumulator in an order that is already a second MFMA operand if the
// contraction index (the key) is enumerated as the accumulator holds it: for
// keys 16 s .. 16 s + 15, lane half h and element j stand for key
// 16 s + 8 (j / 4) + 4 h + j % 4.  The same enumeration of V's rows is what two
// transposing LDS reads (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16
// columns, each receives one column's 4 values) deliver, so O^T = V^T P^T needs
// no exchange of weights between lanes at all.
//
// Online softmax in base 2: m is the running maximum of the scores times
// c = scale log2(e), p = 2^(s c - m); l (float) sums the unrounded weights,
// O (float) accumulates the weights rounded to bf16, the matrix cores' operand
// (relative error 2^-9 of each weight, of random sign: as much as the rounding
// of the output itself).
//
// Rates: a wave's tile of 64 keys x 128 takes 32 MFMAs of 32 cycles (16 for the
// scores, 16 for the values) and about 230 vector instructions; the two to four
// waves per SIMD (by head size) overlap them.  The LDS reads have no bank conflicts in either product.
//
// Layouts measured on the chip: 32x32x16 operands hold row l % 32, k = 8 (l / 32)
// + j, j < 8; the accumulator holds column l % 32, row 8 (i / 4) + 4 (l / 32) +
// i % 4, i < 16.
#pragma once
#include <type_traits>

#include "common.h"

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

namespace moe {

typedef __attribute__((address_space(3))) void at_lds_void;
typedef __attribute__((address_space(3))) s16x4 at_lds_s16x4;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The matrix cores' operand type.  bf16: keys, values and weights as they come.  f16
// (caches held in 4 bits): a code times its block's scale is exact in it (6 significant
// bits, 2^-10 to 2688), and a weight keeps 11 bits.  Its weights are lifted by 2^kLift, so
// that those down to 2^-31 of a row's largest are not lost below its range (2^-24) while the
// largest, 2^(kLift + kSlack) (see weights()) and twice that where a maximum less kLift is
// rounded, by 1 at most, stay under 65504.
struct AttnBf16 {
  typedef bf16x8 v8;
  static constexpr float kLift = 0.0f, kSlack = 8.0f;
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) { return mfma32(a, b, c); }
  static __device__ __forceinline__ uint32_t pair(float a, float b) { return cvt_bf16x2(a, b); }
};
struct AttnF16 {
  typedef f16x8 v8;
  static constexpr float kLift = 7.0f, kSlack = 7.0f;
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
  }
};

// Whether a tile's maximum leaves a row's kept one behind.  Their difference, not the sum m +
// kSlack: of scores past 2^24 that is rounded too, up to where a weight is 2^16, which f16 does
// not hold.  (bf16 holds any weight.)
template <class T>
__device__ __forceinline__ bool has_grown(float mx, float m) {
  return T::kLift == 0.0f ? mx > m + T::kSlack : mx - m > T::kSlack;
}

// a * b rounded, whatever comes after it
__device__ __forceinline__ float mul_rounded(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}
// Scores times c, less base, are formed in one rounding; base itself, the maximum's, was
// rounded before.  Of scores over 2^20 (base 2) that difference would pass 2^-4 and lift
// f16 weights out of their range: there s c is rounded like the maximum's.  The row's
// own choice: (c, 1) or (1, c), to multiply the scores with before and in the exponent.
__device__ __forceinline__ float2 split_scale(float base, float c) {
  return fabsf(base) > 1048576.0f ? float2{c, 1.0f} : float2{1.0f, c};
}

// 8 query values as f16, times 2^-e.  e takes a row's largest magnitude to [2^14, 2^15): a
// value of bf16's 8 bits is then exact down to 2^-28 of the largest and off by 2^-39 of it
// below.  The row's scores are multiplied by 2^e (AttnWave and the like take that with
// their scale).
__device__ __forceinline__ f16x8 query_f16(u32x4 w, int e) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = AttnF16::pair(ldexpf(bf16_lo(w[i]), -e), ldexpf(bf16_hi(w[i]), -e));
  return __builtin_bit_cast(f16x8, r);
}
__device__ __forceinline__ float query_most(u32x4 w, float most) {
#pragma unroll
  for (int i = 0; i < 4; ++i) most = fmaxf(most, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
  return most;
}
__device__ __forceinline__ int query_exponent(float most) {
  return most == 0.0f ? 0 : (int)(__float_as_uint(most) >> 23) - 127 - 14;
}

// max / sum over the two lanes (l, l ^ 32) that share a query row
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Rows of D bf16 in LDS: 16-byte chunk c of row r sits at chunk c ^ at_swz(r).
// A score operand read takes chunk c of 32 rows, a V read 4 chunks of 4
// consecutive rows; the maps spread both over all banks (rows of 128 bytes: two
// to a 256-byte bank sweep; of 384 bytes: alternating halves).
template <int D>
__device__ __forceinline__ int at_swz(int r) {
  if (D == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
  if (D == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  return (r >> 1) & 7;                                              // D == 192 (keys only)
}

// Direct load of 16 bytes per lane into LDS: lane i's bytes land at lds + 16 i.
// As one asm block because the compiler makes every later LDS read that it
// cannot tell apart from the target wait for all loads in flight; here the
// kernel's own waits order them (at_wait_barrier).  No register but m0 is written
// (the compiler sets m0 itself right before a use of its own); the
// wait state between m0 and its use is in the block.
typedef uint32_t at_rsrc __attribute__((ext_vector_type(4)));
__device__ __forceinline__ at_rsrc at_make_rsrc(const void* base) {
  const uint64_t b = (uint64_t)base;
  return at_rsrc{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
}
// (off per lane, uniform on top of it)
__device__ __forceinline__ void at_load_lds(uint32_t lds, at_rsrc r, uint32_t off, uint32_t uniform) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(off), "s"(r), "s"(uniform) : "memory");
}
// The same from a 64-bit address per lane.  ONCE: data that nothing reads again
// (non-temporal cache policy).
template <bool ONCE>
__device__ __forceinline__ void at_load_lds(uint32_t lds, const void* from) {
  if (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" :: "s"(lds), "v"(from) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(from) : "memory");
}
// 4 bytes per lane: lane i's land at lds + 4 i
__device__ __forceinline__ void at_load_lds4(uint32_t lds, const void* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" :: "s"(lds), "v"(from) : "memory");
}
__device__ __forceinline__ uint32_t at_lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// At most N of this wave's direct loads are still in flight.
template <int N>
__device__ __forceinline__ void at_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// Every LDS read of this wave has arrived and at most N of its direct loads are
// still in flight; then the workgroup's barrier.  Nothing moves across.
template <int N>
__device__ __forceinline__ void at_wait_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// NB blocks of 32 keys per tile; DQ-wide keys, DV-wide values
template <int DQ, int DV, int NB, class T = AttnBf16>
struct AttnWave {
  typedef typename T::v8 v8;
  static constexpr int KQ = DQ / 16, OB = DV / 32;
  static constexpr int kKeyBytes = NB * 32 * DQ * 2, kValBytes = NB * 32 * DV * 2;
  v8 q[KQ];
  f32x16 o[OB];
  f32x16 s[NB];
  v8 p[2 * NB];
  float m, l;
  // This lane's byte offsets within a tile: of its first operand chunk of key row
  // l % 32, and of its 8 bytes of the transposing reads of value block 0, lower and
  // upper 8 keys.  The others differ by constants, xored in within the span of the
  // swizzle (KA steps of the keys) and added beyond it.
  static constexpr int KA = DQ == 192 ? 4 : KQ;
  uint32_t k0, v0[2];

  // q: this lane's query row (16-byte aligned).  f16: returns the exponent that its scores lack.
  __device__ __forceinline__ int init(const uint16_t* row, int lane) {
    const int h = lane >> 5, r = lane & 31, g = lane >> 4, i16 = lane & 15;
    int e = 0;
    if constexpr (std::is_same<T, AttnBf16>::value) {
#pragma unroll
      for (int i = 0; i < KQ; ++i) q[i] = __builtin_bit_cast(bf16x8, *(const u32x4*)(row + 16 * i + 8 * h));
    } else {
      u32x4 x[KQ];
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < KQ; ++i) x[i] = *(const u32x4*)(row + 16 * i + 8 * h);
#pragma unroll
      for (int i = 0; i < KQ; ++i) most = query_most(x[i], most);
      e = query_exponent(half_max(most));
#pragma unroll
      for (int i = 0; i < KQ; ++i) q[i] = query_f16(x[i], e);
    }
    k0 = (uint32_t)(r * (DQ * 2) + (h ^ at_swz<DQ>(r)) * 16);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const int row16 = 8 * jj + 4 * h + (i16 >> 2);                // at_swz repeats every 16 rows
      const int chunk = (2 * (g & 1) + ((i16 & 3) >> 1)) ^ at_swz<DV>(row16);
      v0[jj] = (uint32_t)(row16 * (DV * 2) + chunk * 16 + 8 * (i16 & 1));
    }
#pragma unroll
    for (int b = 0; b < OB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;
    m = neg_inf();
    l = 0.0f;
    // The loads are waited for here, not by the first use in the key loop (whose
    // wait would take the direct loads in flight with it, tile after tile); all
    // the rest is done while they are under way.
    asm volatile("" : "+v"(k0), "+v"(v0[0]), "+v"(v0[1]));
#pragma unroll
    for (int i = 0; i < KQ; ++i) asm volatile("" : "+v"(q[i]));
    return e;
  }

  // operand of keys 32 b .. 32 b + 31, columns 16 k .. 16 k + 15
  __device__ __forceinline__ v8 read_k(const uint8_t* ks, int b, int k) const {
    return *(const v8*)(ks + (k0 ^ ((k % KA) * 32)) + (32 * b * (DQ * 2) + (k / KA) * (KA * 32)));
  }
  // operand of value columns 32 b .. 32 b + 31, keys 16 st .. 16 st + 15
  __device__ __forceinline__ v8 read_v(const uint8_t* vs, int st, int b) const {
    s16x4 part[2];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
      part[jj] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at_lds_s16x4*)(vs + (v0[jj] ^ (b * 64)) + 16 * st * (DV * 2)));
    return __builtin_bit_cast(v8, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // V's infinities and NaN as zeros
  __device__ __forceinline__ static bf16x8 finite_only(bf16x8 v) {
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu;
    }
    return __builtin_bit_cast(bf16x8, w);
  }

  // The matrix products take their LDS operands through a queue kAhead deep: the
  // read of operand i + kAhead goes out right after MFMA i, so the LDS latency
  // passes behind kAhead MFMAs of 32 cycles each.  (Left to itself the compiler
  // reads one step ahead and waits for it in each.)
  static constexpr int kAhead = 2;                                  // 3, 4 and 6 measured the same
  static constexpr int kScoreOps = KQ * NB, kValueOps = 2 * NB * OB;
  __device__ __forceinline__ v8 operand(const uint8_t* ks, const uint8_t* vs, int i) const {
    if (i < kScoreOps) return read_k(ks, i % NB, i / NB);
    i -= kScoreOps;
    return read_v(vs, i / OB, i % OB);
  }
  // operands FIRST .. LAST - 1: scores (s must be zero before the first), then values.
  // between(i): work of another kind that is to go out behind MFMA i.
  template <int FIRST, int LAST, class Between>
  __device__ __forceinline__ void products(const uint8_t* ks, const uint8_t* vs, Between between) {
    v8 f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = operand(ks, vs, FIRST + i);
#pragma unroll
    for (int i = FIRST; i < LAST; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      v8& x = f[(i - FIRST) % kAhead];
      if (i < kScoreOps) {
        s[i % NB] = T::mfma(x, q[i / NB], s[i % NB]);
      } else {
        const int j = i - kScoreOps;
        o[j % OB] = T::mfma(x, p[j / OB], o[j % OB]);
      }
      if (i + kAhead < LAST) x = operand(ks, vs, i + kAhead);
      between(i - FIRST);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  struct Nothing {
    __device__ __forceinline__ void operator()(int) const {}
  };
  __device__ __forceinline__ void clear_scores() {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
  }
  // s = the tile's raw scores
  template <class Between = Nothing>
  __device__ __forceinline__ void scores(const uint8_t* ks, Between between = Between()) {
    clear_scores();
    products<0, kScoreOps>(ks, nullptr, between);
  }
  // o += the tile's values times their weights
  template <class Between = Nothing>
  __device__ __forceinline__ void values(const uint8_t* vs, Between between = Between()) {
    products<kScoreOps, kScoreOps + kValueOps>(nullptr, vs, between);
  }
  // this lane's row sees keys 0 .. last of the tile (last may be negative or past the end)
  __device__ __forceinline__ void mask(int lane, int last) {
    const int seen = last - 4 * (lane >> 5);                        // the other part of a key's number is a constant
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + 8 * (i / 4) + (i & 3) <= seen ? s[b][i] : neg_inf();
  }

  // p = the tile's weights.  A row's m is raised, and its l and o scaled, only
  // when its maximum has grown by more than kSlack powers of two: until then
  // weights up to 2^kSlack simply stand (float and bf16 keep their relative
  // precision), and a wave none of whose rows has grown so much skips the
  // multiplications.  The decision is the row's own, so its result does not
  // depend on the rows beside it.
  __device__ __forceinline__ void weights(float c) {
    float mx = neg_inf();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = T::kLift == 0.0f ? half_max(mx) * c : mul_rounded(half_max(mx), c) - T::kLift;
    const bool grown = has_grown<T>(mx, m);
    if (__any(grown)) {
      const float alpha = grown ? __builtin_amdgcn_exp2f(m - mx) : 1.0f;
      m = grown ? mx : m;
      l *= alpha;
#pragma unroll
      for (int b = 0; b < OB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= alpha;
    }
    // a row that has seen no key (or only scores of -inf) keeps m = -inf; its
    // weights are 2^-inf = 0
    const float base = m == neg_inf() ? 0.0f : m;
    if constexpr (T::kLift != 0.0f) {
      const float2 f = split_scale(base, c);
      if (__any(f.y == 1.0f)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = mul_rounded(s[b][i], f.x);
      }
      c = f.y;
    }
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] = __builtin_amdgcn_exp2f(fmaf(s[b][i + j], c, -base));
          sum += w[j];
        }
        p[2 * b + i / 8] = __builtin_bit_cast(
            v8, u32x4{T::pair(w[0], w[1]), T::pair(w[2], w[3]), T::pair(w[4], w[5]), T::pair(w[6], w[7])});
      }
    l += half_sum(sum);
  }

  // values() of a tile with masked places and values that are not all finite.  A
  // weight of 0 times an infinite or NaN value is NaN, so a value that is masked
  // for a row would reach it.  So the product runs on the finite values, and
  // which rows see a +infinity, a -infinity or a NaN in which column is counted
  // by products of 0s and 1s (a positive weight leaves such a value what it is).
  // Few registers and little code rather than speed.
  __device__ __forceinline__ void values_careful(const uint8_t* vs, int lane, int last) {
#pragma unroll
    for (int st = 0; st < 2 * NB; ++st)
#pragma unroll
      for (int b = 0; b < OB; ++b) {
        o[b] = mfma32(finite_only(read_v(vs, st, b)), p[st], o[b]);
        __builtin_amdgcn_sched_barrier(0);
      }
    const int seen = last - 4 * (lane >> 5);
#pragma unroll
    for (int st = 0; st < 2 * NB; ++st) {
      u32x4 w;                                                      // 1.0 where the row sees the key
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 16 * st + 8 * (j / 2) + 2 * (j & 1);
        w[j] = (key <= seen ? 0x3F80u : 0u) | (key + 1 <= seen ? 0x3F800000u : 0u);
      }
      p[st] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {                          // +infinity, -infinity, NaN
      // the kind's bit patterns: (x & care) - first < count
      const uint32_t care = kind == 2 ? 0x7FFFu : 0xFFFFu, count = kind == 2 ? 0x7Fu : 1u;
      const uint32_t first = kind == 0 ? 0x7F80u : (kind == 1 ? 0xFF80u : 0x7F81u);
      const float value = kind == 0 ? -neg_inf() : (kind == 1 ? neg_inf() : __builtin_nanf(""));
#pragma unroll
      for (int b = 0; b < OB; ++b) {
        f32x16 z;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
#pragma unroll
        for (int st = 0; st < 2 * NB; ++st) {
          u32x4 w = __builtin_bit_cast(u32x4, read_v(vs, st, b));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = ((w[j] & care) - first < count ? 0x3F80u : 0u) | (((w[j] >> 16) & care) - first < count ? 0x3F800000u : 0u);
          z = mfma32(__builtin_bit_cast(bf16x8, w), p[st], z);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] += z[i] > 0.0f ? value : 0.0f;
      }
    }
  }
};

// The same for few query rows: RB blocks of 16 rows against 32 keys, on 16x16x32
// MFMAs.  Lane l holds row l % 16 of each block and, g = l / 16, the scores of
// keys 4 g + i and 16 + 4 g + i (i < 4); in that order they are the second
// product's operand, and V's rows 4 g .. 4 g + 3 and 16 + 4 g .. come by one
// transposing read each.  Half the matrix work and half the softmax of the 32-row
// form where at most 16 rows are real.
__device__ __forceinline__ float quarter_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <int DQ, int DV, int RB>
struct AttnWave16 {
  static constexpr int KQ = DQ / 32, OB = DV / 16, KA = DQ == 192 ? 2 : KQ;
  static constexpr int kKeyBytes = 32 * DQ * 2, kValBytes = 32 * DV * 2;
  bf16x8 q[RB][KQ];
  f32x4 o[RB][OB], s[RB][2];
  bf16x8 p[RB];
  float m[RB], l[RB];
  uint32_t ka[KA], va[OB];                                          // this lane's offsets in a tile; the rest are constants

  __device__ __forceinline__ void offsets(int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int k = 0; k < KA; ++k) ka[k] = (uint32_t)(r * (DQ * 2) + ((4 * k + g) ^ at_swz<DQ>(r)) * 16);
#pragma unroll
    for (int b = 0; b < OB; ++b) {
      const int row = 4 * g + (r >> 2);                             // at_swz repeats every 16 rows
      va[b] = (uint32_t)(row * (DV * 2) + ((2 * b + ((r & 3) >> 1)) ^ at_swz<DV>(row)) * 16 + 8 * (r & 1));
    }
  }
  // row: this lane's query row of block rb; all blocks' rows are loaded before settle()
  __device__ __forceinline__ void init(int rb, const uint16_t* row, int lane) {
#pragma unroll
    for (int k = 0; k < KQ; ++k) q[rb][k] = __builtin_bit_cast(bf16x8, *(const u32x4*)(row + 32 * k + 8 * (lane >> 4)));
#pragma unroll
    for (int b = 0; b < OB; ++b) o[rb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[rb] = neg_inf();
    l[rb] = 0.0f;
  }
  __device__ __forceinline__ void settle() {                        // waits for the rows, see AttnWave::init
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int k = 0; k < KQ; ++k) asm volatile("" : "+v"(q[rb][k]));
  }
  __device__ __forceinline__ void scores(const uint8_t* ks) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) s[rb][0] = s[rb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KQ; ++k)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bf16x8 kf = *(const bf16x8*)(ks + ka[k % KA] + (16 * b * (DQ * 2) + (k / KA) * (KA * 64)));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb][b] = mfma16(kf, q[rb][k], s[rb][b]);
      }
  }
  // keys past `last` are not there
  __device__ __forceinline__ void mask(int lane, int last) {
    const int seen = last - 4 * (lane >> 4);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[rb][b][i] = 16 * b + i <= seen ? s[rb][b][i] : neg_inf();
  }
  // as AttnWave::weights
  __device__ __forceinline__ void weights(float c) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      float mx = neg_inf();
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[rb][b][i]);
      mx = quarter_max(mx) * c;
      const bool grown = mx > m[rb] + 8.0f;
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
      float w[8], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = __builtin_amdgcn_exp2f(fmaf(s[rb][j / 4][j % 4], c, -base));
        sum += w[j];
      }
      p[rb] = __builtin_bit_cast(
          bf16x8, u32x4{cvt_bf16x2(w[0], w[1]), cvt_bf16x2(w[2], w[3]), cvt_bf16x2(w[4], w[5]), cvt_bf16x2(w[6], w[7])});
      l[rb] += quarter_sum(sum);
    }
  }
  __device__ __forceinline__ void values(const uint8_t* vs) {
#pragma unroll
    for (int b = 0; b < OB; ++b) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at_lds_s16x4*)(vs + va[b]));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at_lds_s16x4*)(vs + va[b] + 16 * (DV * 2)));
      const bf16x8 vf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) o[rb][b] = mfma16(vf, p[rb], o[rb][b]);
    }
  }
};

}  // namespace moe
