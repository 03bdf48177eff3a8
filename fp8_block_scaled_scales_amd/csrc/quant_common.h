// Device helpers shared by the kernels that write FP8 codes with block factors
// (quant_fp8.hip, norm_fp8.hip, epilogue_bwd.hip): element kinds, the
// factor and division rule, FP8 conversion and reductions across a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "race_check.h"

namespace dg {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Input element kinds: 0 FP32, 1 BF16, 2 FP16 (the library's DG_IN_* codes).
template <int IN>
struct InKind {
  static constexpr int kBytes = IN == 0 ? 4 : 2;  // bytes per element
  static constexpr int kPerLoad = 16 / kBytes;     // elements per 16-byte load
  static constexpr int kQuads = kPerLoad / 4;      // groups of four per load
};

// Elements 4*H .. 4*H+3 of a 16-byte load, as FP32 (exact for every kind).
// A 32-bit word holds two 16-bit elements, the first in its low half. BF16 is
// the high half of an FP32 pattern; FP16 converts exactly.
template <int IN, int H>
__device__ __forceinline__ v4f widen(v4u w) {
  if constexpr (IN == 0) {
    return __builtin_bit_cast(v4f, w);
  } else {
    const unsigned a = H ? w.z : w.x, b = H ? w.w : w.y;
    if constexpr (IN == 1) {
      return (v4f){__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                   __uint_as_float(b & 0xFFFF0000u)};
    } else {
      const v2h ha = __builtin_bit_cast(v2h, a), hb = __builtin_bit_cast(v2h, b);
      return (v4f){(float)ha.x, (float)ha.y, (float)hb.x, (float)hb.y};
    }
  }
}

__device__ __forceinline__ float amax4(v4f v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v2u16 abs_bits2(unsigned w) { return __builtin_bit_cast(v2u16, w & 0x7FFF7FFFu); }

// max |x| over the elements of one 16-byte load. For 16-bit input the max is
// taken on the bit patterns: with the sign bit cleared, the patterns of
// finite BF16 or FP16 values order as the magnitudes do, so a packed 16-bit
// integer max finds the largest, which is then widened once. Nothing widened
// here stays live until the encode pass, which widens its own copies.
template <int IN>
__device__ __forceinline__ float amax_load(v4u w) {
  if constexpr (IN == 0) {
    return amax4(widen<IN, 0>(w));
  } else {
    const v2u16 m = __builtin_elementwise_max(__builtin_elementwise_max(abs_bits2(w.x), abs_bits2(w.y)),
                                              __builtin_elementwise_max(abs_bits2(w.z), abs_bits2(w.w)));
    const unsigned top = m.x > m.y ? m.x : m.y;
    if constexpr (IN == 1) return __uint_as_float(top << 16);
    else return (float)__builtin_bit_cast(_Float16, (unsigned short)top);
  }
}

// A block's factor: amax / fmax (correctly rounded), or 1.0 where that is
// zero: an all-zero block, or one whose amax is so small that the quotient
// underflows (no factor of zero to divide by; 1.0 encodes its values, all
// below fmax * 2^-150, under 2^-134, as zeros).
__device__ __forceinline__ float block_scale(float amax, float fmax) {
  const float s = amax / fmax;
  return s > 0.0f ? s : 1.0f;
}

// Division by a block's scale s, rounded as the correctly rounded FP32 divide
// rounds it, without a divide per element. inv = RN(1/s) is computed once per
// block (a correctly rounded divide); per element q0 = RN(x * inv) lies within
// 1.5 ulp of x/s, one correction q1 = RN(q0 + RN(x - q0*s) * inv) (the
// remainder exact under the FMA) brings it within one ulp, and a second
// correction then gives RN(x/s) by Markstein's theorem on FMA-based division
// (P. Markstein, "IA-64 and Elementary Functions", 2000; also the chapter on
// division with an FMA in the Handbook of Floating-Point Arithmetic): with a
// correctly rounded reciprocal and a quotient within one ulp, the corrected
// quotient is the correctly rounded one. The theorem asks that nothing
// overflows or underflows: s and 1/s normal (the caller's uniform test,
// recip_ok; blocks outside it divide per element) and x/s at most the
// format's largest value. A quotient in FP32's subnormal range may come out
// wrong in its last bits, but every such value is far below half the smallest
// FP8 subnormal and encodes to a signed zero either way; the sign is x's (an
// input -0 gives -0, where the corrections alone would give +0).
__device__ __forceinline__ bool recip_ok(float s) { return s >= 0x1p-120f && s <= 0x1p120f; }

__device__ __forceinline__ float div_by_scale(float x, float s, float inv) {
  float q = x * inv;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
  return __builtin_copysignf(q, x);
}

// One DPP move of v across the wave (row_mask, bank_mask all on; every
// source lane exists for the patterns used here).
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Max over each aligned group of L lanes (L = 8, 16, 32 or 64), in every lane
// of the group: within quads by two swaps (DPP quad_perm [1,0,3,2],
// [2,3,0,1]), then each lane against its mirror in the 8-lane half row, which
// leaves the half row's max in every lane, and in the 16-lane row (DPP
// row_half_mirror, row_mirror); beyond 16 lanes, cross-lane shuffles. max is
// exact and order-free.
template <int L>
__device__ __forceinline__ float group_max(float m) {
  static_assert(L == 8 || L == 16 || L == 32 || L == 64, "group");
  m = fmaxf(m, dpp_f<0xB1>(m));
  m = fmaxf(m, dpp_f<0x4E>(m));
  m = fmaxf(m, dpp_f<0x141>(m));
  if constexpr (L >= 16) m = fmaxf(m, dpp_f<0x140>(m));
  if constexpr (L >= 32) m = fmaxf(m, __shfl_xor(m, 16, 64));
  if constexpr (L >= 64) m = fmaxf(m, __shfl_xor(m, 32, 64));
  return m;
}

// Two FP8 codes of (x0, x1) packed into the low (HI = false) or high half of
// `old`: FMT 0 E4M3FN, 1 E5M2 (hardware round-to-nearest-even).
template <int FMT, bool HI>
__device__ __forceinline__ int cvt2(float x0, float x1, int old) {
  if constexpr (FMT == 1) return __builtin_amdgcn_cvt_pk_bf8_f32(x0, x1, old, HI);
  else return __builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, old, HI);
}

// Four codes of v / s in one 32-bit word (bytes in element order). FAST (s
// and 1/s normal): |v / s| rounds to at most fmax, since s carries a relative
// error of at most 2^-24. Otherwise s is subnormal or tiny, its own rounding
// can be coarse enough that |v / s| passes fmax, and the quotient saturates
// to +-fmax as FP8's round-to-nearest with saturation takes it (the
// conversion instruction alone does not saturate).
template <int FMT, bool FAST>
__device__ __forceinline__ int encode4(v4f v, float s, float inv) {
  if constexpr (FAST) {
    const int lo = cvt2<FMT, false>(div_by_scale(v.x, s, inv), div_by_scale(v.y, s, inv), 0);
    return cvt2<FMT, true>(div_by_scale(v.z, s, inv), div_by_scale(v.w, s, inv), lo);
  } else {
    constexpr float FMAX = FMT == 1 ? 57344.0f : 448.0f;
    auto sat = [](float y) { return fminf(fmaxf(y, -FMAX), FMAX); };
    const int lo = cvt2<FMT, false>(sat(v.x / s), sat(v.y / s), 0);
    return cvt2<FMT, true>(sat(v.z / s), sat(v.w / s), lo);
  }
}

// Inputs of 64 MB and more, twice the L2s, are read and the outputs made from
// them written nontemporally (ONCE below).
constexpr int64_t kOnceBytes = 64ll << 20;

// E (4 or 8) consecutive elements of kind K as loaded, so that a value waiting
// for its row's reduction costs half a register for 16-bit kinds.
//
// A lane takes eight elements at a time where every operand is 16-bit and four
// where one is FP32 (unit_of), so that it moves 16 bytes of the widest operand
// in one instruction and neighbouring lanes touch neighbouring pieces: copying
// 512 MB in pieces of 32 bytes per lane, two instructions each, runs at 4.18
// TB/s, in single 16-byte pieces at 5.90.
template <int K, int E>
struct Raw {
  static constexpr int W = E * InKind<K>::kBytes / 4;  // words
  unsigned w[W];
};

constexpr int unit_of(int k0, int k1) { return k0 == 0 || k1 == 0 ? 4 : 8; }

typedef unsigned v2u __attribute__((ext_vector_type(2)));

// p: base of a matrix of kind K; e: index of the first element (the address
// is aligned to the E elements' bytes, up to 16). ONCE (here and below):
// nontemporal, for data that is larger than the caches.
template <int K, int E, bool ONCE = false>
__device__ __forceinline__ Raw<K, E> load_raw(const void* p, int64_t e) {
  typedef typename std::conditional<Raw<K, E>::W == 2, v2u, v4u>::type V;
  constexpr int N = sizeof(V) / 4;
  Raw<K, E> r;
  const V* src = reinterpret_cast<const V*>(static_cast<const char*>(p) + e * InKind<K>::kBytes);
#pragma unroll
  for (int i = 0; i < Raw<K, E>::W / N; ++i) {
    const V v = ONCE ? __builtin_nontemporal_load(src + i) : src[i];
#pragma unroll
    for (int k = 0; k < N; ++k) r.w[i * N + k] = v[k];
  }
  return r;
}

template <int K, int E>
__device__ __forceinline__ void widen_raw(const Raw<K, E>& r, float (&f)[E]) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    v4f v;
    if constexpr (K == 0) v = widen<K, 0>((v4u){r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]});
    else v = widen<K, 0>((v4u){r.w[2 * q], r.w[2 * q + 1], 0u, 0u});
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * q + i] = v[i];
  }
}

// FP32 -> kind K, round to nearest even (FP16: past 65504 to infinity).
template <int K, int E>
__device__ __forceinline__ Raw<K, E> round_raw(const float (&f)[E]) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  Raw<K, E> r;
#pragma unroll
  for (int i = 0; i < Raw<K, E>::W; ++i) {
    if constexpr (K == 0) r.w[i] = __float_as_uint(f[i]);
    else if constexpr (K == 1) r.w[i] = __builtin_bit_cast(unsigned, (v2bf){(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
    else r.w[i] = __builtin_bit_cast(unsigned, (v2h){(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
  }
  return r;
}

template <bool ONCE = false, int K, int E>
__device__ __forceinline__ void store_raw(void* p, int64_t e, const Raw<K, E>& r) {
  typedef typename std::conditional<Raw<K, E>::W == 2, v2u, v4u>::type V;
  constexpr int N = sizeof(V) / 4;
  V* dst = reinterpret_cast<V*>(static_cast<char*>(p) + e * InKind<K>::kBytes);
#pragma unroll
  for (int i = 0; i < Raw<K, E>::W / N; ++i) {
    V v;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = r.w[i * N + k];
    if constexpr (ONCE) __builtin_nontemporal_store(v, dst + i);
    else dst[i] = v;
  }
}

// Max over the lanes that share a g-wide segment when a lane holds E of its
// elements: g / E = 8 to 64 lanes (g the same for the whole launch).
template <int E>
__device__ __forceinline__ float segment_max(float m, int g) {
  m = group_max<8>(m);
  if (g / E >= 16) m = fmaxf(m, dpp_f<0x140>(m));
  if (g / E >= 32) m = fmaxf(m, __shfl_xor(m, 16, 64));
  if (g / E >= 64) m = fmaxf(m, __shfl_xor(m, 32, 64));
  return m;
}

template <int E>
__device__ __forceinline__ float amax_of(const float (&y)[E]) {
  float m = amax4((v4f){y[0], y[1], y[2], y[3]});
  if constexpr (E == 8) m = fmaxf(m, amax4((v4f){y[4], y[5], y[6], y[7]}));
  return m;
}

__device__ __forceinline__ float format_max(int fmt) { return fmt == 1 ? 57344.0f : 448.0f; }

// The codes of y / s (fmt 0 E4M3FN, 1 E5M2, the same for the whole launch) to q;
// inv = 1 / s where recip_ok(s).
template <int FMT, bool ONCE, int E>
__device__ __forceinline__ void store_codes_fmt(uint8_t* q, const float (&y)[E], float s, float inv) {
  int c[E / 4];
  const bool fast = recip_ok(s);
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const v4f v = {y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
    if (fast) c[i] = encode4<FMT, true>(v, s, inv);
    else c[i] = encode4<FMT, false>(v, s, inv);
  }
  if constexpr (E == 8) {
    if constexpr (ONCE) __builtin_nontemporal_store((v2i){c[0], c[1]}, reinterpret_cast<v2i*>(q));
    else *reinterpret_cast<v2i*>(q) = (v2i){c[0], c[1]};
  } else {
    if constexpr (ONCE) __builtin_nontemporal_store(c[0], reinterpret_cast<int*>(q));
    else *reinterpret_cast<int*>(q) = c[0];
  }
}

template <bool ONCE = false, int E>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&y)[E], float s, float inv, int fmt) {
  if (fmt == 1) store_codes_fmt<1, ONCE>(q, y, s, inv);
  else store_codes_fmt<0, ONCE>(q, y, s, inv);
}

// Sum over the wave in every lane, in a fixed order: DPP swaps and mirrors
// inside 16-lane rows (as group_max), shuffles across them.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  v += dpp_f<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// A workgroup of RL x CL threads whose thread (rl, cl) holds partial sums of
// columns 8 cl .. 8 cl + 7 of 8 CL: their totals to out, in a fixed order (every
// group of 8 CL threads adds eight rows, then the first adds the groups).
template <int RL, int CL>
__device__ __forceinline__ void column_sums_of_lanes(const float (&acc)[8], float (&red)[RL][8 * CL], float* out) {
  const int cl = threadIdx.x % CL, rl = threadIdx.x / CL;
  DG_STEP_SYNC_WG();
#pragma unroll
  for (int k = 0; k < 8; ++k) red[rl][cl * 8 + k] = acc[k];
  __syncthreads();
  DG_STEP_SYNC_WG();
  const int c = threadIdx.x % (8 * CL), g = threadIdx.x / (8 * CL);
  float v = red[g * 8][c];
#pragma unroll
  for (int i = 1; i < 8; ++i) v += red[g * 8 + i][c];
  __syncthreads();
  DG_STEP_SYNC_WG();
  red[g][c] = v;
  __syncthreads();
  DG_STEP_SYNC_WG();
  if (g == 0) {
#pragma unroll 16
    for (int i = 1; i < RL / 8; ++i) v += red[i][c];
    out[c] = v;
  }
}

}  // namespace dg
