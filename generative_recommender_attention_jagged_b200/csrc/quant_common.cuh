// The low-precision number formats, one definition for every kernel that
// writes or reads them.
//
// 8-bit rows (activations, weight channels): scale = amax / 127 in fp32,
// code = x / scale rounded to the nearest integer, ties to even.
//
// 4-bit rows (one token and head of the cache): with lo = min(0, min x) and
// hi = max(0, max x), scale = (hi - lo) / 15 rounded to bf16, zero point
// z = -lo / scale and code = x / scale + z, both rounded to the nearest
// integer (ties to even) and clamped to 0..15; the element stands for
// scale * (code - z).  0 is always representable and code - z is an integer in
// -15..15, exact in bf16.  A row takes d / 2 bytes; in each group of 8 elements
// (one 32-bit word) nibble i holds element 2 i and nibble i + 4 element 2 i + 1,
// so that (w >> 4 i) & 0x000F000F is the pair of elements (2 i, 2 i + 1).
// Beside it stand the scale and the zero point as two bf16 (one 32-bit word).
//
// Both: a scale below the smallest normal fp32 number makes the row zeros
// (scale 0, codes 0); a row with an infinity or NaN (or whose range overflows)
// gets scale NaN and codes 0, so whatever uses it is NaN as well.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <cfloat>

namespace hstu {
namespace {

constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer (ties to even)

// x / s rounded to the nearest integer, ties to even, for |x / s| < 2^21, as
// kRoundMagic + integer (its low bits are the integer in two's complement).
// The first guess m = rint(x inv) with inv ~ 1 / s is within one of the answer,
// and the remainder x - q s is exact in one FMA (a multiple of the smaller ulp,
// no larger than about s): while it is below s / 2 the guess stands, whatever
// the error of inv, and otherwise (a tie, or a quotient so near one that inv's
// error decided) fix_quotient compares exactly.  A rounded quotient is not exact
// at ties; an IEEE division costs more than guess and test together (three FMA
// pipe operations and one comparison).
__device__ __forceinline__ float guess_quotient(float x, float inv) { return fmaf(x, inv, kRoundMagic); }
// twice the remainder of the guess m
__device__ __forceinline__ float twice_rest(float x, float s, float m) {
  return 2.f * fmaf(kRoundMagic - m, s, x);
}
__device__ __forceinline__ float fix_quotient(float x, float s, float m) {
  const float t = twice_rest(x, s, m);
  const bool odd = __float_as_int(m) & 1;
  if (t > s || (odd && t == s)) m += 1.f;
  if (t < -s || (odd && t == -s)) m -= 1.f;
  return m;
}
__device__ __forceinline__ float round_quotient(float x, float s, float inv) {
  return fix_quotient(x, s, guess_quotient(x, inv));
}

// rounded quotients of 8 elements, as round_quotient
__device__ __forceinline__ void round_quotients8(const float (&x)[8], float s, float inv, float (&m)[8]) {
  bool stands = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = guess_quotient(x[i], inv);
    stands = stands && fabsf(fmaf(kRoundMagic - m[i], s, x[i])) < 0.5f * s;
  }
  if (!stands) {  // about one element in a thousand
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fix_quotient(x[i], s, m[i]);
  }
}

// smallest and largest, NaN if either is NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// packed fp32 pairs (one instruction for two operations, each rounded as its scalar form)
__device__ __forceinline__ uint64_t pack_pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_pair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// x / s for |x / s| < 2^20, s and inv ~ 1 / s normal: the remainder of a first
// product is exact, and adding its share again gives the quotient to half an ulp and
// exactly where it has a short binary fraction (the correction is then off by far less
// than the last bit).  Three operations of the FMA pipe for two quotients.
__device__ __forceinline__ uint64_t quotients(uint64_t x, uint64_t minus_s, uint64_t inv) {
  const uint64_t q = mul_pair(x, inv);
  return fma_pair(fma_pair(q, minus_s, x), inv, q);
}

struct Quant4 {
  float s, inv;   // bf16-exact scale (0: all codes 0) and about its reciprocal
  float z;        // zero point 0..15
  uint32_t meta;  // the stored word: scale | zero << 16 (bf16 bits)
};

// Format of a row with extremes lo <= 0 <= hi (NaN if an element is).  `clamp`: an end
// of the row rounds to a code outside 0..15.
__device__ __forceinline__ Quant4 quant4_of(float lo, float hi, bool& clamp) {
  Quant4 f;
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f));
  const float s = __bfloat162float(sb);
  const bool nan = !(s <= FLT_MAX);  // an infinity, a NaN or a range beyond fp32
  const bool live = !nan && s >= FLT_MIN;
  f.s = live ? s : 0.f;
  f.inv = live ? __frcp_rn(s) : 0.f;
  f.z = live ? fminf(round_quotient(-lo, s, f.inv) - kRoundMagic, 15.f) : 0.f;
  clamp = live && (round_quotient(lo, s, f.inv) - kRoundMagic + f.z < 0.f ||
                   round_quotient(hi, s, f.inv) - kRoundMagic + f.z > 15.f);
  const uint32_t sbits = live ? (uint32_t)__bfloat16_as_ushort(sb) : (nan ? 0x7FC0u : 0u);
  f.meta = sbits | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f.z)) << 16);
  return f;
}

// The word of 8 elements.  A quotient of two bf16 numbers is a half-integer or at
// least 2^-16 away from one (relative), so the rounded quotient decides a bf16 row's
// codes; for fp32 rows one that comes out as a half-integer is compared exactly.  The
// codes are put together as fp32 sums of code * 16^i (at most 65535, exact), four to a
// half of the word.
template <bool BF16>
__device__ __forceinline__ uint32_t quant4_word(float s, float inv, float z, bool clamp, const float (&x)[8]) {
  if (s == 0.f) return 0;
  const uint64_t ms2 = pack_pair(-s, -s), inv2 = pack_pair(inv, inv), magic2 = pack_pair(kRoundMagic, kRoundMagic),
                 back2 = pack_pair(-kRoundMagic, -kRoundMagic);
  uint64_t m[4];  // pairs of elements 2 i, 2 i + 1: kRoundMagic + rounded quotient
  bool half = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q = quotients(pack_pair(x[2 * i], x[2 * i + 1]), ms2, inv2);
    m[i] = add_pair(q, magic2);
    if constexpr (!BF16) {
      float q0, q1, m0, m1;
      unpack_pair(q, q0, q1);
      unpack_pair(add_pair(m[i], back2), m0, m1);
      half = half || fabsf(q0 - m0) == 0.5f || fabsf(q1 - m1) == 0.5f;
    }
  }
  if (!BF16 && half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m0, m1;
      unpack_pair(m[i], m0, m1);
      m[i] = pack_pair(fix_quotient(x[2 * i], s, m0), fix_quotient(x[2 * i + 1], s, m1));
    }
  }
  if (clamp) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m0, m1;
      unpack_pair(m[i], m0, m1);
      m[i] = pack_pair(fminf(fmaxf(m0, kRoundMagic - z), kRoundMagic + 15.f - z),
                   fminf(fmaxf(m1, kRoundMagic - z), kRoundMagic + 15.f - z));
    }
  }
  uint64_t sum = pack_pair(z * 4369.f, z * 4369.f);  // 0x1111
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float w = (float)(1 << (4 * i));
    sum = fma_pair(add_pair(m[i], back2), pack_pair(w, w), sum);
  }
  float even, odd;
  unpack_pair(add_pair(sum, pack_pair(8388608.f, 8388608.f)), even, odd);
  return __byte_perm(__float_as_uint(even), __float_as_uint(odd), 0x5410);
}

// scale and zero point of a stored word
__device__ __forceinline__ float meta_scale(uint32_t meta) { return __uint_as_float(meta << 16); }
__device__ __forceinline__ float meta_zero(uint32_t meta) { return __uint_as_float(meta & 0xFFFF0000u); }

// bit position of element e (0..7) inside its 32-bit word
__host__ __device__ __forceinline__ int nibble_shift(int e) { return 4 * ((e >> 1) + 4 * (e & 1)); }

// packed bf16: smaller / larger of each half, NaN if either is NaN
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 8 consecutive elements of a row as they lie, and the row's extremes packed so
// that one shuffle carries both
template <typename T>
struct Elems8;
template <>
struct Elems8<__nv_bfloat16> {
  using Extremes = uint32_t;  // bf16 pair (-smallest, largest)
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ Extremes extremes() const {
    uint32_t lo = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
    uint32_t hi = max2_nan(max2_nan(w[0], w[1]), max2_nan(w[2], w[3]));
    lo = min2_nan(lo, __byte_perm(lo, lo, 0x1032));
    hi = max2_nan(hi, __byte_perm(hi, hi, 0x1032));
    return __byte_perm(lo ^ 0x80008000u, hi, 0x5410);
  }
  __device__ static __forceinline__ Extremes join(Extremes a, Extremes b) { return max2_nan(a, b); }
  __device__ static __forceinline__ Extremes other(Extremes a, int mask) { return __shfl_xor_sync(~0u, a, mask); }
  // with 0 among them
  __device__ static __forceinline__ float lowest(Extremes a) { return -__uint_as_float(max2_nan(a, 0u) << 16); }
  __device__ static __forceinline__ float highest(Extremes a) { return __uint_as_float(max2_nan(a, 0u) & 0xFFFF0000u); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Elems8<float> {
  using Extremes = float2;
  float e[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    e[0] = a.x, e[1] = a.y, e[2] = a.z, e[3] = a.w, e[4] = b.x, e[5] = b.y, e[6] = b.z, e[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = 0.f;
  }
  __device__ __forceinline__ Extremes extremes() const {
    float lo = e[0], hi = e[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = min_nan(lo, e[i]);
      hi = max_nan(hi, e[i]);
    }
    return make_float2(lo, hi);
  }
  __device__ static __forceinline__ Extremes join(Extremes a, Extremes b) {
    return make_float2(min_nan(a.x, b.x), max_nan(a.y, b.y));
  }
  __device__ static __forceinline__ Extremes other(Extremes a, int mask) {
    return make_float2(__shfl_xor_sync(~0u, a.x, mask), __shfl_xor_sync(~0u, a.y, mask));
  }
  __device__ static __forceinline__ float lowest(Extremes a) { return min_nan(a.x, 0.f); }
  __device__ static __forceinline__ float highest(Extremes a) { return max_nan(a.y, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = e[i];
  }
};

// 8 consecutive elements as fp32
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace
}  // namespace hstu
