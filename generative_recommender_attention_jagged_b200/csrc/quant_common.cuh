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

struct Quant4 {
  float s, inv;   // bf16-exact scale and about its reciprocal
  float z;        // zero point 0..15
  uint32_t meta;  // the stored word: scale | zero << 16 (bf16 bits)
  bool live;      // codes are not all zero
  bool clamp;     // an end of the row rounds to a code outside 0..15
};

// Format of a row with extremes lo <= 0 <= hi (NaN if an element is).
__device__ __forceinline__ Quant4 quant4_of(float lo, float hi) {
  Quant4 f;
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f));
  f.s = __bfloat162float(sb);
  const bool nan = !(f.s <= FLT_MAX);  // an infinity, a NaN or a range beyond fp32
  f.live = !nan && f.s >= FLT_MIN;
  f.inv = f.live ? 1.f / f.s : 0.f;
  f.z = f.live ? fminf(round_quotient(-lo, f.s, f.inv) - kRoundMagic, 15.f) : 0.f;
  f.clamp = f.live && (round_quotient(lo, f.s, f.inv) - kRoundMagic + f.z < 0.f ||
                       round_quotient(hi, f.s, f.inv) - kRoundMagic + f.z > 15.f);
  const uint32_t sbits = f.live ? (uint32_t)__bfloat16_as_ushort(sb) : (nan ? 0x7FC0u : 0u);
  f.meta = sbits | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f.z)) << 16);
  return f;
}

// The word of 8 elements.  The codes are put together as fp32 sums of
// code * 16^i (at most 65535, exact), four to a half of the word.
__device__ __forceinline__ uint32_t quant4_word(const Quant4& f, const float (&x)[8]) {
  if (!f.live) return 0;
  float m[8];
  round_quotients8(x, f.s, f.inv, m);
  if (f.clamp) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fminf(fmaxf(m[i], kRoundMagic - f.z), kRoundMagic + 15.f - f.z);
  }
  float even = f.z * 4369.f, odd = even;  // 0x1111
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    even = fmaf(m[2 * i] - kRoundMagic, (float)(1 << (4 * i)), even);
    odd = fmaf(m[2 * i + 1] - kRoundMagic, (float)(1 << (4 * i)), odd);
  }
  return __byte_perm(__float_as_uint(even + 8388608.f), __float_as_uint(odd + 8388608.f), 0x5410);
}

// scale and zero point of a stored word
__device__ __forceinline__ float meta_scale(uint32_t meta) { return __uint_as_float(meta << 16); }
__device__ __forceinline__ float meta_zero(uint32_t meta) { return __uint_as_float(meta & 0xFFFF0000u); }

// bit position of element e (0..7) inside its 32-bit word
__host__ __device__ __forceinline__ int nibble_shift(int e) { return 4 * ((e >> 1) + 4 * (e & 1)); }

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
