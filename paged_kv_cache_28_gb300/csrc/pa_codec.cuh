// pa_codec.cuh -- the quantised pools' writers' codecs ("KV Cache Engineering for LLM
// Serving", section 8): four consecutive elements of a head vector per lane (D = 128).
#pragma once

#include "pa_common.cuh"

namespace pa {

// x / s in fp32, correctly rounded, by the division itself.
struct ByDivision {
  float s;
  __device__ __forceinline__ float operator()(float x) const { return __fdiv_rn(x, s); }
};

// The same bits from the correctly rounded reciprocal, for many x of one s (Markstein's final
// step: with y = RN(1 / s) and q within one unit of x / s, q + (x - q s) y rounds to RN(x / s)).
// x y is within two units, so the step is taken twice, the first time to come within one.  The
// remainders are exact while nothing underflows: `fits` says that s is far from the ends of the
// range, and an x so far below s that its remainder underflows has code 0 anyway.
struct ByReciprocal {
  float s, y;
  __device__ __forceinline__ explicit ByReciprocal(float scale) : s(scale), y(1.f / scale) {}
  __device__ __forceinline__ bool fits() const { return s > 0x1p-60f && s < 0x1p60f; }
  __device__ __forceinline__ float operator()(float x) const {
    float q = __fmul_rn(x, y);
    q = __fmaf_rn(__fmaf_rn(-q, s, x), y, q);
    q = __fmaf_rn(__fmaf_rn(-q, s, x), y, q);
    return copysignf(q, x);                              // (a zero remainder is +0; s > 0)
  }
};

// E4M3 codes, one byte per element; a lane's four codes are one 32-bit word.
struct Fp8Codec {
  static constexpr int kRowBytes = 128;
  static constexpr float kMaxCode = 448.f;
  static constexpr float kPerCode = 1.f / 448.f;
  using Word = uint32_t;
  template <class Over>
  static __device__ __forceinline__ Word encode_over(const float (&v)[4], const Over &over) {
    if (over.s == 0.f) return 0u;
    return f32x2_to_e4m3x2(over(v[0]), over(v[1])) | (f32x2_to_e4m3x2(over(v[2]), over(v[3])) << 16);
  }
  static __device__ __forceinline__ Word encode(const float (&v)[4], float s) {
    return encode_over(v, ByDivision{s});
  }
  // codes restored with the old scale (one fp32 product each), encoded with the new
  static __device__ __forceinline__ Word reencode(Word c, float old, float s) {
    return reencode_over(c, old, ByDivision{s});
  }
  template <class Over>
  static __device__ __forceinline__ Word reencode_over(Word c, float old, const Over &over) {
    const float2 lo = e4m3x2_to_float2(c), hi = e4m3x2_to_float2(c >> 16);
    const float v[4] = {__fmul_rn(lo.x, old), __fmul_rn(lo.y, old), __fmul_rn(hi.x, old),
                        __fmul_rn(hi.y, old)};
    return encode_over(v, over);
  }
};

// 4-bit codes clip(rint(x / scale), -7, 7) stored as offset-binary nibbles, element 2j in
// the low nibble of byte j; a lane's four codes are one 16-bit word.
template <class Over>
__device__ __forceinline__ uint32_t int4_code(float x, const Over &over) {
  if (over.s == 0.f) return 8u;
  const float c = fminf(fmaxf(rintf(over(x)), -7.f), 7.f);
  return static_cast<uint32_t>(static_cast<int>(c) + 8);
}

struct Int4Codec {
  static constexpr int kRowBytes = 64;
  static constexpr float kMaxCode = 7.f;
  static constexpr float kPerCode = 1.f / 7.f;
  using Word = uint16_t;
  template <class Over>
  static __device__ __forceinline__ Word encode_over(const float (&v)[4], const Over &over) {
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) code |= int4_code(v[e], over) << (4 * e);
    return static_cast<Word>(code);
  }
  static __device__ __forceinline__ Word encode(const float (&v)[4], float s) {
    return encode_over(v, ByDivision{s});
  }
  static __device__ __forceinline__ Word reencode(Word c, float old, float s) {
    return reencode_over(c, old, ByDivision{s});
  }
  template <class Over>
  static __device__ __forceinline__ Word reencode_over(Word c, float old, const Over &over) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = __fmul_rn(static_cast<float>(static_cast<int>((c >> (4 * e)) & 0xF) - 8), old);
    return encode_over(v, over);
  }
};

}  // namespace pa
