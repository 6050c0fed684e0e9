// pa_codec.cuh -- the quantised pools' writers' codecs ("KV Cache Engineering for LLM
// Serving", section 8): four consecutive elements of a head vector per lane (D = 128).
#pragma once

#include "pa_common.cuh"

namespace pa {

// E4M3 codes, one byte per element; a lane's four codes are one 32-bit word.
struct Fp8Codec {
  static constexpr int kRowBytes = 128;
  static constexpr float kMaxCode = 448.f;
  static constexpr float kPerCode = 1.f / 448.f;
  using Word = uint32_t;
  static __device__ __forceinline__ Word encode(const float (&v)[4], float s) {
    if (s == 0.f) return 0u;
    return f32x2_to_e4m3x2(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s)) |
           (f32x2_to_e4m3x2(__fdiv_rn(v[2], s), __fdiv_rn(v[3], s)) << 16);
  }
  // codes restored with the old scale (one fp32 product each), encoded with the new
  static __device__ __forceinline__ Word reencode(Word c, float old, float s) {
    const float2 lo = e4m3x2_to_float2(c), hi = e4m3x2_to_float2(c >> 16);
    const float v[4] = {__fmul_rn(lo.x, old), __fmul_rn(lo.y, old), __fmul_rn(hi.x, old),
                        __fmul_rn(hi.y, old)};
    return encode(v, s);
  }
};

// 4-bit codes clip(rint(x / scale), -7, 7) stored as offset-binary nibbles, element 2j in
// the low nibble of byte j; a lane's four codes are one 16-bit word.
__device__ __forceinline__ uint32_t int4_code(float x, float scale) {
  if (scale == 0.f) return 8u;
  const float c = fminf(fmaxf(rintf(__fdiv_rn(x, scale)), -7.f), 7.f);
  return static_cast<uint32_t>(static_cast<int>(c) + 8);
}

struct Int4Codec {
  static constexpr int kRowBytes = 64;
  static constexpr float kMaxCode = 7.f;
  static constexpr float kPerCode = 1.f / 7.f;
  using Word = uint16_t;
  static __device__ __forceinline__ Word encode(const float (&v)[4], float s) {
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) code |= int4_code(v[e], s) << (4 * e);
    return static_cast<Word>(code);
  }
  static __device__ __forceinline__ Word reencode(Word c, float old, float s) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = __fmul_rn(static_cast<float>(static_cast<int>((c >> (4 * e)) & 0xF) - 8), old);
    return encode(v, s);
  }
};

}  // namespace pa
