// The 8-bit row code: e4m3 codes under one power-of-two scale per row.
//
// Sixteen lanes hold a row, eight channels each.  The scale's exponent comes
// from the bits of the largest magnitude (448 = 1.75 * 2^8, so it is the
// magnitude's own exponent less 8, one more when its mantissa is above 1.75);
// x 2^-e is exact, and the conversion rounds once.
#pragma once

#include "common.cuh"

namespace bpkv {

constexpr int kExpMin = -48, kExpMax = 32;  // range of a row's scale exponent
constexpr int kExpBias = 127;

__host__ __device__ __forceinline__ int rows8_exponent(uint32_t abs_bf16_bits) {
  const int e = (int)(abs_bf16_bits >> 7) - kExpBias - 8 + ((abs_bf16_bits & 0x7fu) > 0x60u ? 1 : 0);
  return e < kExpMin ? kExpMin : e > kExpMax ? kExpMax : e;
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Codes of two values, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The values of two codes as halves (exact).
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return *reinterpret_cast<__half2*>(&r);
}

// Magnitude bits of eight bf16 channels: the largest of each half of the words.
__device__ __forceinline__ uint32_t abs_max(const uint4& w) {
  return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}

// Scale exponent of a row from the 8 bf16 channels w of each of its 16 lanes.
__device__ __forceinline__ int row_exponent(const uint4& w) {
  uint32_t a = abs_max(w);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
  return rows8_exponent(max(a & 0xffffu, a >> 16));
}

__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float s) {
  return e4m3x2(__uint_as_float(a << 16) * s, __uint_as_float(a & 0xffff0000u) * s) |
         (e4m3x2(__uint_as_float(b << 16) * s, __uint_as_float(b & 0xffff0000u) * s) << 16);
}

__device__ __forceinline__ uint2 row_codes(const uint4& w, int e) {
  const float s = exp2i(-e);
  return make_uint2(codes4(w.x, w.y, s), codes4(w.z, w.w, s));
}

// One cache's code arrays and where a sequence's new rows go in them.
struct Rows8Out {
  uint8_t* k8;
  uint8_t* v8;
  uint8_t* kexp;
  uint8_t* vexp;
  int64_t* seq_len;
  int64_t cap;
};

__host__ __device__ __forceinline__ bool rows8_fits(int64_t start, int64_t t_new, int64_t cap) {
  return start >= 0 && start <= cap - t_new;
}

}  // namespace bpkv
