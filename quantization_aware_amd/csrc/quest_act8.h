// The 8-bit activation checkpoint: its format and the lane code shared by the
// kernels that write or read it.
//
// A row is cut into blocks of 32 columns (the last may be shorter).  With
// E the biased fp32 exponent of a block's largest magnitude (0 for zeros and
// fp32 subnormals), an entry x is held as
//   q = clamp(round_to_nearest_even(x * 2^(133 - E)), -127, 127),
// and stands for q * 2^(E - 133): the largest entry has 6 or 7 fraction bits
// left, the others the same absolute step.  The scale is a power of two (the
// E8M0 scale and block of 32 of the OCP Microscaling Formats specification
// v1.0, with its INT8 elements), so both scalings are exact and the one
// rounding is that of q: nothing depends on a division's last bit, every
// value is exact in bf16, and saving what was loaded gives the same bytes.
// A block holding an infinity or NaN has E = 255 and stands for NaN whole.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quest {

constexpr int kAct8Block = 32;

// fp32 <-> the element types.
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));  // round to nearest even
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return f32_to_bf16(v); }

// 8 consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// The magnitude's bit pattern: ordered as the magnitudes, NaN above infinity.
__device__ __forceinline__ uint32_t act8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One entry of a block whose largest magnitude has biased exponent e.
__device__ __forceinline__ int act8_encode(float v, int e) {
  const float q = __builtin_rintf(__builtin_ldexpf(v, 133 - e));
  return e == 255 ? 0 : static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}

// The value of code q under biased exponent e.
__device__ __forceinline__ float act8_decode(int q, int e) {
  return e == 255 ? __builtin_nanf("") : __builtin_ldexpf(static_cast<float>(q), e - 133);
}

// Four codes in a dword, entry 0 lowest.
__device__ __forceinline__ uint32_t act8_pack(int a, int b, int c, int d) {
  return (static_cast<uint32_t>(a) & 255u) | ((static_cast<uint32_t>(b) & 255u) << 8) |
         ((static_cast<uint32_t>(c) & 255u) << 16) | (static_cast<uint32_t>(d) << 24);
}
__device__ __forceinline__ int act8_byte(uint32_t w, int i) { return static_cast<int8_t>(w >> (8 * i)); }

// max over the lanes of an aligned group of 4 (quad) or 32 lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}
__device__ __forceinline__ uint32_t half_wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, 64)));
  return v;
}

}  // namespace quest
