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

// The same at any address that is a multiple of the element's size: global
// memory takes wide accesses there, at no more than the lines they touch.
template <typename T>
__device__ __forceinline__ void load8_at(const T* p, float (&v)[8]) {
  typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
  const u32x4_u a = *reinterpret_cast<const u32x4_u*>(p);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
    const u32x4_u b = *reinterpret_cast<const u32x4_u*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8_at(T* p, const float (&v)[8]) {
  typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<u32x4_u*>(p) =
        u32x4_u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<u32x4_u*>(p + 4 * h) =
          u32x4_u{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                  __float_as_uint(v[4 * h + 3])};
  }
}
__device__ __forceinline__ uint2 load_codes8_at(const int8_t* p) {
  typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));
  const u32x2_u a = *reinterpret_cast<const u32x2_u*>(p);
  return make_uint2(a[0], a[1]);
}
__device__ __forceinline__ void store_codes8_at(int8_t* p, uint2 w) {
  typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));
  *reinterpret_cast<u32x2_u*>(p) = u32x2_u{w.x, w.y};
}

// A group of 8 columns from c (a multiple of 8) of a row of `cols` >= 8 that is
// no whole number of groups.  Every load is 8 wide and behind no branch: the
// row's last group, and any past it, is taken `skip` entries early, so that it
// ends with the row; its first `skip` entries belong to the group before (all 8
// and more: no entry is its own) and count for nothing.
struct Group {
  int at, skip;
  __device__ __forceinline__ Group(int c, int cols) : at(min(c, cols - 8)), skip(c - at) {}
  __device__ __forceinline__ bool own(int i) const { return i >= skip; }
};
// Its own entries to memory (p: entry 0).
template <typename T>
__device__ __forceinline__ void store8_own(T* p, const Group& g, const float (&v)[8]) {
  if (g.skip == 0) {
    store8_at(p, v);
  } else if (g.skip < 8) {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= g.skip) p[i] = from_f32<T>(v[i]);
  }
}
__device__ __forceinline__ void store_codes8_own(int8_t* p, const Group& g, uint2 w) {
  if (g.skip == 0) {
    store_codes8_at(p, w);
  } else if (g.skip < 8) {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= g.skip) p[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// For rows that may be narrower than a group: the `left` entries that a row has
// from p on, 8 or more, a row's last few one by one (the others read as zero), or
// none.
template <typename T>
__device__ __forceinline__ void load8_tail(const T* p, int left, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (left >= 8) {
    load8_at(p, v);
  } else if (left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) v[i] = to_f32(p[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store8_tail(T* p, int left, const float (&v)[8]) {
  if (left >= 8) {
    store8_at(p, v);
  } else if (left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) p[i] = from_f32<T>(v[i]);
  }
}
__device__ __forceinline__ uint2 load_codes8_tail(const int8_t* p, int left) {
  uint2 w = make_uint2(0, 0);
  if (left >= 8) {
    w = load_codes8_at(p);
  } else if (left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) (i < 4 ? w.x : w.y) |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3));
  }
  return w;
}
__device__ __forceinline__ void store_codes8_tail(int8_t* p, int left, uint2 w) {
  if (left >= 8) {
    store_codes8_at(p, w);
  } else if (left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) p[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
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

// 8 entries encoded and decoded.
__device__ __forceinline__ uint2 act8_encode8(const float (&v)[8], int e) {
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = act8_encode(v[i], e);
  return make_uint2(act8_pack(q[0], q[1], q[2], q[3]), act8_pack(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ void act8_decode8(uint2 w, int e, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act8_decode(act8_byte(i < 4 ? w.x : w.y, i & 3), e);
}
__device__ __forceinline__ uint32_t act8_mag8(const float (&v)[8]) {
  uint32_t a = act8_mag(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max(a, act8_mag(v[i]));
  return a;
}

// Four entries, packed: adding 1.5 * 2^23 rounds to a whole number (nearest
// even) and leaves its low byte, in two's complement, lowest.
__device__ __forceinline__ uint32_t act8_encode4(float a, float b, float c, float d, int e) {
  const float in[4] = {a, b, c, d};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __float_as_uint(__builtin_amdgcn_fmed3f(__builtin_ldexpf(in[i], 133 - e), -127.0f, 127.0f) + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0400), hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000C0C);
  return e == 255 ? 0u : lo | hi;
}

// max over the lanes of an aligned group of 4 (quad) or 32 lanes (half wave).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}
// (v_permlane16_swap_b32 of a value with itself leaves rows 0 0 2 2 and 1 1 3 3
// of 16 lanes, v_permlane32_swap_b32 halves 0 0 and 1 1.)
__device__ __forceinline__ uint32_t half_wave_max(uint32_t v) {
  v = quad_max(v);
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x141, 0xF, 0xF, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x140, 0xF, 0xF, true)));
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max(r[0], r[1]);
}
__device__ __forceinline__ uint32_t halves_max(uint32_t v) {  // of lanes l and l ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(r[0], r[1]);
}

}  // namespace quest
