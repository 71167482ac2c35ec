// Products of few rows ("tokens") by many, in 8-bit integers, straight from memory
// into the operand registers of the 16 x 16 x 64 instruction.
//
// Lane l of a fragment holds 16 bytes: row l % 16, codes 16 (l / 16) .. + 15 of
// 64.  The rows of the wide operand (weights) are its A side, 16 at a time; the
// tokens its B side, 16 a group.  Lane l then has token l % 16 and the wide rows
// 4 (l / 16) .. + 3 of a product.  Both operands' sums come from the same
// instruction with ones on the other side, in the same lanes.
//
// Wide codes are signed bytes, or 4-bit codes two in a byte as the quantiser packs
// them (u = c + 8, the even column in the low half).  The latter need three
// operations for eight of them, (d & 0x0F..) and (d >> 4) & 0x0F.., which give the
// even and the odd columns; the tokens' bytes are brought into that order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quest {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// 64 codes of 16 rows a fragment: one of signed bytes, two (even and odd columns
// of 128) of packed ones.
template <bool kPacked>
constexpr int kFewChunk = kPacked ? 128 : 64;
template <bool kPacked>
constexpr int kFewFrags = kPacked ? 2 : 1;

// 16 bytes at `off` of a window of memory: zeros past its end, kNoBytes always so.  With
// a branch around a load the compiler no longer knows how many are on their way, and
// waits for all of them before it uses one.
constexpr int kNoBytes = 0x7FFFFFF0;
typedef __amdgpu_buffer_rsrc_t few_rsrc;
__device__ __forceinline__ few_rsrc few_window(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), static_cast<short>(0), bytes, 0x00020000);
}
__device__ __forceinline__ v4i load_window(few_rsrc r, int off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

__device__ __forceinline__ v4i load_v4i(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

// A lane's 16 bytes of a wide row's chunk as fragments.
template <bool kPacked>
__device__ __forceinline__ void wide_frags(v4i w, v4i (&f)[kFewFrags<kPacked>]) {
  if constexpr (kPacked) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[0][d] = w[d] & 0x0F0F0F0F;
      f[1][d] = (w[d] >> 4) & 0x0F0F0F0F;
    }
  } else {
    f[0] = w;
  }
}

// Eight consecutive bytes' even and odd ones.
__device__ __forceinline__ int even_bytes(int lo, int hi) {
  return static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(hi), static_cast<uint32_t>(lo), 0x06040200u));
}
__device__ __forceinline__ int odd_bytes(int lo, int hi) {
  return static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(hi), static_cast<uint32_t>(lo), 0x07050301u));
}

// What a lane loads of a token's chunk: 16 bytes, or 32 for a packed wide operand.
template <bool kPacked>
struct TokenBytes {
  v4i v[kFewFrags<kPacked>];
};

template <bool kPacked>
__device__ __forceinline__ void token_frags(const TokenBytes<kPacked>& x, v4i (&f)[kFewFrags<kPacked>]) {
  if constexpr (kPacked) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int lo = x.v[d >> 1][2 * (d & 1)], hi = x.v[d >> 1][2 * (d & 1) + 1];
      f[0][d] = even_bytes(lo, hi);
      f[1][d] = odd_bytes(lo, hi);
    }
  } else {
    f[0] = x.v[0];
  }
}

__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v4i ones_i8() { return v4i{0x01010101, 0x01010101, 0x01010101, 0x01010101}; }

// Sums of P strips of 16 wide rows by T groups of 16 tokens.
template <bool kPacked, int P, int T>
struct FewSums {
  v4i acc[P][T] = {}, wide[P] = {}, token[T] = {};

  __device__ __forceinline__ void add(const v4i (&w)[P], const TokenBytes<kPacked> (&x)[T]) {
    constexpr int F = kFewFrags<kPacked>;
    v4i fw[P][F], fx[T][F];
#pragma unroll
    for (int p = 0; p < P; ++p) wide_frags<kPacked>(w[p], fw[p]);
#pragma unroll
    for (int t = 0; t < T; ++t) token_frags<kPacked>(x[t], fx[t]);
#pragma unroll
    for (int f = 0; f < F; ++f) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int t = 0; t < T; ++t) acc[p][t] = mfma_i8(fw[p][f], fx[t][f], acc[p][t]);
        wide[p] = mfma_i8(fw[p][f], ones_i8(), wide[p]);
      }
#pragma unroll
      for (int t = 0; t < T; ++t) token[t] = mfma_i8(ones_i8(), fx[t][f], token[t]);
    }
  }

  // The lane's four of sum (2 w + 1)(2 x + 1) without the constant few_constant
  // (kPacked: the stored u = w + 8).  Unsigned: the terms may wrap, their sum does not.
  __device__ __forceinline__ v4u total(int p, int t) const {
    return 4u * (v4u)acc[p][t] + 2u * (v4u)wide[p] + (kPacked ? -30u : 2u) * (v4u)token[t];
  }
};

// What every sum over k codes adds: k, or for u = w + 8, 2 w + 1 = 2 u - 15, -15 k.
template <bool kPacked>
__device__ __forceinline__ uint32_t few_constant(int k) {
  return static_cast<uint32_t>(kPacked ? -15 * k : k);
}

// A wave's walk over chunks first, first + stride, ... of `chunks`, kAhead of them on
// their way: begin() issues the first loads; run() uses each chunk and issues the load
// kAhead further on.  load(c, i) brings chunk c to place i (zeros for those behind the
// last), use(c, i) takes it from there.
template <int kAhead>
struct FewRing {
  int first, stride, chunks;

  template <typename Load>
  __device__ __forceinline__ void begin(Load load) const {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(first + i * stride, i);
  }
  template <typename Load, typename Use>
  __device__ __forceinline__ void run(Load load, Use use) const {
    for (int c = first; c < chunks; c += kAhead * stride) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int ci = c + i * stride;
        if (ci < chunks) use(ci, i);
        load(ci + kAhead * stride, i);
      }
    }
  }
};

}  // namespace quest
