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

// Adds chunks first, first + stride, ... of `chunks` of signed byte codes to the sums:
// the lane's wide row at w, its token at x; four chunks' loads in flight.
__device__ __forceinline__ void few_run(FewSums<false, 1, 1>& s, const uint8_t* w, const uint8_t* x, int first,
                                        int stride, int chunks, int lane) {
  constexpr int kAhead = 4;
  w += 16 * (lane >> 4);
  x += 16 * (lane >> 4);
  v4i fw[kAhead][1];
  TokenBytes<false> fx[kAhead][1];
  auto load = [&](int c, int i) {
    if (c >= chunks) return;
    fw[i][0] = load_v4i(w + static_cast<int64_t>(c) * 64);
    fx[i][0].v[0] = load_v4i(x + static_cast<int64_t>(c) * 64);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(first + i * stride, i);
  for (int c = first; c < chunks; c += kAhead * stride) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int ci = c + i * stride;
      if (ci < chunks) {
        const v4i cw[1] = {fw[i][0]};
        const TokenBytes<false> cx[1] = {fx[i][0]};
        load(ci + kAhead * stride, i);
        s.add(cw, cx);
      }
    }
  }
}

}  // namespace quest
