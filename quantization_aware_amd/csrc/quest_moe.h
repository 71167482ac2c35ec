// What the kernels of quest_moe_fwd share: a token's choice of experts and the gated
// product's activation.
#pragma once

#include "quest_device.h"
#include "quest_launch.h"
#include "quest_sync.h"

namespace quest {

// A token's logits as they lie in memory, expert 64 i + lane in raw[i] (past the last:
// the last again).  Kept apart from their use, so that other loads can follow at once.
template <int S>
__device__ __forceinline__ void fetch_logits(const MoeLaunch& a, int t, int lane, uint32_t (&raw)[S]) {
  const int64_t row = static_cast<int64_t>(t) * a.experts;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int64_t at = row + min(64 * i + lane, a.experts - 1);
    if (a.logits_bf16)
      raw[i] = static_cast<const uint16_t*>(a.logits)[at];
    else
      raw[i] = static_cast<const uint32_t*>(a.logits)[at];
  }
}

template <int CTRL>
__device__ __forceinline__ int dpp_read_i(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, false);
}

// The largest of all lanes', the same in every lane.
__device__ __forceinline__ int wave_max(int x) {
  x = max(x, dpp_read_i<0xB1>(x));
  x = max(x, dpp_read_i<0x4E>(x));
  x = max(x, dpp_read_i<0x141>(x));
  x = max(x, dpp_read_i<0x140>(x));  // every lane of a row of 16 has the row's
  int r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readlane(x, 16 * i);
  return max(max(r[0], r[1]), max(r[2], r[3]));
}

// Logits as whole numbers of the same order (-0 as 0); kNone for an expert that is not
// taken: past the last, taken already, of logit -inf, and NaN.
constexpr int kNone = -0x7FFFFFFF - 1;
__device__ __forceinline__ int logit_key(float f) {
  const int i = __float_as_int(f + 0.0f);
  return f > -__builtin_inff() ? i ^ ((i >> 31) & 0x7FFFFFFF) : kNone;
}
__device__ __forceinline__ float logit_of(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF)); }

// A token's experts by rank, the largest logit first (of equal ones the lowest index), of
// which the first `ranks` are looked for.  Lane r holds the expert of rank r and (with
// `weights`, for ranks = top) its weight.  found: how many there are, or -1 for a token
// with a NaN or +infinity, whose output is NaN.  S: sets of 64 experts.
struct Choice {
  int found, expert;
  float weight;
};

template <int S>
__device__ __forceinline__ Choice choose(const MoeLaunch& a, int lane, const uint32_t (&raw)[S], int ranks,
                                         bool weights) {
  const int shift = a.logits_bf16 ? 16 : 0;
  int v[S], best = kNone;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const float f = __uint_as_float(raw[i] << shift);
    nan |= f != f;
    v[i] = 64 * i + lane < a.experts ? logit_key(f) : kNone;
    best = max(best, v[i]);
  }
  const int first = wave_max(best);
  const float largest = logit_of(first);
  Choice c{-1, 0, 0.0f};
  if (__builtin_amdgcn_ballot_w64(nan) != 0 || largest == __builtin_inff()) return c;
  float all = 0.0f;
  if (weights && a.over_all)
#pragma unroll
    for (int i = 0; i < S; ++i) all += v[i] == kNone ? 0.0f : expf(logit_of(v[i]) - largest);
  int chosen = kNone;
  for (c.found = 0; c.found < ranks; ++c.found) {
    best = v[0];
#pragma unroll
    for (int i = 1; i < S; ++i) best = max(best, v[i]);
    const int value = c.found == 0 ? first : wave_max(best);
    if (value == kNone) break;
    int e = 0;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      const uint64_t at = __builtin_amdgcn_ballot_w64(v[i] == value);
      if (at) e = 64 * i + __builtin_ctzll(at);
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (64 * i + lane == e) v[i] = kNone;
    if (lane == c.found) c.expert = e, chosen = value;
  }
  if (weights) {
    const float own = lane < c.found ? expf(logit_of(chosen) - largest) : 0.0f;
    c.weight = own / group_sum(a.over_all ? all : own, 6);
  }
  return c;
}

template <int kAct>
__device__ __forceinline__ float activation(float g) {
  if constexpr (kAct == 0) return g / (1.0f + expf(-g));
  return g * (0.5f * erfcf(g * -0.70710678f));
}

}  // namespace quest
