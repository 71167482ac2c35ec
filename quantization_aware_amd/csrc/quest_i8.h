// What the quantiser to codes one a byte shares with the expert layer's kernel that
// quantises h itself: the same constants and order of sums, hence the same bits.
#pragma once

#include "quest_kernels.h"

namespace quest {

// Four values (in steps of Delta) to four signed bytes.
__device__ __forceinline__ uint32_t codes4(const float* v, float kk, float half) {
  int c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = static_cast<int>(__builtin_amdgcn_fmed3f(__builtin_floorf(v[j] * kk), -half, half - 1.0f));
  const uint32_t lo = __builtin_amdgcn_perm(static_cast<uint32_t>(c[1]), static_cast<uint32_t>(c[0]), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(static_cast<uint32_t>(c[3]), static_cast<uint32_t>(c[2]), 0x04000C0Cu);
  return lo | hi;
}

// The packed forward's constants, with the number of levels at run time.
inline FwdConsts i8_consts(int64_t cols, int log_block, int bits, double alpha, double trust) {
  const double n = double(1 << log_block), levels = double(1 << bits);
  FwdConsts k;
  k.alpha = static_cast<float>(alpha);
  k.kk = static_cast<float>((levels - 1.0) / (2.0 * alpha * std::sqrt(n)));
  k.thr = static_cast<float>(alpha * (1.0 + trust / (levels - 1.0)) * std::sqrt(n));
  k.inv_cols = static_cast<float>(1.0 / double(cols));
  k.chunks = 0;
  return k;
}

// The runs of a row that add up within a wave: as many lanes, as a power of two.
inline int i8_log_group(int runs) {
  const int group = runs & -runs;
  return log2_exact(group > 64 ? 64 : group);
}

}  // namespace quest
