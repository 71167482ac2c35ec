// Layer norm, forward and backward, and the form whose backward pass reads the
// normalised input from its 8-bit checkpoint (quest_act8.h).
//
// Forward, per row of C entries (all in fp32):
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps),
//   xhat = (x - mean) rstd,  y = xhat w + b.
// Backward, with a = dy w:
//   dx = rstd (a - sum a / C - xhat sum(a xhat) / C),
//   dw = sum_rows dy xhat,  db = sum_rows dy.
//
// One read of every input: a row's entries stay in the registers of the
// threads that share it (16 for up to 128 entries and 64 for up to 2048, so that
// its sums need no barrier; a workgroup for wider rows, and for those of 513 to 2048
// entries where there are few).  The first sum gives the mean within its rounding;
// the second pass over the registers sums x - near and its square, which gives
// the rest of the mean, where there is more of it than those differences' own
// roundings, and the variance about it, so a large common offset costs no digits.
// The parameter gradients: every workgroup of the backward kernel walks rows,
// keeps its columns' sums in registers and writes them once; a second kernel
// adds the workgroups' sums in a fixed order.  No atomics: the result depends
// on the sizes alone.
#include "quest_act8.h"

#include "quest_launch.h"

namespace quest {
namespace {

template <int kCtrl, int kRowMask>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRowMask, 0xF, false));
}
// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_or_zero<0xB1, 0xF>(v);   // lane ^ 1
  v += dpp_or_zero<0x4E, 0xF>(v);   // lane ^ 2
  v += dpp_or_zero<0x141, 0xF>(v);  // the other quad of 8
  v += dpp_or_zero<0x140, 0xF>(v);  // the other 8 of 16
  v += dpp_or_zero<0x142, 0xA>(v);  // rows 1 and 3 add the row before
  v += dpp_or_zero<0x143, 0xC>(v);  // rows 2 and 3 add row 1
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over the 16 lanes of a row of the wave, in each of them.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_or_zero<0xB1, 0xF>(v);
  v += dpp_or_zero<0x4E, 0xF>(v);
  v += dpp_or_zero<0x141, 0xF>(v);
  return v + dpp_or_zero<0x140, 0xF>(v);
}

// Sums of two values over the TPR threads of a row; `part` holds 2 * TPR / 64
// floats and is free again after the next call's first barrier.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* part) {
  if constexpr (TPR == 16) {
    a = row16_sum(a);
    b = row16_sum(b);
    return;
  }
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      part[2 * wave] = a;
      part[2 * wave + 1] = b;
    }
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      a += part[2 * w];
      b += part[2 * w + 1];
    }
  }
}

// Group j of thread t of a row's TPR threads: 8 neighbouring columns from here.
template <int TPR>
__device__ __forceinline__ int column(int t, int j) {
  return 8 * (t + TPR * j);
}

// A row, or a parameter vector.  kVec (cols a multiple of 8): as a buffer
// resource, whose accesses past the end read zero and write nothing, so that no
// load or store stands behind a branch.  Otherwise by address, in groups whose
// last ends with the row (quest_act8.h; 16384 x 2047 backward 43.3 us, 40.1 for 2048
// columns, 82 with a branch for the last entries); rows of 16 threads, which may
// be narrower than a group, entry by entry at their end.
struct Row {
  __amdgpu_buffer_rsrc_t rsrc;
  uintptr_t at;
  int cols;
};
template <typename T>
__device__ __forceinline__ Row row_at(const void* p, int64_t row, int cols) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(row * cols) * sizeof(T);
  return {__builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), static_cast<short>(0),
                                            cols * static_cast<int>(sizeof(T)), 0x00020000),
          at, cols};
}

// How group j of thread t stands to the row: kClamped, by Group.
template <int TPR, bool kVec>
constexpr bool kClamped = !kVec && TPR >= 64;
template <int TPR, bool kVec>
__device__ __forceinline__ bool inside(int t, int j, int i, int cols) {
  const int c = column<TPR>(t, j);
  if constexpr (kClamped<TPR, kVec>) return Group(c, cols).own(i);
  return c + i < cols;
}

// Entries that are not the group's own as zeros.  Of a row's waves only the last and
// those past it have any: the others pass by on a scalar branch (8000 x 5631 forward
// 46 us, 57 with a select at every entry, on one input; 52 where the inputs change).
template <int TPR, bool kVec>
__device__ __forceinline__ void own_only(int t, int j, int cols, float (&v)[8]) {
  if constexpr (TPR >= 64) {
    if (column<TPR>(__builtin_amdgcn_readfirstlane(t), j) + 8 * 64 <= cols) return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = inside<TPR, kVec>(t, j, i, cols) ? v[i] : 0.0f;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 8 entries of a row of T in group j of thread t; only those `inside` count.
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void fetch(const Row& r, int t, int j, float (&v)[8]) {
  const int c = column<TPR>(t, j);
  if constexpr (kClamped<TPR, kVec>) {
    load8_at(reinterpret_cast<const T*>(r.at) + Group(c, r.cols).at, v);
  } else if constexpr (!kVec) {
    load8_tail(reinterpret_cast<const T*>(r.at) + c, r.cols - c, v);
  } else if constexpr (sizeof(T) == 2) {
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, c * 2, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, c * 4, 0, 0);
    const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, c * 4 + 16, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(lo[i]);
      v[4 + i] = __uint_as_float(hi[i]);
    }
  }
}
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void put(const Row& r, int t, int j, const float (&v)[8]) {
  const int c = column<TPR>(t, j);
  if constexpr (kClamped<TPR, kVec>) {
    const Group g(c, r.cols);
    store8_own(reinterpret_cast<T*>(r.at) + g.at, g, v);
  } else if constexpr (!kVec) {
    store8_tail(reinterpret_cast<T*>(r.at) + c, r.cols - c, v);
  } else if constexpr (sizeof(T) == 2) {
    const u32x4 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    __builtin_amdgcn_raw_buffer_store_b128(w, r.rsrc, c * 2, 0, 0);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 w = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                       __float_as_uint(v[4 * h + 3])};
      __builtin_amdgcn_raw_buffer_store_b128(w, r.rsrc, c * 4 + 16 * h, 0, 0);
    }
  }
}
// The 8-bit checkpoint of such a group: a block is four neighbouring threads.  What
// lies past the row in its last block has no part in the block's exponent (without
// kVec: v is zero there).
template <int TPR, bool kVec>
__device__ __forceinline__ void put_act8(const Row& codes, const Row& scale, int t, int j, const float (&v)[8]) {
  const int c = column<TPR>(t, j);
  const uint32_t mag = !kVec || c < codes.cols ? act8_mag8(v) : 0;
  const int e = static_cast<int>(quad_max(mag) >> 23);
  const uint2 w = act8_encode8(v, e);
  if constexpr (kVec) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{w.x, w.y}, codes.rsrc, c, 0, 0);
  } else if constexpr (kClamped<TPR, kVec>) {
    const Group g(c, codes.cols);
    store_codes8_own(reinterpret_cast<int8_t*>(codes.at) + g.at, g, w);
  } else {
    store_codes8_tail(reinterpret_cast<int8_t*>(codes.at) + c, codes.cols - c, w);
  }
  if ((t & 3) == 0 && c < codes.cols) reinterpret_cast<uint8_t*>(scale.at)[c >> 5] = static_cast<uint8_t>(e);
}
// Parameters of either type.
template <int TPR, bool kVec>
__device__ __forceinline__ void fetch_param(const void* p, bool bf16, int cols, int t, int j, float (&v)[8]) {
  if (bf16)
    fetch<uint16_t, TPR, kVec>(row_at<uint16_t>(p, 0, cols), t, j, v);
  else
    fetch<float, TPR, kVec>(row_at<float>(p, 0, cols), t, j, v);
}

template <int TPR>
constexpr int kBlockThreads = TPR <= 64 ? 256 : TPR;

// Which of a workgroup's rows the thread is at: uniform over a wave, except where rows
// have 16 threads (narrow ones, which go by address: kVec is false for them).
template <int TPR>
__device__ __forceinline__ int sub_row() {
  const int sub = threadIdx.x / TPR;
  return TPR >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub;
}

template <typename T, int TPR, int NC, bool kVec>
__global__ void __launch_bounds__(kBlockThreads<TPR>) quest_norm_fwd_kernel(const NormFwdLaunch a) {
  constexpr int kRows = kBlockThreads<TPR> / TPR;
  __shared__ float part[TPR > 64 ? 2 * TPR / 64 : 1];
  static_assert(TPR >= 64 || !kVec, "a wave's rows share a buffer resource");
  const int t = threadIdx.x % TPR, sub = sub_row<TPR>();
  const int cols = a.cols;
  const float count = static_cast<float>(cols);
  const int blocks = (cols + kAct8Block - 1) / kAct8Block;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  // The parameters in registers across the rows that a workgroup walks (16384 x
  // 2048 bf16 with fp32 parameters: 27.4 us, 31.9 when every row reads them again
  // from the caches); not beside the entries of the widest rows, whose threads
  // have 128 registers.
  constexpr bool kHold = TPR * NC < 4096;
  float w[kHold ? NC : 1][8], b[kHold ? NC : 1][8];
  auto params = [&](int j, float (&wj)[8], float (&bj)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) wj[i] = 1.0f, bj[i] = 0.0f;
    if (a.weight) fetch_param<TPR, kVec>(a.weight, a.param_bf16, cols, t, j, wj);
    if (a.bias) fetch_param<TPR, kVec>(a.bias, a.param_bf16, cols, t, j, bj);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < NC; ++j) params(j, w[j], b[j]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < a.rows; row += stride) {
    const Row x = row_at<T>(a.x, row, cols);
    float v[NC][8];
    float sum = 0.0f, none = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) fetch<T, TPR, kVec>(x, t, j, v[j]);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if constexpr (kClamped<TPR, kVec>) own_only<TPR, kVec>(t, j, cols, v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[j][i];
    }
    row_sum2<TPR>(sum, none, part);
    const float near = sum / count;  // the mean, within the rounding of the sum
    float sq = 0.0f, off = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const bool in = !kVec || column<TPR>(t, j) < cols;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = in ? v[j][i] - near : 0.0f;
      if constexpr (!kVec) own_only<TPR, kVec>(t, j, cols, v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        off += v[j][i];
        sq = fmaf(v[j][i], v[j][i], sq);
      }
    }
    row_sum2<TPR>(sq, off, part);
    // What `near` missed, unless no more than the roundings of x - near come to (at most
    // 2^-24 |x - near| each, and all one way in bf16, whose entries share their low bits):
    // those would be the larger error where the offset is small (16384 x 2048 bf16: mean
    // within 0.03 instead of 0.30 times 2^-24 of the spread, rms).
    off /= count;
    if (fabsf(off) < 0x1p-24f * __builtin_amdgcn_sqrtf(sq / count)) off = 0.0f;  // (an infinity stays)
    const float mean = near + off;
    const float var = sq / count - off * off;
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);  // (NaN stays)
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    const Row y = row_at<T>(a.y, row, cols);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int held = kHold ? j : 0;
      if constexpr (!kHold) params(j, w[0], b[0]);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = (v[j][i] - off) * rstd;
        o[i] = fmaf(v[j][i], w[held][i], b[held][i]);
      }
      put<T, TPR, kVec>(y, t, j, o);
      if (a.codes) {
        if constexpr (!kVec) own_only<TPR, kVec>(t, j, cols, v[j]);
        put_act8<TPR, kVec>(row_at<int8_t>(a.codes, row, cols), row_at<uint8_t>(a.scale, row, blocks), t, j, v[j]);
      }
    }
  }
}

// Where a row's xhat comes from: x, mean and rstd, or the 8-bit checkpoint.
struct XhatRow {
  Row x, scale;
  float mean, rstd;
};
// 8 entries of xhat; only those `inside` are meant.
template <typename T, int TPR, bool kVec, bool kAct8>
__device__ __forceinline__ void fetch_xhat(const XhatRow& r, int t, int j, float (&v)[8]) {
  if constexpr (!kAct8) {
    fetch<T, TPR, kVec>(r.x, t, j, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] - r.mean) * r.rstd;
  } else {
    const int c = column<TPR>(t, j);
    uint2 w;
    int e = 0;
    if constexpr (kVec) {
      const u32x2 q = __builtin_amdgcn_raw_buffer_load_b64(r.x.rsrc, c, 0, 0);
      w = make_uint2(q[0], q[1]);
      e = __builtin_amdgcn_raw_buffer_load_b8(r.scale.rsrc, c >> 5, 0, 0);
    } else if constexpr (kClamped<TPR, kVec>) {
      w = load_codes8_at(reinterpret_cast<const int8_t*>(r.x.at) + Group(c, r.x.cols).at);
      e = reinterpret_cast<const uint8_t*>(r.scale.at)[min(c, r.x.cols - 1) >> 5];
    } else {
      w = load_codes8_tail(reinterpret_cast<const int8_t*>(r.x.at) + c, r.x.cols - c);
      if (c < r.x.cols) e = reinterpret_cast<const uint8_t*>(r.scale.at)[c >> 5];
    }
    act8_decode8(w, e, v);
  }
}
template <typename T, bool kAct8>
__device__ __forceinline__ XhatRow xhat_row(const NormBwdLaunch& a, int64_t row) {
  XhatRow r;
  r.rstd = a.rstd[row];
  if constexpr (kAct8) {
    r.mean = 0.0f;
    r.x = row_at<int8_t>(a.codes, row, a.cols);
    r.scale = row_at<uint8_t>(a.scale, row, (a.cols + kAct8Block - 1) / kAct8Block);
  } else {
    r.mean = a.mean[row];
    r.x = row_at<T>(a.x, row, a.cols);
  }
  return r;
}

// kParams: with the column sums.  Without them it is the dx of the widest rows
// (and of calls that ask for dx alone), whose sums have a kernel of their own.
template <typename T, int TPR, int NC, bool kVec, bool kAct8, bool kParams>
__global__ void __launch_bounds__(kBlockThreads<TPR>) quest_norm_bwd_kernel(const NormBwdLaunch a) {
  constexpr int kRows = kBlockThreads<TPR> / TPR;
  // Rows of 1024 threads, which have 128 registers each: the sums of dy xhat in LDS,
  // each thread's its own, and the weight read again from the caches for every row
  // (2048 x 16384 bf16: 54.8 us, 67.2 with 512 threads and all in registers).
  constexpr bool kWide = kParams && TPR == 1024;
  constexpr bool kSkip = kParams && kClamped<TPR, kVec>;
  constexpr int kSums = kWide ? 8 * NC * TPR : kParams && kRows > 1 ? 2 * 8 * NC * TPR : 1;
  constexpr int kHeld = kParams ? NC : 1, kHeldW = kParams && !kWide ? NC : 1;
  __shared__ float part[TPR > 64 ? 2 * TPR / 64 : 1];
  __shared__ float sums[kSums];  // [2][8 NC TPR], the rows of a workgroup joined one after the other
  static_assert(TPR >= 64 || !kVec, "a wave's rows share a buffer resource");
  const int t = threadIdx.x % TPR, sub = sub_row<TPR>();
  const int cols = a.cols;
  const float inv = 1.0f / static_cast<float>(cols);
  float dw[kWide ? 1 : kHeld][8], db[kHeld][8], w[kHeldW][8];
  auto weight = [&](int j, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    if (a.weight) fetch_param<TPR, kVec>(a.weight, a.param_bf16, cols, t, j, v);
    if constexpr (kSkip) own_only<TPR, kVec>(t, j, cols, v);
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      db[j][i] = 0.0f;
      if constexpr (kWide)
        sums[(8 * j + i) * TPR + t] = 0.0f;
      else
        dw[j][i] = 0.0f;
    }
    if constexpr (kParams && !kWide) weight(j, w[j]);
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < a.rows; row += stride) {
    const Row dy = row_at<T>(a.dy, row, cols);
    const XhatRow xr = xhat_row<T, kAct8>(a, row);
    float g[NC][8], xh[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      fetch<T, TPR, kVec>(dy, t, j, g[j]);
      fetch_xhat<T, TPR, kVec, kAct8>(xr, t, j, xh[j]);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int held = kHeldW > 1 ? j : 0;
      if constexpr (!kParams || kWide) weight(j, w[0]);
      // Entries that are not the group's own count as zero: by own_only where that is the
      // faster (16384 x 2047 from the 8-bit copy 40.7 us, 46.6 with a select at each; 2048
      // columns 36.5 with selects and 48 without; dx alone of 8000 x 5631 69 and 76).
      // Only a clamped group's gradients and weights reach past the row.
      if constexpr (kSkip) {
        own_only<TPR, kVec>(t, j, cols, g[j]);
        own_only<TPR, kVec>(t, j, cols, xh[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = kSkip || inside<TPR, kVec>(t, j, i, cols);
        const float d = !kClamped<TPR, kVec> || in ? g[j][i] : 0.0f, x = in ? xh[j][i] : 0.0f;
        if constexpr (kParams) {
          if constexpr (kWide)
            sums[(8 * j + i) * TPR + t] += d * x;
          else
            dw[j][i] = fmaf(d, x, dw[j][i]);
          db[j][i] += d;
        }
        const float y = d * w[held][i];
        xh[j][i] = x;
        g[j][i] = y;
        s1 += in ? y : 0.0f;
        s2 = fmaf(y, x, s2);
      }
    }
    row_sum2<TPR>(s1, s2, part);
    s1 *= inv;
    s2 *= inv;
    if (a.dx) {
      const Row dx = row_at<T>(a.dx, row, cols);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (g[j][i] - s1 - xh[j][i] * s2) * xr.rstd;
        put<T, TPR, kVec>(dx, t, j, o);
      }
    }
  }
  if constexpr (kParams) {
    if constexpr (kRows > 1) {
      for (int r = 0; r < kRows; ++r) {
        if (sub == r) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int s = (8 * j + i) * TPR + t;
              sums[s] = r == 0 ? dw[j][i] : sums[s] + dw[j][i];
              sums[8 * NC * TPR + s] = r == 0 ? db[j][i] : sums[8 * NC * TPR + s] + db[j][i];
            }
        }
        __syncthreads();
      }
      if (sub != 0) return;
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = (8 * j + i) * TPR + t;
          dw[j][i] = sums[s];
          db[j][i] = sums[8 * NC * TPR + s];
        }
    }
    const Row wdw = row_at<float>(a.workspace, 2 * static_cast<int64_t>(blockIdx.x), cols);
    const Row wdb = row_at<float>(a.workspace, 2 * static_cast<int64_t>(blockIdx.x) + 1, cols);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float sw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (kWide)
          sw[i] = sums[(8 * j + i) * TPR + t];
        else
          sw[i] = dw[j][i];
      }
      put<float, TPR, kVec>(wdw, t, j, sw);
      put<float, TPR, kVec>(wdb, t, j, db[j]);
    }
  }
}

// The column sums alone: workgroup (x, y) takes columns 2048 x ... and rows y,
// y + gridDim.y, ...  For rows too wide for quest_norm_bwd_kernel to hold
// their sums beside their entries, at the price of a second read.
template <typename T, bool kVec, bool kAct8>
__global__ void __launch_bounds__(256) quest_norm_colsum_kernel(const NormBwdLaunch a) {
  const int t = threadIdx.x, j = blockIdx.x;
  const int cols = a.cols;
  float dw[8] = {}, db[8] = {};
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float g[8], xh[8];
    fetch<T, 256, kVec>(row_at<T>(a.dy, row, cols), t, j, g);
    fetch_xhat<T, 256, kVec, kAct8>(xhat_row<T, kAct8>(a, row), t, j, xh);
    // (what is not the group's own is not stored)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
    }
  }
  put<float, 256, kVec>(row_at<float>(a.workspace, 2 * static_cast<int64_t>(blockIdx.y), cols), t, j, dw);
  put<float, 256, kVec>(row_at<float>(a.workspace, 2 * static_cast<int64_t>(blockIdx.y) + 1, cols), t, j, db);
}

// The workgroups' column sums added in a fixed order: slice s of a workgroup
// adds every 16th of them from s for its 32 columns, 16 loads at a time (the last few
// 8 at a time), then the slices are added.  Few columns a workgroup and many loads in
// flight: the sums of 512 workgroups over 2048 columns take 4.2 us (31 us with 4 slices
// of 64 columns and one load at a time, all of it latency).
constexpr int kSlices = 16, kSumCols = 32, kLoads = 16;
template <typename P>
__global__ void __launch_bounds__(kSlices* kSumCols)
    quest_norm_params_kernel(const float* __restrict__ ws, int groups, int cols, P* __restrict__ dw,
                             P* __restrict__ db) {
  __shared__ float part[kSlices][kSumCols];
  const int lane = threadIdx.x % kSumCols, s = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + lane;  // column of [dw | db]
  float v = 0.0f;
  if (c < 2 * cols) {
    const float* p = ws + c;
    const int64_t pitch = 2 * static_cast<int64_t>(cols);
    int g = s;
    for (; g + (kLoads - 1) * kSlices < groups; g += kLoads * kSlices) {
      float x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = p[(g + i * kSlices) * pitch];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v += x[i];
    }
    for (; g < groups; g += 8 * kSlices) {  // the rest: 8 loads together as well
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[min(g + i * kSlices, groups - 1) * pitch];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += g + i * kSlices < groups ? x[i] : 0.0f;
    }
  }
  part[s][lane] = v;
  __syncthreads();
  if (s != 0 || c >= 2 * cols) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) v += part[i][lane];
  if (c < cols) {
    if (dw) dw[c] = from_f32<P>(v);
  } else if (db) {
    db[c - cols] = from_f32<P>(v);
  }
}

// Workgroups of the forward and of dx alone, which walk the rows beyond.  The
// stores of y are ordinary ones: non-temporal they make the norm alone faster
// (23.1 us), but not with the quantiser that reads y next (49.0 us both, 47.6 so).
constexpr int kMaxFwdBlocks = 2048;
// Rows of 513 to 2048 columns that have a workgroup's 256 threads and not a wave's 64,
// whose chain of loads and sums is what a call of few rows takes.  Us with 256 and with 64
// (the backward's with the sums added): forward, bf16, 1 x 2048 2.4 and 3.8, 768 x 2048 3.8
// and 4.0, 1500 x 2048 5.3 and 5.0; fp32 8192 x 2048 22.4 and 23.2, 16384 x 1111 27.9 and
// 27.6; up to 1024 columns 256 x 600 3.1 and 3.0.  Backward, 1500 x 2048 bf16 12.2 and 12.8,
// fp32 13.4 and 14.7; 4096 x 2048 16.0 and 16.6, 18.1 and 20.4; 6000 x 2048 19.4 and 18.2,
// 22.7 and 24.8; 256 x 600 5.6 and 6.2, 400 x 600 7.0 and 6.3.
constexpr bool few_fwd(int64_t rows, int cols, bool f32) {
  return cols > 1024 ? rows <= (f32 ? 8192 : 768) : rows <= 256;
}
constexpr bool few_bwd(int64_t rows, int64_t cols) { return cols > 1024 ? rows <= 4096 : rows <= 256; }
// Rows of 16 threads: 111661 x 19 forward 13.5 us, 49.5 with a wave a row; backward 23.7
// and 49.2.
constexpr int kNarrowCols = 128;
// Widest rows whose backward holds entries and column sums (1024 x 32768 bf16: 89 us
// with the sums in a kernel of their own, 133 in one that spills).
constexpr int kMaxHeldCols = 16384;

template <typename T, int TPR, int NC, bool kVec>
hipError_t fwd(const NormFwdLaunch& a) {
  constexpr int kRows = kBlockThreads<TPR> / TPR;
  const int64_t n = (a.rows + kRows - 1) / kRows;
  hipLaunchKernelGGL((quest_norm_fwd_kernel<T, TPR, NC, kVec>),
                     dim3(static_cast<uint32_t>(n < kMaxFwdBlocks ? n : kMaxFwdBlocks)), dim3(kBlockThreads<TPR>), 0,
                     a.stream, a);
  return hipGetLastError();
}

template <typename T, bool kVec>
hipError_t fwd_width(const NormFwdLaunch& a) {
  if (a.cols <= kNarrowCols) return fwd<T, 16, 1, false>(a);
  if (a.cols <= 512) return fwd<T, 64, 1, kVec>(a);
  if (a.cols <= 2048 && few_fwd(a.rows, a.cols, sizeof(T) == 4)) return fwd<T, 256, 1, kVec>(a);
  if (a.cols <= 1024) return fwd<T, 64, 2, kVec>(a);
  if (a.cols <= 2048) return fwd<T, 64, 4, kVec>(a);
  if (a.cols <= 4096) return fwd<T, 256, 2, kVec>(a);
  if (a.cols <= 8192) return fwd<T, 256, 4, kVec>(a);
  if (a.cols <= 16384) return fwd<T, 1024, 2, kVec>(a);
  return fwd<T, 1024, 4, kVec>(a);
}

template <typename T, int TPR, int NC, bool kVec, bool kParams>
hipError_t bwd(const NormBwdLaunch& a, int groups) {
  if (a.codes)
    hipLaunchKernelGGL((quest_norm_bwd_kernel<T, TPR, NC, kVec, true, kParams>), dim3(groups),
                       dim3(kBlockThreads<TPR>), 0, a.stream, a);
  else
    hipLaunchKernelGGL((quest_norm_bwd_kernel<T, TPR, NC, kVec, false, kParams>), dim3(groups),
                       dim3(kBlockThreads<TPR>), 0, a.stream, a);
  return hipGetLastError();
}

template <typename T, bool kVec>
hipError_t bwd_width(const NormBwdLaunch& a, int groups) {
  if (a.workspace && a.cols > kMaxHeldCols) {
    const dim3 grid((a.cols + 2047) / 2048, groups);
    if (a.codes)
      hipLaunchKernelGGL((quest_norm_colsum_kernel<T, kVec, true>), grid, dim3(256), 0, a.stream, a);
    else
      hipLaunchKernelGGL((quest_norm_colsum_kernel<T, kVec, false>), grid, dim3(256), 0, a.stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dx) return e;
  } else if (a.workspace) {
    if (a.cols <= kNarrowCols) return bwd<T, 16, 1, false, true>(a, groups);
    if (a.cols <= 512) return bwd<T, 64, 1, kVec, true>(a, groups);
    if (a.cols <= 2048 && few_bwd(a.rows, a.cols)) return bwd<T, 256, 1, kVec, true>(a, groups);
    if (a.cols <= 1024) return bwd<T, 64, 2, kVec, true>(a, groups);
    if (a.cols <= 2048) return bwd<T, 64, 4, kVec, true>(a, groups);
    if (a.cols <= 4096) return bwd<T, 256, 2, kVec, true>(a, groups);
    if (a.cols <= 8192) return bwd<T, 256, 4, kVec, true>(a, groups);
    return bwd<T, 1024, 2, kVec, true>(a, groups);
  }
  // dx alone: rows in workgroups of their own, as the forward
  const int64_t per = a.cols <= kNarrowCols ? 16 : a.cols <= 2048 ? 4 : 1, n = (a.rows + per - 1) / per;
  groups = static_cast<int>(n < kMaxFwdBlocks ? n : kMaxFwdBlocks);
  if (a.cols <= kNarrowCols) return bwd<T, 16, 1, false, false>(a, groups);
  if (a.cols <= 512) return bwd<T, 64, 1, kVec, false>(a, groups);
  if (a.cols <= 2048) return bwd<T, 64, 4, kVec, false>(a, groups);
  if (a.cols <= 8192) return bwd<T, 256, 4, kVec, false>(a, groups);
  if (a.cols <= 16384) return bwd<T, 1024, 2, kVec, false>(a, groups);
  return bwd<T, 1024, 4, kVec, false>(a, groups);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdLaunch& a, bool x_bf16) {
  const bool vec = a.cols % 8 == 0;
  if (x_bf16) return vec ? fwd_width<uint16_t, true>(a) : fwd_width<uint16_t, false>(a);
  return vec ? fwd_width<float, true>(a) : fwd_width<float, false>(a);
}

int norm_bwd_groups(int64_t rows, int64_t cols) {
  // rows a workgroup holds at a time
  const int64_t per = cols <= kNarrowCols ? 16 : cols <= 512 || (cols <= 2048 && !few_bwd(rows, cols)) ? 4 : 1;
  // Workgroups: few enough that adding their sums is short, until the rows fill the chip
  // (1000 x 1111 fp32 in 250 and 256 x 8192 bf16 in 128: 9.6 and 13.0 us both kernels, 10.5
  // and 15.7 with up to 512; 4096 x 1024 bf16 in 256 10.3, 13.6 with 1024); then as many as
  // fit it by their registers, or as their sums are soon added.
  const int64_t n = (rows + per - 1) / per;
  const int64_t fit = cols <= kNarrowCols ? 1024 : cols <= 512 ? 2048 : cols <= 1024 ? 1024 : cols <= 8192 ? 512 : 256;
  const int64_t most = n <= 256 ? 128 : n <= 2048 ? 256 : fit;
  if (n == 0) return 0;
  // (and no more of them than the busiest one's share of the rows needs)
  const int64_t turns = (n + most - 1) / most;
  return static_cast<int>((n + turns - 1) / turns);
}

hipError_t launch_norm_bwd(const NormBwdLaunch& a, bool bf16) {
  const int groups = norm_bwd_groups(a.rows, a.cols);
  if (groups > 0) {
    const bool vec = a.cols % 8 == 0;
    const hipError_t e = bf16 ? (vec ? bwd_width<uint16_t, true>(a, groups) : bwd_width<uint16_t, false>(a, groups))
                              : (vec ? bwd_width<float, true>(a, groups) : bwd_width<float, false>(a, groups));
    if (e != hipSuccess) return e;
  }
  if (a.dweight || a.dbias) {
    const dim3 grid((2 * a.cols + kSumCols - 1) / kSumCols), block(kSlices * kSumCols);
    if (a.param_bf16)
      hipLaunchKernelGGL(quest_norm_params_kernel<uint16_t>, grid, block, 0, a.stream, a.workspace, groups,
                         a.cols, static_cast<uint16_t*>(a.dweight), static_cast<uint16_t*>(a.dbias));
    else
      hipLaunchKernelGGL(quest_norm_params_kernel<float>, grid, block, 0, a.stream, a.workspace, groups, a.cols,
                         static_cast<float*>(a.dweight), static_cast<float*>(a.dbias));
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace quest
