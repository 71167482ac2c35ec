// Activation checkpoints in 8 bits: saved (quest_act8_save) and read back
// (quest_act8_load).  The format is in quest_act8.h.
//
// Both are one pass over memory with a few operations an entry: bound by HBM.
// Rows of whole blocks (cols a multiple of 32) are one stretch of memory, in
// which entries 8 t .. 8 t + 7 belong to thread t: 16-byte accesses of bf16,
// 8-byte accesses of codes, and a block is four neighbouring lanes, whose
// maximum is two DPP steps.  Other widths keep those accesses at unaligned
// addresses, four lanes a block, a row's last group ending with the row (Group in
// quest_act8.h; rows narrower than 8 go entry by entry); a workgroup takes a run
// of consecutive blocks of the tensor, whatever rows they are of, so narrow rows
// fill the waves as well as wide ones.  (16384 x 5631 bf16 is saved in 54.4 us and
// read in 53.7, with a branch for the last entries in 75.5 and 62.5; beside 5632
// columns in one run 59.1 and 52.7 against 54.3 and 49.1.)
#include "quest_act8.h"

#include "quest_launch.h"

namespace quest {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // groups of 8 entries a thread handles in one pass, their loads together

// Block number `first` + i of the tensor as (row, block of the row), for a
// workgroup's first block (a 64-bit division, once and uniform) and small i.
struct BlockRun {
  int64_t row;
  uint32_t rem, blocks;
  __device__ __forceinline__ BlockRun(int64_t first, int cols)
      : blocks(static_cast<uint32_t>(cols + kAct8Block - 1) / kAct8Block) {
    row = first / blocks;
    rem = static_cast<uint32_t>(first - row * blocks);
  }
  __device__ __forceinline__ void at(uint32_t i, int64_t& r, int& b) const {
    const uint32_t t = rem + i, q = t / blocks;
    r = row + q;
    b = static_cast<int>(t - q * blocks);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quest_act8_save_flat_kernel(const T* __restrict__ x, int64_t groups, int8_t* __restrict__ codes,
                                uint8_t* __restrict__ scale) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  float v[kUnroll][8];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t g = base + u * kThreads;
    if (g < groups) load8(x + 8 * g, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t g = base + u * kThreads;
    if (g >= groups) break;  // groups is a multiple of 4: a block's lanes stay together
    const int e = static_cast<int>(quad_max(act8_mag8(v[u])) >> 23);
    *reinterpret_cast<uint2*>(codes + 8 * g) = act8_encode8(v[u], e);
    if ((g & 3) == 0) scale[g >> 2] = static_cast<uint8_t>(e);
  }
}

constexpr int kRun = kThreads / 4;  // blocks at a time

// kGroups: rows of 8 columns and more.
template <typename T, bool kGroups>
__global__ void __launch_bounds__(kThreads)
    quest_act8_save_blocks_kernel(const T* __restrict__ x, int64_t total, int cols, int8_t* __restrict__ codes,
                                  uint8_t* __restrict__ scale) {
  const int l = threadIdx.x % 4, sub = threadIdx.x / 4;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kRun * kUnroll); first < total;
       first += static_cast<int64_t>(gridDim.x) * (kRun * kUnroll)) {
    const BlockRun run(first, cols);
    const int last = static_cast<int>(min(total - 1 - first, static_cast<int64_t>(kRun * kUnroll - 1)));
    float v[kUnroll][8];
    int64_t at[kUnroll];
    int col[kUnroll];  // of the row; past it behind the tensor's last block
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int64_t r;
      int b;
      run.at(min(u * kRun + sub, last), r, b);
      const int c = b * kAct8Block + 8 * l;
      col[u] = u * kRun + sub <= last ? c : cols + 8;
      if constexpr (kGroups) {
        const Group g(col[u], cols);
        at[u] = r * cols + g.at;
        load8_at(x + at[u], v[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = g.own(i) ? v[u][i] : 0.0f;
      } else {
        at[u] = r * cols + c;
        load8_tail(x + at[u], cols - col[u], v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = static_cast<int>(quad_max(act8_mag8(v[u])) >> 23);
      if constexpr (kGroups)
        store_codes8_own(codes + at[u], Group(col[u], cols), act8_encode8(v[u], e));
      else
        store_codes8_tail(codes + at[u], cols - col[u], act8_encode8(v[u], e));
      if (l == 0 && col[u] < cols) scale[first + u * kRun + sub] = static_cast<uint8_t>(e);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quest_act8_load_flat_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scale, int64_t groups,
                                T* __restrict__ out) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint2 w[kUnroll];
  int e[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t g = base + u * kThreads;
    if (g < groups) {
      w[u] = *reinterpret_cast<const uint2*>(codes + 8 * g);
      e[u] = scale[g >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t g = base + u * kThreads;
    if (g >= groups) break;
    float v[8];
    act8_decode8(w[u], e[u], v);
    store8(out + 8 * g, v);
  }
}

template <typename T, bool kGroups>
__global__ void __launch_bounds__(kThreads)
    quest_act8_load_blocks_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scale, int64_t total,
                                  int cols, T* __restrict__ out) {
  const int l = threadIdx.x % 4, sub = threadIdx.x / 4;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kRun * kUnroll); first < total;
       first += static_cast<int64_t>(gridDim.x) * (kRun * kUnroll)) {
    const BlockRun run(first, cols);
    const int last = static_cast<int>(min(total - 1 - first, static_cast<int64_t>(kRun * kUnroll - 1)));
    uint2 w[kUnroll];
    int e[kUnroll], col[kUnroll];
    int64_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int64_t r;
      int b;
      const int i = min(u * kRun + sub, last);
      run.at(i, r, b);
      const int c = b * kAct8Block + 8 * l;
      col[u] = u * kRun + sub <= last ? c : cols + 8;
      e[u] = scale[first + i];
      if constexpr (kGroups) {
        at[u] = r * cols + Group(col[u], cols).at;
        w[u] = load_codes8_at(codes + at[u]);
      } else {
        at[u] = r * cols + c;
        w[u] = load_codes8_tail(codes + at[u], cols - col[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[8];
      act8_decode8(w[u], e[u], v);
      if constexpr (kGroups)
        store8_own(out + at[u], Group(col[u], cols), v);
      else
        store8_tail(out + at[u], cols - col[u], v);
    }
  }
}

// Workgroups of the block kernels, at most 2^20 (they walk the blocks beyond).
uint32_t block_grid(int64_t total) {
  const int64_t per = kRun * kUnroll, n = (total + per - 1) / per;
  return static_cast<uint32_t>(n < (1 << 20) ? n : (1 << 20));
}

template <typename T>
hipError_t save(const T* x, int64_t rows, int cols, int8_t* codes, uint8_t* scale, hipStream_t stream) {
  const int64_t total = rows * ((cols + kAct8Block - 1) / kAct8Block);
  if (cols % kAct8Block == 0) {
    const int64_t groups = rows * cols / 8, per = kThreads * kUnroll;
    hipLaunchKernelGGL(quest_act8_save_flat_kernel<T>, dim3(static_cast<uint32_t>((groups + per - 1) / per)),
                       dim3(kThreads), 0, stream, x, groups, codes, scale);
  } else if (cols >= 8) {
    hipLaunchKernelGGL((quest_act8_save_blocks_kernel<T, true>), dim3(block_grid(total)), dim3(kThreads), 0, stream, x, total, cols, codes, scale);
  } else {
    hipLaunchKernelGGL((quest_act8_save_blocks_kernel<T, false>), dim3(block_grid(total)), dim3(kThreads), 0, stream, x, total, cols, codes, scale);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t load(const int8_t* codes, const uint8_t* scale, int64_t rows, int cols, T* out, hipStream_t stream) {
  const int64_t total = rows * ((cols + kAct8Block - 1) / kAct8Block);
  if (cols % kAct8Block == 0) {
    const int64_t groups = rows * cols / 8, per = kThreads * kUnroll;
    hipLaunchKernelGGL(quest_act8_load_flat_kernel<T>, dim3(static_cast<uint32_t>((groups + per - 1) / per)),
                       dim3(kThreads), 0, stream, codes, scale, groups, out);
  } else if (cols >= 8) {
    hipLaunchKernelGGL((quest_act8_load_blocks_kernel<T, true>), dim3(block_grid(total)), dim3(kThreads), 0, stream, codes, scale, total, cols, out);
  } else {
    hipLaunchKernelGGL((quest_act8_load_blocks_kernel<T, false>), dim3(block_grid(total)), dim3(kThreads), 0, stream, codes, scale, total, cols, out);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act8_save(const void* x, bool x_is_bf16, int64_t rows, int cols, int8_t* codes, uint8_t* scale,
                            hipStream_t stream) {
  if (x_is_bf16) return save(static_cast<const uint16_t*>(x), rows, cols, codes, scale, stream);
  return save(static_cast<const float*>(x), rows, cols, codes, scale, stream);
}

hipError_t launch_act8_load(const int8_t* codes, const uint8_t* scale, int64_t rows, int cols, void* out,
                            bool out_is_bf16, hipStream_t stream) {
  if (out_is_bf16) return load(codes, scale, rows, cols, static_cast<uint16_t*>(out), stream);
  return load(codes, scale, rows, cols, static_cast<float*>(out), stream);
}

}  // namespace quest
