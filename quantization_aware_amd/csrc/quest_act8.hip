// Activation checkpoints in 8 bits: saved (quest_act8_save) and read back
// (quest_act8_load).  The format is in quest_act8.h.
//
// Both are one pass over memory with a few operations an entry: bound by HBM.
// Rows of whole blocks (cols a multiple of 32) are one stretch of memory, in
// which entry 8 t .. 8 t + 7 of the tensor belongs to lane t: 16-byte
// accesses of bf16, 8-byte accesses of codes, and a block is four
// neighbouring lanes, whose maximum is two DPP steps.  Other widths go a row
// per wave, an entry per lane, a block per half wave.
#include "quest_act8.h"

#include "quest_launch.h"

namespace quest {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRowBlocks = 1 << 20;  // workgroups of the row-per-wave kernels, which walk the rows beyond
constexpr int kUnroll = 4;  // groups of 8 entries a thread handles in one pass, their loads together

__device__ __forceinline__ int64_t first_row() {
  return static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
}
__device__ __forceinline__ int64_t row_stride() { return static_cast<int64_t>(gridDim.x) * (kThreads / 64); }
uint32_t row_blocks(int64_t rows) {
  const int64_t n = (rows + kThreads / 64 - 1) / (kThreads / 64);
  return static_cast<uint32_t>(n < kMaxRowBlocks ? n : kMaxRowBlocks);
}

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
    uint32_t a = act8_mag(v[u][0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = max(a, act8_mag(v[u][i]));
    const int e = static_cast<int>(quad_max(a) >> 23);
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = act8_encode(v[u][i], e);
    *reinterpret_cast<uint2*>(codes + 8 * g) =
        make_uint2(act8_pack(q[0], q[1], q[2], q[3]), act8_pack(q[4], q[5], q[6], q[7]));
    if ((g & 3) == 0) scale[g >> 2] = static_cast<uint8_t>(e);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quest_act8_save_rows_kernel(const T* __restrict__ x, int64_t rows, int cols, int8_t* __restrict__ codes,
                                uint8_t* __restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int blocks = (cols + kAct8Block - 1) / kAct8Block;
  for (int64_t row = first_row(); row < rows; row += row_stride()) {
    const T* xr = x + row * cols;
    int8_t* cr = codes + row * cols;
    uint8_t* sr = scale + row * blocks;
    for (int c0 = 0; c0 < cols; c0 += 64 * kUnroll) {
      float v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + 64 * u + lane;
        v[u] = c < cols ? to_f32(xr[c]) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + 64 * u + lane;
        const int e = static_cast<int>(half_wave_max(act8_mag(v[u])) >> 23);
        if (c < cols) {
          cr[c] = static_cast<int8_t>(act8_encode(v[u], e));
          if ((lane & 31) == 0) sr[c >> 5] = static_cast<uint8_t>(e);
        }
      }
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
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act8_decode(act8_byte(i < 4 ? w[u].x : w[u].y, i & 3), e[u]);
    store8(out + 8 * g, v);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quest_act8_load_rows_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scale, int64_t rows,
                                int cols, T* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int blocks = (cols + kAct8Block - 1) / kAct8Block;
  for (int64_t row = first_row(); row < rows; row += row_stride()) {
#pragma unroll 4
    for (int c = lane; c < cols; c += 64)
      out[row * cols + c] = from_f32<T>(act8_decode(codes[row * cols + c], scale[row * blocks + (c >> 5)]));
  }
}

template <typename T>
hipError_t save(const T* x, int64_t rows, int cols, int8_t* codes, uint8_t* scale, hipStream_t stream) {
  if (cols % kAct8Block == 0) {
    const int64_t groups = rows * cols / 8, per = kThreads * kUnroll;
    hipLaunchKernelGGL(quest_act8_save_flat_kernel<T>, dim3(static_cast<uint32_t>((groups + per - 1) / per)),
                       dim3(kThreads), 0, stream, x, groups, codes, scale);
  } else {
    hipLaunchKernelGGL(quest_act8_save_rows_kernel<T>, dim3(row_blocks(rows)),
                       dim3(kThreads), 0, stream, x, rows, cols, codes, scale);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t load(const int8_t* codes, const uint8_t* scale, int64_t rows, int cols, T* out, hipStream_t stream) {
  if (cols % kAct8Block == 0) {
    const int64_t groups = rows * cols / 8, per = kThreads * kUnroll;
    hipLaunchKernelGGL(quest_act8_load_flat_kernel<T>, dim3(static_cast<uint32_t>((groups + per - 1) / per)),
                       dim3(kThreads), 0, stream, codes, scale, groups, out);
  } else {
    hipLaunchKernelGGL(quest_act8_load_rows_kernel<T>, dim3(row_blocks(rows)),
                       dim3(kThreads), 0, stream, codes, scale, rows, cols, out);
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
