// Building blocks of the FP6 product kernels (gfx950): buffer resources, loads
// into LDS, waits and the fragment layout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace quest {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kFrag = 64 * 24;             // one 32-row x 64-k fragment
constexpr int kBlock = 2 * kFrag;          // one 32-row x 128-k block
constexpr int kNowhereOff = 0x7FFFFFF0;    // past every window: stores there are dropped

// Raw buffer resource: base, byte count, 32-bit raw format; out-of-range
// loads return zero and out-of-range stores are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

// The same resource as four dwords, for the asm loads below.
__device__ __forceinline__ i32x4 raw_rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return i32x4{static_cast<int32_t>(static_cast<uint32_t>(a)), static_cast<int32_t>((a >> 32) & 0xFFFFu),
               static_cast<int32_t>(bytes), 0x00020000};
}

// Two floats to bf16 with round to nearest even (the gfx950 conversion instruction).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// 16 bytes from global memory into LDS at lds_base + 16 * lane.  Written as
// asm so that the compiler's wait counting leaves these loads alone: each
// stage is read only after an explicit vmcnt wait and a barrier.  The load
// has no register results.
__device__ __forceinline__ void dma16(uint32_t lds_base, int32_t voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_base), "v"(voff), "s"(rsrc)
               : "memory");
}

// 4 bytes from global memory into LDS at lds_base + 4 * lane (as dma16).
__device__ __forceinline__ void dma4(uint32_t lds_base, int32_t voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds_base), "v"(voff), "s"(rsrc)
               : "memory");
}

// s_waitcnt with only the vector-memory counter limited (lgkm and exp left
// open); the count's low four bits go to bits 3..0, the high two to 15..14.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt(0x3F70 | (N & 15) | ((N >> 4) << 14));
}

// A workgroup barrier that waits for this wave's LDS accesses only (a
// __syncthreads would also wait for every load and store in flight).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
}

// Tile index -> (tm, tn): groups of 8 tile rows, walked column by column.
__device__ __forceinline__ void tile_at(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int group = 8 * tiles_n;
  const int first_m = (pid / group) * 8;
  const int gm = min(tiles_m - first_m, 8);
  tm = first_m + (pid % group) % gm;
  tn = (pid % group) / gm;
}

// Compute units of the current device (cached per device; concurrent first
// calls on one device may both query it and store the same value).
inline int device_cus() {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int cus = cached[dev].load(std::memory_order_relaxed);
  if (cus == 0) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    cached[dev].store(cus, std::memory_order_relaxed);
  }
  return cus;
}

}  // namespace quest
