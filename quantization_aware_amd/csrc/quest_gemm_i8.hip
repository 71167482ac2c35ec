// Product of two tensors of codes in 8-bit integers, with a scale per row of each.
//
// A row of b-bit codes c (signed bytes) with clip scale s stands for
// (2 c + 1) s / (2^b - 1), so with the step D = 2 s / (2^b - 1)
//   y[i][j] = D_a[i] D_b[j] T / 4,
//   T = sum_k (2 a + 1)(2 b + 1) = 4 sum_k a b + 2 (sum_k a + sum_k b) + K.
// sum_k a b comes from the int8 matrix instructions; the two row sums are taken
// from the same fragments.  For b = 8, 2 c + 1 needs nine bits, which is why the
// half is kept out of the matrix product.  Every sum is exact: |T| <= K 255^2 is
// below 2^31 for K <= 32768, and T itself is what the (wrapping) 32-bit terms add
// up to.  The roundings are those of quest_gemm: 2 / (2^b - 1) and D for both
// operands, D_a D_b, T to fp32, the product, and the output type.  Where
// |T| < 2^24 both products give the same bits.
#include <type_traits>

#include "quest_launch.h"
#include "quest_mma.h"

namespace quest {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kStageK = 64;  // bytes of k in a stage

__device__ __forceinline__ int sum4(v4i f, int acc) {
#pragma unroll
  for (int d = 0; d < 4; ++d) acc = __builtin_amdgcn_sdot4(f[d], 0x01010101, acc, false);
  return acc;
}

// A workgroup of WM x WN waves computes 32 IB WM rows by 32 JB WN columns.
// Both operands are row-major bytes; a stage is 64 bytes of k of every row, four
// 16-byte chunks a row, straight from memory into LDS.  Chunk c of row r lies in
// slot c ^ swizzle(r): the 16 lanes of a fragment read that LDS serves together
// then cover all banks (and so do 8 lanes of half of them).
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) ^ (r >> 3)) & 1 | ((r >> 1) & 2); }

template <typename Out, bool kVec, int WM, int WN, int IB, int JB, int kMinWaves>
__global__ void __launch_bounds__(64 * WM * WN, kMinWaves) quest_gemm_i8_kernel(const GemmI8Launch g) {
  constexpr int kWaves = WM * WN;
  constexpr int kTileM = 32 * IB * WM, kTileN = 32 * JB * WN;
  constexpr int kStageA = kTileM * kStageK, kStageB = kTileN * kStageK, kStage = kStageA + kStageB;
  constexpr int kOut = static_cast<int>(sizeof(Out));
  constexpr int kPer = 16 / kOut;  // outputs per 16-byte chunk
  constexpr int kLanesPerRow = 32 * JB / kPer;
  constexpr int kPitch = 32 * JB * kOut + 16;  // slab row pitch in bytes
  constexpr int kLoadsA = kStageA / 1024 / kWaves, kLoadsB = kStageB / 1024 / kWaves;
  constexpr int kLoads = kLoadsA + kLoadsB;  // loads one wave issues per stage
  static_assert(kLoadsA * kWaves * 1024 == kStageA && kLoadsB * kWaves * 1024 == kStageB, "stages split evenly");
  static_assert(kWaves * 32 * kPitch <= 3 * kStage, "the waves' slabs fit the stage buffers");
  static_assert(IB <= WN && JB <= WM, "the waves that share a fragment sum it once");
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kStage + 8 * (kTileM + kTileN)];
  int* const sums = reinterpret_cast<int*>(lds + 3 * kStage);                    // of the tile's rows of a, then of b
  float* const fac = reinterpret_cast<float*>(sums + kTileM + kTileN);  // and their clip scales

  const int m = g.m, n = g.n, k = g.k;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int lane = tid & 63;
  const int r32 = lane & 31, h = lane >> 5;
  const int stages = k / kStageK;
  const int tiles_m = (m + kTileM - 1) / kTileM, tiles_n = (n + kTileN - 1) / kTileN;
  // Workgroups are dealt to the 8 XCDs round-robin; each XCD takes a
  // contiguous range of tiles, whose operands then share its L2.
  int pid = blockIdx.x, tm, tn;
  const int full = static_cast<int>(gridDim.x) & ~7;
  if (pid < full) pid = (pid & 7) * (full >> 3) + (pid >> 3);
  tile_at(pid, tiles_m, tiles_n, tm, tn);
  const int row0 = tm * kTileM, col0 = tn * kTileN;

  // (rows past the end lie outside the windows and read as zeros)
  const i32x4 ra = raw_rsrc(g.a + static_cast<size_t>(row0) * k, static_cast<uint32_t>(min(m - row0, kTileM)) * k);
  const i32x4 rb = raw_rsrc(g.b + static_cast<size_t>(col0) * k, static_cast<uint32_t>(min(n - col0, kTileN)) * k);
  auto stage_mem = [&](auto bi) -> uint8_t* { return lds + decltype(bi)::value * kStage; };
  // A wave instruction brings 16 rows' 64 bytes: lane l chunk (l % 4) ^ swizzle
  // of row l / 4 (16 rows on, the swizzle is the same).
  const int fetch_off = (lane >> 2) * k + 16 * ((lane & 3) ^ swizzle(lane >> 2));
  auto fetch = [&](int st, auto bi) {
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(stage_mem(bi)));
#pragma unroll
    for (int u = 0; u < kLoadsA; ++u) {
      const int t = wave + kWaves * u;
      dma16(__builtin_amdgcn_readfirstlane(base + 1024 * t), fetch_off + 16 * t * k + st * kStageK, ra);
    }
#pragma unroll
    for (int u = 0; u < kLoadsB; ++u) {
      const int t = wave + kWaves * u;
      dma16(__builtin_amdgcn_readfirstlane(base + kStageA + 1024 * t), fetch_off + 16 * t * k + st * kStageK, rb);
    }
  };
  // A wave's fragments.  The WN waves of a band of rows share its IB fragments:
  // wave wn takes them from fragment wn on, and sums its first one.
  const int lane_off[2] = {r32 * kStageK + 16 * (h ^ swizzle(r32)), r32 * kStageK + 16 * ((2 + h) ^ swizzle(r32))};
  auto row_block = [&](int i) { return wm * IB + (i + wn) % IB; };
  auto col_block = [&](int j) { return wn * JB + (j + wm) % JB; };
  auto frag = [&](auto bi, int op, int blk, int ks) -> v4i {
    const uint8_t* s = stage_mem(bi) + op * kStageA + blk * (32 * kStageK) + lane_off[ks];
    return *reinterpret_cast<const v4i*>(s);
  };

  v16i acc[JB][IB];
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int i = 0; i < IB; ++i) acc[j][i] = v16i{};
  int sum_a = 0, sum_b = 0;

  // The clip scales, 64 a load (entries past the end as zeros); where there are
  // fewer loads than waves, some waves repeat one.
  constexpr int kScaleLoads = (kTileM + kTileN) / 64;
#pragma unroll
  for (int u = 0; u < (kScaleLoads + kWaves - 1) / kWaves; ++u) {
    const int t = (wave + kWaves * u) % kScaleLoads;
    const bool of_a = t < kTileM / 64;
    const int first = of_a ? row0 + 64 * t : col0 + 64 * t - kTileM;
    const int left = __builtin_amdgcn_readfirstlane(max(min((of_a ? m : n) - first, 64), 0));
    const float* src = (of_a ? g.sa : g.sb) + first;
    const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(fac + 64 * t));
    dma4(__builtin_amdgcn_readfirstlane(to), lane * 4, raw_rsrc(src, left * 4));
  }
  // Three stage buffers, two stages ahead; stages past the last are the last one
  // again, so that every wait counts the same loads.
  fetch(0, I0{});
  fetch(stages > 1 ? 1 : 0, I1{});
  auto step = [&](int s, auto bi, auto b2) {
    wait_vmcnt<kLoads>();  // stage s has landed (s + 1 may be in flight)
    lds_barrier();         // for every wave, and all reads of stage s - 1 are done
    fetch(s + 2 < stages ? s + 2 : stages - 1, b2);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v4i fa[IB], fb[JB];
#pragma unroll
      for (int i = 0; i < IB; ++i) fa[i] = frag(bi, 0, row_block(i), ks);
#pragma unroll
      for (int j = 0; j < JB; ++j) fb[j] = frag(bi, 1, col_block(j), ks);
#pragma unroll
      for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int i = 0; i < IB; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[j][i], 0, 0, 0);
      sum_a = sum4(fa[0], sum_a);
      sum_b = sum4(fb[0], sum_b);
    }
  };
  int s = 0;
  for (; s + 3 <= stages; s += 3) {
    step(s, I0{}, I2{});
    step(s + 1, I1{}, I0{});
    step(s + 2, I2{}, I1{});
  }
  if (s < stages) step(s++, I0{}, I2{});
  if (s < stages) step(s++, I1{}, I0{});

  // The row sums (both halves of a wave hold one each) to where every wave finds them.
  sum_a += __shfl_xor(sum_a, 32);
  sum_b += __shfl_xor(sum_b, 32);
  if (wn < IB && h == 0) sums[32 * row_block(0) + r32] = sum_a;
  if (wm < JB && h == 1) sums[kTileM + 32 * col_block(0) + r32] = sum_b;
  wait_vmcnt<0>();  // no load into LDS in flight before the buffers become the slabs
  lds_barrier();

  uint8_t* slab = lds + wave * 32 * kPitch;
  const auto rout = make_rsrc(static_cast<Out*>(g.out) + static_cast<size_t>(row0) * n,
                              static_cast<uint32_t>(min(m - row0, kTileM)) * static_cast<uint32_t>(n) * kOut);
  auto slab_fence = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  float4 fb[JB][4];
  int4 tb[JB][4];
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = 32 * col_block(j) + 8 * q + 4 * h;  // the lane's columns c .. c + 3 of the tile
      const float4 w = *reinterpret_cast<const float4*>(&fac[kTileM + c]);
      fb[j][q] = make_float4(w.x * g.kb, w.y * g.kb, w.z * g.kb, w.w * g.kb);
      tb[j][q] = *reinterpret_cast<const int4*>(&sums[kTileM + c]);
    }
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int r = 32 * row_block(i) + r32;
    const float fa = fac[r] * g.ka;
    const int ta = 2 * sums[r] + k;
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int cl = 32 * ((j + wm) % JB) + 8 * q + 4 * h;  // column within the wave's 32 JB
        const int t[4] = {tb[j][q].x, tb[j][q].y, tb[j][q].z, tb[j][q].w};
        const float f[4] = {fb[j][q].x, fb[j][q].y, fb[j][q].z, fb[j][q].w};
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (unsigned: the terms may wrap, their sum does not)
          const uint32_t v = 4u * static_cast<uint32_t>(acc[j][i][4 * q + e]) + 2u * static_cast<uint32_t>(t[e]) +
                             static_cast<uint32_t>(ta);
          y[e] = (static_cast<float>(static_cast<int>(v)) * 0.25f) * (fa * f[e]);
        }
        uint8_t* d = slab + r32 * kPitch + cl * kOut;
        if constexpr (kOut == 4) {
          *reinterpret_cast<u32x4*>(d) =
              u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
        } else {
          *reinterpret_cast<u32x2*>(d) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        }
      }
    slab_fence();
#pragma unroll
    for (int t = 0; t < 32 * kLanesPerRow / 64; ++t) {
      const int sr = t * (64 / kLanesPerRow) + lane / kLanesPerRow, sc = (lane % kLanesPerRow) * kPer;
      const int row = 32 * row_block(i) + sr;  // within the tile
      const int col = col0 + wn * 32 * JB + sc;
      const uint8_t* src = slab + sr * kPitch + sc * kOut;
      if constexpr (kVec) {
        // n is a multiple of kPer: a chunk is wholly inside or wholly past the row
        const int off = col < n ? (row * n + col) * kOut : kNowhereOff;
        __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(src), rout, off, 0, 0);
      } else if (row0 + row < m && col < n) {
        store_chunk<Out>(static_cast<Out*>(g.out) + static_cast<int64_t>(row0 + row) * n + col, src, n - col);
      }
    }
    slab_fence();
  }
}

template <typename Out, bool kVec, int WM, int WN, int IB, int JB, int kMinWaves>
hipError_t launch_tiles(const GemmI8Launch& g) {
  constexpr int kTileM = 32 * IB * WM, kTileN = 32 * JB * WN;
  const int tiles = ((g.m + kTileM - 1) / kTileM) * ((g.n + kTileN - 1) / kTileN);
  hipLaunchKernelGGL((quest_gemm_i8_kernel<Out, kVec, WM, WN, IB, JB, kMinWaves>), dim3(tiles), dim3(64 * WM * WN), 0,
                     g.stream, g);
  return hipGetLastError();
}

template <typename Out, bool kVec>
hipError_t launch(const GemmI8Launch& g) {
  return launch_tiles<Out, kVec, 2, 2, 2, 2, 2>(g);
}

}  // namespace

hipError_t launch_gemm_i8(const GemmI8Launch& g, bool out_bf16) {
  if (out_bf16) return g.n % 8 == 0 ? launch<uint16_t, true>(g) : launch<uint16_t, false>(g);
  return g.n % 4 == 0 ? launch<float, true>(g) : launch<float, false>(g);
}

}  // namespace quest
