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
//
// Large products are bound by the matrix cores, and there by power: 16384 x 2048 -> 5632
// takes 205 to 215 us back to back, 1.75 to 1.85 POP/s (a library's product of the same
// codes to int32, without scales, 215; instructions alone on such data 3.5 POP/s, on zeros
// 4.5).  What is between: writing the 185 MB of outputs (some 50 us of it without the epilogue), the
// loads (40 without them) and the row sums (2 to 12).  Sums by dot products after the
// four products of a part, not between them: there they stall the matrix cores (+ 26 us).
// Outputs written through the L2 (sc0 sc1) leave it to the operands: 17 us less than
// plain stores; non-temporal ones gain 14 here and lose 9 at 16384 x 2048 -> 2048.
// 2048 x 5632 -> 2048 takes 30.2 us (its 256 tiles read 12 TB/s from the L2; 4 waves of
// 64 x 64 each instead of 8, or three stages, change nothing), 4096 x 2048 -> 5632 58, 333
// x 960 -> 1001 to fp32 5.8, 48 x 2048 -> 5632 7.3 and one row 2048 -> 2048 3.9 us (medians
// of a kernel trace).  The last is latency.  At 17 to 128 rows each workgroup takes all
// stages of k, and narrow outputs leave compute units without one: 48 x 2048 -> 5632 is 88
// workgroups of 16 stages, for 2.5 us of bytes.
#include <type_traits>

#include "quest_few.h"
#include "quest_launch.h"
#include "quest_mma.h"

namespace quest {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kWriteThrough = 17;  // cache policy of the outputs' stores: sc0 and sc1
constexpr int kStageK = 128;  // bytes of k in a stage: a row's whole cache line

// A row's `left` last elements out of 16 bytes, at any multiple of T's size: in one
// store, or the row's last few one by one.
template <typename T>
__device__ __forceinline__ void store_part(T* dst, u32x4 v, int left) {
  typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(1)));
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  if (left >= kPer) {
    *reinterpret_cast<u32x4_u*>(dst) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer - 1; ++e)
    if (e < left) dst[e] = __builtin_bit_cast(T, static_cast<typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type>(
        sizeof(T) == 2 ? v[e / 2] >> (16 * (e & 1)) : v[e]));
}

// A workgroup of WM x WN waves computes a tile of 32 IB WM rows by 32 JB WN columns.
// Both operands are row-major bytes; a stage is 128 bytes of k of every row (a whole
// cache line), eight 16-byte chunks a row, straight from memory into LDS.  Chunk c of
// row r lies in slot c ^ swizzle(r): the 16 lanes of a fragment read that LDS serves
// together then cover all banks, and so do 8 lanes of half of them.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

template <int WM, int WN, int IB, int JB, int NB>
constexpr int kTileLds = 32 * (IB * WM + JB * WN) * (NB * kStageK + 8);

template <typename Out, bool kVec, int WM, int WN, int IB, int JB, int NB>
__device__ __forceinline__ void i8_tile(const GemmI8Launch& g, int row0, int col0, uint8_t* lds) {
  constexpr int kWaves = WM * WN;
  constexpr int kTileM = 32 * IB * WM, kTileN = 32 * JB * WN;
  constexpr int kStageA = kTileM * kStageK, kStageB = kTileN * kStageK, kStage = kStageA + kStageB;
  constexpr int kOut = static_cast<int>(sizeof(Out));
  constexpr int kLoadsA = kStageA / 1024 / kWaves, kLoadsB = kStageB / 1024 / kWaves;
  constexpr int kLoads = kLoadsA + kLoadsB;  // loads one wave issues per stage
  constexpr int kScaleLoads = (kTileM + kTileN) / 64, kScaleEach = (kScaleLoads + kWaves - 1) / kWaves;
  static_assert(kLoadsA * kWaves * 1024 == kStageA && kLoadsB * kWaves * 1024 == kStageB, "stages split evenly");
  // The waves that share a fragment sum it once.
  constexpr int kSumA = (IB + WN - 1) / WN, kSumB = (JB + WM - 1) / WM;
  static_assert(IB % kSumA == 0 && JB % kSumB == 0, "every wave sums as many");
  constexpr int kRows = kTileM + kTileN;
  int* const sums = reinterpret_cast<int*>(lds + NB * kStage);  // of the tile's rows of a, then of b
  float* const fac = reinterpret_cast<float*>(sums + kRows);    // and their clip scales

  const int m = g.m, n = g.n, k = g.k;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int wm = wave / WN, wn = wave % WN;
  // (renew hides the lane from the compiler, which would keep one phase's addresses
  // through the other)
  int lane = tid & 63;
  auto renew = [&]() { asm volatile("" : "+v"(lane)); };
  const int stages = (k + kStageK - 1) / kStageK;
  auto stage_mem = [&](auto bi) -> uint8_t* { return lds + decltype(bi)::value * kStage; };

  // (rows past the end lie outside the windows and read as zeros; a half tile may lie
  // wholly past n)
  const i32x4 ra = raw_rsrc(g.a + static_cast<size_t>(row0) * k, static_cast<uint32_t>(min(m - row0, kTileM)) * k);
  const int cols = __builtin_amdgcn_readfirstlane(max(min(n - col0, kTileN), 0));
  const i32x4 rb = raw_rsrc(g.b + static_cast<size_t>(col0) * k, static_cast<uint32_t>(cols) * k);
  // The clip scales, 64 a load (entries past the end as zeros); where there are fewer
  // loads than waves, some waves repeat one.
#pragma unroll
  for (int u = 0; u < kScaleEach; ++u) {
    const int i = (wave + kWaves * u) % kScaleLoads;
    const bool of_a = i < kTileM / 64;
    const int first = of_a ? row0 + 64 * i : col0 + 64 * i - kTileM;
    const int left = __builtin_amdgcn_readfirstlane(max(min((of_a ? m : n) - first, 64), 0));
    const float* src = (of_a ? g.sa : g.sb) + first;
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(fac + 64 * i));
    dma4(__builtin_amdgcn_readfirstlane(at), lane * 4, raw_rsrc(src, left * 4));
  }
  // A wave instruction brings 8 rows: lane l chunk (l % 8) ^ swizzle of row l / 8 (and, 8
  // rows on, ^ 1).  Chunks past k (a multiple of 64) are zeros: the upper half of the
  // last stage, and stages past it.
  auto fetch = [&](int st, auto bi) {
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(stage_mem(bi)));
    const int row = lane >> 3, chunk = (lane & 7) ^ swizzle(row);
    const int at0 = row * k + st * kStageK + 16 * chunk, at1 = row * k + st * kStageK + 16 * (chunk ^ 1);
    const bool past = st * kStageK + 16 * chunk >= k;  // (the same for both)
    auto one = [&](int t, uint32_t to, i32x4 rsrc) {
      const int off = past ? kNowhereOff : (t & 1 ? at1 : at0) + 8 * t * k;
      dma16(__builtin_amdgcn_readfirstlane(to + 1024 * t), off, rsrc);
    };
#pragma unroll
    for (int u = 0; u < kLoadsA; ++u) one(wave + kWaves * u, base, ra);
#pragma unroll
    for (int u = 0; u < kLoadsB; ++u) one(wave + kWaves * u, base + kStageA, rb);
  };
  // A wave's fragments.  The WN waves of a band of rows share its IB fragments: wave wn
  // takes them from fragment kSumA wn on, and sums its first kSumA.
  auto row_block = [&](int i) { return wm * IB + (i + kSumA * wn) % IB; };
  auto col_block = [&](int j) { return wn * JB + (j + kSumB * wm) % JB; };
  auto index = [](auto i) { return std::integral_constant<int, decltype(i)::value % NB>{}; };
  auto each_buffer = [&](auto f) {  // f(0), f(1), ... f(NB - 1)
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    if constexpr (NB > 2) f(std::integral_constant<int, 2>{});
    if constexpr (NB > 3) f(std::integral_constant<int, 3>{});
  };
  each_buffer([&](auto i) {
    if constexpr (decltype(i)::value < NB - 1) fetch(decltype(i)::value, i);
  });
  v16i acc[JB][IB];
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int i = 0; i < IB; ++i) acc[j][i] = v16i{};
  v4i sum_a[kSumA] = {}, sum_b[kSumB] = {};  // (four each: a chain of them would wait for itself)
  renew();
  int lane_off[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int r32 = lane & 31, h = lane >> 5;
    lane_off[ks] = r32 * kStageK + 16 * ((2 * ks + h) ^ swizzle(r32));
  }
  auto frag = [&](auto bi, int op, int blk, int ks) -> v4i {
    return *reinterpret_cast<const v4i*>(stage_mem(bi) + op * kStageA + blk * (32 * kStageK) + lane_off[ks]);
  };
  v4i f0a[IB], f0b[JB], f1a[IB], f1b[JB];
  auto read = [&](auto bi, int ks, v4i (&fa)[IB], v4i (&fb)[JB]) {
#pragma unroll
    for (int i = 0; i < IB; ++i) fa[i] = frag(bi, 0, row_block(i), ks);
#pragma unroll
    for (int j = 0; j < JB; ++j) fb[j] = frag(bi, 1, col_block(j), ks);
  };
  auto multiply = [&](const v4i (&fa)[IB], const v4i (&fb)[JB]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int i = 0; i < IB; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[j][i], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
#pragma unroll
      for (int i = 0; i < kSumA; ++i) sum_a[i][d] = __builtin_amdgcn_sdot4(fa[i][d], 0x01010101, sum_a[i][d], false);
#pragma unroll
      for (int j = 0; j < kSumB; ++j) sum_b[j][d] = __builtin_amdgcn_sdot4(fb[j][d], 0x01010101, sum_b[j][d], false);
    }
  };
  constexpr int kInFlight = (NB - 2) * kLoads;
  wait_vmcnt<kInFlight>();  // stage 0 has landed
  lds_barrier();
  read(std::integral_constant<int, 0>{}, 0, f0a, f0b);
  // Step s lies in buffer i; the one before i held s - 1, whose reads every wave
  // finished before the last barrier, and receives s + NB - 1.  A step's products come
  // in four parts, each while the next one's fragments are read.
  auto step = [&](int s, auto i) {
    constexpr int I = decltype(i)::value;
    fetch(s + NB - 1, index(std::integral_constant<int, I + NB - 1>{}));
    read(i, 1, f1a, f1b);
    multiply(f0a, f0b);
    read(i, 2, f0a, f0b);
    multiply(f1a, f1b);
    read(i, 3, f1a, f1b);
    multiply(f0a, f0b);
    wait_vmcnt<kInFlight>();  // step s + 1's stage has landed
    lds_barrier();            // for every wave, and all reads of this one are done
    read(index(std::integral_constant<int, I + 1>{}), 0, f0a, f0b);
    multiply(f1a, f1b);
  };
  int s = 0;
  for (; s + NB <= stages; s += NB) each_buffer([&](auto i) { step(s + decltype(i)::value, i); });
  const int left = stages - s;
  each_buffer([&](auto i) {
    if (decltype(i)::value < left) step(s + decltype(i)::value, i);
  });

  // The row sums (both halves of a wave hold one each) to where every wave finds them.
  renew();
  const int r32 = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < kSumA; ++i) {
    int v = sum_a[i][0] + sum_a[i][1] + sum_a[i][2] + sum_a[i][3];
    v += __shfl_xor(v, 32);
    if (kSumA * wn < IB && h == 0) sums[32 * row_block(i) + r32] = v;
  }
#pragma unroll
  for (int j = 0; j < kSumB; ++j) {
    int v = sum_b[j][0] + sum_b[j][1] + sum_b[j][2] + sum_b[j][3];
    v += __shfl_xor(v, 32);
    if (kSumB * wm < JB && h == 1) sums[kTileM + 32 * col_block(j) + r32] = v;
  }
  lds_barrier();
  // A wave's column factors and sums: 16 columns a lane of each block of 32.
  float fb[JB][16];
  uint32_t tb[JB][16];
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = kTileM + 32 * col_block(j) + 8 * q + 4 * h;
      const float4 f = *reinterpret_cast<const float4*>(&fac[c]);
      const int4 t = *reinterpret_cast<const int4*>(&sums[c]);
      fb[j][4 * q] = f.x * g.kb, fb[j][4 * q + 1] = f.y * g.kb, fb[j][4 * q + 2] = f.z * g.kb;
      fb[j][4 * q + 3] = f.w * g.kb;
      tb[j][4 * q] = 2u * t.x, tb[j][4 * q + 1] = 2u * t.y, tb[j][4 * q + 2] = 2u * t.z, tb[j][4 * q + 3] = 2u * t.w;
    }
  const auto rout = make_rsrc(static_cast<Out*>(g.out) + static_cast<size_t>(row0) * n,
                              static_cast<uint32_t>(min(m - row0, kTileM)) * static_cast<uint32_t>(n) * kOut);
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int rr = 32 * row_block(i) + r32;
    const float fa = fac[rr] * g.ka;
    const uint32_t ta = 2u * static_cast<uint32_t>(sums[rr]) + static_cast<uint32_t>(k);
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        // (unsigned: the terms may wrap, their sum does not; g.ka holds the quarter)
        const uint32_t v = 4u * static_cast<uint32_t>(acc[j][i][e]) + (tb[j][e] + ta);
        y[e] = static_cast<float>(static_cast<int>(v)) * (fa * fb[j][e]);
      }
      // Whole 64-byte pieces of rows: a lane has four columns of every eight; the lane
      // 16 away, and for bf16 first the one 32 away, trade them for neighbouring ones.
      // Then chunk c of lane l is row 16 c' + l % 16, c' and the column from its place.
      constexpr int kDwords = 4 * kOut;
      uint32_t w[kDwords];
      if constexpr (kOut == 4) {
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(y[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
        // quad q's dwords 2 q, 2 q + 1: the halves trade quads 0, 2 and 1, 3
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const auto s2 = __builtin_amdgcn_permlane32_swap(w[d], w[d + 4], false, false);
          w[d] = s2[0], w[d + 4] = s2[1];
        }
        // lane half h: columns 16 h .. + 15 in the order of dwords 0 1 4 5 2 3 6 7
        const uint32_t x2 = w[2], x3 = w[3];
        w[2] = w[4], w[3] = w[5], w[4] = x2, w[5] = x3;
      }
#pragma unroll
      for (int p = 0; p < kDwords / 8; ++p) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const auto s2 = __builtin_amdgcn_permlane16_swap(w[8 * p + d], w[8 * p + 4 + d], false, false);
          w[8 * p + d] = s2[0], w[8 * p + 4 + d] = s2[1];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = 32 * row_block(i) + 16 * c + (lane & 15);
          // fp32: 32 bytes of quad 2 p + (l / 16) % 2; bf16: the half's 8-column pieces
          const int cl = kOut == 4 ? 8 * (2 * p + ((lane >> 4) & 1)) + 4 * h : 16 * h + 8 * ((lane >> 4) & 1);
          const int col = col0 + 32 * col_block(j) + cl;
          const u32x4 chunk = {w[8 * p + 4 * c], w[8 * p + 4 * c + 1], w[8 * p + 4 * c + 2], w[8 * p + 4 * c + 3]};
          if constexpr (kVec) {
            // n is a multiple of kPer: a chunk is wholly inside or wholly past the row
            const int off = col < n ? (row * n + col) * kOut : kNowhereOff;
            __builtin_amdgcn_raw_buffer_store_b128(chunk, rout, off, 0, kWriteThrough);
          } else if (row0 + row < m && col < n) {
            store_part(static_cast<Out*>(g.out) + static_cast<int64_t>(row0 + row) * n + col, chunk, n - col);
          }
        }
      }
    }
  }
}

// Workgroups are dealt to the 8 XCDs round-robin; each XCD takes a contiguous range of
// `count` tiles, whose operands then share its L2 (the last count % 8 keep their own).
__device__ __forceinline__ int tile_of_workgroup(int bid, int count) {
  const int full = count & ~7;
  return bid < full ? (bid & 7) * (full >> 3) + (bid >> 3) : bid;
}

template <typename Out, bool kVec, int WM, int WN, int IB, int JB, int NB>
__global__ void __launch_bounds__(64 * WM * WN, 1) quest_gemm_i8_kernel(const GemmI8Launch g) {
  constexpr int kTileM = 32 * IB * WM, kTileN = 32 * JB * WN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTileLds<WM, WN, IB, JB, NB>];
  int tm, tn;
  tile_at(tile_of_workgroup(blockIdx.x, gridDim.x), (g.m + kTileM - 1) / kTileM, (g.n + kTileN - 1) / kTileN, tm, tn);
  i8_tile<Out, kVec, WM, WN, IB, JB, NB>(g, tm * kTileM, tn * kTileN, lds);
}

// 256 x 256 tiles, one workgroup a compute unit at a time.  The last `halves` / 2 tiles
// are done as halves of 128 columns: half of them first and half of them last, so that
// the compute units end together and do not store their tiles at the same time.
template <typename Out, bool kVec>
__global__ void __launch_bounds__(512, 1) quest_gemm_i8_large_kernel(const GemmI8Launch g, int halves) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTileLds<2, 4, 4, 2, 2>];
  const int tiles_m = (g.m + 255) >> 8, tiles_n = (g.n + 255) >> 8, full = tiles_m * tiles_n - halves / 2;
  const int first = halves / 2 & ~7, bid = blockIdx.x;  // halves before the full tiles
  int tm, tn;
  if (bid >= first && bid < first + full) {
    tile_at(tile_of_workgroup(bid - first, full), tiles_m, tiles_n, tm, tn);
    i8_tile<Out, kVec, 2, 4, 4, 2, 2>(g, tm * 256, tn * 256, lds);
  } else {
    const int h = tile_of_workgroup(bid < first ? bid : bid - full, halves);
    tile_at(full + (h >> 1), tiles_m, tiles_n, tm, tn);
    i8_tile<Out, kVec, 2, 4, 4, 1, 2>(g, tm * 256, tn * 256 + (h & 1) * 128, lds);
  }
}

template <typename Out, bool kVec, int WM, int WN, int IB, int JB, int NB>
hipError_t launch_tiles(const GemmI8Launch& g) {
  constexpr int kTileM = 32 * IB * WM, kTileN = 32 * JB * WN;
  const int tiles = ((g.m + kTileM - 1) / kTileM) * ((g.n + kTileN - 1) / kTileN);
  hipLaunchKernelGGL((quest_gemm_i8_kernel<Out, kVec, WM, WN, IB, JB, NB>), dim3(tiles), dim3(64 * WM * WN),
                     0, g.stream, g);
  return hipGetLastError();
}

template <typename Out, bool kVec>
hipError_t launch_large(const GemmI8Launch& g, int cus) {
  const int tiles = ((g.m + 255) / 256) * ((g.n + 255) / 256), last = tiles % cus;
  const int halves = tiles > cus && 2 * last <= cus ? 2 * last : 0;
  hipLaunchKernelGGL((quest_gemm_i8_large_kernel<Out, kVec>), dim3(tiles + halves / 2), dim3(512), 0, g.stream, g,
                     halves);
  return hipGetLastError();
}

// At most 16 rows of one operand ("tokens": a's rows, or with kSwap b's): a workgroup
// takes 16 rows of the other; its 8 waves share k and add their exact sums through LDS.
template <typename Out, bool kSwap>
__global__ void __launch_bounds__(512) quest_gemm_i8_few_kernel(const GemmI8Launch g) {
  constexpr int kWaves = 8;
  __shared__ __attribute__((aligned(16))) uint32_t part[kWaves][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int tokens = kSwap ? g.n : g.m, rows = kSwap ? g.m : g.n, k = g.k;
  const int row0 = blockIdx.x * 16;
  // (rows past the last read as zeros)
  const few_rsrc rw = few_window((kSwap ? g.a : g.b) + static_cast<int64_t>(row0) * k, min(rows - row0, 16) * k);
  const few_rsrc rx = few_window(kSwap ? g.b : g.a, tokens * k);
  const int at = (lane & 15) * k + 16 * (lane >> 4);
  constexpr int kAhead = 4;
  const FewRing<kAhead> ring{wave, kWaves, k / 64};
  v4i fw[kAhead][1];
  TokenBytes<false> fx[kAhead][1];
  auto load = [&](int c, int i) {
    const int off = c < ring.chunks ? at + c * 64 : kNoBytes;
    fw[i][0] = load_window(rw, off);
    fx[i][0].v[0] = load_window(rx, off);
  };
  FewSums<false, 1, 1> s;
  ring.begin(load);
  ring.run(load, [&](int, int i) { s.add(fw[i], fx[i]); });
  *reinterpret_cast<v4u*>(&part[wave][(lane & 15) * 16 + 4 * (lane >> 4)]) = s.total(0, 0);
  __syncthreads();
  const int token = tid / 16, row = row0 + tid % 16;
  if (tid >= 256 || token >= tokens || row >= rows) return;
  uint32_t v = few_constant<false>(k);
#pragma unroll
  for (int i = 0; i < kWaves; ++i) v += part[i][tid];
  const int i = kSwap ? row : token, j = kSwap ? token : row;
  const float y = static_cast<float>(static_cast<int>(v)) * ((g.sa[i] * g.ka) * (g.sb[j] * g.kb));
  Out* const out = static_cast<Out*>(g.out) + static_cast<int64_t>(i) * g.n + j;
  if constexpr (sizeof(Out) == 2)
    *out = static_cast<Out>(pack_bf16x2(y, 0.0f));
  else
    *out = y;
}

// What a variant takes, about, in microseconds: rounds of as many tiles as lie on the
// compute units at a time (`each` a unit), of e + s per stage; a last round of at most
// one tile a unit goes at s1 per stage.
struct Variant {
  int rows, cols, each;
  float e, s1, s;
};
float cost(const GemmI8Launch& g, const Variant& v, int cus) {
  const int64_t tiles = static_cast<int64_t>((g.m + v.rows - 1) / v.rows) * ((g.n + v.cols - 1) / v.cols);
  const int64_t at_once = static_cast<int64_t>(cus) * v.each;
  const int64_t last = tiles % at_once;
  const float stages = static_cast<float>((g.k + kStageK - 1) / kStageK);
  float t = static_cast<float>(tiles / at_once) * (v.e + v.s * stages);
  if (last) t += (v.e + (last <= cus ? v.s1 : v.s) * stages) * (v.rows == 256 && tiles > cus && 2 * last <= cus ? 0.55f : 1.0f);
  return t;
}

template <typename Out, bool kVec>
hipError_t launch(const GemmI8Launch& g) {
  const int cus = device_cus();
  // Few rows of one operand and not too many bytes of the other: 1 x 2048 -> 2048 takes 3.9 us (6.9 in 64 x 64
  // tiles), 5 x 5632 -> 2048 6.7 (12.6), 16 x 2048 -> 5632 7.4 (7.2), 16 x 8192 -> 8192 18.2 (17.8).
  constexpr int64_t kFewBytes = int64_t(1) << 25;
  if (g.m <= 16 && static_cast<int64_t>(g.n) * g.k <= kFewBytes) {
    hipLaunchKernelGGL((quest_gemm_i8_few_kernel<Out, false>), dim3((g.n + 15) / 16), dim3(512), 0, g.stream, g);
    return hipGetLastError();
  }
  if (g.n <= 16 && static_cast<int64_t>(g.m) * g.k <= kFewBytes) {
    hipLaunchKernelGGL((quest_gemm_i8_few_kernel<Out, true>), dim3((g.m + 15) / 16), dim3(512), 0, g.stream, g);
    return hipGetLastError();
  }
  // Largest tiles first: of equal estimates the one that reads less.  Times of a stage
  // as measured on 256 compute units.
  constexpr Variant kVariants[] = {
      {256, 256, 1, 4.0f, 1.75f, 1.75f}, {128, 128, 2, 2.5f, 0.85f, 1.1f}, {128, 128, 1, 2.2f, 0.6f, 0.6f},
      {128, 64, 2, 2.4f, 0.4f, 0.8f},    {64, 64, 2, 2.2f, 0.28f, 0.42f}};
  int best = 0;
  float least = 0.0f;
  for (int i = 0; i < 5; ++i) {
    const float t = cost(g, kVariants[i], cus);
    if (i == 0 || t < least) best = i, least = t;
  }
  switch (best) {
    case 0: return launch_large<Out, kVec>(g, cus);
    case 1: return launch_tiles<Out, kVec, 2, 2, 2, 2, 2>(g);
    case 2: return launch_tiles<Out, kVec, 2, 4, 2, 1, 4>(g);
    case 3: return launch_tiles<Out, kVec, 2, 2, 2, 1, 3>(g);
    default: return launch_tiles<Out, kVec, 2, 2, 1, 1, 4>(g);
  }
}

}  // namespace

hipError_t launch_gemm_i8(const GemmI8Launch& g, bool out_bf16) {
  if (out_bf16) return g.n % 8 == 0 ? launch<uint16_t, true>(g) : launch<uint16_t, false>(g);
  return g.n % 4 == 0 ? launch<float, true>(g) : launch<float, false>(g);
}

}  // namespace quest
