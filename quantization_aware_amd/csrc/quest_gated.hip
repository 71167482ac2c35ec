// The gated feed-forward product of quantised operands and its backward pass.
//
//   g = Q(x) Q(gate)^T,  u = Q(x) Q(up)^T,  h = act(g) * u,
// with the operands of quest_gemm: FP6 E2M3 levels, tiled in blocks of 32 rows
// x 128 columns (include/quest.h).  Both products, the activation and the
// product are one kernel: g and u never leave the registers in more than the
// 8 bits of their checkpoints (quest_act8.h), which the training form writes.
// The levels' products are quarter-integers whose sums stay below 2^22, so the
// fp32 accumulation is exact in any order, and
//   g[i][j] = acc[i][j] * ((sx[i] kx) * (sg[j] kw)),  k = 2 / (2^bits - 1),
// has six roundings (two of them of kx and kw) and then the activation's.
//
// Kernel: a workgroup of 4 waves computes 64 kB rows x 64 kB columns of h.  The
// two weight operands' blocks of 32 columns stand side by side in a stage of
// LDS, so that a wave holds its gate and up accumulators (kB blocks of 32
// columns by kB blocks of 32 rows each) in the same lanes and registers: lane l
// has row l % 32 and 4 consecutive columns per register quad of both.
// kB = 2: two workgroups share a compute unit, each with two stages of 36 KB;
// one's waits, activations and stores run beside the other's products.
// 16384 x 2048 -> 5632 takes 258 us (2.93 PFLOP/s), 296 us with both
// checkpoints; the products alone 212.  Bound by the bytes through LDS: a stage
// moves 110 KB (36 written, 74 read) for 64 matrix instructions, and of 256 us
// the loop without the loads into LDS saves 43, without the fragment reads 20,
// without both 79, with half the matrix instructions 23.  Power sets the clock (1.85
// to 1.96 of 2.4 GHz; matrix cores 34% and LDS 44% busy, 29% and 41% with checkpoints).
// (256-row tiles of 8 waves, one workgroup a compute unit walking its tiles, the
// next one's first stages requested before the stores: 252 and 306 us.)
// kB = 1: four times the workgroups, for products whose larger tiles would
// leave compute units without one; 256 rows take 10.5 us (15.4 with kB = 2).
#include <type_traits>

#include "quest_act8.h"
#include "quest_launch.h"
#include "quest_mma.h"

namespace quest {
namespace {

// act(g) and act'(g).  kFast (silu): the hardware's reciprocal and exp2 (about
// 2^-22 relative), for values that are rounded to bf16 next; fp32 results of silu
// take the full-precision functions.  gelu is normal_cdf's for both.
template <bool kFast>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (kFast) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
  return 1.0f / (1.0f + expf(-g));
}
// Phi(g), the normal distribution function, and exp(-g^2 / 2).  For z = |g| / sqrt(2),
// erfc(z) exp(z^2) is smooth in t = 1 / (1 + 0.325 z); the polynomial is its minimax fit
// in relative error over z <= 9.4 (4.6e-8; beyond, exp(-z^2) is below fp32), halved.  Both
// signs and the tail keep their digits: within (g^2 + 9) 2^-24 relative, most of it the
// rounding of g^2.  About 14 operations, against some 60 and a branch of erfcf.
__device__ __forceinline__ float normal_cdf(float g, float& dens) {
  dens = __builtin_amdgcn_exp2f(g * g * -0.72134752f);
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.2298097f, 1.0f));
  float p = -0.0790198296f;
  p = fmaf(p, t, 0.293662339f);
  p = fmaf(p, t, -0.283676565f);
  p = fmaf(p, t, 0.306698561f);
  p = fmaf(p, t, -0.0359165892f);
  p = fmaf(p, t, 0.120484531f);
  p = fmaf(p, t, 0.0854686797f);
  p = fmaf(p, t, 0.0923278406f);
  p = fmaf(p, t, -2.89869931e-5f);
  const float q = dens * p;
  return g < 0.0f ? q : 1.0f - q;
}

template <bool kFast>
__device__ __forceinline__ float act_value(float g, int act) {
  if (act == 0) return g * sigmoid<kFast>(g);
  float dens;
  return g * normal_cdf(g, dens);
}
template <bool kFast>
__device__ __forceinline__ void act_both(float g, int act, float& value, float& slope) {
  if (act == 0) {
    const float s = sigmoid<kFast>(g);
    value = g * s;
    slope = fmaf(value, 1.0f - s, s);
  } else {
    float dens;
    const float phi = normal_cdf(g, dens);
    value = g * phi;
    slope = fmaf(g * 0.398942280f, dens, phi);
  }
}

// 16 bytes of LDS to a row's `left` last elements of T at any multiple of T's
// size: in one store, or the row's last few one by one.
template <typename T>
__device__ __forceinline__ void store_chunk(T* dst, const uint8_t* src, int left) {
  typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(1)));
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  if (left >= kPer) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(src);
    *reinterpret_cast<u32x4_u*>(dst) = v;
  } else {
    for (int e = 0; e < left; ++e) dst[e] = reinterpret_cast<const T*>(src)[e];
  }
}

template <typename Out, int kB>
constexpr int kSlabPitch = 32 * kB * static_cast<int>(sizeof(Out)) + 16;  // bytes of a slab's row, 32 rows a slab

// What a wave does with its sums of gate (acc[0 .. kB - 1]) and up (the others) of
// rows row0 + row1 .. and columns wcol ..: its kB blocks of 32 rows, each through
// the wave's slab of LDS, so that a row's 32 kB columns leave together.
// fx_at, fg_at, fu_at: Delta's factors of those rows and columns.  The windows
// start at row0 and hold `rows_left` rows.
template <typename Out, int kB, bool kVec, bool kAct8, int kAct>
__device__ __forceinline__ void gated_epilogue(const GatedLaunch& a, v16f (&acc)[2 * kB][kB], const float* fx_at,
                                               const float* fg_at, const float* fu_at, uint8_t* slab, int row0,
                                               int row1, int rows_left, int wcol, int lane) {
  constexpr int kOut = static_cast<int>(sizeof(Out));
  constexpr int kPer = 16 / kOut;               // outputs per 16-byte chunk
  constexpr int kLanesPerRow = 32 * kB / kPer;  // a wave's columns
  constexpr int kPitch = kSlabPitch<Out, kB>;
  constexpr int kCodes = 32 * kB;  // a row's codes of gate, then up's
  static_assert(2 * kCodes + 16 <= kPitch, "the codes fit the slab");
  const int m = a.m;
  const auto rout = make_rsrc(static_cast<Out*>(a.out) + static_cast<size_t>(row0) * m,
                              static_cast<uint32_t>(rows_left) * static_cast<uint32_t>(m) * kOut);
  const int r32 = lane & 31, h = lane >> 5;
  auto slab_fence = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const float fx = fx_at[32 * i + r32];
    uint32_t code[2][kB][4];  // [gate, up][block][quad]
    int ex[2][kB];
#pragma unroll
    for (int jj = 0; jj < kB; ++jj) {
      // Columns past m have clip scale 0, so g = u = 0 there.
      float mg = 0.0f, mu = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int cl = 32 * jj + 8 * q + 4 * h;  // column within the wave's
        const float4 sg = *reinterpret_cast<const float4*>(&fg_at[cl]);
        const float4 su = *reinterpret_cast<const float4*>(&fu_at[cl]);
        const float kg[4] = {sg.x, sg.y, sg.z, sg.w}, ku[4] = {su.x, su.y, su.z, su.w};
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gv = acc[jj][i][4 * q + e] * (fx * kg[e]);
          const float uv = acc[kB + jj][i][4 * q + e] * (fx * ku[e]);
          y[e] = act_value<kOut == 2>(gv, kAct) * uv;
          if constexpr (kAct8) {
            acc[jj][i][4 * q + e] = gv;
            acc[kB + jj][i][4 * q + e] = uv;
            mg = __builtin_elementwise_maximum(mg, fabsf(gv));  // (NaN stays, as in act8_mag's order)
            mu = __builtin_elementwise_maximum(mu, fabsf(uv));
          }
        }
        uint8_t* d = slab + r32 * kPitch + cl * kOut;
        if constexpr (kOut == 4) {
          *reinterpret_cast<u32x4*>(d) =
              u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
        } else {
          *reinterpret_cast<u32x2*>(d) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        }
      }
      if constexpr (kAct8) {
        // the block's other 16 columns are in lane ^ 32
        ex[0][jj] = static_cast<int>(halves_max(act8_mag(mg)) >> 23);
        ex[1][jj] = static_cast<int>(halves_max(act8_mag(mu)) >> 23);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            code[p][jj][q] = act8_encode4(acc[kB * p + jj][i][4 * q], acc[kB * p + jj][i][4 * q + 1],
                                          acc[kB * p + jj][i][4 * q + 2], acc[kB * p + jj][i][4 * q + 3], ex[p][jj]);
      }
    }
    slab_fence();
#pragma unroll
    for (int t = 0; t < 32 * kLanesPerRow / 64; ++t) {
      const int sr = t * (64 / kLanesPerRow) + lane / kLanesPerRow, sc = (lane % kLanesPerRow) * kPer;
      const int row = row1 + 32 * i + sr, col = wcol + sc;
      const uint8_t* src = slab + sr * kPitch + sc * kOut;
      if constexpr (kVec) {
        const int off = col < m ? (row * m + col) * kOut : kNowhereOff;
        __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(src), rout, off, 0, 0);
      } else if (row < rows_left) {
        store_chunk<Out>(static_cast<Out*>(a.out) + static_cast<int64_t>(row0 + row) * m + col, src, m - col);
      }
    }
    slab_fence();
    if constexpr (kAct8) {
      const int blocks = (m + 31) >> 5;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int jj = 0; jj < kB; ++jj)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint32_t*>(slab + r32 * kPitch + kCodes * p + 32 * jj + 8 * q + 4 * h) = code[p][jj][q];
      slab_fence();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const auto rc = make_rsrc((p ? a.up_codes : a.gate_codes) + static_cast<size_t>(row0) * m,
                                  static_cast<uint32_t>(rows_left) * static_cast<uint32_t>(m));
        const auto re = make_rsrc((p ? a.up_scale : a.gate_scale) + static_cast<size_t>(row0) * blocks,
                                  static_cast<uint32_t>(rows_left) * static_cast<uint32_t>(blocks));
#pragma unroll
        for (int t = 0; t < kB; ++t) {
          const int sr = t * (32 / kB) + lane / (2 * kB), sc = (lane % (2 * kB)) * 16;
          const int row = row1 + 32 * i + sr, col = wcol + sc;
          const uint8_t* src = slab + sr * kPitch + kCodes * p + sc;
          if constexpr (kVec) {
            const int off = col < m ? row * m + col : kNowhereOff;
            __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(src), rc, off, 0, 0);
          } else if (row < rows_left) {
            store_chunk<int8_t>((p ? a.up_codes : a.gate_codes) + static_cast<int64_t>(row0 + row) * m + col, src,
                                m - col);
          }
        }
        // the exponents: with two blocks, the lower lanes the first one's
        const int blk = (wcol >> 5) + (kB == 2 ? h : 0);
        const int e = kB == 2 && h ? ex[p][kB - 1] : ex[p][0];
        __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(e), re,
                                             blk < blocks ? (row1 + 32 * i + r32) * blocks + blk : kNowhereOff, 0, 0);
      }
      slab_fence();
    }
  }
}

// kS: groups of 4 waves that share the tile, group g taking every kS-th stage from g,
// in stage buffers of its own; their exact sums are added at the end.
template <typename Out, int kB, int kS, bool kVec, bool kAct8, int kAct>
__global__ void __launch_bounds__(256 * kS, 4 / kB) quest_gated_tiles_kernel(const GatedLaunch a) {
  constexpr int kTile = 64 * kB;             // rows and columns of h of a workgroup
  constexpr int kOpStage = 2 * kB * kBlock;  // one operand's blocks of a stage
  constexpr int kStage = 3 * kOpStage;       // x, gate and up
  constexpr int kSlab = 32 * kSlabPitch<Out, kB>;
  static_assert(4 * kSlab <= 2 * kStage, "the waves' slabs fit the stage buffers");
  static_assert(kS == 1 || kB == 1, "a group's sums fit its stage buffers");
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kS * kStage + 3 * kTile * 4];
  float* const fac = reinterpret_cast<float*>(lds + 2 * kS * kStage);  // clip scales: kTile each of x, gate and up

  const int n = a.n, m = a.m, k = a.k;
  const int tid = threadIdx.x;
  const int group = kS == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid) >> 8;
  const int wave = (__builtin_amdgcn_readfirstlane(tid) >> 6) & 3;  // of the group
  const int wm = wave >> 1, wn = wave & 1;
  const int lane = tid & 63;
  uint8_t* const own = lds + group * 2 * kStage;  // the group's buffers
  auto stage_mem = [&](auto bi) -> uint8_t* { return own + decltype(bi)::value * kStage; };
  const int stages = k >> 7, steps = (stages + kS - 1) / kS;
  const uint32_t rb_bytes = static_cast<uint32_t>(stages) * kBlock;  // one 32-row block, all of k
  const int tiles_m = (n + kTile - 1) / kTile, tiles_n = (m + kTile - 1) / kTile;
  // Workgroups are dealt to the 8 XCDs round-robin; each XCD takes a
  // contiguous range of tiles, whose operand blocks then share its L2.
  int pid = blockIdx.x, tm, tn;
  const int full = static_cast<int>(gridDim.x) & ~7;
  if (pid < full) pid = (pid & 7) * (full >> 3) + (pid >> 3);
  tile_at(pid, tiles_m, tiles_n, tm, tn);
  const int row0 = tm * kTile, col0 = tn * kTile;

  const int rb_x = (n + 31) >> 5, rb_w = (m + 31) >> 5;
  const i32x4 rx =
      raw_rsrc(a.x + static_cast<size_t>(tm) * 2 * kB * rb_bytes, min(rb_x - tm * 2 * kB, 2 * kB) * rb_bytes);
  const uint32_t w_bytes = min(rb_w - tn * 2 * kB, 2 * kB) * rb_bytes;
  const i32x4 rg = raw_rsrc(a.gate + static_cast<size_t>(tn) * 2 * kB * rb_bytes, w_bytes);
  const i32x4 ru = raw_rsrc(a.up + static_cast<size_t>(tn) * 2 * kB * rb_bytes, w_bytes);

  // The clip scales, 64 a load (entries past the end as zeros): kB of each, in turn by the waves.
  auto fetch_scales = [&](int op, const float* src, int left) {
#pragma unroll
    for (int v = 0; v < kB; ++v) {
      if (((op * kB + v) & 3) != wave) continue;
      const int first = 64 * v;
      const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(fac + op * kTile + first));
      dma4(__builtin_amdgcn_readfirstlane(to), lane * 4,
           raw_rsrc(src + first, __builtin_amdgcn_readfirstlane(max(min(left - first, 64), 0)) * 4));
    }
  };
  if (group == 0) {
    fetch_scales(0, a.sx + row0, n - row0);
    fetch_scales(1, a.sg + col0, m - col0);
    fetch_scales(2, a.su + col0, m - col0);
  }

  // Stage st into LDS: 6 kB wave instructions for each operand, spread over the
  // waves (for kB = 1, where they are one and a half a wave, from another wave on
  // for each operand).  A stage past the last, which some groups' last step has,
  // lies outside the windows and is zeros.
  auto fetch_stage = [&](int step, auto bi) {
    const int st = step * kS + group;
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(stage_mem(bi)));
    auto fetch_operand = [&](int op, i32x4 rsrc) {
#pragma unroll
      for (int v = 0; v < (6 * kB + 3) / 4; ++v) {
        const int t = ((wave + 2 * op) & 3) + 4 * v;
        if (6 * kB % 4 == 0 || t < 6 * kB) {
          const int blk = t / 3, part = t % 3;
          const int at = blk * static_cast<int>(rb_bytes) + st * kBlock + part * 1024 + lane * 16;
          const int off = kS == 1 || st < stages ? at : kNowhereOff;
          dma16(__builtin_amdgcn_readfirstlane(base + op * kOpStage + blk * kBlock + part * 1024), off, rsrc);
        }
      }
    };
    fetch_operand(0, rx);
    fetch_operand(1, rg);
    fetch_operand(2, ru);
  };
  // Fragment (block rbk of x (op 0), gate (1) or up (2), k-half ks): this lane's 24 bytes.
  auto frag = [&](auto bi, int op, int rbk, int ks) -> v8i {
    const u32x2* s =
        reinterpret_cast<const u32x2*>(stage_mem(bi) + op * kOpStage + rbk * kBlock + ks * kFrag + lane * 24);
    const u32x2 x0 = s[0], x1 = s[1], x2 = s[2];
    return v8i{static_cast<int>(x0[0]), static_cast<int>(x0[1]), static_cast<int>(x1[0]),
               static_cast<int>(x1[1]), static_cast<int>(x2[0]), static_cast<int>(x2[1]), 0, 0};
  };

  fetch_stage(0, I0{});
  v16f acc[2 * kB][kB];
#pragma unroll
  for (int j = 0; j < 2 * kB; ++j)
#pragma unroll
    for (int i = 0; i < kB; ++i) acc[j][i] = v16f{};
  // One stage: bi holds it; the other buffer held the stage before, whose reads
  // every wave finished before the barrier, and receives the next one.
  auto step = [&](int s, auto bi, auto bn) {
    wait_vmcnt<0>();  // this wave's part of stage s has landed (it had a stage's time)
    lds_barrier();
    if (s + 1 < steps) fetch_stage(s + 1, bn);
    v8i fx[2][kB], fw[2][2 * kB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < kB; ++i) fx[h][i] = frag(bi, 0, wm * kB + i, h);
#pragma unroll
      for (int j = 0; j < 2 * kB; ++j) fw[h][j] = frag(bi, 1 + j / kB, wn * kB + j % kB, h);
    }
    // A wave at its products goes before one at its loads or its epilogue (16384 x 2048 ->
    // 5632: 261.1 to 259.7 us, with checkpoints 300.2 to 297.2).
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2 * kB; ++j)
#pragma unroll
        for (int i = 0; i < kB; ++i)
          acc[j][i] =
              __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[h][j], fx[h][i], acc[j][i], 2, 2, 0, 127, 0, 127);
    __builtin_amdgcn_s_setprio(0);
  };
  // Delta's factors, once for all (between the first barrier and the last).
  auto delta = [&]() {
    for (int t = tid; t < 3 * kTile; t += 256 * kS) fac[t] *= t < kTile ? a.kx : a.kw;
  };
  int s = 0;
  for (; s + 2 <= steps; s += 2) {
    step(s, I0{}, I1{});
    if (s == 0) delta();
    step(s + 1, I1{}, I0{});
  }
  if (s < steps) step(s, I0{}, I1{});
  if (steps == 1) delta();
  lds_barrier();  // every wave's reads are done before the buffers are reused
  if constexpr (kS > 1) {
    typedef float v4f __attribute__((ext_vector_type(4)));
    v4f* const sums = reinterpret_cast<v4f*>(lds) + (tid & 255);  // [group][2 kB * kB * 4][256]
    constexpr int kQuads = 2 * kB * kB * 4;
    static_assert(kQuads * 256 * 16 <= 2 * kStage, "a group's sums fit its stage buffers");
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < 2 * kB; ++j)
#pragma unroll
        for (int i = 0; i < kB; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sums[(group * kQuads + (j * kB + i) * 4 + q) * 256] =
                v4f{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
    }
    lds_barrier();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < kS; ++g)
#pragma unroll
      for (int j = 0; j < 2 * kB; ++j)
#pragma unroll
        for (int i = 0; i < kB; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v4f v = sums[(g * kQuads + (j * kB + i) * 4 + q) * 256];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][i][4 * q + e] += v[e];
          }
  }

  gated_epilogue<Out, kB, kVec, kAct8, kAct>(a, acc, fac + wm * 32 * kB, fac + kTile + wn * 32 * kB,
                                             fac + 2 * kTile + wn * 32 * kB, lds + wave * kSlab, row0, wm * 32 * kB,
                                             min(n - row0, kTile), col0 + wn * 32 * kB, lane);
}

// Few rows (a decode step): the weights are the work, each read once.  A workgroup takes
// 16 kCt columns of h and all n <= 16 kT rows; its 8 waves take every 8th chunk
// of 128 of k, straight from memory into the operand registers of the 16 x 16 x
// 128 instruction (lane l: row l % 16, run l / 16 of the chunk, 24 bytes), and
// add their exact sums through LDS.  kCt is 1, which gives the most workgroups,
// or 2 where the 8-bit checkpoints need blocks of 32 columns in one place.
// Bound by the latency of one pass over the weights: 1 x 2048 -> 5632 takes 5.4 us, 48
// rows 7.2 (7.8 with 64 x 64 tiles, whatever the rows), 17.4 MB.
typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kFewWaves = 8;

__device__ __forceinline__ v8i load_run(const uint8_t* p) {
  typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
  const u32x4_a8 lo = *reinterpret_cast<const u32x4_a8*>(p);
  const u32x2 hi = *reinterpret_cast<const u32x2*>(p + 16);
  return v8i{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
             static_cast<int>(hi[0]), static_cast<int>(hi[1]), 0, 0};
}

template <typename Out, int kT, int kCt, bool kAct8>
__global__ void __launch_bounds__(64 * kFewWaves) quest_gated_few_kernel(const GatedLaunch a) {
  constexpr int kCols = 16 * kCt, kTile = 16 * kT * kCols;  // outputs of a workgroup
  __shared__ __attribute__((aligned(16))) float part[kFewWaves][2][kTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int n = a.n, m = a.m, chunks = a.k >> 7;
  const int64_t rb_bytes = static_cast<int64_t>(chunks) * kBlock;
  const int col0 = blockIdx.x * kCols;
  // Byte of run l / 16 of chunk 0 of operand row r.
  auto run_at = [&](int r) -> int64_t {
    const int j = lane >> 4;
    return (r >> 5) * rb_bytes + (j >> 1) * kFrag + (32 * (j & 1) + (r & 31)) * 24;
  };
  const uint8_t* px[kT];
  const uint8_t* pw[2][kCt];
#pragma unroll
  for (int t = 0; t < kT; ++t) px[t] = a.x + run_at(min(16 * t + (lane & 15), n - 1));  // rows past n: the last again
#pragma unroll
  for (int c = 0; c < kCt; ++c) {
    const int64_t at = run_at(col0 + 16 * c + (lane & 15));
    pw[0][c] = a.gate + at;
    pw[1][c] = a.up + at;
  }
  v4f acc[2][kCt][kT];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int c = 0; c < kCt; ++c)
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[p][c][t] = v4f{};
  v8i fw[2][kCt], fx[kT];
  auto fetch_chunk = [&](int ch) {
    const int64_t off = static_cast<int64_t>(ch) * kBlock;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int c = 0; c < kCt; ++c) fw[p][c] = load_run(pw[p][c] + off);
#pragma unroll
    for (int t = 0; t < kT; ++t) fx[t] = load_run(px[t] + off);
  };
  if (wave < chunks) fetch_chunk(wave);
  for (int ch = wave; ch < chunks; ch += kFewWaves) {
    v8i w[2][kCt], x[kT];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int c = 0; c < kCt; ++c) w[p][c] = fw[p][c];
#pragma unroll
    for (int t = 0; t < kT; ++t) x[t] = fx[t];
    if (ch + kFewWaves < chunks) fetch_chunk(ch + kFewWaves);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int c = 0; c < kCt; ++c)
          acc[p][c][t] =
              __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[p][c], x[t], acc[p][c][t], 2, 2, 0, 127, 0, 127);
  }
  // lane l has row 16 t + l % 16 and columns 16 c + 4 (l / 16) .. + 3
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int c = 0; c < kCt; ++c)
#pragma unroll
      for (int t = 0; t < kT; ++t)
        *reinterpret_cast<v4f*>(&part[wave][p][(16 * t + (lane & 15)) * kCols + 16 * c + 4 * (lane >> 4)]) =
            acc[p][c][t];
  __syncthreads();
  const int blocks = (m + 31) >> 5;
  for (int o = tid; o < kTile; o += 64 * kFewWaves) {
    const int row = o / kCols, col = col0 + o % kCols;
    if (!kAct8 && (row >= n || col >= m)) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      g += part[w][0][o];
      u += part[w][1][o];
    }
    const bool in = row < n && col < m;
    if (in) {
      const float fx = a.sx[row] * a.kx;
      g *= fx * (a.sg[col] * a.kw);
      u *= fx * (a.su[col] * a.kw);
      static_cast<Out*>(a.out)[static_cast<int64_t>(row) * m + col] =
          from_f32<Out>(act_value<sizeof(Out) == 2>(g, a.act) * u);
    }
    if constexpr (kAct8) {  // a half wave is a row's block of 32 columns
      const int eg = static_cast<int>(half_wave_max(in ? act8_mag(g) : 0u) >> 23);
      const int eu = static_cast<int>(half_wave_max(in ? act8_mag(u) : 0u) >> 23);
      if (in) {
        const int64_t at = static_cast<int64_t>(row) * m + col, se = static_cast<int64_t>(row) * blocks + (col >> 5);
        a.gate_codes[at] = static_cast<int8_t>(act8_encode(g, eg));
        a.up_codes[at] = static_cast<int8_t>(act8_encode(u, eu));
        if ((lane & 31) == 0) {
          a.gate_scale[se] = static_cast<uint8_t>(eg);
          a.up_scale[se] = static_cast<uint8_t>(eu);
        }
      }
    }
  }
}

// Backward: 8 columns a thread, a row a workgroup at a time.  kGroups: rows of a
// whole number of groups of 8 (2), others of 8 columns and more (1: unaligned, the
// last group ending with the row, see Group), narrower ones (0).  A streaming
// kernel: 8.06 bytes an entry in bf16; 16384 x 5632 takes 136 to 154 us, 4.8 to 5.5
// TB/s (fp32 259).  Rows under some 2000 columns leave part of their workgroup idle:
// 16384 x 1024 22 us, x 256 12, x 20 10.
template <typename T, int kGroups, int kAct>
__global__ void __launch_bounds__(256) quest_gated_bwd_kernel(const GatedBwdLaunch a) {
  const int cols = a.cols, blocks = (cols + kAct8Block - 1) / kAct8Block;
  constexpr bool kFast = sizeof(T) == 2;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dh = static_cast<const T*>(a.dh) + row * cols;
    const int8_t* gc = a.gate_codes + row * cols;
    const int8_t* uc = a.up_codes + row * cols;
    const uint8_t* gs = a.gate_scale + row * blocks;
    const uint8_t* us = a.up_scale + row * blocks;
    T* dg = static_cast<T*>(a.out) + row * 2 * cols;
    T* du = dg + cols;
    for (int c = threadIdx.x * 8; c < cols; c += 256 * 8) {
      const Group at(kGroups == 1 ? c : 0, kGroups == 1 ? cols : 8);
      float d[8], g[8], u[8];
      uint2 wg, wu;
      if constexpr (kGroups == 2) {
        load8(dh + c, d);
        wg = *reinterpret_cast<const uint2*>(gc + c);
        wu = *reinterpret_cast<const uint2*>(uc + c);
      } else if constexpr (kGroups == 1) {
        load8_at(dh + at.at, d);
        wg = load_codes8_at(gc + at.at);
        wu = load_codes8_at(uc + at.at);
      } else {
        load8_tail(dh + c, cols - c, d);
        wg = load_codes8_tail(gc + c, cols - c);
        wu = load_codes8_tail(uc + c, cols - c);
      }
      act8_decode8(wg, gs[c >> 5], g);
      act8_decode8(wu, us[c >> 5], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float value, slope;
        act_both<kFast>(g[i], kAct, value, slope);
        g[i] = d[i] * u[i] * slope;
        u[i] = d[i] * value;
      }
      if constexpr (kGroups == 2) {
        store8(dg + c, g);
        store8(du + c, u);
      } else if constexpr (kGroups == 1) {
        store8_own(dg + at.at, at, g);
        store8_own(du + at.at, at, u);
      } else {
        store8_tail(dg + c, cols - c, g);
        store8_tail(du + c, cols - c, u);
      }
    }
  }
}

template <typename Out, int kB, int kS, bool kVec>
hipError_t launch_tiles(const GatedLaunch& g) {
  constexpr int kTile = 64 * kB;
  const dim3 grid(((g.n + kTile - 1) / kTile) * ((g.m + kTile - 1) / kTile)), block(256 * kS);
  if (g.gate_codes && g.act == 0)
    hipLaunchKernelGGL((quest_gated_tiles_kernel<Out, kB, kS, kVec, true, 0>), grid, block, 0, g.stream, g);
  else if (g.gate_codes)
    hipLaunchKernelGGL((quest_gated_tiles_kernel<Out, kB, kS, kVec, true, 1>), grid, block, 0, g.stream, g);
  else if (g.act == 0)
    hipLaunchKernelGGL((quest_gated_tiles_kernel<Out, kB, kS, kVec, false, 0>), grid, block, 0, g.stream, g);
  else
    hipLaunchKernelGGL((quest_gated_tiles_kernel<Out, kB, kS, kVec, false, 1>), grid, block, 0, g.stream, g);
  return hipGetLastError();
}

template <typename Out, bool kVec>
hipError_t launch_tiles(const GatedLaunch& g) {
  const int cus = device_cus();
  const int large = ((g.n + 127) / 128) * ((g.m + 127) / 128), small = ((g.n + 63) / 64) * ((g.m + 63) / 64);
  // 64 x 64 tiles until the larger ones are a round and a quarter (2048 -> 5632, us): 512
  // rows, 176 larger tiles, 14.4 against 16.1; 700, 264, 19.2 and 21.0; 1024, 352, 27.1 and 25.4.
  if (4 * large >= 5 * cus) return launch_tiles<Out, 2, 1, kVec>(g);
  // Long sums in few tiles are shared by four groups of waves: 357 x 7424 -> 1792 18.6
  // against 27.5, 1365 x 8064 -> 256 19.4 and 29.3, but 128 x 2048 -> 5632 8.2 and 8.0.
  if (small <= cus && g.k >= 4096) return launch_tiles<Out, 1, 4, kVec>(g);
  return launch_tiles<Out, 1, 1, kVec>(g);
}

template <typename Out, int kT>
hipError_t launch_few(const GatedLaunch& g) {
  const dim3 block(64 * kFewWaves);
  if (g.gate_codes)
    hipLaunchKernelGGL((quest_gated_few_kernel<Out, kT, 2, true>), dim3((g.m + 31) / 32), block, 0, g.stream, g);
  else
    hipLaunchKernelGGL((quest_gated_few_kernel<Out, kT, 1, false>), dim3((g.m + 15) / 16), block, 0, g.stream, g);
  return hipGetLastError();
}

template <typename Out>
hipError_t launch_fwd(const GatedLaunch& g) {
  if (g.n <= 16) return launch_few<Out, 1>(g);
  if (g.n <= 32) return launch_few<Out, 2>(g);
  if (g.n <= 64) return launch_few<Out, 4>(g);
  // Rows whose chunks of 16 codes and of 16 bytes of output start on 16 bytes.
  return g.m % 16 == 0 ? launch_tiles<Out, true>(g) : launch_tiles<Out, false>(g);
}

template <typename T, int kGroups>
hipError_t launch_bwd(const GatedBwdLaunch& a) {
  const dim3 grid(static_cast<uint32_t>(a.rows < (1 << 20) ? a.rows : (1 << 20)));
  if (a.act == 0)
    hipLaunchKernelGGL((quest_gated_bwd_kernel<T, kGroups, 0>), grid, dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL((quest_gated_bwd_kernel<T, kGroups, 1>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_bwd(const GatedBwdLaunch& a) {
  return a.cols % 8 == 0 ? launch_bwd<T, 2>(a) : a.cols > 8 ? launch_bwd<T, 1>(a) : launch_bwd<T, 0>(a);
}

}  // namespace

hipError_t launch_gated_fwd(const GatedLaunch& g, bool out_bf16) {
  return out_bf16 ? launch_fwd<uint16_t>(g) : launch_fwd<float>(g);
}

hipError_t launch_gated_bwd(const GatedBwdLaunch& a, bool bf16) {
  return bf16 ? launch_bwd<uint16_t>(a) : launch_bwd<float>(a);
}

}  // namespace quest
