// A whole mixture-of-experts layer for a few tokens, on quantised weights.
//
//   y_t = sum over the experts e that token t takes of p_te Q(h_te) Q(down_e)^T,
//   h_te = act(Q(x_t) Q(gate_e)^T) * (Q(x_t) Q(up_e)^T),
// where a token takes the top_k experts with the largest logits (of equal ones the
// lowest index) and p is the softmax over those, or over all.  Products are sums of
// whole numbers (quest_few.h): T = sum (2 a + 1)(2 b + 1) exact, a product
// D_a D_b T / 4 as quest_gemm_i8's.  h stays in fp32 and is quantised to h_bits
// by the kernel of quest_quantize_fwd_i8.
//
// With few tokens the chosen experts' weights are the work, and each is read once.
// The grids count the most experts that can be chosen ("slots", min(experts, n top_k)),
// since the choice is known on the device only.  Kernels:
//   route    one workgroup: each token's experts and their weights; each slot's expert
//            and its tokens;
//   gated    (some tiles of 16 columns of h, slot): h goes to the workspace, a row for
//            each token and rank of the expert among the token's;
//   (h is quantised)
//   down     (some tiles of 32 output columns, slot): the same of h's codes by down;
//   combine  the top_k products of each token, weighted, in the order of their rank.
// No atomics on results: the sums' order is fixed.  The workspace need not be set.
// (With the choice found by every workgroup of gated and down instead of the first
// kernel, their code is some 20 KB, and one token's gated kernel took 17.5 us.)
#include <type_traits>

#include "quest_device.h"
#include "quest_few.h"
#include "quest_launch.h"

namespace quest {
namespace {

constexpr int kSets = kMoeMaxExperts / 64;  // of 64 experts
constexpr int kWaves = 8;
constexpr float kNone = -__builtin_inff();

// A workgroup barrier that waits for this wave's LDS accesses only: loads of weights
// stay in flight across it (a __syncthreads waits for them).
__device__ __forceinline__ void lds_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A token's logits as they lie in memory, expert 64 i + lane in raw[i] (past the last:
// the last again).  Kept apart from their use, so that several tokens' loads overlap.
__device__ __forceinline__ void fetch_logits(const MoeLaunch& a, int t, int lane, uint32_t (&raw)[kSets]) {
  const int64_t row = static_cast<int64_t>(t) * a.experts;
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    raw[i] = 0;
    if (64 * i < a.experts) {
      const int64_t at = row + min(64 * i + lane, a.experts - 1);
      if (a.logits_bf16)
        raw[i] = static_cast<const uint16_t*>(a.logits)[at];
      else
        raw[i] = static_cast<const uint32_t*>(a.logits)[at];
    }
  }
}

// Their values: -inf past the last expert, and for NaN (which no comparison finds; the
// combining kernel gives NaN for such a token).  Returns whether the lane saw a NaN.
__device__ __forceinline__ bool decode_logits(const MoeLaunch& a, int lane, const uint32_t (&raw)[kSets],
                                              float (&v)[kSets]) {
  const int shift = a.logits_bf16 ? 16 : 0;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const float f = __uint_as_float(raw[i] << shift);
    nan |= f != f;
    v[i] = 64 * i + lane < a.experts && f == f ? f : kNone;
  }
  return nan;
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float x) {
  return fmaxf(x, dpp_read<CTRL>(x));
}

// The largest of all lanes' (no NaN among them), the same in every lane.
__device__ __forceinline__ float wave_max(float x) {
  x = dpp_max<0xB1>(x);
  x = dpp_max<0x4E>(x);
  x = dpp_max<0x141>(x);
  x = dpp_max<0x140>(x);  // every lane of a row of 16 has the row's
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 16 * i));
  return fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
}

__device__ __forceinline__ float max_of(const float (&v)[kSets]) {
  return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
}

// Takes the largest logit (of equal ones the lowest index) out of v: its expert, or -1.
__device__ __forceinline__ int take_largest(float (&v)[kSets], int lane, float& value) {
  value = wave_max(max_of(v));
  if (value == kNone) return -1;
  int e = -1;
#pragma unroll
  for (int i = kSets - 1; i >= 0; --i) {
    const uint64_t at = __builtin_amdgcn_ballot_w64(v[i] == value);
    if (at) e = 64 * i + __builtin_ctzll(at);
  }
#pragma unroll
  for (int i = 0; i < kSets; ++i)
    if (64 * i + lane == e) v[i] = kNone;
  return e;
}

constexpr int kRouteWaves = 16, kEach = kMoeMaxTokens / kRouteWaves;  // tokens a wave
__global__ void __launch_bounds__(64 * kRouteWaves) quest_moe_route_kernel(const MoeLaunch a) {
  __shared__ uint32_t takes[kMoeMaxExperts][2];  // a bit for each token that takes the expert
  __shared__ uint8_t rank[kMoeMaxTokens][kMoeMaxExperts];
  __shared__ int before[kSets + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  uint32_t raw[kEach][kSets];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i * kRouteWaves < a.n) fetch_logits(a, min(wave + i * kRouteWaves, a.n - 1), lane, raw[i]);
  if (tid < 2 * kMoeMaxExperts) takes[tid >> 1][tid & 1] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = wave + i * kRouteWaves;
    if (t >= a.n) break;
    float v[kSets];
    const bool nan = __builtin_amdgcn_ballot_w64(decode_logits(a, lane, raw[i], v)) != 0;
    const float largest = wave_max(max_of(v));
    // No product of a token with a NaN or +infinity is used: its output is NaN.
    const bool undefined = nan || largest == __builtin_inff();
    float all = 0.0f;
    if (a.over_all)
#pragma unroll
      for (int j = 0; j < kSets; ++j) all += v[j] == kNone ? 0.0f : expf(v[j] - largest);
    int found = 0;
    float own = 0.0f;  // lane r: the exponential of the expert of rank r
    for (; found < a.top && !undefined; ++found) {
      float value;
      const int e = take_largest(v, lane, value);
      if (e < 0) break;
      if (lane == 0) {
        atomicOr(&takes[e][t >> 5], 1u << (t & 31));
        rank[t][e] = static_cast<uint8_t>(found);
      }
      if (lane == found) own = expf(value - largest);
    }
    const float sum = group_sum(a.over_all ? all : own, 6);
    if (lane < found) a.weight[t * a.top + lane] = own / sum;
    if (lane == 0) a.found[t] = undefined ? -1 : found;
  }
  __syncthreads();
  // Thread e < 256: expert e's slot is the number of chosen experts before it.
  uint64_t mine = 0;
  int below = 0;
  if (tid < kMoeMaxExperts) {
    mine = takes[tid][0] | static_cast<uint64_t>(takes[tid][1]) << 32;
    const uint64_t used = __builtin_amdgcn_ballot_w64(mine != 0);
    below = __builtin_popcountll(used & ((uint64_t(1) << lane) - 1));
    if (lane == 0) before[wave] = __builtin_popcountll(used);
  }
  __syncthreads();
  if (tid >= kMoeMaxExperts) return;
  int total = 0;
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    if (i < wave) below += before[i];
    total += before[i];
  }
  if (tid == 0) *a.active = total;
  if (mine) {
    MoeSlot& s = a.slot[below];
    s.expert = tid;
    s.count = __builtin_popcountll(mine);
    for (int i = 0; mine; ++i, mine &= mine - 1) {
      const int t = __builtin_ctzll(mine);
      s.entry[i] = static_cast<uint16_t>(t | rank[t][tid] << 8);
    }
  }
}

template <int kAct>
__device__ __forceinline__ float activation(float g) {
  if constexpr (kAct == 0) return g / (1.0f + expf(-g));
  return g * (0.5f * erfcf(g * -0.70710678f));
}

// Products of one slot's tokens by its expert's rows, T groups of 16 tokens at a time:
// gated (a tile is 16 columns of h: a strip of 16 rows of gate and one of up) or down
// (32 columns: two strips).  KS waves share a tile, taking every KS-th chunk of the
// contraction, and the workgroup's 8 / KS tiles at a time make one step of its walk.
// The tokens' codes lie in LDS in the order of the fragments; where they do not fit
// (`segment` chunks at a time), they are brought again for every step.  A wave's loads of
// weights go straight to its registers and run kAhead chunks ahead, into its next tile:
// with KS = 1 no wave waits for another.
// kMode: kDown, or the gated product's activation.
constexpr int kDown = -1;
template <bool kPacked, int T, int KS, int kMode>
__global__ void __launch_bounds__(64 * kWaves) quest_moe_product_kernel(const MoeLaunch a, int segment) {
  constexpr bool kGated = kMode != kDown;
  constexpr int F = kFewFrags<kPacked>, kChunk = kFewChunk<kPacked>, kAhead = 4;
  constexpr int kCols = kGated ? 16 : 32, kTiles = kWaves / KS;
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];
  __shared__ uint16_t entries[kMoeMaxTokens];
  __shared__ __attribute__((aligned(16))) uint32_t part[KS > 1 ? kWaves : 1][2][KS > 1 ? T * 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6, ks = wave % KS;
  const int len = kGated ? a.k : a.m, rows = kGated ? a.m : a.k;
  const int tiles = rows / kCols, chunks = (len + kChunk - 1) / kChunk;
  const int segments = (chunks + segment - 1) / segment, pitch = segment * kChunk + 16;
  const int64_t row_bytes = kPacked ? len / 2 : len;
  if (static_cast<int>(blockIdx.y) >= *a.active) return;
  const MoeSlot& slot = a.slot[blockIdx.y];
  const int e = slot.expert, count = slot.count;
  if (tid < count) entries[tid] = slot.entry[tid];
  const int64_t first = (static_cast<int64_t>(e) * rows + (lane & 15)) * row_bytes;
  const uint8_t* const wide[2] = {(kGated ? a.gate : a.down) + first,
                                  kGated ? a.up + first : a.down + first + 16 * row_bytes};
  // Lanes of the last chunk's upper half may lie past the row: they read its first bytes
  // and count as zeros.
  const bool short_end = kPacked && (len & 127) != 0 && (lane & 32);
  const int mine = (chunks - ks + KS - 1) / KS;             // the wave's chunks ks, ks + KS, ...
  const int steps = (mine + kAhead - 1) / kAhead * kAhead;  // in whole rounds of the ring
  const int stride = gridDim.x * kTiles;
  v4i w[kAhead][2];
  auto load = [&](int tile, int i, v4i (&to)[2]) {
    if (i < mine && tile < tiles) {
      const int chunk = ks + i * KS;
      const int64_t off = static_cast<int64_t>(tile) * kCols * row_bytes + chunk * 64 +
                          (short_end && chunk == chunks - 1 ? 0 : 16 * g);
      to[0] = load_v4i(wide[0] + off);
      to[1] = load_v4i(wide[1] + off);
    }
  };
  int tile = blockIdx.x * kTiles + wave / KS;
  auto begin = [&]() {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(tile, i, w[i]);
  };
  begin();
  lds_sync();
  for (int t0 = 0; t0 < count; t0 += 16 * T) {
    const int here = min(count - t0, 16 * T);
    // Codes of chunks segment s on, 32 columns a thread at a time; columns past the row as zeros.
    auto stage = [&](int s) {
      const int blocks = min(segment, chunks - s * segment) * (kChunk / 32);
      for (int j = tid; j < here * blocks; j += 64 * kWaves) {
        const int i = j / blocks, c = (j - i * blocks) * 32, col = s * segment * kChunk + c;
        const int entry = entries[t0 + i];
        const uint8_t* x = kGated ? a.x + static_cast<int64_t>(entry & 255) * len
                                  : a.hc + (static_cast<int64_t>(entry & 255) * a.top + (entry >> 8)) * len;
        v4i v[2] = {};
        if (col < len) v[0] = load_v4i(x + col), v[1] = load_v4i(x + col + 16);
        if constexpr (kPacked) {
          TokenBytes<true> b{{v[0], v[1]}};
          token_frags<true>(b, v);
        }
        v4i* to = reinterpret_cast<v4i*>(codes + i * pitch + c);
        to[0] = v[0], to[1] = v[1];
      }
    };
    if (t0 > 0) {
      tile = blockIdx.x * kTiles + wave / KS;
      begin();
      lds_sync();  // the last group's codes have been read
    }
    stage(0);
    lds_sync();
    // (every wave makes the same steps: those without a tile only wait with the others)
    for (int base = blockIdx.x * kTiles; base < tiles; base += stride, tile += stride) {
      FewSums<kPacked, 2, T> s;
      for (int seg = 0; seg < segments; ++seg) {
        if (segments > 1 && (seg > 0 || base != static_cast<int>(blockIdx.x) * kTiles)) {
          lds_sync();
          stage(seg);
          lds_sync();
        }
        const int last = seg + 1 < segments ? (seg + 1) * (segment / KS) : steps;
        for (int i0 = seg * (segment / KS); i0 < last; i0 += kAhead) {
#pragma unroll
          for (int r = 0; r < kAhead; ++r) {
            const int i = i0 + r, chunk = ks + i * KS;
            if (i < mine && tile < tiles) {
              const bool off = short_end && chunk == chunks - 1;
              v4i fw[2][F];
#pragma unroll
              for (int p = 0; p < 2; ++p) wide_frags<kPacked>(off ? v4i{} : w[r][p], fw[p]);
              const uint8_t* x = codes + (lane & 15) * pitch + (chunk - seg * segment) * kChunk + (kChunk / 4) * g;
#pragma unroll
              for (int f = 0; f < F; ++f) {
#pragma unroll
                for (int t = 0; t < T; ++t) {
                  const v4i fx = load_v4i(x + 16 * t * pitch + 16 * f);
#pragma unroll
                  for (int p = 0; p < 2; ++p) s.acc[p][t] = mfma_i8(fw[p][f], fx, s.acc[p][t]);
                  s.token[t] = mfma_i8(ones_i8(), fx, s.token[t]);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) s.wide[p] = mfma_i8(fw[p][f], ones_i8(), s.wide[p]);
              }
            }
            if (i + kAhead < steps)
              load(tile, i + kAhead, w[r]);
            else
              load(tile + stride, i + kAhead - steps, w[r]);
          }
        }
      }
      // Four consecutive columns of a token: T_p of the strips to outputs.
      auto finish = [&](int p, int i, int tile_, int c, v4u sum0, v4u sum1) {
        const int entry = entries[t0 + i], row = (entry & 255) * a.top + (entry >> 8);
        const int col = tile_ * kCols + 16 * p + c;
        const int64_t ws = static_cast<int64_t>(e) * rows + col;
        const uint32_t add = few_constant<kPacked>(len);
        float y[4];
        if constexpr (kGated) {
          const float x_step = a.sx[entry & 255] * a.kx;
          const float4 sg = *reinterpret_cast<const float4*>(a.sg + ws), su = *reinterpret_cast<const float4*>(a.su + ws);
          const float fg[4] = {sg.x, sg.y, sg.z, sg.w}, fu[4] = {su.x, su.y, su.z, su.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float gv = (static_cast<float>(static_cast<int>(sum0[q] + add)) * 0.25f) * (x_step * (fg[q] * a.kw));
            const float uv = (static_cast<float>(static_cast<int>(sum1[q] + add)) * 0.25f) * (x_step * (fu[q] * a.kw));
            y[q] = activation<kMode>(gv) * uv;
          }
        } else {
          const float x_step = a.hs[row] * a.kh;
          const float4 sd = *reinterpret_cast<const float4*>(a.sd + ws);
          const float fd[4] = {sd.x, sd.y, sd.z, sd.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            y[q] = (static_cast<float>(static_cast<int>(sum0[q] + add)) * 0.25f) * (x_step * (fd[q] * a.kw));
        }
        float* to = (kGated ? a.h : a.y) + static_cast<int64_t>(row) * rows + col;
        *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
      };
      if constexpr (KS == 1) {
        if (tile < tiles)
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const int i = 16 * t + (lane & 15);
            if (i < here) {
              finish(0, i, tile, 4 * g, s.total(0, t), s.total(1, t));
              if (!kGated) finish(1, i, tile, 4 * g, s.total(1, t), v4u{});
            }
          }
      } else {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int t = 0; t < T; ++t)
            *reinterpret_cast<v4u*>(&part[wave][p][(16 * t + (lane & 15)) * 16 + 4 * g]) = s.total(p, t);
        lds_sync();
        // Quads of the step's outputs: tile, (down: strip,) token, 4 columns.
        constexpr int kStrips = kGated ? 1 : 2;
        for (int o = tid; o < kTiles * kStrips * T * 64; o += 64 * kWaves) {
          const int q = o % (T * 64), p = kGated ? 0 : o / (T * 64) % 2, of = o / (T * 64 * kStrips);
          const int i = q / 4;
          if (i >= here || base + of >= tiles) continue;
          v4u sum0 = {}, sum1 = {};
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            sum0 += *reinterpret_cast<const v4u*>(&part[of * KS + j][p][4 * q]);
            if (kGated) sum1 += *reinterpret_cast<const v4u*>(&part[of * KS + j][1][4 * q]);
          }
          finish(p, i, base + of, 4 * (q % 4), sum0, sum1);
        }
        lds_sync();
      }
    }
  }
}

// Four columns a thread: the products of a token's experts, weighted, in the order of
// their rank.
template <typename Out>
__global__ void __launch_bounds__(256) quest_moe_combine_kernel(const MoeLaunch a) {
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.k) return;
  const int found = a.found[t];
  float y[4] = {};
  const float* part = a.y + static_cast<int64_t>(t) * a.top * a.k + c;
  for (int r = 0; r < found; ++r) {
    const float p = a.weight[t * a.top + r];
    const float4 w = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(r) * a.k);
    y[0] = fmaf(p, w.x, y[0]), y[1] = fmaf(p, w.y, y[1]), y[2] = fmaf(p, w.z, y[2]), y[3] = fmaf(p, w.w, y[3]);
  }
  if (found < 0) y[0] = y[1] = y[2] = y[3] = __builtin_nanf("");
  Out* out = static_cast<Out*>(a.out) + static_cast<int64_t>(t) * a.k + c;
  if constexpr (sizeof(Out) == 2)
    *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  else
    *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
}

template <bool kPacked, int T, int KS, int kMode>
hipError_t launch_product(const MoeLaunch& a, int tiles, int chunks) {
  constexpr int kChunk = kFewChunk<kPacked>, kTiles = kWaves / KS;
  // All chunks at a time if they fit in LDS, else whole rounds of every wave's ring of loads.
  constexpr int kLds = 159 * 1024 - (KS > 1 ? kWaves * 2 * T * 1024 : 0);  // of 160 KB, beside the sums
  constexpr int kFit = (kLds / (16 * T) - 16) / kChunk, kRound = 4 * KS, kMost = kFit / kRound * kRound;
  static_assert(kMost >= kRound, "a segment holds a round");
  int segment = chunks;
  if (chunks > kFit) {
    const int parts = (chunks + kMost - 1) / kMost;
    segment = ((chunks + parts - 1) / parts + kRound - 1) / kRound * kRound;
  }
  const size_t lds = static_cast<size_t>(16 * T) * (segment * kChunk + 16);
  // Workgroups walk tiles, so that finding and bringing the tokens is paid once for
  // several, down to about three workgroups a compute unit.
  const int each = (tiles + kTiles - 1) / kTiles;
  const int walk = static_cast<int>((static_cast<int64_t>(each) * a.slots + 767) / 768);
  hipLaunchKernelGGL((quest_moe_product_kernel<kPacked, T, KS, kMode>), dim3((each + walk - 1) / walk, a.slots),
                     dim3(64 * kWaves), lds, a.stream, a, segment);
  return hipGetLastError();
}

template <bool kPacked, int kMode>
hipError_t launch_products(const MoeLaunch& a) {
  constexpr bool kGated = kMode != kDown;
  // Two groups of 16 tokens at once where an expert has more than 10 on average.
  const bool two = static_cast<int64_t>(a.n) * a.top > 10 * static_cast<int64_t>(a.experts);
  const int tiles = kGated ? a.m / 16 : a.k / 32;
  const int chunks = ((kGated ? a.k : a.m) + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>;
  auto run = [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    return two ? launch_product<kPacked, 2, KS < 8 ? KS : 4, kMode>(a, tiles, chunks)
               : launch_product<kPacked, 1, KS, kMode>(a, tiles, chunks);
  };
  // As few waves a tile as keep some 16 waves a compute unit busy.
  const int64_t waves = static_cast<int64_t>(tiles) * a.slots;
  if (waves >= 4096 || chunks < 2) return run(std::integral_constant<int, 1>{});
  if (waves >= 2048 || chunks < 4) return run(std::integral_constant<int, 2>{});
  if (waves >= 1024 || chunks < 8) return run(std::integral_constant<int, 4>{});
  return run(std::integral_constant<int, 8>{});
}

template <bool kPacked>
hipError_t launch(const MoeLaunch& a, bool out_bf16) {
  hipLaunchKernelGGL(quest_moe_route_kernel, dim3(1), dim3(64 * kRouteWaves), 0, a.stream, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  err = a.act == 0 ? launch_products<kPacked, 0>(a) : launch_products<kPacked, 1>(a);
  if (err != hipSuccess) return err;
  FwdLaunch q;
  q.rows = static_cast<int64_t>(a.n) * a.top;
  q.cols = a.m;
  q.alpha = a.halpha;
  q.trust = 1.0;
  q.allow_mfma = false;
  q.codes = a.hc;
  q.scale = a.hs;
  q.mask = nullptr;
  q.dq = nullptr;
  q.stream = a.stream;
  err = launch_fwd_i8(a.h, 0, a.log_block, a.h_bits, q);
  if (err != hipSuccess) return err;
  err = launch_products<kPacked, kDown>(a);
  if (err != hipSuccess) return err;
  const dim3 grid((a.k + 1023) / 1024, a.n);
  if (out_bf16)
    hipLaunchKernelGGL((quest_moe_combine_kernel<uint16_t>), grid, dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL((quest_moe_combine_kernel<float>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(const MoeLaunch& a, bool packed, bool out_bf16) {
  return packed ? launch<true>(a, out_bf16) : launch<false>(a, out_bf16);
}

}  // namespace quest
