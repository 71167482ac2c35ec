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
// since the choice is known on the device only; every workgroup finds its slot's
// expert and that expert's tokens from the logits.  Kernels:
//   gated    (some tiles of 16 columns of h, slot): the waves share k, sums meet in
//            LDS; h goes to the workspace, a row for each token and expert rank;
//   (h is quantised)
//   down     (some tiles of 32 output columns, slot): the same of h's codes by down;
//   combine  the top_k products of each token, weighted, in the order of their rank.
// No atomics on results: the sums' order is fixed.  The workspace need not be set.
#include <type_traits>

#include "quest_device.h"
#include "quest_few.h"
#include "quest_launch.h"

namespace quest {
namespace {

constexpr int kMaxTokens = 64;   // one wave's lanes
constexpr int kSets = 4;         // 64 experts each: 256 in all
constexpr int kWaves = 8;
constexpr float kNone = -__builtin_inff();

struct List {
  int token[kMaxTokens];  // token | rank << 8 of the slot's expert, in the tokens' order
  int rank_of[kMaxTokens];
  uint32_t chosen[2 * kSets];  // a bit for each expert that some token takes
  int count;
};

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

// How many experts come before e for a token, or -1 where e is none of its first top.
__device__ __forceinline__ int rank_of(const float (&v)[kSets], int e, int top, int lane) {
  float own = kNone;
#pragma unroll
  for (int i = 0; i < kSets; ++i)
    if ((e >> 6) == i) own = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[i]), e & 63));
  int before = 0;
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int j = 64 * i + lane;
    before += __builtin_popcountll(__builtin_amdgcn_ballot_w64(v[i] > own || (v[i] == own && j < e)));
  }
  return own != kNone && before < top ? before : -1;
}

// The slot's expert and its tokens, for a workgroup of kWaves waves; returns the
// expert, or -1 for a slot without one.  Fewer slots than experts: slot s is the
// s-th expert that any token takes; otherwise it is expert s.  A wave looks at up to
// kEach tokens, whose logits it loads together.
constexpr int kEach = kMaxTokens / kWaves;
__device__ __forceinline__ int find_tokens(const MoeLaunch& a, int slot, List& list, int tid) {
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const bool compact = a.slots < a.experts;
  int e = slot;
  float v[kEach][kSets];
  {
    uint32_t raw[kEach][kSets];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i * kWaves < a.n) fetch_logits(a, min(wave + i * kWaves, a.n - 1), lane, raw[i]);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i * kWaves < a.n) decode_logits(a, lane, raw[i], v[i]);
  }
  if (compact) {
    if (tid < 2 * kSets) list.chosen[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (wave + i * kWaves < a.n) {
        float left[kSets];
#pragma unroll
        for (int j = 0; j < kSets; ++j) left[j] = v[i][j];
        for (int r = 0; r < a.top; ++r) {
          float value;
          const int found = take_largest(left, lane, value);
          if (found < 0) break;
          if (lane == 0) atomicOr(&list.chosen[found >> 5], 1u << (found & 31));
        }
      }
    __syncthreads();
    int left = slot;
    e = -1;
#pragma unroll
    for (int w = 0; w < 2 * kSets; ++w) {
      uint32_t bits = __builtin_amdgcn_readfirstlane(list.chosen[w]);
      const int here = __builtin_popcount(bits);
      if (e < 0) {
        if (left < here) {
          for (; left > 0; --left) bits &= bits - 1;
          e = 32 * w + __builtin_ctz(bits);
        } else {
          left -= here;
        }
      }
    }
    if (e < 0) return -1;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (wave + i * kWaves < a.n) {
      const int r = rank_of(v[i], e, a.top, lane);
      if (lane == 0) list.rank_of[wave + i * kWaves] = r;
    }
  __syncthreads();
  if (wave == 0) {
    const int r = lane < a.n ? list.rank_of[lane] : -1;
    const uint64_t takes = __builtin_amdgcn_ballot_w64(r >= 0);
    if (r >= 0) list.token[__builtin_popcountll(takes & ((uint64_t(1) << lane) - 1))] = lane | r << 8;
    if (lane == 0) list.count = __builtin_popcountll(takes);
  }
  __syncthreads();
  return e;
}

__device__ __forceinline__ float activation(float g, int act) {
  if (act == 0) return g / (1.0f + expf(-g));
  return g * (0.5f * erfcf(g * -0.70710678f));
}

// Products of one slot's tokens by its expert's rows, T groups of 16 tokens at a time:
// gated (h of 16 columns a tile, from gate and up) or down (32 columns a tile).  A
// wave takes every 8th chunk of the contraction; its tokens' chunks, up to NC, stay in
// its registers while the workgroup walks tiles tile0, tile0 + gridDim.x, ..., and
// its loads of weights run kAhead chunks ahead, into the next tile.  NC = 0: any
// length, the tokens' chunks read again for every tile.
template <bool kPacked, int T, int NC, bool kGated>
__global__ void __launch_bounds__(64 * kWaves) quest_moe_product_kernel(const MoeLaunch a) {
  constexpr int F = kFewFrags<kPacked>, kChunk = kFewChunk<kPacked>;
  constexpr int kCols = kGated ? 16 : 32;
  __shared__ List list;
  __shared__ __attribute__((aligned(16))) uint32_t part[2][kWaves][2][T * 256];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int e = find_tokens(a, blockIdx.y, list, tid);
  if (e < 0) return;
  const int count = __builtin_amdgcn_readfirstlane(list.count);
  const int len = kGated ? a.k : a.m, rows = kGated ? a.m : a.k;
  const int tiles = rows / kCols, chunks = (len + kChunk - 1) / kChunk;
  const int64_t row_bytes = kPacked ? len / 2 : len;
  const int64_t first = (static_cast<int64_t>(e) * rows + (lane & 15)) * row_bytes;
  const uint8_t* const wide[2] = {(kGated ? a.gate : a.down) + first,
                                  kGated ? a.up + first : a.down + first + 16 * row_bytes};
  // Lanes of the last chunk's upper half may lie past the row: they read its first bytes
  // (at_end) and count as zeros.
  const bool short_end = kPacked && (len & 127) != 0 && (lane & 32);
  const int at = 16 * g, at_end = short_end ? 0 : at;
  int buf = 0;
  for (int t0 = 0; t0 < count; t0 += 16 * T) {
    const uint8_t* xp[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      // (past the last token: the last again, whose sums are not used)
      const int entry = list.token[min(t0 + 16 * t + (lane & 15), count - 1)];
      xp[t] = kGated ? a.x + static_cast<int64_t>(entry & 255) * len
                     : a.hc + (static_cast<int64_t>(entry & 255) * a.top + (entry >> 8)) * len;
    }
    constexpr int kRegs = NC ? NC : 1;
    v4i fx[kRegs][T][F], token[T] = {};
    if constexpr (NC > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int chunk = c * kWaves + wave;
        if (chunk < chunks) {
          const bool off = short_end && chunk == chunks - 1;
#pragma unroll
          for (int t = 0; t < T; ++t) {
            TokenBytes<kPacked> x;
#pragma unroll
            for (int f = 0; f < F; ++f) {
              x.v[f] = load_v4i(xp[t] + chunk * kChunk + (off ? 0 : kChunk / 4 * g) + 16 * f);
              if (off) x.v[f] = v4i{};
            }
            token_frags<kPacked>(x, fx[c][t]);
          }
        }
      }
    }
    constexpr int kAhead = NC == 0 ? 1 : NC < 4 ? NC : 4;
    v4i w[kAhead][2];
    auto load = [&](int tile, int c, v4i (&to)[2]) {
      const int chunk = c * kWaves + wave;
      if (chunk < chunks && tile < tiles) {
        const int64_t off = static_cast<int64_t>(tile) * kCols * row_bytes + chunk * 64 +
                            (chunk == chunks - 1 ? at_end : at);
        to[0] = load_v4i(wide[0] + off);
        to[1] = load_v4i(wide[1] + off);
      }
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(blockIdx.x, i, w[i]);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c * kWaves + wave < chunks)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int f = 0; f < F; ++f) token[t] = mfma_i8(ones_i8(), fx[c][t][f], token[t]);
    }
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      FewSums<kPacked, 2, T> s;
      if constexpr (NC > 0) {
#pragma unroll
        for (int t = 0; t < T; ++t) s.token[t] = token[t];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          constexpr int kMod = kAhead;
          const int chunk = c * kWaves + wave;
          if (chunk < chunks) {
            v4i fw[2][F];
            const bool off = short_end && chunk == chunks - 1;
#pragma unroll
            for (int p = 0; p < 2; ++p) wide_frags<kPacked>(off ? v4i{} : w[c % kMod][p], fw[p]);
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int t = 0; t < T; ++t) s.acc[p][t] = mfma_i8(fw[p][f], fx[c][t][f], s.acc[p][t]);
                s.wide[p] = mfma_i8(fw[p][f], ones_i8(), s.wide[p]);
              }
          }
          if (c + kAhead < NC)
            load(tile, c + kAhead, w[c % kMod]);
          else
            load(tile + gridDim.x, c + kAhead - NC, w[c % kMod]);
        }
      } else {
        const int64_t off = static_cast<int64_t>(tile) * kCols * row_bytes;
        const uint8_t* const wp[2] = {wide[0] + off, wide[1] + off};
        few_run<kPacked, 2, T, 2>(s, wp, xp, wave, kWaves, chunks, len, lane);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < T; ++t)
          *reinterpret_cast<v4u*>(&part[buf][wave][p][(16 * t + (lane & 15)) * 16 + 4 * g]) = s.total(p, t);
      __syncthreads();
      // (the buffer is written again after the next tile's barrier, which follows these reads)
      auto sum = [&](int p, int o) {
        uint32_t v = few_constant<kPacked>(len);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += part[buf][i][p][o];
        return static_cast<float>(static_cast<int>(v)) * 0.25f;
      };
      for (int o = tid; o < (kGated ? 1 : 2) * T * 256; o += 64 * kWaves) {
        const int p = kGated ? 0 : o / (T * 256), q = o % (T * 256);
        const int i = t0 + q / 16, col = tile * kCols + 16 * p + q % 16;
        if (i >= count) continue;
        const int entry = list.token[i], row = (entry & 255) * a.top + (entry >> 8);
        const int64_t ws = static_cast<int64_t>(e) * rows + col;
        if constexpr (kGated) {
          const float fx_ = a.sx[entry & 255] * a.kx;
          const float gv = sum(0, q) * (fx_ * (a.sg[ws] * a.kw)), uv = sum(1, q) * (fx_ * (a.su[ws] * a.kw));
          a.h[static_cast<int64_t>(row) * rows + col] = activation(gv, a.act) * uv;
        } else {
          a.y[static_cast<int64_t>(row) * rows + col] = sum(p, q) * ((a.hs[row] * a.kh) * (a.sd[ws] * a.kw));
        }
      }
      buf ^= 1;
    }
  }
}

// Four columns a thread: the products of a token's experts, weighted, in the order of
// their rank.  Every wave finds the token's weights itself.
template <typename Out>
__global__ void __launch_bounds__(256) quest_moe_combine_kernel(const MoeLaunch a) {
  __shared__ float weight[4][kMoeMaxTop];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x) >> 6;
  const int t = blockIdx.y;
  uint32_t raw[kSets];
  float v[kSets];
  fetch_logits(a, t, lane, raw);
  const bool nan = __builtin_amdgcn_ballot_w64(decode_logits(a, lane, raw, v)) != 0;
  const float largest = wave_max(max_of(v));
  float sum = 0.0f;
  if (a.over_all) {
#pragma unroll
    for (int i = 0; i < kSets; ++i) sum += v[i] == kNone ? 0.0f : expf(v[i] - largest);
    sum = group_sum(sum, 6);
  }
  int found = 0;
  for (; found < a.top; ++found) {
    float value;
    if (take_largest(v, lane, value) < 0) break;
    const float p = expf(value - largest);
    if (!a.over_all) sum += p;
    if (lane == 0) weight[wave][found] = p;
  }
  const float inv = 1.0f / sum;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.k) return;
  float y[4] = {};
  const float* part = a.y + static_cast<int64_t>(t) * a.top * a.k + c;
  for (int r = 0; r < found; ++r) {
    const float p = weight[wave][r] * inv;
    const float4 w = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(r) * a.k);
    y[0] = fmaf(p, w.x, y[0]), y[1] = fmaf(p, w.y, y[1]), y[2] = fmaf(p, w.z, y[2]), y[3] = fmaf(p, w.w, y[3]);
  }
  if (nan) y[0] = y[1] = y[2] = y[3] = __builtin_nanf("");
  Out* out = static_cast<Out*>(a.out) + static_cast<int64_t>(t) * a.k + c;
  if constexpr (sizeof(Out) == 2)
    *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  else
    *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
}

template <bool kPacked, int T, int NC, bool kGated>
hipError_t launch_product(const MoeLaunch& a) {
  const int tiles = kGated ? a.m / 16 : a.k / 32;
  // Workgroups walk tiles so that finding the tokens is paid once for several, down to
  // about four workgroups a compute unit.
  const int64_t total = static_cast<int64_t>(tiles) * a.slots;
  const int walk = static_cast<int>((total + 1023) / 1024);
  hipLaunchKernelGGL((quest_moe_product_kernel<kPacked, T, NC, kGated>), dim3((tiles + walk - 1) / walk, a.slots),
                     dim3(64 * kWaves), 0, a.stream, a);
  return hipGetLastError();
}

template <bool kPacked, bool kGated>
hipError_t launch_products(const MoeLaunch& a) {
  // Two groups of 16 tokens at once where an expert has more than 10 on average.
  const bool two = static_cast<int64_t>(a.n) * a.top > 10 * static_cast<int64_t>(a.experts);
  const int chunks = ((kGated ? a.k : a.m) + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>;
  const int each = (chunks + kWaves - 1) / kWaves;
  auto run = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    if constexpr (!kPacked || NC < 8)  // (two groups' codes of 8192 columns do not fit the registers)
      if (two) return launch_product<kPacked, 2, NC, kGated>(a);
    return launch_product<kPacked, 1, NC, kGated>(a);
  };
  if (each <= 2) return run(std::integral_constant<int, 2>{});
  if (each <= 4) return run(std::integral_constant<int, 4>{});
  if (each <= 8) return run(std::integral_constant<int, 8>{});
  if constexpr (!kPacked)
    if (each <= 16) return run(std::integral_constant<int, 16>{});
  if constexpr (kGated) return launch_product<kPacked, 1, 0, true>(a);
  return hipErrorInvalidValue;  // (down's length is at most kMoeMaxWidth)
}

template <bool kPacked>
hipError_t launch(const MoeLaunch& a, bool out_bf16) {
  hipError_t err = launch_products<kPacked, true>(a);
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
  err = launch_products<kPacked, false>(a);
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
