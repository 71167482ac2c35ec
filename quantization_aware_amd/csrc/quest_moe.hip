// A whole mixture-of-experts layer for a few tokens, on quantised weights.
//
//   y_t = sum over the experts e that token t takes of p_te Q(h_te) Q(down_e)^T,
//   h_te = act(Q(x_t) Q(gate_e)^T) * (Q(x_t) Q(up_e)^T),
// where a token takes the top_k experts with the largest logits (of equal ones the
// lowest index) and p is the softmax over those, or over all.  Products are sums of
// whole numbers (quest_few.h): T = sum (2 a + 1)(2 b + 1) exact, a product
// D_a D_b T / 4 as quest_gemm_i8's.  h stays in fp32 and is quantised to h_bits
// with its Hadamard transform as by quest_quantize_fwd_i8.
//
// With few tokens the chosen experts' weights are the work, and each is read once.
// Three kernels, whose grids count the most experts that can be chosen ("slots",
// min(experts, n top_k)), since the choice is known on the device only:
//   gated   (16 columns of h, slot): every workgroup finds its slot's expert and that
//           expert's tokens from the logits, 8 waves share k, sums meet in LDS, h goes
//           to the workspace, a row for each token and rank of the expert in it;
//   down    (128 output columns, slot): the tokens' h is transformed and quantised
//           into LDS by the workgroup, each wave multiplies it by 16 rows of down;
//           the products go to the workspace;
//   combine the top_k products of each token are added in the order of their rank.
// No atomics on results: the sums' order is fixed.  The workspace need not be set.
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

// A token's logits, expert 64 i + lane in v[i]: -inf past the last expert, and for
// NaN (which no comparison finds; the combining kernel gives NaN for such a token).
template <typename L>
__device__ __forceinline__ void load_logits(const L* row, int experts, int lane, float (&v)[kSets]) {
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int e = 64 * i + lane;
    v[i] = kNone;
    if (64 * i < experts) {
      const L raw = row[min(e, experts - 1)];
      float f;
      if constexpr (sizeof(L) == 2)
        f = __uint_as_float(static_cast<uint32_t>(raw) << 16);
      else
        f = raw;
      v[i] = e < experts && f == f ? f : kNone;
    }
  }
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
// s-th expert that any token takes; otherwise it is expert s.
template <typename L>
__device__ __forceinline__ int find_tokens(const MoeLaunch& a, int slot, List& list, int tid) {
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const L* logits = static_cast<const L*>(a.logits);
  int e = slot;
  if (a.slots < a.experts) {
    if (tid < 2 * kSets) list.chosen[tid] = 0;
    __syncthreads();
    for (int t = wave; t < a.n; t += kWaves) {
      float v[kSets];
      load_logits(logits + static_cast<int64_t>(t) * a.experts, a.experts, lane, v);
      for (int r = 0; r < a.top; ++r) {
        float value;
        const int found = take_largest(v, lane, value);
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
      if (e < 0 && left < here) {
        for (; left > 0; --left) bits &= bits - 1;
        e = 32 * w + __builtin_ctz(bits);
      }
      left -= e < 0 ? here : 0;
    }
    if (e < 0) return -1;
  }
  for (int t = wave; t < a.n; t += kWaves) {
    float v[kSets];
    load_logits(logits + static_cast<int64_t>(t) * a.experts, a.experts, lane, v);
    const int r = rank_of(v, e, a.top, lane);
    if (lane == 0) list.rank_of[t] = r;
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

// h of 16 columns for the tokens of one slot's expert, T groups of 16 of them at a time.
template <bool kPacked, int T, typename L>
__global__ void __launch_bounds__(64 * kWaves) quest_moe_gated_kernel(const MoeLaunch a) {
  __shared__ List list;
  __shared__ __attribute__((aligned(16))) uint32_t part[kWaves][2][T * 256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int e = find_tokens<L>(a, blockIdx.y, list, tid);
  if (e < 0) return;
  const int count = __builtin_amdgcn_readfirstlane(list.count);
  const int m = a.m, k = a.k, col0 = blockIdx.x * 16;
  const int64_t row_bytes = kPacked ? k / 2 : k;
  const int64_t at = (static_cast<int64_t>(e) * m + col0 + (lane & 15)) * row_bytes;
  const uint8_t* const wp[2] = {a.gate + at, a.up + at};
  const int chunks = (k + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>;
  for (int t0 = 0; t0 < count; t0 += 16 * T) {
    const uint8_t* xp[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      // (past the last token: the last again, whose sums are not used)
      const int entry = list.token[min(t0 + 16 * t + (lane & 15), count - 1)];
      xp[t] = a.x + static_cast<int64_t>(entry & 255) * k;
    }
    FewSums<kPacked, 2, T> s;
    few_run<kPacked, 2, T, 2>(s, wp, xp, wave, kWaves, chunks, k, lane);
    if (t0 > 0) __syncthreads();  // the last group's sums have been read
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int t = 0; t < T; ++t)
        *reinterpret_cast<v4u*>(&part[wave][p][(16 * t + (lane & 15)) * 16 + 4 * (lane >> 4)]) = s.total(p, t);
    __syncthreads();
    for (int o = tid; o < T * 256; o += 64 * kWaves) {
      const int i = t0 + o / 16, col = col0 + o % 16;
      if (i >= count) break;
      uint32_t g = few_constant<kPacked>(k), u = g;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        g += part[w][0][o];
        u += part[w][1][o];
      }
      const int entry = list.token[i], token = entry & 255, rank = entry >> 8;
      const float fx = a.sx[token] * a.kx;
      const int64_t ws = static_cast<int64_t>(e) * m + col;
      const float gv = (static_cast<float>(static_cast<int>(g)) * 0.25f) * (fx * (a.sg[ws] * a.kw));
      const float uv = (static_cast<float>(static_cast<int>(u)) * 0.25f) * (fx * (a.su[ws] * a.kw));
      a.h[(static_cast<int64_t>(token) * a.top + rank) * m + col] = activation(gv, a.act) * uv;
    }
  }
}

// Butterflies between lanes d apart.
template <int D>
__device__ __forceinline__ float lane_xor(float x) {
  static_assert(D == 1 || D == 2 || D == 4 || D == 8 || D == 16, "lanes within half a wave");
  if constexpr (D == 1) return dpp_read<0xB1>(x);
  if constexpr (D == 2) return dpp_read<0x4E>(x);
  if constexpr (D == 8) return dpp_read<0x128>(x);  // row_ror:8
  return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(x), 0x1F | D << 10));
}
template <int D>
__device__ __forceinline__ void butterfly(float (&v)[8], int lane) {
  const float sign = lane & D ? -1.0f : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaf(sign, v[j], lane_xor<D>(v[j]));
}

// Unnormalised transform of blocks of `block` entries, 8 a lane.
__device__ __forceinline__ void transform8(float (&v)[8], int block, int lane) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((j & s) == 0) {
        const float x = v[j], y = v[j + s];
        v[j] = x + y;
        v[j + s] = x - y;
      }
  butterfly<1>(v, lane);
  butterfly<2>(v, lane);
  butterfly<4>(v, lane);
  if (block >= 128) butterfly<8>(v, lane);
  if (block >= 256) butterfly<16>(v, lane);
}

// Products of the tokens' quantised h by 128 rows of down.
template <bool kPacked, int T, typename L>
__global__ void __launch_bounds__(64 * kWaves) quest_moe_down_kernel(const MoeLaunch a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];  // 16 T rows of `pitch` bytes
  __shared__ List list;
  __shared__ float step[16 * T];
  __shared__ int code_sum[16 * T];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int e = find_tokens<L>(a, blockIdx.y, list, tid);
  if (e < 0) return;
  const int count = __builtin_amdgcn_readfirstlane(list.count);
  const int m = a.m, k = a.k;
  const int pitch = moe_code_pitch(m);
  const int chunks = (m + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>;
  const int row = (blockIdx.x * kWaves + wave) * 16;  // the wave's 16 output columns
  const int64_t row_bytes = kPacked ? m / 2 : m;
  const int64_t first = static_cast<int64_t>(e) * k + min(row, k - 16);
  const uint8_t* const wp[1] = {a.down + (first + (lane & 15)) * row_bytes};
  for (int t0 = 0; t0 < count; t0 += 16 * T) {
    const int here = min(count - t0, 16 * T);
    if (t0 > 0) __syncthreads();  // the last group's codes have been read
    for (int i = wave; i < here; i += kWaves) {
      const int entry = list.token[t0 + i];
      const float* h = a.h + (static_cast<int64_t>(entry & 255) * a.top + (entry >> 8)) * m;
      float ss = 0.0f;
      for (int c = 8 * lane; c < m; c += 512) {
        const float4 p = *reinterpret_cast<const float4*>(h + c), q = *reinterpret_cast<const float4*>(h + c + 4);
        ss = fmaf(p.x, p.x, fmaf(p.y, p.y, fmaf(p.z, p.z, fmaf(p.w, p.w, ss))));
        ss = fmaf(q.x, q.x, fmaf(q.y, q.y, fmaf(q.z, q.z, fmaf(q.w, q.w, ss))));
      }
      ss = group_sum(ss, 6);
      const float ms = ss * a.inv_m;
      const float kk = ms > 0.0f ? a.hkk * __builtin_amdgcn_rsqf(ms) : 0.0f;  // (a row of zeros: the middle codes)
      int sum = 0;
      for (int c = 8 * lane; c - 8 * lane < m; c += 512) {
        float v[8] = {};
        if (c < m) {
          const float4 p = *reinterpret_cast<const float4*>(h + c), q = *reinterpret_cast<const float4*>(h + c + 4);
          v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
        }
        transform8(v, a.block, lane);  // (a block's lanes lie wholly before or past the row's end)
        int w[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint32_t b = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // packed weights: the even columns first
            const float x = kPacked ? v[2 * j + d] : v[4 * d + j];
            const int q = static_cast<int>(__builtin_amdgcn_fmed3f(__builtin_floorf(x * kk), -a.h_half, a.h_half - 1.0f));
            b |= (static_cast<uint32_t>(q) & 255u) << (8 * j);
          }
          w[d] = static_cast<int>(b);
        }
        if (c < m) {
          sum = __builtin_amdgcn_sdot4(w[0], 0x01010101, __builtin_amdgcn_sdot4(w[1], 0x01010101, sum, false), false);
          uint8_t* to = codes + i * pitch;
          if constexpr (kPacked) {  // of 32 columns: 16 even ones, then the odd ones
            to += (c & ~31) + (c & 31) / 2;
            *reinterpret_cast<int*>(to) = w[0];
            *reinterpret_cast<int*>(to + 16) = w[1];
          } else {
            *reinterpret_cast<int2*>(to + c) = make_int2(w[0], w[1]);
          }
        }
      }
      const float total = group_sum(static_cast<float>(sum), 6);  // (whole numbers below 2^24)
      if (lane == 0) {
        step[i] = a.halpha * __builtin_amdgcn_sqrtf(ms) * a.kh;
        code_sum[i] = static_cast<int>(total);
      }
    }
    __syncthreads();
    if (row >= k) continue;
    v4i acc[T] = {}, wide = {};
    const int g = lane >> 4;
    for (int c = 0; c < chunks; ++c) {
      constexpr int F = kFewFrags<kPacked>;
      const bool on = !kPacked || c * 128 + 32 * g < m;
      v4i w = load_v4i(wp[0] + static_cast<int64_t>(c) * 64 + 16 * (on ? g : 0));
      if (!on) w = v4i{};
      v4i f[F];
      wide_frags<kPacked>(w, f);
#pragma unroll
      for (int q = 0; q < F; ++q) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          v4i x = load_v4i(codes + (16 * t + (lane & 15)) * pitch + c * kFewChunk<kPacked> +
                           (kPacked ? 32 * g + 16 * q : 16 * g));
          if (kPacked && !on) x = v4i{};
          acc[t] = mfma_i8(f[q], x, acc[t]);
        }
        wide = mfma_i8(f[q], ones_i8(), wide);
      }
    }
    const float4 sd = *reinterpret_cast<const float4*>(a.sd + static_cast<int64_t>(e) * k + row + 4 * g);
    const float fd[4] = {sd.x * a.kw, sd.y * a.kw, sd.z * a.kw, sd.w * a.kw};
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int i = 16 * t + (lane & 15);
      if (i >= here) continue;
      const int entry = list.token[t0 + i];
      const uint32_t add = few_constant<kPacked>(m) + (kPacked ? -30u : 2u) * static_cast<uint32_t>(code_sum[i]);
      const v4u sum = 4u * (v4u)acc[t] + 2u * (v4u)wide + add;
      const float fx = step[i];
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = (static_cast<float>(static_cast<int>(sum[q])) * 0.25f) * (fx * fd[q]);
      *reinterpret_cast<float4*>(a.y + (static_cast<int64_t>(entry & 255) * a.top + (entry >> 8)) * k + row + 4 * g) =
          make_float4(y[0], y[1], y[2], y[3]);
    }
  }
}

// Four columns a thread: the products of a token's experts, weighted, in the order of
// their rank.  Every wave finds the token's weights itself.
template <typename Out, typename L>
__global__ void __launch_bounds__(256) quest_moe_combine_kernel(const MoeLaunch a) {
  __shared__ float weight[4][kMoeMaxTop];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x) >> 6;
  const int t = blockIdx.y;
  const L* row = static_cast<const L*>(a.logits) + static_cast<int64_t>(t) * a.experts;
  float v[kSets];
  load_logits(row, a.experts, lane, v);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kSets; ++i)
    if (64 * i + lane < a.experts) {
      const L raw = row[64 * i + lane];
      if constexpr (sizeof(L) == 2)
        bad |= (raw & 0x7FFFu) > 0x7F80u;
      else
        bad |= raw != raw;
    }
  const bool nan = __builtin_amdgcn_ballot_w64(bad) != 0;
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

template <bool kPacked, typename L>
hipError_t launch(const MoeLaunch& a, bool out_bf16) {
  constexpr int T = 1;
  hipLaunchKernelGGL((quest_moe_gated_kernel<kPacked, T, L>), dim3(a.m / 16, a.slots), dim3(64 * kWaves), 0, a.stream,
                     a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const size_t lds = static_cast<size_t>(16 * T) * moe_code_pitch(a.m);
  hipLaunchKernelGGL((quest_moe_down_kernel<kPacked, T, L>), dim3((a.k + 127) / 128, a.slots), dim3(64 * kWaves), lds,
                     a.stream, a);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 grid((a.k + 1023) / 1024, a.n);
  if (out_bf16)
    hipLaunchKernelGGL((quest_moe_combine_kernel<uint16_t, L>), grid, dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL((quest_moe_combine_kernel<float, L>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(const MoeLaunch& a, bool packed, bool logits_bf16, bool out_bf16) {
  if (packed) return logits_bf16 ? launch<true, uint16_t>(a, out_bf16) : launch<true, float>(a, out_bf16);
  return logits_bf16 ? launch<false, uint16_t>(a, out_bf16) : launch<false, float>(a, out_bf16);
}

}  // namespace quest
