// The mixture-of-experts layer of quest_moe_fwd for few tokens, in two kernels.
//
// With few tokens hardly two of them share an expert: each pair of a token and one of its
// experts is taken by itself, and what the general form (quest_moe.hip) does in kernels
// of their own between the products is done again by every workgroup that needs it:
//   gated  (16 columns of h, pair): one wave looks for the pair's expert among the
//          token's logits, while the token's codes are on their way; 4 waves share the
//          contraction.  One workgroup a token writes the choice down for the next kernel.
//   down   (16 output columns, token): 8 waves share the token's experts and their
//          contractions.  h of all of them is quantised to LDS while the first weights
//          are on their way; the weighted sum over the experts follows through LDS.
// Every value is computed by the operations of the general form, in their order: the
// results are the same bits.
//
// What bounds it is latency: one token of top 8 of 64 experts of 2048 x 1024 at 4 bits
// takes 8.2 + 8.7 us (the general form's five kernels 25.2), of which its 25 MB are 5.2 at
// a copy's rate; two launches, the logits and then the weights behind them, and h and
// then its transform are the rest.  Measured against it: all waves looking for the expert
// themselves 17.5 together, 8 waves in gated 15.7 (but 33.4 instead of 30.8 for three
// tokens), 16 in down 16.2 (but 33.2 instead of 29.6 for four), 8 chunks ahead 17.4.
#include <cmath>

#include "quest_few.h"
#include "quest_i8.h"
#include "quest_launch.h"
#include "quest_moe.h"

namespace quest {
namespace {

constexpr int kAhead = 4, kAheadDown = 4;  // chunks of weights on their way

// A row's chunks.  The last one's upper half may lie past the row, and counts as zeros.
template <bool kPacked>
struct Chunks {
  int count;
  bool short_end;  // this lane's part of the last chunk lies past the row
  __device__ __forceinline__ Chunks(int len, int lane)
      : count((len + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>),
        short_end(kPacked && (len & 127) != 0 && (lane & 32)) {}
  // Whether this lane's part of chunk c lies past the row.
  __device__ __forceinline__ bool none(int c) const { return c >= count || (short_end && c == count - 1); }
};

constexpr int kGatedWaves = 4, kDownWaves = 8;
template <bool kPacked, int kAct, int S>
__global__ void __launch_bounds__(64 * kGatedWaves) quest_moe_few_gated_kernel(const MoeLaunch a) {
  constexpr int kWaves = kGatedWaves, F = kFewFrags<kPacked>;
  __shared__ __attribute__((aligned(16))) uint32_t part[kWaves][2][16];
  __shared__ int shared_expert;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int t = blockIdx.y / a.top, rank = blockIdx.y - t * a.top, col0 = blockIdx.x * 16;
  uint32_t raw[S];
  if (wave == 0) fetch_logits(a, t, lane, raw);
  const Chunks<kPacked> chunks(a.k, lane);
  const FewRing<kAhead> ring{wave, kWaves, chunks.count};
  const few_rsrc rx = few_window(a.x + static_cast<int64_t>(t) * a.k, a.k);
  TokenBytes<kPacked> fx[kAhead][1];
  auto load_x = [&](int c, int i) {
#pragma unroll
    for (int f = 0; f < F; ++f) fx[i][0].v[f] = load_window(rx, c * kFewChunk<kPacked> + (16 * F) * g + 16 * f);
  };
  ring.begin(load_x);
  const float x_step = a.sx[t] * a.kx;
  const bool writes = blockIdx.x == 0 && rank == a.top - 1 && wave == 0;
  if (wave == 0) {
    const Choice choice = choose(a, lane, raw, rank + 1, writes);
    if (lane == rank) shared_expert = choice.found > rank ? choice.expert : -1;
    if (writes) {
      if (lane < choice.found) {
        a.weight[t * a.top + lane] = choice.weight;
        a.slot[t * a.top + lane].expert = choice.expert;
      }
      if (lane == 0) a.found[t] = choice.found;
    }
  }
  lds_barrier();
  const int expert = __builtin_amdgcn_readfirstlane(shared_expert);
  if (expert < 0) return;
  const int64_t row0 = static_cast<int64_t>(expert) * a.m + col0;
  const int row_bytes = kPacked ? a.k / 2 : a.k;
  const few_rsrc rw[2] = {few_window(a.gate + row0 * row_bytes, 16 * row_bytes),
                        few_window(a.up + row0 * row_bytes, 16 * row_bytes)};
  v4i fw[kAhead][2];
  auto load_w = [&](int c, int i) {
    const int off = chunks.none(c) ? kNoBytes : (lane & 15) * row_bytes + c * 64 + 16 * g;
#pragma unroll
    for (int p = 0; p < 2; ++p) fw[i][p] = load_window(rw[p], off);
  };
  ring.begin(load_w);
  const float fg = tid < 16 ? a.sg[row0 + tid] * a.kw : 0.0f, fu = tid < 16 ? a.su[row0 + tid] * a.kw : 0.0f;
  FewSums<kPacked, 2, 1> s;
  ring.run(
      [&](int c, int i) {
        load_x(c, i);
        load_w(c, i);
      },
      [&](int, int i) { s.add(fw[i], fx[i]); });
  // (every token column of the products is the same token)
  if ((lane & 15) == 0)
#pragma unroll
    for (int p = 0; p < 2; ++p) *reinterpret_cast<v4u*>(&part[wave][p][4 * g]) = s.total(p, 0);
  lds_barrier();
  if (tid >= 16) return;
  uint32_t sum[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    sum[p] = few_constant<kPacked>(a.k);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum[p] += part[w][p][tid];
  }
  const float gv = (static_cast<float>(static_cast<int>(sum[0])) * 0.25f) * (x_step * fg);
  const float uv = (static_cast<float>(static_cast<int>(sum[1])) * 0.25f) * (x_step * fu);
  a.h[static_cast<int64_t>(blockIdx.y) * a.m + col0 + tid] = activation<kAct>(gv) * uv;
}

// log_ks: log2 of the waves that share an expert's contraction.
template <bool kPacked, int LOGN, typename Out>
__global__ void __launch_bounds__(64 * kDownWaves)
    quest_moe_few_down_kernel(const MoeLaunch a, FwdConsts q, float half, int log_group, int log_ks) {
  constexpr int kWaves = kDownWaves;
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];  // h's, a row of m for each rank
  __shared__ float part[64 * kWaves];                              // sums of squares
  __shared__ float clip[kMoeMaxTop], weight[kMoeMaxTop];
  __shared__ __attribute__((aligned(16))) uint32_t sums[kMoeMaxTop][16];  // of the ranks' waves
  __shared__ float prod[kMoeMaxTop][16];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6;
  const int t = blockIdx.y, col0 = blockIdx.x * 16, m = a.m;
  Out* const out = static_cast<Out*>(a.out) + static_cast<int64_t>(t) * a.k + col0;
  auto store = [&](float y) {
    if constexpr (sizeof(Out) == 2)
      out[tid] = static_cast<Out>(pack_bf16x2(y, 0.0f));
    else
      out[tid] = y;
  };
  // (what lies behind the ranks that were found is brought along with them, and not used)
  const int found = a.found[t];
  const int expert = a.slot[t * a.top + min(lane, a.top - 1)].expert;  // lane r: of rank r
  const int row_bytes = kPacked ? m / 2 : m;
  const Chunks<kPacked> chunks(m, lane);
  const int ks = wave & ((1 << log_ks) - 1), each = kWaves >> log_ks;
  const FewRing<kAheadDown> ring{ks, 1 << log_ks, chunks.count};
  int rank = wave >> log_ks;
  few_rsrc rw;
  v4i fw[kAheadDown][1];
  auto load_w = [&](int c, int i) {
    fw[i][0] = load_window(rw, chunks.none(c) ? kNoBytes : (lane & 15) * row_bytes + c * 64 + 16 * g);
  };
  auto begin = [&]() {
    if (rank >= found) return;
    const int e = __builtin_amdgcn_readlane(expert, rank);
    rw = few_window(a.down + (static_cast<int64_t>(e) * a.k + col0) * row_bytes, 16 * row_bytes);
    ring.begin(load_w);
  };
  // h of `at_once` ranks at a time to codes, a lane a run of 32 entries, as
  // quest_fwd_i8_kernel; waves without a row go straight to their weights.
  const int runs = m / RUN, at_once = 64 * kWaves / runs, lrow = tid / runs, run = tid - lrow * runs;
  const int per_row = runs >> log_group;
  for (int r0 = 0; r0 < a.top; r0 += at_once) {
    const int row = r0 + lrow;
    const bool works = wave * 64 < min(at_once, a.top - r0) * runs, active = lrow < at_once && row < a.top;
    if (r0 > 0 && per_row > 1) lds_barrier();  // the last rows' sums have been read
    uint32_t raw[RUN];
    if (works) {
      const u32x4* const src = reinterpret_cast<const u32x4*>(
          a.h + static_cast<int64_t>(t * a.top + (active ? row : 0)) * m + (active ? run : 0) * RUN);
#pragma unroll
      for (int i = 0; i < RUN / 4; ++i) {
        const u32x4 w = src[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[4 * i + j] = w[j];
      }
    }
    if (r0 == 0) begin();
    float v[RUN], ss, tau;
    if (works) {
      tau = fwd_transform<float, LOGN>(raw, v, ss, tid);
      ss = group_sum(ss, log_group);
      if (per_row > 1 && (tid & ((1 << log_group) - 1)) == 0) part[tid >> log_group] = ss;
    }
    if (per_row > 1) {
      lds_barrier();
      ss = 0.0f;
      if (active)
        for (int i = 0; i < per_row; ++i) ss += part[lrow * per_row + i];
    }
    if (active) {
      const RowConsts c = row_consts(ss, tau, q);
      if (run == 0) clip[row] = c.scale;
      u32x4* const to = reinterpret_cast<u32x4*>(codes + row * m + run * RUN);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        to[i] = u32x4{codes4(v + 16 * i, c.kk, half), codes4(v + 16 * i + 4, c.kk, half),
                      codes4(v + 16 * i + 8, c.kk, half), codes4(v + 16 * i + 12, c.kk, half)};
    }
  }
  if (tid < found) weight[tid] = a.weight[t * a.top + tid];
  // thread (rank, column) of the last step: its factor
  const int of = max(min(tid >> 4, found - 1), 0);
  const int of_expert = __shfl(expert, of);  // (by every lane: lane `of` need not be one of the threads below)
  const float fd = tid < 16 * found ? a.sd[static_cast<int64_t>(of_expert) * a.k + col0 + (tid & 15)] * a.kw : 0.0f;
  if (found <= 0) {
    if (tid < 16) store(found < 0 ? __builtin_nanf("") : 0.0f);
    return;
  }
  lds_barrier();
  for (; rank < found; rank += each) {
    if (rank >= each) begin();
    FewSums<kPacked, 1, 1> s;
    const uint8_t* const x = codes + rank * m + (kPacked ? 32 : 16) * g;
    ring.run(load_w, [&](int c, int i) {
      TokenBytes<kPacked> fx[1];
#pragma unroll
      for (int f = 0; f < kFewFrags<kPacked>; ++f)
        fx[0].v[f] = chunks.none(c) ? v4i{} : load_v4i(x + c * kFewChunk<kPacked> + 16 * f);
      s.add(fw[i], fx);
    });
    if ((lane & 15) == 0) *reinterpret_cast<v4u*>(&sums[(rank << log_ks) + ks][4 * g]) = s.total(0, 0);
  }
  lds_barrier();
  if (tid < 16 * found) {
    uint32_t sum = few_constant<kPacked>(m);
    for (int i = 0; i < 1 << log_ks; ++i) sum += sums[(of << log_ks) + i][tid & 15];
    prod[of][tid & 15] = (static_cast<float>(static_cast<int>(sum)) * 0.25f) * ((clip[of] * a.kh) * fd);
  }
  lds_barrier();
  if (tid >= 16) return;
  float y = 0.0f;
  for (int r = 0; r < found; ++r) y = fmaf(weight[r], prod[r][tid], y);
  store(y);
}

template <bool kPacked, int kAct>
hipError_t launch_gated(const MoeLaunch& a) {
  const auto kernel = a.experts <= 64    ? quest_moe_few_gated_kernel<kPacked, kAct, 1>
                      : a.experts <= 128 ? quest_moe_few_gated_kernel<kPacked, kAct, 2>
                                         : quest_moe_few_gated_kernel<kPacked, kAct, kMoeMaxExperts / 64>;
  hipLaunchKernelGGL(kernel, dim3(a.m / 16, a.n * a.top), dim3(64 * kGatedWaves), 0, a.stream, a);
  return hipGetLastError();
}

template <bool kPacked, typename Out>
hipError_t launch_down(const MoeLaunch& a) {
  const int runs = a.m / RUN;
  int log_ks = __builtin_ctz(kDownWaves);  // a power of two of waves a rank
  while (log_ks > 0 && (kDownWaves >> log_ks) < a.top) --log_ks;
  const FwdConsts q = i8_consts(a.m, a.log_block, a.h_bits, a.halpha, 1.0);
  const float half = static_cast<float>(1 << (a.h_bits - 1));
  const dim3 grid(a.k / 16, a.n);
  const size_t lds = static_cast<size_t>(a.top) * a.m;
  const int log_group = i8_log_group(runs);
  const auto kernel = a.log_block == 6   ? quest_moe_few_down_kernel<kPacked, 6, Out>
                      : a.log_block == 7 ? quest_moe_few_down_kernel<kPacked, 7, Out>
                                         : quest_moe_few_down_kernel<kPacked, 8, Out>;
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kDownWaves), lds, a.stream, a, q, half, log_group, log_ks);
  return hipGetLastError();
}

template <bool kPacked>
hipError_t launch(const MoeLaunch& a, bool out_bf16) {
  const hipError_t err = a.act == 0 ? launch_gated<kPacked, 0>(a) : launch_gated<kPacked, 1>(a);
  if (err != hipSuccess) return err;
  return out_bf16 ? launch_down<kPacked, uint16_t>(a) : launch_down<kPacked, float>(a);
}

}  // namespace

// This form reads an expert's weights again for each token that takes it, mostly from
// caches, but spends some 10 us less on launches and what lies between the products.  It
// pays as long as the bytes that are read again, with top of the experts taken by each
// token at random, stay below some 42 MB: with this form and the general one, in us, 6
// tokens of top 8 of 64 experts of 2048 x 1024 at 4 bits (40.0 MB) 42.0 and 47.5, 8 (69 MB)
// 52.1 and 45.1; 16 of top 3 of 13 of 704 x 448 at 8 bits (33 MB) 17.9 and 20.9, 24 (56 MB)
// 23.6 and 20.7.  A workgroup of gated costs as much as some 32 KB whatever it reads: 12 of
// top 4 of 32 of 1024 x 512 at 4 bits (so counted 29 MB) 21.8 and 22.9, 16 (43 MB) 24.9 and
// 22.5.  For up to 4 tokens, where the general form's wide instructions are emptier still,
// below 100 MB: 4 of top 2 of 8 of 2048 x 5632 at 8 bits (88 MB) 50.6 and 57.4, 2 of top 4
// of 4 of 4096 x 7168 (352 MB) 137.5 and 85.3.  One token reads nothing again: of top 4 of
// those 78.6 and 85.0.  LDS holds the codes of a token's h.
bool moe_is_few(int n, int experts, int top, int k, int m, bool packed) {
  if (n > 32 || top * m > 1 << 16) return false;
  const double pairs = n * top, bytes = 3.0 * m * k / (packed ? 2 : 1);
  const double chosen = experts * (1.0 - std::pow(1.0 - double(top) / experts, n));
  const double most = n <= 4 ? 100e6 : 42e6, each = 32e3 * m / 16;
  return pairs * (bytes > each ? bytes : each) - chosen * bytes <= most;
}

hipError_t launch_moe_few(const MoeLaunch& a, bool packed, bool out_bf16) {
  return packed ? launch<true>(a, out_bf16) : launch<false>(a, out_bf16);
}

}  // namespace quest
