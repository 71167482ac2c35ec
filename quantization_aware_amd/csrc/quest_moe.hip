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
//   route    a wave for each token: its experts and their weights (all in one workgroup
//            took 12 us for 64 tokens of top 8 of 128 instead of 4.8);
//   gated    (some tiles of 16 columns of h, slot): first which expert the slot's is and
//            which tokens take it; h goes to the workspace, a row for each token and rank
//            of the expert among the token's;
//   (h is quantised)
//   down     (some tiles of 32 output columns, slot): the same of h's codes by down;
//   combine  the top_k products of each token, weighted, in the order of their rank.
// No atomics on results: the sums' order is fixed.  The workspace need not be set.
//
// What bounds it is reading the weights: 64 tokens of top 8 of 128 experts of 2048 x 768 at
// 4 bits, 302 MB, take 43.0 us in gated and 24.5 in down, 4.7 and 4.1 TB/s (a copy of 2 GiB
// reaches 4.84); of 8 experts of 2048 x 5632 at 8 bits, 277 MB, 40.6 and 22.2 (4.5 and
// 4.2; in other runs up to 44.4 and 24.5).  That needs every load issued without a branch around it: with one, each wait was
// for all loads on their way, 50 and 26 us, 54 and 28.5.  The other three kernels are some
// 5 us each.
#include <type_traits>

#include "quest_few.h"
#include "quest_launch.h"
#include "quest_moe.h"

namespace quest {
namespace {

constexpr int kWaves = 8, kAhead = 4;  // chunks of weights on their way

// A wave a token.  The choice goes where the kernel after the next puts products: the
// expert of each rank, -1 for none.
template <int S>
__global__ void __launch_bounds__(64) quest_moe_route_kernel(const MoeLaunch a) {
  const int t = blockIdx.x, lane = threadIdx.x;
  uint32_t raw[S];
  fetch_logits(a, t, lane, raw);
  const Choice c = choose(a, lane, raw, a.top, true);
  if (lane < a.top) reinterpret_cast<int16_t*>(a.y)[t * a.top + lane] = lane < c.found ? c.expert : -1;
  if (lane < c.found) a.weight[t * a.top + lane] = c.weight;
  if (lane == 0) a.found[t] = c.found;
}

// Slot s of the chosen experts, in order of their index.  find() gives its expert, or -1
// if there are fewer; collect() its tokens in order (token | rank << 8) and their count.
// Every thread of the workgroup calls both.
struct SlotSearch {
  static constexpr int kThreads = 64 * kWaves, kEach = kMoeMaxTokens * kMoeMaxTop / kThreads;
  struct Shared {
    uint32_t used[kMoeMaxExperts / 32];  // a bit an expert
    int expert;
    int hits[kEach * kWaves];
  };
  const MoeLaunch& a;
  Shared& sh;
  int16_t mine[kEach];

  __device__ __forceinline__ int find(int s) {
    const int tid = threadIdx.x;
    const int16_t* const choice = reinterpret_cast<const int16_t*>(a.y);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int p = tid + j * kThreads;
      mine[j] = p < a.n * a.top ? choice[p] : -1;
    }
    if (tid < kMoeMaxExperts / 32) sh.used[tid] = 0;
    if (tid == 0) sh.expert = -1;
    lds_barrier();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (mine[j] >= 0) atomicOr(&sh.used[mine[j] >> 5], 1u << (mine[j] & 31));
    lds_barrier();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kMoeMaxExperts / 32; ++w) {
      const int in_w = __builtin_popcount(sh.used[w]);
      if (w < tid >> 5) before += in_w;
      total += in_w;
    }
    if (s >= total) return -1;
    if (tid < kMoeMaxExperts) {
      const uint32_t word = sh.used[tid >> 5];
      before += __builtin_popcount(word & ((1u << (tid & 31)) - 1));
      if ((word >> (tid & 31) & 1) && before == s) sh.expert = tid;
    }
    lds_barrier();
    return __builtin_amdgcn_readfirstlane(sh.expert);
  }

  __device__ __forceinline__ int collect(int e, uint16_t* entries) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t at[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      at[j] = __builtin_amdgcn_ballot_w64(mine[j] == e);
      if (lane == 0) sh.hits[j * kWaves + wave] = __builtin_popcountll(at[j]);
    }
    lds_barrier();
    int count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (j * kThreads >= a.n * a.top) break;
      int before = count + __builtin_popcountll(at[j] & ((uint64_t(1) << lane) - 1));
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int h = sh.hits[j * kWaves + w];
        if (w < wave) before += h;
        count += h;
      }
      if (mine[j] == e) {
        const int p = tid + j * kThreads, t = p / a.top;
        entries[before] = static_cast<uint16_t>(t | (p - t * a.top) << 8);
      }
    }
    lds_barrier();
    return count;
  }
};

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
  constexpr int F = kFewFrags<kPacked>, kChunk = kFewChunk<kPacked>;
  constexpr int kCols = kGated ? 16 : 32, kTiles = kWaves / KS;
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];
  __shared__ uint16_t entries[kMoeMaxTokens];
  __shared__ __attribute__((aligned(16))) uint32_t part[KS > 1 ? kWaves : 1][2][KS > 1 ? T * 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid) >> 6, ks = wave % KS;
  const int len = kGated ? a.k : a.m, rows = kGated ? a.m : a.k;
  const int tiles = rows / kCols, chunks = (len + kChunk - 1) / kChunk;
  const int segments = (chunks + segment - 1) / segment, pitch = segment * kChunk + 16;
  const int row_bytes = kPacked ? len / 2 : len;
  __shared__ SlotSearch::Shared shared;
  SlotSearch search{a, shared};
  MoeSlot& slot = a.slot[blockIdx.y];
  int e, count;
  uint16_t entry = 0;
  if constexpr (kGated) {
    e = search.find(blockIdx.y);
    if (e < 0) {
      if (blockIdx.x == 0 && tid == 0) slot.expert = -1;
      return;
    }
  } else {
    e = slot.expert, count = slot.count;
    if (e < 0) return;
    if (wave == 0) entry = slot.entry[lane];  // (those behind the last hold anything)
  }
  // Both strips of a tile's rows, in windows of the expert's matrices.
  const int64_t first = static_cast<int64_t>(e) * rows * row_bytes;
  const int size = rows * row_bytes, second = kGated ? 0 : 16 * row_bytes;
  const few_rsrc wide[2] = {few_window((kGated ? a.gate : a.down) + first, size),
                          few_window((kGated ? a.up : a.down) + first + second, size - second)};
  // (lanes of the last chunk's upper half may lie past the row)
  const bool short_end = kPacked && (len & 127) != 0 && (lane & 32);
  const int mine = (chunks - ks + KS - 1) / KS;             // the wave's chunks ks, ks + KS, ...
  const int steps = (mine + kAhead - 1) / kAhead * kAhead;  // in whole rounds of the ring
  const int stride = gridDim.x * kTiles;
  v4i w[kAhead][2];
  auto load = [&](int tile, int i, v4i (&to)[2]) {
    const int chunk = ks + i * KS, at = tile * kCols * row_bytes + (lane & 15) * row_bytes + chunk * 64 + 16 * g;
    const bool none = i >= mine || tile >= tiles || (short_end && chunk == chunks - 1);
#pragma unroll
    for (int p = 0; p < 2; ++p) to[p] = load_window(wide[p], none ? kNoBytes : at);
  };
  int tile = blockIdx.x * kTiles + wave / KS;
  auto begin = [&]() {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(tile, i, w[i]);
  };
  begin();
  if constexpr (kGated) {
    count = search.collect(e, entries);
    if (blockIdx.x == 0) {  // for the other product
      if (tid == 0) slot.expert = e, slot.count = count;
      if (tid < count) slot.entry[tid] = entries[tid];
    }
  } else {
    if (wave == 0) entries[lane] = entry;
    lds_barrier();
  }
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
      lds_barrier();  // the last group's codes have been read
    }
    stage(0);
    lds_barrier();
    // (every wave makes the same steps: those without a tile only wait with the others)
    for (int base = blockIdx.x * kTiles; base < tiles; base += stride, tile += stride) {
      FewSums<kPacked, 2, T> s;
      for (int seg = 0; seg < segments; ++seg) {
        if (segments > 1 && (seg > 0 || base != static_cast<int>(blockIdx.x) * kTiles)) {
          lds_barrier();
          stage(seg);
          lds_barrier();
        }
        const int last = seg + 1 < segments ? (seg + 1) * (segment / KS) : steps;
        for (int i0 = seg * (segment / KS); i0 < last; i0 += kAhead) {
#pragma unroll
          for (int r = 0; r < kAhead; ++r) {
            const int i = i0 + r, chunk = ks + i * KS;
            if (i < mine && tile < tiles) {
              v4i fw[2][F];
#pragma unroll
              for (int p = 0; p < 2; ++p) wide_frags<kPacked>(w[r][p], fw[p]);
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
            const bool next = i + kAhead >= steps;
            load(next ? tile + stride : tile, next ? i + kAhead - steps : i + kAhead, w[r]);
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
        lds_barrier();
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
        lds_barrier();
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
  constexpr int kFit = (kLds / (16 * T) - 16) / kChunk, kRound = kAhead * KS, kMost = kFit / kRound * kRound;
  static_assert(kMost >= kRound, "a segment holds a round");
  int segment = chunks;
  if (chunks > kFit) {
    const int parts = (chunks + kMost - 1) / kMost;
    segment = ((chunks + parts - 1) / parts + kRound - 1) / kRound * kRound;
  }
  const size_t lds = static_cast<size_t>(16 * T) * (segment * kChunk + 16);
  // Workgroups walk tiles, so that finding and bringing the tokens is paid once for
  // several: at most two a compute unit, and as many as leave the fullest unit the fewest
  // steps.  (64 tokens of 128 experts: gated in 256 workgroups 42.8 us, in 384 49.0, in 768
  // 42.8; of 8 wide experts in 256 44.0, in 704 48.0.)
  const int each = (tiles + kTiles - 1) / kTiles, cus = device_cus();
  int wide = 1, least = 0x7FFFFFFF;
  for (int w = 1; w <= each && (w == 1 || w * a.slots <= 2 * cus); ++w) {
    const int steps = (w * a.slots + cus - 1) / cus * ((each + w - 1) / w);
    if (steps <= least) wide = w, least = steps;
  }
  hipLaunchKernelGGL((quest_moe_product_kernel<kPacked, T, KS, kMode>), dim3(wide, a.slots),
                     dim3(64 * kWaves), lds, a.stream, a, segment);
  return hipGetLastError();
}

template <bool kPacked, int kMode>
hipError_t launch_products(const MoeLaunch& a) {
  constexpr bool kGated = kMode != kDown;
  // Two groups of 16 tokens at once where an expert has more than 10 on average (a layer of 48 or
  // 64 tokens in us, one group and two: 16 an expert 102.5 and 66.9, 46.6 and 35.7; 12 an
  // expert 47.1 and 43.8; 8 an expert 55.9 and 52.4, but 37.0 and 41.5, 46.5 and 53.9; 4 an
  // expert 74.0 and 75.3).
  const bool two = static_cast<int64_t>(a.n) * a.top > 10 * static_cast<int64_t>(a.experts);
  const int tiles = kGated ? a.m / 16 : a.k / 32;
  const int chunks = ((kGated ? a.k : a.m) + kFewChunk<kPacked> - 1) / kFewChunk<kPacked>;
  // (the sums of 8 waves and two groups would leave no LDS for a round of codes)
  auto run = [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    return two ? launch_product<kPacked, 2, KS < 8 ? KS : 4, kMode>(a, tiles, chunks)
               : launch_product<kPacked, 1, KS, kMode>(a, tiles, chunks);
  };
  // As few waves a tile as keep some 16 waves a compute unit busy, each with a chunk.  (A
  // layer of 64 tokens in us with 1, 2, 4 waves a tile of one product: 24 tiles a unit
  // 74.6, 72.7, 75.0 and with 8 84.4; 11 a unit 74.2, 67.0, 70.2; 4 a unit 39.4, 34.9, 38.0;
  // 2 a unit 103.0, 76.7, 66.7; half a tile a unit 84.0, 57.4, 43.6.  Runs of the same
  // choice differ by up to 2.5.)
  const int64_t waves = static_cast<int64_t>(tiles) * a.slots, cus = device_cus();
  if (waves >= 16 * cus || chunks < 2) return run(std::integral_constant<int, 1>{});
  if (waves >= 8 * cus || chunks < 4) return run(std::integral_constant<int, 2>{});
  if (waves >= 4 * cus || chunks < 8) return run(std::integral_constant<int, 4>{});
  return run(std::integral_constant<int, 8>{});
}

template <bool kPacked>
hipError_t launch(const MoeLaunch& a, bool out_bf16) {
  const auto route = a.experts <= 64    ? quest_moe_route_kernel<1>
                     : a.experts <= 128 ? quest_moe_route_kernel<2>
                                        : quest_moe_route_kernel<kMoeMaxExperts / 64>;
  hipLaunchKernelGGL(route, dim3(a.n), dim3(64), 0, a.stream, a);
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
  if (moe_is_few(a.n, a.experts, a.top, a.k, a.m, packed)) return launch_moe_few(a, packed, out_bf16);
  return packed ? launch<true>(a, out_bf16) : launch<false>(a, out_bf16);
}

}  // namespace quest
