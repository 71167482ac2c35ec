// Codes one a byte: the quantiser that writes the operand of the 8-bit integer
// product (quest_gemm_i8, quest_moe_fwd), and its way back to values.
//
// A row's entries after the blockwise Hadamard transform, y, become
//   c = clamp(floor(y / Delta), -2^(b-1), 2^(b-1) - 1),  Delta = 2 s / (2^b - 1),
// with s = alpha_b RMS, and stand for (c + 1/2) Delta: the codes of
// quest_quantize_fwd less 2^(b-1), as signed bytes for every b.  floor of the
// product is exact, so a code is off only where the transform's own roundings
// (and the one of y / Delta) move an entry across a level's edge; adding 2^(b-1)
// first, as packed codes are made, rounds y / Delta to 2^-17 at b = 8 and moves
// eight times as many.
#include "quest_i8.h"

namespace quest {
namespace {

extern __shared__ u32x4 i8_lds[];

// A workgroup holds rows_per_wg whole rows, a lane a run of 32 entries, as in
// quest_fwd_rows_kernel; rows within a wave need no LDS for their sums.  Bound by its
// bytes: 16384 x 2048 bf16 with the mask, 105 MB, 22.5 us (4.7 TB/s, a copy's 4.84).
template <typename In, int LOGN>
__global__ void __launch_bounds__(1024)
    quest_fwd_i8_kernel(const In* __restrict__ x, int64_t rows, int runs_per_row, int rows_per_wg, int log_group,
                        FwdConsts k, float half, uint8_t* __restrict__ codes, float* __restrict__ scale,
                        uint32_t* __restrict__ mask) {
  constexpr int U = sizeof(In) * 2;
  float* const part = reinterpret_cast<float*>(i8_lds + (blockDim.x >> 6) * 64 * U);
  const int64_t wg = blockIdx.x;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int lrow = tid / runs_per_row;
  const int run_in_row = tid - lrow * runs_per_row;
  const int64_t total_runs = rows * runs_per_row;
  const int64_t wg_first_run = wg * rows_per_wg * runs_per_row;
  const int wave_tid0 = __builtin_amdgcn_readfirstlane(tid) & ~63;

  uint32_t raw[4 * U];
  u32x4* const stage = i8_lds + (wave_tid0 >> 6) * 64 * U;
  wave_load_runs<U>(x, (wg_first_run + wave_tid0) * U, total_runs * U, lane, stage, raw);
  float v[RUN];
  float ss;
  const float tau = fwd_transform<In, LOGN>(raw, v, ss, tid);

  ss = group_sum(ss, log_group);
  const int per_row = runs_per_row >> log_group;
  if (per_row > 1) {
    if ((tid & ((1 << log_group) - 1)) == 0) part[tid >> log_group] = ss;
    __syncthreads();
    ss = 0.f;
    if (lrow < rows_per_wg) {
      const float* pr = part + lrow * per_row;
      for (int i = 0; i < per_row; ++i) ss += pr[i];
    }
  }
  // Lanes past the workgroup's rows compute on whatever they loaded (DPP needs
  // whole quads); their stores fall outside the workgroup's windows.
  const uint32_t wg_runs = static_cast<uint32_t>(rows_per_wg * runs_per_row);
  const RowConsts c = row_consts(ss, tau, k);
  const rsrc_t scale_r = window_at(scale, wg * rows_per_wg * 4, rows * 4, rows_per_wg * 4);
  const int scale_off = (run_in_row == 0 && lrow < rows_per_wg) ? lrow * 4 : kNowhere;
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(c.scale), scale_r, scale_off, 0, 0);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = codes4(v + 4 * j, c.kk, half);
  const rsrc_t codes_r = window_at(codes, wg_first_run * 32, total_runs * 32, wg_runs * 32);
  __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, codes_r, tid * 32, 0, 0);
  __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4], w[5], w[6], w[7]}, codes_r, tid * 32 + 16, 0, 0);
  if (mask) {
    uint32_t mw = 0u;
    push16_abs_le(mw, v + 16, c.thr);
    push16_abs_le(mw, v, c.thr);
    const rsrc_t mask_r = window_at(mask, wg_first_run * 4, total_runs * 4, wg_runs * 4);
    __builtin_amdgcn_raw_buffer_store_b32(mw, mask_r, tid * 4, 0, kNonTemporal);
  }
}

// Values (2 c + 1) s / (2^b - 1) of 16 codes a thread; cols is a multiple of 64.  At most
// kDequantChunks of 16 a launch: the index, its division by the row's length and the outputs'
// 16-byte pieces, up to 4 i + 3, are counted in 32 bits.  Bound by its bytes: 18432 x 2048
// to bf16, 113 MB, 20.7 us (5.5 TB/s).
constexpr int64_t kDequantChunks = int64_t(1) << 30;
template <typename Out>
__global__ void __launch_bounds__(256)
    quest_dequant_i8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scale, uint32_t chunks,
                            uint32_t chunks_per_row, float levels, Out* __restrict__ out) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= chunks) return;
  const float c = scale[i / chunks_per_row] / levels;
  const u32x4 w = reinterpret_cast<const u32x4*>(codes)[i];
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int code = static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
    v[j] = static_cast<float>(2 * code + 1) * c;
  }
  if constexpr (sizeof(Out) == 2) {
    u32x4* o = reinterpret_cast<u32x4*>(out) + 2 * i;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      o[q] = u32x4{pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                   pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7])};
  } else {
    float4* o = reinterpret_cast<float4*>(out) + 4 * i;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  }
}

// quest_bwd_kernel with fp32 gradients in and bf16 out: the gradients of products in
// 8-bit integers are rounded once.  Bound by its bytes: 18432 x 2048, 231 MB, 37.1 us (6.2 TB/s).
template <int LOGN>
__global__ void __launch_bounds__(256)
    quest_bwd_narrow_kernel(const float* __restrict__ grad, const uint32_t* __restrict__ mask, int64_t total_runs,
                            uint16_t* __restrict__ grad_out) {
  __shared__ u32x4 stage_all[4][64 * 8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x) >> 6;
  const int64_t run0 = static_cast<int64_t>(blockIdx.x) * 256 + wave * 64;
  const uint32_t m =
      __builtin_amdgcn_raw_buffer_load_b32(window_at(mask, run0 * 4, total_runs * 4, 64 * 4), lane * 4, 0, kNonTemporal);
  uint32_t raw[RUN], narrow[RUN / 2];
  wave_load_runs<8>(grad, run0 * 8, total_runs * 8, lane, stage_all[wave], raw);
  float v[RUN];
  widen_run_masked(raw, m, v);
  const float k = fwht_block<LOGN>(v, lane) * BlockConst<LOGN>::rsqrt_n;
#pragma unroll
  for (int j = 0; j < RUN; ++j) v[j] *= k;
  narrow_run(v, narrow);
  wave_store_runs<4>(grad_out, run0 * 4, total_runs * 4, lane, stage_all[wave], narrow);
}

template <typename In, int LOGN>
hipError_t launch_fwd(const In* x, int bits, const FwdLaunch& a) {
  const int runs = static_cast<int>(a.cols / RUN);
  const FwdConsts k = i8_consts(a.cols, LOGN, bits, a.alpha, a.trust);
  // Whole rows: the fewest that fill whole waves, and then up to 256 lanes.
  int rows_per_wg = 64 / gcd_int(runs, 64);
  if (rows_per_wg * runs > 1024) rows_per_wg = 1024 / runs;
  if (rows_per_wg < 1) rows_per_wg = 1;
  while (rows_per_wg * runs <= 128) rows_per_wg *= 2;
  // Few rows are spread over the compute units, since their time is a workgroup's (in one
  // kernel trace, 5 x 5632 in fp32 in 2 workgroups of 11 waves 4.8 us, in 5 of 3 waves 3.8;
  // 700 x 960 5.8 and 4.0).
  const int64_t spread = a.rows / (2 * device_cus());
  if (rows_per_wg > spread) rows_per_wg = spread < 1 ? 1 : static_cast<int>(spread);
  const int threads = ((rows_per_wg * runs + 63) / 64) * 64;
  const int64_t grid = (a.rows + rows_per_wg - 1) / rows_per_wg;
  const size_t lds = static_cast<size_t>(threads) * (sizeof(In) * 32) + static_cast<size_t>(threads) * 4;
  hipLaunchKernelGGL((quest_fwd_i8_kernel<In, LOGN>), dim3(static_cast<uint32_t>(grid)), dim3(threads), lds, a.stream,
                     x, a.rows, runs, rows_per_wg, i8_log_group(runs), k, static_cast<float>(1 << (bits - 1)), a.codes, a.scale,
                     reinterpret_cast<uint32_t*>(a.mask));
  return hipGetLastError();
}

template <typename In>
hipError_t launch_fwd_block(const In* x, int log_block, int bits, const FwdLaunch& a) {
  switch (log_block) {
    case 6: return launch_fwd<In, 6>(x, bits, a);
    case 7: return launch_fwd<In, 7>(x, bits, a);
    default: return launch_fwd<In, 8>(x, bits, a);
  }
}

}  // namespace

hipError_t launch_fwd_i8(const void* x, int x_is_bf16, int log_block, int bits, const FwdLaunch& a) {
  if (x_is_bf16) return launch_fwd_block(static_cast<const uint16_t*>(x), log_block, bits, a);
  return launch_fwd_block(static_cast<const float*>(x), log_block, bits, a);
}

hipError_t launch_trust_bwd_narrow(const float* grad, const uint8_t* mask, int64_t rows, int64_t cols, int log_block,
                                   void* grad_out, hipStream_t stream) {
  const int64_t runs = rows * (cols / RUN);
  const auto kernel = log_block == 6   ? quest_bwd_narrow_kernel<6>
                      : log_block == 7 ? quest_bwd_narrow_kernel<7>
                                       : quest_bwd_narrow_kernel<8>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>((runs + 255) / 256)), dim3(256), 0, stream, grad,
                     reinterpret_cast<const uint32_t*>(mask), runs, static_cast<uint16_t*>(grad_out));
  return hipGetLastError();
}

hipError_t launch_dequantize_i8(const uint8_t* codes, const float* scale, int64_t rows, int64_t cols, int bits,
                                void* out, int out_is_bf16, hipStream_t stream) {
  const float levels = static_cast<float>((1 << bits) - 1);
  const int64_t per_row = cols / 16, most = kDequantChunks / per_row;  // rows a launch
  for (int64_t row = 0; row < rows; row += most) {
    const int64_t chunks = (rows - row < most ? rows - row : most) * per_row;
    const dim3 grid(static_cast<uint32_t>((chunks + 255) / 256));
    if (out_is_bf16)
      hipLaunchKernelGGL((quest_dequant_i8_kernel<uint16_t>), grid, dim3(256), 0, stream, codes + row * cols,
                         scale + row, static_cast<uint32_t>(chunks), static_cast<uint32_t>(per_row), levels,
                         static_cast<uint16_t*>(out) + row * cols);
    else
      hipLaunchKernelGGL((quest_dequant_i8_kernel<float>), grid, dim3(256), 0, stream, codes + row * cols, scale + row,
                         static_cast<uint32_t>(chunks), static_cast<uint32_t>(per_row), levels,
                         static_cast<float*>(out) + row * cols);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace quest
