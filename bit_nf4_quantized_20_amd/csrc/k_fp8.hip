// k_fp8.hip -- the 8-bit format's element-wise kernels: a weight to codes and
// scales (one scale per 128 x 128 block), codes to bf16, and activations to
// codes and scales (one scale per row and 128 columns).  All are one pass
// over their data and bound by HBM.
#include "common.hpp"
#include "fp8_format.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
}  // namespace

// One workgroup of 256 threads per 128 x 128 block: thread t holds four
// consecutive columns 4 (t % 32) of rows t / 32 + 8 i, i = 0..15, so a wave's
// load covers two 512-byte row pieces and the whole 64 KiB block is in flight
// before the first value is used.  Rows and columns past the matrix read as
// zero and are not written.  28672 x 8192: 203 us, 5.8 TB/s (a copy of 2 GiB
// reaches 4.84).
__global__ __launch_bounds__(256) void k_fp8_quantize(const float* __restrict__ w, int64_t rows, int64_t cols,
                                                      uint32_t col_blocks, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  const int t = threadIdx.x, lane = t & 63;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / col_blocks) * kF8Block;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x % col_blocks) * kF8Block;
  const int nr = static_cast<int>(rows - r0 < kF8Block ? rows - r0 : kF8Block);
  const int nc = static_cast<int>(cols - c0 < kF8Block ? cols - c0 : kF8Block);
  const int row = t >> 5, col = 4 * (t & 31);
  const bool live_c = col < nc;
  const float* base = w + (r0 + row) * cols + c0 + col;
  f32x4 v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (live_c && row + 8 * i < nr)
      v[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(base + static_cast<int64_t>(8 * i) * cols));
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, abs_bits(v[i][e]));
  m = max16_u32(m);
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  __shared__ uint32_t s_m[4];
  if (lane == 0) s_m[t >> 6] = m;
  __syncthreads();
  m = max(max(s_m[0], s_m[1]), max(s_m[2], s_m[3]));
  const uint32_t b = f8_scale_byte(m);
  const float inv = f8_inv_scale(b);
  if (t == 0) scales[blockIdx.x] = static_cast<uint8_t>(b);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (live_c && row + 8 * i < nr)
      *reinterpret_cast<uint32_t*>(codes + (r0 + row + 8 * i) * cols + c0 + col) =
          f8_pack4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
}

// One workgroup per 128 x 128 block: thread t takes 16 codes at column
// 16 (t % 8) of rows t / 8 + 32 i.  code 2^e is exact in fp32; the rounding to
// bf16 is exact too unless the value is below bf16's normal range.  28672 x 8192:
// 139 us, 5.1 TB/s.
__global__ __launch_bounds__(256) void k_fp8_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int64_t rows,
                                                        int64_t cols, uint32_t col_blocks,
                                                        uint16_t* __restrict__ out) {
  const int t = threadIdx.x;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / col_blocks) * kF8Block;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x % col_blocks) * kF8Block;
  const int64_t c = c0 + 16 * (t & 7);
  const float f = f8_scale(scales[blockIdx.x]);
  u32x4 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + (t >> 3) + 32 * i;
    q[i] = u32x4{0u, 0u, 0u, 0u};
    if (r < rows && c < cols) q[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + r * cols + c));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + (t >> 3) + 32 * i;
    uint32_t o[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[i][d]), false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[i][d]), true);
      o[2 * d] = pack_bf16x2(lo[0] * f, lo[1] * f);
      o[2 * d + 1] = pack_bf16x2(hi[0] * f, hi[1] * f);
    }
    if (r < rows && c < cols) {
      u32x4* dst = reinterpret_cast<u32x4*>(out + r * cols + c);
      dst[0] = u32x4{o[0], o[1], o[2], o[3]};
      dst[1] = u32x4{o[4], o[5], o[6], o[7]};
    }
  }
}

// The activations' codes alone (fp8_rows_tile), where there is no adapter.
__global__ __launch_bounds__(256) void k_fp8_rows(Fp8Rows a) { fp8_rows_tile(a, blockIdx.x); }

hipError_t launch_fp8_quantize(const float* w, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               hipStream_t s) {
  const int64_t cb = ceil_div(cols, kF8Block);
  hipLaunchKernelGGL(k_fp8_quantize, dim3(static_cast<uint32_t>(cb * ceil_div(rows, kF8Block))), dim3(256), 0, s, w,
                     rows, cols, static_cast<uint32_t>(cb), codes, scales);
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                 uint16_t* out, hipStream_t s) {
  const int64_t cb = ceil_div(cols, kF8Block);
  hipLaunchKernelGGL(k_fp8_dequantize, dim3(static_cast<uint32_t>(cb * ceil_div(rows, kF8Block))), dim3(256), 0, s,
                     codes, scales, rows, cols, static_cast<uint32_t>(cb), out);
  return hipGetLastError();
}

hipError_t launch_fp8_rows(const Fp8Rows& a, hipStream_t s) {
  hipLaunchKernelGGL(k_fp8_rows, dim3(static_cast<uint32_t>(fp8_rows_blocks(a))), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
