// fp8_format.hpp -- the 8-bit block-scaled format: e4m3 codes (OCP: bias 7,
// largest finite 448, no infinities) with one power-of-two scale per block,
// stored as its biased exponent (byte b = 2^(b - 127)).
//
// For a block whose largest magnitude is a, the scale is 2^e with e the least
// integer such that a 2^-e <= 448 = 1.75 2^8.  Writing a = m 2^p, 1 <= m < 2,
// that is e = p - 8 for m <= 1.75 and p - 7 above; it comes from a's bits with
// one integer addition (adding 2^23 - 1 - (0.75 2^23) carries into the
// exponent exactly when m > 1.75).  e is held to >= -127; an all-zero block
// has byte 0.  Because the scale is a power of two, w 2^-e and code 2^e are
// exact in fp32, so a code is one rounding of the weight, and
// v_mfma_scale applies the scales inside the matrix cores at no cost.  The
// price against a free fp32 scale is at most one bit of the block's range at
// its bottom end (the largest code lies in (224, 448] instead of at 448); the
// codes' relative precision is the same.
#pragma once

#include "common.hpp"
#include "nf4_format.hpp"

namespace qlora {

constexpr int kF8Block = 128;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// scale byte of a block whose largest |value| has the fp32 bits a (a finite)
__host__ __device__ constexpr uint32_t f8_scale_byte(uint32_t a) {
  // exponent field of a (p + 127), plus 1 where the fraction exceeds 0.75
  const int e = static_cast<int>((a + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}
static_assert(f8_scale_byte(0x43e00000u) == 127, "448 -> 2^0");
static_assert(f8_scale_byte(0x43e00001u) == 128, "above 448 -> 2^1");
static_assert(f8_scale_byte(0x43600000u) == 126 && f8_scale_byte(0) == 0, "224 -> 2^-1, 0 -> byte 0");

// 2^(b - 127) and 2^(127 - b) as fp32 for a scale byte b <= 248
__device__ __forceinline__ float f8_scale(uint32_t b) {
  return __builtin_bit_cast(float, b == 0 ? 0x00400000u : b << 23);
}
__device__ __forceinline__ float f8_inv_scale(uint32_t b) { return __builtin_bit_cast(float, (254u - b) << 23); }

// four fp32 -> four e4m3 codes (round to nearest even)
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, false)));
}
// max over each aligned group of 16 lanes
__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
  v = dpp_max_u32<kDppQuadXor1>(v);
  v = dpp_max_u32<kDppQuadXor2>(v);
  v = dpp_max_u32<kDppRowHalfMirror>(v);
  return dpp_max_u32<kDppRowMirror>(v);
}

// Activations x [T][ldx] bf16 (columns 0 .. K - 1) -> codes [T][Kp], scale
// bytes in groups of four K-blocks, [ceil(KB / 4)][ldsc] dwords, row t's at
// column t: 16 lanes hold one row's 128 columns, eight each.  Columns K .. Kp
// (Kp = K rounded up to 128) become zero codes; scale bytes past the last
// block or row are not written.  A workgroup of 256 threads takes kF8RowsPer
// rows of 16 blocks, all loads before the first use: that keeps enough bytes
// in flight where few workgroups fit a CU (k_lora_front).  4096 x 14336: 10 us.
constexpr int kF8RowsPer = 4;
inline int64_t fp8_rows_blocks(const Fp8Rows& a) {
  return ceil_div(a.T, kF8RowsPer) * ceil_div(static_cast<int64_t>(a.KB), int64_t(16));
}
__device__ __forceinline__ void fp8_rows_tile(const Fp8Rows& a, uint32_t blk) {
  const uint32_t pieces = (a.KB + 15) / 16;
  const int64_t row = static_cast<int64_t>(blk / pieces) * kF8RowsPer;
  const uint32_t kb = blk % pieces * 16 + (threadIdx.x >> 4);
  const int sub = threadIdx.x & 15;
  const uint32_t col = kb * kF8Block + 8 * sub;
  u32x4 v[kF8RowsPer];
#pragma unroll
  for (int i = 0; i < kF8RowsPer; ++i) {
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (col < a.K && row + i < a.T) v[i] = *reinterpret_cast<const u32x4*>(a.x + (row + i) * a.ldx + col);
  }
  if (kb >= a.KB) return;
#pragma unroll
  for (int i = 0; i < kF8RowsPer; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max((v[i][d] << 16) & 0x7fffffffu, v[i][d] & 0x7fff0000u));
    m = max16_u32(m);
    const uint32_t b = f8_scale_byte(m);
    const float inv = f8_inv_scale(b);
    u32x2 o;
#pragma unroll
    for (int d = 0; d < 2; ++d)
      o[d] = f8_pack4(bf16_lo(v[i][2 * d]) * inv, bf16_hi(v[i][2 * d]) * inv, bf16_lo(v[i][2 * d + 1]) * inv,
                      bf16_hi(v[i][2 * d + 1]) * inv);
    if (row + i < a.T) {
      *reinterpret_cast<u32x2*>(a.codes + ((row + i) * a.KB + kb) * kF8Block + 8 * sub) = o;
      if (sub == 0) a.scales[((kb >> 2) * a.ldsc + row + i) * 4 + (kb & 3)] = static_cast<uint8_t>(b);
    }
  }
}

// The K splits of a product [M][N], N % 32 == 0: fragment (m / 32, n / 32) of
// split z is 4 KB of fp32, laid out as the matrix cores leave it: piece g = 0 ..
// 3 of lane l (16 bytes) holds row l % 32, columns 8 g + 4 (l / 32) .. + 3.  A
// store instruction then writes 1 KB in one piece; by rows it would touch 32
// rows of 32 bytes (301 x 4096 outputs of 4096 codes in four splits: 17.9 us by
// rows, 15.4 us this way).
__device__ __forceinline__ f32x4* fp8_part_frag(float* part, int64_t z, int64_t mf, int64_t nf, int64_t M, int64_t N) {
  return reinterpret_cast<f32x4*>(part) + ((z * ceil_div(M, 32) + mf) * (N / 32) + nf) * 256;
}
// C = bf16(splits added in order): a wave adds two pieces of a fragment, eight
// splits in flight; its halves swap one piece so that a lane stores 16 bytes.
inline int64_t fp8_sum_blocks(int64_t M, int64_t N) { return ceil_div(ceil_div(M, 32) * (N / 32), 2); }
__device__ __forceinline__ void fp8_sum_tile(const float* part, int S, int64_t M, int64_t N, uint16_t* C, int64_t wg) {
  const int lane = threadIdx.x & 63, h = lane >> 5, wv = threadIdx.x >> 6, j = wv & 1;
  const int64_t id = wg * 2 + (wv >> 1), nfs = N / 32, mf = id / nfs, nf = id % nfs;
  if (mf * 32 >= M) return;
  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  const f32x4* src = fp8_part_frag(const_cast<float*>(part), 0, mf, nf, M, N) + 128 * j + lane;
  const int64_t stride = ceil_div(M, 32) * nfs * 256;
  for (int z0 = 0; z0 < S; z0 += 8) {
    f32x4 v[8][2];
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int g = 0; g < 2; ++g) v[u][g] = z0 + u < S ? src[(z0 + u) * stride + 64 * g] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < S)
#pragma unroll
        for (int g = 0; g < 2; ++g) acc[g] += v[u][g];
  }
  // half h keeps piece 2 j + h and gives the other away
  u32x2 p[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) p[g] = u32x2{pack_bf16x2(acc[g][0], acc[g][1]), pack_bf16x2(acc[g][2], acc[g][3])};
  const u32x2 mine = h == 0 ? p[0] : p[1], away = h == 0 ? p[1] : p[0];
  u32x2 got;
#pragma unroll
  for (int d = 0; d < 2; ++d) got[d] = static_cast<uint32_t>(__shfl_xor(static_cast<int>(away[d]), 32));
  const u32x2 lo = h == 0 ? mine : got, hi = h == 0 ? got : mine;
  const int64_t m = mf * 32 + (lane & 31);
  if (m < M) *reinterpret_cast<u32x4*>(C + m * N + nf * 32 + 16 * j + 8 * h) = u32x4{lo[0], lo[1], hi[0], hi[1]};
}

}  // namespace qlora
