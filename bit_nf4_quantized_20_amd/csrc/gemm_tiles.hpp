// gemm_tiles.hpp -- what the MFMA GEMM kernels (bf16 / NF4 and 8-bit) share:
// the swizzled 128-byte LDS rows, tiles copied straight from global memory
// into LDS, and the XCD-aware order of the output tiles.
#pragma once

#include "common.hpp"

namespace qlora {

namespace {

constexpr int kBK = 64;

// 16-byte chunk swizzle of a 128-byte LDS row.  A fragment read has 32
// lanes on 32 consecutive rows at one chunk; the key (row & 7) ^ (row >> 3 & 1)
// gives every 8 consecutive rows distinct chunks (32-bank view) and every 16
// consecutive rows distinct (row parity, chunk) pairs (64-bank view), so the
// reads are conflict-free either way.  Writes cover whole rows, so any
// per-row permutation is conflict-free for them.
__device__ __forceinline__ int swz(int row, int chunk) {
  return chunk ^ ((row & 7) ^ ((row >> 3) & 1));
}

constexpr int kBufferWord3 = 0x00020000;  // raw buffer resource, 32-bit data format
constexpr int kStream = 2;                // cache policy nt: streamed once

// A buffer resource for rows [row0, nrows) of a row-major matrix (ld
// elements per row, elem_bytes each): loads past the last row return zeros
// without a branch.  The size is capped at 2^31 - 1 bytes; a tile's own rows
// start at offset 0, so only rows far past the tile could fall beyond it.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int64_t ld, int64_t row0,
                                                            int64_t nrows, int elem_bytes) {
  const uint64_t bytes = static_cast<uint64_t>(nrows > row0 ? nrows - row0 : 0) * ld * elem_bytes;
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(static_cast<const uint8_t*>(base) + row0 * ld * elem_bytes), 0,
      static_cast<int>(bytes < 0x7fffffffu ? bytes : 0x7fffffffu), kBufferWord3);
}

// bf16 tile rows [ROWS][64] of a K-contiguous matrix copied straight into
// LDS by NW waves: ROWS/8 blocks of 1 KB, one wave instruction each.  Lane L
// of a block lands at LDS byte 16 L of the block, i.e. row 8 blk + L/8,
// position L % 8, so it loads the global chunk that the swizzle puts there
// (the XOR swizzle is its own inverse).  Rows past the matrix read as zero.
template <int ROWS, int NW>
struct DtlTile {
  static constexpr int kPerWave = ROWS / 8 / NW;
  __amdgpu_buffer_rsrc_t rs;
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(const uint16_t* base, int64_t ld, int64_t row0, int64_t nrows, int wv, int lane) {
    rs = rows_rsrc(base, ld, row0, nrows, 2);
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int row = (i * NW + wv) * 8 + (lane >> 3);
      voff[i] = static_cast<uint32_t>((row * ld + swz(row, lane & 7) * 8) * 2);
    }
  }
  __device__ __forceinline__ void load(uint16_t* lds, int wv, int64_t k0) const {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * NW + wv) * 512), 16, voff[i],
          static_cast<int>(k0 * 2), 0, 0);
  }
};

__device__ __forceinline__ bf16x8 lds_frag(const uint16_t* lds, int row, int chunk) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * kBK + swz(row, chunk) * 8);
  return __builtin_bit_cast(bf16x8, v);
}

// XCD-aware tile order.  Workgroups are dispatched round-robin over the 8
// XCDs (linear id % 8), and each XCD has its own L2.  The tiles are renumbered
// so that XCD x runs a contiguous stretch of the tile sequence, and the
// sequence walks groups of 8 M-tiles column by column, so the ~32 workgroups an
// XCD runs at once cover a compact block of C and share A and B panels in
// that XCD's L2.
constexpr int kXcds = 8;
constexpr int kGroupM = 8;
__device__ __forceinline__ void xcd_tile(int64_t gm, int64_t gn, int64_t& mt, int64_t& nt) {
  const int64_t total = gm * gn;
  const int64_t lin = static_cast<int64_t>(blockIdx.y) * gm + blockIdx.x;
  int64_t t = lin;
  if (total % kXcds == 0) t = (lin % kXcds) * (total / kXcds) + lin / kXcds;
  const int64_t per_group = kGroupM * gn;
  const int64_t g = t / per_group;
  const int64_t gm_g = (gm - g * kGroupM) < kGroupM ? (gm - g * kGroupM) : kGroupM;
  const int64_t in_g = t - g * per_group;
  mt = g * kGroupM + in_g % gm_g;
  nt = in_g / gm_g;
}

}  // namespace

}  // namespace qlora
