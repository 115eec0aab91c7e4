// k_fp8_decode.hip -- forward of an 8-bit weight for up to 16 tokens, bound by
// the weight's bytes:
//   Y = X_hat W_hat^T + s (X A^T) B^T
// A workgroup of eight waves takes the 16-row tiles blockIdx, blockIdx +
// gridDim, ...; its waves split the 128-column blocks of the reduction.  A
// block meets v_mfma_scale_f32_16x16x128 once: lane (n = l % 16, g = l / 16)
// holds the codes of columns 16 g .. + 15 and 64 + 16 g .. + 15 of row n (A
// operand: 16 rows x 128 columns) and of token n (B operand).
//
// The activations are quantized by the workgroup itself, once: a lane loads
// its columns of token n, the four lanes of a token find their scale together,
// and the codes (8 registers per block) stay in registers for all its tiles.
// The weight's rows are copied into LDS (16 rows x 512 bytes, a chunk of four
// blocks, per wave; two rows per copy, so a copy reads 512 contiguous bytes
// twice) and read back as fragments: loaded straight into registers, every
// load touches 16 rows, which took 22.2 us for 14336 x 4096 at one token against
// 14.5.  A chunk is copied while the one before it is computed, across tile
// borders.  Measured (graph of 30 calls over three weights, one token): 14336
// x 4096 13.9 us (4.2 TB/s), 4096 x 4096 7.7 us, of which about 5 are the
// launch, the first loads and the sums; 16 tokens 15.3 and 9.3 us.
//
// The adapter joins the same sums: wave v takes the ranks 32 v .. + 31, B's
// rows as they lie in memory against s U as a bf16 hi + lo pair.  The waves'
// sums meet in LDS with one barrier per tile, and one wave (another one each
// tile) adds and stores them.
//
// Where U = X A^T is formed here (r <= 16 and at most one workgroup per CU, so
// that A is not read by more workgroups than the extra launch costs), the same
// activations meet A's rows unquantized in v_mfma_f32_16x16x32_bf16.
#include <type_traits>

#include "common.hpp"
#include "fp8_format.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {
constexpr int kWaves = 8;
constexpr int kBufferWord3 = 0x00020000;
constexpr int kStream = 2;                  // cache policy nt: streamed once
constexpr uint32_t kPastEnd = 0x80000000u;  // past every buffer (all < 2^31 bytes)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), kBufferWord3);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

struct DecodeF8 {
  const uint8_t* codes; const uint8_t* scales;
  uint32_t in;
  int64_t out;
  const uint16_t* X;
  int T;
  const uint16_t* A; const uint16_t* B;
  int r;
  float s;
  const float* U;
  uint16_t* Y;
};
}  // namespace

// NC: most chunks (of four 128-column blocks) of a wave; a wave's range may be
// shorter: the blocks past it read as zero and touch no memory.
template <int NC, bool kU>
__global__ __launch_bounds__(64 * kWaves, 2) void k_fp8_decode(DecodeF8 p) {
  constexpr int NBW = 4 * NC;
  constexpr int kChunkBytes = 16 * 512;
  __shared__ __attribute__((aligned(1024))) uint8_t s_w0[kWaves * kChunkBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s_w1[kWaves * kChunkBytes];
  __shared__ f32x4 s_acc[2][kWaves][64];
  __shared__ f32x4 s_u[kU ? kWaves : 1][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4, T = p.T, r = p.r;
  const uint32_t in = p.in;
  const int KB = static_cast<int>((in + kF8Block - 1) / kF8Block);
  const int b0 = KB * wv / kWaves, nb = KB * (wv + 1) / kWaves - b0;
  const int tiles = static_cast<int>(p.out / 16), step = gridDim.x;

  // this lane's byte offset of block i, half h, in a row of codes; past the
  // end for columns past the row (the last block may hold 64) and blocks past
  // the range
  auto col_off = [&](int i, int h) {
    int gg = g;
    __asm__ volatile("" : "+v"(gg));
    const uint32_t col = static_cast<uint32_t>(b0 + i) * kF8Block + 64 * h + 16 * gg;
    return col | (i < nb && col < in ? 0u : kPastEnd);
  };
  const uint32_t wrow = static_cast<uint32_t>(n) * in;
  // copies chunk c of a tile: row 2 q + lane / 32 at LDS byte 512 row, 16-byte
  // piece k of a row at k ^ row (the fragments' 16 rows then read 16 places)
  auto copy = [&](int tile, int c, uint8_t* stage) {
    const __amdgpu_buffer_rsrc_t rw = rsrc(p.codes + static_cast<int64_t>(tile < tiles ? tile : 0) * 16 * in,
                                           tile < tiles ? 16 * in : 0);
    int l = lane;
    __asm__ volatile("" : "+v"(l));  // the offsets are formed here each time, not kept in registers for every chunk
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = 2 * q + (l >> 5), piece = (l & 31) ^ row;
      const uint32_t col = static_cast<uint32_t>(b0 + 4 * c) * kF8Block + 16 * piece;
      const uint32_t off = 4 * c + (piece >> 3) < nb && col < in ? static_cast<uint32_t>(row) * in + col : kPastEnd;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (__attribute__((address_space(3))) void*)(stage + wv * kChunkBytes + 1024 * q), 16, off, 0, 0, kStream);
    }
  };
  // lane l: scale byte of block l of the wave's range
  auto load_s = [&](int tile) {
    const int rows = tile < tiles ? tile / (kF8Block / 16) : 0;
    return static_cast<int>(__builtin_amdgcn_raw_buffer_load_b8(
        rsrc(p.scales + static_cast<int64_t>(rows) * KB + b0, nb), lane, 0, 0));
  };
  int tile = blockIdx.x;
  int sw = load_s(tile);
  copy(tile, 0, s_w0);

  // X's codes and scales; U's partial products
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.X, static_cast<uint32_t>(T) * in * 2);
  const __amdgpu_buffer_rsrc_t ra = rsrc(p.A, kU ? static_cast<uint32_t>(r) * in * 2 : 0);
  const uint32_t xrow = n < T ? wrow * 2 : kPastEnd;
  // A's 16 rows of two blocks at a time (512 bytes a row) go through stage 1,
  // idle until the first tile, like the weight's rows
  auto copy_a = [&](int pair) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = 2 * q + (lane >> 5), piece = (lane & 31) ^ row;
      const uint32_t col = static_cast<uint32_t>(b0 + 2 * pair) * kF8Block + 8 * piece;
      const bool live = row < r && 2 * pair + (piece >> 4) < nb && col < in;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ra, (__attribute__((address_space(3))) void*)(s_w1 + wv * kChunkBytes + 1024 * q), 16,
          live ? (static_cast<uint32_t>(row) * in + col) * 2 : kPastEnd, 0, 0, 0);
    }
  };
  if constexpr (kU) copy_a(0);
  i32x8 fx[NBW];
  int sx[(NBW + 3) / 4];
  f32x4 uacc = {0.f, 0.f, 0.f, 0.f};
  struct Acts {
    u32x4 x[4];
  };
  auto load_x = [&](Acts& v, int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t c = col_off(i, q >> 1), at = (c & ~kPastEnd) * 2 + 16 * (q & 1), off = c & kPastEnd;
      v.x[q] = load16(rx, ((xrow & ~kPastEnd) + at) | off | (xrow & kPastEnd));
    }
  };
  constexpr int kRing = 4;  // blocks of activations in flight
  Acts xa[kRing];
#pragma unroll
  for (int i = 0; i < kRing; ++i) load_x(xa[i], i);
#pragma unroll
  for (int i = 0; i < NBW; ++i) {
    const Acts& v = xa[i % kRing];
    if constexpr (kU)
      if (i % 2 == 0) {
        if (i > 0) copy_a(i / 2);
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): A's rows (and the first tile's codes) are in LDS
        __builtin_amdgcn_sched_barrier(0);
      }
    if (i % 4 == 0) sx[i / 4] = 0;
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int d = 0; d < 4; ++d) m = max(m, max((v.x[q][d] << 16) & 0x7fffffffu, v.x[q][d] & 0x7fff0000u));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    const uint32_t sb = f8_scale_byte(m);
    const float inv = f8_inv_scale(sb);
    sx[i / 4] |= static_cast<int>(sb << (8 * (i % 4)));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
        fx[i][2 * q + d] =
            static_cast<int>(f8_pack4(bf16_lo(v.x[q][2 * d]) * inv, bf16_hi(v.x[q][2 * d]) * inv,
                                      bf16_lo(v.x[q][2 * d + 1]) * inv, bf16_hi(v.x[q][2 * d + 1]) * inv));
      if constexpr (kU) {
        // columns 16 g + 8 (q % 2) and 64 further: piece 2 g + q % 2 (+ 8) of the block's 16
        const int piece = 16 * (i & 1) + 8 * (q >> 1) + 2 * g + (q & 1);
        const u32x4 a = *reinterpret_cast<const u32x4*>(s_w1 + wv * kChunkBytes + 512 * n + ((piece ^ n) << 4));
        uacc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(a), frag(v.x[q]), uacc, 0, 0, 0);
      }
    }
    // the codes are formed here, not at their uses: the loaded values' registers
    // are free before the next load takes them
    __asm__ volatile("" : "+v"(fx[i]), "+v"(sx[i / 4]));
    __builtin_amdgcn_sched_barrier(0);
    if (i + kRing < NBW) load_x(xa[i % kRing], i + kRing);
    __builtin_amdgcn_sched_barrier(0);
  }
  // s U of this wave's 32 ranks: lane (token n, g) ranks 8 g .. + 7, hi and lo
  const int j0 = 32 * wv + 8 * g;
  float u8[8];
  if constexpr (kU) {  // r <= 16: the waves' sums in order, all in wave 0
    s_u[wv][lane] = uacc;  // D[rank 4 g + e][token n]
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e;
      float u = 0.f;
      if (j < 16) {
#pragma unroll
        for (int v = 0; v < kWaves; ++v) u += s_u[v][16 * (j >> 2) + n][j & 3];
      }
      u8[e] = n < T && j < r ? p.s * u : 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) u8[e] = n < T && j0 + e < r ? p.s * p.U[n * r + j0 + e] : 0.f;
  }
  uint32_t uh[4], ul[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split_bf16x2(u8[2 * e], u8[2 * e + 1], uh[e], ul[e]);
  const bf16x8 fuh = frag(u32x4{uh[0], uh[1], uh[2], uh[3]}), ful = frag(u32x4{ul[0], ul[1], ul[2], ul[3]});
  const bool adapter = 32 * wv < r;  // (uniform)
  auto load_b = [&](int t) {         // row n of tile t, ranks 8 g .. + 7 of the wave's; zero past the last rank
    u32x4 v = {0u, 0u, 0u, 0u};
    if (!adapter || t >= tiles) return v;
    const __amdgpu_buffer_rsrc_t rb = rsrc(p.B + static_cast<int64_t>(t) * 16 * r, 32 * r);
    if (r % 8 == 0) return load16(rb, j0 < r ? static_cast<uint32_t>(n * r + j0) * 2 : kPastEnd);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(
          rb, j0 + e < r ? static_cast<uint32_t>(n * r + j0 + e) * 2 : kPastEnd, 0, 0);
      v[e >> 1] |= b << (16 * (e & 1));
    }
    return v;
  };
  u32x4 bt = load_b(tile);

  // chunk c of a tile from one stage while the next chunk's copies run into the other
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](int t, auto cc, uint8_t* now, uint8_t* other) {
    constexpr int c = decltype(cc)::value;
    __builtin_amdgcn_sched_barrier(0);
    copy(c + 1 < NC ? t : t + step, c + 1 < NC ? c + 1 : 0, other);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0f78);  // vmcnt(8): all but the eight copies just issued have landed
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* base = now + wv * kChunkBytes + 512 * n;
    auto block = [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const u32x4 a = *reinterpret_cast<const u32x4*>(base + (((8 * i + g) ^ n) << 4));
      const u32x4 b = *reinterpret_cast<const u32x4*>(base + (((8 * i + 4 + g) ^ n) << 4));
      const i32x8 fw = {static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                        static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          fw, fx[4 * c + i], acc, 0, 0, 0, __builtin_amdgcn_readlane(sw, 4 * c + i), i, sx[c]);
    };
    block(std::integral_constant<int, 0>{});
    block(std::integral_constant<int, 1>{});
    block(std::integral_constant<int, 2>{});
    block(std::integral_constant<int, 3>{});
  };
  int turn = 0;
  auto finish = [&](int t, int next_s) {
    sw = next_s;
    if (adapter) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(bt), fuh, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(bt), ful, acc, 0, 0, 0);
      bt = load_b(t + step);
    }
    s_acc[turn & 1][wv][lane] = acc;  // D[row 4 g + e][token n]
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    // a barrier for the sums in LDS alone (a fence would also wait for the
    // copies in flight); also: the sums of two turns ago are read
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    if (wv == turn % kWaves && n < T) {
      // rows 4 g .. + 3 of token n: the waves' sums in order
      f32x4 y = s_acc[turn & 1][0][lane];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) y += s_acc[turn & 1][v][lane];
      *reinterpret_cast<u32x2*>(p.Y + static_cast<int64_t>(n) * p.out + static_cast<int64_t>(t) * 16 + 4 * g) =
          u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    }
    ++turn;
  };
  using C0 = std::integral_constant<int, 0>;
  if constexpr (NC == 1) {
    for (; tile < tiles; tile += 2 * step) {
      int next_s = load_s(tile + step);
      chunk(tile, C0{}, s_w0, s_w1);
      finish(tile, next_s);
      if (tile + step >= tiles) break;
      next_s = load_s(tile + 2 * step);
      chunk(tile + step, C0{}, s_w1, s_w0);
      finish(tile + step, next_s);
    }
  } else {
    static_assert(NC == 2, "a tile starts in stage 0");
    for (; tile < tiles; tile += step) {
      const int next_s = load_s(tile + step);
      chunk(tile, C0{}, s_w0, s_w1);
      chunk(tile, std::integral_constant<int, 1>{}, s_w1, s_w0);
      finish(tile, next_s);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no copy is left when the workgroup's LDS goes
}

// Up to 8192 columns: with 16 blocks a wave (in = 14336) the codes of the
// activations no longer fit the registers, and one token took 24.9 us for 4096
// rows against 18.3 by the GEMM (with r = 16 27.7 against 29.0).
bool fp8_decode_fits(int64_t T, int64_t in) { return T <= kDecodeMaxT && in <= 8 * kWaves * kF8Block; }
bool fp8_decode_fuses(int64_t out, int64_t in, int64_t r) { return r <= 16 && out <= 16 * 256 && in <= 4 * kWaves * kF8Block; }

hipError_t launch_fp8_decode(const uint8_t* codes, const uint8_t* scales, int64_t out, int64_t in, const uint16_t* X,
                             int64_t T, const uint16_t* A, const uint16_t* B, int64_t r, float s, const float* u,
                             uint16_t* Y, hipStream_t st) {
  const DecodeF8 p{codes, scales, static_cast<uint32_t>(in), out, X, static_cast<int>(T), A, B, static_cast<int>(r),
                   s, u, Y};
  const int64_t tiles = out / 16, per_wave = ceil_div(ceil_div(in, kF8Block), kWaves);
  const int cus0 = device_cus();
  const int64_t cus = cus0 > 0 ? cus0 : 256;
  const bool fuse = r > 0 && u == nullptr;
  // one workgroup per CU, fewer where that evens out the tiles
  const int64_t rounds = ceil_div(tiles, cus);
  const dim3 grid(static_cast<uint32_t>(ceil_div(tiles, rounds))), block(64 * kWaves);
  if (fuse) hipLaunchKernelGGL((k_fp8_decode<1, true>), grid, block, 0, st, p);
  else if (per_wave <= 4) hipLaunchKernelGGL((k_fp8_decode<1, false>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((k_fp8_decode<2, false>), grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace qlora
