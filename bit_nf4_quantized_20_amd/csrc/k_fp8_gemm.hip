// k_fp8_gemm.hip -- the 8-bit block-scaled matrix product for gfx950:
//   C[m][n] = sum_k a_hat[m][k] w_hat[n][k]  +  sum_j act1[m][j] wt1[n][j]
// a_hat: e4m3 codes with a power-of-two scale per row and 128 columns;
// w_hat: e4m3 codes with one per 128 x 128 block, read as it is (the forward,
// n = W's rows) or transposed (dX: n = W's columns, k = its rows).  The second
// segment is the adapter, as bf16 hi/lo pairs (gemm_tiles / launch_lora_down
// layouts), added to the same fp32 accumulators before the one rounding.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes a row scale and a column scale per
// instruction, so a 128-wide K-step is two matrix instructions with the same
// scale operands and the scales cost nothing: no per-block rescaling of the
// accumulators on the vector unit.  The weight tile is the A operand, the
// activations B, so a lane ends up with four consecutive n of one row m.
// The matrix cores align an instruction's products before they add them: on
// normal data that leaves 1.5e-5 of the result's size (measured against 64
// bits), which does not grow with the number of steps (the accumulators are
// fp32), against 1.7e-3 for the final rounding to bf16.
//
// A 128-column K-step of 8-bit codes is 128 bytes per row, the same tile row
// that the bf16 kernels use, so tiles are copied straight into LDS with the
// same swizzle.  Within a K-step the order of k is free as long as both
// operands agree: a lane takes the 16-byte chunks 4 j + h and 4 j + 2 + h (h =
// lane / 32) of sub-step j, the conflict-free pattern of the bf16 fragments.
// The transposed tile is stored as it lies in memory (128 rows of k, BN
// columns) and its fragments are read with gfx950's transposing LDS loads.
#include <type_traits>

#include "common.hpp"
#include "fp8_format.hpp"
#include "gemm_tiles.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {

constexpr int kStep = kF8Block;           // K codes (and bytes) per step
constexpr uint32_t kPastEnd = 0x80000000u;

// Weight rows [ROWS] x 128 bytes straight into LDS; the matrix's last K-step
// may hold only 64 codes per row, whose upper chunks then read as zero.
template <int ROWS, int NW>
struct F8Tile {
  static constexpr int kPerWave = ROWS / 8 / NW;
  static_assert(kPerWave >= 1 && NW % 2 == 0, "tile rows");
  __amdgpu_buffer_rsrc_t rs;
  uint32_t voff[kPerWave];
  bool upper;  // this lane copies a chunk of columns 64 .. 127

  __device__ __forceinline__ void init(const uint8_t* base, int64_t ld, int64_t row0, int64_t nrows, int wv, int lane) {
    rs = rows_rsrc(base, ld, row0, nrows, 1);
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int row = (i * NW + wv) * 8 + (lane >> 3);
      voff[i] = static_cast<uint32_t>(row * ld + swz(row, lane & 7) * 16);
    }
    upper = swz(wv * 8 + (lane >> 3), lane & 7) >= 4;  // the same for every i (NW is even)
  }
  __device__ __forceinline__ void load(uint16_t* lds, int wv, int64_t k0, bool half) const {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * NW + wv) * 512), 16,
          half && upper ? kPastEnd : voff[i], static_cast<int>(k0), 0, 0);
  }
};

// Transposed weight tile: rows k0 .. k0 + 127 of W, BN of its columns, kept
// row by row in LDS (BN bytes each).  16-byte chunk c of row k sits at chunk
// c ^ key(k): a fragment read takes 8 consecutive rows at two adjacent chunks
// per 32 lanes, and the key spreads those over all 64 banks.
template <int BN>
__device__ __forceinline__ int f8t_key(int k) {
  return BN == 256 ? 2 * (k & 7) : 2 * ((k >> 1) & 3);
}
template <int BN, int NW>
struct F8TileT {
  static constexpr int kLanesPerRow = BN / 16;
  static constexpr int kRowsPerCopy = 64 / kLanesPerRow;
  static constexpr int kPerWave = kStep / kRowsPerCopy / NW;
  static_assert(BN == 256 || BN == 128, "tile columns");
  const uint8_t* base;
  int64_t ld, nrows;
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(const uint8_t* w, int64_t ldw, int64_t n0, int64_t rows, int wv, int lane) {
    base = w;
    ld = ldw;
    nrows = rows;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int k = (i * NW + wv) * kRowsPerCopy + lane / kLanesPerRow;
      const int64_t col = n0 + (((lane % kLanesPerRow) ^ f8t_key<BN>(k)) * 16);
      // columns past the matrix read nothing (their outputs are not stored)
      voff[i] = col < ldw ? static_cast<uint32_t>(k * ldw + col) : kPastEnd;
    }
  }
  __device__ __forceinline__ void load(uint16_t* lds, int wv, int64_t k0, bool) const {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(base, ld, k0, nrows, 1);  // rows past the last read zero
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * NW + wv) * 512), 16, voff[i], 0, 0, 0);
  }
};

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
               static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}
// fragment of row `row` (n or m), sub-step j of an N-row-major tile
__device__ __forceinline__ i32x8 f8_frag(const uint16_t* lds, int row, int j, int h) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(lds + row * 64 + swz(row, 4 * j + h) * 8);
  const u32x4 b = *reinterpret_cast<const u32x4*>(lds + row * 64 + swz(row, 4 * j + 2 + h) * 8);
  return join(a, b);
}
// The same k of columns n0 .. n0 + 31 from a transposed tile.
// ds_read_b64_tr_b8 hands each group of 16 lanes an 8 x 16 block transposed:
// lane i of the group supplies the address of row i / 2 at columns 8 (i % 2)
// .. + 7 and receives column i of the eight rows.
template <int BN>
__device__ __forceinline__ i32x8 f8_frag_tr(const uint16_t* lds, int n0, int j) {
  const int l = threadIdx.x & 63, i = l & 15, G = l >> 4;
  const int chunk = (n0 >> 4) + (G & 1);
  i32x8 f;
#pragma unroll
  for (int q = 0; q < 2; ++q)     // the two 16-row pieces of this lane's k
#pragma unroll
    for (int s = 0; s < 2; ++s) {  // eight rows each
      const int k = 16 * (4 * j + 2 * q + (G >> 1)) + 8 * s + (i >> 1);
      const uint8_t* p = reinterpret_cast<const uint8_t*>(lds) + k * BN + ((chunk ^ f8t_key<BN>(k)) << 4) + 8 * (i & 1);
      const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) i32x2*)(const_cast<uint8_t*>(p)));
      f[4 * q + 2 * s] = v[0];
      f[4 * q + 2 * s + 1] = v[1];
    }
  return f;
}

struct F8Args {
  int64_t M, N, K;
  const uint8_t* xq; int64_t ldx;            // activation codes [M][ldx], ldx = K rounded up to 128
  const uint32_t* xs; int64_t ldxs;          // their scales [K / 512][ldxs]: four K-blocks' bytes per row, ldxs >= M in whole tiles
  const uint8_t* w; int64_t ldw, wrows;      // weight codes [wrows][ldw]
  const uint8_t* ws; int64_t ws_n, ws_k;     // scale byte of block (n / 128, k / 128): ws[nb ws_n + kb ws_k]
  int64_t ws_bytes;
  const uint16_t* act1; int64_t lda1;        // adapter segment (K1 = 0: none)
  const uint16_t* wt1; int64_t ldw1;
  int64_t K1;
  uint16_t* C; int64_t ldc;
  // split-K: workgroup z takes K-steps [z ks, (z + 1) ks) (ks % 4 == 0), split 0 also the adapter,
  // and writes fp32 partials (fp8_part_frag) instead of C
  float* part; int64_t ks;
  int64_t gm, gn;                            // output tiles (one flat grid dimension)
};

}  // namespace

// BM x BN tile, WM x WN waves, K-steps of 128 codes through two LDS stages.
// Within a step the matrix instructions of the first 64 codes and the first
// fragment's of the second run, then comes the step's one wait and barrier:
// every wave holds the rest of the step in registers, so the stage takes the
// copies of step e + 2 while the second half is computed, and step e + 1's have
// had a whole step in flight.  The activation fragments are single (each is
// read anew behind its last use).  The scale bytes of four steps sit in one
// register per activation fragment (op_sel picks the byte) and are fetched four
// steps ahead.  4096 x 4096 -> 14336: 262 us with the barrier at the step's end
// and both operands' fragments doubled, 230 this way (2.1 PF/s); 4 waves of 128 x
// 128 took 252.  What bounds it is the issue of this sequence: the matrix cores
// are busy for 244 k cycles, 122 us at the 2.0 GHz of these runs, and with
// neither copies nor LDS reads the same instruction order still took 183; the
// LDS reads and the copies with their one wait a step are the rest.
template <int BM, int BN, int WM, int WN, bool kTr>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_fp8_gemm(F8Args p) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static_assert(TN <= 128 && 128 % TN == 0, "a wave's columns share one scale block");
  __shared__ __attribute__((aligned(1024))) uint16_t s_act0[BM * 64];
  __shared__ __attribute__((aligned(1024))) uint16_t s_act1[BM * 64];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt0[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt1[BN * 64];
  uint16_t* const s_act[2] = {s_act0, s_act1};
  uint16_t* const s_wt[2] = {s_wt0, s_wt1};

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv % WM, wn = wv / WM;
  int64_t mt, nt;
  xcd_tile(p.gm, p.gn, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * BN;
  const int r32 = lane & 31, h = lane >> 5;

  f32x16 acc[FN][FM];
#pragma unroll
  for (int a = 0; a < FN; ++a)
#pragma unroll
    for (int c = 0; c < FM; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.f;

  const bool split = p.part != nullptr;
  const int64_t all = (p.K + kStep - 1) / kStep;
  const int64_t first = split ? blockIdx.z * p.ks : 0;
  const int64_t last = split && first + p.ks < all ? first + p.ks : all;  // steps [first, last)
  const bool odd_tail = p.K % kStep != 0;

  // fragments of sub-step j: the weight's for all FN, one of the activations'
  auto read_w = [&](i32x8 (&f)[FN], const uint16_t* sw, int j) {
#pragma unroll
    for (int a = 0; a < FN; ++a) {
      if constexpr (kTr) f[a] = f8_frag_tr<BN>(sw, wn * TN + a * 32, j);
      else f[a] = f8_frag(sw, wn * TN + a * 32 + r32, j, h);
    }
  };
  auto read_a = [&](const uint16_t* sa, int c, int j) { return f8_frag(sa, wm * TM + c * 32 + r32, j, h); };

  // scales of four steps: one dword per activation fragment, the weight's four bytes in one
  struct Scales { int a[FM]; int w; };
  const uint32_t xso = static_cast<uint32_t>(m0 + wm * TM + r32) * 4;
  const __amdgpu_buffer_rsrc_t rws = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.ws), 0, static_cast<int>(p.ws_bytes < 0x7fffffff ? p.ws_bytes : 0x7fffffff), kBufferWord3);
  const uint32_t wso = static_cast<uint32_t>((n0 + wn * TN) / kF8Block * p.ws_n);
  auto load_xs = [&](Scales& s, int64_t e) {  // steps e .. e + 3, e % 4 == 0 (past the last: any group)
    const int64_t g = e < all ? e / 4 : 0;
    const uint8_t* base = reinterpret_cast<const uint8_t*>(p.xs + g * p.ldxs) + xso;
#pragma unroll
    for (int c = 0; c < FM; ++c) s.a[c] = *reinterpret_cast<const int*>(base + 128 * c);
  };
  auto load_ws = [&](int (&raw)[4], int64_t e) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      raw[u] = __builtin_amdgcn_raw_buffer_load_b8(rws, wso + static_cast<uint32_t>((e + u) * p.ws_k), 0, 0);
  };
  auto pack_ws = [&](Scales& s, const int (&raw)[4]) { s.w = raw[0] | raw[1] << 8 | raw[2] << 16 | raw[3] << 24; };

  auto mfma_col = [&](const i32x8 (&w)[FN], const i32x8& f, int c, const Scales& s, auto uc) {
    constexpr int U = decltype(uc)::value;
    __builtin_amdgcn_s_setprio(1);  // matrix instructions go ahead of the other wave's loads
#pragma unroll
    for (int a = 0; a < FN; ++a)
      acc[a][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[a], f, acc[a][c], 0, 0, U, s.w, U, s.a[c]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);  // the operand registers may be loaded anew from here on
  };

  if (last > first) {
    DtlTile<BM, NW> ta;
    std::conditional_t<kTr, F8TileT<BN, NW>, F8Tile<BN, NW>> tw;
    ta.init(reinterpret_cast<const uint16_t*>(p.xq), p.ldx / 2, m0, p.M, wv, lane);
    tw.init(p.w, p.ldw, n0, p.wrows, wv, lane);
    auto copy_act = [&](int64_t e, uint16_t* sa) {  // steps past the end re-read the last one
      ta.load(sa, wv, (e < last ? e : last - 1) * (kStep / 2));
    };
    auto copy_wt = [&](int64_t e, uint16_t* sw) {
      const int64_t k = e < last ? e : last - 1;
      tw.load(sw, wv, k * kStep, odd_tail && k == all - 1);
    };
    Scales cur, nxt;
    int raw[4];
    load_xs(cur, first);
    load_ws(raw, first);
    copy_act(first, s_act0);
    copy_wt(first, s_wt0);
    __builtin_amdgcn_s_waitcnt(0);
    pack_ws(cur, raw);
    __syncthreads();
    copy_act(first + 1, s_act1);
    copy_wt(first + 1, s_wt1);
    i32x8 w0[FN], w1[FN], fa[FM];
    read_w(w0, s_wt0, 0);
#pragma unroll
    for (int c = 0; c < FM; ++c) fa[c] = read_a(s_act0, c, 0);
    auto step = [&](int64_t e, auto uc) {
      constexpr int U = decltype(uc)::value, B = U & 1;
      read_w(w1, s_wt[B], 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < FM; ++c) {
        mfma_col(w0, fa[c], c, cur, uc);
        fa[c] = read_a(s_act[B], c, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      mfma_col(w1, fa[0], 0, cur, uc);
      __builtin_amdgcn_sched_barrier(0);
      // this wave holds the rest of step e, so stage B is free once every
      // wave is here; step e + 1's copies, in flight since the last such
      // point, have landed
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if constexpr (U == 0) {
        load_xs(nxt, e + 4);
        load_ws(raw, e + 4);
      }
      if constexpr (U == 1) pack_ws(nxt, raw);
      read_w(w0, s_wt[B ^ 1], 0);
      fa[0] = read_a(s_act[B ^ 1], 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 1; c < FM; ++c) {
        mfma_col(w1, fa[c], c, cur, uc);
        fa[c] = read_a(s_act[B ^ 1], c, 0);
        __builtin_amdgcn_sched_barrier(0);
        // step e + 2 into the free stage, behind the first reads
        if (c == 1) copy_act(e + 2, s_act[B]);
        if (c == (FM > 2 ? 2 : 1)) copy_wt(e + 2, s_wt[B]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (FM == 1) {
        copy_act(e + 2, s_act[B]);
        copy_wt(e + 2, s_wt[B]);
      }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    int64_t e = first;
    for (; e + 4 <= last; e += 4) {
      step(e, I0{});
      step(e + 1, I1{});
      step(e + 2, I2{});
      step(e + 3, I3{});
      cur = nxt;
    }
    if (e < last) step(e, I0{});
    if (e + 1 < last) step(e + 1, I1{});
    if (e + 2 < last) step(e + 2, I2{});
  }

  // adapter segment: a few bf16 steps of 64 through stage 0
  if (p.K1 > 0 && (!split || blockIdx.z == 0)) {
    DtlTile<BM, NW> ta;
    DtlTile<BN, NW> tw;
    ta.init(p.act1, p.lda1, m0, p.M, wv, lane);
    tw.init(p.wt1, p.ldw1, n0, p.N, wv, lane);
    for (int64_t e = 0; e < p.K1 / kBK; ++e) {
      __syncthreads();  // every wave is done reading stage 0
      ta.load(s_act0, wv, e * kBK);
      tw.load(s_wt0, wv, e * kBK);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 fw[FN], fa[FM];
#pragma unroll
        for (int a = 0; a < FN; ++a) fw[a] = lds_frag(s_wt0, wn * TN + a * 32 + r32, 2 * j + h);
#pragma unroll
        for (int c = 0; c < FM; ++c) fa[c] = lds_frag(s_act0, wm * TM + c * 32 + r32, 2 * j + h);
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
          for (int c = 0; c < FM; ++c)
            acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[a], fa[c], acc[a][c], 0, 0, 0);
      }
    }
  }

  if (BN != 256 && split) {  // 256 x 256 tiles are never split
#pragma unroll
    for (int c = 0; c < FM; ++c)
#pragma unroll
      for (int a = 0; a < FN; ++a) {
        const int64_t m = m0 + wm * TM + c * 32, n = n0 + wn * TN + a * 32;
        if (m >= p.M || n >= p.N) continue;
        f32x4* dst = fp8_part_frag(p.part, blockIdx.z, m / 32, n / 32, p.M, p.N) + lane;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          dst[64 * g] = f32x4{acc[a][c][4 * g], acc[a][c][4 * g + 1], acc[a][c][4 * g + 2], acc[a][c][4 * g + 3]};
      }
    return;
  }
  // each wave parks its TM x TN block in LDS (rows of TN / 8 16-byte pieces,
  // piece q of row r at q ^ (r % 8)) and stores whole rows back, 64 pieces per
  // instruction; lane: m = r32 of fragment c, n = 32 a + 8 g + 4 h + 0 .. 3
  constexpr int kArrays = BM == BN ? 4 : 2, kPerArray = NW / kArrays, kPieces = TN / 8, kRowsPer = 64 / kPieces;
  constexpr int kKey = (kPieces < 8 ? kPieces : 8) - 1;
  static_assert(TM * TN * kPerArray <= BN * 64, "the waves' blocks fit the stage arrays");
  __builtin_amdgcn_s_waitcnt(0);  // the copies behind the last step have landed
  __syncthreads();                // every wave is done reading the stages
  const int array = wv / kPerArray;
  uint16_t* const s_c = (array == 0 ? s_wt0 : array == 1 ? s_wt1 : array == 2 ? s_act0 : s_act1) + (wv % kPerArray) * (TM * TN);
#pragma unroll
  for (int c = 0; c < FM; ++c)
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = c * 32 + r32, piece = 4 * a + g;
        *reinterpret_cast<u32x2*>(s_c + row * TN + ((piece ^ (row & kKey)) * 8) + 4 * h) =
            u32x2{pack_bf16x2(acc[a][c][4 * g], acc[a][c][4 * g + 1]),
                  pack_bf16x2(acc[a][c][4 * g + 2], acc[a][c][4 * g + 3])};
      }
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's block is in LDS
#pragma unroll
  for (int i = 0; i < TM / kRowsPer; ++i) {
    const int row = kRowsPer * i + lane / kPieces, piece = lane % kPieces;
    const int64_t m = m0 + wm * TM + row, n = n0 + wn * TN + 8 * piece;
    const u32x4 v = *reinterpret_cast<const u32x4*>(s_c + row * TN + ((piece ^ (row & kKey)) * 8));
    if (m < p.M && n < p.N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p.C + m * p.ldc + n));
  }
}

__global__ __launch_bounds__(256) void k_fp8_split_sum(const float* part, int S, int64_t M, int64_t N, uint16_t* C) {
  fp8_sum_tile(part, S, M, N, C, blockIdx.x);
}

template __global__ void k_fp8_gemm<256, 256, 2, 4, false>(F8Args);
template __global__ void k_fp8_gemm<256, 256, 2, 4, true>(F8Args);
template __global__ void k_fp8_gemm<128, 128, 2, 2, false>(F8Args);
template __global__ void k_fp8_gemm<128, 128, 2, 2, true>(F8Args);
template __global__ void k_fp8_gemm<64, 128, 2, 2, false>(F8Args);
template __global__ void k_fp8_gemm<64, 128, 2, 2, true>(F8Args);
template __global__ void k_fp8_gemm<32, 128, 1, 4, false>(F8Args);
template __global__ void k_fp8_gemm<32, 128, 1, 4, true>(F8Args);

namespace {
// Rows of a tile: 256 x 256 tiles where they give every CU one (2048 tokens,
// 14336 columns: 109 us, 4096 tokens 2.1 PF/s), else 128 x 128, which hold two
// workgroups per CU (1024 tokens 71 us, 2048 tokens by 4096 columns 46 us for
// 4096 codes).  Below, the grid is filled by splitting K and lower tiles waste
// fewer rows of matrix instructions and partial sums; 4096 -> 14336, 32 / 64 /
// 128 rows: 33 tokens 19.6 / 21.0 / 21.8 us, 64 tokens 20.4 / 21.4 / 21.8, 128
// tokens 24.1 / 23.6 / 26.1, 256 tokens 36.6 / 26.8 / 31.3, 512 tokens - / 52.0 / 36.3.
int f8_tile(int64_t M, int64_t N) {
  if (M <= 64) return 32;
  if (M <= 256) return 64;
  return ceil_div(M, 256) * ceil_div(N, 256) >= 256 ? 256 : 128;
}
}  // namespace

// Split-K: grids below two workgroups per CU (of a 256-CU part; the count
// depends on the shape only) split K into ranges of at least eight steps, at
// most 16, with at most 64 MiB of partials.  Ranges of four steps (eight): 64
// tokens 4096 x 4096 17.9 us (16.2); K = 1088 in two ranges (unsplit): 301 tokens
// 19.5 us (14.5).  One workgroup per CU (two): 301 tokens 4096 x 14336 50.7 us
// (40.5); four per CU 50.1.
int fp8_splits(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kTarget = 512, kMaxSplits = 16, kMaxPartBytes = int64_t(64) << 20;
  if (M <= 0 || N <= 0) return 1;
  const int64_t bm = f8_tile(M, N);
  if (bm == 256) return 1;
  const int64_t steps = ceil_div(K, kStep);
  int64_t S = kTarget / (ceil_div(M, bm) * ceil_div(N, 128));
  if (S > kMaxSplits) S = kMaxSplits;
  if (S > ceil_div(steps, 8)) S = ceil_div(steps, 8);
  if (S > kMaxPartBytes / (M * N * 4)) S = kMaxPartBytes / (M * N * 4);
  if (S < 2 || steps < 16) return 1;  // a short K: the sum's launch costs more than the steps it saves
  const int64_t ks = round_up(ceil_div(steps, S), 4);
  return static_cast<int>(ceil_div(steps, ks));
}

size_t fp8_split_bytes(int64_t M, int64_t N, int64_t K) {
  const int S = fp8_splits(M, N, K);
  return S > 1 ? static_cast<size_t>(S) * round_up(M, 32) * N * 4 : 0;
}

hipError_t launch_fp8_gemm(const F8Gemm& g, hipStream_t s) {
  const bool tr = g.transposed;
  F8Args a{};
  a.M = g.M;
  a.N = tr ? g.cols : g.rows;
  a.K = tr ? g.rows : g.cols;
  a.xq = g.xq;
  a.ldx = round_up(a.K, kF8Block);
  a.xs = reinterpret_cast<const uint32_t*>(g.xs);
  a.ldxs = fp8_row_pitch(g.M);
  a.w = g.codes;
  a.ldw = g.cols;
  a.wrows = g.rows;
  const int64_t cb = ceil_div(g.cols, kF8Block);
  a.ws = g.scales;
  a.ws_n = tr ? 1 : cb;
  a.ws_k = tr ? cb : 1;
  a.ws_bytes = cb * ceil_div(g.rows, kF8Block);
  a.act1 = g.act1; a.lda1 = g.lda1; a.wt1 = g.wt1; a.ldw1 = g.ldw1; a.K1 = g.K1;
  a.C = g.C;
  a.ldc = a.N;
  const int S = fp8_splits(a.M, a.N, a.K);
  const int bm = f8_tile(a.M, a.N), bn = bm == 256 ? 256 : 128;
  a.gm = ceil_div(a.M, bm);
  a.gn = ceil_div(a.N, bn);
  dim3 grid(static_cast<uint32_t>(a.gm * a.gn), 1, 1);
  if (S > 1) {
    a.part = g.part;
    a.ks = round_up(ceil_div(ceil_div(a.K, kStep), S), 4);
    grid.z = static_cast<uint32_t>(S);
  }
  if (bm == 256) {
    if (tr) hipLaunchKernelGGL((k_fp8_gemm<256, 256, 2, 4, true>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_gemm<256, 256, 2, 4, false>), grid, dim3(512), 0, s, a);
  } else if (bm == 128) {
    if (tr) hipLaunchKernelGGL((k_fp8_gemm<128, 128, 2, 2, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_gemm<128, 128, 2, 2, false>), grid, dim3(256), 0, s, a);
  } else if (bm == 64) {
    if (tr) hipLaunchKernelGGL((k_fp8_gemm<64, 128, 2, 2, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_gemm<64, 128, 2, 2, false>), grid, dim3(256), 0, s, a);
  } else {
    if (tr) hipLaunchKernelGGL((k_fp8_gemm<32, 128, 1, 4, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_gemm<32, 128, 1, 4, false>), grid, dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && S > 1 && !g.keep_parts) {
    hipLaunchKernelGGL(k_fp8_split_sum, dim3(static_cast<uint32_t>(fp8_sum_blocks(a.M, a.N))), dim3(256), 0, s,
                       static_cast<const float*>(g.part), S, a.M, a.N, a.C);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qlora
