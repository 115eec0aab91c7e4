// k_head.hip -- softmax cross entropy through a frozen output head W [V][H] with
// the gradient of the hidden rows, a piece of the vocabulary at a time; the
// logits exist only in registers.  With s = X W^T log2 e and the label's column y:
//   loss = log(1 + sum_{v != y} 2^(s_v - s_y)),   lse = ln 2 log2 sum 2^s_v
//   dX   = dloss (sum_{v != y} p_v W_v - (1 - p_y) W_y)
// The label's column is kept out of the sums: 1 - p_y is then a sum of positive
// terms, not what is left of 1, and a row that is nearly sure of its label keeps
// the digits of its small loss and gradient.
//
// dX needs no second look at the logits: with E = 2^(s - reference) in bf16,
// sum_v p_v W_v is E W over the row's sum of E, and the sum is known at the end.
// A running maximum as reference would scale what was accumulated, and the tiles
// of one piece that do not know of each other, at nearly every step; but bf16
// has fp32's exponents, so the reference is a multiple of kHeadCell = 128 (a
// "cell", from the tile's maximum), and within its cell E lies below 2^64 and
// the row's largest above 2^-64: what E loses is below 2^-62 of the largest.
// Nearly all logits of a model are in cell 0; where a row's tiles differ,
// k_head_rows scales its E, and what was accumulated before is scaled by the
// next product.  (E's own rounding, 2^-9 of each term, is unbiased and stays
// below dX's.)
//
// k_head_logits (X W^T, weight rows as the matrix cores' first operand, then the
// softmax's part in the epilogue) and k_head_grad (E W, the weight read
// K-row-major through transposing LDS loads) share one main loop: BM x 256 x 64
// tiles, four waves of BM/2 x 128, LDS stages filled by copies straight from
// global memory, fragments of a sub-step read during the one before.
#include <type_traits>

#include "common.hpp"
#include "gemm_tiles.hpp"
#include "nf4_format.hpp"
#include "fp8_format.hpp"

namespace qlora {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();
constexpr int kNW = 4, kBN = 256, kWN = 128;  // waves (2 x 2), tile and wave columns

// x 2^(kHeadCell d), d <= 0 a whole number of cells (two cells and more give 0
// or, of an infinity or a NaN, what it was)
__device__ __forceinline__ float down_cells(float x, float d) {
  return ldexpf(x, static_cast<int>(kHeadCell) * static_cast<int>(fmaxf(d, -4.f)));
}
__device__ __forceinline__ float cell_of(float s) { return rintf(s * (1.f / kHeadCell)); }

// joins (c, s) and (c2, s2), sums in units of 2^(kHeadCell c); c = -inf: nothing
__device__ __forceinline__ void join(float& c, float& s, float c2, float s2) {
  if (c2 == c) {
    s += s2;
  } else if (c2 > c) {
    s = s2 + down_cells(s, c - c2);
    c = c2;
  } else {
    s += down_cells(s2, c2 - c);
  }
}

// Tiles of 64 columns (K), copied straight from global memory into LDS, 1 KB a wave
// instruction and whole 128-byte lines: in halves of lines the second-level cache gets
// twice the requests and bounds the kernel (4096 x 4096 x 16128: 485 us).
//
// Where a tile's data begin and how many bytes from there may be read (the rest
// reads as 0; bytes = 0: nothing is read).
struct Source {
  const uint16_t* base;
  int bytes;
};
__device__ __forceinline__ Source rows_source(const uint16_t* p, int64_t ld, int64_t row0, int64_t rows, int64_t col0) {
  const int64_t n = ((rows - row0) * ld - col0) * 2;
  return Source{p + row0 * ld + col0, static_cast<int>(n < 0x7fffffff ? n : 0x7fffffff)};
}

// ROWS rows of a K-contiguous matrix, as lds_frag reads them.
template <int ROWS>
struct RowTile {
  static constexpr int kPerWave = ROWS / 8 / kNW;
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(int64_t ld, int wv, int lane) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int row = (i * kNW + wv) * 8 + (lane >> 3);
      voff[i] = static_cast<uint32_t>((row * ld + swz(row, lane & 7) * 8) * 2);
    }
  }
  // step k's pieces [first, first + count) of the kPerWave
  __device__ __forceinline__ void load(uint16_t* lds, int wv, const Source& s, int k, int first, int count) const {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(s.base), 0, s.bytes, kBufferWord3);
    const int at = s.bytes != 0 ? k * kBK * 2 : 0;
#pragma unroll
    for (int i = first; i < first + count && i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * kNW + wv) * 512), 16, voff[i], at, 0, 0);
  }
};

// K-row-major weight tile: 64 rows of W (K) by kBN columns, swizzled by tswz for
// col_frag.  A wave instruction copies two rows; lane L lands at 16-byte chunk L % 32 of
// row L / 32 and loads the chunk that belongs there.  Columns past H read the next
// row (never stored), rows past the piece read 0: the resource starts at the step's
// first row (a piece is below 2^31 bytes).
struct ColTile {
  static constexpr int kPerWave = kBK / 2 / kNW;
  int pitch;  // bytes of a row
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(int64_t ld, int wv, int lane) {
    pitch = static_cast<int>(ld * 2);
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int k = (i * kNW + wv) * 2 + (lane >> 5);
      voff[i] = static_cast<uint32_t>((k * ld + ((lane & 31) ^ tswz(k)) * 8) * 2);
    }
  }
  __device__ __forceinline__ void load(uint16_t* lds, int wv, const Source& s, int k, int first, int count) const {
    const int64_t at = static_cast<int64_t>(k) * (kBK * pitch);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(s.base) + at), 0,
        static_cast<int>(at < s.bytes ? s.bytes - at : 0), kBufferWord3);
#pragma unroll
    for (int i = first; i < first + count && i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * kNW + wv) * 512), 16, voff[i], 0, 0, 0);
  }
};

// Fragments of v_mfma_f32_16x16x32_bf16: lane l holds row l % 16 and the eight k from
// 32 j + 8 (l / 16) on.  (This shape and not 32 x 32 x 16: per product it moves half
// of the accumulators and draws less power, which is what bounds the matrix
// cores on random operands: 2050 against 1765 TFLOP/s of nothing but matrix instructions.)
__device__ __forceinline__ bf16x8 row_frag(const uint16_t* lds, int row0, int j) {
  const int l = threadIdx.x & 63;
  return lds_frag(lds, row0 + (l & 15), 4 * j + (l >> 4));
}
// of columns n0 .. n0 + 15 of a ColTile: each group of 16 lanes gets the transposed
// blocks of its eight k (as lds_frag_tr)
__device__ __forceinline__ bf16x8 col_frag(const uint16_t* lds, int n0, int j) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  const int l = threadIdx.x & 63, i = l & 15, n = n0 + 4 * (i & 3);
  v4s v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 32 * j + 8 * (l >> 4) + 4 * h + (i >> 2);
    v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s*)(const_cast<uint16_t*>(lds) + k * kBN + (((n >> 3) ^ tswz(k)) << 3) + (n & 4)));
  }
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// acc[a][c] += weight fragments times activation fragments over a tile's K-steps [k0,
// k0 + steps) of 64; acc[a][c][i] holds row m = wm BM/2 + 16 c + lane % 16 of the
// tile and column n = 128 wn + 16 a + 4 (lane / 16) + i.
//
// Two LDS stages of activations and three of weights, each an array of its own and
// its index a compile-time constant, so that the compiler sees that the copies into one
// stage do not alias the fragment reads of another.  A step is two sub-steps of FN = 8
// groups of matrix instructions, one group per weight fragment.  Fragments are read
// ahead: a weight's six groups before its use, into the register of one that is used
// up, the activations' under the middle of the sub-step before.  After group 1 of the
// second sub-step all of the step's fragments have been read and a barrier frees its
// stages; it also waits for what the next step reads.  The copies of two steps on
// (activations) go out behind it and have a sub-step to land, those of three steps on
// (weights) under the next sub-step and have three.
//
// A workgroup takes one tile after another without a break in this: the steps count on
// into the next tile (steps is rounded up to the six after which both rings are back
// where they began, with copies of zeros), so that its first copies and fragments
// are under way during the last steps and the epilogue.
template <int BM, class TW>
struct HeadLoop {
  static constexpr int FN = kWN / 16, FM = BM / 32;
  static_assert(FN == 8, "the order of the reads below");
  static constexpr bool kTr = std::is_same_v<TW, ColTile>;
  typedef f32x4 Acc[FN][FM];
  uint16_t *s_act[2], *s_wt[3];
  int wv;
  RowTile<BM> ta;
  TW tw;
  int k0, steps;          // of this tile (and of the next, where there is one)
  Source a[2], w[2];      // this tile's and the next one's (bytes 0: none)
  bf16x8 fw[FN], fa[2][FM];

  __device__ __forceinline__ bf16x8 act(int b, int j, int i) const {
    return row_frag(s_act[b], (wv & 1) * (BM / 2) + i * 16, j);
  }
  __device__ __forceinline__ bf16x8 wt(int b, int j, int i) const {
    const int n0 = (wv >> 1) * kWN + i * 16;
    if constexpr (kTr) return col_frag(s_wt[b], n0, j);
    else return row_frag(s_wt[b], n0, j);
  }
  // In assembly, so that the accumulators stay where they are: of the builtin's the
  // compiler moves some at every turn of the loop.  It knows what the operands wait
  // for, but not when the result is there: settle() before the first and after the last.
  __device__ __forceinline__ static void mfma(f32x4& acc, const bf16x8& w, const bf16x8& x) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(w), "v"(x));
  }
  __device__ __forceinline__ static void settle(Acc& acc) {
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int c = 0; c < FM; ++c) asm volatile("" : "+a"(acc[a][c]));
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int c = 0; c < FM; ++c) asm volatile("" : "+a"(acc[a][c]));
  }
  // (not __syncthreads, which would wait for every copy)
  __device__ __forceinline__ static void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  static constexpr int wait_code(int copies) { return (copies & 15) | ((copies >> 4) << 14) | 0x70; }  // lgkmcnt(0) too

  __device__ __forceinline__ static int padded(int n) { return (n + 5) / 6 * 6; }
  static constexpr int kA = RowTile<BM>::kPerWave, kW = TW::kPerWave;  // copies of a wave and step
  // step e counted from this tile's first
  __device__ __forceinline__ static Source source(const Source (&s)[2], int e, int steps, int turn) {
    return Source{e < turn ? s[0].base : s[1].base, e < steps ? s[0].bytes : e < turn || e - turn >= steps ? 0 : s[1].bytes};
  }
  __device__ __forceinline__ void copy_a(int e, int b, int first, int count) const {
    const int turn = padded(steps);
    ta.load(s_act[b], wv, source(a, e, steps, turn), e < turn ? k0 + e : e - turn, first, count);
  }
  __device__ __forceinline__ void copy_w(int e, int b, int first, int count) const {
    const int turn = padded(steps);
    tw.load(s_wt[b], wv, source(w, e, steps, turn), e < turn ? k0 + e : e - turn, first, count);
  }

  // the first copies and fragments of a workgroup's first tile
  __device__ __forceinline__ void begin() {
    copy_a(0, 0, 0, kA);
    copy_w(0, 0, 0, kW);
    copy_w(1, 1, 0, kW);
    copy_a(1, 1, 0, kA);
    __builtin_amdgcn_s_waitcnt(wait_code(kA + kW));
    barrier();
#pragma unroll
    for (int i = 0; i < 6; ++i) fw[i] = wt(0, 0, i);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[0][i] = act(0, 0, i);
  }
  __device__ __forceinline__ void tile(Acc& acc) {
    settle(acc);
    // step e; A, W: its stages
    auto step = [&](int e, auto ac, auto wc) {
      constexpr int A = decltype(ac)::value, W = decltype(wc)::value, NA = A ^ 1, NW = (W + 1) % 3;
      constexpr int kPer = (FM + 3) / 4, kWG = (kW + FN - 1) / FN, kAG = (kA + 3) / 4;
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        if (g < 2) fw[g + 6] = wt(W, 0, g + 6);
        else fw[g - 2] = wt(W, 1, g - 2);
        if (g >= 2 && g < 6)
#pragma unroll
          for (int i = (g - 2) * kPer; i < (g - 1) * kPer && i < FM; ++i) fa[1][i] = act(A, 1, i);
        copy_w(e + 2, (W + 2) % 3, g * kWG, kWG);
#pragma unroll
        for (int c = 0; c < FM; ++c) mfma(acc[g][c], fw[g], fa[0][c]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        if (g == 0) {
          fw[6] = wt(W, 1, 6);
          fw[7] = wt(W, 1, 7);
        }
        if (g == 2) {
          __builtin_amdgcn_s_waitcnt(wait_code(kW));
          barrier();
        }
        if (g >= 2) fw[g - 2] = wt(NW, 0, g - 2);
        if (g >= 2 && g < 6)
#pragma unroll
          for (int i = (g - 2) * kPer; i < (g - 1) * kPer && i < FM; ++i) fa[0][i] = act(NA, 0, i);
        if (g >= 4) copy_a(e + 2, A, (g - 4) * kAG, kAG);
#pragma unroll
        for (int c = 0; c < FM; ++c) mfma(acc[g][c], fw[g], fa[1][c]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    for (int e = 0; e < steps; e += 6) {
      step(e, I0{}, I0{});
      step(e + 1, I1{}, I1{});
      step(e + 2, I0{}, I2{});
      step(e + 3, I1{}, I0{});
      step(e + 4, I0{}, I1{});
      step(e + 5, I1{}, I2{});
    }
    settle(acc);
  }
};

template <int FN, int FM>
__device__ __forceinline__ void clear(f32x4 (&acc)[FN][FM]) {
#pragma unroll
  for (int a = 0; a < FN; ++a)
#pragma unroll
    for (int c = 0; c < FM; ++c) acc[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
}

__device__ __forceinline__ void tile_at(int64_t t, int64_t gm, int64_t gn, int64_t& mt, int64_t& nt) {
  const int64_t per_group = kGroupM * gn, g = t / per_group, left = gm - g * kGroupM;
  const int64_t rows = left < kGroupM ? left : kGroupM, in_g = t - g * per_group;
  mt = g * kGroupM + in_g % rows;
  nt = in_g / rows;
}

// max of three (fmaxf would quiet each operand with an instruction of its own; a NaN is
// passed over either way)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
// over the four lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float max_quarters(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = max3(__builtin_bit_cast(float, static_cast<uint32_t>(x[0])), __builtin_bit_cast(float, static_cast<uint32_t>(x[1])), v);
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto y = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return max3(__builtin_bit_cast(float, static_cast<uint32_t>(y[0])), __builtin_bit_cast(float, static_cast<uint32_t>(y[1])), v);
}
__device__ __forceinline__ float sum_quarters(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __builtin_bit_cast(float, static_cast<uint32_t>(x[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(x[1]));
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto y = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __builtin_bit_cast(float, static_cast<uint32_t>(y[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(y[1]));
}

// The softmax's part of a wave's BM/2 x 128 logits, rows from m0 and columns from n0
// on: the row's cell and sum, the label's logit, E.  (Stores of 16 bytes a lane, 64 a
// row and instruction.  Through LDS they would be whole rows, but the stages already
// hold the next tile.)  Bound by the vector unit, a third of it exponentials.
template <int BM, bool kE>
__device__ __forceinline__ void reduce_tile(const HeadPiece& p, const f32x4 (&acc)[kWN / 16][BM / 32], int64_t m0, int64_t n0) {
  constexpr int FN = kWN / 16, FM = BM / 32;
  const int lane = threadIdx.x & 63, r16 = lane & 15, quarter = lane >> 4;
  const int left = static_cast<int>(p.n - n0 < kWN ? p.n - n0 : kWN);  // valid columns; behind them -inf
  const int64_t block = n0 / kHeadCols;
  // the rows' labels and cells, all loads ahead of the first store (rows past the
  // last one read its)
  const int rows = static_cast<int>(p.T - m0 < BM / 2 ? p.T - m0 : BM / 2);  // this wave's; <= 0: none
  if (rows <= 0) return;
  int label[FM];  // the label's column here, -1: elsewhere
  float before[FM];
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    const int row = c * 16 + r16, at_row = row < rows ? row : rows - 1;
    const uint64_t at = static_cast<uint64_t>(p.labels[m0 + at_row]) - static_cast<uint64_t>(p.v0 + n0);
    label[c] = at < static_cast<uint64_t>(left) && row < rows ? static_cast<int>(at) : -1;
    before[c] = p.first ? -kInf : p.c_in[m0 + at_row];
  }
  // E's rows from m0 on; stores behind the last are dropped
  const uint64_t e_bytes = static_cast<uint64_t>(rows) * p.lde * 2;
  const __amdgpu_buffer_rsrc_t e_rs = __builtin_amdgcn_make_buffer_rsrc(
      kE ? p.E + m0 * p.lde : nullptr, 0, static_cast<int>(e_bytes < 0x7fffffff ? e_bytes : 0x7fffffff), kBufferWord3);
  const uint32_t e_pitch = static_cast<uint32_t>(p.lde * 2);
  const uint32_t e_off = r16 * e_pitch + static_cast<uint32_t>(n0 * 2) + 32 * (quarter & 1) + 16 * (quarter >> 1);
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    // E and sum of the logits s, in units of 2^ref
    const auto finish = [&](const float (&s)[FN][4], float scale, float cell) {
      const float ref = cell == -kInf ? 0.f : cell * kHeadCell;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int a = 0; a < FN; a += 2) {
        uint32_t q[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[a + k][i], scale, -ref));
            sum[k] += e[i];
          }
          q[k][0] = pack_bf16x2(e[0], e[1]);
          q[k][1] = pack_bf16x2(e[2], e[3]);
        }
        if constexpr (kE) {
          // lanes 16 .. 31 and 48 .. 63 of fragment a change places with lanes 0 .. 15
          // and 32 .. 47 of a + 1: each lane then has eight columns in a row
          const auto x = __builtin_amdgcn_permlane16_swap(q[0][0], q[1][0], false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(q[0][1], q[1][1], false, false);
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], y[0], x[1], y[1]}, e_rs, e_off + c * 16 * e_pitch + 32 * a, 0, 0);
        }
      }
      const float total = sum_quarters(sum[0] + sum[1]);
      if (quarter == 0 && c * 16 + r16 < rows) {
        p.tile_c[block * p.T + m0 + c * 16 + r16] = cell;
        p.tile_s[block * p.T + m0 + c * 16 + r16] = total;
      }
    };
    const auto largest = [&](const float (&s)[FN][4]) {
      float top = -kInf;
#pragma unroll
      for (int a = 0; a < FN; ++a) top = max3(s[a][2], s[a][3], max3(s[a][0], s[a][1], top));
      return max_quarters(top);
    };
    float s[FN][4];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[a][i] = acc[a][c][i];
    const float top = largest(s);
    // s - ref is one fused multiply-add.  Its product is not rounded, the cell's was:
    // from 2^31 on they would be further apart than a cell, so of such rows (from
    // 2^23 on) the products are rounded first.
    if (left == kWN && !__any(label[c] >= 0 || fabsf(top) >= 0x1p23f)) {
      finish(s, kLog2e, fmaxf(before[c], cell_of(top * kLog2e)));
    } else {
      // (the accumulators are left as they are: changed in a branch, all of them would
      // be copied out of the matrix cores' registers)
      float target = 0.f, u[FN][4];
      const int mine = label[c] >= 0 ? label[c] - 4 * quarter : -1;
#pragma unroll
      for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool hit = mine == 16 * a + i;
          const float v = acc[a][c][i] * kLog2e;
          target = hit ? v : target;  // the label's logit goes aside
          u[a][i] = hit || 16 * a + 4 * quarter + i >= left ? -kInf : v;
        }
      if (label[c] >= 0 && ((label[c] >> 2) & 3) == quarter) p.target[m0 + c * 16 + r16] = target;
      const float most = largest(u);
      finish(u, 1.f, most == -kInf ? before[c] : fmaxf(before[c], cell_of(most)));
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace

// kE: with E (the gradient's call); else the sums alone.
template <int BM, bool kE>
__global__ __launch_bounds__(256, 1) void k_head_logits(HeadPiece p) {
  constexpr int FN = kWN / 16, FM = BM / 32, WM = BM / 2;
  __shared__ __attribute__((aligned(1024))) uint16_t s_a0[BM * kBK], s_a1[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_w0[kBN * kBK], s_w1[kBN * kBK], s_w2[kBN * kBK];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
  // This workgroup's tiles: XCD x (workgroups x, x + 8, ...) has a contiguous eighth
  // of the sequence, which walks groups of kGroupM row tiles column by column.
  const int64_t gm = ceil_div(p.T, BM), gn = ceil_div(p.n, kBN), total = gm * gn;
  const int64_t xcd = blockIdx.x % kXcds, stride = gridDim.x / kXcds, end = total * (xcd + 1) / kXcds;
  int64_t t = total * xcd / kXcds + blockIdx.x / kXcds;
  if (t >= end) return;

  using TW = RowTile<kBN>;
  HeadLoop<BM, TW> loop{{s_a0, s_a1}, {s_w0, s_w1, s_w2}, wv};
  loop.ta.init(p.H, wv, lane);
  loop.tw.init(p.H, wv, lane);
  loop.k0 = 0;
  loop.steps = static_cast<int>(p.H / kBK);
  int64_t m0, n0, m1 = 0, n1 = 0;
  tile_at(t, gm, gn, m0, n0);
  m0 *= BM;
  n0 *= kBN;
  loop.a[0] = rows_source(p.X, p.H, m0, p.T, 0);
  loop.w[0] = rows_source(p.W, p.H, n0, p.n, 0);
  bool more = false;
  const auto look_ahead = [&]() {
    more = t + stride < end;
    loop.a[1] = Source{p.X, 0};
    loop.w[1] = Source{p.W, 0};
    if (more) {
      tile_at(t + stride, gm, gn, m1, n1);
      m1 *= BM;
      n1 *= kBN;
      loop.a[1] = rows_source(p.X, p.H, m1, p.T, 0);
      loop.w[1] = rows_source(p.W, p.H, n1, p.n, 0);
    }
  };
  look_ahead();
  loop.begin();
  for (;;) {
    f32x4 acc[FN][FM];
    clear(acc);
    loop.tile(acc);
    reduce_tile<BM, kE>(p, acc, m0 + wm * WM, n0 + wn * kWN);
    if (!more) break;
    m0 = m1;
    n0 = n1;
    loop.a[0] = loop.a[1];
    loop.w[0] = loop.w[1];
    t += stride;
    look_ahead();
  }
  __builtin_amdgcn_s_waitcnt(0);  // copies behind the last step
}

// loss and lse of a row from its label's logit t and the sum over the others,
// and what the gradient takes: the others' share of the total, and the factor of what
// was accumulated in units of the others' cell over the total
struct RowLoss {
  float loss, lse, rest, factor;
};
__device__ __forceinline__ RowLoss row_loss(float c, float s, bool has, float t) {
  RowLoss r{0.f, 0.f, 0.f, 0.f};
  float cell = c, total = s;
  if (has) {
    cell = fmaxf(c, t == -kInf ? c : cell_of(t));
    const float d = t - (cell == -kInf ? 0.f : cell * kHeadCell);
    const float scale = c == cell ? 1.f : down_cells(1.f, c - cell), others = c == cell ? s : s * scale;
    total = others + __builtin_amdgcn_exp2f(d);
    // 2^-d times the others, where that is in range
    r.loss = d > -40.f ? log1pf(others * __builtin_amdgcn_exp2f(-d)) : (__builtin_amdgcn_logf(total) - d) * kLn2;
    const float inv = 1.f / total;
    r.rest = others * inv;
    r.factor = scale * inv;
  }
  r.lse = ((cell == -kInf ? 0.f : cell * kHeadCell) + __builtin_amdgcn_logf(total)) * kLn2;
  return r;
}

// Workgroup x: 64 rows; its 16 waves share the piece's blocks of 128 columns.
// Workgroup y scales the E of blocks 16 y, ... of those rows where the block's cell is
// below the row's (one wave instruction a row and block; rare).  Without E the last
// piece's launch writes loss and lse.  Bound by the latency of one round of loads.
constexpr int kRowWaves = 16;
__global__ __launch_bounds__(64 * kRowWaves) void k_head_rows(HeadPiece p, HeadFinish f) {
  __shared__ float sc[kRowWaves][64], ss[kRowWaves][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const bool live = m < p.T;
  const int blocks = static_cast<int>(p.lde / kHeadCols);
  float c = -kInf, s = 0.f;
  for (int t = wv; t < blocks; t += 8 * kRowWaves) {
    float tc[8], ts[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = live && t + kRowWaves * u < blocks;
      tc[u] = in ? p.tile_c[(t + kRowWaves * u) * p.T + m] : -kInf;
      ts[u] = in ? p.tile_s[(t + kRowWaves * u) * p.T + m] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) join(c, s, tc[u], ts[u]);
  }
  sc[wv][lane] = c;
  ss[wv][lane] = s;
  __syncthreads();
  const float before = live && !p.first ? p.c_in[m] : -kInf;
  c = before;
  s = live && !p.first ? p.s_in[m] : 0.f;
#pragma unroll
  for (int i = 0; i < kRowWaves; ++i) join(c, s, sc[i][lane], ss[i][lane]);
  if (blockIdx.y == 0 && wv == 0 && live) {
    if (f.loss != nullptr) {
      const int64_t y = f.labels[m];
      const bool has = y >= 0 && y < f.V;
      const RowLoss r = row_loss(c, s, has, has ? f.target[m] : 0.f);
      f.loss[m] = r.loss;
      if (f.lse != nullptr) f.lse[m] = r.lse;
    } else {
      p.c_out[m] = c;
      p.s_out[m] = s;
      if (p.E != nullptr) p.factor[m] = before == c ? 1.f : down_cells(1.f, before - c);
    }
  }
  if (p.E == nullptr) return;
  for (int t = blockIdx.y * kRowWaves + wv; t < blocks; t += gridDim.y * kRowWaves) {
    const float tc = live ? p.tile_c[t * p.T + m] : c;
    uint64_t todo = __ballot(live && tc != c && tc != -kInf);
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, tc - c), l));
      uint32_t* at = reinterpret_cast<uint32_t*>(p.E + (static_cast<int64_t>(blockIdx.x) * 64 + l) * p.lde +
                                                 static_cast<int64_t>(t) * kHeadCols + 2 * lane);
      const uint32_t v = *at;
      *at = pack_bf16x2(down_cells(bf16_lo(v), d), down_cells(bf16_hi(v), d));
    }
  }
}

template <int BM>
__global__ __launch_bounds__(256, 1) void k_head_grad(HeadPiece p, float* part, int ks) {
  constexpr int FN = kWN / 16, FM = BM / 32, WM = BM / 2;
  __shared__ __attribute__((aligned(1024))) uint16_t s_a0[BM * kBK], s_a1[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_w0[kBN * kBK], s_w1[kBN * kBK], s_w2[kBN * kBK];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1, r16 = lane & 15, quarter = lane >> 4;
  int64_t mt, nt;
  xcd_tile(gridDim.x, gridDim.y, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * kBN;
  const int k0 = static_cast<int>(blockIdx.z) * ks, end = static_cast<int>(p.lde / kBK);
  const int steps = k0 + ks < end ? ks : end > k0 ? end - k0 : 0;

  f32x4 acc[FN][FM];
  clear(acc);
  if (steps > 0) {
    HeadLoop<BM, ColTile> loop{{s_a0, s_a1}, {s_w0, s_w1, s_w2}, wv};
    loop.ta.init(p.lde, wv, lane);
    loop.tw.init(p.H, wv, lane);
    loop.k0 = k0;
    loop.steps = steps;
    loop.a[0] = rows_source(p.E, p.lde, m0, p.T, 0);
    loop.w[0] = rows_source(p.W, p.H, 0, p.n, n0);
    loop.a[1] = Source{p.E, 0};
    loop.w[1] = Source{p.W, 0};
    loop.begin();
    loop.tile(acc);
    __builtin_amdgcn_s_waitcnt(0);  // copies behind the last step
  }
  float* const dst = part + blockIdx.z * p.T * p.H;
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    const int64_t m = m0 + wm * WM + c * 16 + r16;
    if (m >= p.T) continue;
    const float f = p.first ? 0.f : p.factor[m];
#pragma unroll
    for (int a = 0; a < FN; ++a) {
      const int64_t n = n0 + wn * kWN + a * 16 + 4 * quarter;
      if (n >= p.H) continue;
      f32x4* at = reinterpret_cast<f32x4*>(dst + m * p.H + n);
      f32x4 v = acc[a][c];
      if (!p.first) {
        const f32x4 old = *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += f == 1.f ? old[i] : f * old[i];
      }
      *at = v;
    }
  }
}

// Columns col .. col + 7 of the label's row of W.
__device__ __forceinline__ void label_row(const HeadFinish& f, int64_t y, int64_t col, float (&w)[8]) {
  const int64_t at = y * f.H + col;
  if (f.W.w16 != nullptr) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(f.W.w16 + at);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      w[2 * d] = bf16_lo(v[d]);
      w[2 * d + 1] = bf16_hi(v[d]);
    }
  } else if (f.W.scale8 != nullptr) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(f.W.codes + at);
    const float s = f8_scale(f.W.scale8[y / kF8Block * ceil_div(f.H, kF8Block) + col / kF8Block]);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[d]), false);
      const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[d]), true);
      w[4 * d] = a[0] * s;
      w[4 * d + 1] = a[1] * s;
      w[4 * d + 2] = b[0] * s;
      w[4 * d + 3] = b[1] * s;
    }
  } else {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(f.W.codes + at / 2);
    const int64_t blk = at / 64;
    const float a = f.W.absmax_q != nullptr ? dq_absmax(f.W.absmax_q[blk], f.W.scale[blk >> 8]) : f.W.scale[blk];
    uint32_t o[4];
    lookup8(make_table(a), v, o);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      w[2 * d] = bf16_lo(o[d]);
      w[2 * d + 1] = bf16_hi(o[d]);
    }
  }
}

// dX, loss and lse: workgroup (row, 2048 columns).
__global__ __launch_bounds__(256) void k_head_finish(HeadFinish f) {
  const int64_t m = blockIdx.x, col = blockIdx.y * 2048 + threadIdx.x * 8;
  const int64_t y = f.labels[m];
  const bool has = y >= 0 && y < f.V;
  const RowLoss r = row_loss(f.c[m], f.s[m], has, has ? f.target[m] : 0.f);
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    f.loss[m] = r.loss;
    if (f.lse != nullptr) f.lse[m] = r.lse;
  }
  if (col >= f.H) return;
  u32x4 o = {0u, 0u, 0u, 0u};
  if (has) {
    const float g = f.dloss[m];
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    for (int z = 0; z < f.splits; z += 8) {  // in order, eight splits in flight
      f32x4 u[8][2];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float* src = f.part + ((z + k < f.splits ? z + k : 0) * f.T + m) * f.H + col;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          u[k][h] = z + k < f.splits ? *reinterpret_cast<const f32x4*>(src + 4 * h) : f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * h + e] += u[k][h][e];
    }
    label_row(f, y, col, w);
#pragma unroll
    for (int d = 0; d < 4; ++d)
      o[d] = pack_bf16x2(g * (v[2 * d] * r.factor - r.rest * w[2 * d]), g * (v[2 * d + 1] * r.factor - r.rest * w[2 * d + 1]));
  }
  *reinterpret_cast<u32x4*>(f.dX + m * f.H + col) = o;
}

#define HEAD_KERNELS(BM)                                       \
  template __global__ void k_head_logits<BM, true>(HeadPiece);  \
  template __global__ void k_head_logits<BM, false>(HeadPiece); \
  template __global__ void k_head_grad<BM>(HeadPiece, float*, int);
HEAD_KERNELS(64) HEAD_KERNELS(96) HEAD_KERNELS(128) HEAD_KERNELS(160) HEAD_KERNELS(192) HEAD_KERNELS(224) HEAD_KERNELS(256)

namespace {
constexpr int64_t kHeadCus = 256;  // of the part; fixed, so that sizes depend on shapes only

// Rows of a tile.  A round of tiles (one a CU) of 64, 128, 192 and 256 rows takes 53,
// 68, 95 and 107 us at 4096 columns, about 36 + 0.28 rows: the shorter ones read more
// weights a product, so which is best goes by how they fill the rounds.  Measured with
// one height throughout (64 / 128 / 192 / 256), gradient calls: 40 x 50021 x 2304 136 /
// 140 / 146 / 150 us, 200 x 32000 x 4096 203 / 174 / 192 / 200, 301 x 50021 x 2304 350 /
// 285 / 226 / 250, 1024 x 32000 x 4096 722 / 495 / 508 / 440.
constexpr int kHeights[] = {64, 96, 128, 160, 192, 224, 256};
constexpr int64_t height_cost(int rows) { return 128 + rows; }

int logits_rows(int64_t T, int64_t n) {
  int best = 0;
  int64_t least = 0;
  for (int rows : kHeights) {
    const int64_t cost = ceil_div(ceil_div(T, rows) * ceil_div(n, kBN), kHeadCus) * height_cost(rows);
    if (best == 0 || cost < least) best = rows, least = cost;
  }
  return best;
}

// The rows of a tile of E W and the ranges of the vocabulary, each of 1024 columns or
// more: as many as give every CU a workgroup.
struct GradShape {
  int rows, splits;
};
GradShape grad_shape(int64_t T, int64_t H, int64_t n) {
  GradShape best{0, 1};
  int64_t least = 0;
  const int64_t steps = round_up(n, kHeadTile) / kBK;
  for (int rows : kHeights) {
    const int64_t tiles = ceil_div(T, rows) * ceil_div(H, kBN);
    int64_t S = kHeadCus / tiles;
    if (S > steps / 16) S = steps / 16;
    if (S < 1) S = 1;
    const int64_t cost = ceil_div(tiles * S, kHeadCus) * ceil_div(steps, S) * height_cost(rows);
    if (best.rows == 0 || cost < least) best = GradShape{rows, static_cast<int>(S)}, least = cost;
  }
  return best;
}

template <class F>
void with_rows(int rows, F f) {
  if (rows == 64) f(std::integral_constant<int, 64>{});
  else if (rows == 96) f(std::integral_constant<int, 96>{});
  else if (rows == 128) f(std::integral_constant<int, 128>{});
  else if (rows == 160) f(std::integral_constant<int, 160>{});
  else if (rows == 192) f(std::integral_constant<int, 192>{});
  else if (rows == 224) f(std::integral_constant<int, 224>{});
  else f(std::integral_constant<int, 256>{});
}
}  // namespace

hipError_t launch_head_logits(const HeadPiece& p, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(kHeadCus));  // a multiple of the XCDs' number
  with_rows(logits_rows(p.T, p.n), [&](auto b) {
    constexpr int BM = decltype(b)::value;
    if (p.E != nullptr) hipLaunchKernelGGL((k_head_logits<BM, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_head_logits<BM, false>), grid, dim3(256), 0, s, p);
  });
  return hipGetLastError();
}

hipError_t launch_head_rows(const HeadPiece& p, const HeadFinish& f, hipStream_t s) {
  const int64_t blocks = p.lde / kHeadCols;
  const int64_t ys = p.E == nullptr ? 1 : blocks < 8 * kRowWaves ? ceil_div(blocks, kRowWaves) : 8;
  hipLaunchKernelGGL(k_head_rows, dim3(static_cast<uint32_t>(ceil_div(p.T, 64)), static_cast<uint32_t>(ys)),
                     dim3(64 * kRowWaves), 0, s, p, f);
  return hipGetLastError();
}

int head_splits(int64_t T, int64_t H, int64_t n) { return grad_shape(T, H, n).splits; }

hipError_t launch_head_grad(const HeadPiece& p, float* part, int splits, hipStream_t s) {
  // (the last piece and the last round may be smaller: the number of splits stays)
  const int rows = grad_shape(p.T, p.H, p.n).rows;
  const dim3 grid(static_cast<uint32_t>(ceil_div(p.T, rows)), static_cast<uint32_t>(ceil_div(p.H, kBN)),
                  static_cast<uint32_t>(splits));
  const int ks = static_cast<int>(ceil_div(p.lde / kBK, splits));
  with_rows(rows, [&](auto b) {
    constexpr int BM = decltype(b)::value;
    hipLaunchKernelGGL((k_head_grad<BM>), grid, dim3(256), 0, s, p, part, ks);
  });
  return hipGetLastError();
}

hipError_t launch_head_finish(const HeadFinish& f, hipStream_t s) {
  hipLaunchKernelGGL(k_head_finish, dim3(static_cast<uint32_t>(f.T), static_cast<uint32_t>(ceil_div(f.H, 2048))), dim3(256),
                     0, s, f);
  return hipGetLastError();
}

}  // namespace qlora
