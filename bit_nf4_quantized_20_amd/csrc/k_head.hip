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
// next product.  (E's own rounding, up to 2^-8 of each term, is unbiased and over a whole
// dX an eighth of dX's own, 2e-4 beside 1.7e-3; where one term is nearly all of a row's sum, it is
// as large.  E W of 2^24 columns stays in fp32 for weights below 2^39.)
//
// k_head_logits (X W^T, weight rows as the matrix cores' first operand, then the
// softmax's part in the epilogue) and k_head_grad (E W, the weight read
// K-row-major through transposing LDS loads) share one main loop: BM x BN x 64
// tiles, four waves of BM/2 x BN/2, LDS stages filled by copies straight from
// global memory, fragments of a sub-step read during the one before.  4- and 8-bit
// weights come through registers instead and are turned into bf16 on their way into
// LDS (up to kHeadCodesTokens rows; the caller writes them out in bf16 for more).
//
// Measured: loss of 1 x 32000 x 4096 58 to 62 us (262 MB, 4.2 to 4.5 TB/s), of 64 rows in NF4 59;
// gradient of 301 x 50021 x 2304 204 us, of 4096 x 128000 x 4096 6.3 ms, 1360 TFLOP/s.  A
// 256 x 256 tile takes 1.4 us a step of 64, 1.5 PFLOP/s, where the matrix cores on random
// operands are bound by power, and 10 us in front of and behind its steps; with few rows HBM
// bounds or, of 4- and 8-bit weights, the codes' way to the products: through registers, put in
// order, into LDS, past a barrier and out again (2.4 million weights of 4 bits a us; k_decode_stream,
// which has none of that, reaches 5.3).
#include <type_traits>

#include "common.hpp"
#include "gemm_tiles.hpp"
#include "head_shapes.hpp"
#include "nf4_format.hpp"
#include "fp8_format.hpp"

namespace qlora {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();
constexpr int kNW = 4;  // waves, 2 x 2
static_assert(kHeadStep == kBK, "tiles and their choice agree on a step");

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
  const int64_t n = rows > row0 ? ((rows - row0) * ld - col0) * 2 : 0;
  return Source{p + row0 * ld + col0, static_cast<int>(n < 0x7fffffff ? n : 0x7fffffff)};
}

// ROWS rows of a K-contiguous matrix, as lds_frag reads them.
template <int ROWS>
struct RowTile {
  static constexpr bool kQuant = false, kTr = false;
  using Src = Source;
  struct Set {};
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

// K-row-major weight tile: 64 rows of W (K) by BN columns, swizzled by tswz for
// col_frag.  A wave instruction copies two or four rows; lane L lands at 16-byte chunk
// L % kChunks of row L / kChunks and loads the chunk that belongs there.  Columns past H read the next
// row (never stored), rows past the piece read 0: the resource starts at the step's
// first row (a piece is below 2^31 bytes).
template <int BN>
struct ColTile {
  static constexpr bool kQuant = false, kTr = true;
  using Src = Source;
  struct Set {};
  static constexpr int kChunks = BN / 8, kRows = 64 / kChunks, kPerWave = kBK / kRows / kNW;
  int pitch;  // bytes of a row
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(int64_t ld, int wv, int lane) {
    pitch = static_cast<int>(ld * 2);
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int k = (i * kNW + wv) * kRows + lane / kChunks;
      voff[i] = static_cast<uint32_t>((k * ld + ((lane % kChunks) ^ tswz(k)) * 8) * 2);
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

// A tile of a 4- or 8-bit weight on its way into LDS: a lane has BN / 4 weights of a row
// (within one NF4 block), loads their codes and scales into registers two steps ahead of the
// step that writes them to LDS in bf16, where row_frag (kCols: col_frag) reads them.
// Rows past the piece are codes of 0 with scales of 0.
enum { kBf16, kNf4, kFp8 };
struct CodeSource {
  const uint8_t* codes;
  const uint8_t* q;      // NF4: 8-bit absmax, or null; 8 bits: scale bytes
  const float* scale;    // NF4
  int bytes, q_bytes;    // of codes (0: nothing is read) and q
  int phase;             // NF4: blocks of scale's first group in front of codes
};
template <int BN, int F, bool kCols>
struct CodeTile {
  static constexpr bool kQuant = true, kTr = kCols;
  static constexpr int kOwn = BN / 4, kLoads = kOwn / (F == kNf4 ? 32 : 16);  // 16 bytes of codes each
  static constexpr int kPerWave = kLoads + (F == kNf4 ? 2 : 1);  // loads of a step
  static constexpr int kRowShift = F == kNf4 ? 1 : 0;            // 2^-kRowShift bytes a weight
  using Src = CodeSource;
  struct Set {
    u32x4 codes[kLoads];
    uint32_t q;
    float s;
  };
  uint32_t H, voff, block;
  int lds_row, lds_chunk;  // this lane's first element and first chunk
  bool dq;
  Nf4Table table;
  float s8;
  __device__ __forceinline__ void init(int64_t h, int wv, int lane, int64_t n0, bool q) {
    H = static_cast<uint32_t>(h);
    dq = q;
    // (columns: 16 lanes have 16 rows and one chunk, so that their LDS writes meet
    // no bank twice, and a wave reads 16 rows of 256 columns)
    const uint32_t row = kCols ? wv * 16 + (lane & 15) : wv * kOwn + (lane & (kOwn - 1));
    const uint32_t first = kOwn * (kCols ? lane >> 4 : lane / kOwn), col = static_cast<uint32_t>(n0) + first;
    voff = (row * H + col) >> kRowShift;
    if constexpr (F == kNf4) block = row * (H / 64) + col / 64;
    else block = kCols ? col / kF8Block : row / kF8Block * ((H + kF8Block - 1) / kF8Block);
    lds_row = row * (kCols ? BN : kBK);
    lds_chunk = first / 8;
    key = kCols ? tswz(row) : swz(row, 0);
  }
  int key;
  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), kBufferWord3);
  }
  __device__ __forceinline__ void load(Set& c, const Src& s, int k) const {
    const int64_t ahead = kCols ? static_cast<int64_t>(k) * kBK * H >> kRowShift : 0;
    const __amdgpu_buffer_rsrc_t rs = rsrc(s.codes + ahead, s.bytes > ahead ? s.bytes - ahead : 0);
    const int soff = kCols || s.bytes == 0 ? 0 : k * kBK >> kRowShift;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      c.codes[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, voff + 16 * i, soff, 0));
    if constexpr (F == kNf4) {
      const uint32_t b = block + (kCols ? static_cast<uint32_t>(k) * H : k);
      const int blocks = s.bytes >> 5, scales = blocks != 0 ? (blocks + s.phase + kGroup - 1) / kGroup : 0;
      c.q = __builtin_amdgcn_raw_buffer_load_b8(rsrc(s.q, dq ? blocks : 0), b, 0, 0);
      c.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                          rsrc(s.scale, dq ? scales * 4 : blocks * 4),
                                          (dq ? (b + s.phase) / kGroup : b) * 4, 0, 0));
    } else {
      const uint32_t b = block + (k >> 1) * (kCols ? (H + kF8Block - 1) / kF8Block : 1);
      c.q = __builtin_amdgcn_raw_buffer_load_b8(rsrc(s.q, s.bytes != 0 ? s.q_bytes : 0), b, 0, 0);
    }
  }
  // The lane's weights 8 g .. 8 g + 7 into LDS in eight parts of about four instructions,
  // g and u in turn: as many as the matrix cores take in behind one of theirs.
  static constexpr int kParts = 8;
  __device__ __forceinline__ void write(uint16_t* lds, const Set& c, int g, int u) {
    if constexpr (F == kNf4) {
      const uint32_t w = c.codes[g / 4][g % 4];
      if (g == 0 && u == 0) table = make_table(dq ? dq_absmax(c.q, c.s) : c.s);
      if (u == 0 || u == 3) {
        sel = (u == 0 ? w : w >> 4) & 0x07070707u;
        pick = __builtin_amdgcn_bitop3_b32(u == 0 ? w >> 1 : w >> 5, 0x04040404u, 0x03020100u, 0xEA);
      }
      if (u == 1) o[0] = lookup_plane(table.lo, sel, pick);
      if (u == 2) o[1] = lookup_plane(table.hi, sel, pick);
      if (u == 4) o[2] = lookup_plane(table.lo, sel, pick);
      if (u == 5) o[3] = lookup_plane(table.hi, sel, pick);
      if (u == 6) {
        const uint32_t e0 = perm(o[1], o[0], 0x05010400u), e1 = perm(o[1], o[0], 0x07030602u);  // (w0, w2), (w4, w6)
        const uint32_t o0 = perm(o[3], o[2], 0x05010400u), o1 = perm(o[3], o[2], 0x07030602u);  // (w1, w3), (w5, w7)
        o[0] = e0;
        o[1] = e1;
        o[2] = o0;
        o[3] = o1;
      }
      if (u == 7)
        *reinterpret_cast<u32x4*>(lds + lds_row + (((lds_chunk + g) ^ key) << 3)) =
            u32x4{perm(o[2], o[0], 0x05040100u), perm(o[2], o[0], 0x07060302u), perm(o[3], o[1], 0x05040100u),
                  perm(o[3], o[1], 0x07060302u)};
    } else {
      if (g == 0 && u == 0) s8 = f8_scale(c.q);
      if (u % 2 == 0) {
        const int v = static_cast<int>(c.codes[g / 2][g % 2 * 2 + u / 4]);
        const auto a = u % 4 == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8(v, false) : __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
        o[u / 2] = pack_bf16x2(a[0] * s8, a[1] * s8);
      }
      if (u == 7) *reinterpret_cast<u32x4*>(lds + lds_row + (((lds_chunk + g) ^ key) << 3)) = u32x4{o[0], o[1], o[2], o[3]};
    }
  }
  uint32_t sel, pick, o[4];
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
template <int BN>
__device__ __forceinline__ bf16x8 col_frag(const uint16_t* lds, int n0, int j) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  const int l = threadIdx.x & 63, i = l & 15, n = n0 + 4 * (i & 3);
  v4s v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 32 * j + 8 * (l >> 4) + 4 * h + (i >> 2);
    v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s*)(const_cast<uint16_t*>(lds) + k * BN + (((n >> 3) ^ tswz(k)) << 3) + (n & 4)));
  }
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// LDS stages.  Of activations three beside codes, where LDS holds them (the wait for a
// stage is also one for the codes asked for before it, and those come from HBM).  Tiles of
// 128 columns of a bf16 weight, one a CU, wait for HBM: four of both (64 x 32000 x 4096 70
// us instead of 75, 1 x 16000 x 2048 18.8 and 21.6; five 70 and 19.5, six 71.5 and 20.4).
constexpr int kDeep = 4;
constexpr int act_stages(int BM, int BN, bool codes) {
  return codes ? BM <= (BN == 128 ? 64 : 160) ? 3 : 2 : BN == 128 ? kDeep : 2;
}
constexpr int weight_stages(int BN, bool codes) { return !codes && BN == 128 ? kDeep : 3; }

// acc[a][c] += weight fragments times activation fragments over a tile's K-steps [k0,
// k0 + steps) of 64; acc[a][c][i] holds row m = wm BM/2 + 16 c + lane % 16 of the
// tile and column n = wn BN/2 + 16 a + 4 (lane / 16) + i.
//
// NA LDS stages of activations and NW of weights, each an array of its own and
// its index a compile-time constant, so that the compiler sees that the copies into one
// stage do not alias the fragment reads of another.  A step is two sub-steps of FN
// groups of matrix instructions, one group per weight fragment.  Fragments are read
// ahead: a weight's FN - 2 groups before its use, into the register of one that is used
// up, the activations' under the middle of the sub-step before.  After group 1 of the
// second sub-step all of the step's fragments have been read and a barrier frees its
// stages; it also waits for what the next step reads.  The copies of NA steps on
// (activations) go out behind it and have at least a sub-step to land, those of NW
// steps on (weights) under the next sub-step and have at least three.  Codes are asked for NA
// steps before they go to LDS, two steps before their products.
//
// A workgroup takes one tile after another without a break in this: the steps count on
// into the next tile (steps is rounded up to the six, with NA > 2 to a multiple of NA of at
// least six, after which the rings are back where they began, with copies of zeros), so
// that its first copies and fragments are under way during the last steps and the
// epilogue.
template <int BM, int BN, class TW>
struct HeadLoop {
  static constexpr int NA = act_stages(BM, BN, TW::kQuant), NW = weight_stages(BN, TW::kQuant);
  // codes become bf16 between the products (of 64 rows: in front of them, there are too few)
  static constexpr bool kSpread = BM > 64;
  static constexpr int FN = BN / 32, FM = BM / 32, kHalf = FN / 2;
  static_assert(FN == 8 || FN == 4, "the order of the reads below");
  static constexpr bool kTr = TW::kTr, kQuant = TW::kQuant;
  typedef f32x4 Acc[FN][FM];
  uint16_t *s_act[NA], *s_wt[NW];
  int wv;
  RowTile<BM> ta;
  TW tw;
  int k0, steps;          // of this tile (and of the next, where there is one)
  Source a[2];            // this tile's and the next one's (bytes 0: none)
  typename TW::Src w[2];
  typename TW::Set set[NA];
  bf16x8 fw[FN], fa[2][FM];

  __device__ __forceinline__ void stages(uint16_t* const (&a)[kDeep], uint16_t* const (&w)[kDeep]) {
#pragma unroll
    for (int i = 0; i < NA; ++i) s_act[i] = a[i];
#pragma unroll
    for (int i = 0; i < NW; ++i) s_wt[i] = w[i];
  }
  __device__ __forceinline__ bf16x8 act(int b, int j, int i) const {
    return row_frag(s_act[b], (wv & 1) * (BM / 2) + i * 16, j);
  }
  __device__ __forceinline__ bf16x8 wt(int b, int j, int i) const {
    const int n0 = (wv >> 1) * (BN / 2) + i * 16;
    if constexpr (kTr) return col_frag<BN>(s_wt[b], n0, j);
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

  __device__ __forceinline__ static int padded(int n) { return NA == 2 ? (n + 5) / 6 * 6 : (n < 6 ? 6 + NA - 1 : n + NA - 1) / NA * NA; }
  static constexpr int kA = RowTile<BM>::kPerWave, kW = TW::kPerWave;  // copies of a wave and step
  // step e counted from this tile's first
  template <class S>
  __device__ __forceinline__ static S source(const S (&s)[2], int e, int steps, int turn) {
    S r = e < turn ? s[0] : s[1];
    r.bytes = e < steps ? s[0].bytes : e < turn || e - turn >= steps ? 0 : s[1].bytes;
    return r;
  }
  __device__ __forceinline__ void copy_a(int e, int b, int first, int count) const {
    const int turn = padded(steps);
    ta.load(s_act[b], wv, source(a, e, steps, turn), e < turn ? k0 + e : e - turn, first, count);
  }
  __device__ __forceinline__ void copy_w(int e, int b, int first, int count) const {
    const int turn = padded(steps);
    if constexpr (!kQuant) tw.load(s_wt[b], wv, source(w, e, steps, turn), e < turn ? k0 + e : e - turn, first, count);
  }
  __device__ __forceinline__ void codes(int e, int b) {
    const int turn = padded(steps);
    if constexpr (kQuant) tw.load(set[b], source(w, e, steps, turn), e < turn ? k0 + e : e - turn);
  }

  // group g of sub-step j, with its share of the codes' way into LDS between the products
  __device__ __forceinline__ void products(Acc& acc, int g, int j, uint16_t* lds, int b) {
#pragma unroll
    for (int c = 0; c < FM; ++c) {
      mfma(acc[g][c], fw[g], fa[j][c]);
      if constexpr (kQuant && kSpread) {
        constexpr int kShare = TW::kParts / 2;  // a group's
        const int G = j * FN + g;
#pragma unroll
        for (int i = (c * kShare + FM - 1) / FM; i < ((c + 1) * kShare + FM - 1) / FM; ++i)
          tw.write(lds, set[b], G / 2, G % 2 * kShare + i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // the first copies and fragments of a workgroup's first tile
  __device__ __forceinline__ void begin() {
    copy_a(0, 0, 0, kA);
    if constexpr (kQuant) {
      codes(0, 0);
      codes(1, 1);
      copy_a(1, 1, 0, kA);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int g = 0; g < FN * TW::kParts; ++g) tw.write(s_wt[b], set[b], g / TW::kParts, g % TW::kParts);
      }
#pragma unroll
      for (int b = 0; b < NA; ++b) codes(2 + b, b);
      if constexpr (NA == 3) copy_a(2, 2, 0, kA);
      __builtin_amdgcn_s_waitcnt(wait_code(0));
    } else if constexpr (NA == kDeep) {
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        if (e > 0) copy_a(e, e, 0, kA);
        if (e < kDeep - 1) copy_w(e, e, 0, kW);
      }
      __builtin_amdgcn_s_waitcnt(wait_code((kDeep - 2) * (kA + kW) + kA));
    } else {
      copy_w(0, 0, 0, kW);
      copy_w(1, 1, 0, kW);
      copy_a(1, 1, 0, kA);
      __builtin_amdgcn_s_waitcnt(wait_code(kA + kW));
    }
    barrier();
#pragma unroll
    for (int i = 0; i < FN - 2; ++i) fw[i] = wt(0, 0, i);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[0][i] = act(0, 0, i);
  }
  __device__ __forceinline__ void tile(Acc& acc) {
    settle(acc);
    // step e; A, W: its stages
    auto step = [&](int e, auto ac, auto wc) {
      constexpr int A = decltype(ac)::value, W = decltype(wc)::value, A1 = (A + 1) % NA, W1 = (W + 1) % NW, WL = (W + NW - 1) % NW;
      constexpr int kPer = (FM + kHalf - 1) / kHalf, kWG = (kW + FN - 1) / FN, kAG = (kA + kHalf - 1) / kHalf;
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        if (g < 2) fw[g + FN - 2] = wt(W, 0, g + FN - 2);
        else fw[g - 2] = wt(W, 1, g - 2);
        if (g >= 2 && g < 2 + kHalf)
#pragma unroll
          for (int i = (g - 2) * kPer; i < (g - 1) * kPer && i < FM; ++i) fa[1][i] = act(A, 1, i);
        copy_w(e + NW - 1, WL, g * kWG, kWG);
        if constexpr (kQuant && !kSpread) {
#pragma unroll
          for (int u = 0; u < TW::kParts; ++u) tw.write(s_wt[WL], set[A], g, u);
          if (g == FN - 1) codes(e + 2 + NA, A);
        }
        products(acc, g, 0, s_wt[WL], A);
      }
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        if (g == 0) {
          fw[FN - 2] = wt(W, 1, FN - 2);
          fw[FN - 1] = wt(W, 1, FN - 1);
        }
        if (g == 2) {
          __builtin_amdgcn_s_waitcnt(wait_code(NA == 2 ? kW : NA == NW && !kQuant ? (NA - 2) * (kA + kW) : 2 * kW + kA));
          barrier();
        }
        if (g >= 2) fw[g - 2] = wt(W1, 0, g - 2);
        if (g >= 2 && g < 2 + kHalf)
#pragma unroll
          for (int i = (g - 2) * kPer; i < (g - 1) * kPer && i < FM; ++i) fa[0][i] = act(A1, 0, i);
        if (g >= kHalf) copy_a(e + NA, A, (g - kHalf) * kAG, kAG);
        products(acc, g, 1, s_wt[WL], A);
      }
      if constexpr (kQuant && kSpread) codes(e + 2 + NA, A);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    if constexpr (NA == 2) {
      for (int e = 0; e < steps; e += 6) {
        step(e, I0{}, I0{});
        step(e + 1, I1{}, I1{});
        step(e + 2, I0{}, I2{});
        step(e + 3, I1{}, I0{});
        step(e + 4, I0{}, I1{});
        step(e + 5, I1{}, I2{});
      }
    } else {
      for (int e = 0, n = padded(steps); e < n; e += NA) {
        step(e, I0{}, I0{});
        step(e + 1, I1{}, I1{});
        step(e + 2, I2{}, I2{});
        if constexpr (NA > 3) step(e + 3, std::integral_constant<int, 3 % NA>{}, std::integral_constant<int, 3 % NW>{});
      }
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

// (there are below 2^31 tiles; the results are told to be the same in all lanes)
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t gm, uint32_t gn, int64_t& mt, int64_t& nt) {
  const uint32_t per_group = kGroupM * gn, g = t / per_group, left = gm - g * kGroupM;
  const uint32_t rows = left < kGroupM ? left : kGroupM, in_g = t - g * per_group;
  mt = __builtin_amdgcn_readfirstlane(g * kGroupM + in_g % rows);
  nt = __builtin_amdgcn_readfirstlane(in_g / rows);
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
template <int BM, int BN, bool kE>
__device__ __forceinline__ void reduce_tile(const HeadPiece& p, const f32x4 (&acc)[BN / 32][BM / 32], int64_t m0, int64_t n0) {
  constexpr int FN = BN / 32, FM = BM / 32, WN = BN / 2;
  const int lane = threadIdx.x & 63, r16 = lane & 15, quarter = lane >> 4;
  const int left = static_cast<int>(p.n <= n0 ? 0 : p.n - n0 < WN ? p.n - n0 : WN);  // valid columns; behind them -inf
  const int64_t block = n0 / WN;
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
    if (left == WN && !__any(label[c] >= 0 || fabsf(top) >= 0x1p23f)) {
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

// the piece's rows from n0 on
template <int F>
__device__ __forceinline__ auto weight_source(const HeadPiece& p, int64_t n0) {
  if constexpr (F == kBf16) {
    return rows_source(p.W, p.H, n0, p.n, 0);
  } else {
    const int64_t kb = ceil_div(p.H, int64_t(kF8Block)), at = n0 * p.H, rows = p.n > n0 ? p.n - n0 : 0;
    const int64_t n = rows * p.H >> (F == kNf4 ? 1 : 0);
    CodeSource s{};
    s.codes = p.q.codes + (F == kNf4 ? at / 2 : at);
    s.bytes = static_cast<int>(n < 0x7fffffff ? n : 0x7fffffff);
    if constexpr (F == kNf4) {
      s.q = p.q.absmax_q + at / kBlock;
      s.phase = static_cast<int>(at / kBlock % kGroup);
      s.scale = p.q.scale + at / (p.q.absmax_q != nullptr ? kGroupElems : kBlock);
    } else {
      s.q = p.q.scale8 + n0 / kF8Block * kb;
      s.q_bytes = static_cast<int>(ceil_div(rows, int64_t(kF8Block)) * kb);
    }
    return s;
  }
}

// A tile's stages, each an array of its own (those that are not used take no space)
#define HEAD_STAGES(NA, NW)                                                                                          \
  __shared__ __attribute__((aligned(1024))) uint16_t s_a0[BM * kBK], s_a1[BM * kBK], s_a2[NA > 2 ? BM * kBK : 1], s_a3[NA > 3 ? BM * kBK : 1]; \
  __shared__ __attribute__((aligned(1024))) uint16_t s_w0[BN * kBK], s_w1[BN * kBK], s_w2[BN * kBK], s_w3[NW > 3 ? BN * kBK : 1]; \
  uint16_t* const s_a[kDeep] = {s_a0, s_a1, s_a2, s_a3};                                                              \
  uint16_t* const s_w[kDeep] = {s_w0, s_w1, s_w2, s_w3};

// kE: with E (the gradient's call); else the sums alone.
template <int BM, int BN, bool kE, int F>
__global__ __launch_bounds__(256, BN == 128 && F != kBf16 ? 2 : 1) void k_head_logits(HeadPiece p) {
  constexpr int FN = BN / 32, FM = BM / 32, WM = BM / 2;
  HEAD_STAGES(act_stages(BM, BN, F != kBf16), weight_stages(BN, F != kBf16))

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
  // This workgroup's tiles: XCD x (workgroups x, x + 8, ...) has a contiguous eighth
  // of the sequence, which walks groups of kGroupM row tiles column by column.
  const uint32_t gm = static_cast<uint32_t>(ceil_div(p.T, BM)), gn = static_cast<uint32_t>(p.lde / BN), total = gm * gn;
  const uint32_t xcd = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
  const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(total) * (xcd + 1) / kXcds);
  uint32_t t = static_cast<uint32_t>(static_cast<uint64_t>(total) * xcd / kXcds) + blockIdx.x / kXcds;
  if (t >= end) return;

  using TW = std::conditional_t<F == kBf16, RowTile<BN>, CodeTile<BN, F, false>>;
  HeadLoop<BM, BN, TW> loop;
  loop.stages(s_a, s_w);
  loop.wv = wv;
  loop.ta.init(p.H, wv, lane);
  if constexpr (F == kBf16) loop.tw.init(p.H, wv, lane);
  else loop.tw.init(p.H, wv, lane, 0, p.q.absmax_q != nullptr);
  loop.k0 = 0;
  loop.steps = static_cast<int>(p.H / kBK);
  int64_t m0, n0, m1 = 0, n1 = 0;
  tile_at(t, gm, gn, m0, n0);
  m0 *= BM;
  n0 *= BN;
  loop.a[0] = rows_source(p.X, p.H, m0, p.T, 0);
  loop.w[0] = weight_source<F>(p, n0);
  bool more = false;
  const auto look_ahead = [&]() {
    more = t + stride < end;
    loop.a[1] = Source{p.X, 0};
    loop.w[1] = weight_source<F>(p, p.n);
    if (more) {
      tile_at(t + stride, gm, gn, m1, n1);
      m1 *= BM;
      n1 *= BN;
      loop.a[1] = rows_source(p.X, p.H, m1, p.T, 0);
      loop.w[1] = weight_source<F>(p, n1);
    }
  };
  look_ahead();
  loop.begin();
  for (;;) {
    f32x4 acc[FN][FM];
    clear(acc);
    loop.tile(acc);
    reduce_tile<BM, BN, kE>(p, acc, m0 + wm * WM, n0 + wn * (BN / 2));
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
    // The others over the label's own, wherever that quotient is finite: the difference of
    // the logarithms is off by 2^-24 |d|, which is all of a small loss (label at -30, others at -60:
    // -2.6e-6 or 0 instead of 3e-11).  It is not finite only where the loss is large.
    const float ratio = others * __builtin_amdgcn_exp2f(-d);
    r.loss = ratio < kInf ? log1pf(ratio) : (__builtin_amdgcn_logf(total) - d) * kLn2;
    const float inv = 1.f / total;
    r.rest = others * inv;
    r.factor = scale * inv;
  }
  r.lse = ((cell == -kInf ? 0.f : cell * kHeadCell) + __builtin_amdgcn_logf(total)) * kLn2;
  return r;
}

// Workgroup x: 16 rows, which its 16 waves have four times each: 64 shares of the
// piece's blocks of p.cols columns.  Workgroup y scales the E of blocks 64 y, ... of
// those rows where the block's cell is below the row's (one wave instruction a row and
// block; rare).  Without E the last piece's launch writes loss and lse.  Bound by the
// latency of one round of loads.
constexpr int kRowWaves = 16, kRowShares = 4 * kRowWaves;
__global__ __launch_bounds__(64 * kRowWaves) void k_head_rows(HeadPiece p, HeadFinish f) {
  __shared__ float sc[kRowShares][16], ss[kRowShares][16];
  const int lane = threadIdx.x & 63, r16 = lane & 15, share = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16, m = m0 + r16;
  const bool live = m < p.T;
  const int blocks = static_cast<int>(p.lde / p.cols);
  float c = -kInf, s = 0.f;
  for (int t = share; t < blocks; t += 8 * kRowShares) {
    float tc[8], ts[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = live && t + kRowShares * u < blocks;
      tc[u] = in ? p.tile_c[(t + kRowShares * u) * p.T + m] : -kInf;
      ts[u] = in ? p.tile_s[(t + kRowShares * u) * p.T + m] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) join(c, s, tc[u], ts[u]);
  }
  sc[share][r16] = c;
  ss[share][r16] = s;
  __syncthreads();
  // each wave for itself: a quarter of the shares a lane, then the quarters in order
  const int first = (lane >> 4) * (kRowShares / 4);
  c = -kInf;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kRowShares / 4; ++i) join(c, s, sc[first + i][r16], ss[first + i][r16]);
  const float before = live && !p.first ? p.c_in[m] : -kInf;
  float rc = before, rs = live && !p.first ? p.s_in[m] : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) join(rc, rs, __shfl(c, 16 * i + r16), __shfl(s, 16 * i + r16));
  if (blockIdx.y == 0 && threadIdx.x < 16 && live) {
    if (f.loss != nullptr) {
      const int64_t y = f.labels[m];
      const bool has = y >= 0 && y < f.V;
      const RowLoss r = row_loss(rc, rs, has, has ? f.target[m] : 0.f);
      f.loss[m] = r.loss;
      if (f.lse != nullptr) f.lse[m] = r.lse;
    } else {
      p.c_out[m] = rc;
      p.s_out[m] = rs;
      if (p.E != nullptr) p.factor[m] = before == rc ? 1.f : down_cells(1.f, before - rc);
    }
  }
  if (p.E == nullptr) return;
  for (int t0 = blockIdx.y * kRowShares + share / 4 * 4; t0 < blocks; t0 += gridDim.y * kRowShares) {
    const int t = t0 + (lane >> 4);
    const float tc = live && t < blocks ? p.tile_c[t * p.T + m] : -kInf;
    uint64_t todo = __ballot(tc != rc && tc != -kInf);
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, tc - rc), l));
      if (2 * lane >= p.cols) continue;
      uint32_t* at = reinterpret_cast<uint32_t*>(p.E + (m0 + (l & 15)) * p.lde + static_cast<int64_t>(t0 + (l >> 4)) * p.cols +
                                                 2 * lane);
      const uint32_t v = *at;
      *at = pack_bf16x2(down_cells(bf16_lo(v), d), down_cells(bf16_hi(v), d));
    }
  }
}

template <int BM, int BN, int F>
__global__ __launch_bounds__(256, BN == 128 ? 2 : 1) void k_head_grad(HeadPiece p, float* part, int ks) {
  constexpr int FN = BN / 32, FM = BM / 32, WM = BM / 2;
  HEAD_STAGES(act_stages(BM, BN, F != kBf16), weight_stages(BN, F != kBf16))

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1, r16 = lane & 15, quarter = lane >> 4;
  int64_t mt, nt;
  xcd_tile(gridDim.x, gridDim.y, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * BN;
  const int k0 = static_cast<int>(blockIdx.z) * ks, end = static_cast<int>(p.lde / kBK);
  const int steps = k0 + ks < end ? ks : end > k0 ? end - k0 : 0;

  f32x4 acc[FN][FM];
  clear(acc);
  if (steps > 0) {
    using TW = std::conditional_t<F == kBf16, ColTile<BN>, CodeTile<BN, F, true>>;
    HeadLoop<BM, BN, TW> loop;
    loop.stages(s_a, s_w);
    loop.wv = wv;
    loop.ta.init(p.lde, wv, lane);
    if constexpr (F == kBf16) loop.tw.init(p.H, wv, lane);
    else loop.tw.init(p.H, wv, lane, n0, p.q.absmax_q != nullptr);
    loop.k0 = k0;
    loop.steps = steps;
    loop.a[0] = rows_source(p.E, p.lde, m0, p.T, 0);
    if constexpr (F == kBf16) {
      loop.w[0] = rows_source(p.W, p.H, 0, p.n, n0);
      loop.w[1] = Source{p.W, 0};
    } else {
      loop.w[0] = loop.w[1] = weight_source<F>(p, 0);
      loop.w[1].bytes = 0;
    }
    loop.a[1] = Source{p.E, 0};
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
      const int64_t n = n0 + wn * (BN / 2) + a * 16 + 4 * quarter;
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

#define HEAD_LOGITS(BM, BN, F)                                        \
  template __global__ void k_head_logits<BM, BN, true, F>(HeadPiece);  \
  template __global__ void k_head_logits<BM, BN, false, F>(HeadPiece);
#define HEAD_KERNELS(BM, BN, F) \
  HEAD_LOGITS(BM, BN, F) template __global__ void k_head_grad<BM, BN, F>(HeadPiece, float*, int);
#define HEAD_CODES(F)                                                                                     \
  HEAD_KERNELS(32, 128, F) HEAD_KERNELS(64, 128, F) HEAD_KERNELS(128, 128, F) HEAD_KERNELS(96, 256, F) HEAD_KERNELS(128, 256, F) \
  HEAD_KERNELS(160, 256, F) HEAD_KERNELS(192, 256, F) HEAD_KERNELS(256, 256, F)
HEAD_LOGITS(64, 128, kBf16)
HEAD_KERNELS(64, 256, kBf16) HEAD_KERNELS(96, 256, kBf16) HEAD_KERNELS(128, 256, kBf16) HEAD_KERNELS(160, 256, kBf16)
HEAD_KERNELS(192, 256, kBf16) HEAD_KERNELS(224, 256, kBf16) HEAD_KERNELS(256, 256, kBf16)
HEAD_CODES(kNf4)
HEAD_CODES(kFp8)

namespace {
template <int N>
using Int = std::integral_constant<int, N>;
// f(tile rows, tile columns, format)
template <class Fn>
void with_kernel(TileShape t, const HeadWeight& q, Fn f) {
  const auto with = [&](auto fmt) {
    if constexpr (decltype(fmt)::value == kBf16) {
      if (t.cols == 128) return f(Int<64>{}, Int<128>{}, fmt);
      if (t.rows == 64) return f(Int<64>{}, Int<256>{}, fmt);
      if (t.rows == 224) return f(Int<224>{}, Int<256>{}, fmt);
    } else {
      if (t.cols == 128 && t.rows == 32) return f(Int<32>{}, Int<128>{}, fmt);
      if (t.cols == 128 && t.rows == 64) return f(Int<64>{}, Int<128>{}, fmt);
      if (t.cols == 128) return f(Int<128>{}, Int<128>{}, fmt);
    }
    if (t.rows == 96) return f(Int<96>{}, Int<256>{}, fmt);
    if (t.rows == 128) return f(Int<128>{}, Int<256>{}, fmt);
    if (t.rows == 160) return f(Int<160>{}, Int<256>{}, fmt);
    if (t.rows == 192) return f(Int<192>{}, Int<256>{}, fmt);
    f(Int<256>{}, Int<256>{}, fmt);
  };
  if (q.codes == nullptr) with(Int<kBf16>{});
  else if (q.scale8 == nullptr) with(Int<kNf4>{});
  else with(Int<kFp8>{});
}
}  // namespace

hipError_t launch_head_logits(const HeadPiece& p, hipStream_t s) {
  const TileShape t = logits_shape(p.T, p.n, p.q.codes != nullptr);
  const dim3 grid(static_cast<uint32_t>(t.cols == 128 && p.q.codes != nullptr ? 2 * kHeadCus : kHeadCus));  // a multiple of the XCDs' number
  with_kernel(t, p.q, [&](auto bm, auto bn, auto fmt) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, F = decltype(fmt)::value;
    if (p.E != nullptr) hipLaunchKernelGGL((k_head_logits<BM, BN, true, F>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_head_logits<BM, BN, false, F>), grid, dim3(256), 0, s, p);
  });
  return hipGetLastError();
}

hipError_t launch_head_rows(const HeadPiece& p, const HeadFinish& f, hipStream_t s) {
  const int64_t blocks = p.lde / p.cols;
  const int64_t ys = p.E == nullptr ? 1 : blocks < 8 * kRowShares ? ceil_div(blocks, kRowShares) : 8;
  hipLaunchKernelGGL(k_head_rows, dim3(static_cast<uint32_t>(ceil_div(p.T, 16)), static_cast<uint32_t>(ys)),
                     dim3(64 * kRowWaves), 0, s, p, f);
  return hipGetLastError();
}

hipError_t launch_head_grad(const HeadPiece& p, float* part, int splits, hipStream_t s) {
  // (the last piece and the last round may be smaller: the number of splits stays)
  const TileShape t = grad_shape(p.T, p.H, p.n, p.q.codes != nullptr).tile;
  const dim3 grid(static_cast<uint32_t>(ceil_div(p.T, t.rows)), static_cast<uint32_t>(ceil_div(p.H, t.cols)),
                  static_cast<uint32_t>(splits));
  const int ks = static_cast<int>(ceil_div(p.lde / kBK, splits));
  with_kernel(t, p.q, [&](auto bm, auto bn, auto fmt) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, F = decltype(fmt)::value;
    if constexpr (F != kBf16 || BN == 256) hipLaunchKernelGGL((k_head_grad<BM, BN, F>), grid, dim3(256), 0, s, p, part, ks);
  });
  return hipGetLastError();
}

hipError_t launch_head_finish(const HeadFinish& f, hipStream_t s) {
  hipLaunchKernelGGL(k_head_finish, dim3(static_cast<uint32_t>(f.T), static_cast<uint32_t>(ceil_div(f.H, 2048))), dim3(256),
                     0, s, f);
  return hipGetLastError();
}

}  // namespace qlora
