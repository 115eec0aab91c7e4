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
// tiles, eight waves of BM/2 x 64, two LDS stages filled by copies straight from
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
constexpr int kNW = 8, kBN = 256;

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

// K-row-major weight tile: 64 rows of W (K) by kBN columns from n0, swizzled by
// tswz for lds_frag_tr.  A wave instruction copies two rows; lane L lands at
// 16-byte chunk L % 32 of row L / 32 and loads the chunk that belongs there.
// Columns past H read the next row (never stored), rows past the piece read 0:
// the resource starts at the step's first row.
struct DtlTileT {
  static constexpr int kPerWave = kBK / 2 / kNW;
  const uint16_t* base;
  int64_t H, rows;
  uint32_t voff[kPerWave];
  __device__ __forceinline__ void init(const uint16_t* W, int64_t ld, int64_t n0, int64_t nrows, int wv, int lane) {
    base = W;
    H = ld;
    rows = nrows;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int k = (i * kNW + wv) * 2 + (lane >> 5);
      voff[i] = static_cast<uint32_t>((k * ld + n0 + ((lane & 31) ^ tswz(k)) * 8) * 2);
    }
  }
  __device__ __forceinline__ void load(uint16_t* lds, int wv, int64_t k0) const {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(base, H, k0, rows, 2);
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (i * kNW + wv) * 512), 16, voff[i], 0, 0, 0);
  }
};

// acc[a][c] += weight fragments times activation fragments over K-steps [k0,
// k0 + steps); acc[a][c][e] holds row m = wm BM/2 + 32 c + lane % 32 of the
// tile and column n = 64 wn + 32 a + 8 (e / 4) + 4 (lane / 32) + e % 4.
template <int BM, class TW>
struct HeadLoop {
  static constexpr int FN = 2, FM = BM / 64;
  static constexpr bool kTr = std::is_same_v<TW, DtlTileT>;
  typedef bf16x8 Frags[FN + FM];
  uint16_t *s_act[2], *s_wt[2];
  int wv, lane;

  __device__ __forceinline__ void read(Frags& f, int b, int j) const {
    const int half = lane >> 5, r32 = lane & 31, chunk = 2 * j + half, wm = wv & 1, wn = wv >> 1;
#pragma unroll
    for (int a = 0; a < FN; ++a) {
      if constexpr (kTr) f[a] = lds_frag_tr<kBN>(s_wt[b], wn * 64 + a * 32, j);
      else f[a] = lds_frag(s_wt[b], wn * 64 + a * 32 + r32, chunk);
    }
#pragma unroll
    for (int c = 0; c < FM; ++c) f[FN + c] = lds_frag(s_act[b], wm * (BM / 2) + c * 32 + r32, chunk);
  }
  __device__ __forceinline__ static void mfmas(f32x16 (&acc)[FN][FM], const Frags& f) {
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int c = 0; c < FM; ++c)
        acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[a], f[FN + c], acc[a][c], 0, 0, 0);
    // each matrix instruction followed by at most two LDS reads, a copy and
    // address arithmetic
#pragma unroll
    for (int i = 0; i < FN * FM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, kTr ? 2 : 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void run(f32x16 (&acc)[FN][FM], const DtlTile<BM, kNW>& ta, const TW& tw, int64_t k0,
                                      int64_t steps) const {
    const int64_t last = steps - 1;
    auto copy = [&](int64_t e, int b) {  // a step past the end copies the last one again
      const int64_t k = (k0 + (e < last ? e : last)) * kBK;
      ta.load(s_act[b], wv, k);
      tw.load(s_wt[b], wv, k);
    };
    copy(0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    Frags f0, f1;
    read(f0, 0, 0);
    auto step = [&](int64_t e, auto bc) {
      constexpr int B = decltype(bc)::value;
      copy(e + 1, B ^ 1);
      __builtin_amdgcn_s_setprio(1);
      read(f1, B, 1);
      mfmas(acc, f0);
      read(f0, B, 2);
      mfmas(acc, f1);
      read(f1, B, 3);
      mfmas(acc, f0);
      mfmas(acc, f1);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      read(f0, B ^ 1, 0);
    };
    int64_t e = 0;
    for (; e + 2 <= steps; e += 2) {
      step(e, std::integral_constant<int, 0>{});
      step(e + 1, std::integral_constant<int, 1>{});
    }
    if (e < steps) step(e, std::integral_constant<int, 0>{});
  }
};

template <int FN, int FM>
__device__ __forceinline__ void clear(f32x16 (&acc)[FN][FM]) {
#pragma unroll
  for (int a = 0; a < FN; ++a)
#pragma unroll
    for (int c = 0; c < FM; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.f;
}

}  // namespace

template <int BM>
__global__ __launch_bounds__(512, 1) void k_head_logits(HeadPiece p) {
  constexpr int FN = 2, FM = BM / 64, WM = BM / 2;
  __shared__ __attribute__((aligned(1024))) uint16_t s_act0[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_act1[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt0[kBN * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt1[kBN * kBK];
  __shared__ float s_max[4][BM], s_sum[4][BM];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1, r32 = lane & 31, half = lane >> 5;
  int64_t mt, nt;
  xcd_tile(gridDim.x, gridDim.y, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * kBN;

  f32x16 acc[FN][FM];
  clear(acc);
  {
    using TW = DtlTile<kBN, kNW>;
    DtlTile<BM, kNW> ta;
    TW tw;
    ta.init(p.X, p.H, m0, p.T, wv, lane);
    tw.init(p.W, p.H, n0, p.n, wv, lane);
    HeadLoop<BM, TW>{{s_act0, s_act1}, {s_wt0, s_wt1}, wv, lane}.run(acc, ta, tw, 0, p.H / kBK);
  }

  // columns behind the vocabulary count as -inf
  const int64_t left = p.n - n0 - wn * 64;  // valid columns from this wave's first
  if (left < 64) {
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int c = 0; c < FM; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * a + 8 * (e >> 2) + 4 * half + (e & 3) >= left) acc[a][c][e] = -kInf;
  }
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    const int row = wm * WM + c * 32 + r32;
    const int64_t m = m0 + row;
    const int64_t at = m < p.T ? p.labels[m] - p.v0 - n0 - wn * 64 : -1;
    if (__any(at >= 0 && at < 64)) {  // the label's logit goes aside
#pragma unroll
      for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (at == 32 * a + 8 * (e >> 2) + 4 * half + (e & 3)) {
            if (at < left) p.target[m] = acc[a][c][e] * kLog2e;
            acc[a][c][e] = -kInf;
          }
    }
    float top = -kInf;
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[a][c][e]);
    top = fmaxf(top, __shfl_xor(top, 32));
    if (half == 0) s_max[wn][row] = top;
  }
  __syncthreads();  // also: every wave is done reading the stages
  // this wave's 128 x 64 block of E in LDS, rows of eight 16-byte pieces, piece k
  // of row r at slot k ^ (r % 8)
  uint16_t* const s_e = (wv < 2 ? s_act0 : wv < 4 ? s_act1 : wv < 6 ? s_wt0 : s_wt1) + (wv & 1) * (WM * 64);
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    const int row = wm * WM + c * 32 + r32;
    const int64_t m = m0 + row;
    const float top = fmaxf(fmaxf(s_max[0][row], s_max[1][row]), fmaxf(s_max[2][row], s_max[3][row]));
    float cell = top == -kInf ? -kInf : cell_of(top * kLog2e);
    if (!p.first && m < p.T) cell = fmaxf(cell, p.c_in[m]);
    const float ref = cell == -kInf ? 0.f : cell * kHeadCell;
    // s - ref is one fused multiply-add.  Its product is not rounded, the cell's was:
    // from 2^31 on they would be further apart than a cell, so a wave that holds
    // such a row (from 2^23 on) rounds its products first.
    float scale = kLog2e;
    if (__any(fabsf(top) >= 0x1p23f)) {
      scale = 1.f;
#pragma unroll
      for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][c][e] *= kLog2e;
    }
    float sum = 0.f;
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[a][c][4 * g + i], scale, -ref));
          sum += e[i];
        }
        if (p.E != nullptr)
          *reinterpret_cast<u32x2*>(s_e + (c * 32 + r32) * 64 + (((4 * a + g) ^ (row & 7)) * 8) + 4 * half) =
              u32x2{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3])};
      }
    sum += __shfl_xor(sum, 32);
    if (half == 0) s_sum[wn][row] = sum;
    if (wn == 0 && half == 0 && m < p.T) p.tile_c[nt * p.T + m] = cell;
  }
  __syncthreads();
  if (threadIdx.x < BM && m0 + threadIdx.x < p.T)
    p.tile_s[nt * p.T + m0 + threadIdx.x] = s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x] + s_sum[2][threadIdx.x] +
                                            s_sum[3][threadIdx.x];
  if (p.E == nullptr) return;
#pragma unroll
  for (int i = 0; i < WM / 8; ++i) {
    const int row = 8 * i + (lane >> 3), piece = lane & 7;
    const int64_t m = m0 + wm * WM + row;
    const u32x4 v = *reinterpret_cast<const u32x4*>(s_e + row * 64 + ((piece ^ (row & 7)) * 8));
    if (m < p.T) *reinterpret_cast<u32x4*>(p.E + m * p.lde + n0 + wn * 64 + 8 * piece) = v;
  }
}

// Workgroup x: 64 rows; its four waves share the piece's tiles.  Workgroup y
// scales the E of tiles y, y + gridDim.y, ... of those rows where the tile's cell
// is below the row's (one wave instruction a row and tile; rare).
__global__ __launch_bounds__(256) void k_head_rows(HeadPiece p) {
  __shared__ float sc[4][64], ss[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const bool live = m < p.T;
  const int tiles = static_cast<int>(ceil_div(p.n, kHeadTile));
  float c = -kInf, s = 0.f;
  for (int t = wv; t < tiles; t += 16) {
    float tc[4], ts[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = live && t + 4 * u < tiles;
      tc[u] = in ? p.tile_c[(t + 4 * u) * p.T + m] : -kInf;
      ts[u] = in ? p.tile_s[(t + 4 * u) * p.T + m] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) join(c, s, tc[u], ts[u]);
  }
  sc[wv][lane] = c;
  ss[wv][lane] = s;
  __syncthreads();
  const float before = live && !p.first ? p.c_in[m] : -kInf;
  c = before;
  s = live && !p.first ? p.s_in[m] : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) join(c, s, sc[i][lane], ss[i][lane]);
  if (blockIdx.y == 0 && wv == 0 && live) {
    p.c_out[m] = c;
    p.s_out[m] = s;
    if (p.E != nullptr) p.factor[m] = before == c ? 1.f : down_cells(1.f, before - c);
  }
  if (p.E == nullptr) return;
  for (int t = blockIdx.y * 4 + wv; t < tiles; t += gridDim.y * 4) {
    const float tc = live ? p.tile_c[t * p.T + m] : c;
    uint64_t todo = __ballot(live && tc != c && tc != -kInf);
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, tc - c), l));
      u32x2* at = reinterpret_cast<u32x2*>(p.E + (static_cast<int64_t>(blockIdx.x) * 64 + l) * p.lde +
                                           static_cast<int64_t>(t) * kHeadTile + 4 * lane);
      const u32x2 v = *at;
      *at = u32x2{pack_bf16x2(down_cells(bf16_lo(v[0]), d), down_cells(bf16_hi(v[0]), d)),
                  pack_bf16x2(down_cells(bf16_lo(v[1]), d), down_cells(bf16_hi(v[1]), d))};
    }
  }
}

template <int BM>
__global__ __launch_bounds__(512, 1) void k_head_grad(HeadPiece p, float* part, int64_t ks) {
  constexpr int FN = 2, FM = BM / 64, WM = BM / 2;
  __shared__ __attribute__((aligned(1024))) uint16_t s_act0[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_act1[BM * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt0[kBN * kBK];
  __shared__ __attribute__((aligned(1024))) uint16_t s_wt1[kBN * kBK];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1, r32 = lane & 31, half = lane >> 5;
  int64_t mt, nt;
  xcd_tile(gridDim.x, gridDim.y, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * kBN;
  const int64_t k0 = blockIdx.z * ks, end = p.lde / kBK;
  const int64_t steps = k0 + ks < end ? ks : end > k0 ? end - k0 : 0;

  f32x16 acc[FN][FM];
  clear(acc);
  if (steps > 0) {
    DtlTile<BM, kNW> ta;
    DtlTileT tw;
    ta.init(p.E, p.lde, m0, p.T, wv, lane);
    tw.init(p.W, p.H, n0, p.n, wv, lane);
    HeadLoop<BM, DtlTileT>{{s_act0, s_act1}, {s_wt0, s_wt1}, wv, lane}.run(acc, ta, tw, k0, steps);
  }
  float* const dst = part + blockIdx.z * p.T * p.H;
#pragma unroll
  for (int c = 0; c < FM; ++c) {
    const int64_t m = m0 + wm * WM + c * 32 + r32;
    if (m >= p.T) continue;
    const float f = p.first ? 0.f : p.factor[m];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t n = n0 + wn * 64 + a * 32 + 8 * g + 4 * half;
        if (n >= p.H) continue;
        f32x4* at = reinterpret_cast<f32x4*>(dst + m * p.H + n);
        f32x4 v = {acc[a][c][4 * g], acc[a][c][4 * g + 1], acc[a][c][4 * g + 2], acc[a][c][4 * g + 3]};
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

// One workgroup a row.
__global__ __launch_bounds__(256) void k_head_finish(HeadFinish f) {
  const int64_t m = blockIdx.x;
  const int64_t y = f.labels[m];
  const bool has = y >= 0 && y < f.V;
  const float c = f.c[m], s = f.s[m];
  float cell = c, others = s, total = s, loss = 0.f, scale = 1.f;
  if (has) {
    const float t = f.target[m];
    cell = fmaxf(c, t == -kInf ? c : cell_of(t));
    const float d = t - (cell == -kInf ? 0.f : cell * kHeadCell);
    scale = c == cell ? 1.f : down_cells(1.f, c - cell);
    others = c == cell ? s : s * scale;
    total = others + __builtin_amdgcn_exp2f(d);
    // 2^-d times the others, where that is in range
    loss = d > -40.f ? log1pf(others * __builtin_amdgcn_exp2f(-d)) : (__builtin_amdgcn_logf(total) - d) * kLn2;
  }
  if (threadIdx.x == 0) {
    f.loss[m] = loss;
    if (f.lse != nullptr)
      f.lse[m] = ((cell == -kInf ? 0.f : cell * kHeadCell) + __builtin_amdgcn_logf(total)) * kLn2;
  }
  if (f.dX == nullptr) return;
  const float g = has ? f.dloss[m] : 0.f, inv = 1.f / total, rest = others * inv;
  for (int64_t col = threadIdx.x * 8; col < f.H; col += 2048) {
    u32x4 o = {0u, 0u, 0u, 0u};
    if (has) {
      float v[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      for (int z = 0; z < f.splits; ++z) {
        const float* src = f.part + (z * f.T + m) * f.H + col;
        const f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += a[e];
          v[4 + e] += b[e];
        }
      }
      label_row(f, y, col, w);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[d] = pack_bf16x2(g * (v[2 * d] * scale * inv - rest * w[2 * d]),
                           g * (v[2 * d + 1] * scale * inv - rest * w[2 * d + 1]));
    }
    *reinterpret_cast<u32x4*>(f.dX + m * f.H + col) = o;
  }
}

template __global__ void k_head_logits<256>(HeadPiece);
template __global__ void k_head_logits<128>(HeadPiece);
template __global__ void k_head_logits<64>(HeadPiece);
template __global__ void k_head_grad<256>(HeadPiece, float*, int64_t);
template __global__ void k_head_grad<128>(HeadPiece, float*, int64_t);
template __global__ void k_head_grad<64>(HeadPiece, float*, int64_t);

namespace {
constexpr int64_t kHeadCus = 256;  // of the part; fixed, so that sizes depend on shapes only
int head_rows(int64_t T) { return T <= 64 ? 64 : T <= 128 ? 128 : 256; }
}  // namespace

hipError_t launch_head_logits(const HeadPiece& p, hipStream_t s) {
  const int bm = head_rows(p.T);
  const dim3 grid(static_cast<uint32_t>(ceil_div(p.T, bm)), static_cast<uint32_t>(ceil_div(p.n, kBN)));
  if (bm == 64) hipLaunchKernelGGL((k_head_logits<64>), grid, dim3(512), 0, s, p);
  else if (bm == 128) hipLaunchKernelGGL((k_head_logits<128>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((k_head_logits<256>), grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_head_rows(const HeadPiece& p, hipStream_t s) {
  const int64_t tiles = ceil_div(p.n, kHeadTile);
  const int64_t ys = p.E == nullptr ? 1 : tiles < 32 ? ceil_div(tiles, 4) : 8;
  hipLaunchKernelGGL(k_head_rows, dim3(static_cast<uint32_t>(ceil_div(p.T, 64)), static_cast<uint32_t>(ys)), dim3(256),
                     0, s, p);
  return hipGetLastError();
}

// as many ranges of the vocabulary as give every CU a workgroup, each of 16
// steps or more
int head_splits(int64_t T, int64_t H, int64_t n) {
  const int64_t tiles = ceil_div(T, head_rows(T)) * ceil_div(H, kBN), steps = round_up(n, kHeadTile) / kBK;
  int64_t S = kHeadCus / tiles;
  if (S > steps / 16) S = steps / 16;
  return S > 1 ? static_cast<int>(S) : 1;
}

hipError_t launch_head_grad(const HeadPiece& p, float* part, int splits, hipStream_t s) {
  const int bm = head_rows(p.T);
  const dim3 grid(static_cast<uint32_t>(ceil_div(p.T, bm)), static_cast<uint32_t>(ceil_div(p.H, kBN)),
                  static_cast<uint32_t>(splits));
  const int64_t ks = ceil_div(p.lde / kBK, splits);
  if (bm == 64) hipLaunchKernelGGL((k_head_grad<64>), grid, dim3(512), 0, s, p, part, ks);
  else if (bm == 128) hipLaunchKernelGGL((k_head_grad<128>), grid, dim3(512), 0, s, p, part, ks);
  else hipLaunchKernelGGL((k_head_grad<256>), grid, dim3(512), 0, s, p, part, ks);
  return hipGetLastError();
}

hipError_t launch_head_finish(const HeadFinish& f, hipStream_t s) {
  hipLaunchKernelGGL(k_head_finish, dim3(static_cast<uint32_t>(f.T)), dim3(256), 0, s, f);
  return hipGetLastError();
}

}  // namespace qlora
