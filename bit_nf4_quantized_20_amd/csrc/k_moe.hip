// k_moe.hip -- mixture-of-experts operators for gfx950: the router's top-k
// with its gradient, and the whole expert layer for a few tokens over NF4
// experts (k_moe_gate_up + k_moe_down).
#include <type_traits>

#include "common.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {
constexpr float kNegInf = -__builtin_inff();

// ---------------------------------------------------------------- router
// Order of the logits as unsigned integers: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t sort_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}

template <int G>
__device__ __forceinline__ float sum_group(float v) {
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float max_group(float v) {
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
}  // namespace

// One group of G lanes per row; lane i of the group holds logits i + G e,
// e < PER.  k rounds of an arg max over the group: the key of a logit joined
// with its complemented index, so equal logits go to the lower index.  A
// chosen logit's key becomes 0 (no logit has key 0: the smallest, -inf, is
// 0x007fffff).  Bound by the rounds' shuffles, not by memory: 16384 x 128, k = 8,
// 11 us for 9.4 MB; a call from the binding takes 8 us of the host.
template <int G, int PER>
__global__ __launch_bounds__(256) void k_moe_route(const float* __restrict__ logits, int64_t T, int E, int k,
                                                   int renorm, int* __restrict__ ids, float* __restrict__ weights) {
  const int sub = threadIdx.x % G;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / G;
  const bool live = row < T;  // dead groups run along (their loads and stores are off)
  const float* lr = logits + (live ? row : 0) * E;
  float x[PER];
  uint32_t key[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int i = sub + G * e;
    x[e] = live && i < E ? lr[i] : kNegInf;
    key[e] = i < E ? sort_key(x[e]) : 0u;
  }
  float top = 0.f, total = 0.f;  // the largest logit; sum of exp(x - top) over the chosen (renorm) or all
  float mine = 0.f;              // lane j: the j-th chosen logit, lane's id below
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t bk = 0, bi = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e)
      if (key[e] > bk) {
        bk = key[e];
        bi = static_cast<uint32_t>(sub + G * e);
      }
    uint64_t best = (static_cast<uint64_t>(bk) << 32) | (0xffffffffu - bi);
#pragma unroll
    for (int o = G / 2; o >= 1; o >>= 1) {
      const uint64_t other = (static_cast<uint64_t>(static_cast<uint32_t>(__shfl_xor(static_cast<int>(best >> 32), o))) << 32) |
                             static_cast<uint32_t>(__shfl_xor(static_cast<int>(best), o));
      best = other > best ? other : best;
    }
    const int id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    float v = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e)
      if (id == sub + G * e) {
        key[e] = 0;
        v = x[e];
      }
    v = __shfl(v, id % G, G);
    if (j == 0) top = v;
    if (sub == j) {
      mine = v;
      my_id = id;
    }
    if (renorm) total += expf(v - top);
  }
  const bool empty = top == kNegInf;  // nothing but -inf: weights 0
  if (!renorm) {
#pragma unroll
    for (int e = 0; e < PER; ++e)
      if (sub + G * e < E) total += expf(x[e] - top);
    total = sum_group<G>(total);
  }
  if (live && sub < k) {
    ids[row * k + sub] = my_id;
    weights[row * k + sub] = empty ? 0.f : expf(mine - top) / total;
  }
}

// Gradient of the logits: with p the softmax over the chosen logits (renorm)
// or over all, dl_e = p_e (g_e - sum g p), g_e the gradient of e's weight (0
// where e was not chosen).  Ids outside [0, E) count as no choice.  16384 x 128:
// 7.8 us for 17.8 MB.
template <int G, int PER>
__global__ __launch_bounds__(256) void k_moe_route_bwd(const float* __restrict__ logits, const int* __restrict__ ids,
                                                       const float* __restrict__ dw, int64_t T, int E, int k,
                                                       int renorm, float* __restrict__ dl) {
  const int sub = threadIdx.x % G;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / G;
  const bool live = row < T;
  const int64_t rr = live ? row : 0;
  float x[PER], g[PER];
  uint32_t chosen = 0;
  int my_id = -1;
  float my_g = 0.f;
  if (sub < k) {
    my_id = ids[rr * k + sub];
    my_g = dw[rr * k + sub];
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int i = sub + G * e;
    x[e] = i < E ? logits[rr * E + i] : kNegInf;
    g[e] = 0.f;
  }
  for (int j = 0; j < k; ++j) {
    const int id = __shfl(my_id, j, G);
    const float gj = __shfl(my_g, j, G);
#pragma unroll
    for (int e = 0; e < PER; ++e)
      if (id == sub + G * e && id < E) {
        g[e] += gj;
        chosen |= 1u << e;
      }
  }
  float top = kNegInf;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if (renorm && !((chosen >> e) & 1u)) x[e] = kNegInf;
    if (x[e] == kNegInf) g[e] = 0.f;  // a masked choice: no weight, so no infinity or NaN of its gradient either
    top = fmaxf(top, x[e]);
  }
  top = max_group<G>(top);
  float total = 0.f, dot = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    x[e] = x[e] == kNegInf ? 0.f : expf(x[e] - top);
    total += x[e];
    dot += x[e] * g[e];
  }
  total = sum_group<G>(total);
  dot = sum_group<G>(dot);
  // a row of nothing but -inf adds up to 0; the largest of NaNs is -inf too
  // (fmaxf passes them over), but their total is NaN
  const float inv = total == 0.f ? 0.f : 1.0f / total;
  dot *= inv;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    if (live && sub + G * e < E) dl[row * E + sub + G * e] = x[e] * inv * (g[e] - dot);
}

// ------------------------------------------------------------- experts
//
// Both products are the same panel product: 16-row tiles of an expert's NF4
// rows against the columns of the pairs (token, choice) that chose it.  A
// workgroup takes one expert and a range of its rows; kw of its waves share a
// row group and split the reduction, the others take further row groups.  A wave walks its 64-weight blocks in chunks of four (lane (n = l %
// 16, g = l / 16): block g of the chunk of row n): the columns' values of the
// chunk go into registers once and meet RB row tiles, whose codes are
// dequantized in registers (MFMA A operand) with their loads kDepth tiles
// ahead.  The vector unit's 3.5 instructions per weight and HBM bound it
// alike (16 rows x 256 weights: 900 cycles of a SIMD and 2.1 KB), so each
// expert is read and dequantized once for all its pairs of a column tile.
namespace {
constexpr int kPairs = kMoeMaxPairs;
// Shapes of a workgroup: waves, 16-row tiles per wave (RB) and tiles of codes
// in flight (kDepth).  Measured at 9 tokens over 8 experts of 4096 x 14336 /
// 64 tokens over 128 of 2048 x 768, gate and up product: 4 waves, RB 4, depth
// 1 at four waves per SIMD 118 / 68 us; depth 2 at three 125 / 72; depth 4
// at two 144 / 86; 8 waves 149 / 86.  Down product: 8 waves, RB 8, depth 2 77 /
// 37 us; RB 4 89 / 46; 4 waves, RB 8 87 / 36.
constexpr int kUpWaves = 4, kUpTiles = 4, kUpDepth = 1;
constexpr int kDownWaves = 8, kDownTiles = 8, kDownDepth = 2;
constexpr int kFewWaves = 8;  // where there are few workgroups
constexpr uint32_t kPastEnd = 0x80000000u;  // past every buffer (all < 2^31 bytes)
constexpr int kBufferWord3 = 0x00020000;
constexpr int kStreamOnce = 2;              // cache policy nt

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), kBufferWord3);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, int aux) {
  // aux has to be a constant of the instruction
  return __builtin_bit_cast(u32x4, aux ? __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kStreamOnce)
                                       : __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// One lane's 64-weight block: 32 code bytes, absmax code, group scale.
struct Blk {
  u32x4 c0, c1;
  uint32_t q;
  float sc;
};

// An expert's rows (rows x nb blocks from block b of the whole weight on):
// codes, absmax codes, and the group scales from its first block's group on,
// with that block's place in the group.
struct ExpertRows {
  __amdgpu_buffer_rsrc_t rc, rq, rs;
  uint32_t rem;
  __device__ __forceinline__ ExpertRows(const MoeWeight& w, int64_t row0, uint32_t rows, uint32_t nb) {
    const int64_t b = row0 * nb;
    const uint32_t blocks = rows * nb;
    rem = static_cast<uint32_t>(b & 255);
    rc = rsrc(w.codes + b * 32, blocks * 32);
    rq = rsrc(w.absmax_q + b, blocks);
    rs = rsrc(w.scale + (b >> 8), ((rem + blocks + 255) >> 8) * 4);
  }
  // block b (counted from the expert's first row); off = kPastEnd: all zero
  __device__ __forceinline__ void load(Blk& o, uint32_t b, uint32_t off) const {
    o.c0 = load16(rc, (b * 32) | off, 1);
    o.c1 = load16(rc, (b * 32 + 16) | off, 1);
    o.q = __builtin_amdgcn_raw_buffer_load_b8(rq, b | off, 0, 0);
    o.sc = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (((rem + b) >> 8) * 4) | off, 0, 0));
  }
};

__device__ __forceinline__ bf16x8 as_frag(const uint32_t (&w)[4]) {
  return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}

// The pairs of one expert, found by every workgroup from the ids: a slot is
// an expert where there are no more experts than pairs, else a pair, whose
// workgroups work only if it is its expert's first pair.  Returns the expert
// (-1: nothing to do) and leaves its pairs in ascending order at list.  Up to
// 64 pairs every wave does this by itself (no barrier before its first weight
// loads); more are staged in LDS.
template <int NW>
struct PairList {
  int ids[kPairs];
  uint16_t all[kPairs];
  uint16_t per_wave[NW][64];
  int n;
};
__device__ __forceinline__ uint64_t lanes_below() { return (uint64_t(1) << (threadIdx.x & 63)) - 1; }
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
template <int NW>
__device__ __forceinline__ int find_pairs(PairList<NW>& s, const MoeArgs& a, int slot, const uint16_t*& list, int& nc) {
  const int tid = threadIdx.x, lane = tid & 63, P = a.T * a.k;
  if (P <= 64) {
    const int id = lane < P ? a.ids[lane] : -1;
    const int e = a.by_expert ? slot : __builtin_amdgcn_readlane(id, slot);
    if (e < 0 || e >= a.E) return -1;
    const uint64_t hit = __ballot(id == e);
    if (hit == 0 || (!a.by_expert && (hit & ((uint64_t(1) << slot) - 1)) != 0)) return -1;
    uint16_t* mine = s.per_wave[tid >> 6];
    if (id == e) mine[__popcll(hit & lanes_below())] = static_cast<uint16_t>(lane);
    wave_lds_sync();
    list = mine;
    nc = __popcll(hit);
    return e;
  }
  for (int i = tid; i < P; i += 64 * NW) {
    const int e = a.ids[i];
    s.ids[i] = e >= 0 && e < a.E ? e : -1;  // -1: no expert
  }
  __syncthreads();
  const int e = a.by_expert ? slot : s.ids[slot];
  if (tid < 64) {
    int n = 0;
    if (e >= 0)
      for (int b = 0; b < P; b += 64) {
        const bool hit = b + lane < P && s.ids[b + lane] == e;
        const uint64_t m = __ballot(hit);
        if (hit) s.all[n + __popcll(m & lanes_below())] = static_cast<uint16_t>(b + lane);
        n += __popcll(m);
      }
    if (lane == 0) s.n = n;
  }
  __syncthreads();
  list = s.all;
  nc = s.n;
  if (e < 0 || nc == 0 || (!a.by_expert && s.all[0] != slot)) return -1;
  return e;
}

// Workgroup -> slot, row range, and which of the range's column workgroups;
// those are eight apart, on one XCD, so that they share the weights in its L2.
// False: past the last.
__device__ __forceinline__ bool place(const MoeArgs& a, int& slot, int& range, int& col) {
  const int lin = blockIdx.x, w = lin / (8 * a.cols) * 8 + lin % 8;
  col = lin / 8 % a.cols;
  range = w % a.ranges;
  slot = w / a.ranges;
  return slot < a.slots;
}

// acc[r][t] += rows of tile r (row offsets trow[r], in blocks, of this lane's
// row) times the columns of tile t, over blocks [b0, b1).  The columns' values
// lie at colf[t] (byte offsets in rx; kPastEnd: zero column), 128 bytes per
// block, with kHiLo a second plane lo bytes further that is added in.
template <int RB, int NT, bool kHiLo, int kDepth>
__device__ __forceinline__ void panel(f32x4 (&acc)[RB][NT], const ExpertRows& w, const uint32_t (&trow)[RB],
                                      __amdgpu_buffer_rsrc_t rx, const uint32_t (&colf)[NT], uint32_t lo, int b0,
                                      int b1) {
  static_assert(RB % kDepth == 0, "tiles of a chunk use the code registers in turn");
  const int g = (threadIdx.x & 63) >> 4;
  const uint32_t none = kPastEnd;
  Blk buf[kDepth];
#pragma unroll
  for (int r = 0; r < kDepth; ++r) w.load(buf[r], trow[r] + b0 + g, b0 + g < b1 ? 0u : none);
  for (int b = b0; b < b1; b += 4) {
    const uint32_t off = b + g < b1 ? 0u : none, next = b + 4 + g < b1 ? 0u : none;
    bf16x8 xh[8][NT], xl[kHiLo ? 8 : 1][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t at = (colf[t] + static_cast<uint32_t>(b + g) * 128) | off;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u32x4 v = load16(rx, at + 16 * j, 0);
        const uint32_t vi[4] = {v[0], v[1], v[2], v[3]};
        uint32_t o[4];
        to_split_order(vi, o);
        xh[j][t] = as_frag(o);
        if constexpr (kHiLo) {
          const u32x4 u = load16(rx, at + lo + 16 * j, 0);
          const uint32_t ui[4] = {u[0], u[1], u[2], u[3]};
          to_split_order(ui, o);
          xl[j][t] = as_frag(o);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const Blk cur = buf[r % kDepth];
      if (r + kDepth < RB) w.load(buf[r % kDepth], trow[r + kDepth] + b + g, off);
      else w.load(buf[r % kDepth], trow[(r + kDepth) % RB] + b + 4 + g, next);
      const Nf4Table tab = make_table(dq_absmax(cur.q, cur.sc));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t o[4];
        lookup8_split(tab, j < 4 ? cur.c0[j] : cur.c1[j - 4], o);
        const bf16x8 f = as_frag(o);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, xh[j][t], acc[r][t], 0, 0, 0);
          if constexpr (kHiLo) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, xl[j][t], acc[r][t], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // one tile's tables and lookups in registers at a time
    }
  }
}

// Adds the KW waves' accumulators of a row group in wave order; afterwards
// the group's first wave holds the sums.  s: room for half of the waves.
template <int N>
__device__ __forceinline__ void sum_waves(f32x4 (&acc)[N], f32x4 (*s)[N][64], int wv, int kw) {
  const int lane = threadIdx.x & 63, z = wv % kw, grp = wv / kw;
  for (int half = kw / 2; half >= 1; half /= 2) {
    if (z >= half && z < 2 * half) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[grp * (kw / 2) + z - half][i][lane] = acc[i];
    }
    __syncthreads();
    if (z < half) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += s[grp * (kw / 2) + z][i][lane];
    }
    __syncthreads();
  }
}
}  // namespace

// h[p] = silu(Wg_e x) * (Wu_e x) for every pair p of expert e, as a bf16 pair
// hi + lo (16 bits of fraction), so that the down product's operand is not
// rounded to 8 bits before Y's one rounding.  Row group: RB / 2 tiles of the
// gate half and the same of the up half.  NT column tiles of 16 pairs at a time.
template <int RB, int NT, int NW, int kDepth>
__global__ __launch_bounds__(64 * NW, NT == 1 ? (kDepth == 1 ? 4 : 3) : 2) void k_moe_gate_up(MoeArgs a) {
  __shared__ PairList<NW> s;
  __shared__ f32x4 s_acc[NW / 2][RB * NT][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = a.kw;
  int slot, range, col;
  if (!place(a, slot, range, col)) return;
  const uint16_t* list;
  int nc;
  const int e = find_pairs(s, a, slot, list, nc);
  if (e < 0) return;
  const int n = lane & 15;
  constexpr int kHalf = RB / 2;
  const uint32_t nb = static_cast<uint32_t>(a.H / 64);
  const ExpertRows w(a.gate_up, static_cast<int64_t>(e) * 2 * a.I, 2 * static_cast<uint32_t>(a.I), nb);
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.X, static_cast<uint32_t>(a.T) * a.H * 2);
  const int tiles = a.I / 16;
  const int tile0 = (range * (NW / kw) + wv / kw) * kHalf;  // the group's first tile (may lie past the last)
  uint32_t trow[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int t = tile0 + r % kHalf;
    trow[r] = ((r >= kHalf ? a.I : 0) + 16 * (t < tiles ? t : tiles - 1) + n) * nb;
  }
  const int z = wv % kw, b0 = tile0 < tiles ? static_cast<int>(nb * z / kw) : 0;
  const int b1 = tile0 < tiles ? static_cast<int>(nb * (z + 1) / kw) : 0;

  for (int c0 = 16 * NT * col; c0 < nc; c0 += 16 * NT * a.cols) {
    f32x4 acc[RB][NT];
    uint32_t colf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + 16 * t + n;
      colf[t] = c < nc ? static_cast<uint32_t>(list[c] / a.k) * a.H * 2 : kPastEnd;
#pragma unroll
      for (int r = 0; r < RB; ++r) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    panel<RB, NT, false, kDepth>(acc, w, trow, rx, colf, 0, b0, b1);
    sum_waves<RB * NT>(reinterpret_cast<f32x4(&)[RB * NT]>(acc), s_acc, wv, kw);
    if (z != 0) continue;
#pragma unroll
    for (int r = 0; r < kHalf; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = c0 + 16 * t + n;
        if (tile0 + r >= tiles || c >= nc) continue;
        float hv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float gv = acc[r][t][q];
          hv[q] = gv / (1.0f + __expf(-gv)) * acc[r + kHalf][t][q];
        }
        uint32_t h0, h1, l0, l1;
        split_bf16x2(hv[0], hv[1], h0, l0);
        split_bf16x2(hv[2], hv[3], h1, l1);
        uint16_t* dst = a.h + static_cast<int64_t>(list[c]) * 2 * a.I + 16 * (tile0 + r) + 4 * (lane >> 4);
        *reinterpret_cast<u32x2*>(dst) = u32x2{h0, h1};
        *reinterpret_cast<u32x2*>(dst + a.I) = u32x2{l0, l1};
      }
  }
}

// part[p] = Wd_e h[p] in fp32 for every pair p of expert e.  Row group: RB
// tiles.  (Adding the experts inside the kernel, by the last workgroup of a
// row range to arrive, cost a release fence per workgroup: 156 us against 11 at
// one token.)
template <int RB, int NT, int NW, int kDepth>
__global__ __launch_bounds__(64 * NW, 2) void k_moe_down(MoeArgs a) {
  __shared__ PairList<NW> s;
  __shared__ f32x4 s_acc[NW / 2][RB * NT][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = a.kw;
  int slot, range, col;
  if (!place(a, slot, range, col)) return;
  const uint16_t* list;
  int nc;
  const int e = find_pairs(s, a, slot, list, nc);
  if (e < 0) return;
  const int n = lane & 15, tiles = a.H / 16;
  const uint32_t nb = static_cast<uint32_t>(a.I / 64);
  const ExpertRows w(a.down, static_cast<int64_t>(e) * a.H, static_cast<uint32_t>(a.H), nb);
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.h, static_cast<uint32_t>(a.T) * a.k * a.I * 4);
  const int tile0 = (range * (NW / kw) + wv / kw) * RB;
  uint32_t trow[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) trow[r] = (16 * (tile0 + r < tiles ? tile0 + r : tiles - 1) + n) * nb;
  const int z = wv % kw, b0 = tile0 < tiles ? static_cast<int>(nb * z / kw) : 0;
  const int b1 = tile0 < tiles ? static_cast<int>(nb * (z + 1) / kw) : 0;
  for (int c0 = 16 * NT * col; c0 < nc; c0 += 16 * NT * a.cols) {
    f32x4 acc[RB][NT];
    uint32_t colf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + 16 * t + n;
      colf[t] = c < nc ? static_cast<uint32_t>(list[c]) * a.I * 4 : kPastEnd;
#pragma unroll
      for (int r = 0; r < RB; ++r) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    panel<RB, NT, true, kDepth>(acc, w, trow, rx, colf, a.I * 2, b0, b1);
    sum_waves<RB * NT>(reinterpret_cast<f32x4(&)[RB * NT]>(acc), s_acc, wv, kw);
    if (z != 0) continue;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = c0 + 16 * t + n;
        if (tile0 + r < tiles && c < nc)
          *reinterpret_cast<f32x4*>(a.part + static_cast<int64_t>(list[c]) * a.H + 16 * (tile0 + r) +
                                    4 * (lane >> 4)) = acc[r][t];
      }
  }
}

// Y_t = sum_j w_tj part[t k + j], the choices added in order; a thread takes
// four columns of one token.
__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs a) {
  const int v = blockIdx.x * 256 + threadIdx.x, quads = a.H / 4;
  if (v >= a.T * quads) return;
  const int t = v / quads, r = v % quads * 4;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  const float* src = a.part + static_cast<int64_t>(t) * a.k * a.H + r;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    // eight choices' loads in flight; a place that is no choice was not
    // written and does not count, whatever it holds
    f32x4 d[8];
    float w[8];
    bool on[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = j0 + i < a.k ? j0 + i : a.k - 1;
      d[i] = *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(j) * a.H);
      w[i] = a.weights[t * a.k + j];
      const int e = a.ids[t * a.k + j];
      on[i] = j0 + i < a.k && e >= 0 && e < a.E;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = on[i] ? __builtin_fmaf(w[i], d[i][q], y[q]) : y[q];
  }
  *reinterpret_cast<u32x2*>(a.Y + static_cast<int64_t>(t) * a.H + r) =
      u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

// The down product of at most 64 pairs in one launch: a workgroup owns one
// 16-row tile of Y's columns for every token; its waves take (expert, range of
// I) units in turn, leave each pair's 16 sums in LDS, and the workgroup adds
// them per token in the order of the choices.
__global__ __launch_bounds__(64 * kFewWaves) void k_moe_down_few(MoeArgs a) {
  constexpr int kMost = 64;
  __shared__ int s_ids[kMost];
  __shared__ int s_lead[kMost];
  __shared__ uint16_t s_list[kFewWaves][kMost];
  __shared__ f32x4 s_sum[kFewWaves][kMost][4];  // [range][pair]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int P = a.T * a.k;
  // every wave finds the experts met, in the order of their first pairs
  int id = lane < P ? a.ids[lane] : -1;
  if (id < 0 || id >= a.E) id = -1;
  bool first = id >= 0;
  for (int j = 0; j + 1 < P; ++j)
    if (lane > j && __builtin_amdgcn_readlane(id, j) == id) first = false;
  const uint64_t lm = __ballot(first);
  const int leads = __popcll(lm);
  if (wv == 0) {
    s_ids[lane] = id;
    if (first) s_lead[__popcll(lm & lanes_below())] = id;
  }
  __syncthreads();
  const uint32_t nb = static_cast<uint32_t>(a.I / 64);
  // ranges of I per expert: more than one where there are fewer experts than waves
  int ks = leads > 0 ? kFewWaves / leads : 1;
  ks = ks > static_cast<int>(nb) ? static_cast<int>(nb) : ks;
  ks = ks < 1 ? 1 : ks;
  const int n = lane & 15;
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.h, static_cast<uint32_t>(P) * a.I * 4);
  const uint32_t trow[1] = {(16 * blockIdx.x + n) * nb};
  for (int u = wv; u < leads * ks; u += kFewWaves) {
    const int e = __builtin_amdgcn_readfirstlane(s_lead[u / ks]), z = u % ks;
    const uint64_t hit = __ballot(id == e);
    const int nc = __popcll(hit);
    if (id == e) s_list[wv][__popcll(hit & lanes_below())] = static_cast<uint16_t>(lane);
    wave_lds_sync();
    const ExpertRows w(a.down, static_cast<int64_t>(e) * a.H, static_cast<uint32_t>(a.H), nb);
    for (int c0 = 0; c0 < nc; c0 += 16) {
      const int p = c0 + n < nc ? s_list[wv][c0 + n] : -1;
      const uint32_t colf[1] = {p >= 0 ? static_cast<uint32_t>(p) * a.I * 4 : kPastEnd};
      f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
      panel<1, 1, true, 1>(acc, w, trow, rx, colf, a.I * 2, static_cast<int>(nb * z / ks),
                        static_cast<int>(nb * (z + 1) / ks));
      if (p >= 0) s_sum[z][p][lane >> 4] = acc[0][0];
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int v = tid; v < a.T * 4; v += 64 * kFewWaves) {
    const int t = v >> 2, q = v & 3;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.k; ++j) {
      const int p = t * a.k + j;
      if (s_ids[p] < 0) continue;
      f32x4 d = s_sum[0][p][q];
      for (int z = 1; z < ks; ++z) d += s_sum[z][p][q];
      const float w = a.weights[p];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(w, d[i], y[i]);
    }
    *reinterpret_cast<u32x2*>(a.Y + static_cast<int64_t>(t) * a.H + 16 * blockIdx.x + 4 * q) =
        u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  }
}

// ------------------------------------------------------------- launchers
namespace {
// lanes per row and logits per lane: one logit each up to 16 experts, then 16
// lanes up to 128, 32 up to 256 and a whole wave above, with up to 16 logits
// each: the k rounds pay for every halving of the lanes, the logits of a lane
// are compared without a shuffle.  At least k lanes, which hold the results.
template <class F>
void route_shape(int E, int k, F&& f) {
  const int need = E > k ? E : k;
  if (need <= 8) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else if (need <= 16) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (need <= 64) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  else if (need <= 128) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  else if (need <= 256) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}
}  // namespace

namespace {
// rows of one launch: below 2^32 lanes
constexpr int64_t kRouteRows = int64_t(1) << 25;
}  // namespace

hipError_t launch_moe_route(const float* logits, int64_t T, int E, int k, bool renorm, int* ids, float* weights,
                            hipStream_t s) {
  for (int64_t t = 0; t < T; t += kRouteRows) {
    const int64_t n = T - t < kRouteRows ? T - t : kRouteRows;
    route_shape(E, k, [&](auto gc, auto pc) {
      constexpr int G = decltype(gc)::value, PER = decltype(pc)::value;
      hipLaunchKernelGGL((k_moe_route<G, PER>), dim3(static_cast<uint32_t>(ceil_div(n * G, 256))), dim3(256), 0, s,
                         logits + t * E, n, E, k, renorm ? 1 : 0, ids + t * k, weights + t * k);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_moe_route_bwd(const float* logits, const int* ids, const float* dw, int64_t T, int E, int k,
                                bool renorm, float* dlogits, hipStream_t s) {
  for (int64_t t = 0; t < T; t += kRouteRows) {
    const int64_t n = T - t < kRouteRows ? T - t : kRouteRows;
    route_shape(E, k, [&](auto gc, auto pc) {
      constexpr int G = decltype(gc)::value, PER = decltype(pc)::value;
      hipLaunchKernelGGL((k_moe_route_bwd<G, PER>), dim3(static_cast<uint32_t>(ceil_div(n * G, 256))), dim3(256), 0, s,
                         logits + t * E, ids + t * k, dw + t * k, n, E, k, renorm ? 1 : 0, dlogits + t * E);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
constexpr int kLeast = 512;

// Row ranges of one expert's `rows` rows, of which a wave takes rows_wave, and
// the waves that split a reduction of nb 64-weight blocks: as many as keep the
// lanes at least 7/8 busy (a chunk is four blocks), and where that leaves fewer
// than `least` workgroups as many more as have a block at all.  (Short row
// groups, 52 tokens x 4 over 60 experts of 512 x 448: one block per wave 46.5 us,
// this way 38.8; 3 x 4 over 8 of 640 x 3776 44.6 and 33.3.)
void moe_ranges(MoeArgs& a, int rows, int rows_wave, int nb, int waves, int least) {
  auto ranges = [&](int kw) { return static_cast<int>(ceil_div(rows, rows_wave * (waves / kw))); };
  a.kw = waves;
  while (a.kw > 1 && a.kw * round_up(ceil_div(nb, a.kw), 4) * 7 > nb * 8) a.kw /= 2;
  while (a.kw < waves && 2 * a.kw <= nb && int64_t(a.slots) * ranges(a.kw) < least) a.kw *= 2;
  a.ranges = ranges(a.kw);
}
}  // namespace

hipError_t launch_moe(MoeArgs a, hipStream_t s) {
  const int P = a.T * a.k;
  a.by_expert = a.E <= P ? 1 : 0;
  a.slots = a.by_expert ? a.E : P;
  // Two column tiles of 16 at a time above ten pairs per expert on average (many
  // experts then have more than 16): 8 experts of 1216 x 6720, nine each 84.7 us
  // with one, 98.9 with two; fourteen 133 and 111.
  const bool two = P > 10 * a.E;
  // Column tiles of an expert, shared by several workgroups where there are few
  // (61 tokens x 4 over 4 experts of 576 x 2304: 76.8 -> 62.6 us).
  const int col_tiles = static_cast<int>(ceil_div(P, 32 * a.E));
  auto grid = [&]() {
    const int64_t wgs = int64_t(a.slots) * a.ranges;
    a.cols = two && wgs < kLeast ? col_tiles : 1;
    return dim3(static_cast<uint32_t>(round_up(wgs, 8) * a.cols));
  };
  // Tall row groups where those fill the chip, else short ones with the reduction
  // split further: the tall ones dequantize as much for fewer reads of the
  // columns.  Gate and up, tall / short: 7 tokens x 8 over 60 experts of 3392 x
  // 448 (784 units of 32 rows) 72.7 / 61.5 us the layer; with two column tiles 40
  // x 7 over 16 of 512 x 1664 (832) 32.3 / 66.6.
  const bool few_up = int64_t(a.slots) * a.I / 32 < (two ? 512 : 1024);
  if (few_up) moe_ranges(a, a.I, 16, a.H / 64, kFewWaves, kLeast);
  else moe_ranges(a, a.I, 16 * kUpTiles / 2, a.H / 64, kUpWaves, 0);
  const dim3 up = grid(), block_up(64 * (few_up ? kFewWaves : kUpWaves));
  if (few_up && !two) hipLaunchKernelGGL((k_moe_gate_up<2, 1, kFewWaves, 2>), up, block_up, 0, s, a);
  else if (few_up) hipLaunchKernelGGL((k_moe_gate_up<2, 2, kFewWaves, 2>), up, block_up, 0, s, a);
  else if (!two) hipLaunchKernelGGL((k_moe_gate_up<kUpTiles, 1, kUpWaves, kUpDepth>), up, block_up, 0, s, a);
  else hipLaunchKernelGGL((k_moe_gate_up<kUpTiles, 2, kUpWaves, 2>), up, block_up, 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // One launch where the few workgroups of 16 rows have little to do each: 7 pairs
  // of 2496 x 576 22.2 us the layer against 33.2 with two; 42 pairs of 640 x 5504
  // the other way 344 against 111.
  if (P <= 64 && int64_t(P) * a.I <= 16384) {
    hipLaunchKernelGGL(k_moe_down_few, dim3(static_cast<uint32_t>(a.H / 16)), dim3(64 * kFewWaves), 0, s, a);
    return hipGetLastError();
  }
  moe_ranges(a, a.H, 16 * (two ? 4 : kDownTiles), a.I / 64, kDownWaves, 0);
  // as above: short groups below 256 workgroups (15 tokens x 2 over 60 of 704 x
  // 4480, 240 of them, 179 -> 77 us the layer; 5 x 5 over 32 of 1984 x 5440, 400,
  // 96.6 tall, 113.5 short)
  const bool few_down = int64_t(a.slots) * a.ranges < 256;
  if (few_down) moe_ranges(a, a.H, 32, a.I / 64, kDownWaves, kLeast);
  const dim3 down = grid(), block_down(64 * kDownWaves);
  if (few_down && !two) hipLaunchKernelGGL((k_moe_down<2, 1, kDownWaves, kDownDepth>), down, block_down, 0, s, a);
  else if (few_down) hipLaunchKernelGGL((k_moe_down<2, 2, kDownWaves, kDownDepth>), down, block_down, 0, s, a);
  else if (!two) hipLaunchKernelGGL((k_moe_down<kDownTiles, 1, kDownWaves, kDownDepth>), down, block_down, 0, s, a);
  else hipLaunchKernelGGL((k_moe_down<4, 2, kDownWaves, kDownDepth>), down, block_down, 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_sum, dim3(static_cast<uint32_t>(ceil_div(int64_t(a.T) * a.H / 4, 256))), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
