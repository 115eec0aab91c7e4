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
// 0x007fffff).
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
// where e was not chosen).  Ids outside [0, E) count as no choice.
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
    top = fmaxf(top, x[e]);
  }
  top = max_group<G>(top);
  float total = 0.f, dot = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    x[e] = top == kNegInf ? 0.f : (sub + G * e < E ? expf(x[e] - top) : 0.f);
    total += x[e];
    dot += x[e] * g[e];
  }
  total = sum_group<G>(total);
  dot = sum_group<G>(dot);
  const float inv = top == kNegInf ? 0.f : 1.0f / total;
  dot *= inv;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    if (live && sub + G * e < E) dl[row * E + sub + G * e] = x[e] * inv * (g[e] - dot);
}

// ------------------------------------------------------------- experts
namespace {
constexpr int kPairs = kMoeMaxPairs;

// One lane's 64-weight block: 32 code bytes, absmax code, group scale.
struct Blk {
  u32x4 c0, c1;
  uint32_t q;
  float sc;
};

// An expert's rows: pointers to its first code byte and absmax code, the
// group scales from its first block's group on, and that block's place in it.
struct Rows {
  const uint8_t* codes;
  const uint8_t* q;
  const float* scale;
  uint32_t rem;
  __device__ __forceinline__ Rows(const MoeWeight& w, int64_t row, int64_t nb) {
    const int64_t b = row * nb;
    codes = w.codes + b * 32;
    q = w.absmax_q + b;
    scale = w.scale + (b >> 8);
    rem = static_cast<uint32_t>(b & 255);
  }
  // block b (counted from the expert's first row)
  __device__ __forceinline__ void load(Blk& o, uint32_t b, bool live) const {
    o.c0 = o.c1 = u32x4{0u, 0u, 0u, 0u};
    o.q = 0;
    o.sc = 0.f;
    if (live) {
      const u32x4* p = reinterpret_cast<const u32x4*>(codes + static_cast<uint64_t>(b) * 32);
      o.c0 = __builtin_nontemporal_load(p);
      o.c1 = __builtin_nontemporal_load(p + 1);
      o.q = q[b];
      o.sc = scale[(rem + b) >> 8];
    }
  }
};

__device__ __forceinline__ bf16x8 as_frag(const uint32_t (&w)[4]) {
  return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}

// the ids of all pairs into LDS (every thread of the workgroup; a barrier follows in the caller)
__device__ __forceinline__ void stage_ids(int* s_ids, const int* __restrict__ ids, int P, int E, int nthreads) {
  for (int i = threadIdx.x; i < P; i += nthreads) {
    const int e = ids[i];
    s_ids[i] = e >= 0 && e < E ? e : -1;  // -1: no expert
  }
}
// the pairs of expert e in ascending order into list (one wave); their count
__device__ __forceinline__ int list_pairs(const int* s_ids, int P, int e, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int b = 0; b < P; b += 64) {
    const bool hit = b + lane < P && s_ids[b + lane] == e;
    const uint64_t m = __ballot(hit);
    if (hit) list[n + __popcll(m & ((uint64_t(1) << lane) - 1))] = static_cast<uint16_t>(b + lane);
    n += __popcll(m);
  }
  return n;
}
}  // namespace

// h[p] = silu(Wg_e x) * (Wu_e x) for every pair p = (token, choice) of expert
// e.  Workgroup (rb, slot): rows [16 rb, 16 rb + 16) of expert e's gate and up
// halves.  A slot is an expert where there are no more experts than pairs,
// else a pair, whose workgroup works only if it is its expert's first pair:
// either way each expert's weights are read once.  The four waves split the
// 64-weight blocks of the rows; lane (n = l % 16, g = l / 16) dequantizes block
// 4 c + g of row n in registers (MFMA A operand) against token columns (B
// operand: pair n's activations at the same k).
__global__ __launch_bounds__(256) void k_moe_gate_up(MoeArgs a) {
  __shared__ int s_ids[kPairs];
  __shared__ uint16_t s_list[kPairs];
  __shared__ int s_n;
  __shared__ f32x4 s_acc[4][2][4][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int P = a.T * a.k;
  const int blocks = a.I / 16;
  const int rb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
  stage_ids(s_ids, a.ids, P, a.E, 256);
  __syncthreads();
  const int e = a.by_expert ? slot : s_ids[slot];
  if (e < 0) return;
  if (wv == 0) {
    const int n = list_pairs(s_ids, P, e, s_list);
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int nc = s_n;
  if (nc == 0 || (!a.by_expert && s_list[0] != slot)) return;

  const int n = lane & 15, g = lane >> 4;
  const int64_t nb64 = a.H / 64;
  const int nb = static_cast<int>(nb64);
  const Rows wg(a.gate_up, (static_cast<int64_t>(e) * 2) * a.I + 16 * rb, nb64);
  const Rows wu(a.gate_up, (static_cast<int64_t>(e) * 2 + 1) * a.I + 16 * rb, nb64);
  const int b0 = nb * wv / 4, b1 = nb * (wv + 1) / 4;

  auto run = [&](int c0, auto ntc) {
    constexpr int NT = decltype(ntc)::value;  // column tiles of 16 pairs
    f32x4 acc[2][NT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* xp[NT];
    bool on[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + 16 * t + n;
      on[t] = c < nc;
      xp[t] = a.X + static_cast<int64_t>(on[t] ? s_list[c] / a.k : 0) * a.H;
    }
    Blk bg, bu, ng, nu;
    const uint32_t row = static_cast<uint32_t>(n) * nb;
    wg.load(bg, row + b0 + g, b0 + g < b1);
    wu.load(bu, row + b0 + g, b0 + g < b1);
    for (int b = b0; b < b1; b += 4) {
      const bool live = b + g < b1, next = b + 4 + g < b1;
      wg.load(ng, row + b + 4 + g, next);
      wu.load(nu, row + b + 4 + g, next);
      const Nf4Table tg = make_table(dq_absmax(bg.q, bg.sc));
      const Nf4Table tu = make_table(dq_absmax(bu.q, bu.sc));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4 x[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          x[t] = u32x4{0u, 0u, 0u, 0u};
          if (live && on[t]) x[t] = *reinterpret_cast<const u32x4*>(xp[t] + (b + g) * 64 + 8 * j);
        }
        uint32_t w[4];
        lookup8(tg, j < 4 ? bg.c0[j] : bg.c1[j - 4], w);
        const bf16x8 fg = as_frag(w);
        lookup8(tu, j < 4 ? bu.c0[j] : bu.c1[j - 4], w);
        const bf16x8 fu = as_frag(w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8 fx = __builtin_bit_cast(bf16x8, x[t]);
          acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fg, fx, acc[0][t], 0, 0, 0);
          acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fu, fx, acc[1][t], 0, 0, 0);
        }
      }
      bg = ng;
      bu = nu;
    }
    // the waves' partial sums meet in LDS, added in wave order; h as a bf16
    // pair hi + lo (16 bits of fraction), so the down product's operand is not
    // rounded to 8 bits a second time before Y's one rounding
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) s_acc[wv][i][t][lane] = acc[i][t];
    __syncthreads();
    for (int v = tid; v < 64 * NT; v += 256) {
      const int t = v >> 6, l = v & 63;
      const int c = c0 + 16 * t + (l & 15);
      if (c >= nc) continue;
      f32x4 gs = s_acc[0][0][t][l], us = s_acc[0][1][t][l];
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        gs += s_acc[w][0][t][l];
        us += s_acc[w][1][t][l];
      }
      float hv[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) hv[q] = gs[q] / (1.0f + __expf(-gs[q])) * us[q];
      const uint32_t h0 = pack_bf16x2(hv[0], hv[1]), h1 = pack_bf16x2(hv[2], hv[3]);
      const uint32_t l0 = pack_bf16x2(hv[0] - bf16_lo(h0), hv[1] - bf16_hi(h0));
      const uint32_t l1 = pack_bf16x2(hv[2] - bf16_lo(h1), hv[3] - bf16_hi(h1));
      uint16_t* dst = a.h + static_cast<int64_t>(s_list[c]) * 2 * a.I + 16 * rb + 4 * (l >> 4);
      *reinterpret_cast<u32x2*>(dst) = u32x2{h0, h1};
      *reinterpret_cast<u32x2*>(dst + a.I) = u32x2{l0, l1};
    }
  };
  if (nc <= 16) run(0, std::integral_constant<int, 1>{});
  else if (nc <= 32) run(0, std::integral_constant<int, 2>{});
  else
    for (int c = 0; c < nc; c += 64) run(c, std::integral_constant<int, 4>{});
}

// Y_t = sum_j w_tj Wd_e h_tj.  Workgroup b owns rows [16 b, 16 b + 16) of Y's
// columns for every token: its waves take (expert, range of I) units in
// turn, each leaving its pairs' 16 sums in LDS, and the workgroup then adds
// them per token in the order of the choices: no partial sums cross
// workgroups and the order of additions is fixed.
constexpr int kDownWaves = 8;
constexpr int kDownSums = 1024;  // (range, pair) sums of 16 rows held in LDS: 64 KiB
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeArgs a) {
  __shared__ int s_ids[kPairs];
  __shared__ int s_first[kMoeMaxExperts];
  __shared__ uint16_t s_lead[kPairs];
  __shared__ int s_leads;
  __shared__ uint16_t s_list[kDownWaves][kPairs];
  __shared__ float s_sum[kDownSums][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int P = a.T * a.k;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 16;
  stage_ids(s_ids, a.ids, P, a.E, 64 * kDownWaves);
  for (int i = tid; i < a.E; i += 64 * kDownWaves) s_first[i] = P;
  __syncthreads();
  for (int p = tid; p < P; p += 64 * kDownWaves)
    if (s_ids[p] >= 0) atomicMin(&s_first[s_ids[p]], p);
  __syncthreads();
  // the experts met, by their first pair
  if (wv == 0) {
    int m = 0;
    for (int b = 0; b < P; b += 64) {
      const int p = b + lane;
      const bool hit = p < P && s_ids[p] >= 0 && s_first[s_ids[p]] == p;
      const uint64_t mask = __ballot(hit);
      if (hit) s_lead[m + __popcll(mask & ((uint64_t(1) << lane) - 1))] = static_cast<uint16_t>(s_ids[p]);
      m += __popcll(mask);
    }
    if (lane == 0) s_leads = m;
  }
  __syncthreads();
  const int leads = s_leads;
  const int nb = a.I / 64;
  // ranges of I per expert: more than one where there are fewer experts than waves
  int ks = leads > 0 ? kDownWaves / leads : 1;
  ks = ks > kDownSums / P ? kDownSums / P : ks;
  ks = ks > nb / 4 ? nb / 4 : ks;
  ks = ks < 1 ? 1 : ks;

  const int n = lane & 15, g = lane >> 4;
  for (int u = wv; u < leads * ks; u += kDownWaves) {
    const int e = s_lead[u / ks], z = u % ks;
    uint16_t* list = s_list[wv];
    const int nc = list_pairs(s_ids, P, e, list);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const Rows wd(a.down, static_cast<int64_t>(e) * a.H + r0, nb);
    const int b0 = nb * z / ks, b1 = nb * (z + 1) / ks;
    const uint32_t row = static_cast<uint32_t>(n) * nb;
    auto run = [&](int c0, auto ntc) {
      constexpr int NT = decltype(ntc)::value;
      f32x4 acc[NT];
      const uint16_t* hp[NT];
      bool on[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int c = c0 + 16 * t + n;
        on[t] = c < nc;
        hp[t] = a.h + static_cast<int64_t>(on[t] ? list[c] : 0) * 2 * a.I;
      }
      Blk cur, nxt;
      wd.load(cur, row + b0 + g, b0 + g < b1);
      for (int b = b0; b < b1; b += 4) {
        const bool live = b + g < b1;
        wd.load(nxt, row + b + 4 + g, b + 4 + g < b1);
        const Nf4Table tab = make_table(dq_absmax(cur.q, cur.sc));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t w[4];
          lookup8(tab, j < 4 ? cur.c0[j] : cur.c1[j - 4], w);
          const bf16x8 fw = as_frag(w);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            u32x4 hi = u32x4{0u, 0u, 0u, 0u}, lo = hi;
            if (live && on[t]) {
              hi = *reinterpret_cast<const u32x4*>(hp[t] + (b + g) * 64 + 8 * j);
              lo = *reinterpret_cast<const u32x4*>(hp[t] + a.I + (b + g) * 64 + 8 * j);
            }
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, __builtin_bit_cast(bf16x8, hi), acc[t], 0, 0, 0);
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, __builtin_bit_cast(bf16x8, lo), acc[t], 0, 0, 0);
          }
        }
        cur = nxt;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (on[t])
          *reinterpret_cast<f32x4*>(&s_sum[z * P + list[c0 + 16 * t + n]][4 * g]) = acc[t];
    };
    if (nc <= 16) run(0, std::integral_constant<int, 1>{});
    else if (nc <= 32) run(0, std::integral_constant<int, 2>{});
    else
      for (int c = 0; c < nc; c += 64) run(c, std::integral_constant<int, 4>{});
  }
  __syncthreads();
  // token t, rows r0 + 4 q .. + 3
  for (int v = tid; v < a.T * 4; v += 64 * kDownWaves) {
    const int t = v >> 2, q = v & 3;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.k; ++j) {
      const int p = t * a.k + j;
      if (s_ids[p] < 0) continue;
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      for (int z = 0; z < ks; ++z) s += *reinterpret_cast<const f32x4*>(&s_sum[z * P + p][4 * q]);
      const float w = a.weights[p];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(w, s[i], y[i]);
    }
    *reinterpret_cast<u32x2*>(a.Y + static_cast<int64_t>(t) * a.H + r0 + 4 * q) =
        u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  }
}

// ------------------------------------------------------------- launchers
namespace {
// lanes per row and logits per lane: the fewest lanes (at least k, for the
// results) that hold a row with one logit each, up to a wave of 16 each
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

hipError_t launch_moe_route(const float* logits, int64_t T, int E, int k, bool renorm, int* ids, float* weights,
                            hipStream_t s) {
  route_shape(E, k, [&](auto gc, auto pc) {
    constexpr int G = decltype(gc)::value, PER = decltype(pc)::value;
    hipLaunchKernelGGL((k_moe_route<G, PER>), dim3(static_cast<uint32_t>(ceil_div(T * G, 256))), dim3(256), 0, s,
                       logits, T, E, k, renorm ? 1 : 0, ids, weights);
  });
  return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const float* logits, const int* ids, const float* dw, int64_t T, int E, int k,
                                bool renorm, float* dlogits, hipStream_t s) {
  route_shape(E, k, [&](auto gc, auto pc) {
    constexpr int G = decltype(gc)::value, PER = decltype(pc)::value;
    hipLaunchKernelGGL((k_moe_route_bwd<G, PER>), dim3(static_cast<uint32_t>(ceil_div(T * G, 256))), dim3(256), 0, s,
                       logits, ids, dw, T, E, k, renorm ? 1 : 0, dlogits);
  });
  return hipGetLastError();
}

hipError_t launch_moe(MoeArgs a, hipStream_t s) {
  const int P = a.T * a.k;
  a.by_expert = a.E <= P ? 1 : 0;
  const int64_t slots = a.by_expert ? a.E : P;
  hipLaunchKernelGGL(k_moe_gate_up, dim3(static_cast<uint32_t>(a.I / 16 * slots)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_down, dim3(static_cast<uint32_t>(a.H / 16)), dim3(64 * kDownWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
