// k_norm.hip -- root-mean-square norm of bf16 rows with the residual's addition
// in front and 8-bit rows behind (k_norm_fwd), and its gradient (k_norm_bwd,
// k_norm_dw).  With h = bf16(x + res), rstd = 1 / sqrt(mean h^2 + eps):
//   y  = bf16(h rstd w), and y's codes as the 8-bit layer forms them
//   dh = bf16(dres + rstd (g - n mean(g n))),  g = w dy, n = h rstd
//   dw = sum over the rows of dy n
// Both are one pass over their rows and bound by HBM: a row stays in the
// registers of the L lanes that share it (C chunks of eight columns each), so
// nothing is read twice.  8192 rows of 8192 with residual, sum, y and codes: 604 MB
// in 104 to 106 us, 5.7 TB/s; the gradient of 8192 rows of 4096 with dres and dw: 268 MB in
// 45 us, 6.0 TB/s, and 4.9 us of k_norm_dw (a 2 GiB copy reaches 4.8 TB/s, HBM's peak is 8).
#include <type_traits>

#include "common.hpp"
#include "fp8_format.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {

// sum over the L lanes that share a row (L = 16, 64: within a wave; above: the
// workgroup's waves through LDS, two buffers by the parity of the row so that
// one barrier a row is enough)
template <int L, class T>
__device__ __forceinline__ T row_sum(T v, T (*red)[8], int parity) {
  constexpr int kIn = L < 64 ? L : 64;
#pragma unroll
  for (int o = kIn / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) red[parity][threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[parity][0];
#pragma unroll
    for (int i = 1; i < L / 64; ++i) v += red[parity][i];
  }
  return v;
}

// Rows are read once and, in the forward pass, written without being kept in
// front of what the caches hold: 8192 rows of 8192 with residual and codes take
// 8% less time so than with ordinary loads and stores, the gradient of 8192 rows of
// 4096 4% less.  The gradient's own stores are ordinary ones (11% more if not).
__device__ __forceinline__ u32x4 row_load(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
template <class T, class P>
__device__ __forceinline__ void row_store(P* p, const T& v) {
  __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
}

__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = bf16_lo(v[d]);
    f[2 * d + 1] = bf16_hi(v[d]);
  }
}

// f (rh + rl) w.  The remainder's product is held to finite values: with an infinite w it is an
// infinity of either sign or, of a remainder of 0, a NaN, and would make the product's
// infinity one.  (Not w itself, which would take a second set of registers: 8192 x 8192
// without residual 63 us instead of 54.)
__device__ __forceinline__ float scaled(float f, float rh, float rl, float w) {
  constexpr float kMost = 0x1.fffffep127f;
  const float p = f * rh, rest = __builtin_fmaf(f, rl, __builtin_fmaf(f, rh, -p)) * w;
  return __builtin_fmaf(p, w, __builtin_amdgcn_fmed3f(rest, -kMost, kMost));
}

constexpr int norm_threads(int L) { return L < 256 ? 256 : L; }

}  // namespace

template <int L, int C>
__global__ __launch_bounds__(norm_threads(L)) void k_norm_fwd(NormFwd a) {
  constexpr int NT = norm_threads(L), kRows = NT / L;
  __shared__ double red[2][8];
  const int sub = threadIdx.x % L;
  float w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t col = (c * L + sub) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 u = col < a.H ? *reinterpret_cast<const f32x4*>(a.w + col + 4 * i) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) w[c][4 * i + e] = u[e];
    }
  }
  int parity = 0;
  // every thread of a workgroup makes the same number of turns (barriers)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.T; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool live = row < a.T;
    const int64_t at = row * a.H;
    u32x4 v[C], u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t col = (c * L + sub) * 8;
      v[c] = u[c] = u32x4{0u, 0u, 0u, 0u};
      if (live && col < a.H) {
        v[c] = row_load(a.x + at + col);
        if (a.res != nullptr) u[c] = row_load(a.res + at + col);
      }
    }
    // The square sum in 64 bits, which hold the squares of any bf16 values and a sum that is
    // as good as exact: in fp32 a row of finite values from 2^57 on could sum to an infinity, its y
    // to 0, and the sum's own error moved codes.  (8192 x 8192 104.5 us either way.)
    double sum = 0.;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t col = (c * L + sub) * 8;
      float f[8];
      double part = 0.;
      if (a.res != nullptr) {
        float g[8];
        unpack8(v[c], f);
        unpack8(u[c], g);
#pragma unroll
        for (int d = 0; d < 4; ++d) v[c][d] = pack_bf16x2(f[2 * d] + g[2 * d], f[2 * d + 1] + g[2 * d + 1]);
        if (live && col < a.H) row_store(a.h + at + col, v[c]);
      }
      unpack8(v[c], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) part = __builtin_fma(static_cast<double>(f[e]), static_cast<double>(f[e]), part);
      sum += part;
    }
    sum = row_sum<L>(sum, red, parity);
    parity ^= 1;
    // rstd as rh + rl (v_rsq_f64 is within 2^-24, a Newton step squares that), and h rstd w without
    // the products' own roundings: y is rounded to bf16 and on to a code, where a last bit decides
    // over a whole step.
    const double x = __builtin_fma(sum, a.inv_h, static_cast<double>(a.eps)), rough = __builtin_amdgcn_rsq(x);
    const double e = __builtin_fma(-x * rough, rough, 1.);
    const double r = e == e ? __builtin_fma(0.5 * rough, e, rough) : rough;
    const float rstd = static_cast<float>(r), rh = rstd;
    const float rl = rh < __builtin_inff() ? static_cast<float>(r - static_cast<double>(rh)) : 0.f;
    if (live && sub == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    uint32_t bytes = 0;  // L = 16: the row's only group of four blocks
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t col = (c * L + sub) * 8;
      float f[8];
      unpack8(v[c], f);
      u32x4 y;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        y[d] = pack_bf16x2(scaled(f[2 * d], rh, rl, w[c][2 * d]), scaled(f[2 * d + 1], rh, rl, w[c][2 * d + 1]));
      // (columns past H: 0 rstd w is NaN where rstd is not finite)
      if (col >= a.H) y = u32x4{0u, 0u, 0u, 0u};
      if (a.y != nullptr && live && col < a.H) row_store(a.y + at + col, y);
      if (a.codes == nullptr) continue;
      uint32_t m = 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) m = max(m, max((y[d] << 16) & 0x7fffffffu, y[d] & 0x7fff0000u));
      m = max16_u32(m);
      const uint32_t b = f8_scale_byte(m);
      const float inv = f8_inv_scale(b);
      u32x2 o;
#pragma unroll
      for (int d = 0; d < 2; ++d)
        o[d] = f8_pack4(bf16_lo(y[2 * d]) * inv, bf16_hi(y[2 * d]) * inv, bf16_lo(y[2 * d + 1]) * inv,
                        bf16_hi(y[2 * d + 1]) * inv);
      if (live && col < a.Kp) row_store(a.codes + row * a.Kp + col, o);
      if constexpr (L == 16) {
        bytes |= b << (8 * c);
      } else {
        // a wave's 512 columns are one group of four blocks
        const uint32_t b0 = __builtin_amdgcn_readlane(b, 0), b1 = __builtin_amdgcn_readlane(b, 16);
        const uint32_t b2 = __builtin_amdgcn_readlane(b, 32), b3 = __builtin_amdgcn_readlane(b, 48);
        if (live && (threadIdx.x & 63) == 0 && col < a.H)
          *reinterpret_cast<uint32_t*>(a.scales + (static_cast<int64_t>(col / 512) * a.pitch + row) * 4) =
              b0 | b1 << 8 | b2 << 16 | b3 << 24;
      }
    }
    if constexpr (L == 16) {
      if (a.codes != nullptr && live && sub == 0) *reinterpret_cast<uint32_t*>(a.scales + row * 4) = bytes;
    }
  }
}

template <int L, int C>
__global__ __launch_bounds__(norm_threads(L)) void k_norm_bwd(NormBwd a) {
  constexpr int NT = norm_threads(L), kRows = NT / L;
  __shared__ float red[2][8];
  const int sub = threadIdx.x % L;
  float w[C][8], acc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t col = (c * L + sub) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 u = col < a.H ? *reinterpret_cast<const f32x4*>(a.w + col + 4 * i) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[c][4 * i + e] = u[e];
        acc[c][4 * i + e] = 0.f;
      }
    }
  }
  int parity = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.T; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool live = row < a.T;
    const int64_t at = row * a.H;
    u32x4 hv[C], gv[C], rv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t col = (c * L + sub) * 8;
      hv[c] = gv[c] = rv[c] = u32x4{0u, 0u, 0u, 0u};
      if (live && col < a.H) {
        hv[c] = row_load(a.h + at + col);
        gv[c] = row_load(a.dy + at + col);
        if (a.dres != nullptr) rv[c] = row_load(a.dres + at + col);
      }
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float h[8], d[8];
      unpack8(hv[c], h);
      unpack8(gv[c], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[e] * rstd;
        sum += d[e] * w[c][e] * n;
      }
    }
    sum = row_sum<L>(sum, red, parity);
    parity ^= 1;
    const float mean = sum / static_cast<float>(a.H);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t col = (c * L + sub) * 8;
      float h[8], d[8], r[8], o[8];
      unpack8(hv[c], h);
      unpack8(gv[c], d);
      unpack8(rv[c], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[e] * rstd;
        acc[c][e] += d[e] * n;
        o[e] = r[e] + rstd * (d[e] * w[c][e] - n * mean);
      }
      if (live && col < a.H)
        *reinterpret_cast<u32x4*>(a.dh + at + col) = u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                                           pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
    }
  }
  if (a.part == nullptr) return;
  // this row group's sum of dy n, [row groups][H]
  float* dst = a.part + (static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / L) * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t col = (c * L + sub) * 8;
    if (col < a.H) {
      *reinterpret_cast<f32x4*>(dst + col) = f32x4{acc[c][0], acc[c][1], acc[c][2], acc[c][3]};
      *reinterpret_cast<f32x4*>(dst + col + 4) = f32x4{acc[c][4], acc[c][5], acc[c][6], acc[c][7]};
    }
  }
}

// dw[col] = the P partial rows added in a fixed order: wave k of 16 adds rows
// k, k + 16, ..., one column a lane, then the 16 sums in order.  H % 64 == 0.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* part, int P, uint32_t H, float* dw) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const float* src = part + blockIdx.x * 64 + lane;
  float acc = 0.f;
  for (int p = wv; p < P; p += 16 * 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p + 16 * u < P ? src[static_cast<int64_t>(p + 16 * u) * H] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) acc += v[u];
  }
  s[wv][lane] = acc;
  __syncthreads();
  if (wv == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][lane];
    dw[blockIdx.x * 64 + lane] = t;
  }
}

namespace {

// Lanes that share a row and chunks of eight columns a lane, by the row's
// length: the fewest lanes that hold the row in at most four chunks.
struct NormShape { int L, C; };
constexpr NormShape norm_shape(int64_t H) {
  if (H <= 128) return {16, 1};
  if (H <= 256) return {16, 2};
  if (H <= 512) return {16, 4};
  if (H <= 1024) return {64, 2};
  if (H <= 2048) return {64, 4};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return {256, 4};
  return {512, 4};
}

template <class F>
hipError_t with_shape(int64_t H, F f) {
  const NormShape s = norm_shape(H);
  if (s.L == 16 && s.C == 1) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (s.L == 16 && s.C == 2) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  if (s.L == 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  if (s.L == 64 && s.C == 2) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (s.L == 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  if (s.L == 256 && s.C == 2) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (s.L == 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}

// Workgroups of 256 threads.  Forward: one turn each up to 16384 of them (8192 x
// 8192: 2% less time than with eight workgroups a CU that go round).  Gradient: each
// leaves H floats for dw, so two a CU (8192 x 4096: 384 of them take 3% more, 640
// 8%).
constexpr int64_t kNormFwdWgs = 16384;
constexpr int64_t kNormBwdWgs = 512;

int64_t norm_groups(int64_t T, int64_t H, int64_t wgs) {
  const int L = norm_shape(H).L, rows = norm_threads(L) / L;
  const int64_t most = L > 256 ? wgs * 256 / L : wgs, need = ceil_div(T, rows);
  return need < most ? need : most;
}

}  // namespace

int64_t norm_bwd_parts(int64_t T, int64_t H) {
  const int L = norm_shape(H).L;
  return norm_groups(T, H, kNormBwdWgs) * (norm_threads(L) / L);
}

hipError_t launch_norm_fwd(const NormFwd& a, hipStream_t s) {
  return with_shape(a.H, [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, C = decltype(c)::value;
    hipLaunchKernelGGL((k_norm_fwd<L, C>), dim3(static_cast<uint32_t>(norm_groups(a.T, a.H, kNormFwdWgs))),
                       dim3(norm_threads(L)), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_bwd(const NormBwd& a, float* dw, hipStream_t s) {
  const int64_t wgs = norm_groups(a.T, a.H, a.part != nullptr ? kNormBwdWgs : kNormFwdWgs);
  const hipError_t e = with_shape(a.H, [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, C = decltype(c)::value;
    hipLaunchKernelGGL((k_norm_bwd<L, C>), dim3(static_cast<uint32_t>(wgs)), dim3(norm_threads(L)), 0, s, a);
    return hipGetLastError();
  });
  if (e != hipSuccess || a.part == nullptr) return e;
  hipLaunchKernelGGL(k_norm_dw, dim3(a.H / 64), dim3(1024), 0, s, static_cast<const float*>(a.part),
                     static_cast<int>(norm_bwd_parts(a.T, a.H)), a.H, dw);
  return hipGetLastError();
}

}  // namespace qlora
