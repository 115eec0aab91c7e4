// k_adamw.hip -- one AdamW step over many tensors in one launch, states in 32
// or 8 bits.  With g = s grad and t the step's number:
//   m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2
//   p' = p - lr wd p - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// Every element is read and written once: bound by HBM (30 bytes an element
// with fp32 states, a master copy and its bf16 parameter; 18 with 8-bit states).
// The factors of seven projections in 32 layers, 41.9 million elements: 232 us and
// 140 us in 8 bits, 5.4 TB/s both (a 2 GiB copy reaches 4.8).
//
// The 8-bit states are m and r = sqrt(v) as e4m3 codes with one power-of-two
// scale per 128 elements of a tensor (fp8_format.hpp).  r instead of v halves
// the exponents that a block spans: e4m3's 2^17 between the largest and the
// smallest code are 2^35 in v.  The codes are rounded down after the addition of
// a noise u in (0, 1) steps.  To the nearest code a state would stand still: with
// b2 = 0.999 a decaying r loses 0.05% a step, and half a code step is 3 to 6%.
// With the noise its expectation is the value.  An r that is not 0 keeps at
// least the smallest code: m' / sqrt(v') would blow up where v alone went to 0.
// This step's own update takes m' and v' before they are rounded.
#include "common.hpp"
#include "fp8_format.hpp"
#include "nf4_format.hpp"

namespace qlora {

namespace {

// Every bit of x spread over a word: two rounds of shift and odd factor and a last shift, with
// Austin Appleby's published 32-bit constants (public domain).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x85ebca6bu;
  x ^= x >> 13;
  x *= 0xc2b2ae35u;
  return x ^ (x >> 16);
}

// The code of |y| <= 448 (its fp32 bits), rounded down after u = (byte + 1/2) / 256
// steps: in the normal range the low 20 bits of the fraction are the part of a
// step, below 2^-6 the step is 2^-9.  Both sums are exact.
__device__ __forceinline__ uint32_t code_with_noise(float y, uint32_t byte) {
  const uint32_t u = byte * 4096u + 2048u;
  const uint32_t normal = ((__builtin_bit_cast(uint32_t, y) + u) >> 20) - (120u << 3);
  const uint32_t sub = (static_cast<uint32_t>(y * 0x1p29f) + u) >> 20;
  return y < 0x1p-6f ? sub : normal;
}

// x y, rounded: a plain product may be fused into the sum that takes it
__device__ __forceinline__ float rounded(float x, float y) { return __builtin_fmaf(x, y, 0.f); }

}  // namespace

// One workgroup a chunk, eight elements a lane; 16 lanes hold a block of 128.  The
// chunks come from a table in device memory: one launch for any number of tensors.
// The state sums are formed without fused multiply-adds: each is then the two
// rounded products' rounded sum, as fp32 tensor operations form it, and the codes, whose
// borders hang on the last bit, are the same whichever way a step is computed.  (m' with
// the products' remainders: 19 instead of 50 of 42 million codes are another than 64 bits
// would choose, for 146 us instead of 141.)
template <bool k8>
__global__ __launch_bounds__(256) void k_adamw(AdamStep a) {
  const AdamChunk c = a.table[blockIdx.x];
  const int first = threadIdx.x * 8;
  // lanes of a block that begins behind the tensor have neither state nor
  // elements (16 lanes agree); in the last block the rest counts as 0
  if (first / kAdamBlock * kAdamBlock >= c.n) return;
  const int live = c.n - first < 0 ? 0 : c.n - first > 8 ? 8 : c.n - first;
  const int64_t at = c.state + first;
  const float s = a.grad_scale != nullptr ? *a.grad_scale : 1.f;

  float g[8], p[8], m[8], v[8];
  if (live == 8) {
    const f32x4 g0 = *reinterpret_cast<const f32x4*>(c.g + first), g1 = *reinterpret_cast<const f32x4*>(c.g + first + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g[e] = g0[e];
      g[4 + e] = g1[e];
    }
    if (c.master != nullptr) {
      const f32x4 p0 = *reinterpret_cast<const f32x4*>(c.master + first);
      const f32x4 p1 = *reinterpret_cast<const f32x4*>(c.master + first + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = p0[e];
        p[4 + e] = p1[e];
      }
    } else {
      const u32x4 q = *reinterpret_cast<const u32x4*>(c.p + first);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        p[2 * d] = bf16_lo(q[d]);
        p[2 * d + 1] = bf16_hi(q[d]);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] = e < live ? c.g[first + e] : 0.f;
      p[e] = e >= live ? 0.f
             : c.master != nullptr ? c.master[first + e]
                                   : __builtin_bit_cast(float, static_cast<uint32_t>(c.p[first + e]) << 16);
    }
  }
  u32x2 mq, vq;
  uint32_t mb = 0, vb = 0;
  if constexpr (k8) {
    mq = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.m) + at);
    vq = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.v) + at);
    mb = a.ms[at / kAdamBlock];
    vb = a.vs[at / kAdamBlock];
    const float fm = f8_scale(mb), fv = f8_scale(vb);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const auto m0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mq[d]), false);
      const auto m1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mq[d]), true);
      const auto v0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(vq[d]), false);
      const auto v1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(vq[d]), true);
      const float mm[4] = {m0[0], m0[1], m1[0], m1[1]}, rr[4] = {v0[0], v0[1], v1[0], v1[1]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[4 * d + e] = mm[e] * fm;
        const float r = rr[e] * fv;
        v[4 * d + e] = r * r;
      }
    }
  } else {
    const float *pm = static_cast<const float*>(a.m) + at, *pv = static_cast<const float*>(a.v) + at;
    const f32x4 m0 = *reinterpret_cast<const f32x4*>(pm), m1 = *reinterpret_cast<const f32x4*>(pm + 4);
    const f32x4 v0 = *reinterpret_cast<const f32x4*>(pv), v1 = *reinterpret_cast<const f32x4*>(pv + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = m0[e];
      m[4 + e] = m1[e];
      v[e] = v0[e];
      v[4 + e] = v1[e];
    }
  }

  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float ge = a.grad_scale != nullptr ? rounded(g[e], s) : g[e];
    m[e] = rounded(a.b1, m[e]) + rounded(a.c1, ge);
    v[e] = rounded(a.b2, v[e]) + rounded(a.c2, rounded(ge, ge));
    r[e] = sqrtf(v[e]);
    p[e] = p[e] - a.decay * p[e] - a.rate * (m[e] / (r[e] * a.root + a.eps));
    if (e >= live) m[e] = v[e] = r[e] = 0.f;
  }

  if (live == 8) {
    if (c.master != nullptr) {
      *reinterpret_cast<f32x4*>(c.master + first) = f32x4{p[0], p[1], p[2], p[3]};
      *reinterpret_cast<f32x4*>(c.master + first + 4) = f32x4{p[4], p[5], p[6], p[7]};
    }
    if (c.p != nullptr)
      *reinterpret_cast<u32x4*>(c.p + first) = u32x4{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]),
                                                    pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7])};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < live) {
        if (c.master != nullptr) c.master[first + e] = p[e];
        if (c.p != nullptr) c.p[first + e] = static_cast<uint16_t>(pack_bf16x2(p[e], 0.f) & 0xffffu);
      }
  }
  if constexpr (!k8) {
    float *pm = static_cast<float*>(a.m) + at, *pv = static_cast<float*>(a.v) + at;
    *reinterpret_cast<f32x4*>(pm) = f32x4{m[0], m[1], m[2], m[3]};
    *reinterpret_cast<f32x4*>(pm + 4) = f32x4{m[4], m[5], m[6], m[7]};
    *reinterpret_cast<f32x4*>(pv) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(pv + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    // a value that is not finite has no part in its block's scale and stays NaN alone
    uint32_t am = 0, ar = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t xm = __builtin_bit_cast(uint32_t, m[e]) & 0x7fffffffu, xr = __builtin_bit_cast(uint32_t, r[e]) & 0x7fffffffu;
      am = max(am, xm < 0x7f800000u ? xm : 0u);
      ar = max(ar, xr < 0x7f800000u ? xr : 0u);
    }
    mb = f8_scale_byte(max16_u32(am));
    vb = f8_scale_byte(max16_u32(ar));
    const float im = f8_inv_scale(mb), ir = f8_inv_scale(vb);
    mq = vq = u32x2{0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t h = mix32(static_cast<uint32_t>(at / 2 + e / 2) ^ a.key);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t bits = __builtin_bit_cast(uint32_t, m[e + k]);
        uint32_t cm = code_with_noise(__builtin_fabsf(m[e + k]) * im, h >> (16 * k) & 255u);
        uint32_t cr = code_with_noise(r[e + k] * ir, h >> (16 * k + 8) & 255u);
        if (cr == 0 && r[e + k] != 0.f) cr = 1;
        if ((bits & 0x7fffffffu) >= 0x7f800000u) cm = 0x7fu;
        if ((__builtin_bit_cast(uint32_t, r[e + k]) & 0x7fffffffu) >= 0x7f800000u) cr = 0x7fu;
        cm |= bits >> 31 << 7;
        mq[e / 4] |= cm << (8 * (e % 4 + k));
        vq[e / 4] |= cr << (8 * (e % 4 + k));
      }
    }
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.m) + at) = mq;
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.v) + at) = vq;
    if (threadIdx.x % 16 == 0) {
      a.ms[at / kAdamBlock] = static_cast<uint8_t>(mb);
      a.vs[at / kAdamBlock] = static_cast<uint8_t>(vb);
    }
  }
}

hipError_t launch_adamw(const AdamStep& a, bool bits8, hipStream_t s) {
  AdamStep b = a;
  b.key = mix32(a.key);
  const dim3 grid(static_cast<uint32_t>(a.chunks));
  if (bits8) hipLaunchKernelGGL((k_adamw<true>), grid, dim3(256), 0, s, b);
  else hipLaunchKernelGGL((k_adamw<false>), grid, dim3(256), 0, s, b);
  return hipGetLastError();
}

}  // namespace qlora
