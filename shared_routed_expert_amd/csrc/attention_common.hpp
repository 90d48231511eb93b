// What the kernels that read the paged cache share: register types, wave-uniform values, the score cap, e4m3 conversions
// and the split of a line of work into equal parts.
#pragma once
#include "attention.hpp"
#include "common.hpp"

namespace srmoe {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ long uni(long v) {
  const uint32_t lo = (uint32_t)uni((int)(uint32_t)v), hi = (uint32_t)uni((int)(uint32_t)((uint64_t)v >> 32));
  return (long)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ long read_lane(long v, int at) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, at);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), at);
  return (long)(((uint64_t)hi << 32) | lo);
}

// cap tanh(y) in units of log2 e, from x = 2 y log2 e; cap2 = cap log2 e, half_cap = cap / 2 (so half_cap x = cap2 y).
// The quotient cap2 (1 - 2 / (2^x + 1)) is off by some 4 2^-24 of the CAP however small the value is: 2^-16 for caps up
// to 64, about what the products that form the score may be off by, but 0.13 for a cap of 1e6.
// kNear (caps above 64, an instance of their own): |x| < 3/4 (|y| < 0.26) takes the odd polynomial y (1 + x^2 (..)) instead, the least squares
// fit of tanh(y) / y - 1 over that range (off by 0.07 2^-24 of the value): within 14 2^-24 of the VALUE at any cap.
// 16384 tokens, bf16: 1019 us with a cap of 30 and 1211 with one of 100 (no cap: 816); 64 sequences of up to 8192, one
// token each, 36 and 39; trees of 64 tokens 27.7 and 32.4. One instance for both: D = 256 spills, 328 -> 352.
template <bool kNear>
__device__ __forceinline__ float capped(float x, float half_cap, float cap2) {
  const float far = cap2 - 2.f * cap2 * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x) + 1.f);
  if (!kNear) return far;
  const float w = x * half_cap, x2 = x * x;
  const float p = __builtin_fmaf(__builtin_fmaf(-8.87633034e-05f, x2, 1.92208393e-03f), x2, -4.00376075e-02f) * x2;
  return __builtin_fabsf(x) < 0.75f ? __builtin_fmaf(w, p, w) : far;
}
constexpr float kNearCap = 64.f;   // caps above it
enum Cap { kCapNone, kCapSmall, kCapLarge };

// 8 e4m3 codes -> bf16 / float16 (both exact)
__device__ __forceinline__ bf16x8 bf16_of_e4m3(int a, int b) {
  const bf16x2_t p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2_t q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2_t s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}
__device__ __forceinline__ f16x8 f16_of_e4m3(int a, int b) {
  const f16x2 p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const f16x2 q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const f16x2 r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const f16x2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return f16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}

// a / b for a >= 0, b > 0: in 32 bits where they fit (a 64-bit division costs over a hundred instructions)
__device__ __forceinline__ long div_pos(long a, long b) {
  if (((uint64_t)(a | b) >> 32) == 0) return (long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Part w of `parts` covers [begin(w), begin(w + 1)) of `total` units.
struct Parts {
  long q, rem;
  __device__ __forceinline__ Parts(long total, int parts) : q(div_pos(total, parts)), rem(total - q * parts) {}
  __device__ __forceinline__ long begin(int w) const { return q * w + min((long)w, rem); }
  __device__ __forceinline__ int of(long unit) const {   // the part that holds a unit
    const long big = (q + 1) * rem;
    return (int)(unit < big ? div_pos(unit, q + 1) : rem + div_pos(unit - big, q));
  }
};

}  // namespace srmoe
