// The residual's addition and the root-mean-square norm in front of the MoE layer, with the result in bf16 (what the
// router reads) and in e4m3 with scales (what the expert GEMMs read, in place of moe_ffn_quant_x's pass over it):
//   h = x + r,  residual_out = bf16(h),  y = h rstd w,  rstd = (mean h^2 + eps)^-1/2,  codes = e4m3(y / s),
//   s = max |y| / 448 over the row or over 128 columns.
// One reduction serves both the norm and the scale: max |y| = rstd max |h w|.
#include "norm.hpp"
#include "common.hpp"

namespace srmoe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 8 bf16 values of a 16-byte word, widened
__device__ __forceinline__ void widen8(const i32x4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float((uint32_t)v[i] << 16);
    f[2 * i + 1] = __uint_as_float((uint32_t)v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ i32x4 narrow8(const float (&f)[8]) {
  return i32x4{(int)pack_bf16x2(f[0], f[1]), (int)pack_bf16x2(f[2], f[3]), (int)pack_bf16x2(f[4], f[5]),
               (int)pack_bf16x2(f[6], f[7])};
}
enum Quant { kQuantNone, kQuantRow, kQuantBlock };

// LANES == 0: one workgroup per row; with W waves, thread t holds values 8 t .. 8 t + 7 of each of the row's STRIPES stripes of
// 512 W. LANES > 0 (H <= 8 LANES): 256 / LANES rows per workgroup, with nothing to exchange between waves. All of a
// row's loads are issued before the first is used, by addresses alone (lanes past the end load the row's first
// values again and drop them): as branches they waited for each other, 16384 tokens of 5120 232 us instead of 132. x and the
// residual are read once, and residual_out is next read a layer later, so they pass the caches by: 122. y and xq are what the
// router and the experts read next (streamed as well: 129, and nothing gained behind them). Bound by its 757 MB: 119 to 138
// us by the card, 5.5 to 6.4 TB/s.
template <int STRIPES, Quant QUANT, int LANES>
__global__ void __launch_bounds__(STRIPES == 1 ? 256 : (STRIPES == 2 ? 512 : 1024)) add_rms_norm_kernel(const NormArgs a) {
  constexpr int kWaves = STRIPES == 1 ? 4 : (STRIPES == 2 ? 8 : 16);   // at most
  constexpr bool kKeepWeight = STRIPES < 8;                            // in registers
  __shared__ float red[2][kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int tid = LANES ? threadIdx.x % LANES : threadIdx.x;           // among the row's threads
  const int t = LANES ? blockIdx.x * (256 / LANES) + threadIdx.x / LANES : blockIdx.x;
  const bool there = !LANES || t < a.T;
  const size_t row = (size_t)(there ? t : a.T - 1) * a.H;
  const uint16_t* const x = a.x + (size_t)(there ? t : a.T - 1) * a.x_stride;
  int at[STRIPES];
  bool in[STRIPES];
  i32x4 xv[STRIPES], rv[STRIPES];
#pragma unroll
  for (int s = 0; s < STRIPES; ++s) {
    at[s] = (s * (LANES ? LANES : blockDim.x) + tid) * 8;
    in[s] = at[s] < a.H;
    at[s] = in[s] ? at[s] : 0;
    xv[s] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(x + at[s]));
  }
  if (a.residual) {
#pragma unroll
    for (int s = 0; s < STRIPES; ++s)
      rv[s] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(a.residual + row + at[s]));
  }
  auto weights = [&](int s, float (&w)[8]) {
    const float4 p = *reinterpret_cast<const float4*>(a.weight + at[s]);
    const float4 q = *reinterpret_cast<const float4*>(a.weight + at[s] + 4);
    w[0] = p.x; w[1] = p.y; w[2] = p.z; w[3] = p.w; w[4] = q.x; w[5] = q.y; w[6] = q.z; w[7] = q.w;
  };
  float w[STRIPES][8];
  if (kKeepWeight) {
#pragma unroll
    for (int s = 0; s < STRIPES; ++s) weights(s, w[s]);
  }
  float h[STRIPES][8];
  float sum = 0.f, most = 0.f;
#pragma unroll
  for (int s = 0; s < STRIPES; ++s) {
    widen8(xv[s], h[s]);
    if (a.residual) {
      float g[8];
      widen8(rv[s], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[s][i] += g[i];
    }
    if (!kKeepWeight && QUANT == kQuantRow) weights(s, w[s]);
    if (in[s]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum = __builtin_fmaf(h[s][i], h[s][i], sum);
        if (QUANT == kQuantRow) most = fmaxf(most, fabsf(h[s][i] * w[s][i]));
      }
    }
  }
#pragma unroll
  for (int d = 1; d < (LANES ? LANES : 64); d <<= 1) {
    sum += __shfl_xor(sum, d, 64);
    if (QUANT == kQuantRow) most = fmaxf(most, __shfl_xor(most, d, 64));
  }
  if (!LANES) {
    if (lane == 0) {
      red[0][wave] = sum;
      red[1][wave] = most;
    }
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < waves; ++i) {
      sum += red[0][i];
      most = fmaxf(most, red[1][i]);
    }
  }
  const float mean = sum / (float)a.H + a.eps;
  float rstd = 1.f / sqrtf(mean);
  const float products = most;
  most *= rstd;
  // Rows whose squares, or whose products with the weights, leave float32's normal range although y need not (the same answer
  // for all of a row's threads; rows of zeros are among them): h by the power of two that brings its largest near 1, and the
  // sums again. A NaN or an infinity in the row stays what it is. Other rows pay a comparison, within the noise: 64 tokens of
  // 5120 5.9 us with and without, 16384 133, 1024 of 65536 120.7 and 120.6.
  const bool far =
      !(mean >= 0x1p-120f && mean < INFINITY) || (QUANT == kQuantRow && !(products >= 0x1p-126f && products < INFINITY));
  if (__builtin_expect(far, 0)) {
    auto over_row = [&](float v, auto op) {
#pragma unroll
      for (int d = 1; d < (LANES ? LANES : 64); d <<= 1) v = op(v, __shfl_xor(v, d, 64));
      if (LANES) return v;
      __syncthreads();   // what was there has been read
      if (lane == 0) red[0][wave] = v;
      __syncthreads();
      v = red[0][0];
      for (int i = 1; i < waves; ++i) v = op(v, red[0][i]);
      return v;
    };
    auto larger = [](float p, float q) { return fmaxf(p, q); };
    float top = sqrtf(a.eps);
#pragma unroll
    for (int s = 0; s < STRIPES; ++s) {
      if (a.residual_out && in[s] && there) *reinterpret_cast<i32x4*>(a.residual_out + row + at[s]) = narrow8(h[s]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in[s]) top = fmaxf(top, fabsf(h[s][i]));
    }
    top = over_row(top, larger);
    if (top > 0.f && top < INFINITY) {
      const float f = ldexpf(1.f, min(max(-ilogbf(top), -126), 126));
      sum = 0.f;
#pragma unroll
      for (int s = 0; s < STRIPES; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[s][i] *= f;
          if (in[s]) sum = __builtin_fmaf(h[s][i], h[s][i], sum);
        }
      sum = over_row(sum, [](float p, float q) { return p + q; });
      rstd = 1.f / sqrtf(sum / (float)a.H + a.eps * f * f);
    }
    if (QUANT == kQuantRow) {
      most = 0.f;
#pragma unroll
      for (int s = 0; s < STRIPES; ++s) {
        if (!kKeepWeight) weights(s, w[s]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in[s]) most = fmaxf(most, fabsf(h[s][i] * rstd * w[s][i]));
      }
      most = over_row(most, larger);
    }
  }
  float scale = 1.f;
  if (QUANT == kQuantRow) {
    scale = fp8_scale(most);
    if (tid == 0 && there) a.sx[t] = scale;
  }
#pragma unroll
  for (int s = 0; s < STRIPES; ++s) {
    if (!kKeepWeight) weights(s, w[s]);
    float y[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = h[s][i] * rstd * w[s][i];
      m = fmaxf(m, fabsf(y[i]));
    }
    if (QUANT == kQuantBlock) scale = fp8_scale(row16_max(m));   // 128 columns: 16 lanes
    if (!in[s] || !there) continue;
    if (a.residual_out && !far)
      __builtin_nontemporal_store(narrow8(h[s]), reinterpret_cast<i32x4*>(a.residual_out + row + at[s]));
    if (a.y) *reinterpret_cast<i32x4*>(a.y + row + at[s]) = narrow8(y);
    if (QUANT == kQuantNone) continue;
    if (QUANT == kQuantBlock && (lane & 15) == 0) a.sx[(row + at[s]) / kGroup] = scale;
    const ScaleDiv q = scale_div(scale);
    *reinterpret_cast<uint2*>(a.xq + row + at[s]) = make_uint2(
        quant2(q, y[0], y[1]) | quant2(q, y[2], y[3]) << 16, quant2(q, y[4], y[5]) | quant2(q, y[6], y[7]) << 16);
  }
}

template <Quant QUANT>
static hipError_t launch_quant(const NormArgs& a, hipStream_t stream) {
  const int pieces = (a.H + 511) / 512;   // a wave's part of a stripe
  auto whole = [&](auto* kernel, int stripes) {
    hipLaunchKernelGGL(kernel, dim3(a.T), dim3(64 * ((pieces + stripes - 1) / stripes)), 0, stream, a);
  };
  auto several = [&](auto* kernel, int rows) {
    hipLaunchKernelGGL(kernel, dim3((a.T + rows - 1) / rows), dim3(256), 0, stream, a);
  };
  if (a.H <= 128) several(add_rms_norm_kernel<1, QUANT, 16>, 16);
  else if (a.H <= 512) several(add_rms_norm_kernel<1, QUANT, 64>, 4);
  else if (pieces <= 4) whole(add_rms_norm_kernel<1, QUANT, 0>, 1);
  else if (pieces <= 16) whole(add_rms_norm_kernel<2, QUANT, 0>, 2);
  else if (pieces <= 64) whole(add_rms_norm_kernel<4, QUANT, 0>, 4);
  else whole(add_rms_norm_kernel<8, QUANT, 0>, 8);
  return hipGetLastError();
}

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t stream) {
  if (!a.xq) return launch_quant<kQuantNone>(a, stream);
  return a.block ? launch_quant<kQuantBlock>(a, stream) : launch_quant<kQuantRow>(a, stream);
}

}  // namespace srmoe
