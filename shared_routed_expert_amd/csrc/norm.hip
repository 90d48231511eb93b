// The residual's addition and the root-mean-square norm in front of the MoE layer, with the result in bf16 (what the
// router reads) and in e4m3 with scales (what the expert GEMMs read, in place of moe_ffn_quant_x's pass over it):
//   h = x + r,  residual_out = bf16(h),  y = h rstd w,  rstd = (mean h^2 + eps)^-1/2,  codes = e4m3(y / s),
//   s = max |y| / 448 over the row or over 128 columns.
// One reduction serves both the norm and the scale: max |y| = rstd max |h w|.
#include "norm.hpp"
#include "common.hpp"

namespace srmoe {

// 8 bf16 values of a 16-byte word, widened
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

enum Quant { kQuantNone, kQuantRow, kQuantBlock };

// One workgroup of WAVES waves per row, thread t holding values 8 t .. 8 t + 7 of every stripe of 512 WAVES. STRIPES > 0:
// the row's h stays in registers (H <= 512 WAVES STRIPES); 0: any H, x and r are read a second time.
template <int WAVES, int STRIPES, Quant QUANT>
__global__ void __launch_bounds__(64 * WAVES) add_rms_norm_kernel(const NormArgs a) {
  __shared__ float red[2][WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t t = blockIdx.x;
  const uint16_t* const x = a.x + t * a.x_stride;
  const uint16_t* const r = a.residual ? a.residual + t * a.H : nullptr;
  constexpr int kKept = STRIPES > 0 ? STRIPES : 1;
  constexpr int kStride = 512 * WAVES;
  float h[kKept][8];
  auto load = [&](int at, float (&f)[8]) {
    widen8(*reinterpret_cast<const uint4*>(x + at), f);
    if (r) {
      float g[8];
      widen8(*reinterpret_cast<const uint4*>(r + at), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
    }
  };
  float sum = 0.f, most = 0.f;
  auto add = [&](int at, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(f[i], f[i], sum);
    if (QUANT == kQuantRow) {
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(f[i] * a.weight[at + i]));
    }
  };
  if (STRIPES > 0) {
#pragma unroll
    for (int s = 0; s < kKept; ++s) {
      const int at = s * kStride + tid * 8;
      if (at < a.H) {
        load(at, h[s]);
        add(at, h[s]);
      }
    }
  } else {
    for (int at = tid * 8; at < a.H; at += kStride) {
      load(at, h[0]);
      add(at, h[0]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  if (QUANT == kQuantRow) most = wave_max(most);
  if (WAVES > 1) {
    if (lane == 0) {
      red[0][wave] = sum;
      red[1][wave] = most;
    }
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      sum += red[0][i];
      most = fmaxf(most, red[1][i]);
    }
  }
  const float rstd = 1.f / sqrtf(sum / (float)a.H + a.eps);
  float scale = 1.f;
  if (QUANT == kQuantRow) {
    scale = fp8_scale(most * rstd);
    if (tid == 0) a.sx[t] = scale;
  }
  auto store = [&](int at, float (&f)[8], bool in) {
    float y[8];
    if (in && a.residual_out) *reinterpret_cast<uint4*>(a.residual_out + t * a.H + at) = narrow8(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = in ? f[i] * rstd * a.weight[at + i] : 0.f;
    if (in && a.y) *reinterpret_cast<uint4*>(a.y + t * a.H + at) = narrow8(y);
    if (QUANT == kQuantNone) return;
    if (QUANT == kQuantBlock) {   // 128 columns: 16 lanes
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
      scale = fp8_scale(row16_max(m));
      if (in && (lane & 15) == 0) a.sx[t * (a.H / kGroup) + at / kGroup] = scale;
    }
    const ScaleDiv q = scale_div(scale);
    if (in)
      *reinterpret_cast<uint2*>(a.xq + t * a.H + at) = make_uint2(
          quant2(q, y[0], y[1]) | quant2(q, y[2], y[3]) << 16, quant2(q, y[4], y[5]) | quant2(q, y[6], y[7]) << 16);
  };
  if (STRIPES > 0) {
#pragma unroll
    for (int s = 0; s < kKept; ++s) {
      const int at = s * kStride + tid * 8;
      store(at, h[s], at < a.H);
    }
  } else {
    for (int base = 0; base < a.H; base += kStride) {
      const int at = base + tid * 8;
      if (at < a.H) load(at, h[0]);
      store(at, h[0], at < a.H);
    }
  }
}

template <Quant QUANT>
static hipError_t launch_quant(const NormArgs& a, hipStream_t stream) {
  const dim3 grid(a.T);
  if (a.H <= 2048) hipLaunchKernelGGL((add_rms_norm_kernel<4, 1, QUANT>), grid, dim3(256), 0, stream, a);
  else if (a.H <= 4096) hipLaunchKernelGGL((add_rms_norm_kernel<4, 2, QUANT>), grid, dim3(256), 0, stream, a);
  else if (a.H <= 8192) hipLaunchKernelGGL((add_rms_norm_kernel<4, 4, QUANT>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((add_rms_norm_kernel<8, 0, QUANT>), grid, dim3(512), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t stream) {
  if (!a.xq) return launch_quant<kQuantNone>(a, stream);
  return a.block ? launch_quant<kQuantBlock>(a, stream) : launch_quant<kQuantRow>(a, stream);
}

}  // namespace srmoe
