// Per-head RMS norm and rotary embedding of q and k, as in qknorm.hip, with the results
// written where the attention reads them: q to its own rows, k and v into the paged cache
// as bf16 or e4m3. qkv itself is only read.
//
// Work split as in qknorm.hip: D/8 lanes per head, each lane one 16-byte load of 8
// consecutive values; the sum of squares is a butterfly over the head's lanes, a
// rotate-half partner is one lane exchange away. Every head of a token (q, k and v) is one
// group of lanes, so the three kinds share one launch.
#include "attention.hpp"
#include "common.hpp"

namespace srmoe {

// v / scale held to +-448, for its e4m3 code: the division itself (the FMA form of scale_div loses
// the sign of -0 and makes NaN of a quotient that overflows), and NaN kept (a comparison with it is
// false).
__device__ __forceinline__ float fp8_quotient(float v, float scale) {
  const float q = __fdiv_rn(v, scale);
  return q > kFp8Max ? kFp8Max : (q < -kFp8Max ? -kFp8Max : q);
}

template <int LPH>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a) {
  constexpr int D = 8 * LPH;
  constexpr int kHeadsPerWave = kWave / LPH;
  const int lane = threadIdx.x & 63;
  const int heads = a.Hq + 2 * a.Hkv, nqk = a.Hq + a.Hkv;
  const int total = a.T * heads;   // <= 2^20 * 2^10
  const int g = ((int)blockIdx.x * 4 + (threadIdx.x >> 6)) * kHeadsPerWave + lane / LPH;
  const bool valid = g < total;
  // lanes past the last head work on it and store nothing, so that every lane of a head group
  // takes part in the exchanges
  const int gc = valid ? g : total - 1;
  const int t = gc / heads, h = gc - t * heads;
  const int j = lane % LPH;   // dims 8j .. 8j+7 of the head
  const uint4 raw = *reinterpret_cast<const uint4*>(a.qkv + (size_t)t * a.qkv_stride + (size_t)h * D + 8 * j);
  const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_to_f32(r[i] & 0xFFFFu);
    x[2 * i + 1] = bf16_to_f32(r[i] >> 16);
  }
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m, kWave);
    if (h < nqk) {
      const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
      const float* w = (h < a.Hq ? a.qw : a.kw) + 8 * j;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
    }
  }
  if (a.rd) {
    const int half = a.rd >> 1;
    const int pos = min(max(a.positions[t], 0), a.max_pos - 1);
    const float* cs = a.cos_sin + (size_t)pos * a.rd;
    const bool rotated = h < nqk && 8 * j < a.rd;
    if (a.neox) {
      // partner of dim d is d + half (d < half) or d - half: lane j ^ (half / 8)
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_xor(x[i], half >> 3, kWave);
      if (rotated) {
        const bool first = 8 * j < half;
        const int f0 = first ? 8 * j : 8 * j - half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = cs[f0 + i], s = cs[half + f0 + i];
          x[i] = first ? x[i] * c - y[i] * s : x[i] * c + y[i] * s;
        }
      }
    } else if (rotated) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float c = cs[4 * j + q], s = cs[half + 4 * j + q];
        const float u = x[2 * q], v = x[2 * q + 1];
        x[2 * q] = u * c - v * s;
        x[2 * q + 1] = v * c + u * s;
      }
    }
  }
  if (!valid) return;
  uint4 o;
  o.x = pack_bf16x2(x[0], x[1]);
  o.y = pack_bf16x2(x[2], x[3]);
  o.z = pack_bf16x2(x[4], x[5]);
  o.w = pack_bf16x2(x[6], x[7]);
  if (h < a.Hq) {
    *reinterpret_cast<uint4*>(a.q_out + ((size_t)t * a.Hq + h) * D + 8 * j) = o;
    return;
  }
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) return;
  const bool is_v = h >= nqk;
  const int hk = h - (is_v ? nqk : a.Hq);
  const int page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
  const size_t e = (size_t)page * a.page_stride + ((size_t)((hk << a.page_shift) + at)) * D + 8 * j;
  if (a.fp8) {
    const float s = (is_v ? a.v_scale : a.k_scale)[hk];
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3_pack2(fp8_quotient(x[2 * i], s), fp8_quotient(x[2 * i + 1], s));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + e) =
        make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + e) = o;
  }
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  const int heads = a.T * (a.Hq + 2 * a.Hkv);
  const int per_block = 4 * (kWave / (a.D / 8));
  const dim3 grid((unsigned)((heads + per_block - 1) / per_block));
  switch (a.D) {
    case 64: hipLaunchKernelGGL(kv_append_kernel<8>, grid, dim3(256), 0, stream, a); break;
    case 128: hipLaunchKernelGGL(kv_append_kernel<16>, grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL(kv_append_kernel<32>, grid, dim3(256), 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace srmoe
