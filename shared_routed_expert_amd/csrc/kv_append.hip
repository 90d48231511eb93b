// Per-head RMS norm and rotary embedding of q and k, as in qknorm.hip, with the results
// written where the attention reads them: q to its own rows, k and v into the paged cache
// as bf16 or e4m3. qkv itself is only read.
//
// Work split: D/8 lanes per head, each lane 8 consecutive values (one 16-byte load); the sum of
// squares is a butterfly over the head's lanes, a rotate-half partner is one lane exchange
// away. A wavefront takes kGroups groups of 64 / (D/8) heads of ONE token, all loaded before the
// first is used, with the token's position, slot, cosines and sines and the norm weights fetched once
// beside them. Bound by memory latency, then bytes. Two groups per wavefront, measured against one
// and four: 16384 tokens of 12 + 2 heads into e4m3 31 us (35, 31; 118 MB), 5000 tokens of 96 + 16 heads 55 us (68,
// 56; 288 MB, 5.2 TB/s); one group where all wavefronts are resident at once: 64 tokens 3.7 us (two: 4.6).
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

template <int LPH, int kGroups>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a, const int chunks) {
  constexpr int D = 8 * LPH;
  constexpr int kHeadsPerWave = kWave / LPH;
  const int lane = threadIdx.x & 63;
  const int heads = a.Hq + 2 * a.Hkv, nqk = a.Hq + a.Hkv;
  const int wave = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + (threadIdx.x >> 6));
  const int t = wave / chunks;
  if (t >= a.T) return;
  const int h0 = (wave - t * chunks) * (kGroups * kHeadsPerWave) + lane / LPH;   // and every kHeadsPerWave-th after
  const int j = lane % LPH;   // dims 8j .. 8j+7 of the head
  const uint16_t* row = a.qkv + (size_t)t * a.qkv_stride + 8 * j;
  uint4 raw[kGroups];
#pragma unroll
  for (int u = 0; u < kGroups; ++u)   // lanes past the last head load it again and store nothing
    raw[u] = *reinterpret_cast<const uint4*>(row + (size_t)min(h0 + u * kHeadsPerWave, heads - 1) * D);
  const int slot = a.slots[t];
  const int half = a.rd >> 1;
  const bool rotated = 8 * j < a.rd, first = 8 * j < half;
  float c[8], s[8];
  if (rotated) {
    const int pos = min(max(a.positions[t], 0), a.max_pos - 1);
    const float* cs = a.cos_sin + (size_t)pos * a.rd;
    if (a.neox) {
      const float4* p = reinterpret_cast<const float4*>(cs + (first ? 8 * j : 8 * j - half));
      const float4* q = reinterpret_cast<const float4*>(cs + half + (first ? 8 * j : 8 * j - half));
      const float4 c0 = p[0], c1 = p[1], s0 = q[0], s1 = q[1];
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    } else {
      const float4 c0 = *reinterpret_cast<const float4*>(cs + 4 * j);
      const float4 s0 = *reinterpret_cast<const float4*>(cs + half + 4 * j);
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
    }
  }
  float4 qw[2], kw[2];
  if (a.norm) {
    kw[0] = *reinterpret_cast<const float4*>(a.kw + 8 * j);
    kw[1] = *reinterpret_cast<const float4*>(a.kw + 8 * j + 4);
    const float* w = a.Hq > 0 ? a.qw : a.kw;
    qw[0] = *reinterpret_cast<const float4*>(w + 8 * j);
    qw[1] = *reinterpret_cast<const float4*>(w + 8 * j + 4);
  }
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const int h = h0 + u * kHeadsPerWave;
    const uint32_t r[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
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
        const float4 w0 = h < a.Hq ? qw[0] : kw[0], w1 = h < a.Hq ? qw[1] : kw[1];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
      }
    }
    if (a.rd) {
      if (a.neox) {
        // partner of dim d is d + half (d < half) or d - half: lane j ^ (half / 8)
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_xor(x[i], half >> 3, kWave);
        if (rotated && h < nqk) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * c[i] - y[i] * s[i] : x[i] * c[i] + y[i] * s[i];
        }
      } else if (rotated && h < nqk) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v0 = x[2 * q], v1 = x[2 * q + 1];
          x[2 * q] = v0 * c[q] - v1 * s[q];
          x[2 * q + 1] = v1 * c[q] + v0 * s[q];
        }
      }
    }
    uint4 o;
    o.x = pack_bf16x2(x[0], x[1]);
    o.y = pack_bf16x2(x[2], x[3]);
    o.z = pack_bf16x2(x[4], x[5]);
    o.w = pack_bf16x2(x[6], x[7]);
    if (h < a.Hq) {
      *reinterpret_cast<uint4*>(a.q_out + ((size_t)t * a.Hq + h) * D + 8 * j) = o;
    } else if (h < heads && slot >= 0 && slot < a.num_slots) {
      const bool is_v = h >= nqk;
      const int hk = h - (is_v ? nqk : a.Hq);
      const int page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
      const size_t e = (size_t)page * a.page_stride + ((size_t)((hk << a.page_shift) + at)) * D + 8 * j;
      if (a.fp8) {
        const float scale = (is_v ? a.v_scale : a.k_scale)[hk];
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          code[i] = e4m3_pack2(fp8_quotient(x[2 * i], scale), fp8_quotient(x[2 * i + 1], scale));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + e) =
            make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + e) = o;
      }
    }
  }
}

template <int LPH>
static void launch_heads(const KvAppendArgs& a, hipStream_t stream) {
  constexpr int kHeadsPerWave = kWave / LPH;
  const int groups = (a.Hq + 2 * a.Hkv + kHeadsPerWave - 1) / kHeadsPerWave;
  if ((long)a.T * groups <= 4096) {
    hipLaunchKernelGGL((kv_append_kernel<LPH, 1>), dim3((unsigned)((a.T * groups + 3) / 4)), dim3(256), 0, stream, a,
                       groups);
  } else {
    const int chunks = (groups + 1) / 2;
    hipLaunchKernelGGL((kv_append_kernel<LPH, 2>), dim3((unsigned)((a.T * chunks + 3) / 4)), dim3(256), 0, stream, a,
                       chunks);
  }
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: launch_heads<8>(a, stream); break;
    case 128: launch_heads<16>(a, stream); break;
    default: launch_heads<32>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace srmoe
