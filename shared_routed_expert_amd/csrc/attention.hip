// Attention over the paged cache, in its plainest form: one wavefront per query head of
// a token walks the sequence's keys 64 at a time, a key per lane for the scores and D / 64
// dims per lane for the weighted values, with the running maximum m and sum l of the
// softmax (float32):
//     m' = max(m, max z),  l' = l e^(m - m') + sum e^(z - m'),  o' = o e^(m - m') + sum e^(z - m') v
#include "attention.hpp"
#include "common.hpp"

namespace srmoe {

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(64) attention_plain_kernel(const AttnArgs a) {
  __shared__ float qs[D];
  __shared__ float ps[kWave];
  __shared__ long base[kWave];
  const int lane = threadIdx.x, h = blockIdx.y, hk = h / a.G;
  // sequence of query row blockIdx.x
  const int row = blockIdx.x;
  int s = -1;
  SeqInfo si{};
  for (int i = 0; i < a.S; ++i) {
    si = seq_info(a, i);
    if (row >= si.row0 && row < si.row0 + si.n) {
      s = i;
      break;
    }
  }
  if (s < 0) return;
  const int i = row - si.row0, ctx = si.kv - si.n;
  for (int d = lane; d < D; d += kWave) qs[d] = bf16_to_f32(a.q[(size_t)row * a.q_stride + (size_t)h * D + d]);
  const float ks = kFp8 ? a.k_scale[hk] : 1.f, vs = kFp8 ? a.v_scale[hk] : 1.f;
  const uint64_t mask = a.tree_mask ? a.tree_mask[row] : 0;
  const int pre = a.prefix_lens ? a.prefix_lens[s] : 0;
  const int ps_mask = (1 << a.page_shift) - 1;
  float m = -INFINITY, l = 0.f, o[D / kWave] = {};
  __syncthreads();
  for (int j0 = 0; j0 < si.kv; j0 += kWave) {
    const int j = j0 + lane;
    long e = -1;
    bool see = j < si.kv;
    if (see) {
      const int page = a.block_table[(size_t)s * a.max_pages + (j >> a.page_shift)];
      if (page >= 0 && page < a.num_pages)
        e = (long)page * (long)a.page_stride + (long)((hk << a.page_shift) + (j & ps_mask)) * D;
      const int b = j - ctx;
      see = e >= 0 && (b < 0 || (a.tree_mask ? ((mask >> b) & 1) != 0 : b <= i) || j < pre);
      if (a.tree_mask && b < 0) see = e >= 0;
    }
    float z = -INFINITY;
    if (see) {
      float dot = 0.f;
      for (int d = 0; d < D; ++d) {
        const float k = kFp8 ? e4m3_to_f32(static_cast<const uint8_t*>(a.k_cache)[e + d])
                             : bf16_to_f32(static_cast<const uint16_t*>(a.k_cache)[e + d]);
        dot += qs[d] * k;
      }
      z = dot * ks * a.scale;
      if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
    }
    const float mn = fmaxf(m, wave_max(z));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float p = expf(z - ref), f = expf(m - ref);
    float sum = p;
    for (int w = 1; w < kWave; w <<= 1) sum += __shfl_xor(sum, w, kWave);
    l = l * f + sum;
    m = mn;
    ps[lane] = p;
    base[lane] = see ? e : -1;
    __syncthreads();
    for (int c = 0; c < D / kWave; ++c) o[c] *= f;
    for (int k = 0; k < kWave; ++k) {
      const long b = base[k];
      if (b < 0) continue;
      for (int c = 0; c < D / kWave; ++c) {
        const float v = kFp8 ? e4m3_to_f32(static_cast<const uint8_t*>(a.v_cache)[b + c * kWave + lane])
                             : bf16_to_f32(static_cast<const uint16_t*>(a.v_cache)[b + c * kWave + lane]);
        o[c] += ps[k] * v;
      }
    }
    __syncthreads();
  }
  for (int c = 0; c < D / kWave; ++c)
    a.out[((size_t)row * a.Hq + h) * D + c * kWave + lane] = f32_to_bf16(l > 0.f ? o[c] * vs / l : 0.f);
  if (a.lse && lane == 0) a.lse[(size_t)row * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

size_t attention_workspace_bytes(int, int, int, int, int) { return 0; }

template <bool kFp8>
static void launch_plain(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.T, (unsigned)a.Hq);
  switch (a.D) {
    case 64: hipLaunchKernelGGL((attention_plain_kernel<64, kFp8>), grid, dim3(64), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((attention_plain_kernel<128, kFp8>), grid, dim3(64), 0, stream, a); break;
    default: hipLaunchKernelGGL((attention_plain_kernel<256, kFp8>), grid, dim3(64), 0, stream, a); break;
  }
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
  if (a.k_scale)
    launch_plain<true>(a, stream);
  else
    launch_plain<false>(a, stream);
  return hipGetLastError();
}

}  // namespace srmoe
