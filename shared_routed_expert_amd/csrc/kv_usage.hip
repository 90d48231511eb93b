// What attention weight every cached token has received: column sums of the attention matrix over a call's tokens and the
// query heads of a kv head,
//   usage_j = decay prev_j + sum_{i, g} exp(z_{ig,j} - lse_{ig})     over the rows (i, g) that see key j,
// from q, the cached keys and the attention call's own lse: the weights themselves are never stored.
//
// Keys stay, rows pass. A workgroup's four waves hold KPW keys each in registers, as the A operand of 16x16x32 matrix
// instructions, and the rows come by in tiles of 32 through LDS, one tile ahead. A lane of the result S = K Q^T owns one row
// (its column l & 15) and 4 keys per 16, so a weight is one fma (score, scale, -lse), one exponential, and one fma into
// the lane's own sum of that key; the 16 lanes of a key are added up once, after the last row. lse log2 e is split into
// its float32 value and a factor 2^-remainder that rides in the last fma.
//
// Work split. A segment is one block of 4 KPW keys of a sequence and kv head against all rows that see one of them. All segments
// are laid end to end, each as long as its rows and a fixed cost, and workgroup w takes the w-th of equal parts of that
// line. A segment in several parts leaves one partial sum per part, added in part order by a second kernel (no atomics,
// the same bits every time); calls of at most 32 rows per sequence never split one and have no second kernel.
#include "kv_usage.hpp"
#include "attention_common.hpp"

namespace srmoe {

// One sequence's key blocks: block b (of MB) is seen by the tokens from first(b) on.
struct SeqBlocks {
  int row0, n, kv, ctx, all, MB;   // keys up to `all` are seen by every token (-1: none is)
  __device__ __forceinline__ int first(int b, int KB) const { return b * KB <= all ? 0 : min(b * KB - ctx, n); }
  // cost of blocks 0 .. m - 1 of one head: (n - first) G + fixed each, in closed form
  __device__ __forceinline__ long cost(int m, int KB, int G, int fixed) const {
    const long flat = all >= 0 ? min(MB, all / KB + 1) : 0;                      // blocks that all tokens see
    const long end = n + ctx > 0 ? min((long)MB, ((long)n + ctx + KB - 1) / KB) : 0;   // and that any token sees
    const long to = min((long)m, end);
    long tokens = min((long)m, flat) * n;
    if (to > flat) tokens += (to - flat) * ((long)n + ctx) - (long)KB * ((to * (to - 1) - flat * (flat - 1)) / 2);
    return tokens * G + (long)m * fixed;
  }
};
__device__ __forceinline__ SeqBlocks seq_blocks(const AttnArgs& a, int s, int KB) {
  const SeqInfo q = seq_info(a, s);
  SeqBlocks t;
  t.row0 = q.row0;
  t.n = q.n;
  t.kv = q.kv;
  t.ctx = q.kv - q.tokens;
  t.all = max(t.ctx, (a.prefix_lens ? min(max(a.prefix_lens[s], 0), q.kv) : 0) - 1);
  if (t.all < 0) t.all = -1;
  t.MB = q.n > 0 ? (q.kv + KB - 1) / KB : 0;   // (without tokens the sequence is left alone)
  return t;
}

// A segment that begins in part `first` and ends in a later part `last` (keys == 0: nothing to join)
struct alignas(32) UsageDesc {
  int s, head, k0, keys, first, last;
};

constexpr int kUsageParts = 768;   // three workgroups on each CU
constexpr int kUsageRows = 32;      // rows of a tile

// Where a sequence's weights are, or null: they are not kept
__device__ __forceinline__ size_t usage_at(const UsageArgs& u, int s, int head, bool* kept) {
  const int row = u.usage_rows ? u.usage_rows[s] : s;
  *kept = row >= 0 && row < u.rows;
  return ((size_t)(*kept ? row : 0) * u.a.Hkv + head) * ((size_t)u.a.max_pages << u.a.page_shift);
}

template <int D, bool FP8, Cap CAP>
struct Usage {
  static constexpr int kWaves = 4, kThreads = 64 * kWaves;
  static constexpr int KPW = D == 256 ? 32 : 64;   // keys of a wave: 64 registers of them (32 for D = 64)
  static constexpr int KB = KPW * kWaves, AT = KPW / 16;
  static constexpr int STEPS = D / 32;
  static constexpr int RB = D * (FP8 ? 1 : 2);
  static constexpr int CH = D / 8;                              // 16-byte chunks of a row of q
  static constexpr int LOADS = kUsageRows * CH / kThreads;      // of a thread for a tile
  // What a segment costs besides its rows, in rows (its keys, their sums)
  static constexpr int kSegCost = 64;
};

template <int D, bool FP8, Cap CAP>
__global__ void __launch_bounds__(256, D == 256 || CAP == kCapLarge ? 2 : 3) kv_usage_kernel(const UsageArgs args, const uint64_t magic, const int parts_max,
                                                          const bool joined, float* __restrict__ partials,
                                                          UsageDesc* __restrict__ descs) {
  using C = Usage<D, FP8, CAP>;
  const AttnArgs& a = args.a;
  __shared__ __attribute__((aligned(16))) uint16_t qs[2][kUsageRows * D];
  __shared__ float row_lse[2][kUsageRows], row_fix[2][kUsageRows];
  __shared__ int row_lim[2][kUsageRows];
  __shared__ long scan_sum[C::kWaves];
  __shared__ long found_rem;
  __shared__ int found_s;
  __shared__ SeqBlocks found_seq;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  // -------- which part of the line of segments is this workgroup's: a stretch of sequences per thread
  const int per = (a.S + C::kThreads - 1) / C::kThreads;
  const int s_lo = min(tid * per, a.S), s_hi = min(s_lo + per, a.S);
  long mine = 0;
  for (int s = s_lo; s < s_hi; ++s) {
    const SeqBlocks t = seq_blocks(a, s, C::KB);
    mine += t.cost(t.MB, C::KB, a.G, C::kSegCost) * a.Hkv;
  }
  long incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) scan_sum[wave] = incl;
  __syncthreads();
  long total = 0, before = incl - mine;
#pragma unroll
  for (int i = 0; i < C::kWaves; ++i) {
    if (i < wave) before += scan_sum[i];
    total += scan_sum[i];
  }
  total = uni(total);
  const int parts = (int)min((long)parts_max, (total + C::kSegCost - 1) / C::kSegCost);
  const int w = xcd_tile((int)blockIdx.x, parts);   // consecutive parts on one XCD: neighbouring keys, the same rows
  if (joined) {   // no segment begins in these parts until one is written below
    if (blockIdx.x == 0)
      for (int i = parts + tid; i < parts_max; i += C::kThreads) descs[i] = UsageDesc{0, 0, 0, 0, 0, 0};
    if (w >= 0 && tid == 0) descs[w] = UsageDesc{0, 0, 0, 0, 0, 0};
  }
  if (w < 0 || w >= parts) return;
  const Parts split(total, parts);
  long u = split.begin(w);
  const long u_end = split.begin(w + 1);
  if (mine > 0 && u >= before && u < before + mine) {   // one thread alone
    long r = u - before;
    for (int i = s_lo; i < s_hi; ++i) {
      const SeqBlocks t = seq_blocks(a, i, C::KB);
      const long cost = t.cost(t.MB, C::KB, a.G, C::kSegCost) * a.Hkv;
      if (r < cost) {
        found_s = i;
        found_seq = t;
        found_rem = r;
        break;
      }
      r -= cost;
    }
  }
  __syncthreads();
  auto uniform = [](SeqBlocks t) {
    t.row0 = uni(t.row0); t.n = uni(t.n); t.kv = uni(t.kv); t.ctx = uni(t.ctx); t.all = uni(t.all); t.MB = uni(t.MB);
    return t;
  };
  int s = uni(found_s);
  long rem = uni(found_rem);
  SeqBlocks seq = uniform(found_seq);
  int h, kb;
  {
    const long per_head = seq.cost(seq.MB, C::KB, a.G, C::kSegCost);
    h = uni((int)div_pos(rem, per_head));
    rem -= h * per_head;
    int lo = 0, hi = seq.MB;   // the largest block with cost(block) <= rem, 64 candidates at a time
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) >> 6, at = lo + lane * step;
      const int n = __popcll(__ballot(at < hi && seq.cost(at, C::KB, a.G, C::kSegCost) <= rem));
      lo = uni(lo + (n - 1) * step);
      hi = uni(min(hi, lo + step));
    }
    kb = lo;
    rem -= seq.cost(kb, C::KB, a.G, C::kSegCost);
  }

  const int page_mask = (1 << a.page_shift) - 1;
  const size_t page_bytes = a.page_stride * (FP8 ? 1 : 2);
  int buf = 0;
  while (u < u_end) {
    // -------- the segment: its rows, and this part's share of their tiles (the fixed cost comes first; a part whose share
    // of the front is no tile leaves the segment to the next one, which then begins it)
    const int k0 = kb * C::KB;
    const int i0 = seq.first(kb, C::KB);
    const int rows = (seq.n - i0) * a.G, r0 = i0 * a.G;
    const long seg_end = u - rem + rows + C::kSegCost;
    const bool ends = seg_end <= u_end;
    const int ntiles = (rows + kUsageRows - 1) / kUsageRows;
    const int t0 = (int)(max(rem - C::kSegCost, 0l) / kUsageRows);
    const int t1 = ends ? ntiles : (int)(max(rem + u_end - u - C::kSegCost, 0l) / kUsageRows);
    const bool begins = ntiles > 0 ? t0 == 0 : rem == 0;
    if (ntiles > 0 ? t1 > 0 : begins) {
      const float ks = FP8 ? a.k_scale[h] : 1.f;
      const float c = CAP ? 2.f * kLog2e * a.scale * ks / a.softcap : a.scale * kLog2e * ks;
      const float cap2 = a.softcap * kLog2e, half_cap = 0.5f * a.softcap;
      // -------- this wave's keys: 16 of them lie in one page; those past the end and of pages outside the pool are read
      // from page 0 (every key has sums of its own, and theirs are dropped)
      const int wk = k0 + wave * C::KPW;
      const int my_key = wk + 16 * (lane & (C::AT - 1));
      int id = my_key < seq.kv ? a.block_table[(size_t)s * a.max_pages + (my_key >> a.page_shift)] : -1;
      const uint32_t pages_ok = (uint32_t)__ballot(id >= 0 && id < a.num_pages) & ((1u << C::AT) - 1);
      if (id < 0 || id >= a.num_pages) id = 0;
      const uint8_t* const kc = static_cast<const uint8_t*>(a.k_cache) + ((size_t)h << a.page_shift) * C::RB;
      bf16x8 k[C::AT][C::STEPS];
      if (t0 < t1) {
#pragma unroll
        for (int t = 0; t < C::AT; ++t) {
          const size_t at = (size_t)__builtin_amdgcn_readlane(id, t) * page_bytes +
                            (size_t)((wk + 16 * t) & page_mask) * C::RB;
          const uint8_t* p = kc + at + col * C::RB + quarter * 16;
          if constexpr (FP8) {   // 16 bytes are two steps' 8 values of this lane
#pragma unroll
            for (int st = 0; st < C::STEPS; st += 2) {
              const i32x4 v = *reinterpret_cast<const i32x4*>(p + st * 32);
              k[t][st] = bf16_of_e4m3(v[0], v[1]);
              k[t][st + 1] = bf16_of_e4m3(v[2], v[3]);
            }
          } else {
#pragma unroll
            for (int st = 0; st < C::STEPS; ++st) k[t][st] = *reinterpret_cast<const bf16x8*>(p + st * 64);
          }
        }
      }
      // -------- rows, a tile ahead: chunk c of row r sits at c ^ (r & 15) (D = 64, two rows to LDS's 64 banks: (r >> 1) & 7)
      i32x4 ahead[C::LOADS];
      float ahead_lse = 0.f;
      int ahead_lim = 0;
      auto swizzle = [](int r) { return D == 64 ? (r >> 1) & 7 : r & 15; };
      auto token_of = [&](int r) { return (int)((uint64_t)r * magic >> 40); };
      const int r_end = seq.n * a.G;
      auto fetch = [&](int t) {
#pragma unroll
        for (int y = 0; y < C::LOADS; ++y) {
          const int x = y * C::kThreads + tid, r = min(r0 + t * kUsageRows + x / C::CH, r_end - 1);
          const int tok = token_of(r);
          const uint16_t* p = a.q + (size_t)(seq.row0 + tok) * a.q_stride + (size_t)(h * a.G + r - tok * a.G) * D;
          ahead[y] = *reinterpret_cast<const i32x4*>(p + (x % C::CH) * 8);
        }
        if (tid < kUsageRows) {
          const int r = r0 + t * kUsageRows + tid, tok = token_of(min(r, r_end - 1));
          // rows past the last, and such as saw nothing, add nothing
          ahead_lse = r < r_end ? args.lse[(size_t)(seq.row0 + tok) * a.Hq + h * a.G + r - tok * a.G] : INFINITY;
          if (ahead_lse == -INFINITY) ahead_lse = INFINITY;
          ahead_lim = max(seq.all, seq.ctx + tok) + 1;
        }
      };
      auto put = [&](int b) {
#pragma unroll
        for (int y = 0; y < C::LOADS; ++y) {
          const int x = y * C::kThreads + tid, r = x / C::CH;
          *reinterpret_cast<i32x4*>(&qs[b][r * D + ((x % C::CH) ^ swizzle(r)) * 8]) = ahead[y];
        }
        if (tid < kUsageRows) {
          // lse log2 e = l2 + rest
          constexpr float kLog2eRest = 1.92596299112661746e-8f;
          const float l2 = ahead_lse * kLog2e;
          const float rest = __builtin_fmaf(ahead_lse, kLog2e, -l2) + ahead_lse * kLog2eRest;
          row_lse[b][tid] = l2;
          row_fix[b][tid] = __builtin_fabsf(l2) < 1e30f ? __builtin_amdgcn_exp2f(-rest) : 1.f;
          row_lim[b][tid] = ahead_lim;
        }
      };
      float sum[C::AT][4];
#pragma unroll
      for (int t = 0; t < C::AT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] = 0.f;
      if (t0 < t1) {
        fetch(t0);
        put(buf);
      }
      for (int t = t0; t < t1; ++t) {
        __syncthreads();   // this tile is there, and the other buffer's rows have been read
        if (t + 1 < t1) fetch(t + 1);
        const int first = r0 + t * kUsageRows;
        // every key of this wave is seen by every row of the tile
        const bool all_seen = wk + C::KPW <= seq.ctx + uni(token_of(first)) + 1 || wk + C::KPW <= seq.all + 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (first + 16 * half >= r_end) break;
          const int r = 16 * half + col;
          bf16x8 q[C::STEPS];
#pragma unroll
          for (int st = 0; st < C::STEPS; ++st) {
            const int chunk = FP8 ? 8 * (st >> 1) + 2 * quarter + (st & 1) : 4 * st + quarter;
            q[st] = *reinterpret_cast<const bf16x8*>(&qs[buf][r * D + (chunk ^ swizzle(r)) * 8]);
          }
          const float l2 = row_lse[buf][r], fix = row_fix[buf][r];
          const int lim = row_lim[buf][r];
#pragma unroll
          for (int t4 = 0; t4 < C::AT; ++t4) {
            v4f z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < C::STEPS; ++st) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[t4][st], q[st], z, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float p = __builtin_amdgcn_exp2f(CAP ? capped<CAP == kCapLarge>(z[e] * c, half_cap, cap2) - l2
                                                   : __builtin_fmaf(z[e], c, -l2));
              if (!all_seen) p = wk + 16 * t4 + 4 * quarter + e < lim ? p : 0.f;
              sum[t4][e] = __builtin_fmaf(p, fix, sum[t4][e]);
            }
          }
        }
        buf ^= 1;
        if (t + 1 < t1) put(buf);
      }
      // -------- a key's sum over its 16 lanes; lane (quarter, col) takes key 16 (col / 4) + 4 quarter + col % 4
      float v = 0.f;
#pragma unroll
      for (int t = 0; t < C::AT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sum[t][e];
          x += dpp_f32<kDppXor1>(x);
          x += dpp_f32<kDppXor2>(x);
          x += dpp_f32<kDppRowHalfMirror>(x);
          x += dpp_f32<kDppRowMirror>(x);
          v = col == 4 * t + e ? x : v;
        }
      if (col < 4 * C::AT) {
        if (!((pages_ok >> (col >> 2)) & 1)) v = 0.f;
        const int at = wave * C::KPW + 16 * (col >> 2) + 4 * quarter + (col & 3), j = k0 + at;
        if (begins && (ends || ntiles == 0)) {
          bool kept;
          const size_t base = usage_at(args, s, h, &kept);
          if (kept && j < seq.kv)
            args.usage[base + j] = args.prev && j < seq.ctx ? __builtin_fmaf(args.decay, args.prev[base + j], v) : v;
        } else {
          partials[(size_t)(2 * w + (begins ? 1 : 0)) * C::KB + at] = v;
        }
      }
      if (joined && tid == 0 && begins && !(ends || ntiles == 0))
        descs[w] = UsageDesc{s, h, k0, min(C::KB, seq.kv - k0), w, split.of(seg_end - 1)};
    }

    // -------- the next segment
    u = min(u_end, seg_end);
    rem = 0;
    if (++kb >= seq.MB) {
      kb = 0;
      if (++h >= a.Hkv && u < u_end) {
        h = 0;
        do seq = uniform(seq_blocks(a, ++s, C::KB));
        while (seq.MB == 0);
      }
    }
  }
}

// Adds the partial sums of segments that span several parts, in part order: workgroup w the one that begins in part w.
__global__ void __launch_bounds__(256) kv_usage_join_kernel(const UsageArgs args, const int KB,
                                                            const float* __restrict__ partials,
                                                            const UsageDesc* __restrict__ descs) {
  const UsageDesc d = descs[blockIdx.x];
  const int at = threadIdx.x, j = d.k0 + at;
  if (at >= d.keys) return;
  bool kept;
  const size_t base = usage_at(args, d.s, d.head, &kept);
  if (!kept) return;
  float v = partials[(size_t)(2 * d.first + 1) * KB + at];
  for (int p = d.first + 1; p <= d.last; ++p) v += partials[(size_t)(2 * p) * KB + at];
  const SeqInfo q = seq_info(args.a, d.s);
  args.usage[base + j] = args.prev && j < q.kv - q.tokens ? __builtin_fmaf(args.decay, args.prev[base + j], v) : v;
}

size_t kv_usage_workspace_bytes(int D) {
  const size_t KB = D == 256 ? Usage<256, false, kCapNone>::KB : Usage<128, false, kCapNone>::KB;
  return kUsageParts * (2 * KB * 4 + sizeof(UsageDesc));
}

template <int D, bool FP8, Cap CAP>
static hipError_t launch_usage(const UsageArgs& u, hipStream_t stream) {
  using C = Usage<D, FP8, CAP>;
  const AttnArgs& a = u.a;
  float* partials = static_cast<float*>(a.ws);
  UsageDesc* descs = reinterpret_cast<UsageDesc*>(partials + 2 * (size_t)kUsageParts * C::KB);
  const bool joined = (long)a.max_q * a.G > kUsageRows;   // (one tile is one part's)
  const uint64_t magic = (1ull << 40) / (uint64_t)a.G + 1;   // row / G = row magic >> 40: row G < 2^40
  hipLaunchKernelGGL((kv_usage_kernel<D, FP8, CAP>), dim3(kUsageParts), dim3(C::kThreads), 0, stream, u, magic, kUsageParts,
                     joined, partials, descs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !joined) return e;
  hipLaunchKernelGGL(kv_usage_join_kernel, dim3(kUsageParts), dim3(C::KB), 0, stream, u, C::KB, (const float*)partials,
                     (const UsageDesc*)descs);
  return hipGetLastError();
}

template <int D, bool FP8>
static hipError_t launch_usage_cap(const UsageArgs& u, hipStream_t stream) {
  if (u.a.softcap == 0.f) return launch_usage<D, FP8, kCapNone>(u, stream);
  return u.a.softcap <= kNearCap ? launch_usage<D, FP8, kCapSmall>(u, stream) : launch_usage<D, FP8, kCapLarge>(u, stream);
}

template <int D>
static hipError_t launch_usage_dim(const UsageArgs& u, hipStream_t stream) {
  return u.a.k_scale ? launch_usage_cap<D, true>(u, stream) : launch_usage_cap<D, false>(u, stream);
}

hipError_t launch_kv_usage(const UsageArgs& u, hipStream_t stream) {
  switch (u.a.D) {
    case 64: return launch_usage_dim<64>(u, stream);
    case 128: return launch_usage_dim<128>(u, stream);
    default: return launch_usage_dim<256>(u, stream);
  }
}

}  // namespace srmoe
