// What attention weight every cached token has received: column sums of the attention matrix over a call's tokens and the
// query heads of a kv head,
//   usage_j = decay prev_j + sum_{i, g} exp(z_{ig,j} - lse_{ig})     over the rows (i, g) that see key j,
// from q, the cached keys and the attention call's own lse: the weights themselves are never stored.
//
// Two kernels by how many rows (token, head of the group) a sequence may have.
//
// More than 32: keys stay, rows pass. A workgroup's four waves hold 64 keys each in registers (32 at D = 256), as the A operand
// of 32x32x16 matrix instructions, and the rows come by in tiles of 128 (64) through LDS, straight from global memory, one
// tile ahead. A lane of the result S = K Q^T owns one row (its column l & 31) and 16 keys per 32, so a weight is one fma
// (score, scale, -lse), one exponential, and one fma into the lane's own sum of that key; the 32 lanes of a key are added
// up once, after the last row. lse log2 e is split into its float32 value and a factor 2^-remainder that rides in the last
// fma. The weights of one 32 x 32 tile are computed between the products of the next one. (16x16x32 products took 41 and
// 139 us in the two cases below instead of 38 and 126: twice the instructions for the same keys.)
//   Work split. A segment is one block of the workgroup's keys of a sequence and kv head against all rows that see one of them.
// All segments are laid end to end, each as long as its rows and a fixed cost, and workgroup w takes the w-th of 512 equal
// parts of that line, two workgroups on a CU: one's vector work beside the other's products. A segment in several parts
// leaves one partial sum per part, added in part order by a second kernel (no atomics, the same bits every time).
//   What bounds it: the vector unit and the matrix cores in turn, 3 vector instructions for 64 weights against D / 8 cycles of
// the matrix core. Two prompts of 4096 tokens behind 1904 cached ones, 12 heads of 128, take 116 to 126 us by the card (790
// to 860 TFLOP/s, matrix cores 37% busy), 4 of them for the sums, with a cap of 30 174, of 100 221. The last 64 tokens of
// 131072 cached in e4m3 take 34 to 37 (700 to 755 TFLOP/s), of which some 2 find the parts, 3 to 6 wait for the keys, 4 are
// the sums. One workgroup per CU with 128 keys a wave: 191 and 34. At D = 256 a wave holds one tile of 32 keys, so its weights
// have no products beside them: two prompts of 4096 after 1904, 8 heads, 154 to 160 us (830 to 860 TFLOP/s).
//
// At most 32 (decoding): bound by the keys' bytes; see kv_usage_few_kernel. 64 single tokens over up to 8192 keys, 82 MB, take
// 20 to 22 us (3.7 to 4.1 TB/s, a launch included), 43 MB in e4m3 15, 162 MB of 8 heads of 256 30 to 32.
#include "kv_usage.hpp"
#include "attention_common.hpp"

#include <type_traits>

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

constexpr int kUsageParts = 512;   // two workgroups on each CU

// All sequences' costs laid end to end: up to 64 of them one per lane, in every wave by itself; more, a stretch of them per
// thread of the workgroup (and barriers).
struct Line {
  SeqBlocks own;        // of this lane's sequence, S <= 64
  int s_lo, s_hi;
  long total, before, mine;
};
__device__ __forceinline__ SeqBlocks uniform(SeqBlocks t) {
  t.row0 = uni(t.row0); t.n = uni(t.n); t.kv = uni(t.kv); t.ctx = uni(t.ctx); t.all = uni(t.all); t.MB = uni(t.MB);
  return t;
}
__device__ __forceinline__ SeqBlocks lane_of(const SeqBlocks& t, int lane) {
  SeqBlocks u;
  u.row0 = __builtin_amdgcn_readlane(t.row0, lane);
  u.n = __builtin_amdgcn_readlane(t.n, lane);
  u.kv = __builtin_amdgcn_readlane(t.kv, lane);
  u.ctx = __builtin_amdgcn_readlane(t.ctx, lane);
  u.all = __builtin_amdgcn_readlane(t.all, lane);
  u.MB = __builtin_amdgcn_readlane(t.MB, lane);
  return u;
}
// The next sequence with key blocks, looked for 64 at a time; false where there is none. (One by one, each waits for the
// last one's lengths: 2 sequences of 40 tokens, the first and the last of 8192, 1430 us instead of 75, of 65536 11,300 instead of
// 432. One more by itself before the 64 costs registers: D = 256, two prompts of 4096, 166 us instead of 160.)
__device__ __forceinline__ bool next_seq(const AttnArgs& a, int KB, int& s, SeqBlocks& seq) {
  for (int at = s + 1; at < a.S; at += 64) {
    const SeqBlocks t = seq_blocks(a, min(at + (int)(threadIdx.x & 63), a.S - 1), KB);   // (lanes past the last one look at it)
    const uint64_t some = __ballot(t.MB > 0);
    if (some) {
      const int first = __ffsll((unsigned long long)some) - 1;
      s = at + first;
      seq = lane_of(t, first);
      return true;
    }
  }
  return false;
}
template <class F>   // cost(SeqBlocks) of a sequence
__device__ __forceinline__ Line lay_line(const AttnArgs& a, int KB, F cost, long* scan_sum /* LDS, 4 */) {
  const int tid = threadIdx.x, lane = tid & 63;
  Line l{};
  const bool few = a.S <= 64;
  const int per = few ? 1 : (a.S + 255) / 256;
  l.s_lo = min((few ? lane : tid) * per, a.S);
  l.s_hi = min(l.s_lo + per, a.S);
  for (int s = l.s_lo; s < l.s_hi; ++s) {
    l.own = seq_blocks(a, s, KB);
    l.mine += cost(l.own);
  }
  long incl = l.mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  l.before = incl - l.mine;
  if (few) {
    l.total = read_lane(incl, 63);
    return l;
  }
  if (lane == 63) scan_sum[tid >> 6] = incl;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < tid >> 6) l.before += scan_sum[i];
    l.total += scan_sum[i];
  }
  l.total = uni(l.total);
  return l;
}
// The sequence in which `unit` lies, and how far into it; S <= 64: for this wave, else the one thread that knows writes it
struct Place {
  int s;
  long rem;
};
__device__ __forceinline__ Place place_few(const Line& l, long unit, SeqBlocks& seq) {
  const int s = __ffsll((unsigned long long)__ballot(l.mine > 0 && unit >= l.before && unit < l.before + l.mine)) - 1;
  seq = lane_of(l.own, s);
  return {s, unit - read_lane(l.before, s)};
}
template <class F>
__device__ __forceinline__ void place_many(const AttnArgs& a, const Line& l, int KB, F cost, long unit, Place* to) {
  if (!(l.mine > 0 && unit >= l.before && unit < l.before + l.mine)) return;
  long r = unit - l.before;
  for (int s = l.s_lo; s < l.s_hi; ++s) {
    const long c = cost(seq_blocks(a, s, KB));
    if (r < c) {
      *to = {s, r};
      return;
    }
    r -= c;
  }
}

// Where a sequence's weights are, or null: they are not kept
__device__ __forceinline__ size_t usage_at(const UsageArgs& u, int s, int head, bool* kept) {
  const int row = u.usage_rows ? u.usage_rows[s] : s;
  *kept = row >= 0 && row < u.rows;
  return ((size_t)(*kept ? row : 0) * u.a.Hkv + head) * ((size_t)u.a.max_pages << u.a.page_shift);
}

// lse log2 e = l2 + rest, the remainder as a factor; rows that saw nothing add nothing
struct RowLse {
  float l2, fix;
};
__device__ __forceinline__ RowLse row_lse_of(float lse) {
  constexpr float kLog2eRest = 1.92596299112661746e-8f;   // log2 e minus its float32 value
  if (lse == -INFINITY) lse = INFINITY;
  const float l2 = lse * kLog2e;
  const float rest = __builtin_fmaf(lse, kLog2e, -l2) + lse * kLog2eRest;
  return {l2, __builtin_fabsf(l2) < 1e30f ? __builtin_amdgcn_exp2f(-rest) : 1.f};
}

// A key's 16 lanes added up: sums[t][e] of lane (quarter, col) is that of key 16 t + 4 quarter + e, row col; lane
// (quarter, col) gets the sum of key 16 (col / 4) + 4 quarter + col % 4.
__device__ __forceinline__ float column_sum(const float (*sums)[4], int col) {
  float v = 0.f;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = sums[t][e];
      x += dpp_f32<kDppXor1>(x);
      x += dpp_f32<kDppXor2>(x);
      x += dpp_f32<kDppRowHalfMirror>(x);
      x += dpp_f32<kDppRowMirror>(x);
      v = col == 4 * t + e ? x : v;
    }
  return v;
}

// 32 keys as the A operand of 32x32x16 products, from global memory (pages hold 16 at least: two addresses)
template <int D, bool FP8>
__device__ __forceinline__ void load_keys32(const uint8_t* lo, const uint8_t* hi, int lane, bf16x8 (&k)[D / 16]) {
  const uint8_t* p = (lane & 16 ? hi : lo) + (lane & 15) * (FP8 ? D : 2 * D) + (lane >> 5) * 16;
  if constexpr (FP8) {   // 16 bytes are two steps' 8 values of this lane
#pragma unroll
    for (int st = 0; st < D / 16; st += 2) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(p + st * 16);
      k[st] = bf16_of_e4m3(v[0], v[1]);
      k[st + 1] = bf16_of_e4m3(v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int st = 0; st < D / 16; ++st) k[st] = *reinterpret_cast<const bf16x8*>(p + st * 32);
  }
}
template <bool FP8>
__device__ __forceinline__ int q_chunk32(int st, int half) {
  return FP8 ? 4 * (st >> 1) + 2 * half + (st & 1) : 2 * st + half;
}
// A key's 32 lanes added up, for two tiles: entry i of lane (half, row) is that of key 8 (i / 4) + 4 half + i % 4; the lane
// with lane & 15 = i gets the sum of that key, of the odd tile where lane & 16.
__device__ __forceinline__ float column_sum32(const float (&even)[16], const float (&odd)[16], int lane) {
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {   // the odd 16 lanes of the one against the even ones of the other
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(even[i]), __float_as_uint(odd[i]), false, false);
    float x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    x += dpp_f32<kDppXor1>(x);
    x += dpp_f32<kDppXor2>(x);
    x += dpp_f32<kDppRowHalfMirror>(x);
    x += dpp_f32<kDppRowMirror>(x);
    v = (lane & 15) == i ? x : v;
  }
  return v;
}
// which 16-byte chunk of a row of q goes with step st of 16x16x32 products
template <bool FP8>
__device__ __forceinline__ int q_chunk(int st, int quarter) {
  return FP8 ? 8 * (st >> 1) + 2 * quarter + (st & 1) : 4 * st + quarter;
}

// r / G for r < 256, with magic = 2^16 / G + 1
__device__ __forceinline__ int near_token(int r, uint32_t magic) { return (int)(__umul24((uint32_t)r, magic) >> 16); }

template <Cap CAP>
struct Weight {   // exp(z - lse) of a score q.k
  float c, half_cap, cap2;
  __device__ __forceinline__ Weight(const AttnArgs& a, float ks)
      : c(CAP ? 2.f * kLog2e * a.scale * ks / a.softcap : a.scale * kLog2e * ks),
        half_cap(0.5f * a.softcap),
        cap2(a.softcap * kLog2e) {}
  __device__ __forceinline__ float operator()(float dot, float l2) const {
    return __builtin_amdgcn_exp2f(CAP ? capped<CAP == kCapLarge>(dot * c, half_cap, cap2) - l2
                                      : __builtin_fmaf(dot, c, -l2));
  }
};

// 16 bytes per lane to LDS address `lds` + 16 * lane, from base + off, or from an address of its own (in asm: the compiler
// would wait for it before any later LDS read)
__device__ __forceinline__ void load_lds16_at(uint32_t lds, const void* p) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(uni((int)lds)), "v"(p) : "memory");
}
__device__ __forceinline__ void load_lds16_near(uint32_t lds, uint32_t off, const void* base) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(uni((int)lds)), "v"(off), "s"(uni((long)base))
               : "memory");
}

template <int D, bool FP8, Cap CAP>
struct Usage {
  static constexpr int kWaves = 4, kThreads = 64 * kWaves;
  static constexpr int KPW = D == 256 ? 32 : 64;    // keys of a wave: 64 registers of them (32 for D = 64)
  static constexpr int ROWS = D == 256 ? 64 : 128;  // rows of a tile
  static constexpr int KB = KPW * kWaves, AT = KPW / 32;
  static constexpr int STEPS = D / 16;
  static constexpr int CH = D / 8;                              // 16-byte chunks of a row of q
  static constexpr int RPL = 64 / CH;                           // rows of a wave's load (1 KB)
  static constexpr int LOADS = ROWS / RPL / kWaves;       // of a wave for a tile
  // What a segment costs besides its rows, in rows (its keys, their sums)
  static constexpr int kSegCost = 256;
  static constexpr int LDS = 2 * ROWS * D * 2;
};

template <int D, bool FP8, Cap CAP>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
kv_usage_kernel(const UsageArgs args, const uint64_t magic, const uint32_t magic_near, const int parts_max,
                float* __restrict__ partials, UsageDesc* __restrict__ descs) {
  using C = Usage<D, FP8, CAP>;
  const AttnArgs& a = args.a;
  extern __shared__ __attribute__((aligned(1024))) uint16_t qs[];   // two tiles
  __shared__ float row_l2[2][C::ROWS], row_fix[2][C::ROWS];
  __shared__ long scan_sum[C::kWaves];
  __shared__ Place found;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  // -------- which part of the line of segments is this workgroup's
  auto cost = [&](const SeqBlocks& t) { return t.cost(t.MB, C::KB, a.G, C::kSegCost) * a.Hkv; };
  const Line line = lay_line(a, C::KB, cost, scan_sum);
  const long total = line.total;
  const int parts = (int)min((long)parts_max, (total + C::kSegCost - 1) / C::kSegCost);
  const int w = xcd_tile((int)blockIdx.x, parts);   // consecutive parts on one XCD: neighbouring keys, the same rows
  // no segment begins in these parts until one is written below
  if (blockIdx.x == 0)
    for (int i = parts + tid; i < parts_max; i += C::kThreads) descs[i] = UsageDesc{0, 0, 0, 0, 0, 0};
  if (w >= 0 && tid == 0) descs[w] = UsageDesc{0, 0, 0, 0, 0, 0};
  if (w < 0 || w >= parts) return;
  const Parts split(total, parts);
  long u = split.begin(w);
  const long u_end = split.begin(w + 1);
  Place at;
  SeqBlocks seq;
  if (a.S <= 64) {
    at = place_few(line, u, seq);
  } else {
    place_many(a, line, C::KB, cost, u, &found);
    __syncthreads();
    at = {uni(found.s), uni(found.rem)};
    seq = uniform(seq_blocks(a, at.s, C::KB));
  }
  int s = at.s;
  long rem = at.rem;
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
  const uint32_t qs_off = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)qs;
  // chunk c of row r sits at c ^ swizzle(r): 16 rows' same chunk on different banks (D = 64: two rows span the 64 banks)
  auto swizzle = [](int r) { return D == 64 ? (r >> 1) & 7 : r & 15; };
  // bytes between a token's last row and the next token's first: 32-bit offsets within a tile where they are few
  const bool near_rows = a.q_stride - (size_t)a.G * D < 1u << 22;
  const uint32_t gap = (uint32_t)(a.q_stride - (size_t)a.G * D) * 2;
  // Of two waves on a SIMD the older one is served first, and the younger one's part would end last by a third: the workgroups
  // that come second go ahead instead (a prompt's last 64 tokens 38.5 -> 35.6 us, two prompts of 4096 127 -> 123).
  if (blockIdx.x >= kUsageParts / 2) __builtin_amdgcn_s_setprio(1);
  int buf = 0;
  while (u < u_end) {
    // -------- the segment: its rows, and this part's share of their tiles (the fixed cost comes first; a part whose share
    // of the front is no tile leaves the segment to the next one, which then begins it)
    const int k0 = kb * C::KB;
    const int i0 = seq.first(kb, C::KB);
    const int rows = (seq.n - i0) * a.G, r0 = i0 * a.G, r_end = seq.n * a.G;
    const long seg_end = u - rem + rows + C::kSegCost;
    const bool ends = seg_end <= u_end;
    const int ntiles = (rows + C::ROWS - 1) / C::ROWS;
    const int t0 = (int)(max(rem - C::kSegCost, 0l) / C::ROWS);
    const int t1 = ends ? ntiles : (int)(max(rem + u_end - u - C::kSegCost, 0l) / C::ROWS);
    const bool begins = ntiles > 0 ? t0 == 0 : rem == 0;
    if (ntiles > 0 ? t1 > 0 : begins) {
      const Weight<CAP> weight(a, FP8 ? a.k_scale[h] : 1.f);
      // -------- rows of tile t to LDS, and their lse, which one wave takes at a time
      const uint16_t* const qh = a.q + (size_t)seq.row0 * a.q_stride + (size_t)h * a.G * D;
      auto token_of = [&](int r) { return (int)((uint64_t)r * magic >> 40); };   // r / G
      float ahead = INFINITY;   // the lse of one of the next tile's rows, in the waves whose turn it is
      auto fetch = [&](int t, int b) {
        const int first = r0 + t * C::ROWS, tok0 = uni(token_of(first)), last = min(C::ROWS, r_end - first) - 1;
        const uint16_t* const q0 = qh + (size_t)tok0 * a.q_stride;
        const int lead = first - tok0 * a.G;   // rows of its first token before the tile
        auto loads = [&](auto near) {
#pragma unroll
          for (int y = 0; y < C::LOADS; ++y) {
            const int x = y * C::kWaves + wave;   // (rows past the last repeat it)
            const int at = x * C::RPL + lane / C::CH, r = lead + min(at, last), tok = near_token(r, magic_near);
            const uint32_t lds = qs_off + b * (C::ROWS * D * 2) + x * 1024, chunk = ((lane % C::CH) ^ swizzle(at)) * 16;
            if (near) load_lds16_near(lds, __umul24(tok, gap) + r * (2 * D) + chunk, q0);
            else load_lds16_at(lds, reinterpret_cast<const uint8_t*>(q0 + tok * (a.q_stride - a.G * D) + r * D) + chunk);
          }
        };
        if (near_rows) loads(std::true_type{});
        else loads(std::false_type{});
        if (tid / C::ROWS == t % (C::kThreads / C::ROWS)) {
          const int r = lead + min(tid & (C::ROWS - 1), last), tok = near_token(r, magic_near);
          ahead = args.lse[(size_t)(seq.row0 + tok0 + tok) * a.Hq + h * a.G + r - tok * a.G];
        }
      };
      auto put_lse = [&](int t, int b) {   // (not in fetch: a use of what it loads would wait for the rows as well)
        if (tid / C::ROWS != t % (C::kThreads / C::ROWS)) return;
        const int at = tid & (C::ROWS - 1);
        const RowLse f = row_lse_of(r0 + t * C::ROWS + at < r_end ? ahead : INFINITY);
        row_l2[b][at] = f.l2;
        row_fix[b][at] = f.fix;
      };
      if (t0 < t1) fetch(t0, buf);
      // -------- this wave's keys: 16 of them lie in one page; those past the end and of pages outside the pool are read
      // from page 0 (every key has sums of its own, and theirs are dropped)
      const int wk = k0 + wave * C::KPW;
      const int my_key = wk + 16 * (lane & (2 * C::AT - 1));
      int id = my_key < seq.kv ? a.block_table[(size_t)s * a.max_pages + (my_key >> a.page_shift)] : -1;
      const uint32_t pages_ok = (uint32_t)__ballot(id >= 0 && id < a.num_pages) & ((1u << 2 * C::AT) - 1);
      if (id < 0 || id >= a.num_pages) id = 0;
      const uint8_t* const kc = static_cast<const uint8_t*>(a.k_cache) + ((size_t)h << a.page_shift) * (FP8 ? D : 2 * D);
      auto rows_of = [&](int i) {   // of the 16 keys from wk + 16 i on
        return kc + (size_t)__builtin_amdgcn_readlane(id, i) * page_bytes +
               (size_t)((wk + 16 * i) & page_mask) * (FP8 ? D : 2 * D);
      };
      bf16x8 k[C::AT][C::STEPS];
      if (t0 < t1) {
#pragma unroll
        for (int t = 0; t < C::AT; ++t) load_keys32<D, FP8>(rows_of(2 * t), rows_of(2 * t + 1), lane, k[t]);
      }
      if (t0 < t1) put_lse(t0, buf);
      // the keys are here before the loop: a wait for them inside would wait for the next tile's rows as well
#pragma unroll
      for (int t = 0; t < C::AT; ++t)
#pragma unroll
        for (int st = 0; st < C::STEPS; ++st) asm volatile("" ::"v"(__builtin_bit_cast(i32x4, k[t][st])));
      float sum[C::AT][16];
#pragma unroll
      for (int t = 0; t < C::AT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[t][e] = 0.f;
      // tile t is there, and the other buffer's rows have been read
      auto arrive = [&](int t) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (t + 1 < t1) fetch(t + 1, buf ^ 1);
      };
      auto leave = [&](int t) {
        buf ^= 1;
        if (t + 1 < t1) put_lse(t + 1, buf);
      };
      auto step = [&](int t, auto masked) {
        arrive(t);
        const int first = r0 + t * C::ROWS, groups = (min(C::ROWS, r_end - first) + 31) >> 5;
        const uint16_t* const rows_q = qs + buf * (C::ROWS * D);
        bf16x8 q[C::STEPS];
        float l2 = 0.f, fix = 0.f, next_l2, next_fix;
        auto read = [&](int g, int st) {
          const int r = 32 * g + col;
          q[st] = *reinterpret_cast<const bf16x8*>(&rows_q[r * D + (q_chunk32<FP8>(st, half) ^ swizzle(r)) * 8]);
        };
        auto read_lse = [&](int g) {
          next_l2 = row_l2[buf][32 * g + col];
          next_fix = row_fix[buf][32 * g + col];
        };
        v16f z[2];
        // A stage: the weights of 32 keys and 32 rows beside the products of the next 32 keys, or of the next rows' first
        // ones; a group's last products hand their operands' registers to the next group's rows as they go.
        auto group = [&](int g, auto last) {
          // (rows past the last add nothing: their lse is infinite)
          const int lim =
              masked ? max(seq.all, seq.ctx + token_of(min(first + 32 * g + col, r_end - 1))) + 1 - wk - 4 * half : 0;
          l2 = next_l2;
          fix = next_fix;
#pragma unroll
          for (int i = 0; i < C::AT; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const bool hand_over = !last && i + 2 == C::AT;
            const bool products = C::AT > 1 && (i + 1 < C::AT || !last);   // (one tile: nothing to stand beside)
            const int next = (i + 1) % C::AT;
            if (products) {
              z[next & 1] = v16f{};
#pragma unroll
              for (int st = 0; st < C::STEPS; ++st) {
                z[next & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[next][st], q[st], z[next & 1], 0, 0, 0);
                if (hand_over) read(g + 1, st);
              }
              if (hand_over) read_lse(g + 1);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p = weight(z[i & 1][e], l2);
              if (masked) p = 32 * i + 8 * (e / 4) + e % 4 < lim ? p : 0.f;
              sum[i][e] = __builtin_fmaf(p, fix, sum[i][e]);
            }
            if (products && !masked && CAP == kCapNone) {
#pragma unroll
              for (int x = 0; x < C::STEPS; ++x) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a product
                if (hand_over) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (x > 0) __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);
              }
            }
          }
        };
        auto begin = [&](int g) {
#pragma unroll
          for (int st = 0; st < C::STEPS; ++st) read(g, st);
          read_lse(g);
          z[0] = v16f{};
#pragma unroll
          for (int st = 0; st < C::STEPS; ++st)
            z[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[0][st], q[st], z[0], 0, 0, 0);
        };
        if constexpr (C::AT == 1) {
          for (int g = 0; g < groups; ++g) {
            begin(g);
            group(g, std::true_type{});
          }
        } else {
          begin(0);
          for (int g = 0; g + 1 < groups; ++g) group(g, std::false_type{});
          group(groups - 1, std::true_type{});
        }
        leave(t);
      };
      // later rows see more: tiles whose last row sees no key of this wave come first, and once a tile's first row sees every one,
      // all that follow do
      int t = t0;
      for (; t < t1 && max(seq.ctx + uni(token_of(min(r0 + (t + 1) * C::ROWS, r_end) - 1)), seq.all) < wk; ++t) {
        arrive(t);
        leave(t);
      }
      for (; t < t1 && wk + C::KPW > max(seq.ctx + uni(token_of(r0 + t * C::ROWS)), seq.all) + 1; ++t) step(t, std::true_type{});
      for (; t < t1; ++t) step(t, std::false_type{});
      const float total_weight = column_sum32(sum[0], sum[C::AT - 1], lane);   // (every lane takes part)
      if (C::AT == 2 || col < 16) {
        const int in_wave = 32 * (col >> 4) + 8 * ((col & 15) >> 2) + 4 * half + (col & 3);
        const float v = (pages_ok >> (in_wave >> 4)) & 1 ? total_weight : 0.f;
        const int at = wave * C::KPW + in_wave, j = k0 + at;
        if (begins && (ends || ntiles == 0)) {
          bool kept;
          const size_t base = usage_at(args, s, h, &kept);
          if (kept && j < seq.kv)
            args.usage[base + j] = args.prev && j < seq.ctx ? __builtin_fmaf(args.decay, args.prev[base + j], v) : v;
        } else {
          partials[(size_t)(2 * w + (begins ? 1 : 0)) * C::KB + at] = v;
        }
      }
      if (tid == 0 && begins && !(ends || ntiles == 0))
        descs[w] = UsageDesc{s, h, k0, min(C::KB, seq.kv - k0), w, split.of(seg_end - 1)};
    }

    // -------- the next segment
    u = min(u_end, seg_end);
    rem = 0;
    if (++kb >= seq.MB) {
      kb = 0;
      if (++h >= a.Hkv && u < u_end) {
        h = 0;
        if (!next_seq(a, C::KB, s, seq)) return;
      }
    }
  }
}

// Few rows per sequence and kv head (GROUPS times 16; a decoding step): every wave walks a stretch of 16-key tiles of its own,
// the rows in its registers. The stretches are equal parts of all sequences' and heads' tiles laid end to end; a
// tile is one wave's, so nothing is joined. Bound by the keys' bytes: they go to LDS in whole rows, 1 KB a load (straight to the
// operand's registers, 64 bytes of a row at a time, 64 sequences of up to 8192 tokens took 22.1 us).
template <int D, bool FP8>
struct Few {
  static constexpr int RB = D * (FP8 ? 1 : 2);                 // bytes of a key's row
  static constexpr int CPR = RB / 16;                          // its 16-byte chunks
  static constexpr int AT = RB == 512 ? 2 : 4;                 // tiles at a time
  static constexpr int LOADS = AT * 16 * RB / 1024;
  static constexpr int LDS = 4 * AT * 16 * RB;                 // of four waves
  // chunk c of row r sits at c ^ swizzle(r): 16 rows' same chunk on different banks
  static __device__ __forceinline__ int swizzle(int r) { return CPR >= 16 ? r & 15 : (CPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3); }
};
constexpr int kFewWaves = 2048;   // two on every SIMD
template <int D, bool FP8, Cap CAP, int GROUPS>
__global__ void __launch_bounds__(256, 2) kv_usage_few_kernel(const UsageArgs args, const uint32_t magic_near) {
  using F = Few<D, FP8>;
  constexpr int KB = 16, AT = F::AT, STEPS = D / 32;
  extern __shared__ __attribute__((aligned(1024))) uint8_t stages[];
  const AttnArgs& a = args.a;
  __shared__ long scan_sum[4];
  __shared__ Place found[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  auto cost = [&](const SeqBlocks& t) { return (long)t.MB * a.Hkv; };
  const Line line = lay_line(a, KB, cost, scan_sum);
  const int block = xcd_tile((int)blockIdx.x, (int)gridDim.x);
  const Parts split(line.total, 4 * (int)gridDim.x);
  if (a.S > 64) {   // the sequences in which this workgroup's waves begin
#pragma unroll
    for (int i = 0; i < 4; ++i) place_many(a, line, KB, cost, split.begin(4 * block + i), &found[i]);
    __syncthreads();
  }
  long u = split.begin(4 * block + wave);
  const long u_end = split.begin(4 * block + wave + 1);
  if (u >= u_end) return;
  Place at;
  SeqBlocks seq;
  if (a.S <= 64) {
    at = place_few(line, u, seq);
  } else {
    at = {uni(found[wave].s), uni(found[wave].rem)};
    seq = uniform(seq_blocks(a, at.s, KB));
  }
  int s = at.s, h, kb;
  h = uni((int)div_pos(at.rem, seq.MB));
  kb = uni((int)(at.rem - (long)h * seq.MB));
  const int page_mask = (1 << a.page_shift) - 1;
  const size_t page_bytes = a.page_stride * (FP8 ? 1 : 2);
  uint8_t* const mine_lds = stages + wave * (F::LDS / 4);
  const uint32_t mine_off = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)mine_lds;
  while (u < u_end) {
    // -------- one sequence and head: its rows, then its tiles, AT at a time
    const int rows = seq.n * a.G, tiles = (int)min((long)(seq.MB - kb), u_end - u);
    bf16x8 q[GROUPS][STEPS];
    RowLse row[GROUPS];
    int lim[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int r = min(16 * g + col, rows - 1), tok = near_token(r, magic_near);
      const uint16_t* p = a.q + (size_t)(seq.row0 + tok) * a.q_stride + (size_t)(h * a.G + r - tok * a.G) * D;
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
        q[g][st] = *reinterpret_cast<const bf16x8*>(p + q_chunk<FP8>(st, quarter) * 8);
      float l = args.lse[(size_t)(seq.row0 + tok) * a.Hq + h * a.G + r - tok * a.G];
      if (16 * g + col >= rows) l = INFINITY;   // adds nothing
      row[g] = row_lse_of(l);
      lim[g] = max(seq.all, seq.ctx + tok) + 1;
    }
    const Weight<CAP> weight(a, FP8 ? a.k_scale[h] : 1.f);
    const uint8_t* const kc = static_cast<const uint8_t*>(a.k_cache) + ((size_t)h << a.page_shift) * (FP8 ? D : 2 * D);
    bool kept;
    const size_t base = usage_at(args, s, h, &kept);
    const int* const table = a.block_table + (size_t)s * a.max_pages;
    int id = 0;
    for (int t = 0; t < tiles; t += AT) {
      if (t % 64 == 0) {   // page ids of 64 tiles at a time, one per lane
        const int key = (kb + t + lane) * 16;
        id = t + lane < tiles ? table[key >> a.page_shift] : -1;
      }
      const int k0 = (kb + t) * 16, here = min(AT, tiles - t);
      const uint32_t pages_ok = (uint32_t)(__ballot(id >= 0 && id < a.num_pages) >> (t % 64)) & ((1u << AT) - 1);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the last tiles have been read
#pragma unroll
      for (int x = 0; x < F::LOADS; ++x) {   // (tiles past the stretch and of pages outside the pool: page 0's, dropped)
        constexpr int kRows = 1024 / F::RB;
        const int i = x * kRows / 16, r = x * kRows % 16 + lane / F::CPR;
        const int page = (pages_ok >> i) & 1 ? __builtin_amdgcn_readlane(id, (t + i) % 64) : 0;
        const uint8_t* p = kc + (size_t)page * page_bytes + (size_t)((k0 + 16 * i) & page_mask) * F::RB;
        load_lds16_near(mine_off + x * 1024, r * F::RB + (((lane % F::CPR) ^ F::swizzle(r)) << 4), p);
      }
      const int at = 16 * (col >> 2) + 4 * quarter + (col & 3), j = k0 + at;
      const bool mine_too = kept && col < 4 * here && j < seq.kv;
      const float old = mine_too && args.prev && j < seq.ctx ? args.prev[base + j] : 0.f;
      float sum[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        bf16x8 k[STEPS];
        const uint8_t* const rows_k = mine_lds + (16 * i + col) * F::RB;
        auto chunk = [&](int c) { return *reinterpret_cast<const i32x4*>(rows_k + ((c ^ F::swizzle(col)) << 4)); };
        if constexpr (FP8) {   // 16 bytes are two steps' 8 values of this lane
#pragma unroll
          for (int st = 0; st < STEPS; st += 2) {
            const i32x4 v = chunk(2 * st + quarter);
            k[st] = bf16_of_e4m3(v[0], v[1]);
            k[st + 1] = bf16_of_e4m3(v[2], v[3]);
          }
        } else {
#pragma unroll
          for (int st = 0; st < STEPS; ++st) k[st] = __builtin_bit_cast(bf16x8, chunk(4 * st + quarter));
        }
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          v4f z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = 0; st < STEPS; ++st) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[st], q[g][st], z, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = k0 + 16 * i + 4 * quarter + e < lim[g] ? weight(z[e], row[g].l2) : 0.f;
            sum[i][e] = __builtin_fmaf(p, row[g].fix, sum[i][e]);
          }
        }
      }
      const float v = column_sum(sum, col);
      if (mine_too) args.usage[base + j] = __builtin_fmaf(args.decay, old, (pages_ok >> (col >> 2)) & 1 ? v : 0.f);
    }
    u += tiles;
    kb = 0;
    if (++h >= a.Hkv && u < u_end) {
      h = 0;
      if (!next_seq(a, KB, s, seq)) return;
    }
  }
}

// Adds the partial sums of segments that span several parts, in part order: workgroup w the one that begins in part w.
__global__ void __launch_bounds__(512) kv_usage_join_kernel(const UsageArgs args, const int KB,
                                                            const float* __restrict__ partials,
                                                            const UsageDesc* __restrict__ descs) {
  const UsageDesc d = descs[blockIdx.x];
  const int at = threadIdx.x, j = d.k0 + at;
  if (at >= d.keys) return;
  bool kept;
  const size_t base = usage_at(args, d.s, d.head, &kept);
  if (!kept) return;
  float v = partials[(size_t)(2 * d.first + 1) * KB + at];
  for (int p = d.first + 1; p <= d.last; p += 16) {   // 16 loads at a time
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = partials[(size_t)(2 * min(p + i, d.last)) * KB + at];
#pragma unroll
    for (int i = 0; i < 16; ++i) v += p + i <= d.last ? x[i] : 0.f;
  }
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
  using F = Few<D, FP8>;
  const AttnArgs& a = u.a;
  // r / G: r magic >> 40 where r < 2^20 G, r magic_near >> 16 where r < 256
  const uint64_t magic = (1ull << 40) / (uint64_t)a.G + 1;
  const uint32_t magic_near = (1u << 16) / (uint32_t)a.G + 1;
  const long rows = (long)a.max_q * a.G;
  if (rows <= 32) {
    const long tiles = (long)a.S * a.Hkv * ((((long)a.max_pages << a.page_shift) + 15) / 16);   // at most
    const int grid = (int)min((long)kFewWaves / 4, (tiles + 3) / 4);
    if (rows <= 16)
      hipLaunchKernelGGL((kv_usage_few_kernel<D, FP8, CAP, 1>), dim3(grid), dim3(256), F::LDS, stream, u, magic_near);
    else
      hipLaunchKernelGGL((kv_usage_few_kernel<D, FP8, CAP, 2>), dim3(grid), dim3(256), F::LDS, stream, u, magic_near);
    return hipGetLastError();
  }
  float* partials = static_cast<float*>(a.ws);
  UsageDesc* descs = reinterpret_cast<UsageDesc*>(partials + 2 * (size_t)kUsageParts * C::KB);
  hipLaunchKernelGGL((kv_usage_kernel<D, FP8, CAP>), dim3(kUsageParts), dim3(C::kThreads), C::LDS, stream, u, magic, magic_near,
                     kUsageParts, partials, descs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
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
