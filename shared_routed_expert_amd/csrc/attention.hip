// Attention over the paged cache on the matrix cores, for drafted trees, single tokens and
// prompt chunks alike.
//
// Rows. The query heads that share a kv head read the same keys, so a tile's rows are (token,
// head of the group) pairs: TB = M / G tokens of a sequence times its G heads, M = 32 RW rows.
// A segment is one such tile against all keys it sees. Row r of a tile sees key j when j <
// lim_r, or when j is a drafted token whose bit is set in the row's mask word; causal order, a
// prefix and a tree are all of this form.
//
// Products. Scores are taken transposed, S^T = K Q^T (32x32x16 matrix instructions): a lane then
// owns one row (its column l & 31) and 16 keys per 32x32 tile, so the running maximum and sum
// of the softmax are sums in registers plus one exchange with lane l ^ 32, and a change of the
// maximum scales O^T by one number per lane. The weights, rounded to 16 bits, are already the B
// operand of O^T += V^T P^T when the keys of a 16-key step are counted as (half h of the wave,
// j < 8) -> key 8 (j / 4) + 4 h + j % 4; V's transposing LDS reads fetch them in that order.
//   m' = max(m, max z),  O' = O 2^(m - m') + sum 2^(z - m') v,  l' = l 2^(m - m') + sum 2^(z - m')
// (z in units of log2 e). m only moves when a score exceeds it by more than 8: until then the
// weights are at most 2^8 in bf16. In float16 they are 2^7 larger, so that the row's largest is 2^7 to
// 2^15 (float16 ends below 2^16) and its subnormals, 2^-24 apart, lose at most 2^-32 of the largest weight.
//
// Keys and values go to LDS straight from global memory (16 bytes a lane), 16-byte chunks swapped
// within a row by the source address (chunk c of key k sits at c ^ swizzle(k)), so that both
// the row-wise reads of K and the transposing reads of V use all banks.
//
// Two arrangements of a workgroup's waves:
//   RW == 1 (decode, small trees): every wave walks keys of its own through its own two LDS
//     stages, with no barrier; the KW waves' sums are joined at the end of the segment.
//   KW == 1 (larger trees, prompts): RW waves with rows of their own share each key tile; two such
//     workgroups per CU, one's matrix work beside the other's vector work.
//
// Work split. The segments of all sequences, heads and row tiles are laid end to end, each as
// long as the keys it sees; workgroup w takes the w-th of equal parts of that line, so ragged
// batches and causal triangles balance without a host-side plan. A segment that spans several
// parts leaves one partial (O, m, l) per part in the workspace, joined by a second kernel in
// part order (no atomics; the same bits every time). Many segments that are all short beside a part are taken
// whole instead, one per workgroup, with nothing to join (share_for).
//
// What bounds it, measured (one call, join included). Decode: bytes; 24 sequences of up to 16384 tokens on 8 kv
// heads 151 us (0.93 GB, 6.1 TB/s), 64 of up to 8192 on one 35 us (160 MB). Prompts: the matrix cores and
// the vector unit in turn; 16384 tokens of 12 heads 838 us (983 TFLOP/s), over e4m3 860, 4096 tokens 78 us. Small
// calls: latency; one sequence of 777 tokens 13 us, 8 trees of 64 tokens over up to 4099 26 us.
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
constexpr float kMoveMax = 8.0f;    // a running maximum moves when a score exceeds it by this (base 2)
constexpr float kHalfBias = 7.0f;   // float16 weights are 2^this larger
static_assert(kMoveMax + kHalfBias <= 15.0f, "the largest weight is a finite float16");

// 16-byte chunk swap of key k's row (CPR chunks of it), for LDS's 64 banks of 4 bytes: 16 consecutive
// keys' same chunk (a step of K's reads) and the 64 or 32 bytes of {4h..4h+3} (8-bit: and 8+4h..) of a
// transposing read of V fall on different banks (rows of 128 and 64 bytes: 2 and 4 rows span the
// banks, so the low key bits need no swap).
__device__ __forceinline__ int swizzle(int k, int cpr) {
  const int low = (k >> 2) & 3;
  return cpr >= 16 ? ((k & 3) << 2) | low : (cpr == 8 ? ((k & 2) << 1) | low : low);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ float swap_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
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

// 16 bytes per lane from base + voff to LDS address `lds` + 16 * lane. In asm, because the
// compiler would wait for every such load in flight before any later LDS read; wait_vm counts them.
// kOnce: the bytes are read by this wave alone and passed through the caches as such (decode of 24
// sequences of up to 16384 tokens, 0.93 GB: 170 us without, 152 us with).
template <bool kOnce>
__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t voff, const uint8_t* base) {
  // (the LDS address goes in as m0 itself, so that the compiler knows what the register holds; a wait state after it)
  if (kOnce)
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"{m0}"(uni((int)lds)), "v"(voff), "s"(uni((long)base))
                 : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(uni((int)lds)), "v"(voff), "s"(uni((long)base))
                 : "memory");
}

// LDS reads and matrix instructions stay on their side of this; other arithmetic may cross.
__device__ __forceinline__ void fence_reads() { __builtin_amdgcn_sched_barrier(0x0006 | 0x0400); }
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

// ------------------------------------------------------------------------------- the work split
// One sequence's row tiles: tile i (of MT) sees the first vis(i) = max(lo, ctx + min(n, (i + 1) TB))
// keys (lo: what every row may see at least: its prefix, or all keys under a tree mask).
struct SeqTiles {
  int row0, n, kv, ctx, lo, MT;
  __device__ __forceinline__ int vis(int i, int TB) const { return max(lo, ctx + min(n, (i + 1) * TB)); }
  // cost of tiles 0..mt-1 of one head: vis + fixed each, in closed form (fixed: what a segment costs
  // besides its keys, in keys); 1 each where segments are taken whole (fixed < 0)
  __device__ __forceinline__ long cost(int mt, int TB, int fixed) const {
    if (fixed < 0) return mt;
    const long star = lo > ctx ? min(MT, (lo - ctx) / TB) : 0;   // the tiles with ctx + (i + 1) TB <= lo
    long f = (long)mt * fixed + min((long)mt, star) * lo;
    if (mt > star) {
      f += (mt - star) * ctx + (long)TB * (((long)mt * (mt + 1) - star * (star + 1)) / 2);
      if (mt == MT) f -= (long)ctx + (long)MT * TB - max(lo, ctx + n);
    }
    return f;
  }
};
__device__ __forceinline__ SeqTiles seq_tiles(const AttnArgs& a, int s, int TB) {
  const SeqInfo q = seq_info(a, s);
  SeqTiles t;
  t.row0 = q.row0;
  t.n = q.n;
  t.kv = q.kv;
  t.ctx = q.kv - q.tokens;
  t.lo = a.tree_mask ? q.kv : (a.prefix_lens ? min(max(a.prefix_lens[s], 0), q.kv) : 0);
  t.MT = (q.n + TB - 1) / TB;
  return t;
}

// a sequence that is the same for the whole wave, in scalar registers
__device__ __forceinline__ SeqTiles uniform(SeqTiles t) {
  t.row0 = uni(t.row0); t.n = uni(t.n); t.kv = uni(t.kv); t.ctx = uni(t.ctx); t.lo = uni(t.lo); t.MT = uni(t.MT);
  return t;
}

// How the segments are shared out: equal parts of the line, whole segments, or either by the lengths that the
// kernel finds (a launch of both: as many workgroups as there can be segments, and the join).
enum Share { kEqualParts, kWholeSegments, kByLengths };

// A segment that begins in part `first` and ends in a later part `last` (rows == 0: nothing to join)
struct alignas(32) PartDesc {
  int row0, rows, head, first, last;
};

// a / b for a >= 0, b > 0: in 32 bits where they fit (a 64-bit division costs over a hundred instructions)
__device__ __forceinline__ long div_pos(long a, long b) {
  if (((uint64_t)(a | b) >> 32) == 0) return (long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Workgroups that are resident at once with tiles of M rows, and so the most parts of the line
constexpr int parts_of(int M) { return M == 128 ? 512 : 256; }

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

// -------------------------------------------------------------------------------------- the kernel
template <int D, bool FP8, int RW, int KW, int NK, Cap CAP>
struct Attn {
  static constexpr int kWaves = RW * KW;
  static constexpr int M = 32 * RW;
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int RB = D * ES;             // bytes of a key's row
  static constexpr int CPR = RB / 16;           // its 16-byte chunks
  static constexpr int RPI = 64 / CPR;          // rows per 1 KB load
  static constexpr int TILE = NK * RB;          // bytes of a K (or V) tile
  static constexpr int NX = TILE / 1024;        // loads per tile
  static constexpr int XW = NX / RW;            // of one wave
  static constexpr int STAGE = 2 * TILE;
  static constexpr int LDS = 2 * STAGE * KW;
  static constexpr int KT = NK / 32;            // 32-key tiles of scores
  static constexpr int DT = D / 32;
  static constexpr int STEPS = D / 16;
  // bf16 weights are split in two (16 bits of them) where memory sets the pace and the second product is
  // free (decode of 64 sequences takes as long, its error is 0.0017 of the output instead of 0.0023, that of the
  // output's own rounding). Tiles of more rows round them once (64 trees of 5 tokens 42 us, split 52; a prompt of
  // 4096 tokens 77 and 97, of 16384 805 and 1143).
  static constexpr bool kSplit = !FP8 && RW == 1;
  // What a segment costs besides its keys, in keys (its q, its first tile's latency, its result: about
  // 5 us, a tile of 64 keys 1.2 to 1.7)
  static constexpr int kSegCost = RW == 1 ? 192 : 256;
  // A part's cost in keys is at least this (eight waves, 128 and 256: 20 sequences of 2 tokens over up to
  // 3000 keys 17.5 and 20 us, 20 of 3000 keys 19.4 and 16.5, one of 3000 15.3 and 14.8)
  static constexpr int kMinPart = RW == 1 ? (KW < 4 ? 64 : 128) : 4 * NK;
  static constexpr int SLOT = M * D + 2 * M;    // floats of a partial: O [M][D], then m and l per row
  // Shared tiles of D = 256: q and O^T alone are 192 of the 256 registers that two workgroups per CU leave
  // (a chunk of 8192 tokens of 8 heads: bf16 352 us, one workgroup 475; e4m3 330 and 440). LDS is then
  // read fewer products ahead and its addresses are formed anew for each tile; kept, they spill.
  static constexpr bool kTight = RW == 4 && D == 256;
  static_assert(NX % RW == 0 && RPI <= 16 && NK <= 64, "tile shape");
  static_assert(KW == 1 || M * D * 4 <= 2 * STAGE, "the waves' sums are joined in their stages");
};

template <int D, bool FP8, int RW, int KW, int NK, Cap CAP>
__global__ void __launch_bounds__(64 * RW * KW)
__attribute__((amdgpu_waves_per_eu(RW == 4 || KW == 8 ? 2 : 1, RW == 4 || KW == 8 ? 2 : 1))) attention_kernel(
    const AttnArgs a, const int TB, const int parts_max, const Share share, const int desc_tiles,
    float* __restrict__ partials, PartDesc* __restrict__ descs) {
  using C = Attn<D, FP8, RW, KW, NK, CAP>;
  constexpr int kThreads = 64 * C::kWaves;
  extern __shared__ __attribute__((aligned(1024))) uint8_t sm[];
  __shared__ long scan_sum[C::kWaves];
  __shared__ int scan_max[C::kWaves];
  __shared__ long found_rem;
  __shared__ int found_s;
  __shared__ SeqTiles found_seq;
  __shared__ float row_m[KW][C::M], row_l[KW][C::M];
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int half = lane >> 5, col = lane & 31;
  bool whole = share == kWholeSegments;
  // -------- which part of the line of segments is this workgroup's
  // Up to 64 sequences: one per lane, in every wave by itself. More: a stretch of them per thread, and
  // two barriers.
  const bool few = a.S <= 64;
  const int per = few ? 1 : (a.S + kThreads - 1) / kThreads, place = few ? lane : tid;
  const int s_lo = min(place * per, a.S), s_hi = min(s_lo + per, a.S);
  long mine = 0, segments = 0;   // this place's stretch of the line, and its segments
  int longest = 0;
  SeqTiles own{};
  for (int s = s_lo; s < s_hi; ++s) {
    own = seq_tiles(a, s, TB);
    mine += own.cost(own.MT, TB, whole ? -1 : C::kSegCost) * a.Hkv;
    if (share == kByLengths && own.MT > 0) {
      segments += (long)own.MT * a.Hkv;
      longest = max(longest, own.vis(own.MT - 1, TB) + C::kSegCost);   // the last tile sees the most
    }
  }
  // the line's length, and what lies before this place
  long total, before;
  auto scan = [&]() {
    long incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    total = read_lane(incl, 63), before = incl - mine;
    if (!few) {
      if (lane == 0) scan_sum[wave] = total;
      __syncthreads();
      total = 0;
#pragma unroll
      for (int i = 0; i < C::kWaves; ++i) {
        if (i < wave) before += scan_sum[i];
        total += scan_sum[i];
      }
      total = uni(total);
    }
  };
  scan();
  constexpr int kPartsMost = parts_of(C::M);
  if constexpr (KW == 1) {
    // Whole where no segment is longer than 5/8 of an equal part: a workgroup that takes such a one last is no more than
    // that behind. Whole and split by the longest's share of a part: 0.29 453 and 484 us (4096 tokens of 96 heads), 0.55 160
    // and 178 (200 prompts of 10 tokens behind up to 1400), 0.61 840 and 865 (one of 16384 tokens), 0.67 530 and 499 (2048
    // tokens of 96 heads beside 64 sequences of 8192), 0.89 1197 and 849 (16384 tokens behind one sequence of 24000).
    if (share == kByLengths) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) longest = max(longest, __shfl_xor(longest, d, 64));
      if (!few) {
        if (lane == 0) scan_max[wave] = longest;
        __syncthreads();   // (scan_sum has been read as well)
#pragma unroll
        for (int i = 0; i < C::kWaves; ++i) longest = max(longest, scan_max[i]);
      }
      whole = 8l * uni(longest) * kPartsMost <= 5 * total;
      if (whole) {
        mine = segments;
        scan();
      }
    }
  }
  const int fixed = whole ? -1 : C::kSegCost;
  const int parts_split = share == kByLengths ? kPartsMost : parts_max;
  const int parts = whole ? (int)min((long)parts_max, total)
                          : (int)min((long)parts_split, (total + C::kMinPart - 1) / C::kMinPart);
  // Split: consecutive parts on one XCD (they walk neighbouring keys), however many there are on all
  // XCDs alike. Whole: the last tiles of a sequence, which see the most keys, first.
  const int w = whole ? parts_max - 1 - (int)blockIdx.x : xcd_tile((int)blockIdx.x, parts);
  if (share != kWholeSegments && desc_tiles == 0) {   // no segment begins in these parts until one is written below
    if (blockIdx.x == 0)
      for (int i = (whole ? 0 : parts) + tid; i < parts_split; i += kThreads) descs[i] = PartDesc{0, 0, 0, 0, 0};
    if (!whole && w >= 0 && tid == 0) descs[w] = PartDesc{0, 0, 0, 0, 0};
  }
  if (w < 0 || w >= parts) return;
  const Parts split(total, parts);
  long u = split.begin(w);
  const long u_end = split.begin(w + 1);
  const bool here = mine > 0 && u >= before && u < before + mine;   // one place alone
  int s;
  long rem;
  SeqTiles seq;
  if (few) {
    s = __ffsll((unsigned long long)__ballot(here)) - 1;
    rem = u - read_lane(before, s);
    seq.row0 = __builtin_amdgcn_readlane(own.row0, s);
    seq.n = __builtin_amdgcn_readlane(own.n, s);
    seq.kv = __builtin_amdgcn_readlane(own.kv, s);
    seq.ctx = __builtin_amdgcn_readlane(own.ctx, s);
    seq.lo = __builtin_amdgcn_readlane(own.lo, s);
    seq.MT = __builtin_amdgcn_readlane(own.MT, s);
  } else {
    if (here) {
      long r = u - before;
      for (int i = s_lo; i < s_hi; ++i) {
        const SeqTiles t = seq_tiles(a, i, TB);
        const long cost = t.cost(t.MT, TB, fixed) * a.Hkv;
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
    s = uni(found_s);
    rem = uni(found_rem);
    seq = uniform(found_seq);
  }
  int h, mt;
  {
    const long per_head = seq.cost(seq.MT, TB, fixed);
    h = uni((int)div_pos(rem, per_head));
    rem -= h * per_head;
    int lo = 0, hi = seq.MT;   // the largest tile with cost(tile) <= rem, 64 candidates at a time
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) >> 6, at = lo + lane * step;
      const int n = __popcll(__ballot(at < hi && seq.cost(at, TB, fixed) <= rem));
      lo = uni(lo + (n - 1) * step);
      hi = uni(min(hi, lo + step));
    }
    mt = lo;
    rem -= seq.cost(mt, TB, fixed);
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)sm;
  uint8_t* const stages = sm + kw * 2 * C::STAGE;
  const uint32_t stages_off = lds0 + kw * 2 * C::STAGE;
  const int page_mask = (1 << a.page_shift) - 1;
  const size_t page_bytes = a.page_stride * C::ES;
  const float scale2 = a.scale * kLog2e;
  constexpr float kBias = FP8 ? kHalfBias : 0.0f;

  // -------- this wave's LDS read addresses (see the layout above)
  int k_addr, v_addr, v_addr2;
  {
    k_addr = col * C::RB + ((half ^ swizzle(col, C::CPR)) << 4);
    const int dh = (lane >> 4) & 1, i = lane & 15;
    if (FP8) {
      const int r = i >> 1, key = 4 * half + (r & 3) + 8 * (r >> 2);
      v_addr = key * C::RB + ((dh ^ swizzle(key, C::CPR)) << 4) + 8 * (i & 1);
      v_addr2 = 0;
    } else {
      const int key = 4 * half + (i >> 2), c = 2 * dh + ((i & 3) >> 1);
      v_addr = key * C::RB + ((c ^ swizzle(key, C::CPR)) << 4) + 8 * (i & 1);
      v_addr2 = (key + 8) * C::RB + ((c ^ swizzle(key + 8, C::CPR)) << 4) + 8 * (i & 1);
    }
  }

  while (u < u_end) {
    // -------- the segment: rows, keys, and this part's share of its tiles
    const int vis = seq.vis(mt, TB);
    const long seg_cost = whole ? 1 : vis + C::kSegCost;
    const long seg_end = u - rem + seg_cost;
    const bool ends = seg_end <= u_end;
    const int ntiles = (vis + NK - 1) / NK;
    // The fixed cost comes first: the part in which a segment begins takes that much fewer keys. The part
    // after a border starts where the part before it stops. A part whose share of the front is no tile
    // leaves the segment to the next one, which then begins it; no tile at all (nothing is seen) belongs
    // to its first unit.
    const int t0 = (int)(max(rem - C::kSegCost, 0l) / NK);
    const int t1 = ends ? ntiles : (int)(max(rem + u_end - u - C::kSegCost, 0l) / NK);
    const bool begins = ntiles > 0 ? t0 == 0 : rem == 0;
    const bool mine_too = ntiles > 0 ? t1 > 0 : begins;
    if (mine_too) {
    const int tok0 = mt * TB, rows = min(TB, seq.n - tok0) * a.G;
    const int row0 = seq.row0 + tok0;
    const float ks = FP8 ? a.k_scale[h] : 1.f, vs = FP8 ? a.v_scale[h] : 1.f;
    // Not 0 where scale * ks underflows: a masked score of -inf times 0 would be NaN. The smallest float32 instead moves
    // a score by less than 2^-21 whatever q.k is.
    const float c = CAP ? 2.f * kLog2e * a.scale * ks / a.softcap : fmaxf(scale2 * ks, 0x1p-149f);
    const float cap2 = a.softcap * kLog2e, half_cap = 0.5f * a.softcap;
    const int* table = a.block_table + (size_t)s * a.max_pages;
    const int pages_used = (seq.kv + page_mask) >> a.page_shift;
    const uint8_t* const kc = static_cast<const uint8_t*>(a.k_cache) + ((size_t)h << a.page_shift) * C::RB;
    const uint8_t* const vc = static_cast<const uint8_t*>(a.v_cache) + ((size_t)h << a.page_shift) * C::RB;

    // this wave's tiles: all of the part's (shared), or a stretch of its own
    const int wt0 = RW == 1 ? t0 + (int)((long)(t1 - t0) * kw / KW) : t0;
    const int wt1 = RW == 1 ? t0 + (int)((long)(t1 - t0) * (kw + 1) / KW) : t1;

    // -------- page ids: 64 at a time, one per lane; pages outside the pool (and past the last
    // cached token) are read as page 0 and masked
    int pg = 0, pg_base = -64;
    bool careful = false;   // a page outside the pool was met
    auto fetch_ids = [&](int first) { return first + lane < pages_used ? table[first + lane] : 0; };
    auto take_ids = [&](int first, int id) {
      pg_base = first;
      const bool bad = id < 0 || id >= a.num_pages;
      careful = careful || __ballot(bad) != 0;
      pg = bad ? 0 : id;
    };
    auto group_offset = [&](int key) -> size_t {   // of rows key .. key + 15 in kc and vc
      const int id = __builtin_amdgcn_readlane(pg, (key >> a.page_shift) - pg_base);
      return (size_t)id * page_bytes + (size_t)(key & page_mask) * C::RB;
    };
    // a tile's keys lie in pages [key0 >> shift, (key0 + NK - 1) >> shift]: at most 4 of them
    auto pages_for = [&](int key0) {
      const int i = key0 >> a.page_shift;
      if (i + (NK - 1) / 16 >= pg_base + 64) take_ids(i, fetch_ids(i));
    };
    auto issue = [&](const uint8_t* cache, uint32_t lds, int key0) {
#pragma unroll
      for (int y = 0; y < C::XW; ++y) {
        const int x = rw * C::XW + y;
        const int row = x * C::RPI;
        const uint8_t* base = cache + group_offset(key0 + (row & ~15)) + (row & 15) * C::RB;
        const int lr = lane / C::CPR;
        const uint32_t voff = lr * C::RB + (((lane % C::CPR) ^ swizzle(row + lr, C::CPR)) << 4);
        load_lds16<RW == 1>(lds + x * 1024, voff, base);
      }
    };
    // is the 16-key group that holds `key` in a page of the pool
    auto group_ok = [&](int key) -> bool {
      if (key >= seq.kv) return false;
      const int id = table[key >> a.page_shift];
      return id >= 0 && id < a.num_pages;
    };
    // V rows that no cached token stands behind may hold anything: zero, since 0 * NaN is NaN
    auto zero_rows = [&](uint8_t* v, int key0) {
#pragma unroll
      for (int y = 0; y < C::XW; ++y) {
        const int x = rw * C::XW + y;
        const int key = key0 + x * C::RPI + lane / C::CPR;
        if (key >= seq.kv || (careful && !group_ok(key)))
          *reinterpret_cast<uint4*>(v + x * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
    };

    const int first_page = wt0 * NK >> a.page_shift;
    const int first_ids = fetch_ids(first_page);
    bf16x8 q[C::STEPS];
    int lim;
    uint64_t word;
    // rows past the tile's last repeat it and are not stored
    const int r = min(rw * 32 + col, rows - 1);
    const int tok = r / a.G, qrow = row0 + tok;
    const uint16_t* p = a.q + (size_t)qrow * a.q_stride + (size_t)(h * a.G + r - tok * a.G) * D;
#pragma unroll
    for (int st = 0; st < C::STEPS; ++st) {
      const int d = FP8 ? 32 * (st >> 1) + 16 * half + 8 * (st & 1) : 16 * st + 8 * half;
      q[st] = *reinterpret_cast<const bf16x8*>(p + d);
    }
    if (a.tree_mask) {
      lim = max(seq.ctx, 0);
      word = a.tree_mask[qrow] & (~0ull >> (64 - min(seq.kv - seq.ctx, 64)));
    } else {
      lim = max(seq.lo, seq.ctx + tok0 + tok + 1);
      word = 0;
    }
    take_ids(first_page, first_ids);
    // q is here before the key loop: a wait for it inside would wait for the tiles in flight too
    auto wait_q = [&]() {
#pragma unroll
      for (int st = 0; st < C::STEPS; ++st) asm volatile("" ::"v"(__builtin_bit_cast(i32x4, q[st])));
    };
    // keys below this are seen by every row
    const int all_see = a.tree_mask ? max(seq.ctx, 0) : max(seq.lo, seq.ctx + tok0 + 1);

    v16f o[C::DT];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < C::DT; ++d) o[d] = v16f{};

    // -------- scores of one key tile. Each product's operand is read from LDS kAhead products
    // earlier, and the fences keep that order: left alone, the compiler reads right before use and every
    // product waits for its own read.
    v16f sc[C::KT];
    auto scores = [&](const uint8_t* kt_lds) {
#pragma unroll
      for (int t = 0; t < C::KT; ++t) sc[t] = v16f{};
      constexpr int kReads = C::KT * C::STEPS / (FP8 ? 2 : 1);   // 16 bytes: one step of bf16, two of e4m3
      constexpr int kAhead = C::kTight ? (FP8 ? 2 : 3) : (FP8 ? 3 : 6);
      i32x4 raw[kReads];
      auto read = [&](int i) {
        const int t = i % C::KT, st = i / C::KT;
        raw[i] = *reinterpret_cast<const i32x4*>(kt_lds + t * 32 * C::RB + (k_addr ^ (st * 32)));
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) read(i);
      fence_reads();
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        if (i + kAhead < kReads) read(i + kAhead);
        fence_reads();
        const int t = i % C::KT, st = i / C::KT;
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bf16x8 k = bf16_of_e4m3(raw[i][2 * e], raw[i][2 * e + 1]);
            sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[2 * st + e], sc[t], 0, 0, 0);
          }
        } else {
          const bf16x8 k = __builtin_bit_cast(bf16x8, raw[i]);
          sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[st], sc[t], 0, 0, 0);
        }
        fence_reads();
      }
    };

    // -------- the softmax step in four pieces: caps and masks, the rows' maxima, a moved maximum, and
    // the weights as the next product's operand
    bf16x8 pb[NK / 16], pl[NK / 16];
    f16x8 pf[NK / 16];
    auto mask = [&](int key0) {
      if constexpr (CAP != kCapNone) {
#pragma unroll
        for (int t = 0; t < C::KT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[t][i] = capped<CAP == kCapLarge>(sc[t][i] * c, half_cap, cap2);
      }
      if (key0 + NK <= all_see && !careful) return;
      // bit k: key0 + k is seen
      const int n = lim - key0;
      uint64_t see = n >= 64 ? ~0ull : (n <= 0 ? 0ull : ~0ull >> (64 - n));
      if (a.tree_mask) {
        const int b = key0 - seq.ctx;   // the first key's bit
        see |= b >= 64 || b <= -64 ? 0ull : (b >= 0 ? word >> b : word << -b);
      }
      if (careful) {
#pragma unroll
        for (int g = 0; g < NK / 16; ++g)
          if (!group_ok(key0 + 16 * g)) see &= ~(0xFFFFull << (16 * g));
      }
      see >>= 4 * half;
#pragma unroll
      for (int t = 0; t < C::KT; ++t) {
        const uint32_t bits = (uint32_t)(see >> (32 * t));
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = (bits >> (8 * (i / 4) + i % 4)) & 1 ? sc[t][i] : -INFINITY;
      }
    };
    float mx;   // the row's largest score of the tile, in units of log2 e
    auto maxima = [&]() {
      float v = sc[0][0];
#pragma unroll
      for (int t = 0; t < C::KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) v = fmaxf(v, sc[t][i]);
      v = swap_max(v);
      mx = (CAP ? v : v * c) - kBias;
    };
    auto move_max = [&]() {
      if (!__any(mx > m + kMoveMax)) return;
      const float mn = fmaxf(m, mx);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    };
    auto weights = [&]() {
      const float ms = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < C::KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(CAP ? sc[t][i] - ms : __builtin_fmaf(sc[t][i], c, -ms));
          sum += p;
          if constexpr (FP8) {
            pf[2 * t + i / 8][i % 8] = (_Float16)p;
          } else {
            pb[2 * t + i / 8][i % 8] = (__bf16)p;
            if constexpr (C::kSplit) pl[2 * t + i / 8][i % 8] = (__bf16)(p - (float)(__bf16)p);
          }
        }
      l += sum;
    };

    auto values = [&](const uint8_t* v) {
      constexpr int kReads = NK / 16 * C::DT;
      constexpr int kAhead = C::kTight ? 2 : 4;
      i32x4 raw[kReads];
      auto read = [&](int i) {
        const int st = i / C::DT, d = i % C::DT;
        if constexpr (FP8) {
          const i32x2 r = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2*)(v + st * 16 * C::RB + (v_addr ^ (32 * d))));
          raw[i][0] = r[0];
          raw[i][1] = r[1];
        } else {
          const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(v + st * 16 * C::RB + (v_addr ^ (64 * d)))));
          const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(v + st * 16 * C::RB + (v_addr2 ^ (64 * d)))));
          raw[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) read(i);
      fence_reads();
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        if (i + kAhead < kReads) read(i + kAhead);
        fence_reads();
        const int st = i / C::DT, d = i % C::DT;
        const bf16x8 vb = __builtin_bit_cast(bf16x8, raw[i]);
        if constexpr (FP8)
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f16_of_e4m3(raw[i][0], raw[i][1]), pf[st], o[d], 0, 0, 0);
        else
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb, pb[st], o[d], 0, 0, 0);
        if constexpr (C::kSplit) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb, pl[st], o[d], 0, 0, 0);
        fence_reads();
      }
    };

    // -------- the key loop
    if constexpr (RW == 1) {
      // this wave's own tiles; two stages in flight. Loads are issued in the order K0 V0 K1 V1 | K2
      // (after the scores of tile 0) V2 (after its values) ..., so with L = NX loads per tile the
      // ones younger than K_t are V_t K_t+1 V_t+1, and those younger than V_t K_t+1 V_t+1 K_t+2
      constexpr int L = C::NX;
      for (int t = wt0; t < min(wt0 + 2, wt1); ++t) {
        const uint32_t st = stages_off + ((t - wt0) & 1) * C::STAGE;
        pages_for(t * NK);
        issue(kc, st, t * NK);
        issue(vc, st + C::TILE, t * NK);
      }
      wait_q();
      for (int t = wt0; t < wt1; ++t) {
        const int b = (t - wt0) & 1, left = wt1 - 1 - t;
        uint8_t* const st = stages + b * C::STAGE;
        const uint32_t st_off = stages_off + b * C::STAGE;
        if (left == 0) wait_vm<L>();
        else wait_vm<3 * L>();
        scores(st);
        if (left >= 2) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // K_t has been read
          pages_for((t + 2) * NK);
          issue(kc, st_off, (t + 2) * NK);
        }
        mask(t * NK);
        maxima();
        move_max();
        weights();
        if (left == 0) wait_vm<0>();
        else if (left == 1) wait_vm<2 * L>();
        else wait_vm<3 * L>();
        if ((t + 1) * NK > seq.kv || careful) {
          zero_rows(st + C::TILE, t * NK);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        values(st + C::TILE);
        if (left >= 2) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // V_t has been read
          issue(vc, st_off + C::TILE, (t + 2) * NK);
        }
      }
    } else {
      // the waves share a tile: loaded one tile ahead into the other stage, one barrier per tile.
      // Matrix work goes ahead of the other workgroup's vector work (16384 tokens over e4m3: 864 -> 843 us).
      // bf16: the odd wave slot of a SIMD (hardware id, low bit) ahead of the even one as well, since two that
      // share the matrix core in turn also end together and then want the vector unit together (a prompt of
      // 4096 tokens 84 -> 81 us, of 96 heads 474 -> 460, 16384 tokens at D = 64 370 -> 355; over e4m3,
      // where conversions keep the vector unit busy, 867 -> 883).
      const bool ahead = !FP8 && (__builtin_amdgcn_s_getreg(4 | 3 << 11) & 1);
      auto matrix_work = [&]() {
        if (ahead) __builtin_amdgcn_s_setprio(3);
        else __builtin_amdgcn_s_setprio(1);
      };
      if (t0 < t1) {
        pages_for(t0 * NK);
        issue(kc, stages_off, t0 * NK);
        issue(vc, stages_off + C::TILE, t0 * NK);
      }
      wait_q();
      for (int t = t0; t < t1; ++t) {
        const int b = (t - t0) & 1;
        uint8_t* const st = stages + b * C::STAGE;
        if constexpr (C::kTight) asm volatile("" : "+v"(k_addr), "+v"(v_addr), "+v"(v_addr2));
        wait_vm<0>();
        if ((t + 1) * NK > seq.kv || careful) zero_rows(st + C::TILE, t * NK);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (t + 1 < t1) {
          const uint32_t nx = stages_off + (b ^ 1) * C::STAGE;
          pages_for((t + 1) * NK);
          issue(kc, nx, (t + 1) * NK);
          issue(vc, nx + C::TILE, (t + 1) * NK);
        }
        matrix_work();
        scores(st);
        __builtin_amdgcn_s_setprio(0);
        mask(t * NK);
        maxima();
        move_max();
        weights();
        matrix_work();
        values(st + C::TILE);
        __builtin_amdgcn_s_setprio(0);
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // before the stages are filled again
    }

    // -------- the segment's result, or this part's partial (a sum of 0: the row sees nothing; a NaN in
    // q leaves a NaN sum, and NaN is what the row gets)
    const bool complete = begins && (ends || ntiles == 0);
    float* const slot = partials + (size_t)(2 * w + (begins ? 1 : 0)) * C::SLOT;
    if constexpr (KW == 1) {
      const int r = rw * 32 + col;
      const float sum = swap_sum(l);
      if (r < rows) {
        if (complete) {
          const int tok = r / a.G, head = h * a.G + r - tok * a.G;
          const size_t at = (size_t)(row0 + tok) * a.Hq + head;
          const float f = sum != 0.f ? vs / sum : 0.f;
#pragma unroll
          for (int d = 0; d < C::DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint2*>(a.out + at * D + 32 * d + 8 * i + 4 * half) =
                  make_uint2(pack_bf16x2(o[d][4 * i] * f, o[d][4 * i + 1] * f),
                             pack_bf16x2(o[d][4 * i + 2] * f, o[d][4 * i + 3] * f));
          if (a.lse && half == 0) a.lse[at] = sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
        } else {
#pragma unroll
          for (int d = 0; d < C::DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(slot + (size_t)r * D + 32 * d + 8 * i + 4 * half) =
                  make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
          if (half == 0) {
            slot[C::M * D + r] = m;
            slot[C::M * D + C::M + r] = sum;
          }
        }
      }
    } else {
      // every wave's O, [row][D] float32 with chunks swapped by row, in its own stages
      const float sum = swap_sum(l);
      if (half == 0) {
        row_m[kw][col] = m;
        row_l[kw][col] = sum;
      }
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int chunk = (8 * d + 2 * i + half) ^ (col & 15);
          *reinterpret_cast<float4*>(stages + col * D * 4 + chunk * 16) =
              make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
        }
      __syncthreads();
      for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c4 = i % (D / 4);
        float top = row_m[0][r];
#pragma unroll
        for (int k = 1; k < KW; ++k) top = fmaxf(top, row_m[k][r]);
        float sum = 0.f, v0 = 0.f, v1 = 0.f, v2 = 0.f, v3 = 0.f;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(row_m[k][r] - top);
          const float4 v = *reinterpret_cast<const float4*>(sm + k * 2 * C::STAGE + r * D * 4 + ((c4 ^ (r & 15)) * 16));
          sum += f * row_l[k][r];
          v0 += f * v.x; v1 += f * v.y; v2 += f * v.z; v3 += f * v.w;
        }
        if (complete) {
          const int tok = r / a.G, head = h * a.G + r - tok * a.G;
          const size_t at = (size_t)(row0 + tok) * a.Hq + head;
          const float f = sum != 0.f ? vs / sum : 0.f;
          *reinterpret_cast<uint2*>(a.out + at * D + 4 * c4) =
              make_uint2(pack_bf16x2(v0 * f, v1 * f), pack_bf16x2(v2 * f, v3 * f));
          if (a.lse && c4 == 0) a.lse[at] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(slot + (size_t)r * D + 4 * c4) = make_float4(v0, v1, v2, v3);
          if (c4 == 0) {
            slot[C::M * D + r] = top;
            slot[C::M * D + C::M + r] = sum;
          }
        }
      }
      __syncthreads();   // the stages are free again
    }
    if (begins && tid == 0 && !whole) {
      if (desc_tiles > 0)
        descs[((size_t)s * a.Hkv + h) * desc_tiles + mt] =
            PartDesc{row0, complete ? 0 : rows, h, w, complete ? w : split.of(seg_end - 1)};
      else if (!complete)
        descs[w] = PartDesc{row0, rows, h, w, split.of(seg_end - 1)};
    }
    }

    // -------- the next segment
    u = min(u_end, seg_end);
    rem = 0;
    if (++mt >= seq.MT) {
      mt = 0;
      if (++h >= a.Hkv && u < u_end) {
        h = 0;
        do seq = uniform(seq_tiles(a, ++s, TB));
        while (seq.n == 0);
      }
    }
  }
}

// Joins the partials of segments that span several parts: workgroup (i, y) takes rows of the
// segment of description i. There is one description per segment, or, where that would be many, one per
// part for the segment that begins in it and goes on. D / 4 lanes read a partial's row (16 bytes
// each); the workgroup's groups of such lanes stand side by side on `side` partials of a row (few
// partials: on rows of their own), and each has kBatch of them in flight, so that neither a segment
// split over the whole card nor 128 rows of two partials each wait for memory more than a few times.
// Bound by a launch and its tail (64 sequences, 3 MB: 4.6 us), then bytes (one prompt of 4096 tokens, 59 MB: 11.8
// us, 5.0 TB/s).
constexpr int kJoinThreads = 256;
template <int D, int kBatch>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const int M, const PartDesc& d, const int side,
                                          const float* __restrict__ partials, float4* acc, float* acc_l, float* acc_m) {
  constexpr int LPR = D / 4;
  constexpr int kGroups = kJoinThreads / LPR;
  const int w = d.first, count = d.last - w + 1;
  const int rows_at_once = kGroups / side;
  const size_t slot = (size_t)M * D + 2 * M;
  const int c4 = threadIdx.x % LPR, g = threadIdx.x / LPR, p0 = g % side;
  const float vs = a.v_scale ? a.v_scale[d.head] : 1.f;
  for (int base = blockIdx.y * rows_at_once; base < d.rows; base += gridDim.y * rows_at_once) {
    const int r = min(base + g / side, d.rows - 1);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = p0; p < count; p += kBatch * side) {
      float pm[kBatch], pl[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = w + min(p + i * side, count - 1);
        const float* s = partials + (size_t)(at == w ? 2 * w + 1 : 2 * at) * slot;
        pm[i] = s[(size_t)M * D + r];
        pl[i] = p + i * side < count ? s[(size_t)M * D + M + r] : 0.f;
        v[i] = *reinterpret_cast<const float4*>(s + (size_t)r * D + 4 * c4);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (pl[i] != 0.f) {   // an empty partial says nothing, one of NaN makes the row NaN
          const float mn = fmaxf(m, pm[i]);
          const float f = __builtin_amdgcn_exp2f(m - mn), e = __builtin_amdgcn_exp2f(pm[i] - mn);
          m = mn;
          l = l * f + pl[i] * e;
          o.x = o.x * f + v[i].x * e;
          o.y = o.y * f + v[i].y * e;
          o.z = o.z * f + v[i].z * e;
          o.w = o.w * f + v[i].w * e;
        }
    }
    if (side > 1) {
      acc[threadIdx.x] = o;
      if (c4 == 0) {
        acc_m[g] = m;
        acc_l[g] = l;
      }
      __syncthreads();
      if (p0 == 0) {
        float mx = m;
        for (int i = 1; i < side; ++i) mx = fmaxf(mx, acc_m[g + i]);
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < side; ++i) {
          const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(acc_m[g + i] - mx);
          const float4 v = acc[(g + i) * LPR + c4];
          l += f * acc_l[g + i];
          o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
        }
        m = mx;
      }
      __syncthreads();
    }
    if (p0 == 0 && base + g / side < d.rows) {
      const int tok = r / a.G;
      const size_t at = (size_t)(d.row0 + tok) * a.Hq + d.head * a.G + r - tok * a.G;
      const float f = l != 0.f ? vs / l : 0.f;
      *reinterpret_cast<uint2*>(a.out + at * D + 4 * c4) =
          make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
      if (a.lse && c4 == 0) a.lse[at] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnArgs a, const int M, const int TB,
                                                                      const int desc_tiles,
                                                                      const float* __restrict__ partials,
                                                                      const PartDesc* __restrict__ descs) {
  constexpr int kGroups = kJoinThreads / (D / 4);
  __shared__ float4 acc[kJoinThreads];
  __shared__ float acc_l[kGroups], acc_m[kGroups];
  const PartDesc d = descs[blockIdx.x];
  if (desc_tiles > 0) {   // a tile that its sequence does not have has no description
    const int s = (int)blockIdx.x / (desc_tiles * a.Hkv), mt = (int)blockIdx.x % desc_tiles;
    if (mt * TB >= seq_info(a, s).n) return;
  }
  if (d.rows == 0) return;
  const int count = d.last - d.first + 1;
  int side = 1;
  while (side < kGroups && side * 8 < count) side *= 2;
  if (count <= 2) join_rows<D, 2>(a, M, d, side, partials, acc, acc_l, acc_m);
  else if (count <= 4) join_rows<D, 4>(a, M, d, side, partials, acc, acc_l, acc_m);
  else join_rows<D, 8>(a, M, d, side, partials, acc, acc_l, acc_m);
}

// ------------------------------------------------------------------------------------- the launch
// Parts of the line of segments = workgroups, all resident at once: one per CU (256), or two with shared
// tiles. One per CU there too where a part would see few keys, for half the partials: `segments` at most
// of at most `keys` keys. One and two per CU measured, by keys per part of two: 275 44 and 51 us (one
// prompt of 1500 tokens, D = 256), 450 29.8 and 31.7 (trees of 64 tokens), 512 46 and 55 (trees of 20 tokens,
// D = 256), 1125 41 and 42 (trees of 16 tokens, e4m3), 2048 67 and 60 (trees of 5 tokens, 96 heads), 3280 101 and 85
// (one prompt of 4096 tokens).
static int parts_for(int M, long segments, long keys) {
  return M == 128 && segments * keys < 512l * 1024 ? 256 : parts_of(M);
}

// Whether a workgroup takes a whole segment (no partials, no join) rather than an equal part of the
// line: `segments` as the rows of q say, `keys` as the block table allows at most. Whole and split
// measured, shared tiles: 1639 segments of one 16384-token prompt 868 and 1007 us; about 500 of up to
// 1024 keys 37 and 54; 100 of up to 250 keys 15 and 22; 409 of up to 4096 keys 98 and 92. A wave's own
// keys: 256 sequences of up to 1000 keys 21 and 30; 3 of up to 200 13 and 15; one of 777 19 and 15.
// Where a table of more than 4096 keys may hold a long segment among many, the kernel looks (2048 tokens of 96
// heads with one sequence of 131072 cached tokens: split 254 us, whole 2589; the two alone 158 and 89).
static Share share_for(bool shared_tiles, long segments, long keys) {
  if (keys <= 512) return kWholeSegments;
  if (!shared_tiles) return segments >= 128 && keys <= 1024 ? kWholeSegments : kEqualParts;
  if (segments >= 256 && keys <= 2048) return kWholeSegments;
  if (segments >= 1536) return keys <= 4096 ? kWholeSegments : kByLengths;
  return kEqualParts;
}

// Rows of a workgroup's tile for calls of at most max_q tokens per sequence: 32 with a wave's own
// keys where they hold a sequence's whole query group, else 128 sharing them (60 rows of 5 tokens,
// 64 sequences of up to 8192: 44 us; two 32-row tiles per wave of own keys: 53).
static int tile_rows(int max_q, int G) { return (long)max_q * G <= 32 ? 32 : 128; }
static size_t slot_floats(int M, int D) { return (size_t)M * D + 2 * M; }

size_t attention_workspace_bytes(int S, int max_q, int Hq, int Hkv, int D) {
  (void)S;
  const int M = tile_rows(max_q, Hq / Hkv);
  return parts_of(M) * 2 * (slot_floats(M, D) * 4 + sizeof(PartDesc));
}

template <int D, bool FP8, int RW, int KW, int NK, Cap CAP>
static hipError_t launch_one(const AttnArgs& a, hipStream_t stream) {
  using C = Attn<D, FP8, RW, KW, NK, CAP>;
  auto* kernel = attention_kernel<D, FP8, RW, KW, NK, CAP>;
  constexpr int kParts = parts_of(C::M);
  float* partials = static_cast<float*>(a.ws);
  PartDesc* descs = reinterpret_cast<PartDesc*>(partials + 2 * kParts * slot_floats(C::M, D));
  const int TB = C::M / a.G;
  // segments by the rows of q alone (a device-side count would come too late); one per sequence where a
  // tile holds its whole query group
  const long segments = (long)a.Hkv * (KW == 1 ? a.T / TB : min(a.S, a.T));
  const long bound = (long)a.Hkv * ((a.T + TB - 1) / TB + a.S);
  const long keys = (long)a.max_pages << a.page_shift;
  // (every workgroup reads every sequence's lengths: not for thousands of sequences)
  const Share share = bound <= 1l << 22 && a.S <= 4096 ? share_for(KW == 1, segments, keys) : kEqualParts;
  const int tiles = (a.max_q + TB - 1) / TB;
  const long most = (long)a.S * a.Hkv * tiles;   // segments, if every sequence had max_q tokens
  const bool by_segment = share == kEqualParts && most <= 2 * kParts;
  const int parts = share == kEqualParts ? parts_for(C::M, min(most, bound), keys) : kParts;
  const int grid = share == kEqualParts ? parts : (int)bound;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * C::kWaves), C::LDS, stream, a, TB, grid, share,
                     by_segment ? tiles : 0, partials, descs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || share == kWholeSegments) return e;
  // about as many workgroups as are resident at once, and no more than a segment has rows
  const int rows = (int)min((long)C::M, (long)a.max_q * a.G);
  const int y = by_segment ? max(1, min((int)(2048 / most), min(rows, 32))) : 4;
  hipLaunchKernelGGL(attention_join_kernel<D>, dim3(by_segment ? (int)most : parts, y), dim3(kJoinThreads), 0,
                     stream, a, C::M, TB, by_segment ? tiles : 0, (const float*)partials, (const PartDesc*)descs);
  return hipGetLastError();
}

template <int D, bool FP8, Cap CAP>
static hipError_t launch_rows(const AttnArgs& a, hipStream_t stream) {
  // A wave's own keys: as many waves as LDS holds two stages for, two per SIMD where that is eight, so that one
  // converts and exponentiates beside the other's loads (e4m3, eight waves of 32 keys and four of 64: 64
  // sequences of up to 8192 27.3 and 30.0 us, 3 of 131072 30.9 and 34.2; D = 64, 64 sequences, 2 kv heads, bf16 37.7 and
  // 39.3; D = 256, four of 32 keys and two: 41.4 and 48.6).
  constexpr int NKs = FP8 && D == 64 ? 64 : 32;
  constexpr int KWs = D == 64 || (FP8 && D == 128) ? 8 : (FP8 || D == 128 ? 4 : 2);
  if (tile_rows(a.max_q, a.G) == 32) return launch_one<D, FP8, 1, KWs, NKs, CAP>(a, stream);
  return launch_one<D, FP8, 4, 1, D == 256 ? 32 : 64, CAP>(a, stream);
}

template <int D, bool FP8>
static hipError_t launch_cap(const AttnArgs& a, hipStream_t stream) {
  if (a.softcap == 0.f) return launch_rows<D, FP8, kCapNone>(a, stream);
  return a.softcap <= kNearCap ? launch_rows<D, FP8, kCapSmall>(a, stream) : launch_rows<D, FP8, kCapLarge>(a, stream);
}

template <int D>
static hipError_t launch_dim(const AttnArgs& a, hipStream_t stream) {
  return a.k_scale ? launch_cap<D, true>(a, stream) : launch_cap<D, false>(a, stream);
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_dim<64>(a, stream);
    case 128: return launch_dim<128>(a, stream);
    default: return launch_dim<256>(a, stream);
  }
}

}  // namespace srmoe
