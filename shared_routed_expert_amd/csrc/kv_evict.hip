// Eviction from the paged cache: per kv head, a sequence of n > limit cached tokens keeps its first `sinks`, its last
// `recent`, and the m = budget - sinks - recent of largest usage between them (equal ones: the earlier), in order of position.
//
// Selection, one workgroup per sequence and kv head. Usage as an unsigned integer of the same order; the m-th largest is
// found by up to three passes over the row (12, 10 and 10 bits, counted in LDS), which say what it is, T, and how many of the
// values equal to T are kept, r; they end where all values of a prefix are kept. The place of token j among the kept is then
// (tokens before j that are protected or above T) + min(r, tokens before j equal to T): counted per wave's stretch of the row,
// added up, and written out. Bound by one CU's vector unit and its counting in LDS, not by bytes. (11, 11 and 10 bits: 0.5 us
// more in 16384 tokens, since usage crowds a few bins.)
//
// The kept tokens' keys and values then go to the sequence's new pages, which no sequence reads in this call: every row is read
// once and written once, by any workgroup at any time, and pages that other sequences share are left whole.
#include "kv_usage.hpp"
#include "common.hpp"

namespace srmoe {

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kBins = 4096 + 2 * 1024;   // of passes over 12, 10 and 10 bits

// Order of floats as that of unsigned integers: NaN lowest, then -infinity upwards, the zeros equal
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t o = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  return v != v ? 0u : o;
}

__device__ __forceinline__ int cached_tokens(const EvictArgs& a, int s) {
  return min(max(a.kv_lens[s], 0), a.max_pages << a.page_shift);
}

// A token as the selection sees it: protected ones above all orders, those past the end among the lowest (they come last of
// their equals, so none is kept)
constexpr uint32_t kProtected = 0xFFFFFFFFu, kTop = 0xFF800000u /* +infinity */;

// What the workgroup shares: the bins of every pass, cleared together.
struct Select {
  uint32_t counts[kBins];
  int wave_sum[kSelWaves], wave_eq[kSelWaves];
  int found_bin, found_left, found_count;
};

// A wave takes a stretch of the row, 256 tokens at a time, four a lane. HELD > 0: the stretch is at most HELD such steps and
// stays in registers, usage and order (16 steps spill); else each pass reads it again, four loads in flight. A cut of one
// sequence of 2112 tokens takes 11 to 12 us, of 32768 26, of 131072 76 (112 with each token's place compared in every
// pass), the move included.
template <int HELD>
__device__ __forceinline__ void select(const EvictArgs& a, Select& sh, const float* usage, float* out, int32_t* kept, int n) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = a.sinks, hi = n - a.recent;   // those that are chosen among
  const int stretch = (n + 256 * kSelWaves - 1) / (256 * kSelWaves) * 256;
  const int w_lo = min(wave * stretch, n), w_hi = min(w_lo + stretch, n);
  const int steps = (w_hi - w_lo + 255) / 256;
  // the four tokens from j on (rows are 16-byte aligned, and as long as whole pages; no row: all are equal)
  auto load4 = [&](int j) {
    return usage && j < w_hi ? *reinterpret_cast<const float4*>(usage + j) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto orders = [&](int j0, const float4& v) {   // of the 256 tokens from j0 on
    uint4 o = make_uint4(order_of(v.x), order_of(v.y), order_of(v.z), order_of(v.w));
    if (j0 >= lo && j0 + 256 <= hi) return o;   // none is protected or past the end
    const int j = j0 + 4 * lane;
    auto mark = [&](int at, uint32_t& one) {
      if (at < lo || at >= hi) one = at < n ? kProtected : 0;
    };
    mark(j, o.x), mark(j + 1, o.y), mark(j + 2, o.z), mark(j + 3, o.w);
    return o;
  };
  constexpr int kKept = HELD > 0 ? HELD : 1;
  float4 held[kKept];
  uint4 held_orders[kKept];
  if (HELD > 0) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) held[i] = load4(w_lo + 256 * i + 4 * lane);
  }
  for (int i = tid; i < kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0, 0, 0, 0);
  if (HELD > 0) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) held_orders[i] = orders(w_lo + 256 * i, held[i]);
  }
  __syncthreads();
  auto each = [&](auto f) {   // f(first token of the lane's four, their orders, their usage)
    if (HELD > 0) {
#pragma unroll
      for (int i = 0; i < kKept; ++i)
        if (i < steps) f(w_lo + 256 * i + 4 * lane, held_orders[i], held[i]);
    } else {
      constexpr int kAtOnce = 4;   // loads in flight
      for (int i0 = 0; i0 < steps; i0 += kAtOnce) {
        float4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) v[i] = load4(w_lo + 256 * (i0 + i) + 4 * lane);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int j0 = w_lo + 256 * (i0 + i);
          if (i0 + i < steps) f(j0 + 4 * lane, orders(j0, v[i]), v[i]);
        }
      }
    }
  };

  // -------- T, bits from the top, and r
  int left = a.budget - a.sinks - a.recent;   // how many of the values that begin with the prefix are kept
  uint32_t T = kTop;                          // (left == 0: none is above it, and none of those equal to it is kept)
  uint32_t prefix = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    if (left == 0) break;
    const int shift = pass == 0 ? 20 : (pass == 1 ? 10 : 0), bits = pass == 0 ? 12 : 10, bins = 1 << bits;
    uint32_t* const counts = sh.counts + (pass == 0 ? 0 : (pass == 1 ? 4096 : 4096 + 1024));
    each([&](int, const uint4& four, const float4&) {
      const uint32_t o[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = pass == 0 || o[e] >> shift >> bits == prefix;
        const uint32_t bin = (o[e] >> shift) & (bins - 1);
        const uint64_t who = __ballot(in);
        if (who == 0) continue;
        // where all lanes count in one bin (values alike), one of them adds them all
        const int lead = __ffsll((unsigned long long)who) - 1;
        const uint32_t one = (uint32_t)__builtin_amdgcn_readlane((int)bin, lead);
        if (__ballot(in && bin != one) == 0) {
          if (lane == lead) atomicAdd(&counts[one], (uint32_t)__popcll(who));
        } else if (in) {
          atomicAdd(&counts[bin], 1u);
        }
      }
    });
    __syncthreads();
    // the bin that holds the left-th largest: bins from the top, four a thread (the protected ones' is left out)
    const int low = bins - 4 * (tid + 1);
    uint4 c = make_uint4(0, 0, 0, 0);
    if (low >= 0) c = *reinterpret_cast<const uint4*>(counts + low);
    if (pass == 0 && tid == 0) c.w = 0;
    const int c4[4] = {(int)c.w, (int)c.z, (int)c.y, (int)c.x}, sum = c4[0] + c4[1] + c4[2] + c4[3];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (lane == 63) sh.wave_sum[wave] = incl;
    __syncthreads();
    int above = incl - sum;
#pragma unroll
    for (int k = 0; k < kSelWaves; ++k) above += k < wave ? sh.wave_sum[k] : 0;
    if (left > above && left <= above + sum) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (left > above && left <= above + c4[e]) {
          sh.found_bin = low + 3 - e;
          sh.found_left = left - above;
          sh.found_count = c4[e];
        }
        above += c4[e];
      }
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)sh.found_bin;
    left = sh.found_left;
    T = prefix << shift;
    if (pass < 2 && left == sh.found_count && T > 0) {   // all values of this prefix are kept: the rest of their bits is not needed
      T -= 1;
      left = 0;
    }
  }

  // -------- the places of the kept: tokens before a lane's e-th are those of all lanes before it and its own e
  struct Marks {
    uint64_t above[4], equal[4];   // lanes whose e-th token is protected or above T, or equal to it
  };
  auto look = [&](const uint4& four) {
    const uint32_t o[4] = {four.x, four.y, four.z, four.w};
    Marks m;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m.above[e] = __ballot(o[e] > T);
      m.equal[e] = __ballot(o[e] == T);
    }
    return m;
  };
  auto all_of = [](const uint64_t (&m)[4]) { return __popcll(m[0]) + __popcll(m[1]) + __popcll(m[2]) + __popcll(m[3]); };
  auto before = [](const uint64_t (&m)[4]) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      n = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m[e] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m[e], (uint32_t)n));
    return n;
  };
  int n_above = 0, n_equal = 0;
  each([&](int, const uint4& four, const float4&) {
    const Marks m = look(four);
    n_above += all_of(m.above);
    n_equal += all_of(m.equal);
  });
  __syncthreads();   // (wave_sum has been read; and with the row held, all of it has been)
  if (lane == 0) {
    sh.wave_sum[wave] = n_above;
    sh.wave_eq[wave] = n_equal;
  }
  __syncthreads();
  n_above = n_equal = 0;
#pragma unroll
  for (int k = 0; k < kSelWaves; ++k) {
    n_above += k < wave ? sh.wave_sum[k] : 0;
    n_equal += k < wave ? sh.wave_eq[k] : 0;
  }
  each([&](int j, const uint4& four, const float4& usage4) {
    const Marks m = look(four);
    const float v[4] = {usage4.x, usage4.y, usage4.z, usage4.w};
    int at_a = n_above + before(m.above), at_e = n_equal + before(m.equal);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool up = (m.above[e] >> lane) & 1, eq = (m.equal[e] >> lane) & 1;
      const int to = at_a + min(at_e, left);
      // (never budget or more, unless another sequence of the same row writes it meanwhile)
      if ((up || (eq && at_e < left)) && to < a.budget) {
        kept[to] = j + e;
        if (HELD > 0 && usage) out[to] = v[e];   // (out may be usage: nobody reads it any more)
      }
      at_a += up;
      at_e += eq;
    }
    n_above += all_of(m.above);
    n_equal += all_of(m.equal);
  });
  if (HELD > 0) return;

  // -------- a long row's usage, which may be written where it is read: place i is at most kept[i], so that a step's places lie
  // before every later step's sources, and its own have all been read at the barrier
  __threadfence_block();
  __syncthreads();
  if (!usage) return;
  for (int i0 = 0; i0 < a.budget; i0 += 4 * kSelThreads) {
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kSelThreads + tid;
      if (i < a.budget) v[k] = usage[min((uint32_t)kept[i], (uint32_t)n - 1)];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kSelThreads + tid;
      if (i < a.budget) out[i] = v[k];
    }
  }
}

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const EvictArgs a) {
  __shared__ __attribute__((aligned(16))) Select sh;
  const int s = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int n = cached_tokens(a, s);
  if (h == 0 && threadIdx.x == 0) a.new_lens[s] = n > a.limit ? a.budget : n;
  if (n <= a.limit) return;
  const int row = a.usage_rows ? a.usage_rows[s] : s;
  const bool known = row >= 0 && row < a.rows;
  const size_t base = ((size_t)(known ? row : 0) * a.Hkv + h) * ((size_t)a.max_pages << a.page_shift);
  const float* const usage = known ? a.usage + base : nullptr;
  float* const out = a.new_usage + base;
  int32_t* const kept = a.kept + ((size_t)s * a.Hkv + h) * a.budget;
  constexpr int kStep = 256 * kSelWaves;
  if (n <= kStep) select<1>(a, sh, usage, out, kept, n);
  else if (n <= 4 * kStep) select<4>(a, sh, usage, out, kept, n);
  else if (n <= 8 * kStep) select<8>(a, sh, usage, out, kept, n);
  else select<0>(a, sh, usage, out, kept, n);
}

// Rows of keys and values to the new pages: 16 bytes a lane, two rows of each a thread (four: one sequence of 2112 tokens 12.1 us
// instead of 11.5, the others alike). They are read past the caches (64 sequences in e4m3 48 -> 43 us) and written through
// them, to the attention that reads them next. Bytes set the pace: 24 sequences on 8 heads, 0.8 GB, at 4.9 to 5.1 TB/s.
typedef int i32x4 __attribute__((ext_vector_type(4)));
constexpr int kMoveThreads = 256, kMoveEach = 2;
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const EvictArgs a, const int lanes /* of a row */) {
  const int s = blockIdx.y / a.Hkv, h = blockIdx.y % a.Hkv;
  const int n = cached_tokens(a, s);
  if (n <= a.limit) return;
  const int32_t* const kept = a.kept + ((size_t)s * a.Hkv + h) * a.budget;
  const int at_once = kMoveThreads / lanes, lane = threadIdx.x % lanes;
  const int first = blockIdx.x * kMoveEach * at_once + threadIdx.x / lanes;
  const int mask = (1 << a.page_shift) - 1;
  const size_t rb = (size_t)lanes * 16, head = (size_t)h << a.page_shift;
  i32x4 k[kMoveEach], v[kMoveEach];
  size_t to[kMoveEach];
  bool go[kMoveEach];
#pragma unroll
  for (int x = 0; x < kMoveEach; ++x) {
    const int i = first + x * at_once;
    go[x] = i < a.budget;
    k[x] = v[x] = i32x4{0, 0, 0, 0};
    if (!go[x]) continue;
    const int j = (int)min((uint32_t)kept[i], (uint32_t)n - 1);
    const int src = a.block_table[(size_t)s * a.max_pages + (j >> a.page_shift)];
    const int dst = a.new_table[(size_t)s * a.new_max_pages + (i >> a.page_shift)];
    go[x] = dst >= 0 && dst < a.num_pages;
    to[x] = (size_t)(go[x] ? dst : 0) * a.page_bytes + (head + (i & mask)) * rb + lane * 16;
    if (src >= 0 && src < a.num_pages) {   // (a token of no page becomes zeros)
      const size_t from = (size_t)src * a.page_bytes + (head + (j & mask)) * rb + lane * 16;
      k[x] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(a.k_cache + from));
      v[x] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(a.v_cache + from));
    }
  }
#pragma unroll
  for (int x = 0; x < kMoveEach; ++x)
    if (go[x]) {
      *reinterpret_cast<i32x4*>(a.k_cache + to[x]) = k[x];
      *reinterpret_cast<i32x4*>(a.v_cache + to[x]) = v[x];
    }
}

hipError_t launch_kv_evict(const EvictArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(kv_select_kernel, dim3(a.S * a.Hkv), dim3(kSelThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int lanes = a.row_bytes / 16, rows = kMoveEach * kMoveThreads / lanes;
  hipLaunchKernelGGL(kv_move_kernel, dim3((a.budget + rows - 1) / rows, a.S * a.Hkv), dim3(kMoveThreads), 0, stream, a,
                     lanes);
  return hipGetLastError();
}

}  // namespace srmoe
