// Eviction from the paged cache: which tokens a head keeps, and moving them together.
//
//   evict    of a sequence's `len` tokens the first `sinks`, the last `recent` and, of those
//            between, the budget - sinks - recent of the largest sums, of equal ones the
//            earlier.  The sums become whole numbers of the same order (sign turned, NaN
//            lowest), and the smallest kept one is found digit by digit from the top: 11, 11
//            and 10 bits, each a histogram of the sums that agree so far and a scan over it.
//            What is larger is kept, and of the equal ones the first that are missing.  Counts
//            are whole numbers, so the order of the histogram's atomics changes nothing.
//            A workgroup does it for sequences of up to 8192 tokens, in LDS; longer ones are cut
//            into up to 16 chunks, a launch a digit, whose histograms go through the workspace.
//   compact  row starts + j of a head takes row keep[j], in place.  The lists rise and no row is
//            before its place, so a workgroup that takes a head's rows in order, reads a run
//            whole and then writes it, never overwrites what is still to be read.  Few long lists
//            go through the workspace instead, by as many workgroups as there are rows.
#include "kv_common.h"
#include "tile_common.h"

namespace tabit {
namespace {

using namespace kv;

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kCopies = 4;       // of a histogram, by lane: fewer lanes meet at one place
constexpr int kWhole = 8192;     // tokens whose numbers one workgroup holds
constexpr int kChunks = 16;      // of a longer sequence, at most

// Whole number of the same order as w: NaN 0, then -infinity ... infinity (-0 as 0).
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  return w != w ? 0u : u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ int count_below(unsigned long long m, int lane) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// Ordered numbers of the sums of tokens i .. i + 3 of a sequence (i a multiple of 4: one page).
__device__ __forceinline__ uint4 load4(const KvEvictArgs& a, const int* table, int h, int i) {
  const KvCacheArgs& c = a.cache;
  const int page = table[i >> c.page_shift];
  if ((unsigned)page >= (unsigned)c.num_pages) return make_uint4(0u, 0u, 0u, 0u);
  const float4 w = *reinterpret_cast<const float4*>(
      a.sums + ((((long long)page * c.heads + h) << c.page_shift) | (i & ((1 << c.page_shift) - 1))));
  return make_uint4(order_of(w.x), order_of(w.y), order_of(w.z), order_of(w.w));
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k, 64);
  return v;
}

// Bits of digit `pass`, from the top.
constexpr int digit_bits(int pass) { return pass < 2 ? kBits : 32 - 2 * kBits; }

// The bin, from the top, in which the count passes `missing`, and the count above it: thread t
// has the counts of bins kBins - 1 - 2 t and the one below.  room: kWaves + 2 ints of LDS.
__device__ __forceinline__ void find_bin(int high, int low, int missing, int* room, int& bin, int& above) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = high + low;
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    const int y = __shfl_up(sum, k, 64);
    sum += lane >= k ? y : 0;
  }
  __syncthreads();
  if (lane == 63) room[wave] = sum;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWaves; ++k) sum += k < wave ? room[k] : 0;
  const int before = sum - high - low;                     // exactly one thread finds its bin
  if (before < missing && sum >= missing) {
    const bool first = before + high >= missing;
    room[kWaves] = kBins - 1 - 2 * (int)threadIdx.x - (first ? 0 : 1);
    room[kWaves + 1] = first ? before : before + high;
  }
  __syncthreads();
  bin = room[kWaves];
  above = room[kWaves + 1];
}

// Writes the kept ones of tokens [from, to) of one wave, four neighbours a lane; get4 gives their
// numbers.  Kept for sure: outside [first, last), and larger than T where any compete; of the equal ones
// as many as are `missing`.  sure, equal: how many of either come before.  COUNT: only counts them.
template <bool COUNT, typename Get>
__device__ __forceinline__ void write_kept(int from, int to, int first, int last, bool any, uint32_t T, int missing,
                                           int& sure, int& equal, int* keep, Get get4) {
  const int lane = threadIdx.x & 63;
  for (int i0 = from; i0 < to; i0 += 256) {
    const int i = i0 + lane * 4;
    const uint4 x = i < to ? get4(i) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
    unsigned long long ms[4], me[4];
    bool s[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = i + e < to, between = i + e >= first && i + e < last;
      s[e] = in && (!between || (any && v[e] > T));
      q[e] = in && between && any && v[e] == T;
      ms[e] = __ballot(s[e]);
      me[e] = __ballot(q[e]);
    }
    if constexpr (!COUNT) {
      int ps = sure, pe = equal;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ps += count_below(ms[e], lane);
        pe += count_below(me[e], lane);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (s[e] || (q[e] && pe < missing)) keep[ps + min(pe, missing)] = i + e;
        ps += s[e];
        pe += q[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sure += __popcll(ms[e]);
      equal += __popcll(me[e]);
    }
  }
}

// Up to kWhole tokens: one workgroup a key head of a sequence, the numbers in LDS.  Bound by what it waits for:
// two loads that depend on each other, then six barriers a digit (2048 tokens of one sequence 8.4 us, up to 8192 of
// 32 sequences, 8 heads, 13.1).
__global__ void __launch_bounds__(kThreads)
kv_evict_kernel(KvEvictArgs a) {
  __shared__ uint32_t hist[kCopies][kBins];
  __shared__ __attribute__((aligned(16))) uint32_t held[kWhole];
  __shared__ int room[kWaves + 2], counted[kWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const int* table = a.table + (long long)b * a.table_stride;
  // (before the length is known: the table has room for max_kv tokens, and what lies past the length
  // is not looked at)
  uint4 mine[kWhole / (kThreads * 4)];
#pragma unroll
  for (int k = 0; k < kWhole / (kThreads * 4); ++k) {
    const int i = (k * kThreads + tid) * 4;
    mine[k] = i < a.max_kv ? load4(a, table, h, i) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int n = min(max(a.kv_lens[b], 0), a.max_kv);
  int* keep = a.keep + ((long long)b * a.cache.heads + h) * a.budget;
  if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
  if (n <= a.budget) {
    for (int j = tid; j < a.budget; j += kThreads) keep[j] = j < n ? j : -1;
    return;
  }
  const int first = a.sinks, last = n - a.recent;          // those between compete: first < last
#pragma unroll
  for (int k = 0; k < kWhole / (kThreads * 4); ++k) *reinterpret_cast<uint4*>(held + (k * kThreads + tid) * 4) = mine[k];
  auto get4 = [&](int i) { return *reinterpret_cast<const uint4*>(held + i); };

  // The smallest kept number T, and how many equal to it are kept
  uint32_t T = 0u;
  int missing = a.budget - a.sinks - a.recent;
  const bool any = missing > 0;
  int shift = 32;
  for (int pass = 0; pass < 3 && any; ++pass) {
    const int bits = digit_bits(pass);
    shift -= bits;
    for (int k = tid; k < kCopies * kBins; k += kThreads) (&hist[0][0])[k] = 0u;
    __syncthreads();
    for (int i = tid * 4; i < n; i += kThreads * 4) {
      const uint4 x = get4(i);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e >= first && i + e < last && (pass == 0 || (v[e] >> (shift + bits)) == T))
          atomicAdd(&hist[lane & (kCopies - 1)][(v[e] >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    const int top = kBins - 1 - 2 * tid;
    int high = 0, low = 0, bin, above;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      high += (int)hist[k][top];
      low += (int)hist[k][top - 1];
    }
    find_bin(high, low, missing, room, bin, above);
    T = T << bits | (uint32_t)bin;
    missing -= above;
  }
  __syncthreads();               // (also where nothing competes: the numbers are in LDS)

  // A wave writes its run of tokens: first counts them, then knows its place
  const int per = ((n + kWaves * 256 - 1) / (kWaves * 256)) * 256;
  const int from = min(wave * per, n), to = min(from + per, n);
  int sure = 0, equal = 0;
  write_kept<true>(from, to, first, last, any, T, missing, sure, equal, keep, get4);
  if (lane == 0) {
    counted[wave][0] = sure;
    counted[wave][1] = equal;
  }
  __syncthreads();
  sure = equal = 0;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    sure += k < wave ? counted[k][0] : 0;
    equal += k < wave ? counted[k][1] : 0;
  }
  write_kept<false>(from, to, first, last, any, T, missing, sure, equal, keep, get4);
}

// ------------------------------------------------------------------ longer sequences
// What a chunk's workgroup of one digit leaves for its own of the next.
struct Found {
  uint32_t T;
  int missing, before;           // kept for sure in the chunks before
};
struct LongPlan {
  int chunks, tokens;            // of one chunk
  uint32_t* hist[2];             // [seqs][heads][chunks][kBins], of every other digit
  Found* found;                  // [seqs][heads][chunks]
};

// PASS 0 counts the first digit of a chunk's tokens; 1 and 2 find a digit from all chunks' counts and
// count the next; 3 finds the last and writes the chunk's kept tokens.  Bound as the other, four times, and in 1 to 3
// by the counts of all chunks, which every workgroup reads before it starts (128 KB, 16 MB a launch of 8 heads): 131072
// tokens of 8 heads 5.6, 9.3, 8.6 and 10.4 us (one workgroup a head for all of it: 146).
template <int PASS>
__global__ void __launch_bounds__(kThreads)
kv_evict_long_kernel(KvEvictArgs a, LongPlan p) {
  __shared__ uint32_t hist[PASS < 3 ? kCopies : 1][PASS < 3 ? kBins : 1];
  __shared__ __attribute__((aligned(16))) uint32_t held[kWhole];
  __shared__ int room[kWaves + 2], counted[kWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // (heads first: the chunks of a head share a die's L2 where the heads are a multiple of eight)
  const int h = blockIdx.x, chunk = blockIdx.y, b = blockIdx.z;
  const int n = min(max(a.kv_lens[b], 0), a.max_kv);
  int* keep = a.keep + ((long long)b * a.cache.heads + h) * a.budget;
  if (n <= a.budget) {
    if constexpr (PASS == 3) {
      if (h == 0 && chunk == 0 && tid == 0) a.new_lens[b] = n;
      for (int j = chunk * kThreads + tid; j < a.budget; j += p.chunks * kThreads) keep[j] = j < n ? j : -1;
    }
    return;
  }
  const long long pair = (long long)b * a.cache.heads + h;
  const int first = a.sinks, last = n - a.recent;
  const int* table = a.table + (long long)b * a.table_stride;
  const int c0 = min(chunk * p.tokens, n), c1 = min(c0 + p.tokens, n);
  uint32_t T = 0u;
  int missing = a.budget - a.sinks - a.recent, before = 0, equal = 0;
  const bool any = missing > 0;
  // The numbers of a chunk that LDS holds are on their way while the last digit is found.
  const bool whole = p.tokens <= kWhole;
  uint4 own[kWhole / (kThreads * 4)];
#pragma unroll
  for (int k = 0; k < kWhole / (kThreads * 4); ++k) {
    const int i = c0 + (k * kThreads + tid) * 4;
    own[k] = whole && i < c1 ? load4(a, table, h, i) : make_uint4(0u, 0u, 0u, 0u);
  }
  if constexpr (PASS > 0) {
    if constexpr (PASS > 1) {
      const Found f = p.found[pair * p.chunks + chunk];
      T = f.T;
      missing = f.missing;
      before = f.before;
    }
    if (any) {
      // thread: two bins of the last digit counted, over all chunks and over those before this one
      const uint32_t* from = p.hist[(PASS - 1) & 1] + pair * p.chunks * kBins;
      const int top = kBins - 1 - 2 * tid;
      int high = 0, low = 0, high_before = 0, low_before = 0, bin, above;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint2 x = k < p.chunks ? *reinterpret_cast<const uint2*>(from + (long long)k * kBins + top - 1) : make_uint2(0u, 0u);
        high += (int)x.y;
        low += (int)x.x;
        high_before += k < chunk ? (int)x.y : 0;
        low_before += k < chunk ? (int)x.x : 0;
      }
      find_bin(high, low, missing, room, bin, above);
      T = T << digit_bits(PASS - 1) | (uint32_t)bin;
      missing -= above;
      int mine = (top > bin ? high_before : 0) + (top - 1 > bin ? low_before : 0);
      int same = (top == bin ? high_before : 0) + (top - 1 == bin ? low_before : 0);
      mine = wave_sum(mine);
      same = wave_sum(same);
      if (lane == 0) {
        counted[wave][0] = mine;
        counted[wave][1] = same;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        before += counted[k][0];
        equal += counted[k][1];
      }
    }
    if (PASS < 3 && tid == 0) p.found[pair * p.chunks + chunk] = {T, missing, before};
  }
#pragma unroll
  for (int k = 0; k < kWhole / (kThreads * 4); ++k) *reinterpret_cast<uint4*>(held + (k * kThreads + tid) * 4) = own[k];
  auto get4 = [&](int i) { return whole ? *reinterpret_cast<const uint4*>(held + (i - c0)) : load4(a, table, h, i); };
  if constexpr (PASS < 3) {
    for (int k = tid; k < kCopies * kBins; k += kThreads) (&hist[0][0])[k] = 0u;
    __syncthreads();
    constexpr int bits = digit_bits(PASS);
    constexpr int shift = PASS == 0 ? 32 - kBits : PASS == 1 ? 32 - 2 * kBits : 0;
    if (any) {
#pragma unroll 2
      for (int i = c0 + tid * 4; i < c1; i += kThreads * 4) {
        const uint4 x = get4(i);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e >= first && i + e < min(last, c1) && (PASS == 0 || (v[e] >> (shift + bits) % 32) == T))
            atomicAdd(&hist[lane & (kCopies - 1)][(v[e] >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    __syncthreads();
    uint32_t* to = p.hist[PASS & 1] + (pair * p.chunks + chunk) * kBins;
    for (int k = tid; k < kBins; k += kThreads) {
      uint32_t sum = 0u;
#pragma unroll
      for (int m = 0; m < kCopies; ++m) sum += hist[m][k];
      to[k] = sum;
    }
  } else {
    __syncthreads();                                       // the numbers are in LDS
    if (h == 0 && chunk == 0 && tid == 0) a.new_lens[b] = a.budget;
    // the first and the last ones before this chunk are kept for sure, too
    before += min(c0, first) + max(c0 - last, 0);
    const int per = ((c1 - c0 + kWaves * 256 - 1) / (kWaves * 256)) * 256;
    const int from = min(c0 + wave * per, c1), to = min(from + per, c1);
    int s = 0, q = 0;
    write_kept<true>(from, to, first, last, any, T, missing, s, q, keep, get4);
    __syncthreads();
    if (lane == 0) {
      counted[wave][0] = s;
      counted[wave][1] = q;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      before += k < wave ? counted[k][0] : 0;
      equal += k < wave ? counted[k][1] : 0;
    }
    write_kept<false>(from, to, first, last, any, T, missing, before, equal, keep, get4);
  }
}

// Up to kChunks chunks of 8192 tokens or more: every workgroup reads all chunks' counts.
size_t long_plan(int seqs, int heads, int max_kv, uint8_t* ws, LongPlan& p) {
  const long long even = ((long long)max_kv + kChunks - 1) / kChunks;
  p.tokens = (int)(even <= kWhole ? kWhole : (even + 4095) / 4096 * 4096);
  p.chunks = (int)(((long long)max_kv + p.tokens - 1) / p.tokens);
  const size_t all = (size_t)seqs * (size_t)heads * (size_t)p.chunks, hist = all * kBins * 4;
  p.hist[0] = reinterpret_cast<uint32_t*>(ws);
  p.hist[1] = reinterpret_cast<uint32_t*>(ws + hist);
  p.found = reinterpret_cast<Found*>(ws + 2 * hist);
  return 2 * hist + all * sizeof(Found);
}

// A row of a head on its way: the codes of key and value in pieces of 16 bytes and a last
// piece of scales (key, value), the sum and whether there is such a row.
template <int NB>
struct Row {
  static constexpr int PIECES = 2 * NB + 1;
};

// Index of token j's row among all rows of the cache, or -1.
__device__ __forceinline__ long long row_of(const KvCacheArgs& c, const int* table, int table_stride, int h, int j) {
  const int pi = j >> c.page_shift;
  if (j < 0 || pi >= table_stride) return -1;
  const int page = table[pi];
  if ((unsigned)page >= (unsigned)c.num_pages) return -1;
  return (((long long)page * c.heads + h) << c.page_shift) | (j & ((1 << c.page_shift) - 1));
}

template <int NB>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (NB == 4) return *reinterpret_cast<const uint32_t*>(p);
  if constexpr (NB == 2) return *reinterpret_cast<const uint16_t*>(p);
  uint32_t v = p[0];
  if constexpr (NB == 3) v |= (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
  return v;
}
template <int NB>
__device__ __forceinline__ void store_scales(uint8_t* p, uint32_t v) {
  if constexpr (NB == 4) {
    *reinterpret_cast<uint32_t*>(p) = v;
  } else if constexpr (NB == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)v;
  } else {
    p[0] = (uint8_t)v;
    if constexpr (NB == 3) {
      p[1] = (uint8_t)(v >> 8);
      p[2] = (uint8_t)(v >> 16);
    }
  }
}

// Piece p of row `at`.
template <int NB>
__device__ __forceinline__ uint4 load_piece(const KvCompactArgs& a, long long at, int p) {
  const KvCacheArgs& c = a.cache;
  if (p < NB) return reinterpret_cast<const uint4*>(c.k_codes)[at * NB + p];
  if (p < 2 * NB) return reinterpret_cast<const uint4*>(c.v_codes)[at * NB + (p - NB)];
  return make_uint4(load_scales<NB>(c.k_scales + at * NB), load_scales<NB>(c.v_scales + at * NB),
                    a.sums != nullptr ? __float_as_uint(a.sums[at]) : 0u, 1u);
}
template <int NB>
__device__ __forceinline__ void store_piece(const KvCompactArgs& a, long long at, int p, uint4 x) {
  const KvCacheArgs& c = a.cache;
  if (p < NB) {
    reinterpret_cast<uint4*>(c.k_codes)[at * NB + p] = x;
  } else if (p < 2 * NB) {
    reinterpret_cast<uint4*>(c.v_codes)[at * NB + (p - NB)] = x;
  } else {
    store_scales<NB>(c.k_scales + at * NB, x.x);
    store_scales<NB>(c.v_scales + at * NB, x.y);
    if (a.sums != nullptr) a.sums[at] = __uint_as_float(x.z);
  }
}

// Rows to the workspace (GATHER), and from there to their places.  blockIdx: rows, head, sequence.
template <int NB, bool GATHER>
__global__ void __launch_bounds__(256)
kv_compact_kernel(KvCompactArgs a) {
  constexpr int PIECES = Row<NB>::PIECES;
  constexpr int ROWS = 256 / PIECES;
  const int r = threadIdx.x / PIECES, p = threadIdx.x % PIECES;
  const int h = blockIdx.y, b = blockIdx.z;
  const int j = blockIdx.x * ROWS + r;
  if (r >= ROWS || j >= min(a.counts[b], a.keep_stride)) return;
  const int* table = a.table + (long long)b * a.table_stride;
  const int from = a.keep[((long long)b * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_stride + j];
  const int start = a.starts != nullptr ? a.starts[b] : 0;
  const long long src = row_of(a.cache, table, a.table_stride, h, from);
  // (a place past 2^31 is none)
  const long long dst = start > 0x7FFFFFFF - j ? -1 : row_of(a.cache, table, a.table_stride, h, start + j);
  if (src < 0 || dst < 0) return;
  uint4* piece = reinterpret_cast<uint4*>(a.ws) +
                 (((long long)b * a.cache.heads + h) * a.keep_stride + j) * PIECES + p;
  if constexpr (GATHER) *piece = load_piece<NB>(a, src, p);
  else store_piece<NB>(a, dst, p, *piece);
}

// In place: one workgroup takes the keys (or values) of one head, kRun rows at a time, which are read
// whole before the first is written.  What comes later lies behind all places written so far.  Bound by rows of
// 64 bytes in any place: 32 lists of 2048 of 8 heads x 128 elements (70 MB read, 73 written) 51 us, 2.8 TB/s.
// 2048, 1024 and 512 rows at a time by a thread each were 74, 54 and 56 us, by half as many threads 71 to 80;
// with the next run's places looked up beside this one's rows 66, with its rows read beside this one's writes 57.
constexpr int kRun = kThreads;
template <int NB>
__global__ void __launch_bounds__(kRun)
kv_compact_run_kernel(KvCompactArgs a) {
  __shared__ long long src[kRun], dst[kRun];
  const int tid = threadIdx.x;
  const int h = blockIdx.x >> 1, b = blockIdx.y;
  const bool keys = (blockIdx.x & 1) == 0;
  const KvCacheArgs& c = a.cache;
  const int* table = a.table + (long long)b * a.table_stride;
  const int* keep = a.keep + ((long long)b * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_stride;
  const int first = tid < a.keep_stride ? keep[tid] : -1;  // (before the count is known)
  const int count = min(a.counts[b], a.keep_stride), start = a.starts != nullptr ? a.starts[b] : 0;
  uint4* codes = reinterpret_cast<uint4*>(keys ? c.k_codes : c.v_codes);
  uint8_t* scales = keys ? c.k_scales : c.v_scales;
  for (int j0 = 0; j0 < count; j0 += kRun) {
    const int j = j0 + tid;
    long long own = -1, own_to = -1;
    if (j < count) {
      own = row_of(c, table, a.table_stride, h, j0 == 0 ? first : keep[j]);
      own_to = start > 0x7FFFFFFF - j ? -1 : row_of(c, table, a.table_stride, h, start + j);
      if (own == own_to || own_to < 0) own = -1;           // (in its place already, or no place)
    }
    src[tid] = own;
    dst[tid] = own_to;
    __syncthreads();
    uint4 x[NB];
    uint32_t s = 0u;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = i * kRun + tid;
      if (src[at / NB] >= 0) x[i] = codes[src[at / NB] * NB + at % NB];
    }
    if (own >= 0) {
      s = load_scales<NB>(scales + own * NB);
      if (keys && a.sums != nullptr) w = a.sums[own];
    }
    tile::wait_vmcnt0();                                   // all of the run is here, in every wave
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = i * kRun + tid;
      if (src[at / NB] >= 0) codes[dst[at / NB] * NB + at % NB] = x[i];
    }
    if (own >= 0) {
      store_scales<NB>(scales + own_to * NB, s);
      if (keys && a.sums != nullptr) a.sums[own_to] = w;
    }
    __syncthreads();                                       // the places of the next run overwrite these
  }
}

// Whether lists go through the workspace: long ones of few heads (one list of 16384 of 8 heads: 12 us there,
// 9 back).
bool through_ws(int seqs, int heads, int keep_stride) {
  return keep_stride > 2 * kRun && (long long)seqs * heads < 64;
}

template <int NB>
hipError_t compact_nb(const KvCompactArgs& a, hipStream_t s) {
  if (!through_ws(a.seqs, a.cache.heads, a.keep_stride)) {
    kv_compact_run_kernel<NB><<<dim3(2u * (unsigned)a.cache.heads, (unsigned)a.seqs), kRun, 0, s>>>(a);
    return hipGetLastError();
  }
  constexpr int ROWS = 256 / Row<NB>::PIECES;
  const dim3 grid((unsigned)(((long long)a.keep_stride + ROWS - 1) / ROWS), (unsigned)a.cache.heads, (unsigned)a.seqs);
  kv_compact_kernel<NB, true><<<grid, 256, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  kv_compact_kernel<NB, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t kv_evict_workspace(int seqs, int heads, int max_kv) {
  LongPlan p;
  return max_kv <= kWhole ? 0 : long_plan(seqs, heads, max_kv, nullptr, p);
}

hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t s) {
  if (a.max_kv <= kWhole) {
    kv_evict_kernel<<<dim3((unsigned)a.cache.heads, (unsigned)a.seqs), kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  LongPlan p;
  long_plan(a.seqs, a.cache.heads, a.max_kv, a.ws, p);
  const dim3 grid((unsigned)a.cache.heads, (unsigned)p.chunks, (unsigned)a.seqs);
  kv_evict_long_kernel<0><<<grid, kThreads, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  kv_evict_long_kernel<1><<<grid, kThreads, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  kv_evict_long_kernel<2><<<grid, kThreads, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  kv_evict_long_kernel<3><<<grid, kThreads, 0, s>>>(a, p);
  return hipGetLastError();
}

size_t kv_compact_workspace(int seqs, int heads, int dim_pad, int keep_stride) {
  if (!through_ws(seqs, heads, keep_stride)) return 0;
  return (size_t)seqs * (size_t)heads * (size_t)keep_stride * (size_t)(2 * (dim_pad / 32) + 1) * 16;
}

hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t s) {
  switch (a.cache.dim_pad) {
    case 32: return compact_nb<1>(a, s);
    case 64: return compact_nb<2>(a, s);
    case 96: return compact_nb<3>(a, s);
    case 128: return compact_nb<4>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tabit
