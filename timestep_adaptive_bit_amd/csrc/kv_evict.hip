// Eviction from the paged cache: which tokens a head keeps, and moving them together.
//
//   evict    of a sequence's `len` tokens the first `sinks`, the last `recent` and, of those
//            between, the budget - sinks - recent of the largest sums, of equal ones the
//            earlier.  The sums become whole numbers of the same order (sign turned, NaN
//            lowest), and the smallest kept one is found digit by digit from the top: 11, 11
//            and 10 bits, each a histogram of the sums that agree so far and a scan over it.
//            What is larger is kept, and of the equal ones the first that are missing.  Counts
//            are whole numbers, so the order of the histogram's atomics changes nothing.
//   compact  row starts + j of a head takes row keep[j], in place.
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kBits = 11, kBins = 1 << kBits;

// Whole number of the same order as w: NaN 0, then -infinity ... infinity (-0 as 0).
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  return w != w ? 0u : u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ int count_below(unsigned long long m, int lane) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// One workgroup: one key head of one sequence.  CAP: sums (as ordered numbers) that are held in
// LDS, read from memory once; a longer sequence reads them again for each pass (CAP 0).
// A lane takes four neighbours, which lie in one page.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
kv_evict_kernel(KvEvictArgs a) {
  constexpr int COPIES = 4;          // of the histogram, by lane: fewer lanes meet at one place
  __shared__ uint32_t hist[COPIES][kBins];
  __shared__ uint32_t held[CAP > 0 ? CAP : 4];
  __shared__ int wave_sum[kWaves][2], found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const KvCacheArgs& c = a.cache;
  const int n = min(max(a.kv_lens[b], 0), a.max_kv);
  int* keep = a.keep + ((long long)b * c.heads + h) * a.budget;
  if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
  if (n <= a.budget) {
    for (int j = tid; j < a.budget; j += kThreads) keep[j] = j < n ? j : -1;
    return;
  }
  const int first = a.sinks, last = n - a.recent;          // those between compete: first < last
  const int* table = a.table + (long long)b * a.table_stride;
  // Ordered numbers of tokens i .. i + 3 (i a multiple of 4; some may lie past n)
  auto load4 = [&](int i) {
    const int page = table[i >> c.page_shift];
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if ((unsigned)page < (unsigned)c.num_pages) {
      const float* p = a.sums + ((((long long)page * c.heads + h) << c.page_shift) | (i & ((1 << c.page_shift) - 1)));
      const float4 w = *reinterpret_cast<const float4*>(p);
      x = make_uint4(order_of(w.x), order_of(w.y), order_of(w.z), order_of(w.w));
    }
    return x;
  };
  if constexpr (CAP > 0) {
    for (int i = tid * 4; i < n; i += kThreads * 4) *reinterpret_cast<uint4*>(held + i) = load4(i);
  }
  auto get4 = [&](int i) {
    if constexpr (CAP > 0) return *reinterpret_cast<const uint4*>(held + i);
    else return load4(i);
  };

  // The smallest kept number T, and how many equal to it are kept
  uint32_t T = 0u;
  int missing = a.budget - a.sinks - a.recent;
  const bool any = missing > 0;
  int shift = 32;
  for (int pass = 0; pass < 3 && any; ++pass) {
    const int bits = pass < 2 ? kBits : 32 - 2 * kBits;
    shift -= bits;
    for (int k = tid; k < COPIES * kBins; k += kThreads) (&hist[0][0])[k] = 0u;
    __syncthreads();
    for (int i = tid * 4; i < n; i += kThreads * 4) {
      const uint4 x = get4(i);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e >= first && i + e < last && (pass == 0 || (v[e] >> (shift + bits)) == T))
          atomicAdd(&hist[lane & (COPIES - 1)][(v[e] >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    // thread: two bins, from the top; how many numbers lie in them and above
    const int top = kBins - 1 - 2 * tid;
    int two[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < COPIES; ++k) {
      two[0] += (int)hist[k][top];
      two[1] += (int)hist[k][top - 1];
    }
    int sum = two[0] + two[1];
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int y = __shfl_up(sum, k, 64);
      sum += lane >= k ? y : 0;
    }
    if (lane == 63) wave_sum[wave][0] = sum;
    __syncthreads();
    for (int k = 0; k < wave; ++k) sum += wave_sum[k][0];
    const int above = sum - two[0] - two[1];               // exactly one thread finds its bin
    if (above < missing && above + two[0] >= missing) {
      found[0] = top;
      found[1] = above;
    } else if (above + two[0] < missing && sum >= missing) {
      found[0] = top - 1;
      found[1] = above + two[0];
    }
    __syncthreads();
    T = T << bits | (uint32_t)found[0];
    missing -= found[1];
    __syncthreads();
  }

  // A wave writes its run of tokens: first counts them, then knows its place
  const int per = ((n + kWaves * 256 - 1) / (kWaves * 256)) * 256;
  const int from = min(wave * per, n), to = min(from + per, n);
  int place = 0, equals = 0;
  for (int phase = 0; phase < 2; ++phase) {
    int sure = 0, equal = 0;
    for (int i0 = from; i0 < to; i0 += 256) {
      const int i = i0 + lane * 4;
      const uint4 x = i < n ? get4(i) : make_uint4(0u, 0u, 0u, 0u);
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
      if (phase == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sure += __popcll(ms[e]);
          equal += __popcll(me[e]);
        }
        continue;
      }
      // before the lane's four: kept for sure, and equal ones, of which the first `missing`
      int ps = place, pe = equals;
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        place += __popcll(ms[e]);
        equals += __popcll(me[e]);
      }
    }
    if (phase == 0) {
      if (lane == 0) {
        wave_sum[wave][0] = sure;
        wave_sum[wave][1] = equal;
      }
      __syncthreads();
      for (int k = 0; k < wave; ++k) {
        place += wave_sum[k][0];
        equals += wave_sum[k][1];
      }
    }
  }
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

template <int NB>
hipError_t compact_nb(const KvCompactArgs& a, hipStream_t s) {
  constexpr int ROWS = 256 / Row<NB>::PIECES;
  const dim3 grid((unsigned)(((long long)a.keep_stride + ROWS - 1) / ROWS), (unsigned)a.cache.heads, (unsigned)a.seqs);
  kv_compact_kernel<NB, true><<<grid, 256, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  kv_compact_kernel<NB, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.cache.heads, (unsigned)a.seqs);
  if (a.max_kv <= 8192) kv_evict_kernel<8192><<<grid, kThreads, 0, s>>>(a);
  else kv_evict_kernel<0><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

size_t kv_compact_workspace(int seqs, int heads, int dim_pad, int keep_stride) {
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
