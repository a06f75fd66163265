// Attention weights summed over a step's rows, per cached token and key head:
//
//   w_j += sum_i exp2(s_ij - L_i),  s_ij = c q'_i . k'_j,  L_i = log2 sum_j exp2(s_ij)
//
// with q', k', c and the visible keys as in the attention kernels.  The result is fp32 and
// stays that exact: q' is five FP6 (E2M3) terms with scales 2^e ... 2^(e-16) per block of 32
// (2^-21 of the block's largest element is lost at most), which go against the key codes
// as stored in the 32x32x64 block-scaled MFMA, and the exponentials take fp32 scores.
//
// Three kernels.  One prepares the rows, 32 a tile, once for all that read them.  The second
// passes over the keys for L: S = K Q'^T, so that a lane has one row and keeps its largest
// score and its sum alone until the end.  The third passes over the keys again for the
// sums: S = Q' K^T, so that a lane has one key and adds up rows in registers; the accumulator
// starts at -L, so what leaves the matrix core goes into the exponential as it is.  Storing the scores
// of the first pass would cost as many bytes as the keys have at eight rows a head, and more than
// the memory holds in long prompts.
//
// Workspace, per 32-row tile: the terms' codes, 1.5 KB each for 64 elements (lane l: row l % 32,
// block l / 32 of the step; 16 and then 8 bytes a lane), and eight bytes of scales a lane; then
// -L of each row, and with `splits` ranges of keys each one's (reference, sum).
#include "kv_query.h"

namespace tabit {
namespace {

using namespace kv;

constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e+38f;
constexpr int TERMS = 5, STEP = TERMS * 1536 + 512;      // bytes of one 64-element step of a tile
constexpr int NUM_CUS = 256;
constexpr int kMaxSplits = 64;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What a launch works on beyond the call's arguments.
struct Plan {
  int row_tiles;         // of 32 rows, a sequence at most
  int head_tiles;        // tile places of a key head: sequences next to each other
  uint8_t* terms;        // [heads][head_tiles][NS][STEP]
  float* minus_l;        // [heads][head_tiles][32]
  float2* stats;         // [splits][heads][head_tiles][32]
  int splits;
};

// Place of row tile rt of sequence b for head hk: sequences of q0 * group rows before them and a
// tile each to round up never meet.
__device__ __forceinline__ long long tile_at(const KvAttnArgs& a, const Plan& p, int b, int hk, int q0, int rt) {
  return (long long)hk * p.head_tiles + (long long)q0 * a.group / 32 + b + rt;
}

template <int NB>
__global__ void __launch_bounds__(64 * ((NB + 1) / 2))
kv_weigh_rows_kernel(KvAttnArgs a, Plan p) {
  constexpr int NS = (NB + 1) / 2;
  const int lane = threadIdx.x & 63, ds = threadIdx.x >> 6;
  const int row = lane & 31, blk = 2 * ds + (lane >> 5);
  const int hk = blockIdx.y, b = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, rr = rt * 32 + row;
  if (rt * 32 >= rows) return;
  uint8_t* to = p.terms + (tile_at(a, p, b, hk, q0, rt) * NS + ds) * STEP;
  float x[32];
  bool ok = true;
  const bool mine = rr < rows && blk < NB;
  if (mine) {
    ok = load_q_block(a, q0 + rr / a.group, hk * a.group + rr % a.group, blk, base2_scale(a), x);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = 0.0f;
  }
  float top = 0.0f, even = 0.0f, odd = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
    even += x[e];
    odd += x[e + 1];
  }
  // an infinity shows in the largest magnitude, NaN in the sums
  ok = ok && finite_f32(top) && even == even && odd == odd;
  // exponent of the first term: the block's largest element is 3.75 to 7.5 of it
  const int ex = max(mx_exponent(__uint_as_float(__float_as_uint(top) + 0x100000u)), 4 * TERMS - 131);
  uint32_t s0 = 0u, s1 = 0u;
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    const int E = ex - 4 * t + 127;
    const float s = __uint_as_float((uint32_t)E << 23);
    v16f lo, hi;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      lo[e] = x[2 * e];
      hi[e] = x[2 * e + 1];
    }
    const v6u w = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(lo, hi, s);
    if (t + 1 < TERMS) {
      const v32f d = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(w, s);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] -= d[e];
    }
    *reinterpret_cast<uint4*>(to + t * 1536 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint2*>(to + t * 1536 + 1024 + lane * 8) = make_uint2(w[4], w[5]);
    // (a row that is not finite has scales that are not a number: its scores are none either)
    const uint32_t byte = ok ? (uint32_t)E : 255u;
    if (t < 4) s0 |= byte << (8 * t);
    else s1 |= byte << (8 * (t - 4));
  }
  *reinterpret_cast<uint2*>(to + TERMS * 1536 + lane * 8) = make_uint2(s0, s1);
}

// A tile's terms in registers.
template <int NB>
struct Terms {
  static constexpr int NS = (NB + 1) / 2;
  v8i q[NS][TERMS];
  uint2 scale[NS];
  __device__ __forceinline__ void load(const uint8_t* from, int lane) {
#pragma unroll
    for (int ds = 0; ds < NS; ++ds) {
      const uint8_t* f = from + ds * STEP;
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        const uint4 w = *reinterpret_cast<const uint4*>(f + t * 1536 + lane * 16);
        const uint2 v = *reinterpret_cast<const uint2*>(f + t * 1536 + 1024 + lane * 8);
        q[ds][t] = v8i{(int)w.x, (int)w.y, (int)w.z, (int)w.w, (int)v.x, (int)v.y, 0, 0};
      }
      scale[ds] = *reinterpret_cast<const uint2*>(f + TERMS * 1536 + lane * 8);
    }
  }
};

// 32 keys as an operand: lane l has key l % 32 and, of each step, block l / 32.
template <int NB>
struct Keys {
  static constexpr int NS = (NB + 1) / 2;
  v4i codes[NS];
  uint32_t scale[NS];
  __device__ __forceinline__ void load(const KvCacheArgs& c, long long row, int lane) {
#pragma unroll
    for (int ds = 0; ds < NS; ++ds) {
      const int blk = 2 * ds + (lane >> 5);
      const bool has = NB % 2 == 0 || blk < NB;      // a block that does not exist is zeros in q'
      codes[ds] = *reinterpret_cast<const v4i*>(c.k_codes + (row * NB + (has ? blk : 0)) * 16);
      const uint32_t s = c.k_scales[row * NB + (has ? blk : 0)];
      scale[ds] = has ? s : 127u;
    }
  }
};

// acc + one term's product; KEYS: the keys are the first operand (rows of the result).
template <bool KEYS_FIRST>
__device__ __forceinline__ v16f term(v4i codes, uint32_t kscale, const v8i& q, uint2 qs, int t, v16f acc) {
  const v8i k = {codes[0], codes[1], codes[2], codes[3], 0, 0, 0, 0};
#define TABIT_TERM(T_, B_, W_)                                                                              \
  if (t == T_)                                                                                              \
    return KEYS_FIRST                                                                                       \
               ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q, acc, 4, 2, 0, (int)kscale, B_, (int)W_) \
               : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(q, k, acc, 2, 4, B_, (int)W_, 0, (int)kscale);
  TABIT_TERM(0, 0, qs.x)
  TABIT_TERM(1, 1, qs.x)
  TABIT_TERM(2, 2, qs.x)
  TABIT_TERM(3, 3, qs.x)
  TABIT_TERM(4, 0, qs.y)
#undef TABIT_TERM
  return acc;
}

// Row of the cache of key j (an existing one where there is none), and whether there is one.
__device__ __forceinline__ bool key_row(const KvAttnArgs& a, const int* table, int hk, int j, int len, long long& row) {
  const KvCacheArgs& c = a.cache;
  int page = -1;
  if (j < len) page = table[j >> c.page_shift];
  const bool there = (unsigned)page < (unsigned)c.num_pages;
  row = (((long long)(there ? page : 0) * c.heads + hk) << c.page_shift) | (there ? j & ((1 << c.page_shift) - 1) : 0);
  return there;
}

// A row that sees nothing, or something that is not a number, adds nothing.
__device__ __forceinline__ bool counts(float sum, float l) { return sum > 0.0f && finite_f32(l); }

__device__ __forceinline__ void write_lse(const KvAttnArgs& a, int q0, int hk, int rr, float sum, float l) {
  a.lse[(long long)(q0 + rr / a.group) * a.q_heads + hk * a.group + rr % a.group] =
      sum == 0.0f ? kNegInf : l * 0.6931471805599453f;
}

// Sum (relative to a reference) and L of row lane % 32 of a tile from its ranges of keys, half of
// them to each half of the wave.
__device__ __forceinline__ float join_ranges(const KvAttnArgs& a, const Plan& p, long long tile, int lane, float& l) {
  const float2* st = p.stats + tile * 32 + (lane & 31);
  const long long stride = (long long)a.cache.heads * p.head_tiles * 32;
  float ref = kLowest, sum = 0.0f;
  for (int s = lane >> 5; s < p.splits; s += 2) {
    const float2 x = st[s * stride];
    const float top = fmaxf(ref, x.x);
    sum = sum * exp2_fast(ref - top) + x.y * exp2_fast(x.x - top);
    ref = top;
  }
  const float top = fmaxf(ref, __shfl_xor(ref, 32, 64));
  sum *= exp2_fast(ref - top);
  sum += __shfl_xor(sum, 32, 64);
  l = top + __builtin_log2f(sum);
  return sum;
}

// L of the rows of one tile over one range of keys: one wave.  64 keys at a time.
template <int NB>
__global__ void __launch_bounds__(256)
kv_weigh_stats_kernel(KvAttnArgs a, Plan p) {
  constexpr int NS = (NB + 1) / 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 31, half = lane >> 5;
  // the waves of a workgroup: ranges of one tile, or tiles of one range
  const unsigned unit = blockIdx.x * 4 + wave, per = (unsigned)p.row_tiles * p.splits;
  const int b = unit / per, hk = blockIdx.y;
  if (b >= a.seqs) return;
  const int sp = unit % per % p.splits;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b);
  const int rt = (rows + 31) / 32 - 1 - (int)(unit % per / p.splits);     // those that see most first
  if (rt < 0) return;
  const int rr = rt * 32 + row;
  const bool row_ok = rr < rows;
  const int seen_hi = seen_keys(a, len, all, min(rt * 32 + 31, rows - 1) / a.group);
  const int seen = row_ok ? seen_keys(a, len, all, rr / a.group) : seen_hi;
  const int seen_lo = seen_keys(a, len, all, rt * 32 / a.group);
  const long long at = tile_at(a, p, b, hk, q0, rt);
  Terms<NB> q;
  q.load(p.terms + at * NS * STEP, lane);
  const int tiles = (int)(((unsigned)seen_hi + 63u) / 64u);
  const int share = (tiles + p.splits - 1) / p.splits;
  const int t0 = min(sp * share, tiles), t1 = min(t0 + share, tiles);
  const int* table = a.table + (long long)b * a.table_stride;

  float ref = kLowest, sum = 0.0f;
  Keys<NB> k[2];
  bool there[2];
  auto fetch = [&](int t) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      long long at_row;
      there[kb] = key_row(a, table, hk, t * 64 + kb * 32 + row, len, at_row);
      k[kb].load(a.cache, at_row, lane);
    }
  };
  if (a.cache.num_pages > 0) {
    for (int t = t0; t < t1; ++t) {
      fetch(t);
      const uint32_t in[2] = {(uint32_t)__ballot(there[0]), (uint32_t)__ballot(there[1])};
      v16f s[2] = {v16f{}, v16f{}};
#pragma unroll
      for (int ds = 0; ds < NS; ++ds)
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) s[kb] = term<true>(k[kb].codes[ds], k[kb].scale[ds], q.q[ds][i], q.scale[ds], i, s[kb]);
      // lane: keys 32 kb + 8 (r / 4) + 4 half + r % 4 of its row
      if (seen_lo - t * 64 < 64 || (in[0] & in[1]) != 0xFFFFFFFFu) {
        const int left = seen - t * 64 - 4 * half;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = 8 * (r >> 2) + (r & 3);
            if (kb * 32 + key >= left || !(in[kb] >> (key + 4 * half) & 1u)) s[kb][r] = kNegInf;
          }
      }
      float top = ref;
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(fmaxf(top, s[0][r]), s[1][r]);
      sum *= exp2_fast(ref - top);
      ref = top;
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        even += exp2_fast(s[0][r] - ref);
        odd += exp2_fast(s[1][r] - ref);
      }
      sum += even + odd;
    }
  }
  const float other = __shfl_xor(ref, 32, 64), top = fmaxf(ref, other);
  sum *= exp2_fast(ref - top);
  sum += __shfl_xor(sum, 32, 64);
  if (half != 0) return;
  if (!row_ok) sum = 0.0f;                       // (rows past the sequence's were not masked)
  if (p.splits > 1) {
    p.stats[((long long)sp * a.cache.heads * p.head_tiles + at) * 32 + row] = make_float2(top, sum);
    return;
  }
  const float l = top + __builtin_log2f(sum);
  p.minus_l[at * 32 + row] = counts(sum, l) ? -l : kNegInf;
  if (a.lse != nullptr && row_ok) write_lse(a, q0, hk, rr, sum, l);
}

// The same of rows whose ranges are joined here, where the caller asked for it.
__global__ void __launch_bounds__(64)
kv_weigh_lse_kernel(KvAttnArgs a, Plan p) {
  const int hk = blockIdx.y, b = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rr = rt * 32 + (threadIdx.x & 31);
  float l;
  const float sum = join_ranges(a, p, tile_at(a, p, b, hk, q0, min(rt, max(n * a.group - 1, 0) / 32)), threadIdx.x, l);
  if (threadIdx.x < 32 && rr < n * a.group) write_lse(a, q0, hk, rr, sum, l);
}

// Sums of KB * 32 keys a wave over all rows that see them.
template <int NB, int KB>
__global__ void __launch_bounds__(256)
kv_weigh_sums_kernel(KvAttnArgs a, Plan p, float* sums, unsigned chunks) {
  constexpr int NS = (NB + 1) / 2;
  __shared__ __attribute__((aligned(16))) float joined[4][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key = lane & 31, half = lane >> 5;
  const int b = blockIdx.x / chunks, hk = blockIdx.y;
  const int j0 = ((int)(blockIdx.x % chunks) * 4 + wave) * KB * 32;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b);
  if (j0 >= len || rows == 0 || a.cache.num_pages == 0) return;
  const int* table = a.table + (long long)b * a.table_stride;
  Keys<NB> k[KB];
  long long place[KB];
  bool there[KB], number[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    there[kb] = key_row(a, table, hk, j0 + kb * 32 + key, len, place[kb]);
    k[kb].load(a.cache, place[kb], lane);
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    uint32_t worst = 0u;
#pragma unroll
    for (int ds = 0; ds < NS; ++ds) worst = max(worst, k[kb].scale[ds]);
    number[kb] = max(worst, (uint32_t)__shfl_xor((int)worst, 32, 64)) != 255u;
  }
  // the first row that sees key j is (j - (len - all)) * group, with the causal mask
  const int old = len - all;
  int first[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const long long f = (long long)(j0 + kb * 32 + key - old) * a.group;
    first[kb] = a.causal ? (int)min(max(f, 0ll), 0x7FFFFFFFll) : 0;
  }
  const long long f0 = a.causal ? (long long)(j0 - old) * a.group : 0;
  const long long f1 = a.causal ? (long long)(min(j0 + KB * 32, len) - 1 - old) * a.group : 0;
  const int rt0 = (int)min(max(f0, 0ll), (long long)rows) / 32, rts = (rows + 31) / 32;
  float w[KB];
  const long long base = tile_at(a, p, b, hk, q0, 0);
  // Scores of rows that add nothing may be no number; they show in the sums, which are then
  // formed once more without them.
  for (bool clean = false;; clean = true) {
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) w[kb] = 0.0f;
  for (int rt = rt0; rt < rts; ++rt) {
    Terms<NB> q;
    q.load(p.terms + (base + rt) * NS * STEP, lane);
    const float* ml = p.minus_l + (base + rt) * 32;
    if (p.splits > 1) {
      float l;
      const float sum = join_ranges(a, p, base + rt, lane, l);
      if (half == 0) joined[wave][key] = counts(sum, l) ? -l : kNegInf;
      ml = joined[wave];
      __builtin_amdgcn_wave_barrier();
    }
    v16f start;          // register r: row 8 (r / 4) + 4 half + r % 4
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const v4f x = *reinterpret_cast<const v4f*>(ml + 2 * r + 4 * half);
#pragma unroll
      for (int e = 0; e < 4; ++e) start[r + e] = x[e];
    }
    __builtin_amdgcn_wave_barrier();
    const bool cut = f1 > (long long)rt * 32;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      v16f s = start;
#pragma unroll
      for (int ds = 0; ds < NS; ++ds)
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i) s = term<false>(k[kb].codes[ds], k[kb].scale[ds], q.q[ds][i], q.scale[ds], i, s);
      if (cut) {
        const int from = first[kb] - rt * 32 - 4 * half;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (8 * (r >> 2) + (r & 3) < from) s[r] = kNegInf;
      }
      if (clean) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = s[r] == s[r] ? s[r] : kNegInf;
      }
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        even += exp2_fast(s[r]);
        odd += exp2_fast(s[r + 1]);
      }
      w[kb] += even + odd;
    }
  }
  bool none = false;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) none = none || (number[kb] && w[kb] != w[kb]);
  if (clean || !__any(none)) break;
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const float total = w[kb] + __shfl_xor(w[kb], 32, 64);
    const int j = j0 + kb * 32 + key;
    if (half != 0 || !there[kb]) continue;
    const float before = a.causal && j >= old ? 0.0f : sums[place[kb]];
    sums[place[kb]] = before + (number[kb] ? total : 0.0f);
  }
}

template <int NB>
hipError_t launch_nb(const KvAttnArgs& a, const Plan& p, float* sums, hipStream_t s) {
  constexpr int NS = (NB + 1) / 2;
  const unsigned heads = (unsigned)a.cache.heads;
  kv_weigh_rows_kernel<NB><<<dim3((unsigned)p.row_tiles * a.seqs, heads), 64 * NS, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const long long units = (long long)p.row_tiles * p.splits * a.seqs;
  kv_weigh_stats_kernel<NB><<<dim3((unsigned)((units + 3) / 4), heads), 256, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (a.lse != nullptr && p.splits > 1) {
    kv_weigh_lse_kernel<<<dim3((unsigned)p.row_tiles * a.seqs, heads), 64, 0, s>>>(a, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.max_kv == 0) return hipSuccess;
  // few rows: 64 keys a wave fill the chip; many: 128 keys share a tile's terms
  if (p.row_tiles <= 4) {
    const unsigned chunks = (unsigned)((a.max_kv + 255ll) / 256);
    kv_weigh_sums_kernel<NB, 2><<<dim3(chunks * a.seqs, heads), 256, 0, s>>>(a, p, sums, chunks);
  } else {
    const unsigned chunks = (unsigned)((a.max_kv + 511ll) / 512);
    kv_weigh_sums_kernel<NB, 4><<<dim3(chunks * a.seqs, heads), 256, 0, s>>>(a, p, sums, chunks);
  }
  return hipGetLastError();
}

// Ranges of keys for the statistics: enough waves to fill the chip (four a SIMD), of at least two
// tiles each.
int splits_of(int seqs, int max_q, int q_heads, int kv_heads, int max_kv) {
  const long long rt = ((long long)max_q * (q_heads / kv_heads) + 31) / 32;
  const long long base = (long long)seqs * kv_heads * rt, tiles = ((long long)max_kv + 63) / 64;
  long long want = (16ll * NUM_CUS + base - 1) / base;
  want = want < tiles / 2 ? want : tiles / 2;
  return (int)(want < 1 ? 1 : want > kMaxSplits ? kMaxSplits : want);
}

// Places, and with a workspace the arrays in it.
size_t plan_of(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv, uint8_t* ws, Plan& p) {
  const int group = q_heads / kv_heads;
  p.row_tiles = (int)(((long long)max_q * group + 31) / 32);
  p.head_tiles = (int)((long long)tokens * group / 32 + 1 + seqs);
  p.splits = splits_of(seqs, max_q, q_heads, kv_heads, max_kv);
  const size_t tiles = (size_t)kv_heads * (size_t)p.head_tiles;
  const size_t terms = tiles * (size_t)((dim_pad + 63) / 64) * STEP, rows = tiles * 32;
  p.terms = ws;
  p.minus_l = reinterpret_cast<float*>(ws + terms);
  p.stats = reinterpret_cast<float2*>(ws + terms + rows * 4);
  return terms + rows * 4 + (p.splits > 1 ? (size_t)p.splits * rows * 8 : 0);
}

}  // namespace

size_t kv_weigh_workspace(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv) {
  Plan p;
  return plan_of(tokens, q_heads, kv_heads, dim_pad, seqs, max_q, max_kv, nullptr, p);
}

hipError_t launch_kv_weigh(const KvAttnArgs& a, float* sums, hipStream_t s) {
  Plan p;
  plan_of(a.tokens, a.q_heads, a.cache.heads, a.cache.dim_pad, a.seqs, a.max_q, a.max_kv,
          reinterpret_cast<uint8_t*>(a.part), p);
  switch (a.cache.dim_pad) {
    case 32: return launch_nb<1>(a, p, sums, s);
    case 64: return launch_nb<2>(a, p, sums, s);
    case 96: return launch_nb<3>(a, p, sums, s);
    case 128: return launch_nb<4>(a, p, sums, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tabit
