// Attention weights summed over a step's rows, per cached token and key head:
//
//   w_j += sum_i exp2(s_ij - L_i),  s_ij = c q'_i . k'_j,  L_i = log2 sum_j exp2(s_ij)
//
// with q', k', c and the visible keys as in the attention kernels.  The result is fp32 and
// stays that exact: q' is five FP6 (E2M3) terms with scales 2^e ... 2^(e-16) per block of 32
// (2^-21 of the block's largest element is lost at most), which go against the key codes
// as stored in the 32x32x64 block-scaled MFMA, and the exponentials take fp32 scores.
//
// Many rows, three kernels.  One prepares the rows, 32 a tile, once for all that read them.  The
// second passes over the keys for L: S = K Q'^T, so that a lane has one row and keeps its sum
// alone until the end.  The third passes over the keys again for the sums: S = Q' K^T, so that a
// lane has one key and adds up rows in registers; the accumulator starts at -L, so what leaves the
// matrix core goes into the exponential as it is.
//
// Up to eight rows a key head (single tokens), two kernels (one for few short sequences, `held`): the first prepares the rows by itself,
// forms the scores with a lane a key, keeps each row's largest score and sum, and leaves the scores in the
// workspace (16 or 32 bytes a key; reading the keys again would be 68 at 128 elements); the second adds up
// their exponentials.
//
// Workspace, many rows, per 32-row tile: the terms' codes, 1.5 KB each for 64 elements (lane l: row
// l % 32, block l / 32 of the step; 16 and then 8 bytes a lane), and eight bytes of scales a lane; then
// -L of each row, and with `splits` ranges of keys each one's (reference, sum).
#include <algorithm>

#include "kv_query.h"
#include "tile_common.h"

namespace tabit {
namespace {

using namespace kv;

constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e+38f;
constexpr int TERMS = 5, STEP = TERMS * 1536 + 512;      // bytes of one 64-element step of a tile
constexpr int NUM_CUS = 256;
constexpr int kMaxSplits = 64;
constexpr int kKeys = 256;       // of a workgroup of the last pass
constexpr int kHeld = 1024;      // whose scores stay in LDS

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What a launch works on beyond the call's arguments.
struct Plan {
  int row_tiles;         // of 32 rows, a sequence at most
  int head_tiles;        // tile places of a key head: sequences next to each other
  uint8_t* terms;        // [heads][head_tiles][NS][STEP]
  float* minus_l;        // [heads][head_tiles][32]
  float2* stats;         // [splits][heads][head_tiles][32]
  int splits;
  float* parts;          // [ranges][seqs][heads][pad]: sums of ranges of row tiles
  int ranges, pad;
};

// Place of row tile rt of sequence b for head hk: sequences of q0 * group rows before them and a
// tile each to round up never meet.
__device__ __forceinline__ long long tile_at(const KvAttnArgs& a, const Plan& p, int b, int hk, int q0, int rt) {
  return (long long)hk * p.head_tiles + (long long)q0 * a.group / 32 + b + rt;
}

// The terms of a block of 32 elements, given to put(t, codes) one by one, and their scale bytes.  A
// block that is not ok or not finite has scales that are not a number, and so have its row's
// scores: an infinity shows in the largest magnitude, NaN in the sums.
template <typename Put>
__device__ __forceinline__ void split_terms(float (&x)[32], bool ok, uint32_t& s0, uint32_t& s1, Put put) {
  float top = 0.0f, even = 0.0f, odd = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
    even += x[e];
    odd += x[e + 1];
  }
  ok = ok && finite_f32(top) && even == even && odd == odd;
  // exponent of the first term: the block's largest element is 3.75 to 7.5 of it
  const int ex = max(mx_exponent(__uint_as_float(__float_as_uint(top) + 0x100000u)), 4 * TERMS - 131);
  s0 = s1 = 0u;
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
    put(t, w);
    const uint32_t byte = ok ? (uint32_t)E : 255u;
    if (t < 4) s0 |= byte << (8 * t);
    else s1 |= byte << (8 * (t - 4));
  }
}

// The rows' terms, a lane a block of 32 elements (3584 rows of 32 heads x 128: 24 us, 57 MB written).
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
  uint32_t s0, s1;
  split_terms(x, ok, s0, s1, [&](int t, v6u w) {
    *reinterpret_cast<uint4*>(to + t * 1536 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint2*>(to + t * 1536 + 1024 + lane * 8) = make_uint2(w[4], w[5]);
  });
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

// Page of key j, -1 where the sequence or the table has none.
__device__ __forceinline__ int key_page(const KvAttnArgs& a, const int* table, int j, int len) {
  return j < len ? table[j >> a.cache.page_shift] : -1;
}
// Row of the cache of key j on that page (an existing one where there is none), and whether there is one.
__device__ __forceinline__ bool key_row(const KvAttnArgs& a, int page, int hk, int j, long long& row) {
  const KvCacheArgs& c = a.cache;
  const bool there = (unsigned)page < (unsigned)c.num_pages;
  row = (((long long)(there ? page : 0) * c.heads + hk) << c.page_shift) | (there ? j & ((1 << c.page_shift) - 1) : 0);
  return there;
}

// 64 keys in LDS: rows of NB 16-byte blocks, whose order within a row is turned by bits of the key so that
// the 16 rows that 16 lanes read at once spread over the banks (48-byte rows spread by themselves), and
// their scale bytes.  They come straight from memory, 16 keys an instruction: those lie in one page.
template <int NB>
struct Stage {
  uint8_t codes[64 * NB * 16];
  uint8_t scales[64 * NB];
  static __device__ __forceinline__ int turned(int key, int blk) {
    return NB == 4 ? blk ^ ((key >> 2) & 3) : NB == 2 ? blk ^ ((key >> 3) & 1) : blk;
  }
  // Asks for keys 16 group .. 16 group + 15, rows `row` .. row + 15 of the cache (a wave; row is uniform).
  __device__ __forceinline__ void bring(const KvCacheArgs& c, long long row, int group, int lane) {
    if (lane < 16 * NB)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(c.k_codes + row * NB * 16 + (lane / NB * NB + turned(lane / NB, lane % NB)) * 16),
          (__attribute__((address_space(3))) void*)(codes + group * 16 * NB * 16), 16, 0, 0);
    if (lane < 4 * NB)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(c.k_scales + row * NB + lane * 4),
                                       (__attribute__((address_space(3))) void*)(scales + group * 16 * NB), 4, 0, 0);
  }
  // Keys 32 kb .. 32 kb + 31 as an operand.
  __device__ __forceinline__ void get(Keys<NB>& k, int kb, int lane) const {
    const int key = kb * 32 + (lane & 31), half = lane >> 5;
    uint32_t w = 0u;
    if constexpr (NB == 4) w = *reinterpret_cast<const uint32_t*>(scales + key * 4) >> (8 * half);
    if constexpr (NB == 2) w = *reinterpret_cast<const uint16_t*>(scales + key * 2) >> (8 * half);
#pragma unroll
    for (int ds = 0; ds < Keys<NB>::NS; ++ds) {
      const int blk = 2 * ds + half;
      const bool has = NB % 2 == 0 || blk < NB;
      k.codes[ds] = *reinterpret_cast<const v4i*>(codes + (key * NB + turned(key, has ? blk : 0)) * 16);
      if constexpr (NB % 2 == 0) k.scale[ds] = w >> (16 * ds);
      else k.scale[ds] = has ? scales[key * NB + blk] : 127u;
    }
  }
};

// First row of the cache of the 16 keys from j on (an existing one where there is none), and how many of
// them there are.
__device__ __forceinline__ int key_rows(const KvAttnArgs& a, int page, int hk, int j, int len, long long& row) {
  const KvCacheArgs& c = a.cache;
  const bool there = (unsigned)page < (unsigned)c.num_pages;
  row = (((long long)(there ? page : 0) * c.heads + hk) << c.page_shift) | (j & ((1 << c.page_shift) - 1) & ~15);
  return there ? min(max(len - j, 0), 16) : 0;
}

// Sequence and key head of a workgroup, which are the fastest index: workgroups go to the chip's eight dies
// in turn, so those that read the same keys (and rows) share a die's L2 where the pairs are a multiple of
// eight, and at least stay together in time.
struct Pair {
  int b, hk, rest;
};
__device__ __forceinline__ Pair pair_of(const KvAttnArgs& a, unsigned id) {
  const unsigned pairs = (unsigned)a.seqs * a.cache.heads, pair = id % pairs;
  return {(int)(pair / a.cache.heads), (int)(pair % a.cache.heads), (int)(id / pairs)};
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

// L of 128 rows, 32 a wave, over one range of keys.  A tile of 64 keys comes to LDS once for all waves, 16
// keys each, while the tile before is worked on (two stages, one barrier a tile).  A wave's tile is
// 20 products, 640 cycles of a matrix core, which take a SIMD 1130 by themselves with random codes (722 with
// constant ones), 1264 with the exponentials and 1478 in here, batches of equal lengths without a mask; causal
// ragged ones 1880.  Bound there by uneven workgroups and their ends: 2.1 waves are on a SIMD of the three that
// fit, and the matrix cores are busy for 36% of the cycles where such products alone keep them so for 57%
// (2 x 2048 rows behind 6144 keys at most, 32 heads over 8: 138 us).  Level or slower: one barrier for two tiles, the chains of products
// fenced or given a priority.
template <int NB>
__global__ void __launch_bounds__(256, 3)
kv_weigh_stats_kernel(KvAttnArgs a, Plan p) {
  constexpr int NS = (NB + 1) / 2;
  __shared__ __attribute__((aligned(1024))) Stage<NB> stage[2];
  __shared__ __attribute__((aligned(16))) int held[2][4];      // of each 16 keys, how many there are
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 31, half = lane >> 5;
  const Pair pair = pair_of(a, blockIdx.x);
  const int b = pair.b, hk = pair.hk;
  const int sp = pair.rest % p.splits;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b), tiles_r = (rows + 31) / 32;
  const int rt0 = ((tiles_r + 3) / 4 - 1 - pair.rest / p.splits) * 4;    // those that see most first
  if (rt0 < 0 || rows == 0) return;
  const int rt = rt0 + wave;
  const bool mine = rt < tiles_r;
  const int rr = rt * 32 + row;
  const bool row_ok = rr < rows;
  const int seen_all = seen_keys(a, len, all, min(rt0 * 32 + 127, rows - 1) / a.group);
  const int seen_hi = mine ? seen_keys(a, len, all, min(rt * 32 + 31, rows - 1) / a.group) : 0;
  const int seen = row_ok ? seen_keys(a, len, all, rr / a.group) : seen_hi;
  const int seen_lo = mine ? seen_keys(a, len, all, rt * 32 / a.group) : 0;
  const long long at = tile_at(a, p, b, hk, q0, rt);
  Terms<NB> q;
  if (mine) q.load(p.terms + at * NS * STEP, lane);
  const int tiles = (int)(((unsigned)seen_all + 63u) / 64u);
  const int share = (tiles + p.splits - 1) / p.splits;
  const int t0 = min(sp * share, tiles), t1 = a.cache.num_pages > 0 ? min(t0 + share, tiles) : t0;
  const int* table = a.table + (long long)b * a.table_stride;

  // Weights are 2^(s - ref): ref stays 0 while a lane's first tile has a largest score within +-40 and
  // its tiles sum up to less than 2^60, so that a tile needs no maximum.
  float ref = 0.0f, sum = 0.0f;
  bool fresh = true, any_fresh = true, any_ref = false;
  auto raise = [&](v16f (&s)[2], bool over) {
    float top = kNegInf;
    asm volatile("" : "+v"(top));                // (else the compiler takes the maximum of every tile)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(fmaxf(top, s[0][r]), s[1][r]);
    const bool first = fresh && top > kNegInf;
    fresh = fresh && !first;
    any_fresh = __any(fresh);
    const float by = (first ? fabsf(top) > 40.0f : over && top > 0.0f) ? top : 0.0f;
    sum *= exp2_fast(first ? 0.0f : -by);
    ref += by;
    any_ref = __any(ref != 0.0f);
    if (__any(by != 0.0f)) {
      s[0] -= by;
      s[1] -= by;
    }
  };
  int page = -1;
  auto pages = [&](int t) {
    const int j = (int)((unsigned)t * 64u) + wave * 16;
    page = t < t1 && j < len ? table[j >> a.cache.page_shift] : -1;
  };
  auto bring = [&](int t) {
    if (t >= t1) return;
    long long at_row;
    const int got = key_rows(a, __builtin_amdgcn_readfirstlane(page), hk, t * 64 + wave * 16, len, at_row);
    stage[(t - t0) & 1].bring(a.cache, at_row, wave, lane);
    if (lane == 0) held[(t - t0) & 1][wave] = got;
  };
  pages(t0);
  bring(t0);
  pages(t0 + 1);
  for (int t = t0; t < t1; ++t) {
    tile::wait_vmcnt0();
    tile::lds_barrier();
    bring(t + 1);
    pages(t + 2);
    if (t * 64 >= seen_hi) continue;
    const Stage<NB>& st = stage[(t - t0) & 1];
    Keys<NB> k[2];
    st.get(k[0], 0, lane);
    st.get(k[1], 1, lane);
    const int4 got = *reinterpret_cast<const int4*>(held[(t - t0) & 1]);
    v16f s[2] = {v16f{}, v16f{}};
#pragma unroll
    for (int ds = 0; ds < NS; ++ds)
#pragma unroll
      for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) s[kb] = term<true>(k[kb].codes[ds], k[kb].scale[ds], q.q[ds][i], q.scale[ds], i, s[kb]);
    if (any_ref) {
      s[0] -= ref;
      s[1] -= ref;
    }
    // lane: keys 32 kb + 8 (r / 4) + 4 half + r % 4 of its row
    if (seen_lo - t * 64 < 64 || got.x + got.y + got.z + got.w != 64) {
      const int left = seen - t * 64 - 4 * half;
      const int in[4] = {got.x - 4 * half, got.y - 4 * half, got.z - 4 * half, got.w - 4 * half};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = 8 * (r >> 2) + (r & 3);
          if (kb * 32 + key >= left || (key & 15) >= in[kb * 2 + (key >> 4)]) s[kb][r] = kNegInf;
        }
    }
    bool over = false;
    float tile;
    for (int pass = 0; pass < 2; ++pass) {
      if (pass == 1 || any_fresh) raise(s, over);
      float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        w[0] += exp2_fast(s[0][r]);
        w[1] += exp2_fast(s[1][r]);
        w[2] += exp2_fast(s[0][r + 1]);
        w[3] += exp2_fast(s[1][r + 1]);
      }
      tile = (w[0] + w[1]) + (w[2] + w[3]);
      over = !(tile < 0x1p60f);
      if (!__any(over)) break;
    }
    sum += tile;
  }
  if (!mine) return;
  if (fresh) ref = kLowest;                      // no key of this range
  const float top = fmaxf(ref, __shfl_xor(ref, 32, 64));
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

// The same of rows whose ranges are joined here, four tiles a workgroup.
__global__ void __launch_bounds__(256)
kv_weigh_join_kernel(KvAttnArgs a, Plan p) {
  const int lane = threadIdx.x & 63;
  const int hk = blockIdx.y, b = blockIdx.x / ((p.row_tiles + 3) / 4);
  const int rt = blockIdx.x % ((p.row_tiles + 3) / 4) * 4 + (threadIdx.x >> 6);
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rr = rt * 32 + (lane & 31);
  if (rt * 32 >= n * a.group) return;
  float l;
  const long long tile = tile_at(a, p, b, hk, q0, rt);
  const float sum = join_ranges(a, p, tile, lane, l);
  if (lane >= 32) return;
  p.minus_l[tile * 32 + lane] = counts(sum, l) ? -l : kNegInf;
  if (a.lse != nullptr && rr < n * a.group) write_lse(a, q0, hk, rr, sum, l);
}

// Sums of 64 keys a wave over all rows that see them; bound as the statistics (150 us there, matrix cores busy for
// 34% of the cycles, 2.2 waves on a SIMD of four).  (128 keys a wave take
// 208 registers and leave two waves a SIMD: 415 us for 315, long prompts, the whole call; a tile's terms in
// registers, not read from LDS for every product, 64 and 128 keys a wave, 166 and 172 us for 147, this kernel.)  The workgroup's waves go over the row
// tiles together: a tile's terms come to LDS once for all, straight from memory, while the tile before is
// worked on (two stages, one barrier a tile).  With more than one range of row tiles, sums
// go to the workspace and are added up by a kernel of their own.
template <int NB>
__global__ void __launch_bounds__(256, 4)
kv_weigh_sums_kernel(KvAttnArgs a, Plan p, float* sums) {
  constexpr int NS = (NB + 1) / 2, BYTES = NS * STEP, KB = 2;
  __shared__ __attribute__((aligned(1024))) uint8_t stage[2][BYTES];
  __shared__ __attribute__((aligned(16))) float minus_l[2][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key = lane & 31, half = lane >> 5;
  const Pair pair = pair_of(a, blockIdx.x);
  const int b = pair.b, hk = pair.hk;
  const int range = pair.rest % p.ranges, chunk = pair.rest / p.ranges;
  static_assert(4 * KB * 32 == kKeys, "four waves");
  const int j00 = chunk * kKeys, j0 = j00 + wave * KB * 32;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b);
  if (j00 >= len || rows == 0 || a.cache.num_pages == 0) return;
  const int* table = a.table + (long long)b * a.table_stride;
  Keys<NB> k[KB];
  long long place[KB];
  bool there[KB], number[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int j = j0 + kb * 32 + key;
    there[kb] = key_row(a, key_page(a, table, j, len), hk, j, place[kb]);
    k[kb].load(a.cache, place[kb], lane);
  }
  // the first row that sees key j is (j - (len - all)) * group, with the causal mask
  const int old = len - all;
  auto first_row = [&](int j) {
    return a.causal ? (int)min((long long)max(j - old, 0) * a.group, 0x7FFFFFFFll) : 0;
  };
  int first[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) first[kb] = first_row(j0 + kb * 32 + key);
  // of the workgroup's and of the wave's keys: the first tile that sees one, and of the wave's the first
  // row that sees all
  const int seen0 = min(first_row(j00), rows) / 32, tiles = (rows + 31) / 32;
  const int rt0 = seen0 + (int)((long long)(tiles - seen0) * range / p.ranges);
  const int rts = seen0 + (int)((long long)(tiles - seen0) * (range + 1) / p.ranges);
  const int mine = j0 < len ? min(first_row(j0), rows) / 32 : rts;
  const int whole = first_row(min(j0 + KB * 32, len) - 1);
  const long long base = tile_at(a, p, b, hk, q0, 0);
  auto bring = [&](int rt) {
    if (rt >= rts) return;
    const uint8_t* from = p.terms + (base + rt) * BYTES;
#pragma unroll
    for (int i = 0; i < BYTES / 1024 / 4; ++i)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(from + (i * 4 + wave) * 1024 + lane * 16),
          (__attribute__((address_space(3))) void*)(stage[(rt - rt0) & 1] + (i * 4 + wave) * 1024), 16, 0, 0);
    if (wave == 0 && lane < 32)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(p.minus_l + (base + rt) * 32 + lane),
                                       (__attribute__((address_space(3))) void*)minus_l[(rt - rt0) & 1], 4, 0, 0);
  };
  float w[KB];
  // Scores of rows that add nothing may be no number; they show in the sums, which are then
  // formed once more without them (by all waves, for their barriers).
  for (bool clean = false;; clean = true) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) w[kb] = 0.0f;
    bring(rt0);
    for (int rt = rt0; rt < rts; ++rt) {
      tile::wait_vmcnt0();
      tile::lds_barrier();
      bring(rt + 1);
      if (rt < mine) continue;
      v16f start;        // -L.  Register r: row 8 (r / 4) + 4 half + r % 4
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const v4f x = *reinterpret_cast<const v4f*>(minus_l[(rt - rt0) & 1] + 2 * r + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) start[r + e] = x[e];
      }
      const uint8_t* st = stage[(rt - rt0) & 1];
      uint2 qs[NS];
#pragma unroll
      for (int ds = 0; ds < NS; ++ds) qs[ds] = *reinterpret_cast<const uint2*>(st + ds * STEP + TERMS * 1536 + lane * 8);
      v16f s[KB];
#pragma unroll
      for (int ds = 0; ds < NS; ++ds)
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i) {
          const uint8_t* f = st + ds * STEP + i * 1536;
          const uint4 x = *reinterpret_cast<const uint4*>(f + lane * 16);
          const uint2 y = *reinterpret_cast<const uint2*>(f + 1024 + lane * 8);
          const v8i q = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, 0, 0};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            s[kb] = term<false>(k[kb].codes[ds], k[kb].scale[ds], q, qs[ds], i, ds == 0 && i == TERMS - 1 ? start : s[kb]);
        }
      const bool cut = whole > rt * 32;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (cut) {
          const int from = first[kb] - rt * 32 - 4 * half;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (8 * (r >> 2) + (r & 3) < from) s[kb][r] = kNegInf;
        }
        if (clean) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[kb][r] = s[kb][r] == s[kb][r] ? s[kb][r] : kNegInf;
        }
        float even = 0.0f, odd = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          even += exp2_fast(s[kb][r]);
          odd += exp2_fast(s[kb][r + 1]);
        }
        w[kb] += even + odd;
      }
    }
    // (a key that is no number itself gets nothing)
    bool none = false;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t worst = 0u;
#pragma unroll
      for (int ds = 0; ds < NS; ++ds) worst = max(worst, k[kb].scale[ds] & 255u);
      number[kb] = max(worst, (uint32_t)__shfl_xor((int)worst, 32, 64)) != 255u;
      none = none || (number[kb] && w[kb] != w[kb]);
    }
    if (clean || !__syncthreads_or(none)) break;
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const float total = w[kb] + __shfl_xor(w[kb], 32, 64);
    const int j = j0 + kb * 32 + key;
    if (half != 0 || !there[kb]) continue;
    const float add = number[kb] ? total : 0.0f;
    if (p.ranges > 1) {
      p.parts[(((long long)range * a.seqs + b) * a.cache.heads + hk) * p.pad + j] = add;
    } else {
      sums[place[kb]] = (a.causal && j >= old ? 0.0f : sums[place[kb]]) + add;
    }
  }
}

// Adds the ranges' parts to the sums, in their order, four keys a thread.
__global__ void __launch_bounds__(256)
kv_weigh_parts_kernel(KvAttnArgs a, Plan p, float* sums, unsigned chunks) {
  const int b = blockIdx.x / chunks, hk = blockIdx.y;
  const int j = ((int)(blockIdx.x % chunks) * 256 + (int)threadIdx.x) * 4;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int len = seq_keys(a, b);
  if (n == 0 || j >= len) return;
  const KvCacheArgs& c = a.cache;
  const int page = a.table[(long long)b * a.table_stride + (j >> c.page_shift)];
  if ((unsigned)page >= (unsigned)c.num_pages) return;
  v4f w = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < p.ranges; ++i)
    w += *reinterpret_cast<const v4f*>(p.parts + (((long long)i * a.seqs + b) * c.heads + hk) * p.pad + j);
  v4f* to = reinterpret_cast<v4f*>(sums + ((((long long)page * c.heads + hk) << c.page_shift) |
                                           (j & ((1 << c.page_shift) - 1))));
  v4f x = *to;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < len) x[e] = (a.causal && j + e >= len - all ? 0.0f : x[e]) + w[e];
  *to = x;
}

// ------------------------------------------------------------------ up to eight rows
struct FewPlan {
  int pad;               // keys that the scores have room for, a sequence
  float* scores;         // [seqs][heads][pad][R], R = 4 or 8
  float2* stats;         // [seqs][heads][splits][8]
  int splits;
};

// The tiles of 64 keys of split sp: a sequence has as many splits as its length needs at the
// share of the longest one there may be.
__device__ __forceinline__ void few_range(const KvAttnArgs& a, int splits, int len, int sp, int& t0, int& t1) {
  const int most = (int)(((unsigned)a.max_kv + 63u) / 64u), share = max((most + splits - 1) / splits, 1);
  const int tiles = (int)(((unsigned)len + 63u) / 64u);
  t0 = min(sp * share, tiles);
  t1 = min(t0 + share, tiles);
}

// Scores of a range of keys of one key head, and each row's (reference, sum) over it.  Its tiles go
// to the waves in runs.  Bound by the keys' bytes and by the longest sequences, which end alone: a wave has two
// tiles on their way to its own LDS while it works on a third (64 rows of up to 8192 keys, 8 key heads of 128:
// 54 us, 4.2 TB/s with the scores that go out).  Level or slower: a third tile on its way, heads as the fastest
// index, four rows held twice so that each half of a wave weighs half of a tile's keys (59 us).
// HELD: at most kHeld keys, whose scores stay in LDS and whose weights this kernel adds up, too.
template <int NB, int R, bool HELD>
__global__ void __launch_bounds__(HELD ? 512 : 256)
kv_weigh_scores_kernel(KvAttnArgs a, FewPlan p, float* sums) {
  constexpr int NS = (NB + 1) / 2, NW = HELD ? 8 : 4, STAGES = 3;
  __shared__ __attribute__((aligned(16))) float held_scores[HELD ? kHeld * R : 1];
  __shared__ float minus_l[8];
  __shared__ __attribute__((aligned(16))) uint32_t terms[TERMS][NB][8][6];
  __shared__ uint2 term_scales[NB][8];
  __shared__ float2 part[NW][8];
  __shared__ __attribute__((aligned(1024))) Stage<NB> stage[NW][STAGES];
  __shared__ int held[NW][STAGES][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key = lane & 31, half = lane >> 5;
  const int hk = blockIdx.y, b = blockIdx.x / p.splits, sp = blockIdx.x % p.splits;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b);
  if (rows == 0) return;
  float2* stats = p.stats + (((long long)b * a.cache.heads + hk) * p.splits + sp) * 8;
  int t0, t1;
  few_range(a, p.splits, len, sp, t0, t1);
  if (t0 >= t1 || a.cache.num_pages == 0) {
    if constexpr (HELD) {
      if (a.lse != nullptr && (int)threadIdx.x < rows) write_lse(a, q0, hk, threadIdx.x, 0.0f, 0.0f);
    } else if (threadIdx.x < 8) {
      stats[threadIdx.x] = make_float2(kLowest, 0.0f);
    }
    return;
  }
  const int per = (t1 - t0 + NW - 1) / NW;
  const int w0 = min(t0 + wave * per, t1), w1 = min(w0 + per, t1);
  const int* table = a.table + (long long)b * a.table_stride;

  // Where the keys of 16 tiles lie, a lane 16 keys, and how many of those there are: one wait for 16 tiles
  // (a load whose wait falls between the tiles' would make each wait for all before it).
  uint32_t at_lo = 0u, at_hi = 0u;
  int got = 0;
  auto bring = [&](int t) {
    if (t >= w1) return;
    const int in = (t - w0) & 15;
    if (in == 0) {
      const int j = (int)((unsigned)(t + (lane >> 2)) * 64u) + 16 * (lane & 3);
      long long row;
      got = key_rows(a, t + (lane >> 2) < w1 && j < len ? table[j >> a.cache.page_shift] : -1, hk, j, len, row);
      at_lo = (uint32_t)row;
      at_hi = (uint32_t)(row >> 32);
    }
    if ((lane >> 2) == in) held[wave][(t - w0) % STAGES][lane & 3] = got;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const long long row = (long long)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)at_hi, in * 4 + g) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)at_lo, in * 4 + g));
      stage[wave][(t - w0) % STAGES].bring(a.cache, row, g, lane);
    }
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) bring(w0 + i);
  // the rows, a lane a block of one, through LDS to the operand's lanes
  for (int i = threadIdx.x; i < 8 * NB; i += NW * 64) {
    const int row = i & 7, blk = i >> 3;
    float x[32];
    bool ok = true;
    if (row < rows) {
      ok = load_q_block(a, q0 + row / a.group, hk * a.group + row % a.group, blk, base2_scale(a), x);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = 0.0f;
    }
    uint32_t s0, s1;
    split_terms(x, ok, s0, s1, [&](int t, v6u w) {
#pragma unroll
      for (int e = 0; e < 6; ++e) terms[t][blk][row][e] = w[e];
    });
    term_scales[blk][row] = make_uint2(s0, s1);
  }
  __syncthreads();
  Terms<NB> q;
#pragma unroll
  for (int ds = 0; ds < NS; ++ds) {
    const int blk = 2 * ds + half;
    const bool mine = key < 8 && blk < NB;       // (as an operand's lane: row l % 32)
    q.scale[ds] = mine ? term_scales[blk][key] : make_uint2(0x7F7F7F7Fu, 0x7Fu);
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      q.q[ds][t] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
      if (mine) {
        const uint32_t* w = terms[t][blk][key];
        q.q[ds][t] = v8i{(int)w[0], (int)w[1], (int)w[2], (int)w[3], (int)w[4], (int)w[5], 0, 0};
      }
    }
  }

  // (of its own keys a thread has place and sum on their way)
  constexpr int OWN = HELD ? kHeld / (NW * 64) : 1;
  long long place[OWN];
  float before[OWN];
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int j = i * NW * 64 + (int)threadIdx.x;
      const bool there = key_row(a, key_page(a, table, j, len), hk, j, place[i]);
      before[i] = there && !(a.causal && j >= len - all) ? sums[place[i]] : 0.0f;
      if (!there) place[i] = -1;
    }
  }

  // register r: row 4 half + r
  float* scores = p.scores + ((long long)b * a.cache.heads + hk) * p.pad * R;
  const int old = len - all;
  float ref[4], sum[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    ref[r] = kLowest;
    sum[r] = 0.0f;
  }
  for (int t = w0; t < w1; ++t) {
    // a tile is asked for by eight instructions, and those of the tile after it may be on their way
    if (t + 1 < w1) tile::wait_vmcnt<8>();
    else tile::wait_vmcnt0();
    __builtin_amdgcn_wave_barrier();
    const int at_stage = (t - w0) % STAGES;
    Keys<NB> k[2];
    stage[wave][at_stage].get(k[0], 0, lane);
    stage[wave][at_stage].get(k[1], 1, lane);
    const int there[2] = {held[wave][at_stage][key >> 4], held[wave][at_stage][2 + (key >> 4)]};
    bring(t + 2);                                // (to the stage that the last tile left)
    float s[2][4];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      v16f x = v16f{};
#pragma unroll
      for (int ds = 0; ds < NS; ++ds)
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i) x = term<false>(k[kb].codes[ds], k[kb].scale[ds], q.q[ds][i], q.scale[ds], i, x);
      const int j = t * 64 + kb * 32 + key;
      const int first = a.causal ? min(max(j - old, 0), 8) * a.group : 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) s[kb][r] = (key & 15) < there[kb] && 4 * half + r >= first ? x[r] : kNegInf;
      if (4 * half < R) {
        const v4f w = {s[kb][0], s[kb][1], s[kb][2], s[kb][3]};
        if constexpr (HELD) *reinterpret_cast<v4f*>(held_scores + j * R + 4 * half) = w;
        else *reinterpret_cast<v4f*>(scores + (long long)j * R + 4 * half) = w;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float top = fmaxf(fmaxf(ref[r], s[0][r]), s[1][r]);
      sum[r] = sum[r] * exp2_fast(ref[r] - top) + (exp2_fast(s[0][r] - top) + exp2_fast(s[1][r] - top));
      ref[r] = top;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      const float top = fmaxf(ref[r], __shfl_xor(ref[r], m, 64));
      sum[r] *= exp2_fast(ref[r] - top);
      sum[r] += __shfl_xor(sum[r], m, 64);
      ref[r] = top;
    }
    if (key == 0) part[wave][4 * half + r] = make_float2(ref[r], sum[r]);
  }
  __syncthreads();
  if (threadIdx.x < 8) {
    float top = kLowest, total = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, part[w][threadIdx.x].x);
#pragma unroll
    for (int w = 0; w < NW; ++w) total += part[w][threadIdx.x].y * exp2_fast(part[w][threadIdx.x].x - top);
    if constexpr (HELD) {
      const float l = top + __builtin_log2f(total);
      minus_l[threadIdx.x] = (int)threadIdx.x < rows && counts(total, l) ? -l : kNegInf;
      if (a.lse != nullptr && (int)threadIdx.x < rows) write_lse(a, q0, hk, threadIdx.x, total, l);
    } else {
      stats[threadIdx.x] = make_float2(top, total);
    }
  }
  if constexpr (HELD) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld / (NW * 64); ++i) {
      const int j = i * NW * 64 + (int)threadIdx.x;
      if (place[i] < 0) continue;
      float w = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r)                // (as below)
        w += minus_l[r] == kNegInf ? 0.0f : exp2_fast(held_scores[j * R + r] + minus_l[r]);
      sums[place[i]] = before[i] + w;
    }
  }
}

// Adds the exponentials of those scores to the sums, a key a thread four times.
template <int R>
__global__ void __launch_bounds__(256)
kv_weigh_add_kernel(KvAttnArgs a, FewPlan p, float* sums, unsigned chunks) {
  __shared__ float2 part[32][8];
  __shared__ float minus_l[8];
  const int b = blockIdx.x / chunks, hk = blockIdx.y;
  const int chunk = (int)(blockIdx.x % chunks);
  const int j0 = chunk * 1024 + (int)threadIdx.x;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group, len = seq_keys(a, b);
  if (rows == 0 || (chunk * 1024 >= len && !(a.lse != nullptr && chunk == 0))) return;
  const KvCacheArgs& c = a.cache;
  v4f s[4][R / 4];
  int page[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + i * 256;
    page[i] = -1;
    if (j < len) {
      page[i] = a.table[(long long)b * a.table_stride + (j >> c.page_shift)];
      const v4f* from = reinterpret_cast<const v4f*>(p.scores + (((long long)b * c.heads + hk) * p.pad + j) * R);
#pragma unroll
      for (int r = 0; r < R / 4; ++r) s[i][r] = from[r];
    }
  }
  const float2* st = p.stats + ((long long)b * c.heads + hk) * p.splits * 8;
  const int row = threadIdx.x & 7;
  float ref = kLowest, sum = 0.0f;
  for (int i = threadIdx.x >> 3; i < p.splits; i += 32) {
    const float2 x = st[i * 8 + row];
    const float top = fmaxf(ref, x.x);
    sum = sum * exp2_fast(ref - top) + x.y * exp2_fast(x.x - top);
    ref = top;
  }
  part[threadIdx.x >> 3][row] = make_float2(ref, sum);
  __syncthreads();
  if (threadIdx.x < 8) {
    const int used = min(p.splits, 32);
    float top = kLowest, total = 0.0f;
    for (int i = 0; i < used; ++i) top = fmaxf(top, part[i][row].x);
    for (int i = 0; i < used; ++i) total += part[i][row].y * exp2_fast(part[i][row].x - top);
    const float l = top + __builtin_log2f(total);
    minus_l[row] = row < rows && counts(total, l) ? -l : kNegInf;
    if (a.lse != nullptr && chunk == 0 && row < rows) write_lse(a, q0, hk, row, total, l);
  }
  __syncthreads();
  const int old = len - all;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + i * 256;
    if ((unsigned)page[i] >= (unsigned)c.num_pages) continue;
    float w = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)                  // (the scores of a row that adds nothing may be no number)
      w += minus_l[r] == kNegInf ? 0.0f : exp2_fast(s[i][r / 4][r % 4] + minus_l[r]);
    float* to = sums + ((((long long)page[i] * c.heads + hk) << c.page_shift) | (j & ((1 << c.page_shift) - 1)));
    *to = (a.causal && j >= old ? 0.0f : *to) + w;
  }
}

// The first row past eight is a step: 64 sequences of 8 and 12 rows a key head x up to 8192 keys 96 and 169 us (8
// key heads of 128), one of 8 and 16 x 1000 keys 11.8 and 19.6.
bool few_rows(const KvAttnArgs& a) { return (long long)a.max_q * a.group <= 8; }

// Ranges of keys: two workgroups a CU, of at least four tiles (one a wave) each.  A workgroup spends about 5 us
// on its start, most of it on the rows' terms, so more of them cost more than they balance (64 rows of up to
// 8192 keys, both kernels: 71 us unsplit, 74 in halves, 79 in thirds, 107 in eighths).
int few_splits(int seqs, int kv_heads, int max_kv) {
  const long long base = (long long)seqs * kv_heads, tiles = ((long long)max_kv + 63) / 64;
  long long want = (2ll * NUM_CUS + base - 1) / base;
  const long long most = (tiles + 3) / 4;
  want = want < most ? want : most;
  return (int)(want < 1 ? 1 : want > 128 ? 128 : want);
}

size_t few_plan_of(int seqs, int kv_heads, int rows, int max_kv, uint8_t* ws, FewPlan& p) {
  const size_t heads = (size_t)seqs * (size_t)kv_heads;
  p.pad = (int)(((long long)max_kv + 63) / 64 * 64);
  p.splits = few_splits(seqs, kv_heads, max_kv);
  const size_t scores = heads * (size_t)p.pad * (rows <= 4 ? 16 : 32);
  p.scores = reinterpret_cast<float*>(ws);
  p.stats = reinterpret_cast<float2*>(ws + scores);
  return scores + heads * (size_t)p.splits * 64;
}

// One kernel for short sequences while each (sequence, key head) has a CU to itself (8 waves; of 128 elements 123 KB of
// LDS with up to four rows, 139 KB with eight).
// Measured under a graph, two kernels and one, 8 key heads of 128: one row x 1000 keys 12.4 and 10.5 us, x 200 10.5
// and 8.6, 16 of 700 (64 elements, 16 heads) 14.5 and 10.1; 64 rows x 1000 18.7 and 19.7, 256 x 500 40 and 60.
bool held(const KvAttnArgs& a) { return a.max_kv <= kHeld && (long long)a.seqs * a.cache.heads <= NUM_CUS; }

template <int NB, int R>
hipError_t launch_few(const KvAttnArgs& a, float* sums, hipStream_t s) {
  const unsigned heads = (unsigned)a.cache.heads;
  if (held(a)) {
    kv_weigh_scores_kernel<NB, R, true><<<dim3((unsigned)a.seqs, heads), 512, 0, s>>>(a, FewPlan{0, nullptr, nullptr, 1}, sums);
    return hipGetLastError();
  }
  FewPlan p;
  few_plan_of(a.seqs, a.cache.heads, R, a.max_kv, reinterpret_cast<uint8_t*>(a.part), p);
  kv_weigh_scores_kernel<NB, R, false><<<dim3((unsigned)(p.splits * a.seqs), heads), 256, 0, s>>>(a, p, sums);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const unsigned chunks = max((unsigned)((a.max_kv + 1023ll) / 1024), 1u);
  kv_weigh_add_kernel<R><<<dim3(chunks * a.seqs, heads), 256, 0, s>>>(a, p, sums, chunks);
  return hipGetLastError();
}

// ------------------------------------------------------------------ more rows
template <int NB>
hipError_t launch_nb(const KvAttnArgs& a, const Plan& p, float* sums, hipStream_t s) {
  constexpr int NS = (NB + 1) / 2;
  const unsigned heads = (unsigned)a.cache.heads;
  kv_weigh_rows_kernel<NB><<<dim3((unsigned)p.row_tiles * a.seqs, heads), 64 * NS, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const unsigned pairs = heads * (unsigned)a.seqs;
  kv_weigh_stats_kernel<NB><<<(unsigned)(p.row_tiles + 3) / 4 * p.splits * pairs, 256, 0, s>>>(a, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (p.splits > 1) {
    kv_weigh_join_kernel<<<dim3((unsigned)((p.row_tiles + 3) / 4) * a.seqs, heads), 256, 0, s>>>(a, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.max_kv == 0) return hipSuccess;
  const unsigned chunks = (unsigned)(((long long)a.max_kv + kKeys - 1) / kKeys);
  kv_weigh_sums_kernel<NB><<<chunks * pairs * (unsigned)p.ranges, 256, 0, s>>>(a, p, sums);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess || p.ranges == 1) return e;
  const unsigned more = (unsigned)((a.max_kv + 1023ll) / 1024);
  kv_weigh_parts_kernel<<<dim3(more * a.seqs, heads), 256, 0, s>>>(a, p, sums, more);
  return hipGetLastError();
}

// Ranges of keys for the statistics and of row tiles for the sums: eight workgroups a CU (two or three
// rounds, so that a causal batch's unequal ones level out), of at least two tiles of keys and eight of
// rows.  Measured, 2 x up to 2048 rows behind up to 6144 keys, 32 heads over 8: sums in 1, 2, 4, 8 and 16
// workgroups a CU 550, 344, 322, 315 and 316 us for the whole call, statistics in 4, 8 and 16 level.
void ranges_of(int seqs, int kv_heads, int max_kv, Plan& p) {
  const long long base = (long long)seqs * kv_heads, tiles = ((long long)max_kv + 63) / 64;
  auto between = [](long long x, long long lo, long long hi) { return (int)(x < lo ? lo : x > hi ? hi : x); };
  const long long wide = base * ((p.row_tiles + 3) / 4);
  p.splits = between((8 * NUM_CUS + wide - 1) / wide, 1, between(tiles / 2, 1, kMaxSplits));
  const long long groups = base * std::max(((long long)max_kv + kKeys - 1) / kKeys, 1ll);
  p.ranges = between((8 * NUM_CUS + groups - 1) / groups, 1, between(p.row_tiles / 8, 1, 16));
}

// Places, and with a workspace the arrays in it.
size_t plan_of(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv, uint8_t* ws, Plan& p) {
  const int group = q_heads / kv_heads;
  p.row_tiles = (int)(((long long)max_q * group + 31) / 32);
  p.head_tiles = (int)((long long)tokens * group / 32 + 1 + seqs);
  ranges_of(seqs, kv_heads, max_kv, p);
  p.pad = (int)(((long long)max_kv + 3) / 4 * 4);
  const size_t tiles = (size_t)kv_heads * (size_t)p.head_tiles;
  const size_t terms = tiles * (size_t)((dim_pad + 63) / 64) * STEP, rows = tiles * 32;
  const size_t stats = p.splits > 1 ? (size_t)p.splits * rows * 8 : 0;
  p.terms = ws;
  p.minus_l = reinterpret_cast<float*>(ws + terms);
  p.stats = reinterpret_cast<float2*>(ws + terms + rows * 4);
  p.parts = reinterpret_cast<float*>(ws + terms + rows * 4 + stats);
  return terms + rows * 4 + stats +
         (p.ranges > 1 ? (size_t)p.ranges * (size_t)seqs * (size_t)kv_heads * (size_t)p.pad * 4 : 0);
}

}  // namespace

bool kv_weigh_fits(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv) {
  const long long most = (1ll << 24) - 1;        // workgroups of 256 threads: 2^32 threads are the limit
  const long long pairs = (long long)seqs * kv_heads;
  if ((long long)max_q * (q_heads / kv_heads) <= 8) {
    FewPlan p;
    few_plan_of(seqs, kv_heads, 8, max_kv, nullptr, p);
    return (long long)p.splits * seqs <= most && ((long long)max_kv / 1024 + 1) * seqs <= most;
  }
  if ((long long)tokens * (q_heads / kv_heads) / 32 + 1 + seqs > 0x7FFFFFFF) return false;    // tile places of a head
  Plan p;
  plan_of(tokens, q_heads, kv_heads, dim_pad, seqs, max_q, max_kv, nullptr, p);
  return (long long)p.row_tiles * seqs <= most && ((p.row_tiles + 3ll) / 4) * p.splits * pairs <= most &&
         ((long long)max_kv / kKeys + 1) * pairs * p.ranges <= most && ((long long)max_kv / 1024 + 1) * seqs <= most;
}

size_t kv_weigh_workspace(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv) {
  const long long rows = (long long)max_q * (q_heads / kv_heads);
  if (rows <= 8) {
    FewPlan p;
    return few_plan_of(seqs, kv_heads, (int)rows, max_kv, nullptr, p);
  }
  Plan p;
  return plan_of(tokens, q_heads, kv_heads, dim_pad, seqs, max_q, max_kv, nullptr, p);
}

template <int NB>
static hipError_t launch_weigh(const KvAttnArgs& a, float* sums, hipStream_t s) {
  if (few_rows(a)) {
    return a.max_q * a.group <= 4 ? launch_few<NB, 4>(a, sums, s) : launch_few<NB, 8>(a, sums, s);
  }
  Plan p;
  plan_of(a.tokens, a.q_heads, a.cache.heads, a.cache.dim_pad, a.seqs, a.max_q, a.max_kv,
          reinterpret_cast<uint8_t*>(a.part), p);
  return launch_nb<NB>(a, p, sums, s);
}

hipError_t launch_kv_weigh(const KvAttnArgs& a, float* sums, hipStream_t s) {
  switch (a.cache.dim_pad) {
    case 32: return launch_weigh<1>(a, sums, s);
    case 64: return launch_weigh<2>(a, sums, s);
    case 96: return launch_weigh<3>(a, sums, s);
    case 128: return launch_weigh<4>(a, sums, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tabit
