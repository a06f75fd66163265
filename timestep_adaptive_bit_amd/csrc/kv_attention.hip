// Attention over the paged MXFP4 cache.
//
//   s_j = c q'.k'_j,  p_j = softmax over the visible keys,  o = (1/32) H32 sum_j p_j v'_j
//
// with q' = H32 R(pos) q padded to blocks of 32 (H32 and the 1/32 only for a
// rotated cache: H32 H32 = 32, so c = scale / 32 and the output is turned back
// once per row).  Keys j < len are visible, with `causal` also only j <= len - n + i
// to query i of the n of a sequence.  A row that sees no key answers 0.
//
// Trees of drafted tokens (TREE) see by a mask: of the last n keys of a sequence those whose bit is set in the
// row's words, 64 of which are lined up with a tile of 64 keys by two loads and a shift, and every key before
// them.  Only tiles that reach into the tree look at it, so it costs nothing beside the rest.
//
// Rows of one key head are packed as (query, head of the group), so the heads
// that share keys share every byte read of them.  A wave takes 64 keys at a time
// and 16 rows:
//
//   scores  S = K Q'^T with the 16x16x128 block-scaled MFMA: the key codes go from
//           memory into the matrix core as they are stored (lane l holds one MX
//           block: key l%16, block l/16), scaled by their E8M0 bytes in the
//           instruction.  q' is three FP6 (E2M3) terms with scales 2^e, 2^(e-4),
//           2^(e-8) per block of 32, e such that the block's largest element is 3.75 to
//           7.5 of 2^e (7.5 is the largest E2M3): what is left of an element is at most
//           2^-12 of 2^e, so below 2^-13 of the largest element.  That is less than bf16
//           loses of elements down to 2^-5 of the largest, and more of smaller ones; it
//           takes 3/4 of the matrix time of one bf16 product.
//   softmax every lane holds one row (l%16) and 16 of the 64 keys, in fp32, base 2.
//           Weights are 2^(s - ref) and their sum runs beside the values'.  Any ref that
//           neither over- nor underflows gives the same relative precision, so it is 0
//           until a row's first visible tile has a largest score beyond +-40 or a tile's
//           weights pass 2^40; then it is raised to the largest score, and what is
//           summed so far is scaled by 2^(old - new).  Weights of 2^-40 to 2^40 times
//           values could leave fp32 where the result does not, so in a row that sees a
//           value scale far from one (kFarLow, kFarHigh) the reference follows what the
//           row has seen: its largest score, or the logarithm of its sum.
//   values  O^T += V^T P^T with the 16x16x32 bf16 MFMA.  The order of the summed
//           keys is free, so it is chosen as the lanes already hold them: P needs
//           no exchange, only its rounding to bf16 (2^-8 of a weight at most; sums stay in
//           fp32).  That is the format the matrix core shares with the values, which
//           become bf16 exactly (a code has 2 bits, a scale eight bits of exponent: fp16
//           has not the range) through LDS and are read transposed by
//           ds_read_b64_tr_b16; a second term of the weights would double the value
//           products.  It makes the output's error 1.3 to 1.5 times that of an fp32
//           form rounded to bf16 (0.0021 - 0.0024 for 0.0016 of the result).
//
// Long caches are split over workgroups (`splits` ranges of whole 64-key tiles of
// each sequence's own length) whose fp32 partial sums a second kernel joins.
#include "../../include/tabit.h"
#include "kv_query.h"
#include "tile_common.h"

namespace tabit {
namespace {

using namespace kv;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr float kNegInf = -__builtin_inff();
constexpr uint32_t kMaxValueScale = 252;   // 6 * 2^(252 - 127) is the largest finite value
// Value scales up to 2^50: sums of weights to 2^67 (2^40 in each of 2^27 tiles), 2^3 for a code
// and 2^5 for the transform stay below 2^128.  From 2^-60 on: the largest weight, 2^-40 or more,
// times half of it is far above 2^-126, so a row's sums keep their bits.
constexpr uint32_t kFarLow = 67, kFarHigh = 177;
// A row with a value scale beyond them has weights of one at most, or of 2^-16 from a large scale
// on: 2^16 of them times the largest finite value stay finite.
constexpr float kFarRoom = 16.0f;
constexpr int kNever = 0x7FFFFFFF;
constexpr int TILE = 64;      // keys a wave takes at a time
constexpr int NUM_CUS = 256;  // MI355X
constexpr int kMaxSplits = 128;
constexpr int kNarrow = 8;    // splits that one lane joins by itself

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bool far_scale(uint32_t s) { return s - kFarLow > kFarHigh - kFarLow; }

// Which of 16 keys have one of a wave's bits (lane % 16: the key), and the lowest of them.
__device__ __forceinline__ uint32_t keys_of(unsigned long long m) {
  m |= m >> 32;
  m |= m >> 16;
  return (uint32_t)m & 0xFFFFu;
}
__device__ __forceinline__ int lowest_key(unsigned long long m) { return __builtin_ctz(keys_of(m)); }

// What a part (reference, sum of weights) of a row is taken relative to when parts are joined: the
// exponent of its sum, so that every part's sum of weights becomes less than one.  A part
// without keys is (-inf, 0).
__device__ __forceinline__ float part_top(float ref, float sum) {
  return ref + (float)__builtin_amdgcn_frexp_expf(sum);
}

// 1 / sum (for a transformed cache 1 / (32 sum)) in two factors: a power of two, which is taken
// before the transform adds 32 elements, so that their sum stays in range and what cancels does so
// exactly, and the rest, which is taken after it.  0 for a row that sees no key.
struct Shares {
  float power, rest;
};
__device__ __forceinline__ Shares shares(float sum, bool had) {
  const int e = __builtin_amdgcn_frexp_expf(sum);
  return {__builtin_amdgcn_ldexpf(had ? 0.03125f : 1.0f, -e),
          sum == 0.0f ? 0.0f : 1.0f / __builtin_amdgcn_ldexpf(sum, -e)};
}

// sum + both bf16 weights of a pair, in fp32.  The rounded weights are summed, not the exact
// ones: what a row's values are multiplied with then adds up to one, and a row that sees one
// key answers that key's value as it is (a tie of its rounding to bf16 may fall either way).
__device__ __forceinline__ float add_pair(uint32_t pair, float sum) {
  const v2bf one = {(__bf16)1.0f, (__bf16)1.0f};
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, pair), one, sum, false);
}

// Byte offset of 16-byte piece `half` of 16-element run `c` of key row `key` in the
// bf16 value tile: rows of RS bytes.  Runs are XORed with bits of the key so that what
// one access touches fills a 256-byte bank window: the 4 keys x 2 runs (or 8 keys x 1
// run) of 32 lanes of a transposed read, and, with the pieces of every other eight
// keys swapped, the 16 keys that 16 lanes write at once.  By the counters that is not
// the whole rule: 39 - 40% of the cycles LDS is active are conflicts in single rows of
// 128 elements, 21 - 25% in chunks (which access has them was not taken apart; LDS is
// active for about a quarter of the time).
template <int RS>
__device__ __forceinline__ int v_off(int key, int c, int half) {
  const int x = RS == 256 ? ((key & 3) << 1 | ((key >> 2) & 1)) : ((key & 2) | ((key >> 2) & 1));
  return key * RS + ((c ^ x) << 5) + ((half ^ ((key >> 3) & 1)) << 4);
}

// Three FP6 terms of a block of 32 with their E8M0 bytes (bytes 0..2 of `scales`).
// A block that is not `ok` or not finite gets scale 255 (not a number) for whatever its
// codes are: its row answers NaN.  An infinity shows in the largest magnitude, NaN in
// the sum (an overflow of the sum itself is an infinity and counts for nothing).
__device__ __forceinline__ void q_terms(float (&x)[32], bool ok, v8i (&q)[3], uint32_t& scales) {
  float top = 0.0f, even = 0.0f, odd = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
    even += x[e];
    odd += x[e + 1];
  }
  ok = ok && finite_f32(top) && even == even && odd == odd;
  // the exponent floor(log2 top) - 2, or one more above 7.5 of it: all terms end at 7.5
  const int ex = max(mx_exponent(__uint_as_float(__float_as_uint(top) + 0x100000u)), -119);
  scales = 0u;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const int E = ex - 4 * t + 127;
    const float s = __uint_as_float((uint32_t)E << 23);
    v16f lo, hi;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      lo[e] = x[2 * e];
      hi[e] = x[2 * e + 1];
    }
    const v6u w = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(lo, hi, s);
    if (t < 2) {
      const v32f d = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(w, s);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] -= d[e];
    }
    q[t] = v8i{(int)w[0], (int)w[1], (int)w[2], (int)w[3], (int)w[4], (int)w[5], 0, 0};
    scales |= (uint32_t)(ok ? E : 255) << (8 * t);
  }
}

// Tiles of n keys, and the first n = TILE t keys cut at len: n and TILE t may be within TILE of
// 2^31, or 2^31 itself.
__device__ __forceinline__ int tiles_of(int n) { return (int)(((unsigned)n + (TILE - 1)) / TILE); }
__device__ __forceinline__ int keys_to(int t, int len) { return (int)min((unsigned)t * TILE, (unsigned)len); }

// The range of tiles [t0, t1) of split `sp`, of `tiles` tiles in all.  A sequence has as
// many splits as its length needs at the share of the longest one there may be, alike in
// length: the workgroups of a ragged batch cost about the same.
__device__ __forceinline__ void split_range(const KvAttnArgs& a, int tiles, int sp, int& t0, int& t1) {
  const int most = tiles_of(a.max_kv), share = max((most + a.splits - 1) / a.splits, 1);
  const int parts = max((tiles + share - 1) / share, 1), per = (tiles + parts - 1) / parts;
  t0 = min(sp * per, tiles);
  t1 = min(t0 + per, tiles);
}

// Where the partial result of split `sp` for row `row` of tokens x q_heads goes: dim_pad
// sums at part_sums, (maximum, sum) at part_stats.  A split without keys writes (-inf, 0)
// and no sums.
__device__ __forceinline__ float* part_sums(const KvAttnArgs& a, int sp, long long row) {
  return a.part + ((long long)sp * a.tokens * a.q_heads + row) * a.cache.dim_pad;
}
__device__ __forceinline__ float2* part_stats(const KvAttnArgs& a, int sp, long long row) {
  const long long rows = (long long)a.tokens * a.q_heads;
  return reinterpret_cast<float2*>(a.part + (long long)a.splits * rows * a.cache.dim_pad) + sp * rows + row;
}

// One workgroup: 16 rows (queries x heads of the group) of one key head of one
// sequence over one range of its keys; the range's tiles go to the waves in runs and
// every wave works by itself until the end.  Bound by the cache's bytes: a wave asks
// for the next tile's codes and scales (8.7 KB at 128 elements) as soon as this one's
// are in LDS or in the matrix core; the values of 32 keys are staged at a time (8 KB of
// LDS a wave), and registers allow three workgroups a CU.
//
// Measured at 32 heads over 8, 128 elements: 64 rows of up to 8192 keys 84 - 87 us (371 MB,
// 4.3 TB/s; 64 of 8192 each 108 us, 5.3 TB/s, what a large copy reaches: the rest is the
// longest sequences, a lone workgroup passing 256 keys in 1.25 us), one row of 131072
// keys 39 us with the join (143 MB, 3.7 TB/s), one row of 1000 keys 13 - 16 us.  A
// workgroup's start costs 6 us (bounds, pages, then codes and tables: three loads that
// depend on each other), which is what short caches take.  Six, eight or twelve waves a
// workgroup level out ragged batches but fill the chip less: 99 to 112 us for 97 then.
template <int NB, bool TREE>
__global__ void __launch_bounds__(256, 3)
kv_attention_rows16_kernel(KvAttnArgs a) {
  constexpr int NW = 4;
  constexpr int DP = NB * 32;
  constexpr int ND = DP / 16;                         // 16-element output blocks
  constexpr int RS = NB <= 2 ? 128 : 256;             // bytes of a staged value row
  constexpr int STAGE = 32 * RS;
  constexpr int MERGE = 16 * (DP + 4) * 4;            // one wave's sums, rows padded against banks
  constexpr int PER_WAVE = STAGE > MERGE ? STAGE : MERGE;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * PER_WAVE + NW * 16 * 8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, g = lane >> 4;
  const int b = blockIdx.z, hk = blockIdx.y;
  const int sp = blockIdx.x % a.splits, row_tile = blockIdx.x / a.splits;
  const KvCacheArgs& c = a.cache;

  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int r0 = row_tile * 16;
  if (r0 >= n * a.group) return;
  const int len = seq_keys(a, b);
  const int qi = (r0 + row) / a.group, qh = hk * a.group + (r0 + row) % a.group;
  const bool row_ok = qi < n;
  const int last = (min(r0 + 16, n * a.group) - 1) / a.group;
  const int seen_hi = seen_keys(a, len, all, last);
  const int seen_lo = TREE ? before_tree(len, all) : seen_keys(a, len, all, r0 / a.group);
  const uint64_t* seen_nodes = TREE ? a.mask + (long long)(q0 + min(qi, n - 1)) * a.mask_words : nullptr;
  const int seen = row_ok ? seen_keys(a, len, all, qi) : seen_hi;     // idle rows hide nothing

  int t0, t1;
  split_range(a, tiles_of(seen_hi), sp, t0, t1);
  if (a.splits > 1 && t0 >= t1) {
    if (threadIdx.x < 16 && row_ok)
      *part_stats(a, sp, (long long)(q0 + qi) * a.q_heads + qh) = make_float2(kNegInf, 0.0f);
    return;
  }
  const int per = (t1 - t0 + NW - 1) / NW;
  const int w0 = min(t0 + wave * per, t1), w1 = min(w0 + per, t1);

  const int* table = a.table + (long long)b * a.table_stride;
  const int in_page = (1 << c.page_shift) - 1;
  // lane: key l%16 and block l/16 of each group of 16 keys, which lie in one page
  const bool has = g < NB;
  const unsigned c_at = row * (DP / 2) + (has ? g * 16 : 0), s_at = row * NB + (has ? g : 0);
  v4i kc[4] = {}, vc[4] = {};
  uint32_t ks[4] = {127u, 127u, 127u, 127u}, vs[4] = {127u, 127u, 127u, 127u};
  // Lane: the page of key group lane % 4 of tile t, -1 past the keys.
  int page;
  auto pages = [&](int t) {
    const int j = (int)((unsigned)t * TILE + 16 * (lane & 3));     // (t may be past the range)
    page = t < w1 && j < len ? table[min(j >> c.page_shift, a.table_stride - 1)] : -1;
  };
  // Codes and scales of tile t.  Where a group has no page, or a key lies past the end, some
  // row of the cache is read all the same and taken out when the tile is used: every group
  // costs four loads at uniform bases and no branch.
  auto fetch = [&](int t) {
    if (t >= w1 || c.num_pages == 0) return;
    const uint32_t pg = (unsigned)page < (unsigned)c.num_pages ? (uint32_t)page : 0u;
    const uint32_t in = (uint32_t)(t * TILE + 16 * (lane & 3)) & (uint32_t)in_page;
    const uint64_t at = ((((uint64_t)pg * (uint32_t)c.heads + (uint32_t)hk) << c.page_shift) | in) * NB;
    // (kept 32 bits wide here, so that the loads take them beside a scalar base)
    uint32_t ca = c_at, sa = s_at;
    asm("" : "+v"(ca), "+v"(sa));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(at >> 32), k) << 32 |
                            (uint32_t)__builtin_amdgcn_readlane((int)at, k);
      kc[k] = *reinterpret_cast<const v4i*>((c.k_codes + base * 16) + ca);
      vc[k] = *reinterpret_cast<const v4i*>((c.v_codes + base * 16) + ca);
      ks[k] = (c.k_scales + base)[sa];
      vs[k] = (c.v_scales + base)[sa];
    }
  };
  // The start is a chain of dependent loads, so each link asks for all it can: what
  // depends on the sequence's bounds alone (pages, positions, query rows), then the table
  // rows and the first tile, which arrives while the queries are turned.
  pages(w0);
  const int hole0 = (int)((unsigned)w0 * TILE >> c.page_shift), hole1 = min(((keys_to(w1, len) - 1) >> c.page_shift) + 1, a.table_stride);
  const int probe = hole0 + lane < hole1 ? table[hole0 + lane] : 0;
  // q': eight elements a thread, through LDS to the B operand (row l%16, block l/16)
  float* qs = reinterpret_cast<float*>(smem);
  constexpr int QROW = DP + 4;
  static_assert(16 * QROW * 4 <= NW * PER_WAVE, "q' fits the staging");
  const int qr = threadIdx.x / (4 * NB), e0 = threadIdx.x % (4 * NB) * 8;
  const int ti = (r0 + qr) / a.group, th = hk * a.group + (r0 + qr) % a.group;
  const bool turns = e0 < a.rope.rope_dim, mine = (int)threadIdx.x < 64 * NB && ti < n && e0 < c.head_dim;
  const int rhalf = a.rope.rope_dim >> 1;
  const bool second = !a.rope.interleaved && e0 >= rhalf;
  const int pair0 = a.rope.interleaved ? e0 >> 1 : second ? e0 - rhalf : e0;
  uint4 own = make_uint4(0, 0, 0, 0), other = own;
  int pos = 0;
  if (mine) {
    const uint16_t* qp = a.q + (long long)(q0 + ti) * a.q_stride + (long long)th * c.head_dim;
    if (turns) {
      pos = a.positions[q0 + ti];
      if (!a.rope.interleaved) other = *reinterpret_cast<const uint4*>(qp + (second ? e0 - rhalf : e0 + rhalf));
    }
    own = *reinterpret_cast<const uint4*>(qp + e0);
  }
  const bool pos_ok = pos >= 0 && pos < a.rope.num_positions;
  float4 cs[4] = {};             // cos, sin: four pairs, or eight
  if (mine && turns && pos_ok) {
    const size_t at = (size_t)pos * rhalf + pair0;
    cs[0] = *reinterpret_cast<const float4*>(a.rope.cos + at);
    cs[2] = *reinterpret_cast<const float4*>(a.rope.sin + at);
    if (!a.rope.interleaved) {
      cs[1] = *reinterpret_cast<const float4*>(a.rope.cos + at + 4);
      cs[3] = *reinterpret_cast<const float4*>(a.rope.sin + at + 4);
    }
  }
  fetch(w0);
  pages(w0 + 1);
  bool holes = (unsigned)probe >= (unsigned)c.num_pages && hole0 + lane < hole1;
  for (int i = hole0 + 64 + lane; i < hole1; i += 64) holes = holes || (unsigned)table[i] >= (unsigned)c.num_pages;
  holes = __any(holes);          // whether a page of the wave's keys is not in the cache
  if ((int)threadIdx.x < 64 * NB) {
    float x[8] = {bf_lo(own.x), bf_hi(own.x), bf_lo(own.y), bf_hi(own.y),
                  bf_lo(own.z), bf_hi(own.z), bf_lo(own.w), bf_hi(own.w)};
    if (mine && turns) {
      if (!pos_ok) {             // no such table row: not a number
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_nanf("");
      } else if (a.rope.interleaved) {
        turn(x[0], x[1], cs[0].x, cs[2].x);
        turn(x[2], x[3], cs[0].y, cs[2].y);
        turn(x[4], x[5], cs[0].z, cs[2].z);
        turn(x[6], x[7], cs[0].w, cs[2].w);
      } else {
        const float y[8] = {bf_lo(other.x), bf_hi(other.x), bf_lo(other.y), bf_hi(other.y),
                            bf_lo(other.z), bf_hi(other.z), bf_lo(other.w), bf_hi(other.w)};
        const float cc[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
        const float ss[8] = {cs[2].x, cs[2].y, cs[2].z, cs[2].w, cs[3].x, cs[3].y, cs[3].z, cs[3].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[e] * cc[e], w = y[e] * ss[e];
          x[e] = second ? u + w : u - w;
        }
      }
    }
    if (c.had) fwht32_lanes(x, lane);
    const float factor = base2_scale(a);
#pragma unroll
    for (int e = 0; e < 8; e += 4)
      *reinterpret_cast<v4f*>(qs + qr * QROW + e0 + e) =
          v4f{x[e] * factor, x[e + 1] * factor, x[e + 2] * factor, x[e + 3] * factor};
  }
  __syncthreads();
  v8i q[3];
  uint32_t q_scales = 0u;
#pragma unroll
  for (int t = 0; t < 3; ++t) q[t] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
  if (has) {
    float x[32];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const v4f y = *reinterpret_cast<const v4f*>(qs + row * QROW + g * 32 + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e + k] = y[k];
    }
    q_terms(x, true, q, q_scales);
  }
  __syncthreads();

  float ref = 0.0f, l = 0.0f, far_room = 0.0f;
  bool fresh = true, any_fresh = true, any_ref = false;      // any: over the wave
  v4f o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  uint8_t* stage = smem + wave * PER_WAVE;

  for (int t = w0; t < w1; ++t) {
    const int j0 = t * TILE;
    v4f s[4];
    if (len - j0 < TILE || holes) {                  // values of rows that were not asked for: zeros
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 16 * k, pi = j >> c.page_shift;
        const bool there = !holes || (pi < a.table_stride && (unsigned)table[pi] < (unsigned)c.num_pages);
        if (!there || row >= len - j) {
          vs[k] = 127u;
          vc[k] = v4i{0, 0, 0, 0};
        }
      }
    }
    // a value scale beyond bf16 (or NaN): the key's scores become NaN, its values zero; one far from
    // one: the rows that see the first such key of the tile (of a tree, any such key) keep their reference
    // near their scores
    int far_from = kNever, high_from = kNever;
    uint64_t far_keys = 0, high_keys = 0;            // (of a tree)
    if (__any(has && max(max(vs[0] - kFarLow, vs[1] - kFarLow), max(vs[2] - kFarLow, vs[3] - kFarLow)) > kFarHigh - kFarLow)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned long long bad = __ballot(has && vs[k] > kMaxValueScale);
        if (((bad >> row) & 0x0001000100010001ull) != 0) {
          ks[k] = 255u;
          vs[k] = 127u;
          vc[k] = v4i{0, 0, 0, 0};
        }
        const unsigned long long far = __ballot(has && far_scale(vs[k]));
        const unsigned long long high = __ballot(has && vs[k] > kFarHigh);
        if constexpr (TREE) {
          far_keys |= (uint64_t)keys_of(far) << (16 * k);
          high_keys |= (uint64_t)keys_of(high) << (16 * k);
        } else {
          if (far != 0) far_from = min(far_from, j0 + 16 * k + lowest_key(far));
          if (high != 0) high_from = min(high_from, j0 + 16 * k + lowest_key(high));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // blocks that do not exist (lanes past NB) are zeros on the side of q
      const v8i ka = {kc[k][0], kc[k][1], kc[k][2], kc[k][3], 0, 0, 0, 0};
      const int kw = has ? (int)ks[k] : 127;
      s[k] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      s[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ka, q[0], s[k], 4, 2, 0, kw, 0, (int)q_scales);
      s[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ka, q[1], s[k], 4, 2, 0, kw, 1, (int)q_scales);
      s[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ka, q[2], s[k], 4, 2, 0, kw, 2, (int)q_scales);
    }
    // lane: keys 16 k + 4 g + r of its row
    if (seen_lo - j0 < TILE || holes) {
      const int left = seen - j0 - 4 * g;
      const uint64_t nodes = TREE ? nodes_from(seen_nodes, a.mask_words, j0 - (len - all)) >> (4 * g) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pi = (j0 + 16 * k) >> c.page_shift;
        const bool there = !holes || (pi < a.table_stride && (unsigned)table[pi] < (unsigned)c.num_pages);
        const int mine = there ? left : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * k + r >= mine || (TREE && !(nodes >> (16 * k + r) & 1))) s[k][r] = kNegInf;
      }
    }
    // weights: as in the kernel for 128 rows, 2^(s - ref) with a reference only where needed
    float sum;
    uint32_t p[8];
    bool over = false;
    const bool any_far = TREE ? far_keys != 0 : far_from != kNever;
    if (any_ref) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] -= ref;
    }
    for (int pass = 0; pass < 2; ++pass) {
      if (pass == 1 || any_far || (any_fresh && __any(fresh && j0 < seen))) {
        float top = kNegInf;
        asm volatile("" : "+v"(top));                // (else the compiler takes the maximum of every tile)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = fmaxf(top, s[k][r]);
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const bool first = fresh && top > kNegInf;
        fresh = fresh && !first;
        any_fresh = __any(fresh);
        const bool up = first ? fabsf(top) > 40.0f : over && top > 0.0f;
        float by = up ? top : 0.0f;
        if (pass == 0 && any_far) {
          float so_far = l + __shfl_xor(l, 16, 64);
          so_far += __shfl_xor(so_far, 32, 64);
          const float m = fmaxf(top, __builtin_amdgcn_logf(so_far));
          bool sees_far = seen > far_from, sees_high = seen > high_from;
          if constexpr (TREE) {
            const uint64_t nodes = nodes_from(seen_nodes, a.mask_words, j0 - (len - all));
            sees_far = (nodes & far_keys) != 0;
            sees_high = (nodes & high_keys) != 0;
          }
          far_room = sees_high ? kFarRoom : far_room;
          if (sees_far && m > kNegInf) by = m + far_room;
        }
        ref += by;
        any_ref = __any(ref != 0.0f);
        if (__any(by != 0.0f)) {
          const float alpha = first ? 1.0f : exp2_fast(-by);
          l *= alpha;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[d] *= alpha;
#pragma unroll
          for (int k = 0; k < 4; ++k) s[k] -= by;
        }
      }
      sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w0_ = exp2_fast(s[k][0]), w1_ = exp2_fast(s[k][1]);
        const float w2_ = exp2_fast(s[k][2]), w3_ = exp2_fast(s[k][3]);
        p[2 * k] = pack_bf16(w0_, w1_);
        p[2 * k + 1] = pack_bf16(w2_, w3_);
        sum = add_pair(p[2 * k + 1], add_pair(p[2 * k], sum));
      }
      unsigned long long m = __ballot(!(sum < 0x1p40f));
      if (m == 0) break;
      m |= m >> 32;
      over = ((m | m >> 16) >> row) & 1;             // in any of the row's four lanes
    }
    l += sum;
    // values, 32 keys at a time through the wave's own staging (LDS serves a wave in order)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (has) {
#pragma unroll
        for (int k = 2 * h; k < 2 * h + 2; ++k) {
          const float f = __uint_as_float(vs[k] << 23);
          const int key = (k & 1) * 16 + row;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = (uint32_t)vc[k][w];
            uint4 y;
            y.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 0));
            y.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 1));
            y.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 2));
            y.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 3));
            *reinterpret_cast<uint4*>(stage + v_off<RS>(key, g * 2 + (w >> 1), w & 1)) = y;
          }
        }
      }
      if (h == 1) {                                    // the tile's registers are free
        fetch(t + 1);                                  // past the range: no loads
        pages(t + 2);
      }
      __builtin_amdgcn_wave_barrier();
      const v8bf w = __builtin_bit_cast(v8bf, make_uint4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]));
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int key = 4 * g + (row >> 2);
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s)(stage + v_off<RS>(key, d, (row >> 1) & 1) + (row & 1) * 8));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s)(stage + v_off<RS>(key + 16, d, (row >> 1) & 1) + (row & 1) * 8));
        const v8bf v = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w, o[d], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves: sums to LDS as [row][d], then 16 rows x NB blocks
  float* sums = reinterpret_cast<float*>(stage);
  float* ml = reinterpret_cast<float*>(smem + NW * PER_WAVE);
#pragma unroll
  for (int d = 0; d < ND; ++d)
    *reinterpret_cast<v4f*>(sums + row * (DP + 4) + d * 16 + g * 4) = o[d];
  if (g == 0) {
    ml[(wave * 16 + row) * 2] = fresh ? kNegInf : ref;
    ml[(wave * 16 + row) * 2 + 1] = l;
  }
  __syncthreads();
  if ((int)threadIdx.x >= 16 * NB) return;
  const int fr = threadIdx.x / NB, fb = threadIdx.x % NB;
  const int fi = (r0 + fr) / a.group, fh = hk * a.group + (r0 + fr) % a.group;
  if (fi >= n) return;
  float M = kNegInf;
#pragma unroll
  for (int w = 0; w < NW; ++w) M = fmaxf(M, part_top(ml[(w * 16 + fr) * 2], ml[(w * 16 + fr) * 2 + 1]));
  M += 2.0f;                                          // four sums: less than one together
  const float base = M == kNegInf ? 0.0f : M;
  float x[32], L = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float f = exp2_fast(ml[(w * 16 + fr) * 2] - base);
    L += f * ml[(w * 16 + fr) * 2 + 1];
    const float* src = reinterpret_cast<const float*>(smem + w * PER_WAVE) + fr * (DP + 4) + fb * 32;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const v4f y = *reinterpret_cast<const v4f*>(src + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e + k] += f * y[k];
    }
  }
  const long long out_row = (long long)(q0 + fi) * a.q_heads + fh;
  if (a.splits > 1) {
    float* dst = part_sums(a, sp, out_row) + fb * 32;
#pragma unroll
    for (int e = 0; e < 32; e += 4) *reinterpret_cast<v4f*>(dst + e) = v4f{x[e], x[e + 1], x[e + 2], x[e + 3]};
    if (fb == 0) *part_stats(a, sp, out_row) = make_float2(M, L);
    return;
  }
  const Shares inv = shares(L, c.had);
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] *= inv.power;
  if (c.had) fwht32_lane(x);
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    const int d = fb * 32 + e;
    if (d < c.head_dim)
      *reinterpret_cast<uint4*>(a.out + out_row * c.head_dim + d) =
          make_uint4(pack_bf16(x[e] * inv.rest, x[e + 1] * inv.rest), pack_bf16(x[e + 2] * inv.rest, x[e + 3] * inv.rest),
                     pack_bf16(x[e + 4] * inv.rest, x[e + 5] * inv.rest), pack_bf16(x[e + 6] * inv.rest, x[e + 7] * inv.rest));
  }
  if (a.lse != nullptr && fb == 0)
    a.lse[out_row] = L == 0.0f ? kNegInf : (M + __builtin_log2f(L)) * 0.6931471805599453f;
}

// Both halves' values of a lane pair (l, l ^ 32), in the order (lanes 0..31, 32..63).
__device__ __forceinline__ void halves(float v, float& lo, float& hi) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  lo = __uint_as_float(r[0]);
  hi = __uint_as_float(r[1]);
}

// s + K_block Q'^T for term `t` of q'; `byte` picks the keys' scale in ksw.
__device__ __forceinline__ v16f score_term(v4i x, const v8i& q, v16f s, int byte, int ksw, int t, int qsw) {
  const v8i k = {x[0], x[1], x[2], x[3], 0, 0, 0, 0};
#define TABIT_TERM(B_, T_) \
  if (byte == B_ && t == T_) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q, s, 4, 2, B_, ksw, T_, qsw);
  TABIT_TERM(0, 0) TABIT_TERM(0, 1) TABIT_TERM(0, 2)
  TABIT_TERM(1, 0) TABIT_TERM(1, 1) TABIT_TERM(1, 2)
  TABIT_TERM(2, 0) TABIT_TERM(2, 1) TABIT_TERM(2, 2)
  TABIT_TERM(3, 0) TABIT_TERM(3, 1) TABIT_TERM(3, 2)
#undef TABIT_TERM
  return s;
}

// One workgroup: 32 NW rows of one key head of one sequence, 32 a wave, over one range
// of its keys.  The 64 keys of a tile are brought in once for all rows: codes and
// scales through registers (loaded a tile ahead, their pages two ahead) into one of two
// LDS stages, the values already as bf16, one barrier a tile.  A wave uses the 32x32
// forms of the same products: scores with 32x32x64 (lane l: one row, l%32, and 32 of
// the 64 keys), values with 32x32x16, P staying in its lanes.
//
// Vector instructions and matrix products share a wave's issue and about balance, so a
// tile costs the vector units one exponential a score, half a rounding to bf16 and half a
// dot product that sums; without a reference (see the top) the scores go to the exponential
// as they leave the matrix core, and what a tile's addresses need is prepared for 64 tiles
// at once.
//
// Measured, the clock settled: 2700 rows x 17776 keys x 30 heads x 64 in 407 - 424 us by the card,
// 16 of it the join (870 - 905 TFLOP/s at 4 flops a key, row and element; a library bf16 product
// of 8192^3 reaches 1207; 446 us in the first 20 calls on an idle card), four causal turns (1024
// to 2048 queries behind caches of up to 6144 keys, 32 heads over 8, 128 elements) at 965
// TFLOP/s of visible keys, 2 x 4096 rows x 300 keys x 16 heads x 72 in 30 - 31 us.  Matrix cores are busy for a third of the cycles, LDS for 30%; a wave
// waits for its turn to issue most of the time.  Level or slower: scores of a tile beside the weights of the one before,
// eight waves a workgroup, 32 keys a step, three stages, heads or sequences as the fastest
// index (causal turns 527 us for 466).  Up to 64 elements three workgroups fit a CU (four
// would spill: 485 us for 409); 96 and 128 elements take 204 and 232 registers, two
// workgroups (three spill: 38 us for 30 at 72 elements).  Seeing value scales far from one and
// keeping sums in range for them costs the first 1.2%, short chunks 1.5%, causal turns nothing.
template <int NB, bool TREE>
__global__ void __launch_bounds__(256, NB <= 2 ? 3 : 2)
kv_attention_rows128_kernel(KvAttnArgs a) {
  constexpr int NW = 4, ROWS = NW * 32;              // waves, rows
  constexpr int DP = NB * 32;
  constexpr int ND = DP / 32;                        // 32-element output blocks
  constexpr int NS = (NB + 1) / 2;                   // 64-element steps of a score
  constexpr int RS = NB <= 2 ? 128 : 256;            // bytes of a staged value row
  constexpr int KB = TILE * DP / 2;                  // bytes of a tile's key codes
  struct Stage {
    uint8_t v[TILE * RS];
    uint8_t k[KB];
    // [block % 2][key % 32]: scale bytes of [key / 32 * 2 + block / 2], then as many marks of keys
    // (of this tile or an earlier one of the stage) whose value scale is far from one
    uint8_t ks[2][32][8];
  };
  __shared__ __attribute__((aligned(1024))) Stage st[2];
  // by stage: the first key so far whose value scale is far from one, and that is far above it.
  // Like the stage's marks written before the barrier that hands a tile over and read in that tile
  // alone, so neither depends on timing.
  __shared__ int2 far_at[2];
  // Of a tree, whose rows see keys by their bits: by stage and wave the last tile that has such keys, which
  // of the wave's 16 they are, and in the upper half those far above.
  __shared__ int2 far_in[TREE ? 2 : 1][NW];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 31, half = lane >> 5;
  const int per = gridDim.x / (unsigned)(a.cache.heads * a.seqs);   // row tiles x splits
  const int at_x = blockIdx.x / (unsigned)per, at_y = blockIdx.x % (unsigned)per;
  const int b = at_x / a.cache.heads, hk = at_x % a.cache.heads;
  const int sp = at_y % a.splits, row_tile = at_y / a.splits;
  const KvCacheArgs& c = a.cache;

  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int rows = n * a.group;
  // the last rows of a causal sequence see most: they start first
  const int tiles_r = (rows + ROWS - 1) / ROWS;
  if (row_tile >= tiles_r) return;
  const int r0 = (tiles_r - 1 - row_tile) * ROWS;
  const int len = seq_keys(a, b);
  const int rr = r0 + wave * 32 + row;
  const bool row_ok = rr < rows;
  const int qi = rr / a.group, qh = hk * a.group + rr % a.group;
  const int seen_all = seen_keys(a, len, all, (min(r0 + ROWS, rows) - 1) / a.group);
  const int seen = row_ok ? seen_keys(a, len, all, qi) : seen_all;   // idle rows mask nothing
  const int first = r0 + wave * 32;
  const int seen_lo = TREE ? before_tree(len, all) : seen_keys(a, len, all, min(first, rows - 1) / a.group);
  const uint64_t* seen_nodes = TREE ? a.mask + (long long)(q0 + min(qi, n - 1)) * a.mask_words : nullptr;
  const int seen_hi = first < rows ? seen_keys(a, len, all, min(first + 31, rows - 1) / a.group) : 0;

  int t0, t1;
  split_range(a, tiles_of(seen_all), sp, t0, t1);
  const long long out_row = (long long)(q0 + qi) * a.q_heads + qh;
  if (a.splits > 1 && t0 >= t1) {
    if (half == 0 && row_ok) *part_stats(a, sp, out_row) = make_float2(kNegInf, 0.0f);
    return;
  }

  // B operands: row l%32, block l/32 of each 64-element step
  v8i q[NS][3];
  uint32_t q_scales[NS];
#pragma unroll
  for (int ds = 0; ds < NS; ++ds) {
    q_scales[ds] = 0u;
#pragma unroll
    for (int t = 0; t < 3; ++t) q[ds][t] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    const int blk = 2 * ds + half;
    if (row_ok && blk < NB) {
      float x[32];
      const bool ok = load_q_block(a, q0 + qi, qh, blk, base2_scale(a), x);
      q_terms(x, ok, q[ds], q_scales[ds]);
    }
  }

  const int in_page = (1 << c.page_shift) - 1;

  // A wave brings in KPW keys of a tile, which lie in one page: their rows are one run of
  // memory at a uniform base, a lane's offset in it never changes.  Key codes: lane =
  // block * KPW + key; value codes: likewise, VH pieces a block where that fits the wave.
  constexpr int KPW = TILE / NW;
  constexpr int VH = 64 / KPW / NB >= 4 ? 4 : 64 / KPW / NB >= 2 ? 2 : 1;
  constexpr int VW = 4 / VH;                         // dwords of a piece
  const int lkey = lane % KPW, unit = lane / KPW;
  const int kblk = unit, vblk = unit / VH, vpart = unit % VH;
  const bool has_k = kblk < NB, has_v = vblk < NB;
  // (lanes without a block read the first one)
  const unsigned k_at = lkey * (DP / 2) + (has_k ? kblk * 16 : 0);
  const unsigned v_at = lkey * (DP / 2) + (has_v ? vblk * 16 + vpart * VW * 4 : 0);
  const unsigned ks_at = lkey * NB + (has_k ? kblk : 0), vs_at = lkey * NB + (has_v ? vblk : 0);
  const int* table = a.table + (long long)b * a.table_stride;
  // Where the wave's 16 keys of 64 tiles lie, a lane a tile: 32 (row / 16) + how many of them
  // are in the cache and the sequence.  One lane-wide computation for 64 tiles (waited for at
  // once: a load whose wait is left to a later tile makes every tile wait) leaves a tile two
  // lane reads and the additions of its bases.
  uint32_t at_lo = 0u, at_hi = 0u;
  auto place = [&](int from) {
    const int j = min(from + lane, t1 - 1) * TILE + wave * KPW;
    const int page = table[min(j >> c.page_shift, a.table_stride - 1)];
    const bool there = (unsigned)page < (unsigned)c.num_pages;
    const uint64_t row = (((uint64_t)(there ? (uint32_t)page : 0u) * (uint32_t)c.heads + (uint32_t)hk) << c.page_shift) |
                         (uint32_t)(j & in_page);
    const uint64_t at = row * 2 + (there ? (uint32_t)min(max(len - j, 0), KPW) : 0u);
    at_lo = (uint32_t)at;
    at_hi = (uint32_t)(at >> 32);
  };
  v4i kc = {}, vc = {};
  uint32_t ks = 127u, vs = 127u;
  int got = 0;                   // keys of the wave's 16 that are in the cache and the sequence
  // Codes and scales of tile t: four loads at uniform bases and no
  // branch.  Without a page, or past the sequence's end, some row of the cache is read all the
  // same and its values are zeroed when they are stored.
  auto fetch = [&](int t) {
    if (t >= t1 || c.num_pages == 0) return;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)at_lo, (t - t0) & 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)at_hi, (t - t0) & 63);
    got = (int)(lo & 31u);
    const uint64_t base = ((uint64_t)hi << 32 | (lo & ~31u)) * NB >> 1;      // row * NB
    // (kept 32 bits wide here, so that the loads take them beside a scalar base)
    uint32_t ka = k_at, va = v_at, ksa = ks_at, vsa = vs_at;
    asm("" : "+v"(ka), "+v"(va), "+v"(ksa), "+v"(vsa));
    kc = *reinterpret_cast<const v4i*>((c.k_codes + base * 16) + ka);
    const uint8_t* vp = (c.v_codes + base * 16) + va;
    if constexpr (VW == 4) {
      vc = *reinterpret_cast<const v4i*>(vp);
    } else if constexpr (VW == 2) {
      const int2 w = *reinterpret_cast<const int2*>(vp);
      vc[0] = w.x;
      vc[1] = w.y;
    } else {
      vc[0] = *reinterpret_cast<const int*>(vp);
    }
    ks = (c.k_scales + base)[ksa];
    vs = (c.v_scales + base)[vsa];
  };
  // Whether a page of the range is not in the cache: its keys are then hidden tile by tile.
  bool holes = false;
  for (int i = (int)((unsigned)t0 * TILE >> c.page_shift) + lane; i < a.table_stride && i <= (keys_to(t1, len) - 1) >> c.page_shift; i += 64)
    holes = holes || (unsigned)table[i] >= (unsigned)c.num_pages;
  holes = __any(holes);
  // 16-byte block `blk` of key row `key`: rows share a 256-byte bank window, the XOR
  // spreads the 16 rows one read touches over it (48-byte rows spread by themselves)
  auto k_off = [](int key, int blk) {
    if constexpr (NB == 4) return key * 64 + ((blk ^ ((key >> 2) & 3)) << 4);
    else if constexpr (NB == 2) return key * 32 + ((blk ^ ((key >> 3) & 1)) << 4);
    else return key * (DP / 2) + (blk << 4);
  };

  // weights are 2^(s - ref); `fresh`: the row has seen no key yet
  float ref = 0.0f, l = 0.0f;
  bool fresh = true;
  v16f o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = v16f{};

  const int skey = wave * KPW + lkey;
  // A value scale beyond bf16 (or NaN): the key's scores become NaN and its values zero,
  // so that rows that do not see the key (weight 0) are not touched by it.
  // One far from one is noted for the tile's readers.
  auto settle = [&](int t) {
    if (got >= KPW && !__any(far_scale(vs))) return;
    asm volatile("");                                // a branch, not selects in every tile
    if (lkey >= got) {                               // rows that were not asked for
      vs = 127u;
      vc = v4i{0, 0, 0, 0};
    }
    const unsigned long long bad = __ballot(vs > kMaxValueScale);
    if (((bad >> lkey) & 0x0001000100010001ull) != 0) {            // lanes of the same key
      ks = 255u;
      vs = 127u;
      vc = v4i{0, 0, 0, 0};
    }
    const unsigned long long far = __ballot(far_scale(vs)), high = __ballot(vs > kFarHigh);
    const int key = (int)((unsigned)t * TILE) + wave * KPW;
    if (has_k && ((far >> lkey) & 0x0001000100010001ull) != 0)
      st[(t - t0) & 1].ks[kblk & 1][skey & 31][4 + (skey >> 5) * 2 + (kblk >> 1)] = 1;
    if constexpr (TREE) {
      if (far != 0 && lane == 0) far_in[(t - t0) & 1][wave] = make_int2(t, (int)(keys_of(far) | keys_of(high) << 16));
    } else {
      if (far != 0 && lane == 0) atomicMin(&far_at[(t - t0) & 1].x, key + lowest_key(far));
      if (high != 0 && lane == 0) atomicMin(&far_at[(t - t0) & 1].y, key + lowest_key(high));
    }
  };
  auto store_keys = [&](Stage& s) {
    if (has_k) {
      *reinterpret_cast<v4i*>(s.k + k_off(skey, kblk)) = kc;
      s.ks[kblk & 1][skey & 31][(skey >> 5) * 2 + (kblk >> 1)] = (uint8_t)ks;
    }
  };
  auto store_values = [&](Stage& s, int w) {         // w: dword of the piece
    if (has_v) {
      const float f = __uint_as_float(vs << 23);
      const uint32_t x = (uint32_t)vc[w];
      uint4 y;
      y.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 0));
      y.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 1));
      y.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 2));
      y.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, f, 3));
      const int g = vpart * VW + w;                  // 16 bytes of the block
      *reinterpret_cast<uint4*>(s.v + v_off<RS>(skey, vblk * 2 + (g >> 1), g & 1)) = y;
    }
  };
  auto store = [&](Stage& s) {
    store_keys(s);
#pragma unroll
    for (int w = 0; w < VW; ++w) store_values(s, w);
  };
  // Scores of a tile.  Lane: keys 32 kb + 8 (r / 4) + 4 half + r % 4 of its row.
  // Returns the lane's marks.
  auto scores = [&](const Stage& s, v16f (&sc)[2]) {
    const int2 ks_far = *reinterpret_cast<const int2*>(s.ks[half][row]);
    const int ksw = ks_far.x;
    sc[0] = sc[1] = v16f{};
#pragma unroll
    for (int ds = 0; ds < NS; ++ds) {
      const int blk = 2 * ds + half;
      v4i x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        if (NB % 2 == 0 || blk < NB) x[kb] = *reinterpret_cast<const v4i*>(s.k + k_off(kb * 32 + row, blk));
      // the two accumulators in turn: neither waits for its own last product
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          sc[kb] = score_term(x[kb], q[ds][t], sc[kb], kb * 2 + ds, ksw, t, (int)q_scales[ds]);
    }
    return ks_far.y;
  };
  // Sets the reference of rows that see their first key, raises it to the largest score in
  // rows that are `over`, and in a row `far` puts it at its largest score or `least`; the scores,
  // relative to it, move along, and what is summed so far is to be scaled by alpha.
  float alpha = 1.0f;
  bool any_fresh = true, any_ref = false, any_alpha = false;     // over the wave
  float far_room = 0.0f;
  uint32_t far_seen = 0u;        // of a tree: the stages in which the row has seen a far value scale
  auto raise = [&](v16f (&sc)[2], bool over, bool far, float least) {
    float top = kNegInf;
    asm volatile("" : "+v"(top));    // (else the compiler takes the maximum of every tile)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(fmaxf(top, sc[0][r]), sc[1][r]);
    float tl, th;
    halves(top, tl, th);
    top = fmaxf(tl, th);
    const bool first = fresh && top > kNegInf;
    fresh = fresh && !first;
    any_fresh = __any(fresh);
    // 2^s is as exact as 2^(s - ref): a reference is needed only for large scores
    const bool up = first ? fabsf(top) > 40.0f : over && top > 0.0f;
    float by = up ? top : 0.0f;
    const float m = fmaxf(top, least);
    if (far && m > kNegInf) by = m + far_room;
    const float f = first ? 1.0f : exp2_fast(-by);   // a fresh row's sums are zero
    ref += by;
    alpha *= f;
    l *= f;
    any_ref = __any(ref != 0.0f);
    any_alpha = __any(alpha != 1.0f);
    if (__any(by != 0.0f)) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) sc[kb] -= by;
    }
  };
  uint32_t p[16];                // pairs of weights, in the order of the value products
  float sum;
  auto weights = [&](const v16f (&sc)[2]) __attribute__((always_inline)) {
    float even = 0.0f, odd = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = exp2_fast(sc[i >> 3][2 * (i & 7)]), y = exp2_fast(sc[i >> 3][2 * (i & 7) + 1]);
      p[i] = pack_bf16(x, y);
      if (i & 1) odd = add_pair(p[i], odd);
      else even = add_pair(p[i], even);
    }
    sum = even + odd;
  };
  // Places of the lane's transposed reads: of key 16 u + key0 (+ 8), run 2 d + run0, beside
  // u keys of 16 rows.  (Opaque, or the compiler forms them from their parts in every tile.)
  uint32_t v_at0[ND], v_at8[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    const int key0 = 4 * half + ((lane & 15) >> 2), run = 2 * d + ((lane >> 4) & 1), piece = (lane >> 1) & 1;
    v_at0[d] = v_off<RS>(key0, run, piece) + (lane & 1) * 8;
    v_at8[d] = v_off<RS>(key0 + 8, run, piece) + (lane & 1) * 8;
    asm volatile("" : "+v"(v_at0[d]), "+v"(v_at8[d]));
  }
  auto values = [&](const Stage& s) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {                    // 16 keys each: the same bits of the XOR
      const v8bf w = __builtin_bit_cast(v8bf, make_uint4(p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]));
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(s.v + v_at0[d] + u * 16 * RS));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(s.v + v_at8[d] + u * 16 * RS));
        const v8bf v = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, w, o[d], 0, 0, 0);
      }
    }
  };

  if (t0 < t1) place(t0);
  fetch(t0);
  if (tid < 2 * 64)              // scale bytes of blocks that do not exist: any finite scale; no marks
    reinterpret_cast<uint2*>(st[tid / 64].ks)[tid % 64] = make_uint2(0x7F7F7F7Fu, 0u);
  if (tid < 2) far_at[tid] = make_int2(kNever, kNever);
  if (TREE && tid < 2 * NW) (&far_in[0][0])[tid] = make_int2(-1, 0);
  __syncthreads();
  settle(t0);
  store(st[0]);
  fetch(t0 + 1);
  tile::lds_barrier();
  for (int t = t0; t < t1; ++t) {
    const Stage& s = st[(t - t0) & 1];
    const int j0 = t * TILE;
    const bool work = j0 < seen_hi;   // else no row of the wave sees the tile, nor a later one
    if (work) {
      v16f sc[2];
      const bool any_far = __any(scores(s, sc) != 0);
      if (seen_lo - j0 < TILE || holes) {
        const int left = seen - j0 - half * 4;
        const uint64_t nodes = TREE ? nodes_from(seen_nodes, a.mask_words, j0 - (len - all)) >> (4 * half) : 0;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int pi = (j0 + kb * 32 + g * 16) >> c.page_shift;
            const bool there = !holes || (pi < a.table_stride && (unsigned)table[pi] < (unsigned)c.num_pages);
            const int mine = there ? left : 0;
#pragma unroll
            for (int r = g * 8; r < g * 8 + 8; ++r)
              if (kb * 32 + (r >> 2) * 8 + (r & 3) >= mine ||
                  (TREE && !(nodes >> (kb * 32 + (r >> 2) * 8 + (r & 3)) & 1)))
                sc[kb][r] = kNegInf;
          }
      }
      if (any_ref) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) sc[kb] -= ref;
      }
      // first pass: rows that see their first key; second: rows whose weights are large
      // (rows apart, so that none depends on its neighbours)
      bool over = false;
      for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1 || (__builtin_expect(any_fresh | any_far, 0) && (any_far || __any(fresh && j0 < seen)))) {
          float least = kNegInf;         // the logarithm of what a row has summed
          bool far = false;
          if (pass == 0 && any_far) {
            if constexpr (TREE) {
              // (what a row has seen is noted by stage, as the marks that bring it here are)
              const uint64_t nodes = nodes_from(seen_nodes, a.mask_words, j0 - (len - all));
              uint64_t far_keys = 0, high_keys = 0;
#pragma unroll
              for (int w = 0; w < NW; ++w) {
                const int2 in = far_in[(t - t0) & 1][w];
                const uint32_t keys = in.x == t ? (uint32_t)in.y : 0u;
                far_keys |= (uint64_t)(keys & 0xFFFFu) << (KPW * w);
                high_keys |= (uint64_t)(keys >> 16) << (KPW * w);
              }
              if ((nodes & high_keys) != 0) far_room = kFarRoom;
              if ((nodes & far_keys) != 0) far_seen |= 1u << ((t - t0) & 1);
              far = (far_seen >> ((t - t0) & 1) & 1u) != 0u;
            } else {
              const int2 from = far_at[(t - t0) & 1];
              if (seen > from.y) far_room = kFarRoom;
              far = seen > from.x;
            }
            float tl, th;
            halves(l, tl, th);
            least = __builtin_amdgcn_logf(tl + th);
          }
          raise(sc, over, far, least);
        }
        weights(sc);
        const unsigned long long m = __ballot(!(sum < 0x1p40f));
        if (m == 0) break;
        over = ((m | m >> 32) >> row) & 1;           // in either of the row's lanes
      }
      l += sum;
      if (any_alpha) {
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= alpha;
        any_alpha = false;
        alpha = 1.0f;
      }
    }
    // The next tile goes to the other stage, whose readers were done before the last barrier,
    // between this tile's weights and values: the loads have had a tile's time to arrive, the
    // writes have the value products to land.  (One place for both kinds of wave: with two, the
    // loads on their way are waited for where the paths meet.)
    settle(t + 1);
    store(st[(t + 1 - t0) & 1]);
    if (((t + 2 - t0) & 63) == 0) place(t + 2);
    fetch(t + 2);                // past the range: no loads
    if (work) values(s);
    tile::lds_barrier();
  }
  {
    float lo, hi;
    halves(l, lo, hi);
    l = lo + hi;
  }
  // lane: elements 32 d + 8 (r / 4) + 4 half + r % 4 of its row
  if (a.splits > 1) {
    if (!row_ok) return;
    float* dst = part_sums(a, sp, out_row) + half * 4;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<v4f*>(dst + d * 32 + g * 8) =
            v4f{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    if (half == 0) *part_stats(a, sp, out_row) = make_float2(fresh ? kNegInf : ref, l);
    return;
  }
  const Shares inv = shares(l, c.had);
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    o[d] *= inv.power;
    if (c.had) {   // element bits 0, 1 and 3, 4 are register bits, bit 2 is the lane half
#pragma unroll
      for (int h = 1; h < 16; h <<= 1) {
        if (h == 4) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            float lo, hi;
            halves(o[d][r], lo, hi);
            o[d][r] = half ? lo - hi : lo + hi;
          }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!(r & h)) {
            const float x = o[d][r], y = o[d][r + h];
            o[d][r] = x + y;
            o[d][r + h] = x - y;
          }
      }
    }
    uint32_t w[4][2];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[g][e] = pack_bf16(o[d][4 * g + 2 * e] * inv.rest, o[d][4 * g + 2 * e + 1] * inv.rest);
    // runs g and g + 1 of eight elements: the low half ends with run g, the high one with g + 1
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      const auto x = __builtin_amdgcn_permlane32_swap(w[g][0], w[g + 1][0], false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(w[g][1], w[g + 1][1], false, false);
      const int at = d * 32 + (g + half) * 8;
      if (row_ok && at < c.head_dim)
        *reinterpret_cast<uint4*>(a.out + out_row * c.head_dim + at) = make_uint4(x[0], y[0], x[1], y[1]);
    }
  }
  if (a.lse != nullptr && half == 0 && row_ok)
    a.lse[out_row] = l == 0.0f ? kNegInf : (ref + __builtin_log2f(l)) * 0.6931471805599453f;
}

// Joins the splits of each row: a lane holds four elements of one row, eight lanes a
// block of 32.  WIDE: the groups of lanes of a workgroup share one row's splits (every
// GROUPS-th each) and add up through LDS, for few rows of many splits; else each has a
// row of its own.  Both orders are fixed.  WIDE asks for all it needs at once, also for ranges
// that turn out to have no keys (their sums were never written and are not used): one row of
// 131072 keys 41 -> 39.5 us.  The other form does not: held for eight splits, it took 2% of
// the video shape's time.
template <int NB, bool WIDE>
__global__ void __launch_bounds__(256)
kv_attention_join_kernel(KvAttnArgs a) {
  constexpr int DP = NB * 32;
  constexpr int LPR = 8 * NB;              // lanes of a row
  constexpr int GROUPS = 256 / LPR;
  __shared__ float part[WIDE ? GROUPS : 1][DP], weight[WIDE ? 256 : 1], stats[8];
  static_assert(kMaxSplits <= 256, "one thread a split");
  const int b = blockIdx.y;
  int q0, all, n;
  seq_rows(a, b, q0, all, n);
  const int gr = threadIdx.x / LPR, li = threadIdx.x % LPR, lane = threadIdx.x & 63;
  const int r = WIDE ? blockIdx.x : blockIdx.x * GROUPS + gr;
  if (WIDE && r >= n * a.q_heads) return;
  const bool ok = gr < GROUPS && r < n * a.q_heads;
  const KvCacheArgs& c = a.cache;
  const long long row = (long long)q0 * a.q_heads + (ok ? r : 0);
  float M = kNegInf, L = 0.0f;
  Shares inv;
  v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (WIDE) {
    // one thread a split: maxima and sums at once, the weights to LDS
    constexpr int MINE = (kMaxSplits + GROUPS - 1) / GROUPS;
    float m = kNegInf, w = 0.0f;
    if ((int)threadIdx.x < a.splits) {
      const float2 st = *part_stats(a, threadIdx.x, row);
      m = st.x;
      w = st.y;
    }
    v4f y[MINE];
#pragma unroll
    for (int k = 0; k < MINE; ++k)
      if (ok && gr + k * GROUPS < a.splits)
        y[k] = *reinterpret_cast<const v4f*>(part_sums(a, gr + k * GROUPS, row) + li * 4);
    const bool none = m == kNegInf && w == 0.0f;     // no keys: there are no sums to read
    M = part_top(m, w);
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor(M, k, 64));
    if (lane == 0) stats[threadIdx.x >> 6] = M;
    __syncthreads();
    M = fmaxf(fmaxf(stats[0], stats[1]), fmaxf(stats[2], stats[3]));
    const float f = exp2_fast(m - (M == kNegInf ? 0.0f : M));
    weight[threadIdx.x] = none ? -1.0f : f;
    w *= f;
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) w += __shfl_xor(w, k, 64);
    if (lane == 0) stats[4 + (threadIdx.x >> 6)] = w;
    __syncthreads();
    L = (stats[4] + stats[5]) + (stats[6] + stats[7]);
    inv = shares(L, c.had);
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int s = gr + k * GROUPS;
      if (ok && s < a.splits && !(weight[s] < 0.0f)) x += weight[s] * inv.power * y[k];
    }
  } else if (ok) {
    for (int s = 0; s < a.splits; ++s) {
      const float2 st = *part_stats(a, s, row);
      M = fmaxf(M, part_top(st.x, st.y));
    }
    M += 3.0f;                                         // up to eight sums: less than one together
    const float base = M == kNegInf ? 0.0f : M;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float2 st = *part_stats(a, s, row);
      if (st.x == kNegInf && st.y == 0.0f) continue;   // no keys: there are no sums to read
      const float f = exp2_fast(st.x - base);
      L += f * st.y;
      x += f * *reinterpret_cast<const v4f*>(part_sums(a, s, row) + li * 4);
    }
  }
  if constexpr (WIDE) {
    if (gr < GROUPS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) part[gr][li * 4 + e] = x[e];
    }
    __syncthreads();
    if (gr == 0) {
      for (int k = 1; k < GROUPS; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += part[k][li * 4 + e];
      }
    }
  }
  if constexpr (!WIDE) {
    static_assert(kNarrow <= 8, "the room of the narrow form");
    inv = shares(L, c.had);
    x *= inv.power;
  }
  if (c.had) {
    float v[4] = {x[0], x[1], x[2], x[3]};
    const float a0 = v[0] + v[1], a1 = v[0] - v[1], a2 = v[2] + v[3], a3 = v[2] - v[3];
    v[0] = a0 + a2; v[1] = a1 + a3; v[2] = a0 - a2; v[3] = a1 - a3;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y = lane_xor<1>(v[e]);
      v[e] = (lane & 1) ? y - v[e] : v[e] + y;
      y = lane_xor<2>(v[e]);
      v[e] = (lane & 2) ? y - v[e] : v[e] + y;
      y = lane_xor<4>(v[e]);
      v[e] = (lane & 4) ? y - v[e] : v[e] + y;
    }
    x = v4f{v[0], v[1], v[2], v[3]};
  }
  if (!ok || (WIDE && gr != 0)) return;
  if (li * 4 < c.head_dim)
    *reinterpret_cast<uint2*>(a.out + row * c.head_dim + li * 4) =
        make_uint2(pack_bf16(x[0] * inv.rest, x[1] * inv.rest), pack_bf16(x[2] * inv.rest, x[3] * inv.rest));
  if (a.lse != nullptr && li == 0)
    a.lse[row] = L == 0.0f ? kNegInf : (M + __builtin_log2f(L)) * 0.6931471805599453f;
}

// Rows of a (sequence, key head) that one workgroup takes: 16 (the keys split over its
// waves) while they fit, else 128.  Measured for up to 16 rows, by 16 and by 128: 64 rows
// of up to 8192 keys 87 and 158 us, one row of 131072 keys 40 and 55, of 1000 keys 15 and
// 18.  At 32 rows neither form is ahead: 64 sequences x 4096 keys 92 and 84 us, one of 131072
// keys 43 and 51; at 16 sequences of 64 rows x 8192 keys 89 and 68 us.  Trees of up to 32 rows of more than
// 64 elements go by 16, too: 16 x 32 rows x up to 8192 keys 46 and 51 us, 64 x 32 x 1000 (72 elements) 44 and
// 58, one of 32 x 1000 16.6 and 18.0; with 64 elements 8 x 32 x 4000 45 and 38, one of 20 x 50000 37 and 34.
inline bool few_rows(int max_q, int group, bool tree, int dim_pad) {
  return (long long)max_q * group <= (tree && dim_pad > 64 ? 32 : 16);
}

template <int NB, bool TREE>
hipError_t launch_nb(const KvAttnArgs& a, hipStream_t s) {
  const bool few = few_rows(a.max_q, a.group, TREE, a.cache.dim_pad);
  const int per = few ? 16 : 128;
  const int row_tiles = (int)(((long long)a.max_q * a.group + per - 1) / per);
  const unsigned per_head = (unsigned)((long long)row_tiles * a.splits);
  hipError_t e = hipSuccess;
  if (few) {
    kv_attention_rows16_kernel<NB, TREE><<<dim3(per_head, (unsigned)a.cache.heads, (unsigned)a.seqs), 256, 0, s>>>(a);
    e = hipGetLastError();
  } else {
    // one axis, which is limited to 2^32 threads: as many sequences a launch as fit
    const long long per_seq = (long long)per_head * a.cache.heads;
    const int most = (int)min(max(((1ll << 24) - 1) / per_seq, 1ll), (long long)a.seqs);
    for (int first = 0; first < a.seqs && e == hipSuccess; first += most) {
      KvAttnArgs part = a;
      part.seqs = min(most, a.seqs - first);
      part.cu_q += first;
      part.kv_lens += first;
      part.table += (long long)first * a.table_stride;
      kv_attention_rows128_kernel<NB, TREE><<<(unsigned)(per_seq * part.seqs), 256, 0, s>>>(part);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || a.splits == 1) return e;
  const long long rows = (long long)a.max_q * a.q_heads;
  // A workgroup a row where there are many splits, 32 / NB rows a workgroup where there
  // are few: always wide costs the video shape (3 splits, 81000 rows) 804 us for 420, narrow up
  // to 32 splits one sequence of 32 rows x 8192 keys 34 us for 17.
  if (a.splits > kNarrow) {
    kv_attention_join_kernel<NB, true><<<dim3((unsigned)rows, (unsigned)a.seqs), 256, 0, s>>>(a);
  } else {
    constexpr int RPW = 256 / (8 * NB);
    kv_attention_join_kernel<NB, false><<<dim3((unsigned)((rows + RPW - 1) / RPW), (unsigned)a.seqs), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

int splits_of(int seqs, int max_q, int q_heads, int kv_heads, int max_kv, bool tree, int dim_pad) {
  if (seqs <= 0 || max_q <= 0 || kv_heads <= 0) return 1;
  const int group = q_heads / kv_heads;
  const bool few = few_rows(max_q, group, tree, dim_pad);
  const long long row_tiles = ((long long)max_q * group + (few ? 15 : 127)) / (few ? 16 : 128);
  const long long base = (long long)seqs * kv_heads * row_tiles;
  const long long tiles = ((long long)max_kv + TILE - 1) / TILE;
  if (few) {
    // Two workgroups a CU, of at least four tiles (one a wave) each: a workgroup spends
    // about 8 us on its start and end, so more of them cost more than they balance (one
    // row of 131072 keys: 64 splits 44 us, 96 45, 128 52 then; 64 rows of 5000 keys: 73 us
    // unsplit, 81 in halves, 79 in thirds; of 1 to 10000 keys: 86, 92 and 81).
    long long want = (2ll * NUM_CUS + base - 1) / base;
    const long long most = (tiles + 3) / 4;
    want = want < most ? want : most;
    if (want > kMaxSplits) want = kMaxSplits;
    return want < 1 ? 1 : (int)want;
  }
  // 128 rows: the splits whose rounds of workgroups over the chip's slots take least.  A
  // range costs its tiles and about six more to start; each split's partial sums cost the
  // chip about one tile's time a row tile in two slots.  Two slots a CU are counted for every
  // head size: up to 64 elements a third workgroup fits, but the three share the vector units,
  // so a round of three takes longer.  By two and by three (64 elements, us): 2700 rows x 17776
  // keys x 30 heads 404 and 423, 17776 x 17776 x 6 504 and 527, 4096 x 4096 x 16 83 and 95, four of
  // 256 x 2048 x 16 28 and 31; 512 x 8192 x 30 54 and 53, two of 1000 x 3000 x 20 58 and 55.
  const long long slots = 2ll * NUM_CUS;
  long long best = 0;
  int splits = 1;
  for (int n = 1; n <= 64 && n <= (tiles + 3) / 4; ++n) {
    const long long rounds = (base * n + slots - 1) / slots;
    const long long cost = rounds * ((tiles + n - 1) / n + 6) + (n > 1 ? (base * n + slots - 1) / slots * 4 : 0);
    if (n == 1 || cost < best) {
      best = cost;
      splits = n;
    }
  }
  return splits;
}

template <bool TREE>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  switch (a.cache.dim_pad) {
    case 32: return launch_nb<1, TREE>(a, s);
    case 64: return launch_nb<2, TREE>(a, s);
    case 96: return launch_nb<3, TREE>(a, s);
    case 128: return launch_nb<4, TREE>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

int kv_attention_splits(int seqs, int max_q, int q_heads, int kv_heads, int max_kv) {
  return splits_of(seqs, max_q, q_heads, kv_heads, max_kv, false, 0);
}

hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t s) { return launch<false>(a, s); }

int kv_tree_splits(int seqs, int max_q, int q_heads, int kv_heads, int max_kv, int dim_pad) {
  return splits_of(seqs, max_q, q_heads, kv_heads, max_kv, true, dim_pad);
}

hipError_t launch_kv_tree_attention(const KvAttnArgs& a, hipStream_t s) { return launch<true>(a, s); }

}  // namespace tabit
