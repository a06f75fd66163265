// Device helpers of the kernels that take query rows to the paged cache (attention, weights):
// a sequence's rows and lengths, and a query prepared as the cached keys are.
#pragma once

#include "kv_common.h"

namespace tabit {
namespace kv {

// Factor of the products q'.k' that gives scores in base 2.
__device__ __forceinline__ float base2_scale(const KvAttnArgs& a) {
  return a.scale * 1.4426950408889634f / (a.cache.had ? 32.0f : 1.0f);
}

// 32 elements of a query row (block `blk` of the head vector), rotated and
// transformed as the cache's keys are, times `factor`.  All loads are issued before
// the first use: elements past the head, and tables outside the rotated part, are
// read at a valid place and replaced.
__device__ __forceinline__ bool load_q_block(const KvAttnArgs& a, int token, int head, int blk,
                                             float factor, float (&x)[32]) {
  const int D = a.cache.head_dim, R = a.rope.rope_dim;
  const uint16_t* p = a.q + (long long)token * a.q_stride + (long long)head * D;
  bool ok = true;
  uint4 own[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e0 = blk * 32 + i * 8;
    own[i] = *reinterpret_cast<const uint4*>(p + (e0 < D ? e0 : 0));
  }
  auto spread = [](uint4 w, float* v) {
    v[0] = bf_lo(w.x); v[1] = bf_hi(w.x); v[2] = bf_lo(w.y); v[3] = bf_hi(w.y);
    v[4] = bf_lo(w.z); v[5] = bf_hi(w.z); v[6] = bf_lo(w.w); v[7] = bf_hi(w.w);
  };
  if (R > 0) {
    const int pos = a.positions[token];
    ok = pos >= 0 && pos < a.rope.num_positions;
    const int half = R >> 1;
    const float* cos = a.rope.cos + (ok ? (size_t)pos * half : 0);
    const float* sin = a.rope.sin + (ok ? (size_t)pos * half : 0);
    if (a.rope.interleaved) {
      float4 c[4], s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e0 = blk * 32 + i * 8, at = e0 < R ? e0 >> 1 : 0;
        c[i] = *reinterpret_cast<const float4*>(cos + at);
        s[i] = *reinterpret_cast<const float4*>(sin + at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        spread(own[i], x + 8 * i);
        if (blk * 32 + i * 8 < R) {
          turn(x[8 * i], x[8 * i + 1], c[i].x, s[i].x);
          turn(x[8 * i + 2], x[8 * i + 3], c[i].y, s[i].y);
          turn(x[8 * i + 4], x[8 * i + 5], c[i].z, s[i].z);
          turn(x[8 * i + 6], x[8 * i + 7], c[i].w, s[i].w);
        }
      }
    } else {
      uint4 other[4];
      float4 c[8], s[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e0 = blk * 32 + i * 8;
        const bool second = e0 >= half;
        const int at = e0 < R ? (second ? e0 - half : e0) : 0;
        other[i] = *reinterpret_cast<const uint4*>(p + (e0 < R ? (second ? e0 - half : e0 + half) : 0));
        const uint32_t sign = second ? 0u : 0x80008000u;   // the first of a pair takes -other sin
        other[i] = make_uint4(other[i].x ^ sign, other[i].y ^ sign, other[i].z ^ sign, other[i].w ^ sign);
        c[2 * i] = *reinterpret_cast<const float4*>(cos + at);
        c[2 * i + 1] = *reinterpret_cast<const float4*>(cos + at + 4);
        s[2 * i] = *reinterpret_cast<const float4*>(sin + at);
        s[2 * i + 1] = *reinterpret_cast<const float4*>(sin + at + 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e0 = blk * 32 + i * 8;
        spread(own[i], x + 8 * i);
        float y[8];
        spread(other[i], y);
        const float cc[8] = {c[2 * i].x, c[2 * i].y, c[2 * i].z, c[2 * i].w,
                             c[2 * i + 1].x, c[2 * i + 1].y, c[2 * i + 1].z, c[2 * i + 1].w};
        const float ss[8] = {s[2 * i].x, s[2 * i].y, s[2 * i].z, s[2 * i].w,
                             s[2 * i + 1].x, s[2 * i + 1].y, s[2 * i + 1].z, s[2 * i + 1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[8 * i + e] * cc[e], w = y[e] * ss[e];
          x[8 * i + e] = e0 >= R ? x[8 * i + e] : u + w;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) spread(own[i], x + 8 * i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (blk * 32 + i * 8 >= D) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * i + e] = 0.0f;
    }
  if (a.cache.had) fwht32_lane(x);
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] *= factor;
  return ok;
}

// First query row of sequence b, its queries, inside [0, tokens], and how many of them are
// computed.
__device__ __forceinline__ void seq_rows(const KvAttnArgs& a, int b, int& q0, int& all, int& n) {
  q0 = min(max(a.cu_q[b], 0), a.tokens);
  all = max(min(a.cu_q[b + 1], a.tokens) - q0, 0);
  n = min(all, a.max_q);
}

__device__ __forceinline__ int seq_keys(const KvAttnArgs& a, int b) {
  return min(max(a.kv_lens[b], 0), a.max_kv);
}

// Keys that query i of `all` sees, of `len`.
__device__ __forceinline__ int seen_keys(const KvAttnArgs& a, int len, int all, int i) {
  return a.causal ? min(max(len - all + i + 1, 0), len) : len;
}

// Trees of drafted tokens.  Keys that every row sees: those before the tree's.
__device__ __forceinline__ int before_tree(int len, int all) { return min(max(len - all, 0), len); }

// Which of nodes [from, from + 64) a row sees, by its row of the mask; keys before the tree
// (negative) are all seen, nodes past the mask's words are not.
__device__ __forceinline__ uint64_t nodes_from(const uint64_t* row, int words, int from) {
  const int w = from >> 6, s = from & 63;
  const uint64_t lo = w < 0 ? ~0ull : w < words ? row[w] : 0ull;
  const uint64_t hi = w + 1 < 0 ? ~0ull : w + 1 < words ? row[w + 1] : 0ull;
  return s == 0 ? lo : lo >> s | hi << (64 - s);
}

}  // namespace kv
}  // namespace tabit
