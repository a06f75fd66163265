// Checks that the entry points of the paged cache and of attention over it share.
#pragma once

#include "api_common.h"

#include <climits>
#include <cmath>

namespace {

constexpr int kMaxHeadDim = 128;

// Shape of a cache and alignment of its arrays; fills the kernels' form of it.
int check_cache(tabit_ctx* ctx, const tabit_kv_cache* c, tabit::KvCacheArgs* out) {
  if (c == nullptr) return fail(ctx, TABIT_EINVAL, "null cache");
  if (c->head_dim < 8 || c->head_dim > kMaxHeadDim || c->head_dim % 8 != 0)
    return fail(ctx, TABIT_ESHAPE, "head_dim must be a multiple of 8 in [8, %d] (got %d)", kMaxHeadDim,
                c->head_dim);
  if (c->num_kv_heads < 1 || c->num_kv_heads > 65535)
    return fail(ctx, TABIT_ESHAPE, "num_kv_heads must be in [1, 65535] (got %d)", c->num_kv_heads);
  if (c->page_size < 16 || (c->page_size & (c->page_size - 1)) != 0 || c->page_size > (1 << 20))
    return fail(ctx, TABIT_ESHAPE, "page_size must be a power of two in [16, 2^20] (got %d)", c->page_size);
  if (c->num_pages < 0) return fail(ctx, TABIT_ESHAPE, "num_pages must be >= 0 (got %d)", c->num_pages);
  if (c->had_block != 0 && c->had_block != 32)
    return fail(ctx, TABIT_ERANGE, "a cache takes had_block 0 or 32 (got %d)", c->had_block);
  if (c->num_pages > 0) {
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
      return fail(ctx, TABIT_EINVAL, "null cache array");
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4))
      return fail(ctx, TABIT_EALIGN, "cache codes must be 16-byte aligned, scales 4-byte");
  }
  out->k_codes = c->k_codes;
  out->k_scales = c->k_scales;
  out->v_codes = c->v_codes;
  out->v_scales = c->v_scales;
  out->num_pages = c->num_pages;
  out->page_shift = __builtin_ctz((unsigned)c->page_size);
  out->heads = c->num_kv_heads;
  out->head_dim = c->head_dim;
  out->dim_pad = (c->head_dim + 31) / 32 * 32;
  out->had = c->had_block == 32;
  return TABIT_OK;
}

int check_rope(tabit_ctx* ctx, const tabit_rope* r, const int32_t* positions, int head_dim,
               tabit::RopeArgs* out) {
  *out = tabit::RopeArgs{};
  if (r == nullptr) return TABIT_OK;
  if (r->cos == nullptr || r->sin == nullptr || positions == nullptr)
    return fail(ctx, TABIT_EINVAL, "a rotation needs cos, sin and positions");
  if (r->rope_dim < 16 || r->rope_dim > head_dim || r->rope_dim % 16 != 0)
    return fail(ctx, TABIT_ESHAPE, "rope_dim must be a multiple of 16 in [16, head_dim = %d] (got %d)",
                head_dim, r->rope_dim);
  if (r->num_positions < 1)
    return fail(ctx, TABIT_ESHAPE, "num_positions must be >= 1 (got %d)", r->num_positions);
  if (!aligned(r->cos, 16) || !aligned(r->sin, 16) || !aligned(positions, 4))
    return fail(ctx, TABIT_EALIGN, "cos and sin must be 16-byte aligned, positions 4-byte");
  out->cos = r->cos;
  out->sin = r->sin;
  out->num_positions = r->num_positions;
  out->rope_dim = r->rope_dim;
  out->interleaved = r->interleaved != 0;
  return TABIT_OK;
}

// Shapes, pointers and alignment of an attention-like call (out_ok: its output is as it should
// be); fills the kernels' form of it but for the splits and the workspace.
int check_attention(tabit_ctx* ctx, const tabit_kv_cache* cache, const tabit_kv_attention_args* a, bool out_ok,
                    tabit::KvAttnArgs* k) {
  int st = check_cache(ctx, cache, &k->cache);
  if (st != TABIT_OK) return st;
  st = check_rope(ctx, a->rope, a->positions, k->cache.head_dim, &k->rope);
  if (st != TABIT_OK) return st;
  if (a->num_tokens < 0 || a->num_seqs < 0 || a->max_q < 0 || a->max_kv < 0)
    return fail(ctx, TABIT_ESHAPE, "num_tokens, num_seqs, max_q and max_kv must be >= 0");
  if (a->num_q_heads < 1 || a->num_q_heads % k->cache.heads != 0)
    return fail(ctx, TABIT_ESHAPE, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)",
                a->num_q_heads, k->cache.heads);
  if (a->num_seqs > 65535) return fail(ctx, TABIT_ESHAPE, "at most 65535 sequences (got %d)", a->num_seqs);
  if (a->q == nullptr || !out_ok || a->cu_q == nullptr || a->kv_lens == nullptr)
    return fail(ctx, TABIT_EINVAL, "null pointer");
  if (a->max_kv > 0 && a->block_table == nullptr) return fail(ctx, TABIT_EINVAL, "null block_table");
  if (a->max_kv > 0 && (a->table_stride < 1 || (int64_t)a->table_stride * cache->page_size < a->max_kv))
    return fail(ctx, TABIT_ESHAPE, "a table row of %d pages of %d tokens does not hold max_kv = %d",
                a->table_stride, cache->page_size, a->max_kv);
  const int64_t row = (int64_t)a->num_q_heads * k->cache.head_dim;
  if (a->q_stride < row || a->q_stride % 8 != 0)
    return fail(ctx, TABIT_ESHAPE, "q_stride must be a multiple of 8 of at least %lld elements",
                (long long)row);
  if (!std::isfinite(a->scale)) return fail(ctx, TABIT_EINVAL, "scale is not finite");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->cu_q, 4) || !aligned(a->kv_lens, 4) ||
      !aligned(a->block_table, 4) || !aligned(a->lse, 4) || !aligned(a->ws, 16))
    return fail(ctx, TABIT_EALIGN, "q, out and ws must be 16-byte aligned, the others 4-byte");
  k->q = a->q;
  k->q_stride = a->q_stride;
  k->tokens = a->num_tokens;
  k->q_heads = a->num_q_heads;
  k->group = a->num_q_heads / k->cache.heads;
  k->cu_q = a->cu_q;
  k->seqs = a->num_seqs;
  k->max_q = a->max_q;
  k->table = a->block_table;
  k->table_stride = a->table_stride;
  k->kv_lens = a->kv_lens;
  k->max_kv = a->max_kv;
  k->scale = a->scale;
  k->causal = a->causal != 0;
  k->positions = a->positions;
  k->out = a->out;
  k->lse = a->lse;
  return TABIT_OK;
}

}  // namespace
