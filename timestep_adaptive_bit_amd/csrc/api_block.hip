// extern "C" entry points of the operators between a block's linears (declared in
// include/tabit.h): the paged MXFP4 cache, attention over it, the block norms.
// Arguments are validated completely before the first HIP call; kernels go to the
// caller's stream; no device memory is allocated here.
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

bool valid_norm(int kind) {
  return kind == TABIT_NORM_NONE || kind == TABIT_NORM_LAYER || kind == TABIT_NORM_RMS;
}

}  // namespace

extern "C" {

int tabit_kv_append(tabit_ctx* ctx, const tabit_kv_cache* cache, const uint16_t* k_bf16,
                    int64_t k_stride, const uint16_t* v_bf16, int64_t v_stride, int num_tokens,
                    const int64_t* slots, const tabit_rope* rope, const int32_t* positions,
                    void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  tabit::KvCacheArgs c;
  int st = check_cache(ctx, cache, &c);
  if (st != TABIT_OK) return st;
  if (num_tokens < 0) return fail(ctx, TABIT_ESHAPE, "num_tokens must be >= 0 (got %d)", num_tokens);
  tabit::RopeArgs r;
  st = check_rope(ctx, rope, positions, c.head_dim, &r);
  if (st != TABIT_OK) return st;
  if (k_bf16 == nullptr || v_bf16 == nullptr || slots == nullptr)
    return fail(ctx, TABIT_EINVAL, "null pointer");
  const int64_t row = (int64_t)c.heads * c.head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(ctx, TABIT_ESHAPE, "token strides must be multiples of 8 of at least %lld elements",
                (long long)row);
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(slots, 8))
    return fail(ctx, TABIT_EALIGN, "k and v must be 16-byte aligned, slots 8-byte");
  if (num_tokens == 0 || c.num_pages == 0) return TABIT_OK;
  return hip_status(ctx,
                    tabit::launch_kv_append(c, k_bf16, k_stride, v_bf16, v_stride, num_tokens, slots, r,
                                            positions, static_cast<hipStream_t>(stream)),
                    "kv_append launch");
}

int tabit_kv_read(tabit_ctx* ctx, const tabit_kv_cache* cache, const int64_t* slots, int num_tokens,
                  uint16_t* k_bf16, uint16_t* v_bf16, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  tabit::KvCacheArgs c;
  int st = check_cache(ctx, cache, &c);
  if (st != TABIT_OK) return st;
  if (num_tokens < 0) return fail(ctx, TABIT_ESHAPE, "num_tokens must be >= 0 (got %d)", num_tokens);
  if (slots == nullptr || k_bf16 == nullptr || v_bf16 == nullptr)
    return fail(ctx, TABIT_EINVAL, "null pointer");
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(slots, 8))
    return fail(ctx, TABIT_EALIGN, "k and v must be 16-byte aligned, slots 8-byte");
  if (num_tokens == 0) return TABIT_OK;
  return hip_status(ctx,
                    tabit::launch_kv_read(c, slots, num_tokens, k_bf16, v_bf16,
                                          static_cast<hipStream_t>(stream)),
                    "kv_read launch");
}

size_t tabit_kv_attention_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads,
                                          int head_dim, int num_seqs, int max_q, int max_kv) {
  if (num_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_seqs <= 0 ||
      max_q <= 0 || max_kv <= 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  const int splits = tabit::kv_attention_splits(num_seqs, max_q, num_q_heads, num_kv_heads, max_kv);
  if (splits <= 1) return 0;
  const size_t rows = (size_t)num_tokens * (size_t)num_q_heads;
  return (size_t)splits * rows * (size_t)((head_dim + 31) / 32 * 32 + 2) * sizeof(float);
}

int tabit_kv_attention(tabit_ctx* ctx, const tabit_kv_cache* cache, const tabit_kv_attention_args* a,
                       void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (a == nullptr) return fail(ctx, TABIT_EINVAL, "null arguments");
  tabit::KvAttnArgs k{};
  int st = check_cache(ctx, cache, &k.cache);
  if (st != TABIT_OK) return st;
  st = check_rope(ctx, a->rope, a->positions, k.cache.head_dim, &k.rope);
  if (st != TABIT_OK) return st;
  if (a->num_tokens < 0 || a->num_seqs < 0 || a->max_q < 0 || a->max_kv < 0)
    return fail(ctx, TABIT_ESHAPE, "num_tokens, num_seqs, max_q and max_kv must be >= 0");
  if (a->num_q_heads < 1 || a->num_q_heads % k.cache.heads != 0)
    return fail(ctx, TABIT_ESHAPE, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)",
                a->num_q_heads, k.cache.heads);
  if (a->num_seqs > 65535) return fail(ctx, TABIT_ESHAPE, "at most 65535 sequences (got %d)", a->num_seqs);
  if (a->q == nullptr || a->out == nullptr || a->cu_q == nullptr || a->kv_lens == nullptr)
    return fail(ctx, TABIT_EINVAL, "null pointer");
  if (a->max_kv > 0 && a->block_table == nullptr) return fail(ctx, TABIT_EINVAL, "null block_table");
  if (a->max_kv > 0 && (a->table_stride < 1 || (int64_t)a->table_stride * cache->page_size < a->max_kv))
    return fail(ctx, TABIT_ESHAPE, "a table row of %d pages of %d tokens does not hold max_kv = %d",
                a->table_stride, cache->page_size, a->max_kv);
  const int64_t row = (int64_t)a->num_q_heads * k.cache.head_dim;
  if (a->q_stride < row || a->q_stride % 8 != 0)
    return fail(ctx, TABIT_ESHAPE, "q_stride must be a multiple of 8 of at least %lld elements",
                (long long)row);
  if (!std::isfinite(a->scale)) return fail(ctx, TABIT_EINVAL, "scale is not finite");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->cu_q, 4) || !aligned(a->kv_lens, 4) ||
      !aligned(a->block_table, 4) || !aligned(a->lse, 4) || !aligned(a->ws, 16))
    return fail(ctx, TABIT_EALIGN, "q, out and ws must be 16-byte aligned, the others 4-byte");
  if (a->num_tokens == 0 || a->num_seqs == 0 || a->max_q == 0) return TABIT_OK;
  k.splits = tabit::kv_attention_splits(a->num_seqs, a->max_q, a->num_q_heads, k.cache.heads, a->max_kv);
  if ((int64_t)a->max_q * a->num_q_heads > INT_MAX / 64 ||
      (int64_t)a->max_q * a->num_q_heads * k.splits * a->num_seqs > INT_MAX)
    return fail(ctx, TABIT_ESHAPE, "max_q * num_q_heads * num_seqs is too large (%d * %d * %d)", a->max_q,
                a->num_q_heads, a->num_seqs);
  const size_t need =
      tabit_kv_attention_workspace_bytes(a->num_tokens, a->num_q_heads, k.cache.heads, k.cache.head_dim,
                                         a->num_seqs, a->max_q, a->max_kv);
  if (need > 0 && a->ws == nullptr) return fail(ctx, TABIT_EINVAL, "null ws (%zu bytes needed)", need);
  if (a->ws_bytes < need)
    return fail(ctx, TABIT_ESHAPE, "ws holds %zu bytes, %zu needed", a->ws_bytes, need);
  k.q = a->q;
  k.q_stride = a->q_stride;
  k.tokens = a->num_tokens;
  k.q_heads = a->num_q_heads;
  k.group = a->num_q_heads / k.cache.heads;
  k.cu_q = a->cu_q;
  k.seqs = a->num_seqs;
  k.max_q = a->max_q;
  k.table = a->block_table;
  k.table_stride = a->table_stride;
  k.kv_lens = a->kv_lens;
  k.max_kv = a->max_kv;
  k.scale = a->scale;
  k.causal = a->causal != 0;
  k.positions = a->positions;
  k.out = a->out;
  k.lse = a->lse;
  k.part = static_cast<float*>(a->ws);
  return hip_status(ctx, tabit::launch_kv_attention(k, static_cast<hipStream_t>(stream)),
                    "kv_attention launch");
}

int tabit_block_norm(tabit_ctx* ctx, const tabit_block_norm_args* a, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (a == nullptr || a->x == nullptr) return fail(ctx, TABIT_EINVAL, "null pointer");
  if (a->rows < 0) return fail(ctx, TABIT_ESHAPE, "rows must be >= 0 (got %d)", a->rows);
  if (a->width < 32 || a->width > 32768 || a->width % 32 != 0)
    return fail(ctx, TABIT_ESHAPE, "width must be a multiple of 32 in [32, 32768] (got %d)", a->width);
  if (!valid_norm(a->post_kind) || !valid_norm(a->pre_kind))
    return fail(ctx, TABIT_EINVAL, "unknown norm kind (post %d, pre %d)", a->post_kind, a->pre_kind);
  if (a->y == nullptr && (a->post_kind != TABIT_NORM_NONE || a->post_weight != nullptr || a->gate != nullptr))
    return fail(ctx, TABIT_EINVAL, "a post norm, its weight or a gate needs y");
  if ((a->post_kind == TABIT_NORM_NONE && a->post_weight != nullptr) ||
      (a->pre_kind == TABIT_NORM_NONE && a->pre_weight != nullptr))
    return fail(ctx, TABIT_EINVAL, "a norm weight needs a norm");
  if (a->x_out == nullptr && a->h == nullptr) return fail(ctx, TABIT_EINVAL, "no output requested");
  if (!std::isfinite(a->res_scale) || !(a->eps >= 0.0f) || !std::isfinite(a->eps))
    return fail(ctx, TABIT_EINVAL, "res_scale must be finite, eps finite and >= 0");
  if (a->h == nullptr && (a->pre_kind != TABIT_NORM_NONE || a->scale != nullptr || a->shift != nullptr))
    return fail(ctx, TABIT_EINVAL, "a pre norm, scale or shift needs h");
  if (a->h != nullptr) {
    if (a->fmt != TABIT_FMT_BF16 && a->fmt != TABIT_FMT_INT8 && a->fmt != TABIT_FMT_MXFP4)
      return fail(ctx, TABIT_EINVAL, "unknown fmt %d", a->fmt);
    const int b = a->had_block;
    if (b != 0 && (a->fmt == TABIT_FMT_BF16 || (b != 32 && (a->fmt == TABIT_FMT_MXFP4 || (b != 64 && b != 128)))))
      return fail(ctx, TABIT_ERANGE, "had_block is 0 for bf16, 0 or 32 for MXFP4, 0, 32, 64 or 128 for INT8 (got %d)", b);
    if (b != 0 && a->width % b != 0)
      return fail(ctx, TABIT_ESHAPE, "width (%d) must be a multiple of had_block (%d)", a->width, b);
    if (a->fmt != TABIT_FMT_BF16 && a->h_scale == nullptr)
      return fail(ctx, TABIT_EINVAL, "a quantized h needs h_scale");
  }
  const bool mod = a->gate != nullptr || a->scale != nullptr || a->shift != nullptr;
  if (mod && a->rows_per_sample < 1)
    return fail(ctx, TABIT_ESHAPE, "rows_per_sample must be >= 1 (got %d)", a->rows_per_sample);
  if (mod && (a->num_samples < 0 || (int64_t)a->num_samples * a->rows_per_sample < a->rows))
    return fail(ctx, TABIT_ESHAPE, "%d samples of %d rows do not hold %d rows", a->num_samples,
                a->rows_per_sample, a->rows);
  if (mod && (a->mod_stride < a->width || a->mod_stride % 8 != 0))
    return fail(ctx, TABIT_ESHAPE, "mod_stride must be a multiple of 8 of at least width elements");
  if (!aligned(a->x, 16) || !aligned(a->y, 16) || !aligned(a->post_weight, 16) ||
      !aligned(a->pre_weight, 16) || !aligned(a->gate, 16) || !aligned(a->scale, 16) ||
      !aligned(a->shift, 16) || !aligned(a->x_out, 16) || !aligned(a->h, 16) ||
      (a->fmt == TABIT_FMT_INT8 && !aligned(a->h_scale, 4)))
    return fail(ctx, TABIT_EALIGN, "misaligned pointer");
  if (a->rows == 0) return TABIT_OK;
  tabit::BlockNormArgs k{};
  k.x = a->x;
  k.y = a->y;
  k.rows = a->rows;
  k.width = a->width;
  k.post_kind = a->post_kind;
  k.pre_kind = a->pre_kind;
  k.post_w = a->post_weight;
  k.pre_w = a->pre_weight;
  k.gate = a->gate;
  k.scale = a->scale;
  k.shift = a->shift;
  k.mod_stride = mod ? a->mod_stride : 0;
  k.rows_per_sample = mod ? a->rows_per_sample : a->rows;   // one sample: weights are read once a wave
  k.res_scale = a->res_scale;
  k.eps = a->eps;
  k.x_out = a->x_out;
  k.h = a->h;
  k.h_scale = a->h_scale;
  k.fmt = a->fmt;
  k.had = a->had_block;
  return hip_status(ctx, tabit::launch_block_norm(k, static_cast<hipStream_t>(stream)),
                    "block_norm launch");
}

}  // extern "C"
