// extern "C" entry points of the operators for serving many requests (declared in
// include/tabit.h): trees of drafted tokens, eviction from the cache, low-rank adapters.
// Arguments are validated completely before the first HIP call; kernels go to the
// caller's stream; no device memory is allocated here.
#include "api_cache.h"

#include <cstdlib>

namespace {

using tabit::kMaxNodes;
constexpr int kMaxKeys = 1 << 30;    // of a sequence: kernels step past the last one by less than as many again

// Sizes that an attention-like launch takes.
int check_grid(tabit_ctx* ctx, const tabit_kv_attention_args* a, int splits) {
  if ((int64_t)a->max_q * a->num_q_heads > INT_MAX / 64 ||
      (int64_t)a->max_q * a->num_q_heads * splits * a->num_seqs > INT_MAX)
    return fail(ctx, TABIT_ESHAPE, "max_q * num_q_heads * num_seqs is too large (%d * %d * %d)", a->max_q,
                a->num_q_heads, a->num_seqs);
  return TABIT_OK;
}

int check_ws(tabit_ctx* ctx, const void* ws, size_t bytes, size_t need) {
  if (need > 0 && ws == nullptr) return fail(ctx, TABIT_EINVAL, "null ws (%zu bytes needed)", need);
  if (bytes < need) return fail(ctx, TABIT_ESHAPE, "ws holds %zu bytes, %zu needed", bytes, need);
  return TABIT_OK;
}

// A block table for sequences of up to max_kv tokens.
int check_table(tabit_ctx* ctx, const int32_t* table, int stride, int num_seqs) {
  if (num_seqs < 0) return fail(ctx, TABIT_ESHAPE, "num_seqs must be >= 0 (got %d)", num_seqs);
  if (num_seqs > 65535) return fail(ctx, TABIT_ESHAPE, "at most 65535 sequences (got %d)", num_seqs);
  if (table == nullptr) return fail(ctx, TABIT_EINVAL, "null block_table");
  if (stride < 1) return fail(ctx, TABIT_ESHAPE, "table_stride must be >= 1 (got %d)", stride);
  return TABIT_OK;
}

bool valid_sizes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int num_seqs, int max_q,
                 int max_kv) {
  return num_tokens > 0 && num_q_heads > 0 && num_kv_heads > 0 && head_dim > 0 && num_seqs > 0 && max_q > 0 &&
         max_kv > 0 && num_q_heads % num_kv_heads == 0;
}

// Whether n bytes at p and m at q share one.
bool meet(const void* p, uint64_t n, const void* q, uint64_t m) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && (a < b ? b - a < n : a - b < m);
}

// Whether `rows` rows of n bytes, `step` bytes (n at least) apart from p on, share a byte with as many of m bytes
// from q on.  Columns of one wider matrix do not.
bool rows_meet(const void* p, int64_t n, int64_t step, const void* q, int64_t m, int64_t q_step, int rows) {
  if (rows == 1) return meet(p, (uint64_t)n, q, (uint64_t)m);
  const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(p), b = (int64_t)reinterpret_cast<uintptr_t>(q);
  if (a + (rows - 1) * step + n <= b || b + (rows - 1) * q_step + m <= a) return false;
  if (step == q_step) {          // row i + k of p and row i of q are b - a - k step apart
    const int64_t d = b - a, k = d >= 0 ? d / step : -((-d + step - 1) / step), r = d - k * step;      // 0 <= r < step
    return (r < n && std::abs(k) < rows) || (step - r < m && std::abs(k + 1) < rows);
  }
  for (int64_t i = 0, j = 0; i < rows && j < rows;) {
    const int64_t x = a + i * step, y = b + j * q_step;
    if (x + n <= y) ++i;
    else if (y + m <= x) ++j;
    else return true;
  }
  return false;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t tabit_kv_tree_attention_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                               int num_seqs, int max_q, int max_kv) {
  if (!valid_sizes(num_tokens, num_q_heads, num_kv_heads, head_dim, num_seqs, max_q, max_kv)) return 0;
  const int splits = tabit::kv_tree_splits(num_seqs, max_q, num_q_heads, num_kv_heads, max_kv, (head_dim + 31) / 32 * 32);
  if (splits <= 1) return 0;
  return (size_t)splits * (size_t)num_tokens * (size_t)num_q_heads * (size_t)((head_dim + 31) / 32 * 32 + 2) *
         sizeof(float);
}

int tabit_kv_tree_attention(tabit_ctx* ctx, const tabit_kv_cache* cache, const tabit_kv_attention_args* a,
                            const uint64_t* mask, int mask_words, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (a == nullptr) return fail(ctx, TABIT_EINVAL, "null arguments");
  tabit::KvAttnArgs k{};
  int st = check_attention(ctx, cache, a, a->out != nullptr, &k);
  if (st != TABIT_OK) return st;
  if (a->causal != 0) return fail(ctx, TABIT_EINVAL, "a tree has its mask: causal must be 0");
  if (a->max_q > kMaxNodes) return fail(ctx, TABIT_ESHAPE, "at most %d nodes of a sequence (got %d)", kMaxNodes, a->max_q);
  if (mask == nullptr) return fail(ctx, TABIT_EINVAL, "null mask");
  if (mask_words < 1 || mask_words < (a->max_q + 63) / 64)
    return fail(ctx, TABIT_ESHAPE, "%d words do not hold the mask of %d nodes", mask_words, a->max_q);
  if (!aligned(mask, 8)) return fail(ctx, TABIT_EALIGN, "mask must be 8-byte aligned");
  if (a->num_tokens == 0 || a->num_seqs == 0 || a->max_q == 0) return TABIT_OK;
  k.splits = tabit::kv_tree_splits(a->num_seqs, a->max_q, a->num_q_heads, k.cache.heads, a->max_kv, k.cache.dim_pad);
  if ((st = check_grid(ctx, a, k.splits)) != TABIT_OK) return st;
  const size_t need = tabit_kv_tree_attention_workspace_bytes(
      a->num_tokens, a->num_q_heads, k.cache.heads, k.cache.head_dim, a->num_seqs, a->max_q, a->max_kv);
  if ((st = check_ws(ctx, a->ws, a->ws_bytes, need)) != TABIT_OK) return st;
  k.part = static_cast<float*>(a->ws);
  k.mask = mask;
  k.mask_words = mask_words;
  return hip_status(ctx, tabit::launch_kv_tree_attention(k, static_cast<hipStream_t>(stream)),
                    "kv_tree_attention launch");
}

int tabit_tree_mask(tabit_ctx* ctx, const int32_t* parents, int num_tokens, const int32_t* cu_q, int num_seqs,
                    int max_q, uint64_t* mask, int mask_words, int32_t* depth, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (num_tokens < 0 || num_seqs < 0 || max_q < 0)
    return fail(ctx, TABIT_ESHAPE, "num_tokens, num_seqs and max_q must be >= 0");
  if (max_q > kMaxNodes) return fail(ctx, TABIT_ESHAPE, "at most %d nodes of a sequence (got %d)", kMaxNodes, max_q);
  if (parents == nullptr || cu_q == nullptr || mask == nullptr) return fail(ctx, TABIT_EINVAL, "null pointer");
  if (mask_words < 1 || mask_words < (max_q + 63) / 64)
    return fail(ctx, TABIT_ESHAPE, "%d words do not hold the mask of %d nodes", mask_words, max_q);
  if (!aligned(mask, 8) || !aligned(parents, 4) || !aligned(cu_q, 4) || !aligned(depth, 4))
    return fail(ctx, TABIT_EALIGN, "mask must be 8-byte aligned, the others 4-byte");
  if (num_tokens == 0 || num_seqs == 0 || max_q == 0) return TABIT_OK;
  return hip_status(ctx,
                    tabit::launch_tree_mask(parents, num_tokens, cu_q, num_seqs, max_q, mask, mask_words, depth,
                                            static_cast<hipStream_t>(stream)),
                    "tree_mask launch");
}

size_t tabit_kv_weigh_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                      int num_seqs, int max_q, int max_kv) {
  if (max_kv > kMaxKeys) return 0;
  // (a call without keys may still ask for lse)
  if (!valid_sizes(num_tokens, num_q_heads, num_kv_heads, head_dim, num_seqs, max_q, max_kv == 0 ? 1 : max_kv)) return 0;
  const int dim_pad = (head_dim + 31) / 32 * 32;
  if (!tabit::kv_weigh_fits(num_tokens, num_q_heads, num_kv_heads, dim_pad, num_seqs, max_q, max_kv)) return 0;
  return tabit::kv_weigh_workspace(num_tokens, num_q_heads, num_kv_heads, dim_pad, num_seqs, max_q, max_kv);
}

int tabit_kv_weigh(tabit_ctx* ctx, const tabit_kv_cache* cache, const tabit_kv_attention_args* a, float* sums,
                   void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (a == nullptr) return fail(ctx, TABIT_EINVAL, "null arguments");
  tabit::KvAttnArgs k{};
  int st = check_attention(ctx, cache, a, true, &k);
  if (st != TABIT_OK) return st;
  if (a->out != nullptr) return fail(ctx, TABIT_EINVAL, "weights have no attention output: out must be NULL");
  if (sums == nullptr && k.cache.num_pages > 0) return fail(ctx, TABIT_EINVAL, "null sums");
  if (!aligned(sums, 16)) return fail(ctx, TABIT_EALIGN, "sums must be 16-byte aligned");
  if (a->max_kv > kMaxKeys) return fail(ctx, TABIT_ESHAPE, "max_kv must be in [0, 2^30] (got %d)", a->max_kv);
  if (a->num_tokens == 0 || a->num_seqs == 0 || a->max_q == 0) return TABIT_OK;
  if (a->max_kv == 0 && a->lse == nullptr) return TABIT_OK;
  if ((st = check_grid(ctx, a, 1)) != TABIT_OK) return st;
  if (!tabit::kv_weigh_fits(a->num_tokens, a->num_q_heads, k.cache.heads, k.cache.dim_pad, a->num_seqs, a->max_q,
                            a->max_kv))
    return fail(ctx, TABIT_ESHAPE, "too many rows or keys for one call (%d sequences of %d rows, %d keys)", a->num_seqs,
                a->max_q, a->max_kv);
  const size_t need = tabit::kv_weigh_workspace(a->num_tokens, a->num_q_heads, k.cache.heads, k.cache.dim_pad,
                                                a->num_seqs, a->max_q, a->max_kv);
  if ((st = check_ws(ctx, a->ws, a->ws_bytes, need)) != TABIT_OK) return st;
  k.part = static_cast<float*>(a->ws);
  return hip_status(ctx, tabit::launch_kv_weigh(k, sums, static_cast<hipStream_t>(stream)), "kv_weigh launch");
}

size_t tabit_kv_evict_workspace_bytes(int num_seqs, int num_kv_heads, int max_kv) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || max_kv <= 0) return 0;
  return tabit::kv_evict_workspace(num_seqs, num_kv_heads, max_kv);
}

int tabit_kv_evict(tabit_ctx* ctx, const tabit_kv_cache* cache, const float* sums, const int32_t* block_table,
                   int table_stride, const int32_t* kv_lens, int num_seqs, int max_kv, int budget, int sinks,
                   int recent, int32_t* keep, int32_t* new_lens, void* ws, size_t ws_bytes, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  tabit::KvEvictArgs k{};
  int st = check_cache(ctx, cache, &k.cache);
  if (st != TABIT_OK) return st;
  st = check_table(ctx, block_table, table_stride, num_seqs);
  if (st != TABIT_OK) return st;
  if (max_kv < 0 || max_kv > kMaxKeys) return fail(ctx, TABIT_ESHAPE, "max_kv must be in [0, 2^30] (got %d)", max_kv);
  if ((int64_t)table_stride * cache->page_size < max_kv)
    return fail(ctx, TABIT_ESHAPE, "a table row of %d pages of %d tokens does not hold max_kv = %d", table_stride,
                cache->page_size, max_kv);
  if (budget < 1 || budget > (1 << 30)) return fail(ctx, TABIT_ESHAPE, "budget must be in [1, 2^30] (got %d)", budget);
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return fail(ctx, TABIT_ESHAPE, "the first %d and last %d tokens do not fit a budget of %d", sinks, recent, budget);
  if (kv_lens == nullptr || keep == nullptr || new_lens == nullptr) return fail(ctx, TABIT_EINVAL, "null pointer");
  if (sums == nullptr && k.cache.num_pages > 0) return fail(ctx, TABIT_EINVAL, "null sums");
  if (!aligned(sums, 16) || !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(keep, 4) ||
      !aligned(new_lens, 4) || !aligned(ws, 16))
    return fail(ctx, TABIT_EALIGN, "sums and ws must be 16-byte aligned, the others 4-byte");
  if (num_seqs == 0) return TABIT_OK;
  if ((st = check_ws(ctx, ws, ws_bytes, tabit_kv_evict_workspace_bytes(num_seqs, k.cache.heads, max_kv))) != TABIT_OK)
    return st;
  // (other workgroups still read the lengths, tables and sums when one writes its outputs)
  const uint64_t seqs = (uint64_t)num_seqs, heads = (uint64_t)k.cache.heads;
  const struct { const void* p; uint64_t n; } in[] = {{kv_lens, seqs * 4}, {block_table, seqs * (uint64_t)table_stride * 4},
                                                      {sums, ((uint64_t)k.cache.num_pages * heads << k.cache.page_shift) * 4}},
                                              out[] = {{new_lens, seqs * 4}, {keep, seqs * heads * (uint64_t)budget * 4}};
  bool met = meet(out[0].p, out[0].n, out[1].p, out[1].n);
  for (const auto& o : out)
    for (const auto& i : in) met = met || meet(o.p, o.n, i.p, i.n);
  if (met) return fail(ctx, TABIT_EINVAL, "keep and new_lens may not overlap each other or what the call reads");
  k.ws = static_cast<uint8_t*>(ws);
  k.sums = sums;
  k.table = block_table;
  k.kv_lens = kv_lens;
  k.table_stride = table_stride;
  k.seqs = num_seqs;
  k.max_kv = max_kv;
  k.budget = budget;
  k.sinks = sinks;
  k.recent = recent;
  k.keep = keep;
  k.new_lens = new_lens;
  return hip_status(ctx, tabit::launch_kv_evict(k, static_cast<hipStream_t>(stream)), "kv_evict launch");
}

size_t tabit_kv_compact_workspace_bytes(int num_seqs, int num_kv_heads, int head_dim, int keep_stride) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || head_dim <= 0 || keep_stride <= 0) return 0;
  return tabit::kv_compact_workspace(num_seqs, num_kv_heads, (head_dim + 31) / 32 * 32, keep_stride);
}

int tabit_kv_compact(tabit_ctx* ctx, const tabit_kv_cache* cache, const int32_t* block_table, int table_stride,
                     int num_seqs, const int32_t* keep, int keep_heads, int keep_stride, const int32_t* counts,
                     const int32_t* starts, float* sums, void* ws, size_t ws_bytes, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  tabit::KvCompactArgs k{};
  int st = check_cache(ctx, cache, &k.cache);
  if (st != TABIT_OK) return st;
  st = check_table(ctx, block_table, table_stride, num_seqs);
  if (st != TABIT_OK) return st;
  if (keep_heads != 1 && keep_heads != k.cache.heads)
    return fail(ctx, TABIT_ESHAPE, "keep_heads must be 1 or %d (got %d)", k.cache.heads, keep_heads);
  if (keep_stride < 0 || keep_stride > (1 << 26))
    return fail(ctx, TABIT_ESHAPE, "keep_stride must be in [0, 2^26] (got %d)", keep_stride);
  if (keep == nullptr || counts == nullptr) return fail(ctx, TABIT_EINVAL, "null pointer");
  if (!aligned(sums, 4) || !aligned(block_table, 4) || !aligned(keep, 4) || !aligned(counts, 4) ||
      !aligned(starts, 4) || !aligned(ws, 16))
    return fail(ctx, TABIT_EALIGN, "ws must be 16-byte aligned, the others 4-byte");
  if (num_seqs == 0 || keep_stride == 0 || k.cache.num_pages == 0) return TABIT_OK;
  const size_t need = tabit_kv_compact_workspace_bytes(num_seqs, k.cache.heads, k.cache.head_dim, keep_stride);
  if ((st = check_ws(ctx, ws, ws_bytes, need)) != TABIT_OK) return st;
  k.table = block_table;
  k.table_stride = table_stride;
  k.seqs = num_seqs;
  k.keep = keep;
  k.keep_heads = keep_heads;
  k.keep_stride = keep_stride;
  k.counts = counts;
  k.starts = starts;
  k.sums = sums;
  k.ws = static_cast<uint8_t*>(ws);
  return hip_status(ctx, tabit::launch_kv_compact(k, static_cast<hipStream_t>(stream)), "kv_compact launch");
}

size_t tabit_adapter_workspace_bytes(int rows, int rank, int num_segments) {
  if (rows <= 0 || rank <= 0 || num_segments <= 0) return 0;
  return 2 * align256((size_t)rows * (size_t)rank * 2);
}

int tabit_adapter_linear(tabit_ctx* ctx, const tabit_adapter_args* a, void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (a == nullptr) return fail(ctx, TABIT_EINVAL, "null arguments");
  if (a->x_fmt != TABIT_FMT_BF16 && a->x_fmt != TABIT_FMT_INT8 && a->x_fmt != TABIT_FMT_MXFP4)
    return fail(ctx, TABIT_EINVAL, "unknown x_fmt %d", a->x_fmt);
  if (a->rows < 0 || a->num_segments < 0 || a->num_adapters < 0)
    return fail(ctx, TABIT_ESHAPE, "rows, num_segments and num_adapters must be >= 0");
  if (a->K < 32 || a->K > 32768 || a->K % 32 != 0 || a->N < 32 || a->N > 32768 || a->N % 32 != 0)
    return fail(ctx, TABIT_ESHAPE, "K and N must be multiples of 32 in [32, 32768] (got %d, %d)", a->K, a->N);
  if (a->rank != 16 && a->rank != 32 && a->rank != 64 && a->rank != 128)
    return fail(ctx, TABIT_ESHAPE, "rank must be 16, 32, 64 or 128 (got %d)", a->rank);
  if (a->x == nullptr || a->cu_rows == nullptr || a->adapter == nullptr || a->y == nullptr || a->out == nullptr)
    return fail(ctx, TABIT_EINVAL, "null pointer");
  if (a->num_adapters > 0 && (a->a == nullptr || a->b == nullptr)) return fail(ctx, TABIT_EINVAL, "null adapters");
  if (a->x_fmt != TABIT_FMT_BF16 && a->x_scale == nullptr) return fail(ctx, TABIT_EINVAL, "codes need x_scale");
  if (a->x_fmt == TABIT_FMT_BF16 && (a->x_stride < a->K || a->x_stride % 8 != 0))
    return fail(ctx, TABIT_ESHAPE, "x_stride must be a multiple of 8 of at least K elements");
  if (a->y_stride < a->N || a->y_stride % 8 != 0 || a->out_stride < a->N || a->out_stride % 8 != 0)
    return fail(ctx, TABIT_ESHAPE, "y_stride and out_stride must be multiples of 8 of at least N elements");
  if (a->out == a->y && a->out_stride != a->y_stride)
    return fail(ctx, TABIT_ESHAPE, "out is y: their strides must be alike");
  if (!aligned(a->x, 16) || !aligned(a->a, 16) || !aligned(a->b, 16) || !aligned(a->y, 16) || !aligned(a->out, 16) ||
      !aligned(a->ws, 16) || !aligned(a->scale, 4) || !aligned(a->cu_rows, 4) || !aligned(a->adapter, 4) ||
      (a->x_fmt == TABIT_FMT_INT8 && !aligned(a->x_scale, 4)))
    return fail(ctx, TABIT_EALIGN, "matrices and ws must be 16-byte aligned, vectors 4-byte");
  if (a->rows == 0 || a->num_segments == 0) return TABIT_OK;
  if (!tabit::adapter_fits(a->rows, a->num_segments, a->rank, a->N))
    return fail(ctx, TABIT_ESHAPE, "too many rows and columns (%d, %d)", a->rows, a->N);
  const size_t need = tabit_adapter_workspace_bytes(a->rows, a->rank, a->num_segments);
  const int st = check_ws(ctx, a->ws, a->ws_bytes, need);
  if (st != TABIT_OK) return st;
  // (workgroups of other columns still read a row of x when one writes its part of out)
  const int64_t x_row = a->x_fmt == TABIT_FMT_BF16 ? 2ll * a->K : a->x_fmt == TABIT_FMT_INT8 ? a->K : a->K / 2;
  if (rows_meet(a->out, 2ll * a->N, 2 * a->out_stride, a->x, x_row, a->x_fmt == TABIT_FMT_BF16 ? 2 * a->x_stride : x_row, a->rows))
    return fail(ctx, TABIT_EINVAL, "out may not overlap x");
  if (a->out != a->y && rows_meet(a->out, 2ll * a->N, 2 * a->out_stride, a->y, 2ll * a->N, 2 * a->y_stride, a->rows))
    return fail(ctx, TABIT_EINVAL, "out may be y or not overlap it");
  tabit::AdapterArgs k{};
  k.x = a->x;
  k.x_scale = a->x_scale;
  k.x_fmt = a->x_fmt;
  k.rows = a->rows;
  k.K = a->K;
  k.N = a->N;
  k.x_stride = a->x_stride;
  k.a = a->a;
  k.b = a->b;
  k.scale = a->scale;
  k.num_adapters = a->num_adapters;
  k.rank = a->rank;
  k.cu_rows = a->cu_rows;
  k.adapter = a->adapter;
  k.segments = a->num_segments;
  k.y = a->y;
  k.y_stride = a->y_stride;
  k.out = a->out;
  k.out_stride = a->out_stride;
  k.hi = static_cast<uint16_t*>(a->ws);
  k.lo = k.hi + need / 4;
  return hip_status(ctx, tabit::launch_adapter_linear(k, static_cast<hipStream_t>(stream)), "adapter_linear launch");
}

int tabit_adapter_rotate(tabit_ctx* ctx, const uint16_t* a, int rows, int K, int had_block, uint16_t* out,
                         void* stream) {
  if (ctx == nullptr) return TABIT_EINVAL;
  if (had_block != 32 && had_block != 64 && had_block != 128)
    return fail(ctx, TABIT_ERANGE, "had_block must be 32, 64 or 128 (got %d)", had_block);
  if (rows < 0 || K < 32 || K > 32768 || K % had_block != 0)
    return fail(ctx, TABIT_ESHAPE, "rows must be >= 0, K a multiple of had_block in [32, 32768] (got %d, %d)", rows, K);
  if ((int64_t)rows * K >= (1ll << 34)) return fail(ctx, TABIT_ESHAPE, "too many rows (%d)", rows);
  if (a == nullptr || out == nullptr) return fail(ctx, TABIT_EINVAL, "null pointer");
  if (!aligned(a, 16) || !aligned(out, 16)) return fail(ctx, TABIT_EALIGN, "a and out must be 16-byte aligned");
  if (rows == 0) return TABIT_OK;
  return hip_status(ctx, tabit::launch_adapter_rotate(a, rows, K, had_block, out, static_cast<hipStream_t>(stream)),
                    "adapter_rotate launch");
}

}  // extern "C"
