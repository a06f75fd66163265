// Internal declarations shared by the HIP translation units of libtabit.
// Not part of the public ABI (see include/tabit.h).
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <map>
#include <string>
#include <tuple>
#include <vector>

namespace tabit {

// ---------------------------------------------------------------- quantizers
// Per-row INT8 quantization with an optional block FWHT (activations and
// weights).  scale_div divides the per-row scale a/127 (1 for activations,
// max(b, 1) for weights).
// gate (optional, every launcher below): device byte holding the format the
// caller's schedule selected; a kernel whose format differs returns at once.
hipError_t launch_quant_int8(const uint16_t* x, int M, int K, int had_block, float scale_div,
                             int8_t* q, float* scale, hipStream_t stream,
                             const uint8_t* gate = nullptr);

// Quantizer of the MLP down projection's input with the GELU (tanh form)
// folded in: codes of blockFWHT_b(bf16(gelu(x))).
hipError_t launch_quant_gelu_int8(const uint16_t* x, int M, int K, int had_block, int8_t* q,
                                  float* scale, hipStream_t stream, const uint8_t* gate = nullptr);

// HQ-DM single Hadamard: codes of the rotated row rotated back, Z = 128 hi + lo
// as two int8 planes; scale = (a / 127) / max(b, 1).
hipError_t launch_quant_hqdm(const uint16_t* x, int M, int K, int had_block, int8_t* q_hi,
                             int8_t* q_lo, float* scale, hipStream_t stream,
                             const uint8_t* gate = nullptr);

// MXFP4 quantization (block 32, optional FWHT32).
hipError_t launch_quant_mx(const uint16_t* x, int M, int K, int had_block,
                           uint8_t* q_fp4, uint8_t* e8m0, hipStream_t stream,
                           const uint8_t* gate = nullptr);

// MXFP4 quantization of bf16(gelu(x)) (the MLP's GELU folded in).
hipError_t launch_quant_gelu_mx(const uint16_t* x, int M, int K, int had_block,
                                uint8_t* q_fp4, uint8_t* e8m0, hipStream_t stream,
                                const uint8_t* gate = nullptr);

// ---------------------------------------------------------------- INT8 GEMM
struct GemmConfig {
  int bm, bn, k_groups;   // wave groups splitting one tile's K stages (1 = none)
};
int gemm_config_count();
GemmConfig gemm_config(int index);
int gemm_config_choose(int M, int N, int K, int num_cus);

// ev0 / ev1 (optional): events stamped with this GEMM kernel's start and stop.
hipError_t launch_gemm_i8(int cfg, bool bitserial, const int8_t* xq, const float* sa,
                          const int8_t* wq, const float* sw, int M, int N, int K, int kbits,
                          uint16_t* y, int32_t* acc, hipStream_t stream,
                          hipEvent_t ev0 = nullptr, hipEvent_t ev1 = nullptr,
                          const uint8_t* gate = nullptr);

// ---------------------------------------------------------------- MXFP4 GEMM
int mx_config_count();
GemmConfig mx_config(int index);
int mx_config_choose(int M, int N, int K, int num_cus);

hipError_t launch_gemm_mxfp4(int cfg, const uint8_t* xq, const uint8_t* xe, const uint8_t* wq,
                             const uint8_t* we, int M, int N, int K, float out_scale,
                             uint16_t* y, float* acc, hipStream_t stream,
                             hipEvent_t ev0 = nullptr, hipEvent_t ev1 = nullptr,
                             const uint8_t* gate = nullptr);

// ---------------------------------------------------------------- plane-major storage
// uint32 P[8][ceil(K/128)][N][4]: word P[b][s][n][j] holds bit b of
// W[n][128s + 32j + i] at bit 8*(i % 4) + i / 4; words past K are zero.
size_t planes_bytes(int N, int K);
hipError_t launch_pack_planes(const int8_t* wq, int N, int K, uint32_t* planes, hipStream_t s);
int plane_config_count();
GemmConfig plane_config(int index);
int plane_config_choose(int M, int N, int K, int num_cus);
hipError_t launch_gemm_planes(int cfg, const int8_t* xq, const float* sa, const uint32_t* wp,
                              const float* sw, int M, int N, int K, int kbits, uint16_t* y,
                              int32_t* acc, hipStream_t stream, hipEvent_t ev0 = nullptr,
                              hipEvent_t ev1 = nullptr, const uint8_t* gate = nullptr);

// ---------------------------------------------------------------- HQ-DM single-Hadamard GEMM
int hqdm_config_count();
GemmConfig hqdm_config(int index);
int hqdm_config_choose(int M, int N, int K, int num_cus);
hipError_t launch_gemm_hqdm(int cfg, const int8_t* xh, const int8_t* xl, const float* sa,
                            const int8_t* wq, const float* sw, int M, int N, int K, int kbits,
                            uint16_t* y, long long* acc, hipStream_t stream,
                            hipEvent_t ev0 = nullptr, hipEvent_t ev1 = nullptr);

// ---------------------------------------------------------------- DMPQ selector
// Gamma = sum |out - in| / sum |in| of a block's hidden states in the fixed
// fp64 order; fmt[l] = Gamma > theta[l] ? INT8 : MXFP4.  rows: M x 2 doubles.
size_t dmpq_workspace_bytes(int M);
hipError_t launch_dmpq_select(const uint16_t* xin, const uint16_t* xout, int M, int H, double* rows,
                              const float* theta, int n_layers, uint8_t* fmt, double* gamma,
                              hipStream_t s);

// ---------------------------------------------------------------- paged MXFP4 cache
// Arrays [num_pages][heads][2^page_shift][dim_pad/2 or dim_pad/32]; dim_pad =
// 32 ceil(head_dim / 32); had: rows hold H32 of the padded vectors.
struct KvCacheArgs {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_pages, page_shift, heads, head_dim, dim_pad, had;
};
// Rotation tables [num_positions][rope_dim/2]; rope_dim 0: no rotation.
struct RopeArgs {
  const float *cos, *sin;
  int num_positions, rope_dim, interleaved;
};
hipError_t launch_kv_append(const KvCacheArgs& c, const uint16_t* k, long long k_stride,
                            const uint16_t* v, long long v_stride, int tokens,
                            const int64_t* slots, const RopeArgs& rope, const int* positions,
                            hipStream_t s);
hipError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int tokens, uint16_t* k,
                          uint16_t* v, hipStream_t s);

// Attention of packed query rows over the cache.  `part` holds, when splits > 1,
// splits x tokens x q_heads partial results: dim_pad sums each, then (max, sum).
struct KvAttnArgs {
  KvCacheArgs cache;
  RopeArgs rope;
  const uint16_t* q;
  long long q_stride;
  int tokens, q_heads, group;
  const int* cu_q;
  int seqs, max_q;
  const int* table;
  int table_stride;
  const int* kv_lens;
  int max_kv;
  float scale;
  int causal;
  const int* positions;
  uint16_t* out;
  float* lse;
  float* part;
  int splits;
  const uint64_t* mask;    // trees: [tokens][mask_words]
  int mask_words;
};
// Number of ranges the keys of one sequence are split into for this problem.
int kv_attention_splits(int seqs, int max_q, int q_heads, int kv_heads, int max_kv);
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t s);

// Trees of drafted tokens: the same with a.mask, a.mask_words.
constexpr int kMaxNodes = 8192;  // of a sequence: tree_mask holds their parents in LDS
int kv_tree_splits(int seqs, int max_q, int q_heads, int kv_heads, int max_kv, int dim_pad);
hipError_t launch_kv_tree_attention(const KvAttnArgs& a, hipStream_t s);
hipError_t launch_tree_mask(const int* parents, int tokens, const int* cu_q, int seqs, int max_q,
                            uint64_t* mask, int mask_words, int* depth, hipStream_t s);

// ---------------------------------------------------------------- eviction
// Sums [num_pages][heads][2^page_shift] += the rows' attention weights; a.part is the workspace.
size_t kv_weigh_workspace(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv);
bool kv_weigh_fits(int tokens, int q_heads, int kv_heads, int dim_pad, int seqs, int max_q, int max_kv);
hipError_t launch_kv_weigh(const KvAttnArgs& a, float* sums, hipStream_t s);

struct KvEvictArgs {
  KvCacheArgs cache;
  const float* sums;
  const int *table, *kv_lens;
  int table_stride, seqs, max_kv, budget, sinks, recent;
  int *keep, *new_lens;
  uint8_t* ws;
};
size_t kv_evict_workspace(int seqs, int heads, int max_kv);
hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t s);

struct KvCompactArgs {
  KvCacheArgs cache;
  const int* table;
  int table_stride, seqs;
  const int* keep;
  int keep_heads, keep_stride;
  const int *counts, *starts;    // starts may be null
  float* sums;                   // may be null
  uint8_t* ws;
};
size_t kv_compact_workspace(int seqs, int heads, int dim_pad, int keep_stride);
hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t s);

// ---------------------------------------------------------------- low-rank adapters
struct AdapterArgs {
  const void *x, *x_scale;
  int x_fmt, rows, K, N;
  long long x_stride;
  const uint16_t *a, *b;
  const float* scale;            // may be null
  int num_adapters, rank;
  const int *cu_rows, *adapter;
  int segments;
  const uint16_t* y;
  long long y_stride;
  uint16_t* out;
  long long out_stride;
  uint16_t *hi, *lo;             // workspace: x A^T in two bf16 terms, [rows][rank] each
};
bool adapter_fits(int rows, int segments, int rank, int N);      // the launches' limits
hipError_t launch_adapter_linear(const AdapterArgs& a, hipStream_t s);
hipError_t launch_adapter_rotate(const uint16_t* a, int rows, int K, int had_block, uint16_t* out,
                                 hipStream_t s);

// ---------------------------------------------------------------- block norms
struct BlockNormArgs {
  const uint16_t *x, *y;
  int rows, width;
  int post_kind, pre_kind;              // TABIT_NORM_*
  const uint16_t *post_w, *pre_w;       // [width] or null
  const uint16_t *gate, *scale, *shift; // [samples][mod_stride] or null
  long long mod_stride;
  int rows_per_sample;
  float res_scale, eps;
  uint16_t* x_out;                      // may be null
  void *h, *h_scale;                    // may be null
  int fmt, had;
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s);

// ---------------------------------------------------------------- matrix-core rate probe
// kind 0: INT8 32x32x32 MFMA; kind 1: FP4 32x32x64 scaled MFMA.  sink holds
// mfma_probe_sink_ints(num_cus) ints.  Returns the operations the launch performs.
size_t mfma_probe_sink_ints(int num_cus);
double launch_mfma_probe(int kind, int iters, int num_cus, int* sink, hipStream_t s,
                         hipEvent_t ev0, hipEvent_t ev1, hipError_t* err);

// Compute units of the current device (cached per device id).
int device_num_cus();

}  // namespace tabit

struct tabit_ctx {
  std::string err;
  int steps = 0;
  int layers = 0;
  std::vector<uint8_t> k_bits;
  std::vector<uint8_t> fmt;
  int force_gemm_cfg = -1;
  int force_mx_cfg = -1;
  int force_plane_cfg = -1;
  int force_hqdm_cfg = -1;
  // autotuned tile configuration per (path, M, N, K); path 2 = MXFP4, 3 = plane-major
  std::map<std::tuple<int, int, int, int>, int> tuned;

  int tuned_cfg(int path, int M, int N, int K) const {
    auto it = tuned.find(std::make_tuple(path, M, N, K));
    return it == tuned.end() ? -1 : it->second;
  }
};
