// Masks of trees of drafted tokens from the nodes' parents.
#include "kv_query.h"

namespace tabit {
namespace {

// One workgroup a sequence; a thread follows the parents of its nodes (every 256th), which fall, through LDS.
// Bound by LDS's latency and the sum of a thread's paths, about 53 ns a step: a chain of 64 nodes 4.5 us, of 256
// 15, of 1024 (2556 steps) 136, of 8192 (135000) 7.2 ms; 8192 nodes whose parents are up to eight before them 1.8 ms.
__global__ void __launch_bounds__(256)
tree_mask_kernel(const int* parents, int tokens, const int* cu_q, int max_q, uint64_t* mask, int words, int* depth) {
  __shared__ int up[kMaxNodes];
  const int b = blockIdx.x;
  const int q0 = min(max(cu_q[b], 0), tokens);
  const int n = min(max(min(cu_q[b + 1], tokens) - q0, 0), max_q);
  for (int i = threadIdx.x; i < n; i += 256) {
    const int p = parents[q0 + i];
    up[i] = p >= 0 && p < i ? p : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    uint64_t* row = mask + (long long)(q0 + i) * words;
    int above = -1;
    int at = i;
    for (int w = words - 1; w >= 0; --w) {
      uint64_t bits = 0;
      for (; at >> 6 >= w; at = up[at]) {            // (64 w may pass 32 bits; of no node, -1, it is below)
        bits |= 1ull << (at & 63);
        ++above;
      }
      row[w] = bits;
    }
    if (depth != nullptr) depth[q0 + i] = above;
  }
}

}  // namespace

hipError_t launch_tree_mask(const int* parents, int tokens, const int* cu_q, int seqs, int max_q,
                            uint64_t* mask, int mask_words, int* depth, hipStream_t s) {
  tree_mask_kernel<<<(unsigned)seqs, 256, 0, s>>>(parents, tokens, cu_q, max_q, mask, mask_words, depth);
  return hipGetLastError();
}

}  // namespace tabit
