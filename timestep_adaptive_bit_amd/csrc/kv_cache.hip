// Paged MXFP4 key / value cache: append with position rotation, and read back.
//
//   append   k' = R(pos) k on the first rope_dim elements of each head (pairs
//            (i, i + rope_dim/2), or (2i, 2i + 1)): (a c - b s, b c + a s) in
//            fp32; k' and v padded with zeros to blocks of 32, each block
//            transformed by H32 when the cache is rotated (had_block 32), then
//            MXFP4: X = clamp(floor(log2 max|y|) - 2, +-127), E2M1 codes of
//            y 2^-X to nearest even.
//   read     H32 (code 2^X) / 32 (or code 2^X), rounded to bf16 once.
//
// A group of GL lanes holds one (token, head): lane i has elements 8i .. 8i + 7
// of key and value, loaded and stored as whole 16- and 4-byte words; a block of
// 32 is four lanes, so the transform's last two stages and the block maximum are
// DPP moves inside a quad.  Every rotation, butterfly and scaling is one rounded
// fp32 operation in a fixed order, so the stored codes are a function of the
// inputs alone.  The kernel moves each byte once and is bound by memory.
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

constexpr int NT = 256;

// Codes and scale byte of one lane's eight elements of a block (four lanes).
__device__ __forceinline__ void mx_encode(float (&v)[8], uint32_t& codes, uint32_t& scale) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  m = fmaxf(m, lane_xor<1>(m));
  m = fmaxf(m, lane_xor<2>(m));
  const int X = mx_exponent(m);
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X: X is at most 125
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= inv;
  codes = e2m1x8(v);
  scale = (uint32_t)(X + 127);
}

template <int GL>
__global__ void __launch_bounds__(NT)
kv_append_kernel(KvCacheArgs c, const uint16_t* __restrict__ k, long long k_stride,
                 const uint16_t* __restrict__ v, long long v_stride, int tokens,
                 const int64_t* __restrict__ slots, RopeArgs rope,
                 const int* __restrict__ positions) {
  const int lane = threadIdx.x & 63;
  const int gl = threadIdx.x % GL;
  const long long pair = (long long)blockIdx.x * (NT / GL) + threadIdx.x / GL;
  const int t = (int)(pair / c.heads), h = (int)(pair % c.heads);
  if (t >= tokens) return;                       // whole groups leave together
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= (long long)c.num_pages << c.page_shift) return;
  const int e0 = gl * 8;
  const int blocks = c.dim_pad / 32;
  bool bad = false;
  float a[8] = {}, b[8] = {};
  if (e0 < c.head_dim) {
    int pos = 0;
    RopeArgs r = rope;
    if (r.rope_dim > 0) {
      pos = positions[t];
      if (pos < 0 || pos >= r.num_positions) {   // no such table row: stored as not a number
        bad = true;
        r.rope_dim = 0;
      }
    }
    load8_turned(k + t * k_stride + (long long)h * c.head_dim, e0, r, pos, a);
    load8(v + t * v_stride + (long long)h * c.head_dim + e0, b);
  }
  if (c.had) {
    fwht32_lanes(a, lane);
    fwht32_lanes(b, lane);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) bad = bad || !finite_f32(a[e]) || !finite_f32(b[e]);
  // one bad element in the head's key or value marks the whole token
  const unsigned long long group = ((1ull << GL) - 1) << (lane / GL * GL);
  bad = (__ballot(bad) & group) != 0;
  uint32_t kc, ks, vc, vs;
  mx_encode(a, kc, ks);
  mx_encode(b, vc, vs);
  if (bad) {   // a query that sees the token answers NaN, others never touch it
    kc = vc = 0u;
    ks = 255u;
    vs = 127u;
  }
  if (e0 >= c.dim_pad) return;
  const long long page = slot >> c.page_shift;
  const long long row = ((page * c.heads + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
  reinterpret_cast<uint32_t*>(c.k_codes)[row * (c.dim_pad / 8) + gl] = kc;
  reinterpret_cast<uint32_t*>(c.v_codes)[row * (c.dim_pad / 8) + gl] = vc;
  if ((gl & 3) == 0) {
    c.k_scales[row * blocks + (gl >> 2)] = (uint8_t)ks;
    c.v_scales[row * blocks + (gl >> 2)] = (uint8_t)vs;
  }
}

// Eight values of packed codes w with scale byte sb: code 2^(sb - 127); NaN for 255.
__device__ __forceinline__ void mx_decode(uint32_t w, uint32_t sb, float (&v)[8]) {
  const float s = __uint_as_float(sb << 23);     // the conversion reads the exponent field alone
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  v[0] = (float)p0[0]; v[1] = (float)p0[1]; v[2] = (float)p1[0]; v[3] = (float)p1[1];
  v[4] = (float)p2[0]; v[5] = (float)p2[1]; v[6] = (float)p3[0]; v[7] = (float)p3[1];
  if (sb == 255u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(0x7FC00000u);
  }
}

__device__ __forceinline__ void write8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                            pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <int GL>
__global__ void __launch_bounds__(NT)
kv_read_kernel(KvCacheArgs c, const int64_t* __restrict__ slots, int tokens,
               uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  const int lane = threadIdx.x & 63;
  const int gl = threadIdx.x % GL;
  const long long pair = (long long)blockIdx.x * (NT / GL) + threadIdx.x / GL;
  const int t = (int)(pair / c.heads), h = (int)(pair % c.heads);
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  const int e0 = gl * 8;
  float a[8] = {}, b[8] = {};
  if (slot >= 0 && slot < (long long)c.num_pages << c.page_shift && e0 < c.dim_pad) {
    const long long page = slot >> c.page_shift;
    const long long row = ((page * c.heads + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
    const int blocks = c.dim_pad / 32;
    mx_decode(reinterpret_cast<const uint32_t*>(c.k_codes)[row * (c.dim_pad / 8) + gl],
              c.k_scales[row * blocks + (gl >> 2)], a);
    mx_decode(reinterpret_cast<const uint32_t*>(c.v_codes)[row * (c.dim_pad / 8) + gl],
              c.v_scales[row * blocks + (gl >> 2)], b);
  }
  if (c.had) {
    fwht32_lanes(a, lane);
    fwht32_lanes(b, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] *= 0.03125f;
      b[e] *= 0.03125f;
    }
  }
  if (e0 >= c.head_dim) return;
  const long long o = pair * c.head_dim + e0;
  write8(k + o, a);
  write8(v + o, b);
}

}  // namespace

hipError_t launch_kv_append(const KvCacheArgs& c, const uint16_t* k, long long k_stride,
                            const uint16_t* v, long long v_stride, int tokens,
                            const int64_t* slots, const RopeArgs& rope, const int* positions,
                            hipStream_t s) {
  const int gl = c.dim_pad <= 64 ? 8 : 16;
  const long long pairs = (long long)tokens * c.heads;
  const unsigned grid = (unsigned)((pairs + NT / gl - 1) / (NT / gl));
  if (gl == 8)
    kv_append_kernel<8><<<grid, NT, 0, s>>>(c, k, k_stride, v, v_stride, tokens, slots, rope, positions);
  else
    kv_append_kernel<16><<<grid, NT, 0, s>>>(c, k, k_stride, v, v_stride, tokens, slots, rope, positions);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int tokens, uint16_t* k,
                          uint16_t* v, hipStream_t s) {
  const int gl = c.dim_pad <= 64 ? 8 : 16;
  const long long pairs = (long long)tokens * c.heads;
  const unsigned grid = (unsigned)((pairs + NT / gl - 1) / (NT / gl));
  if (gl == 8) kv_read_kernel<8><<<grid, NT, 0, s>>>(c, slots, tokens, k, v);
  else kv_read_kernel<16><<<grid, NT, 0, s>>>(c, slots, tokens, k, v);
  return hipGetLastError();
}

}  // namespace tabit
