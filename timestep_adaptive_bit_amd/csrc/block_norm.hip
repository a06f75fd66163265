// Norms before and after a transformer block with the gate, the residual scale,
// the modulation and the next linear's quantizer in one pass over a token:
//
//   x' = r x + gate * N_post(y)             (x' = r x without y)
//   h  = N_pre(x') (1 + scale) + shift
//
// N is the identity, a layer norm (v - mean) / sqrt(var + eps) or an RMS norm
// v / sqrt(mean v^2 + eps), times a weight if there is one; gate, scale and shift
// are rows of H elements, one per sample of rows_per_sample tokens.  Everything
// between the loads and the stores is fp32: h comes from the unrounded x', which
// is rounded to bf16 for its own output alone.  The variance is the mean square
// of the centred values, in registers, so a large common mean costs no bits.
// h leaves as bf16, as INT8 codes with a per-token scale after a block Walsh-
// Hadamard transform (the codes tabit_hadamard_quant_act defines, of the fp32 h),
// or as MXFP4.
//
// One pass: a row is held in registers, eight elements a lane and slot, by TPR
// threads (a wave, or a workgroup for long rows); its sums are butterflies over
// the lanes (and one value per wave through LDS).  Bound by memory: 4 bytes read
// and 2 + 2 (INT8 1, MXFP4 0.53) written per element.
#include "../../include/tabit.h"
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  return v;
}

// Sum (or maximum) over the TPR threads of a row.  `slot` picks one of the LDS
// rows so that consecutive reductions need one barrier each.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*buf)[16], int slot) {
  v = MAX ? wave_max(v) : wave_sum(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[slot][wave] = v;
    __syncthreads();
    v = buf[slot][0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = MAX ? fmaxf(v, buf[slot][w]) : v + buf[slot][w];
  }
  return v;
}

// v <- N(v) with the row's statistics over `width` elements; elements past the
// row are zero and stay so.
template <int TPR, int S>
__device__ __forceinline__ void normalize(float (&v)[S][8], int kind, const uint16_t* w, float eps,
                                          int width, int li, float (*buf)[16], int slot) {
  if (kind == TABIT_NORM_NONE) return;
  const float inv = 1.0f / (float)width;
  const int chunks = width >> 3;
  if (kind == TABIT_NORM_LAYER) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[i][e];
    const float mean = row_reduce<TPR, false>(sum, buf, slot) * inv;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i * TPR + li < chunks)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] -= mean;
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sq += v[i][e] * v[i][e];
  const float rstd = 1.0f / sqrtf(row_reduce<TPR, false>(sq, buf, slot + 1) * inv + eps);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int ch = i * TPR + li;
    if (w != nullptr && ch < chunks) {
      float g[8];
      load8(w + ch * 8, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rstd * g[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= rstd;
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ uint32_t i8x4(float a, float b, float c, float d, float r) {
  const int qa = (int)__builtin_amdgcn_fmed3f(rintf(a * r), -127.0f, 127.0f);
  const int qb = (int)__builtin_amdgcn_fmed3f(rintf(b * r), -127.0f, 127.0f);
  const int qc = (int)__builtin_amdgcn_fmed3f(rintf(c * r), -127.0f, 127.0f);
  const int qd = (int)__builtin_amdgcn_fmed3f(rintf(d * r), -127.0f, 127.0f);
  return (uint32_t)(qa & 0xFF) | ((uint32_t)(qb & 0xFF) << 8) | ((uint32_t)(qc & 0xFF) << 16) |
         ((uint32_t)qd << 24);
}

template <int TPR, int S>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
block_norm_kernel(BlockNormArgs a) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  static_assert(TPR == 64 || TPR == NT, "a row is one wave's or one workgroup's");
  __shared__ float buf[5][16];
  const int li = TPR == NT ? threadIdx.x : threadIdx.x & 63;
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;               // whole rows leave together
  const int chunks = a.width >> 3;
  const size_t at = (size_t)row * a.width;
  const size_t mod = (size_t)(row / a.rows_per_sample) * a.mod_stride;

  float x[S][8];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int ch = i * TPR + li;
    if (ch < chunks) {
      load8(a.x + at + ch * 8, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    }
  }
  if (a.y != nullptr) {
    float t[S][8];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      if (ch < chunks) {
        load8(a.y + at + ch * 8, t[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] = 0.0f;
      }
    }
    normalize<TPR, S>(t, a.post_kind, a.post_w, a.eps, a.width, li, buf, 0);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      if (a.gate != nullptr && ch < chunks) {
        float g[8];
        load8(a.gate + mod + ch * 8, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = a.res_scale * x[i][e] + g[e] * t[i][e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = a.res_scale * x[i][e] + t[i][e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= a.res_scale;
  }
  if (a.x_out != nullptr) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      if (ch < chunks) *reinterpret_cast<uint4*>(a.x_out + at + ch * 8) = pack8(x[i]);
    }
  }
  if (a.h == nullptr) return;

  normalize<TPR, S>(x, a.pre_kind, a.pre_w, a.eps, a.width, li, buf, 2);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int ch = i * TPR + li;
    if (ch < chunks) {
      float g[8];
      if (a.scale != nullptr) {
        load8(a.scale + mod + ch * 8, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= 1.0f + g[e];
      }
      if (a.shift != nullptr) {
        load8(a.shift + mod + ch * 8, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] += g[e];
      }
    }
  }
  if (a.fmt == TABIT_FMT_BF16) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      if (ch < chunks)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + at + ch * 8) = pack8(x[i]);
    }
    return;
  }
  // blocks of 32, 64 and 128 are 4, 8 and 16 consecutive lanes of one slot
  if (a.had > 0) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      fwht32_lanes(x[i], lane);
      if (a.had >= 64) fwht_cross8<4>(x[i], lane);
      if (a.had >= 128) fwht_cross8<8>(x[i], lane);
    }
  }
  if (a.fmt == TABIT_FMT_INT8) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e]));
    top = row_reduce<TPR, true>(top, buf, 4);
    const float r = top > 0.0f ? 127.0f / top : 0.0f;
    if (li == 0) static_cast<float*>(a.h_scale)[row] = top / 127.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      if (ch < chunks)
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.h) + at + ch * 8) =
            make_uint2(i8x4(x[i][0], x[i][1], x[i][2], x[i][3], r),
                       i8x4(x[i][4], x[i][5], x[i][6], x[i][7], r));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {   // MXFP4: a block is four lanes
    const int ch = i * TPR + li;
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e]));
    top = fmaxf(top, lane_xor<1>(top));
    top = fmaxf(top, lane_xor<2>(top));
    const int X = mx_exponent(top);
    const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X: X is at most 125
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] *= inv;
    if (ch < chunks) {
      reinterpret_cast<uint32_t*>(a.h)[at / 8 + ch] = e2m1x8(x[i]);
      if ((ch & 3) == 0) static_cast<uint8_t*>(a.h_scale)[at / 32 + (ch >> 2)] = (uint8_t)(X + 127);
    }
  }
}

template <int TPR, int S>
hipError_t launch(const BlockNormArgs& a, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPW = NT / TPR;
  block_norm_kernel<TPR, S><<<(a.rows + RPW - 1) / RPW, NT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
  const int chunks = a.width / 8;
  if (chunks <= 64) return launch<64, 1>(a, s);
  if (chunks <= 128) return launch<64, 2>(a, s);
  if (chunks <= 192) return launch<64, 3>(a, s);
  if (chunks <= 256) return launch<64, 4>(a, s);
  if (chunks <= 512) return launch<256, 2>(a, s);
  if (chunks <= 1024) return launch<256, 4>(a, s);
  return launch<1024, 4>(a, s);
}

}  // namespace tabit
