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
// or as MXFP4.  What is not finite stays visible: maxima carry NaN, and a row (MXFP4: a
// block) whose largest magnitude is NaN or infinite gets zero codes and a scale of NaN.
//
// A row is held in registers, eight elements a lane and slot, by a wave (or by a
// workgroup for long rows); its sums are DPP butterflies (and one value per wave
// through LDS).  What a sample's rows share -- gate * post weight, (1 + scale) * pre
// weight, shift -- is formed once and kept in registers while a wave walks its rows:
// reading and unpacking five vectors a row cost more vector instructions than the
// norms themselves.  The next row's loads go out before this row's work, since two waves
// a SIMD alone do not keep enough bytes on the way.
//
// Memory bounds it: 4 bytes read and 2 + 2 (INT8 1, MXFP4 0.53) written per element.
// Measured: 17776 x 1920, RMS post and layer pre norm, INT8 after a block of 32: 53 - 56 us
// (76 with the factors read for each row, 60 without the early loads), 4.3 TB/s where a
// large copy reaches 5.2, MXFP4 after a block of 32 55 us (4.0 TB/s); 8192 x 1152 (two samples,
// layer norm, bf16): 17 us, 4.5 TB/s.  At 67 MB of x, INT8 and MXFP4, the widths 512 to 8192 reach
// 4.3 - 5.6 TB/s with modulation or without, 256 reaches 3.0 (half of the lanes are past the row),
// 16384 reaches 3.9 and 32768 1.7, where registers spill.
#include "../../include/tabit.h"
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

// v combined over the 64 lanes, in every lane: inside rows of 16 by DPP (after the
// first two steps a quad agrees, so the mirrored lane stands for the other one), then
// row and half exchanges.
// The larger one, NaN if either is (fmaxf drops it).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <bool MAX>
__device__ __forceinline__ float both(float a, float b) { return MAX ? larger(a, b) : a + b; }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}

template <bool MAX>
__device__ __forceinline__ float wave_all(float v) {
  v = both<MAX>(v, dpp<0xB1>(v));     // quad_perm [1, 0, 3, 2]
  v = both<MAX>(v, dpp<0x4E>(v));     // quad_perm [2, 3, 0, 1]
  v = both<MAX>(v, dpp<0x141>(v));    // row_half_mirror
  v = both<MAX>(v, dpp<0x140>(v));    // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = both<MAX>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return both<MAX>(__uint_as_float(h[0]), __uint_as_float(h[1]));
}

// v combined over the threads of a row.  A row of several waves goes through LDS, one
// slot of `buf` per reduction and parity of the row, so that each needs one barrier.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_all(float v, float (*buf)[16], int slot) {
  v = wave_all<MAX>(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[slot][wave] = v;
    __syncthreads();
    v = buf[slot][0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = both<MAX>(v, buf[slot][w]);
  }
  return v;
}

// Centres v (layer norm) and returns 1 / sqrt(mean square + eps); 1 for no norm.  The
// elements past the row are zero and stay so.
template <int TPR, int S>
__device__ __forceinline__ float statistic(float (&v)[S][8], int kind, float eps, int width, int li,
                                           float (*buf)[16], int slot) {
  if (kind == TABIT_NORM_NONE) return 1.0f;
  const float inv = 1.0f / (float)width;
  const int chunks = width >> 3;
  if (kind == TABIT_NORM_LAYER) {
    float even = 0.0f, odd = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        even += v[i][e];
        odd += v[i][e + 1];
      }
    const float mean = row_all<TPR, false>(even + odd, buf, slot) * inv;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float m = i * TPR + li < chunks ? mean : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] -= m;
    }
  }
  float even = 0.0f, odd = 0.0f;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      even = __builtin_fmaf(v[i][e], v[i][e], even);
      odd = __builtin_fmaf(v[i][e + 1], v[i][e + 1], odd);
    }
  return 1.0f / sqrtf(__builtin_fmaf(row_all<TPR, false>(even + odd, buf, slot + 1), inv, eps));
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}

// INT8 codes of four values: v * r is at most 127 (1 + 2^-24) for the row's largest, so
// adding 1.5 * 2^23 rounds it to the nearest even whole number in the low byte.  r is 0 in a
// row that is not finite: zeros, and NaNs whose low byte is 0 (they are the hardware's or come
// from a bf16, whose lower half is 0).
__device__ __forceinline__ uint32_t i8x4(float a, float b, float c, float d, float r) {
  const uint32_t qa = __float_as_uint(a * r + 12582912.0f), qb = __float_as_uint(b * r + 12582912.0f);
  const uint32_t qc = __float_as_uint(c * r + 12582912.0f), qd = __float_as_uint(d * r + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(qb, qa, 0x0C0C0400u), hi = __builtin_amdgcn_perm(qd, qc, 0x04000C0Cu);
  return lo | hi;
}

// What the rows of a sample share, for the eight elements of chunk ch: gate * post
// weight; (1 + scale) * pre weight and shift.
__device__ __forceinline__ void post_factors(const BlockNormArgs& a, size_t mod, int ch, float (&ga)[8]) {
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) ga[e] = 1.0f;
  if (ch >= a.width >> 3) return;
  if (a.gate != nullptr) load8(a.gate + mod + ch * 8, ga);
  if (a.post_w != nullptr) {
    load8(a.post_w + ch * 8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) ga[e] *= w[e];
  }
}

__device__ __forceinline__ void pre_factors(const BlockNormArgs& a, size_t mod, int ch, float (&gb)[8],
                                            float (&gc)[8]) {
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    gb[e] = 1.0f;
    gc[e] = 0.0f;
  }
  if (ch >= a.width >> 3) return;
  if (a.scale != nullptr) {
    load8(a.scale + mod + ch * 8, gb);
#pragma unroll
    for (int e = 0; e < 8; ++e) gb[e] += 1.0f;
  }
  if (a.pre_w != nullptr) {
    load8(a.pre_w + ch * 8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) gb[e] *= w[e];
  }
  if (a.shift != nullptr) load8(a.shift + mod + ch * 8, gc);
}

template <int TPR, int S>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, TPR > 256 ? 4 : 2)
block_norm_kernel(BlockNormArgs a, int rows_per, int unit0) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  static_assert(TPR == 64 || TPR == NT, "a row is one wave's or one workgroup's");
  __shared__ float buf[TPR > 64 ? 10 : 1][16];
  const int li = TPR == NT ? threadIdx.x : threadIdx.x & 63;
  const int lane = threadIdx.x & 63;
  // this wave's (workgroup's) rows
  const int unit = unit0 + (TPR == NT ? (int)blockIdx.x
                                      : (int)(blockIdx.x * (NT / 64)) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const int row0 = min((long long)unit * rows_per, (long long)a.rows);
  const int row1 = row0 + min(rows_per, a.rows - row0);     // (the sum of the two may pass 2^31)
  const int chunks = a.width >> 3;

  // the longest rows leave no registers for the shared factors or the next row: a
  // workgroup has one row and reads x and the factors at use
  constexpr bool KEEP = TPR <= 256;
  float ga[KEEP ? S : 1][8], gb[KEEP ? S : 1][8], gc[KEEP ? S : 1][8];
  int sample = -1;
  uint4 xn[S], yn[S];   // KEEP: the next row's, on their way while this one is worked on
  auto ask = [&](int row) {
    const size_t at = (size_t)row * a.width;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int ch = i * TPR + li;
      xn[i] = yn[i] = make_uint4(0, 0, 0, 0);
      if (ch < chunks) {
        if (KEEP) xn[i] = *reinterpret_cast<const uint4*>(a.x + at + ch * 8);
        if (a.y != nullptr) yn[i] = *reinterpret_cast<const uint4*>(a.y + at + ch * 8);
      }
    }
  };
  if (row0 < row1) ask(row0);
  for (int row = row0; row < row1; ++row) {
    const size_t at = (size_t)row * a.width;
    const int par = TPR > 64 ? (row & 1) * 5 : 0;
    const size_t mod = (size_t)(row / a.rows_per_sample) * a.mod_stride;
    if (KEEP && row / a.rows_per_sample != sample) {
      sample = row / a.rows_per_sample;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        post_factors(a, mod, i * TPR + li, ga[KEEP ? i : 0]);
        pre_factors(a, mod, i * TPR + li, gb[KEEP ? i : 0], gc[KEEP ? i : 0]);
      }
    }
    uint4 xw[S], yw[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      xw[i] = xn[i];
      yw[i] = yn[i];
    }
    if (KEEP && row + 1 < row1) ask(row + 1);

    float x[S][8];
    if (a.y != nullptr) {
      float t[S][8];
#pragma unroll
      for (int i = 0; i < S; ++i) unpack8(yw[i], t[i]);
      const float r = statistic<TPR, S>(t, a.post_kind, a.eps, a.width, li, buf, par);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (!KEEP && i * TPR + li < chunks)
          xw[i] = *reinterpret_cast<const uint4*>(a.x + at + (i * TPR + li) * 8);
        unpack8(xw[i], x[i]);
        if constexpr (!KEEP) post_factors(a, mod, i * TPR + li, ga[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[i][e] = __builtin_fmaf(t[i][e] * r, ga[KEEP ? i : 0][e], a.res_scale * x[i][e]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (!KEEP && i * TPR + li < chunks)
          xw[i] = *reinterpret_cast<const uint4*>(a.x + at + (i * TPR + li) * 8);
        unpack8(xw[i], x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= a.res_scale;
      }
    }
    if (a.x_out != nullptr) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int ch = i * TPR + li;
        if (ch < chunks) *reinterpret_cast<uint4*>(a.x_out + at + ch * 8) = pack8(x[i]);
      }
    }
    if (a.h == nullptr) continue;

    const float r = statistic<TPR, S>(x, a.pre_kind, a.eps, a.width, li, buf, par + 2);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if constexpr (!KEEP) pre_factors(a, mod, i * TPR + li, gb[0], gc[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[i][e] = __builtin_fmaf(x[i][e] * r, gb[KEEP ? i : 0][e], gc[KEEP ? i : 0][e]);
    }
    if (a.fmt == TABIT_FMT_BF16) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int ch = i * TPR + li;
        if (ch < chunks)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + at + ch * 8) = pack8(x[i]);
      }
      continue;
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
        for (int e = 0; e < 8; ++e) top = larger(top, fabsf(x[i][e]));
      top = row_all<TPR, true>(top, buf, par + 4);
      const bool good = finite_f32(top);
      float q = good && top > 0.0f ? 127.0f / top : 0.0f;
      if (li == 0) static_cast<float*>(a.h_scale)[row] = good ? top / 127.0f : __builtin_nanf("");
      if (q > 0x1p100f) {          // (127 / top would be infinite below 2^-121: both by 2^64, exactly)
        q = 127.0f / (top * 0x1p64f);
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] *= 0x1p64f;
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int ch = i * TPR + li;
        if (ch < chunks)
          *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.h) + at + ch * 8) =
              make_uint2(i8x4(x[i][0], x[i][1], x[i][2], x[i][3], q),
                         i8x4(x[i][4], x[i][5], x[i][6], x[i][7], q));
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {   // MXFP4: a block is four lanes
      const int ch = i * TPR + li;
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; e += 2)   // (as `larger`, which takes 22 registers more here)
        asm("v_maximum3_f32 %0, %0, |%1|, |%2|" : "+v"(top) : "v"(x[i][e]), "v"(x[i][e + 1]));
      top = larger(top, lane_xor<1>(top));
      top = larger(top, lane_xor<2>(top));
      const bool good = finite_f32(top);
      const int X = mx_exponent(top);
      const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X: X is at most 125
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= inv;
      if (ch < chunks) {
        reinterpret_cast<uint32_t*>(a.h)[at / 8 + ch] = good ? e2m1x8(x[i]) : 0u;
        if ((ch & 3) == 0) static_cast<uint8_t*>(a.h_scale)[at / 32 + (ch >> 2)] = (uint8_t)(good ? X + 127 : 255);
      }
    }
  }
}

template <int TPR, int S>
hipError_t launch(const BlockNormArgs& a, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPW = NT / TPR;
  // Rows in runs, one run a wave (workgroup), as many runs as the chip holds at once:
  // then the shared factors are formed once per place.  Three or four times as many
  // took 9 to 19% longer at 17776 x 1920; rows of up to 512 elements, whose factors are
  // few, fill the chip at 8 waves a SIMD and gain 18% over 2.  A row of the longest kind
  // is a run of its own.
  constexpr int kWavesPerSimd = S == 1 ? 8 : S == 2 ? 3 : 2;
  constexpr int kUnits = 256 * 4 * kWavesPerSimd * 64 / TPR;
  const int rows_per = TPR > 256 ? 1 : (a.rows - 1) / kUnits + 1;
  const int units = (a.rows - 1) / rows_per + 1;
  // a launch is limited to 2^32 threads, which rows of the longest kind can pass
  constexpr int kMost = 1 << 21;
  for (int first = 0;; first += kMost) {
    const int n = min(kMost, units - first);
    block_norm_kernel<TPR, S><<<(n + RPW - 1) / RPW, NT, 0, s>>>(a, rows_per, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || units - first <= kMost) return e;
  }
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
  if (chunks <= 2048) return launch<1024, 2>(a, s);
  return launch<1024, 4>(a, s);
}

}  // namespace tabit
