// Device helpers shared by the paged-cache kernels (append, read, attention).
//
// Layout of the cache, per array [num_pages][num_kv_heads][page_size][row]: row
// is Dp/2 bytes of packed E2M1 codes (element 2i in the low nibble) or Dp/32
// E8M0 scale bytes, Dp = 32 ceil(D / 32).  The rows of one page and head are
// contiguous, so 16 tokens of a head are one run of 16 * Dp/2 bytes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "tabit_internal.h"

namespace tabit {
namespace kv {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v32f __attribute__((ext_vector_type(32)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned v6u __attribute__((ext_vector_type(6)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(uint4 a, float (&v)[8]) {
  v[0] = bf_lo(a.x); v[1] = bf_hi(a.x); v[2] = bf_lo(a.y); v[3] = bf_hi(a.y);
  v[4] = bf_lo(a.z); v[5] = bf_hi(a.z); v[6] = bf_lo(a.w); v[7] = bf_hi(a.w);
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}

__device__ __forceinline__ bool finite_f32(float f) {
  return (__float_as_uint(f) & 0x7F800000u) != 0x7F800000u;
}

// fp32 -> bf16 bits of two values, round to nearest even; NaN stays NaN (the
// compiler's conversion, one packed instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const v2bf p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// Value of the lane whose index differs in bit MASK (1, 2: inside a quad by DPP;
// 4, 8, 16: ds_swizzle inside 32 lanes).  With the bound bit set the compiler folds the
// move into the instruction that uses it.
template <int MASK>
__device__ __forceinline__ float lane_xor(float v) {
  int i = __float_as_int(v);
  if constexpr (MASK == 1) i = __builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, true);
  else if constexpr (MASK == 2) i = __builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, true);
  else i = __builtin_amdgcn_ds_swizzle(i, (MASK << 10) | 0x1F);
  return __int_as_float(i);
}

// Butterflies h = 1, 2, 4 of the unnormalized Walsh-Hadamard transform on eight
// consecutive elements of one lane.
__device__ __forceinline__ void fwht8(float (&v)[8]) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; i += 2 * h)
#pragma unroll
      for (int j = i; j < i + h; ++j) {
        const float a = v[j], b = v[j + h];
        v[j] = a + b;
        v[j + h] = a - b;
      }
}

// One cross-lane butterfly: the lane with MASK clear keeps first + second, its
// partner first - second, as partner + (+-own): the sign bit is turned in the lanes
// that subtract, which rounds alike.
template <int MASK>
__device__ __forceinline__ void fwht_cross8(float (&v)[8], int lane) {
  const uint32_t sign = (lane & MASK) ? 0x80000000u : 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = lane_xor<MASK>(v[e]) + __uint_as_float(__float_as_uint(v[e]) ^ sign);
}

// Block-32 transform over four consecutive lanes of eight elements each
// (stages h = 1, 2, 4, then 8 and 16 across lanes).
__device__ __forceinline__ void fwht32_lanes(float (&v)[8], int lane) {
  fwht8(v);
  fwht_cross8<1>(v, lane);
  fwht_cross8<2>(v, lane);
}

// Block-32 transform of 32 elements held by one lane, same stages.
__device__ __forceinline__ void fwht32_lane(float (&v)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int i = 0; i < 32; i += 2 * h)
#pragma unroll
      for (int j = i; j < i + h; ++j) {
        const float a = v[j], b = v[j + h];
        v[j] = a + b;
        v[j + h] = a - b;
      }
}

// Exponent X of the shared MX scale 2^X: floor(log2 top) - 2, in [-127, 127]; 0
// for a zero block.
__device__ __forceinline__ int mx_exponent(float top) {
  const int ex = (int)((__float_as_uint(top) >> 23) & 0xFFu);
  if (top == 0.0f) return 0;
  if (ex == 0) return -127;
  return min(max(ex - 127 - 2, -127), 127);
}

// E2M1 codes of eight values (already divided by the scale), element 2i in the
// low nibble of byte i.  The conversion rounds to nearest even and saturates at
// 6; it keeps the sign of a value that rounds to zero, which is cleared here
// (code 8 becomes 0: adding 7 to a nibble's magnitude carries into its sign bit
// exactly when the magnitude is nonzero).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t x = 0u;
  x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[0], v[1], 1.0f, 0);
  x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[2], v[3], 1.0f, 1);
  x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[4], v[5], 1.0f, 2);
  x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[6], v[7], 1.0f, 3);
  const uint32_t mag = x & 0x77777777u;
  return mag | (x & ((mag + 0x77777777u) & 0x88888888u));
}

// The two rotated elements of one pair: (a c - b s, b c + a s), each product and
// sum rounded to fp32 on its own.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a * c - b * s, y = b * c + a * s;
  a = x;
  b = y;
}

// Elements [e0, e0 + 8) of a head vector, rotated to position row `pos` of the tables.
// rope_dim is a multiple of 16, so in either pairing the eight lie on one side of the
// rotated region and their partners are the eight consecutive elements from
// turn_partner(e0) on (the same eight where pairs are neighbours).
__device__ __forceinline__ int turn_partner(int e0, const RopeArgs& rope) {
  const int half = rope.rope_dim >> 1;
  if (rope.interleaved || e0 >= rope.rope_dim) return e0;
  return e0 >= half ? e0 - half : e0 + half;
}

__device__ __forceinline__ void turned8(uint4 own, uint4 partner, int e0, const RopeArgs& rope, int pos,
                                        float (&v)[8]) {
  unpack8(own, v);
  if (e0 >= rope.rope_dim) return;
  const int half = rope.rope_dim >> 1;
  const size_t row = (size_t)pos * half;
  if (rope.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(rope.cos + row + (e0 >> 1));
    const float4 s = *reinterpret_cast<const float4*>(rope.sin + row + (e0 >> 1));
    turn(v[0], v[1], c.x, s.x);
    turn(v[2], v[3], c.y, s.y);
    turn(v[4], v[5], c.z, s.z);
    turn(v[6], v[7], c.w, s.w);
    return;
  }
  const bool second = e0 >= half;
  const int i0 = second ? e0 - half : e0;
  const float4 c0 = *reinterpret_cast<const float4*>(rope.cos + row + i0);
  const float4 c1 = *reinterpret_cast<const float4*>(rope.cos + row + i0 + 4);
  const float4 s0 = *reinterpret_cast<const float4*>(rope.sin + row + i0);
  const float4 s1 = *reinterpret_cast<const float4*>(rope.sin + row + i0 + 4);
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  // the first of a pair takes -o s: the partner's sign bits are turned
  const uint32_t sign = second ? 0u : 0x80008000u;
  float o[8];
  unpack8(make_uint4(partner.x ^ sign, partner.y ^ sign, partner.z ^ sign, partner.w ^ sign), o);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * c[e] + o[e] * s[e];
}

}  // namespace kv
}  // namespace tabit
