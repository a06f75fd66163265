// Low-rank adapters of many requests at once beside a shared projection:
//
//   out[t] = y[t] + c_a s_t (x[t] A_a^T) B_a^T,   a the adapter of row t's segment, s_t its
//                                               row scale (INT8 codes), x bf16, INT8 or MXFP4
//
// Two kernels.  The first forms h = c s x A^T for tiles of rows of one segment and 16 to 64
// of the adapter's ranks, its waves sharing the sum over K; h goes out as two bf16 terms (2^-16 of
// itself is lost at most).  The second adds h B^T to y: the product starts from y in the
// accumulator, so out is rounded once.  Both use the 16x16x32 bf16 MFMA with operands loaded from
// memory as they lie: x and A (h and B) are contiguous along the summed axis, and a wave's tile
// of A or B is read by nobody else in its workgroup, so LDS would only delay it.
#include "../../include/tabit.h"
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

// Segment and first row of row tile `tile` (of `rows` rows each, none over two segments), or
// false past the last.  Every lane of a wave takes part.
__device__ __forceinline__ bool find_tile(const AdapterArgs& a, int tile, int rows, int lane, int& seg, int& row0,
                                          int& row1) {
  int before = 0;
  for (int s0 = 0; s0 < a.segments; s0 += 64) {
    const int s = s0 + lane;
    int lo = 0, hi = 0;
    if (s < a.segments) {
      lo = min(max(a.cu_rows[s], 0), a.rows);
      hi = min(max(a.cu_rows[s + 1], lo), a.rows);
    }
    const int mine = (hi - lo + rows - 1) / rows;
    int sum = mine;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int y = __shfl_up(sum, k, 64);
      sum += lane >= k ? y : 0;
    }
    const unsigned long long past = __ballot(before + sum > tile);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      seg = s0 + l;
      const int first = before + __shfl(sum - mine, l, 64);
      row0 = __shfl(lo, l, 64) + (tile - first) * rows;
      row1 = min(row0 + rows, __shfl(hi, l, 64));
      return true;
    }
    before += __shfl(sum, 63, 64);
  }
  return false;
}

__device__ __forceinline__ v8bf zero8() { return __builtin_bit_cast(v8bf, make_uint4(0u, 0u, 0u, 0u)); }

// 16 consecutive elements of a row of x, as two operands.
template <int FMT>
struct Rows;
template <>
struct Rows<TABIT_FMT_BF16> {
  struct Raw { uint4 w[2]; };
  static __device__ __forceinline__ Raw load(const AdapterArgs& a, int t, int k) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + t * a.x_stride + k);
    return {p[0], p[1]};
  }
  static __device__ __forceinline__ void get(const Raw& r, v8bf (&x)[2]) {
    x[0] = __builtin_bit_cast(v8bf, r.w[0]);
    x[1] = __builtin_bit_cast(v8bf, r.w[1]);
  }
};
template <>
struct Rows<TABIT_FMT_INT8> {
  struct Raw { uint4 w; };
  static __device__ __forceinline__ Raw load(const AdapterArgs& a, int t, int k) {
    return {*reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.x) + (long long)t * a.K + k)};
  }
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int at) {
    return pack_bf16((float)(int8_t)(w >> at), (float)(int8_t)(w >> (at + 8)));
  }
  static __device__ __forceinline__ void get(const Raw& r, v8bf (&x)[2]) {
    x[0] = __builtin_bit_cast(v8bf, make_uint4(pair(r.w.x, 0), pair(r.w.x, 16), pair(r.w.y, 0), pair(r.w.y, 16)));
    x[1] = __builtin_bit_cast(v8bf, make_uint4(pair(r.w.z, 0), pair(r.w.z, 16), pair(r.w.w, 0), pair(r.w.w, 16)));
  }
};
template <>
struct Rows<TABIT_FMT_MXFP4> {
  struct Raw { uint2 w; uint32_t scale; };
  static __device__ __forceinline__ Raw load(const AdapterArgs& a, int t, int k) {
    return {*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + ((long long)t * a.K + k) / 2),
            static_cast<const uint8_t*>(a.x_scale)[(long long)t * (a.K / 32) + k / 32]};
  }
  static __device__ __forceinline__ v8bf eight(uint32_t w, uint32_t scale) {
    const float s = __uint_as_float(scale << 23);      // the conversion reads the exponent alone
    uint4 y;
    y.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    y.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    y.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    y.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    if (scale == 255u) y = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    return __builtin_bit_cast(v8bf, y);
  }
  static __device__ __forceinline__ void get(const Raw& r, v8bf (&x)[2]) {
    x[0] = eight(r.w.x, r.scale);
    x[1] = eight(r.w.y, r.scale);
  }
};

// h of 16 MR rows and 16 RB ranks.  A wave takes 64 elements of K at a time, every NW-th: lane l
// holds row l % 16 of x (and rank l % 16 of A), 16 consecutive elements from 16 (l / 16) on, the
// first eight for one product and the others for a second.
template <int FMT, int MR, int RB, int NW>
__global__ void __launch_bounds__(NW * 64)
adapter_down_kernel(AdapterArgs a) {
  constexpr int ROWS = 16 * MR, RANKS = 16 * RB;
  __shared__ float part[NW][ROWS][RANKS + 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int seg, row0, row1;
  const unsigned blocks = (unsigned)a.rank / RANKS;
  if (!find_tile(a, blockIdx.x / blocks, ROWS, lane, seg, row0, row1)) return;
  const int ad = a.adapter[seg];
  if ((unsigned)ad >= (unsigned)a.num_adapters) return;
  const int r0 = blockIdx.x % blocks * RANKS;
  const int row = lane & 15, g = lane >> 4;
  const uint16_t* ap = a.a + ((long long)ad * a.rank + r0 + row) * a.K;
  v4f acc[MR][RB];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r) acc[m][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave * 64; k0 < a.K; k0 += NW * 64) {
    const int k = k0 + 16 * g;
    const bool in = k < a.K;                     // (K is a multiple of 32)
    v8bf x[MR][2], w[RB][2];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[r][e] = in ? *reinterpret_cast<const v8bf*>(ap + (long long)16 * r * a.K + k + 8 * e) : zero8();
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      // (rows past the segment read its last row: their products are not kept)
      const auto raw = Rows<FMT>::load(a, min(row0 + 16 * m + row, row1 - 1), in ? k : 0);
      Rows<FMT>::get(raw, x[m]);
      if (!in) x[m][0] = x[m][1] = zero8();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
          acc[m][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][e], w[r][e], acc[m][r], 0, 0, 0);
  }
  // lane: rank l % 16, rows 4 (l / 16) + i
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][16 * m + 4 * g + i][16 * r + row] = acc[m][r][i];
  __syncthreads();
  const float c = a.scale != nullptr ? a.scale[ad] : 1.0f;
  for (int i = threadIdx.x; i < ROWS * RANKS / 2; i += NW * 64) {
    const int t = i / (RANKS / 2), r = i % (RANKS / 2) * 2;
    if (row0 + t >= row1) continue;
    float u = 0.0f, v = 0.0f;
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      u += part[n][t][r];
      v += part[n][t][r + 1];
    }
    float f = c;
    if (FMT == TABIT_FMT_INT8) f *= static_cast<const float*>(a.x_scale)[row0 + t];
    u *= f;
    v *= f;
    const uint32_t hi = pack_bf16(u, v);
    const long long at = (long long)(row0 + t) * a.rank + r0 + r;
    *reinterpret_cast<uint32_t*>(a.hi + at) = hi;
    // (what rounds to infinity has no second term)
    const float ul = u - bf_lo(hi), vl = v - bf_hi(hi);
    *reinterpret_cast<uint32_t*>(a.lo + at) = pack_bf16(finite_f32(ul) ? ul : 0.0f, finite_f32(vl) ? vl : 0.0f);
  }
}

// out of 16 rows and 64 columns a wave: D[n][t] with B the first operand, so that a lane holds one
// row (l % 16) and, over four products with n = 16 (i / 4) + 4 j + i % 4 for row i of product j, 16
// consecutive columns.  R = 16: one product takes both terms of h, [hi | lo] . [B | B].
// WIDE: the workgroup's waves take 64 rows, 16 each, of the same columns; else 16 rows, and each
// wave columns of its own.
template <int R, bool WIDE>
__global__ void __launch_bounds__(256)
adapter_up_kernel(AdapterArgs a) {
  constexpr int ROWS = WIDE ? 64 : 16, COLS = WIDE ? 64 : 256;
  constexpr int KC = R <= 32 ? 1 : R / 32;             // 32-rank chunks
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int seg, row0, row1;
  const unsigned blocks = ((unsigned)a.N + COLS - 1) / COLS;
  if (!find_tile(a, blockIdx.x / blocks, ROWS, lane, seg, row0, row1)) return;
  const int row = lane & 15, g = lane >> 4;
  const int t = row0 + (WIDE ? wave * 16 : 0) + row;
  const int n0 = (int)(blockIdx.x % blocks) * COLS + (WIDE ? 0 : wave * 64);
  if (n0 >= a.N) return;
  const bool in = n0 + 16 * g < a.N, mine = t < row1 && in;
  const int ad = a.adapter[seg];
  const bool has = (unsigned)ad < (unsigned)a.num_adapters;
  if (!has && a.out == a.y) return;
  uint4 yw[2] = {};
  if (mine) {
    const uint4* p = reinterpret_cast<const uint4*>(a.y + t * a.y_stride + n0 + 16 * g);
    yw[0] = p[0];
    yw[1] = p[1];
  }
  v4f acc[4];
  float y[8];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    unpack8(yw[e], y);
    acc[2 * e] = v4f{y[0], y[1], y[2], y[3]};
    acc[2 * e + 1] = v4f{y[4], y[5], y[6], y[7]};
  }
  if (has) {
    const int th = min(t, row1 - 1);
    v8bf hi[KC], lo[KC];
    if constexpr (R == 16) {
      hi[0] = *reinterpret_cast<const v8bf*>((g < 2 ? a.hi : a.lo) + (long long)th * R + 8 * (g & 1));
    } else {
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        hi[kc] = *reinterpret_cast<const v8bf*>(a.hi + (long long)th * R + 32 * kc + 8 * g);
        lo[kc] = *reinterpret_cast<const v8bf*>(a.lo + (long long)th * R + 32 * kc + 8 * g);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (columns past N read the last ones: their products are not kept)
      const int n = min(n0 + 16 * (row >> 2) + 4 * j + (row & 3), a.N - 1);
      const uint16_t* bp = a.b + ((long long)ad * a.N + n) * R;
      if constexpr (R == 16) {
        const v8bf w = *reinterpret_cast<const v8bf*>(bp + 8 * (g & 1));
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, hi[0], acc[j], 0, 0, 0);
      } else {
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          const v8bf w = *reinterpret_cast<const v8bf*>(bp + 32 * kc + 8 * g);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, lo[kc], acc[j], 0, 0, 0);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, hi[kc], acc[j], 0, 0, 0);
        }
      }
    }
  }
  if (!mine) return;
  uint4* o = reinterpret_cast<uint4*>(a.out + t * a.out_stride + n0 + 16 * g);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    o[e] = make_uint4(pack_bf16(acc[2 * e][0], acc[2 * e][1]), pack_bf16(acc[2 * e][2], acc[2 * e][3]),
                      pack_bf16(acc[2 * e + 1][0], acc[2 * e + 1][1]), pack_bf16(acc[2 * e + 1][2], acc[2 * e + 1][3]));
}

// Each row of A times the block transform over 1 / b.  A wave holds 512 elements, eight a lane.
template <int B>
__global__ void __launch_bounds__(256)
adapter_rotate_kernel(const uint16_t* a, long long n, uint16_t* out) {
  const int lane = threadIdx.x & 63;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
  float v[8] = {};
  if (i < n) load8(a + i, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= 1.0f / B;         // first: b of them may pass fp32
  fwht32_lanes(v, lane);
  if constexpr (B >= 64) fwht_cross8<4>(v, lane);
  if constexpr (B >= 128) fwht_cross8<8>(v, lane);
  if (i < n)
    *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                    pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Row tiles of a launch: every segment ends inside one at most.
unsigned tiles(const AdapterArgs& a, int rows) { return (unsigned)((a.rows + rows - 1) / rows + a.segments); }

// Segments of few rows (single tokens): small tiles, more waves on one sum.
bool few_rows(const AdapterArgs& a) { return a.rows <= 16ll * a.segments; }

template <int FMT>
hipError_t down(const AdapterArgs& a, hipStream_t s) {
  if (few_rows(a)) adapter_down_kernel<FMT, 1, 1, 8><<<tiles(a, 16) * (a.rank / 16), 512, 0, s>>>(a);
  else if (a.rank == 16) adapter_down_kernel<FMT, 2, 1, 4><<<tiles(a, 32), 256, 0, s>>>(a);
  else if (a.rank == 32) adapter_down_kernel<FMT, 2, 2, 4><<<tiles(a, 32), 256, 0, s>>>(a);
  else adapter_down_kernel<FMT, 2, 4, 4><<<tiles(a, 32) * (a.rank / 64), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int R>
hipError_t up(const AdapterArgs& a, hipStream_t s) {
  if (few_rows(a)) adapter_up_kernel<R, false><<<tiles(a, 16) * ((a.N + 255) / 256), 256, 0, s>>>(a);
  else adapter_up_kernel<R, true><<<tiles(a, 64) * ((a.N + 63) / 64), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_linear(const AdapterArgs& a, hipStream_t s) {
  const hipError_t e = a.x_fmt == TABIT_FMT_BF16   ? down<TABIT_FMT_BF16>(a, s)
                       : a.x_fmt == TABIT_FMT_INT8 ? down<TABIT_FMT_INT8>(a, s)
                                                   : down<TABIT_FMT_MXFP4>(a, s);
  if (e != hipSuccess) return e;
  switch (a.rank) {
    case 16: return up<16>(a, s);
    case 32: return up<32>(a, s);
    case 64: return up<64>(a, s);
    case 128: return up<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_adapter_rotate(const uint16_t* a, int rows, int K, int had_block, uint16_t* out,
                                 hipStream_t s) {
  const long long n = (long long)rows * K;
  const unsigned grid = (unsigned)((n / 8 + 255) / 256);
  if (had_block == 32) adapter_rotate_kernel<32><<<grid, 256, 0, s>>>(a, n, out);
  else if (had_block == 64) adapter_rotate_kernel<64><<<grid, 256, 0, s>>>(a, n, out);
  else adapter_rotate_kernel<128><<<grid, 256, 0, s>>>(a, n, out);
  return hipGetLastError();
}

}  // namespace tabit
