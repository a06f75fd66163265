// Low-rank adapters of many requests at once beside a shared projection:
//
//   out[t] = y[t] + c_a s_t (x[t] A_a^T) B_a^T,   a the adapter of row t's segment, s_t its
//                                               row scale (INT8 codes), x bf16, INT8 or MXFP4
//
// Two kernels.  The first forms h = c s x A^T for tiles of rows of one segment and 16 to 64 of the adapter's
// ranks, its waves sharing the sum over K; h goes out as two bf16 terms (2^-16 of itself is lost at most).
// The second adds h B^T to y: the product starts from y in the accumulator, so out is rounded once.  Few rows
// at low ranks have one kernel of both parts, with the same bits.  All use the 16x16x32 bf16 MFMA.  x, A and B
// come through LDS, straight from memory by whole lines: loaded as the operands' lanes hold them, 16 rows in
// turn, each lane's 16 bytes were a cache access of their own (60 an instruction; 17776 rows of 1920 to 5760
// by rank 32 took 121 us for the second kernel then, its address units busy throughout).
#include "../../include/tabit.h"
#include "kv_common.h"
#include "tile_common.h"

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

typedef int v2i __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v8bf zero8() { return __builtin_bit_cast(v8bf, make_uint4(0u, 0u, 0u, 0u)); }

typedef const __attribute__((address_space(1))) void* from_t;
typedef __attribute__((address_space(3))) void* to_t;

// Rows of PIECES 16-byte pieces in LDS: piece p of row i lies at place p ^ turned(i) of its row, so that
// the 16 rows that 16 lanes read at once cover the banks' 256 bytes.
template <int PIECES>
__device__ __forceinline__ int turned(int i) {
  return PIECES >= 16 ? i & 15 : (i / (16 / PIECES)) & (PIECES - 1);
}
template <int PIECES>
__device__ __forceinline__ int place(int i, int p) { return (i * PIECES + (p ^ turned<PIECES>(i))) * 16; }

// 64 elements of a row of x: PIECES of 16 bytes; get gives 16 consecutive ones, from 16 g on, as two
// operands.
template <int FMT>
struct Rows;
template <>
struct Rows<TABIT_FMT_BF16> {
  static constexpr int PIECES = 8;
  static __device__ __forceinline__ const void* at(const AdapterArgs& a, int t, int k) {
    return static_cast<const uint16_t*>(a.x) + t * a.x_stride + k;
  }
  static __device__ __forceinline__ void get(const uint8_t* lds, int i, int g, uint32_t, v8bf (&x)[2]) {
    x[0] = *reinterpret_cast<const v8bf*>(lds + place<8>(i, 2 * g));
    x[1] = *reinterpret_cast<const v8bf*>(lds + place<8>(i, 2 * g + 1));
  }
};
template <>
struct Rows<TABIT_FMT_INT8> {
  static constexpr int PIECES = 4;
  static __device__ __forceinline__ const void* at(const AdapterArgs& a, int t, int k) {
    return static_cast<const int8_t*>(a.x) + (long long)t * a.K + k;
  }
  static __device__ __forceinline__ uint32_t pair(int w, int at) {
    return pack_bf16((float)(int8_t)(w >> at), (float)(int8_t)(w >> (at + 8)));
  }
  static __device__ __forceinline__ void get(const uint8_t* lds, int i, int g, uint32_t, v8bf (&x)[2]) {
    // (a vector type, as v8bf: a HIP struct loses the access's alias information, and the compiler then has it
    // wait for every copy that is on its way to LDS, the next step's, too)
    const v4i w = *reinterpret_cast<const v4i*>(lds + place<4>(i, g));
    x[0] = __builtin_bit_cast(v8bf, make_uint4(pair(w[0], 0), pair(w[0], 16), pair(w[1], 0), pair(w[1], 16)));
    x[1] = __builtin_bit_cast(v8bf, make_uint4(pair(w[2], 0), pair(w[2], 16), pair(w[3], 0), pair(w[3], 16)));
  }
};
template <>
struct Rows<TABIT_FMT_MXFP4> {
  static constexpr int PIECES = 2;
  static __device__ __forceinline__ const void* at(const AdapterArgs& a, int t, int k) {
    return static_cast<const uint8_t*>(a.x) + ((long long)t * a.K + k) / 2;
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
  static __device__ __forceinline__ void get(const uint8_t* lds, int i, int g, uint32_t scale, v8bf (&x)[2]) {
    const v2i w = *reinterpret_cast<const v2i*>(lds + place<2>(i, g >> 1) + 8 * (g & 1));
    x[0] = eight((uint32_t)w[0], scale);
    x[1] = eight((uint32_t)w[1], scale);
  }
};

// h of 16 MR rows and 16 RB ranks.  A wave takes 64 elements of K at a time, every NW-th, through LDS of its
// own, a step ahead: lane l holds row l % 16 of x (and rank l % 16 of A), 16 consecutive elements from
// 16 (l / 16) on, the first eight for one product and the others for a second.
template <int FMT, int MR, int RB>
struct Down {
  static constexpr int ROWS = 16 * MR, RANKS = 16 * RB, STAGES = 2;
  static constexpr int XB = ROWS * Rows<FMT>::PIECES * 16, WB = RANKS * 128;        // bytes of a step
  static constexpr int PART = ROWS * (RANKS + 4) * 4;
  static constexpr int PER_WAVE = STAGES * (XB + WB) > PART ? STAGES * (XB + WB) : PART;
};
// Adapter ad's ranks from r0 on of rows row0 .. row1 - 1 (16 MR at most); put(row of the tile, rank, high terms
// of two ranks, low terms).  LATE: the next step is asked for when this one has been read, not before it is waited
// for.  A third step on its way is level in either order.  4 rows of 2240, rank 16, 4.6 us late and 4.8 first, one of
// 12288 in INT8 9.3 and 11.0 (one kernel for both products); 32 rows of 12288, rank 64, 17.7 and 14.3, 17776 of
// 1920 in bf16, rank 32, 101 and 98 (two kernels).
template <int FMT, int MR, int RB, int NW, bool LATE, typename Put>
__device__ __forceinline__ void form_h(const AdapterArgs& a, uint8_t (*smem)[Down<FMT, MR, RB>::PER_WAVE], int ad, int row0,
                                       int row1, int r0, Put put) {
  using X = Rows<FMT>;
  using D = Down<FMT, MR, RB>;
  constexpr int ROWS = D::ROWS, RANKS = D::RANKS, STAGES = D::STAGES, XB = D::XB, WB = D::WB;
  constexpr int XI = (XB + 1023) / 1024, WI = WB / 1024;             // instructions of a step
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, g = lane >> 4;
  // (asked for here, waited for at the end)
  const float c = a.scale != nullptr ? a.scale[ad] : 1.0f;
  constexpr int PAIRS = RANKS / 2, MINE = (ROWS * PAIRS + NW * 64 - 1) / (NW * 64);
  float f[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    f[i] = 1.0f;
    if (FMT == TABIT_FMT_INT8)
      f[i] = static_cast<const float*>(a.x_scale)[min(row0 + (i * NW * 64 + (int)threadIdx.x) / PAIRS, row1 - 1)];
  }
  const uint16_t* ap = a.a + ((long long)ad * a.rank + r0) * a.K;
  v4f acc[MR][RB];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r) acc[m][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t scale[STAGES][MR];
  // Rows past the segment read its last one, pieces past K (a multiple of 32) the row's first: neither is
  // kept.
  auto ask = [&](int step) {
    const int k0 = (step * NW + wave) * 64;
    if (k0 >= a.K) return;
    uint8_t* to = smem[wave] + step % STAGES * (XB + WB);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int s = i * 64 + lane, r = s / X::PIECES, p = (s % X::PIECES) ^ turned<X::PIECES>(r);
      const int k = k0 + p * (64 / X::PIECES);
      if (XB >= 1024 || s < XB / 16)
        __builtin_amdgcn_global_load_lds((from_t)X::at(a, min(row0 + r, row1 - 1), k < a.K ? k : 0), (to_t)(to + i * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int s = i * 64 + lane, r = s / 8, k = k0 + ((s % 8) ^ turned<8>(r)) * 8;
      __builtin_amdgcn_global_load_lds((from_t)(ap + (long long)r * a.K + (k < a.K ? k : 0)), (to_t)(to + XB + i * 1024), 16, 0, 0);
    }
    if constexpr (FMT == TABIT_FMT_MXFP4) {
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        const int k = k0 + 16 * g;
        scale[step % STAGES][m] = static_cast<const uint8_t*>(
            a.x_scale)[(long long)min(row0 + 16 * m + row, row1 - 1) * (a.K / 32) + (k < a.K ? k : 0) / 32];
      }
    }
  };
  ask(0);
  for (int step = 0;; ++step) {
    const int k0 = (step * NW + wave) * 64;
    if (k0 >= a.K) break;
    if (!LATE) ask(step + 1);
    if (!LATE && k0 + NW * 64 < a.K) tile::wait_vmcnt<XI + WI>();     // this step's are here, the next one's not
    else tile::wait_vmcnt0();
    __builtin_amdgcn_wave_barrier();
    const uint8_t* st = smem[wave] + step % STAGES * (XB + WB);
    v8bf x[MR][2], w[RB][2];
#pragma unroll
    for (int m = 0; m < MR; ++m) X::get(st, 16 * m + row, g, FMT == TABIT_FMT_MXFP4 ? scale[step % STAGES][m] : 0u, x[m]);
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) w[r][e] = *reinterpret_cast<const v8bf*>(st + XB + place<8>(16 * r + row, 2 * g + e));
    if (LATE) {
      __builtin_amdgcn_wave_barrier();
      ask(step + 1);
    }
    if (k0 + 64 > a.K && k0 + 16 * g >= a.K) {
#pragma unroll
      for (int m = 0; m < MR; ++m) x[m][0] = x[m][1] = zero8();
#pragma unroll
      for (int r = 0; r < RB; ++r) w[r][0] = w[r][1] = zero8();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
          acc[m][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][e], w[r][e], acc[m][r], 0, 0, 0);
    __builtin_amdgcn_wave_barrier();             // (LDS serves a wave in order: its reads are before what comes)
  }
  // lane: rank l % 16, rows 4 (l / 16) + i
  float* part = reinterpret_cast<float*>(smem[wave]);
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[(16 * m + 4 * g + i) * (RANKS + 4) + 16 * r + row] = acc[m][r][i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int t = (i * NW * 64 + (int)threadIdx.x) / PAIRS, r = (i * NW * 64 + (int)threadIdx.x) % PAIRS * 2;
    if (t >= ROWS || row0 + t >= row1) continue;
    float u = 0.0f, v = 0.0f;
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      const float2 x = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(smem[n]) + t * (RANKS + 4) + r);
      u += x.x;
      v += x.y;
    }
    u *= c * f[i];
    v *= c * f[i];
    const uint32_t hi = pack_bf16(u, v);
    // (what rounds to infinity has no second term)
    const float ul = u - bf_lo(hi), vl = v - bf_hi(hi);
    put(t, r, hi, pack_bf16(finite_f32(ul) ? ul : 0.0f, finite_f32(vl) ? vl : 0.0f));
  }
}

template <int FMT, int MR, int RB, int NW>
__global__ void __launch_bounds__(NW * 64)
adapter_down_kernel(AdapterArgs a) {
  using D = Down<FMT, MR, RB>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW][D::PER_WAVE];
  int seg, row0, row1;
  const unsigned blocks = (unsigned)a.rank / D::RANKS;
  if (!find_tile(a, blockIdx.x / blocks, D::ROWS, threadIdx.x & 63, seg, row0, row1)) return;
  const int ad = a.adapter[seg];
  if ((unsigned)ad >= (unsigned)a.num_adapters) return;
  const int r0 = blockIdx.x % blocks * D::RANKS;
  form_h<FMT, MR, RB, NW, false>(a, smem, ad, row0, row1, r0, [&](int t, int r, uint32_t hi, uint32_t lo) {
    const long long at = (long long)(row0 + t) * a.rank + r0 + r;
    *reinterpret_cast<uint32_t*>(a.hi + at) = hi;
    *reinterpret_cast<uint32_t*>(a.lo + at) = lo;
  });
}

// Columns n0 + 8 i + j of B as row 16 j + i of 128 in LDS (those past N read the last one and are not kept), every
// EACH-th instruction of them from `from` on.
template <int R, int EACH>
__device__ __forceinline__ void bring_b(const AdapterArgs& a, const uint16_t* bp, int n0, uint8_t* to, int from, int lane) {
  constexpr int PIECES = R / 8;
#pragma unroll
  for (int i = from; i < 128 * R * 2 / 1024; i += EACH) {
    const int s = i * 64 + lane, q = s / PIECES, p = (s % PIECES) ^ turned<PIECES>(q & 15);
    const int n = min(n0 + 8 * (q & 15) + (q >> 4), a.N - 1);
    __builtin_amdgcn_global_load_lds((from_t)(bp + (long long)n * R + p * 8), (to_t)(to + i * 1024), 16, 0, 0);
  }
}

// acc (rows 4 (l / 16) + r, columns 8 (l % 16) + j) + h . B of those columns
template <int R, int KC>
__device__ __forceinline__ void add_up(const uint8_t* stage, const v8bf (&hi)[KC], const v8bf (&lo)[KC], int row, int g, v4f (&acc)[8]) {
  constexpr int PIECES = R / 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint8_t* b = stage + j * 16 * R * 2;
    if constexpr (R == 16) {
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[0], *reinterpret_cast<const v8bf*>(b + place<PIECES>(row, g & 1)), acc[j], 0, 0, 0);
    } else {
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        const v8bf w = *reinterpret_cast<const v8bf*>(b + place<PIECES>(row, 4 * kc + g));
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[kc], w, acc[j], 0, 0, 0);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[kc], w, acc[j], 0, 0, 0);
      }
    }
  }
}

__device__ __forceinline__ void start_from(const uint4 (&y)[4], v4f (&acc)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float v[8];
    unpack8(y[r], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j][r] = v[j];
  }
}

__device__ __forceinline__ uint4 row_of(const v4f (&acc)[8], int r) {
  return make_uint4(pack_bf16(acc[0][r], acc[1][r]), pack_bf16(acc[2][r], acc[3][r]),
                    pack_bf16(acc[4][r], acc[5][r]), pack_bf16(acc[6][r], acc[7][r]));
}

// out of 16 rows a wave, 128 columns at a time: h is the first operand and product j takes columns
// 8 i + j (i = l % 16), so that a lane holds eight consecutive columns of four rows, and 16 lanes read and
// write 256 bytes of a row at once.  R = 16: one product takes both terms of h, [hi | lo] . [B | B].
// WIDE: the workgroup's waves take 64 rows, 16 each, of the same columns, which they bring to LDS together;
// else 16 rows, and each wave columns of its own.
template <int R, bool WIDE>
__global__ void __launch_bounds__(256)
adapter_up_kernel(AdapterArgs a, int cols) {
  constexpr int ROWS = WIDE ? 64 : 16, COLS = 128;
  constexpr int KC = R <= 32 ? 1 : R / 32;             // 32-rank chunks
  constexpr int BYTES = COLS * R * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WIDE ? 2 : 4][BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int seg, row0, row1;
  const unsigned blocks = ((unsigned)a.N + cols - 1) / cols;
  if (!find_tile(a, blockIdx.x / blocks, ROWS, lane, seg, row0, row1)) return;
  const int row = lane & 15, g = lane >> 4;
  const int ad = a.adapter[seg];
  const bool has = (unsigned)ad < (unsigned)a.num_adapters;
  if (!has && a.out == a.y) return;
  const int t0 = row0 + (WIDE ? wave * 16 : 0);
  constexpr int STRIDE = WIDE ? COLS : 4 * COLS;
  const int first = (int)(blockIdx.x % blocks) * cols + (WIDE ? 0 : wave * COLS);
  const int last = min((int)(blockIdx.x % blocks + 1) * cols, a.N);
  const uint16_t* bp = a.b + (long long)(has ? ad : 0) * a.N * R;
  auto bring = [&](int n0, uint8_t* to) {
    if (has && n0 < last) bring_b<R, WIDE ? 4 : 1>(a, bp, n0, to, WIDE ? wave : 0, lane);
  };
  uint8_t* stage = smem[WIDE ? 0 : wave];
  bring(first, stage);
  v8bf hi[KC], lo[KC];
  if (has) {
    const int th = min(t0 + row, row1 - 1);
    if constexpr (R == 16) {
      hi[0] = *reinterpret_cast<const v8bf*>((g < 2 ? a.hi : a.lo) + (long long)th * R + 8 * (g & 1));
    } else {
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        hi[kc] = *reinterpret_cast<const v8bf*>(a.hi + (long long)th * R + 32 * kc + 8 * g);
        lo[kc] = *reinterpret_cast<const v8bf*>(a.lo + (long long)th * R + 32 * kc + 8 * g);
      }
    }
  }
  int at = 0;
  for (int n0 = first; n0 < last; n0 += STRIDE) {
    // lane: rows t0 + 4 g + r, columns n0 + 8 (l % 16) on
    const int n = n0 + 8 * row;
    uint4 y[4] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n < a.N && t0 + 4 * g + r < row1) y[r] = *reinterpret_cast<const uint4*>(a.y + (t0 + 4 * g + r) * a.y_stride + n);
    tile::wait_vmcnt0();
    if constexpr (WIDE) {
      tile::lds_barrier();
      bring(n0 + STRIDE, smem[at ^ 1]);
      stage = smem[at];
      at ^= 1;
    } else {
      __builtin_amdgcn_wave_barrier();
    }
    v4f acc[8];
    start_from(y, acc);
    if (has) add_up<R, KC>(stage, hi, lo, row, g, acc);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n < a.N && t0 + 4 * g + r < row1)
        *reinterpret_cast<uint4*>(a.out + (t0 + 4 * g + r) * a.out_stride + n) = row_of(acc, r);
    if constexpr (!WIDE) {
      __builtin_amdgcn_wave_barrier();
      bring(n0 + STRIDE, stage);
    }
  }
}

// Both at once, for few rows and low ranks: every workgroup (16 rows, 1024 columns, 128 a wave) forms h for itself.
template <int FMT, int R>
__global__ void __launch_bounds__(512)
adapter_few_kernel(AdapterArgs a) {
  using D = Down<FMT, 1, R / 16>;
  constexpr int NW = 8, COLS = 128, KC = 1, BYTES = COLS * R * 2;
  static_assert(R <= 32, "one operand of h");
  // (one array: with two, the compiler tells their copies apart and has reads of one wait for all of its copies)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NW * (BYTES + D::PER_WAVE)];
  auto stage = reinterpret_cast<uint8_t (*)[BYTES]>(lds);
  auto smem = reinterpret_cast<uint8_t (*)[D::PER_WAVE]>(lds + NW * BYTES);
  auto h = reinterpret_cast<uint16_t (*)[16][R]>(smem[0]);         // [2][16][R]: both terms, when x and A are done with
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, g = lane >> 4;
  int seg, row0, row1;
  const unsigned blocks = ((unsigned)a.N + NW * COLS - 1) / (NW * COLS);
  if (!find_tile(a, blockIdx.x / blocks, 16, lane, seg, row0, row1)) return;
  const int ad = a.adapter[seg];
  const bool has = (unsigned)ad < (unsigned)a.num_adapters;
  if (!has && a.out == a.y) return;
  const int n0 = (int)(blockIdx.x % blocks) * NW * COLS + wave * COLS, n = n0 + 8 * row;
  uint4 y[4] = {};
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n < a.N && row0 + 4 * g + r < row1) y[r] = *reinterpret_cast<const uint4*>(a.y + (row0 + 4 * g + r) * a.y_stride + n);
  v4f acc[8];
  if (has) {
    if (n0 < a.N) bring_b<R, 1>(a, a.b + (long long)ad * a.N * R, n0, stage[wave], 0, lane);
    static_assert(16 * R / 2 <= NW * 64, "at most two ranks a thread");
    int t = -1, r = 0;
    uint32_t high = 0u, low = 0u;
    form_h<FMT, 1, R / 16, NW, true>(a, smem, ad, row0, row1, 0, [&](int t_, int r_, uint32_t hi, uint32_t lo) {
      t = t_;
      r = r_;
      high = hi;
      low = lo;
    });
    __syncthreads();
    if (t >= 0) {
      *reinterpret_cast<uint32_t*>(&h[0][t][r]) = high;
      *reinterpret_cast<uint32_t*>(&h[1][t][r]) = low;
    }
    tile::wait_vmcnt0();
    __syncthreads();
    // (rows past the segment have no h, and no place)
    const v8bf hi[1] = {R == 16 ? *reinterpret_cast<const v8bf*>(&h[g >> 1][row][8 * (g & 1)]) : *reinterpret_cast<const v8bf*>(&h[0][row][8 * g])};
    const v8bf lo[1] = {*reinterpret_cast<const v8bf*>(&h[1][row][R == 16 ? 0 : 8 * g])};
    start_from(y, acc);
    add_up<R, KC>(stage[wave], hi, lo, row, g, acc);
  } else {
    start_from(y, acc);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n < a.N && row0 + 4 * g + r < row1)
      *reinterpret_cast<uint4*>(a.out + (row0 + 4 * g + r) * a.out_stride + n) = row_of(acc, r);
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
long long tiles_of(int rows, int segments, int tile) { return ((long long)rows + tile - 1) / tile + segments; }
unsigned tiles(const AdapterArgs& a, int tile) { return (unsigned)tiles_of(a.rows, a.segments, tile); }

// Segments of few rows (single tokens): small tiles, more waves on one sum.
bool few_rows(int rows, int segments) { return rows <= 16ll * segments; }
bool few_rows(const AdapterArgs& a) { return few_rows(a.rows, a.segments); }
// One kernel for both, where reading A again for every 1024 columns costs less than a launch: up to 32 MB in all.
// Measured under a graph, two kernels and one: 4 rows of 2240 to 2240, rank 16 (0.9 MB) 7.0 and 4.6 us; 32 rows
// of 4096 to 6144, ranks 16 (26 MB) and 32 (53 MB) 8.9 and 6.8, 9.2 and 12.5; 64 of 2240 to 2240, rank 32 (28 MB)
// 8.5 and 7.4; 256 of 1152 to 1152, ranks 16 (20 MB) and 32 (40 MB) 10.1 and 7.4, 11.9 and 15.0.
bool at_once(const AdapterArgs& a) {
  return few_rows(a) && a.rank <= 32 &&
         (long long)tiles(a, 16) * ((a.N + 1023) / 1024) * a.rank * a.K * 2 <= (1ll << 25);
}

// Measured, 64 rows of 4096 in INT8, rank 64, 40 adapters: 4, 8 and 16 waves 12.5, 9.1 and 8.6 us, one row of
// 2240 in each of four segments 4.5, 3.8 and 4.2 (8 waves are 8.1 us now for the first).  17776 rows of 1920, rank
// 32: 16, 32 and 64 rows by four waves 25, 19.5 and 19.6 (17.5 now), 32 by eight 24.5; a third stage 25.5 (13 us
// where the rows come from a cache; 2.6 TB/s, A from the L2 as often as x from memory).
template <int FMT>
hipError_t down(const AdapterArgs& a, hipStream_t s) {
  if (few_rows(a)) adapter_down_kernel<FMT, 1, 1, 8><<<tiles(a, 16) * (a.rank / 16), 512, 0, s>>>(a);
  else if (a.rank == 16) adapter_down_kernel<FMT, 2, 1, 4><<<tiles(a, 32), 256, 0, s>>>(a);
  else if (a.rank == 32) adapter_down_kernel<FMT, 2, 2, 4><<<tiles(a, 32), 256, 0, s>>>(a);
  else adapter_down_kernel<FMT, 2, 4, 4><<<tiles(a, 32) * (a.rank / 64), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t few(const AdapterArgs& a, hipStream_t s) {
  const unsigned grid = tiles(a, 16) * ((a.N + 1023) / 1024);
  if (a.rank == 16) adapter_few_kernel<FMT, 16><<<grid, 512, 0, s>>>(a);
  else adapter_few_kernel<FMT, 32><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}

// Columns of a workgroup: 512 (128 a wave) of single tokens, 256 of many rows (17776 rows to 5760, rank 32, in
// 128, 256, 512 and 1024: both kernels 92, 92, 100 and 103 us; 74 of it this one, 5.5 TB/s).
template <int R>
hipError_t up(const AdapterArgs& a, hipStream_t s) {
  if (few_rows(a)) adapter_up_kernel<R, false><<<tiles(a, 16) * ((a.N + 511) / 512), 256, 0, s>>>(a, 512);
  else adapter_up_kernel<R, true><<<tiles(a, 64) * ((a.N + 255) / 256), 256, 0, s>>>(a, 256);
  return hipGetLastError();
}

}  // namespace

bool adapter_fits(int rows, int segments, int rank, int N) {
  // 2^32 threads a launch, in workgroups of 512 or 256
  return few_rows(rows, segments)
             ? tiles_of(rows, segments, 16) * (rank / 16) < (1ll << 23) && tiles_of(rows, segments, 16) * ((N + 511) / 512) < (1ll << 24)
             : tiles_of(rows, segments, 32) * ((rank + 63) / 64) < (1ll << 24) && tiles_of(rows, segments, 64) * ((N + 255) / 256) < (1ll << 24);
}

hipError_t launch_adapter_linear(const AdapterArgs& a, hipStream_t s) {
  if (at_once(a))
    return a.x_fmt == TABIT_FMT_BF16   ? few<TABIT_FMT_BF16>(a, s)
           : a.x_fmt == TABIT_FMT_INT8 ? few<TABIT_FMT_INT8>(a, s)
                                       : few<TABIT_FMT_MXFP4>(a, s);
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
