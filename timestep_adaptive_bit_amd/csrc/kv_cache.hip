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
// inputs alone.
//
// Each byte moves once.  Measured at 17776 tokens x 30 heads x 64, rotated in neighbour
// pairs, had_block 32: append 52 us (3.4 TB/s; 26 us for its loads alone, and the table
// rows, the transform and the stores add 6 to 9 us each: the vector units are 75% busy
// and the memory system is not full), read 34 us (5.0 TB/s, what a large copy reaches).
// Two heads a lane sharing a table row took 50 us, in four more kernels; not kept.
#include "kv_common.h"

namespace tabit {
namespace {

using namespace kv;

constexpr int NT = 256;

// Codes and scale byte of one lane's eight elements of a block (four lanes); m is the
// largest magnitude of the lane's.
__device__ __forceinline__ void mx_encode(float (&v)[8], float m, uint32_t& codes, uint32_t& scale) {
  m = fmaxf(m, lane_xor<1>(m));
  m = fmaxf(m, lane_xor<2>(m));
  const int X = mx_exponent(m);
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X: X is at most 125
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= inv;
  codes = e2m1x8(v);
  scale = (uint32_t)(X + 127);
}

// The (token, head) of this group of GL lanes: a workgroup has a tile of `hb` = 1, 2 or
// 4 heads, which divide the head count, times as many tokens as fit, so that it reads
// runs of hb vectors and a head's rows of consecutive slots are one run of one
// workgroup's: spread over workgroups of different dies, 32 bytes each, a line of codes
// went through four L2s.
struct Place {
  int t, h;
};
template <int GL>
__device__ __forceinline__ Place place(int heads, int hb_shift) {
  const unsigned tiles = (unsigned)heads >> hb_shift;         // head tiles, the fastest index
  const unsigned tt = blockIdx.x / tiles, th = blockIdx.x - tt * tiles;
  const int g = threadIdx.x / GL;
  return {(int)(tt * ((NT / GL) >> hb_shift)) + (g >> hb_shift),
          (int)(th << hb_shift) + (g & ((1 << hb_shift) - 1))};
}

// Byte offset of a valid slot's scales; its codes are at 16 times that.
__device__ __forceinline__ uint64_t scale_at(const KvCacheArgs& c, int64_t slot, int h) {
  const uint32_t page = (uint32_t)(slot >> c.page_shift), in = (uint32_t)slot & ((1u << c.page_shift) - 1);
  const uint64_t row = (((uint64_t)page * (uint32_t)c.heads + (uint32_t)h) << c.page_shift) | in;
  return row * (uint32_t)(c.dim_pad >> 5);
}

// Whether any of v is NaN or infinite: infinities stand out in the
// largest magnitude m, NaN in a sum (which may also overflow, and then is infinite).
__device__ __forceinline__ bool any_bad(const float (&v)[8], float m) {
  float s = v[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) s += v[e];
  return s != s || !finite_f32(m);
}

template <int GL>
__global__ void __launch_bounds__(NT)
kv_append_kernel(KvCacheArgs c, int hb_shift, const uint16_t* __restrict__ k, long long k_stride,
                 const uint16_t* __restrict__ v, long long v_stride, int tokens,
                 const int64_t* __restrict__ slots, RopeArgs rope,
                 const int* __restrict__ positions) {
  const int lane = threadIdx.x & 63;
  const int gl = threadIdx.x % GL;
  const auto [t, h] = place<GL>(c.heads, hb_shift);
  if (t >= tokens) return;                       // whole groups leave together
  const int e0 = gl * 8;
  // everything but the tables' rows is asked for at once
  const int64_t slot = slots[t];
  int pos = rope.rope_dim > 0 ? positions[t] : 0;
  uint4 kw = make_uint4(0, 0, 0, 0), ko = kw, vw = kw;
  if (e0 < c.head_dim) {
    const uint16_t* kp = k + t * k_stride + (long long)h * c.head_dim;
    kw = *reinterpret_cast<const uint4*>(kp + e0);
    if (!rope.interleaved && e0 < rope.rope_dim)
      ko = *reinterpret_cast<const uint4*>(kp + turn_partner(e0, rope));
    vw = *reinterpret_cast<const uint4*>(v + t * v_stride + (long long)h * c.head_dim + e0);
  }
  if (slot < 0 || slot >= (long long)c.num_pages << c.page_shift) return;
  bool bad = false;
  if (rope.rope_dim > 0 && (pos < 0 || pos >= rope.num_positions)) {
    bad = true;                                  // no such table row: stored as not a number
    pos = 0;
  }
  float a[8], b[8];
  turned8(kw, ko, e0, rope, pos, a);
  unpack8(vw, b);
  if (c.had) {
    fwht32_lanes(a, lane);
    fwht32_lanes(b, lane);
  }
  float ma = 0.0f, mb = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ma = fmaxf(ma, fabsf(a[e]));
    mb = fmaxf(mb, fabsf(b[e]));
  }
  bad = bad || any_bad(a, ma) || any_bad(b, mb);
  // one bad element in the head's key or value marks the whole token
  const unsigned long long group = ((1ull << GL) - 1) << (lane / GL * GL);
  bad = (__ballot(bad) & group) != 0;
  uint32_t kc, ks, vc, vs;
  mx_encode(a, ma, kc, ks);
  mx_encode(b, mb, vc, vs);
  if (bad) {   // a query that sees the token answers NaN, others never touch it
    kc = vc = 0u;
    ks = 255u;
    vs = 127u;
  }
  if (e0 >= c.dim_pad) return;
  const uint64_t at = scale_at(c, slot, h);
  *reinterpret_cast<uint32_t*>(c.k_codes + at * 16 + gl * 4) = kc;
  *reinterpret_cast<uint32_t*>(c.v_codes + at * 16 + gl * 4) = vc;
  if ((gl & 3) == 0) {
    c.k_scales[at + (gl >> 2)] = (uint8_t)ks;
    c.v_scales[at + (gl >> 2)] = (uint8_t)vs;
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
kv_read_kernel(KvCacheArgs c, int hb_shift, const int64_t* __restrict__ slots, int tokens,
               uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  const int lane = threadIdx.x & 63;
  const int gl = threadIdx.x % GL;
  const auto [t, h] = place<GL>(c.heads, hb_shift);
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  const int e0 = gl * 8;
  float a[8] = {}, b[8] = {};
  if (slot >= 0 && slot < (long long)c.num_pages << c.page_shift && e0 < c.dim_pad) {
    const uint64_t at = scale_at(c, slot, h);
    mx_decode(*reinterpret_cast<const uint32_t*>(c.k_codes + at * 16 + gl * 4), c.k_scales[at + (gl >> 2)], a);
    mx_decode(*reinterpret_cast<const uint32_t*>(c.v_codes + at * 16 + gl * 4), c.v_scales[at + (gl >> 2)], b);
  }
  if (c.had) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {      // (first, and exactly: 32 of them could pass fp32)
      a[e] *= 0.03125f;
      b[e] *= 0.03125f;
    }
    fwht32_lanes(a, lane);
    fwht32_lanes(b, lane);
  }
  if (e0 >= c.head_dim) return;
  const long long o = ((long long)t * c.heads + h) * c.head_dim + e0;
  write8(k + o, a);
  write8(v + o, b);
}

// Tokens go in pieces, so that a launch has fewer than 2^24 workgroups (2^32 threads are
// the limit).
template <typename Launch>
hipError_t in_pieces(const KvCacheArgs& c, int tokens, Launch launch) {
  const int gl = c.dim_pad <= 64 ? 8 : 16;
  const int hb_shift = c.heads % 4 == 0 ? 2 : c.heads % 2 == 0 ? 1 : 0;
  const int per = (NT / gl) >> hb_shift, tiles = c.heads >> hb_shift;
  const int piece = max(1, (1 << 23) / tiles) * per;
  for (long long first = 0; first < tokens; first += piece) {   // first + piece may pass 2^31
    const int n = (int)min((long long)piece, tokens - first);
    launch(gl, hb_shift, (unsigned)((n + per - 1) / per * tiles), first, n);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_append(const KvCacheArgs& c, const uint16_t* k, long long k_stride,
                            const uint16_t* v, long long v_stride, int tokens,
                            const int64_t* slots, const RopeArgs& rope, const int* positions,
                            hipStream_t s) {
  return in_pieces(c, tokens, [&](int gl, int hb_shift, unsigned grid, long long first, int n) {
    auto* kernel = gl == 8 ? &kv_append_kernel<8> : &kv_append_kernel<16>;
    kernel<<<grid, NT, 0, s>>>(c, hb_shift, k + first * k_stride, k_stride, v + first * v_stride,
                               v_stride, n, slots + first, rope,
                               positions == nullptr ? nullptr : positions + first);
  });
}

hipError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int tokens, uint16_t* k,
                          uint16_t* v, hipStream_t s) {
  return in_pieces(c, tokens, [&](int gl, int hb_shift, unsigned grid, long long first, int n) {
    const long long o = first * c.heads * c.head_dim;
    auto* kernel = gl == 8 ? &kv_read_kernel<8> : &kv_read_kernel<16>;
    kernel<<<grid, NT, 0, s>>>(c, hb_shift, slots + first, n, k + o, v + o);
  });
}

}  // namespace tabit
