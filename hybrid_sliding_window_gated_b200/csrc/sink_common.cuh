// sink_common.cuh -- what the sink-attention kernels share, most of it the
// backward's: fp16 warp MMAs, the order in which a row's 128 dims lie in its
// operand tiles, rows' scales, and the gate's two sigmoids.
//
// Order of the dims.  A contraction over the 128 dims may run over them in any
// order as long as both operands use the same one, and the columns of a product
// may come out in any order.  Both orders below are chosen so that a thread of
// an m16n8k16 fragment (lane = 4 * row + c, c = 0..3) finds what it needs in
// its own registers and in 16-byte pieces of a row:
//   K', q' ("rope order"): position 16 kk + m (m < 8, kk < 3) is the first and
//     position 16 kk + 8 + m the second dim of rotated pair 8 kk + m, so both
//     dims of a pair sit in one thread of the A fragment.  Pairs past rot_dim/2
//     are dims (2 j, 2 j + 1), with the identity rotation.  Dims 48..63 fill
//     k-step 3 and dims 64..127 k-steps 4..7 such that thread c holds dims
//     48 + 4 c .. + 3 and 32 m + 8 c .. + 7.
//   V ("split order"): dim 32 m + 8 c + 2 q + e at position 32 m + 8 q + 2 c + e:
//     thread c of the product's fragment holds dims 32 m + 8 c .. + 7.
#pragma once
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "sink_internal.h"
#include "warp_mma.cuh"

namespace swa {
namespace snk {

constexpr int kRowBytes = kHeadDim * 2;             // one row of a tile
constexpr int kTileBytes = kSinkTile * kRowBytes;   // 16 KiB
constexpr int kSinkBytes = kMaxSink * kRowBytes;    // 4 KiB
constexpr int kRopeDims = 2 * kMaxPairs;            // dims 0..47 hold every rotated pair

// D (16x8 fp32) += A (16x16) * B (16x8), fp16.  Not volatile: a pure
// function of registers, which the compiler may move between other work.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float bf16_f32(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Dims of rotated pair j (j < 24): (j, j + P) below P = rot_dim / 2, and the
// unrotated dims (2 j, 2 j + 1) from there on.
__device__ __forceinline__ int pair_lo(int j, int P) { return j < P ? j : 2 * j; }
__device__ __forceinline__ int pair_hi(int j, int P) { return j < P ? j + P : 2 * j + 1; }

// Byte offset of 16-byte chunk c of row r of a K', V, q' or dA tile: eight rows
// at one chunk index lie in eight different 16-byte bank groups.
__device__ __forceinline__ uint32_t row_off(int r, int c) {
  return static_cast<uint32_t>(r * kRowBytes + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Power of two not below every |w| (1 for all-zero weights): q' and k' are held
// in fp16 divided by it, so |q'| / c <= sqrt(128) whatever the weights.
__device__ __forceinline__ float pow2_ceil(float m) {
  if (!(m > 0.0f) || m == INFINITY) return 1.0f;
  int e;
  const float f = frexpf(m, &e);  // m = f 2^e, f in [1/2, 1)
  e = f == 0.5f ? e - 1 : e;
  return ldexpf(1.0f, min(max(e, -100), 100));
}

// A K row's part held by one lane: rotated pair `lane` (lanes < 24) and dims
// 48 + 4 lane .. + 3 (lanes < 20).
struct KRow {
  uint16_t lo, hi;
  uint2 rest;
};

__device__ __forceinline__ KRow load_k_row(const uint16_t* row, int lane, int dlo, int dhi) {
  KRow x;
  x.lo = x.hi = 0;
  x.rest = make_uint2(0u, 0u);
  if (row != nullptr) {
    if (lane < kMaxPairs) {
      x.lo = __ldg(row + dlo);
      x.hi = __ldg(row + dhi);
    }
    if (lane < 20) x.rest = __ldg(reinterpret_cast<const uint2*>(row + kRopeDims + 4 * lane));
  }
  return x;
}

// Byte offset inside a row (chunk, byte) of the two word pairs of lane's `rest`
// dims in rope order.
__device__ __forceinline__ void rest_pos(int lane, int* chunk0, int* byte) {
  if (lane < 4) {  // dims 48 + 4 c: k-step 3
    *chunk0 = 6;
    *byte = 4 * lane;
  } else {         // dims 64 + 32 m + 8 c + 4 h: k-step 4 + 2 m + h
    const int a = lane - 4;
    *chunk0 = 2 * (4 + 2 * (a >> 3) + (a & 1));
    *byte = 4 * ((a & 7) >> 1);
  }
}

// k' / ck of N rows, fp16, in rope order into rows r0 .. of `tile`; w_* are this lane's
// weights divided by ck, rot its pair's rotation at each row's position.  eps of a row that
// only fills up a tile is not 0, so that the row's zeros stay zeros.  A row that has no
// finite k' (an infinity or NaN, or all zeros with eps = 0) becomes zeros too: a masked
// pair's 0 x NaN would reach the sums of the rows around it, and where the pair is visible
// the query's lse is NaN, and P with it.  The rows' chains of shuffles run side by side.
template <int N>
__device__ __forceinline__ void store_k_rows(uint8_t* tile, int r0, const KRow (&x)[N], int lane,
                                             float w_lo, float w_hi, float4 w_rest,
                                             const float2 (&rot)[N], const float (&eps)[N]) {
  float ss[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float lo = bf16_f32(x[e].lo), hi = bf16_f32(x[e].hi);
    const float a0 = bf16_lo(x[e].rest.x), a1 = bf16_hi(x[e].rest.x);
    const float a2 = bf16_lo(x[e].rest.y), a3 = bf16_hi(x[e].rest.y);
    ss[e] = lo * lo + hi * hi + a0 * a0 + a1 * a1 + a2 * a2 + a3 * a3;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int e = 0; e < N; ++e) ss[e] += __shfl_xor_sync(0xffffffffu, ss[e], o);
  uint32_t pair[N], r01[N], r23[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float rinv = rsqrtf(ss[e] * (1.0f / kHeadDim) + eps[e]);
    const float u = bf16_f32(x[e].lo) * rinv * w_lo, v = bf16_f32(x[e].hi) * rinv * w_hi;
    pair[e] = pack_f16x2(u * rot[e].x - v * rot[e].y, v * rot[e].x + u * rot[e].y);
    r01[e] = pack_f16x2(bf16_lo(x[e].rest.x) * rinv * w_rest.x,
                        bf16_hi(x[e].rest.x) * rinv * w_rest.y);
    r23[e] = pack_f16x2(bf16_lo(x[e].rest.y) * rinv * w_rest.z,
                        bf16_hi(x[e].rest.y) * rinv * w_rest.w);
    const float f = ss[e] * rinv;  // NaN for inf * 0, 0 * inf and NaN
    if (f != f) pair[e] = r01[e] = r23[e] = 0u;
  }
  int c0, by;
  rest_pos(lane, &c0, &by);
  const int kk = lane >> 3, m = lane & 7;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int r = r0 + e;
    if (lane < kMaxPairs) {
      *reinterpret_cast<uint16_t*>(tile + row_off(r, 2 * kk) + 2 * m) =
          static_cast<uint16_t>(pair[e]);
      *reinterpret_cast<uint16_t*>(tile + row_off(r, 2 * kk + 1) + 2 * m) =
          static_cast<uint16_t>(pair[e] >> 16);
    }
    if (lane < 20) {
      *reinterpret_cast<uint32_t*>(tile + row_off(r, c0) + by) = r01[e];
      *reinterpret_cast<uint32_t*>(tile + row_off(r, c0 + 1) + by) = r23[e];
    }
  }
}

// The largest |v| of N rows whose dims 4 lane .. + 3 this lane holds (bf16 pairs).
// bf16 magnitudes order as their bit patterns do (an inf or NaN counts as inf).
template <int N>
__device__ __forceinline__ void v_absmax(const uint2 (&v)[N], float (&m)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const uint32_t a = __vmaxu2(v[e].x & 0x7fff7fffu, v[e].y & 0x7fff7fffu);
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(a & 0xffffu, a >> 16));
    m[e] = __uint_as_float(min(top, 0x7f80u) << 16);
  }
}
// Dims 4 lane .. + 3 of a V row times f, fp16, in split order into row r of `tile`:
// they are 32 m + 8 c + 2 q .. with q = 0 or 2, words q and q + 1 of the group.
__device__ __forceinline__ void store_v_row(uint8_t* tile, int r, uint2 v, int lane, float f) {
  const int m = lane >> 3, c = (lane & 7) >> 1, q = 2 * (lane & 1);
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m + q) + 4 * c) =
      pack_f16x2(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m + q + 1) + 4 * c) =
      pack_f16x2(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
}

// 2^x for a whole x in [-126, 127]
__device__ __forceinline__ float pow2i(float x) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<int>(x) + 127) << 23);
}
// Exponent a of a V row of the forward, which enters as the fp16 of v 2^a.  Rows whose
// largest entry lies in [2^-6, 2^7) all have kVExp: entries down to 2^-25, 2^-19 of the
// largest at least, keep their bf16 bits.  Any other row's largest goes to [2^8, 2^9),
// which keeps entries down to 2^-33 of it.  kZeroRow: a row of zeros, which no scale
// concerns.  kBadRow: a row that is not finite, which is summed apart.  Tiles whose rows all have kVExp
// skip the scaling of P: 4 x 4096 tokens of 32 heads take 220 us, else 399 us.
constexpr float kVExp = 8.0f, kZeroRow = 127.0f, kBadRow = -128.0f;
__device__ __forceinline__ float v_exp(float m) {
  if (m == 0.0f) return kZeroRow;
  if (!(m < INFINITY)) return kBadRow;
  if (m >= 0.015625f && m < 128.0f) return kVExp;
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 255u) - 127;
  return static_cast<float>(min(126, 8 - e));  // at least 8 - 127
}

// sigmoid(g) and 1 - sigmoid(g) = sigmoid(-g) of two values, each off by at most 1.03e-4 of
// itself, where dA's rounding to fp16 is 4.9e-4 and dg's to bf16 3.9e-3: with e = exp(-|g|)
// and r = 1 / (1 + e) they are r and e r, or the other way round (the evaluation of
// sigmoid2, kept to both halves; with a reciprocal instruction per value instead the
// backward's rows took 190 us where this took 170).
__device__ __forceinline__ float2 sigmoid_both(float2 g, float2* rest) {
  constexpr float kL2e = 1.4426950408889634f;
  const float2 e = make_float2(ex2_approx(-fabsf(g.x) * kL2e), ex2_approx(-fabsf(g.y) * kL2e));
  const float2 d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  float2 r = __ffma2_rn(d, make_float2(0.32286211f, 0.32286211f),
                        make_float2(-1.45351115f, -1.45351115f));
  r = __ffma2_rn(r, d, make_float2(2.12052006f, 2.12052006f));
  const float2 t = __ffma2_rn(make_float2(-d.x, -d.y), r, make_float2(1.0f, 1.0f));
  r = __ffma2_rn(r, t, r);
  const float2 er = __fmul2_rn(e, r);
  *rest = make_float2(g.x >= 0.0f ? er.x : r.x, g.y >= 0.0f ? er.y : r.y);
  return make_float2(g.x >= 0.0f ? r.x : er.x, g.y >= 0.0f ? r.y : er.y);
}

// The largest |w| of the norm weights, by the 32 lanes of a warp.
__device__ __forceinline__ float warp_absmax(const float* w, int lane) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(__ldg(w + lane + 32 * i)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ void pdl_start() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The raw row of x as floats, as far as a fragment's thread c covers it: pairs 8 kk + 2 c + e and
// dims 48 + 4 c .., 64 + 8 c .., 96 + 8 c ...
struct RawRow {
  float lo[6], hi[6], rest[20];
};
// Dim of rest[i] (thread c), and its weight.
__device__ __forceinline__ int rest_dim(int i, int c) {
  return i < 4 ? 48 + 4 * c + i : (i < 12 ? 64 + 8 * c + (i - 4) : 96 + 8 * c + (i - 12));
}
__device__ __forceinline__ float raw_rinv(const RawRow& x, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 6; ++i) s += x.lo[i] * x.lo[i] + x.hi[i] * x.hi[i];
#pragma unroll
  for (int i = 0; i < 20; ++i) s += x.rest[i] * x.rest[i];
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  return rsqrtf(s * (1.0f / kHeadDim) + eps);
}

}  // namespace snk
}  // namespace swa
