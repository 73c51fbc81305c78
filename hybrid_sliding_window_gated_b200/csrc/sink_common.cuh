// sink_common.cuh -- what the sink-attention kernels share: fp16 / bf16 warp
// MMAs, the order in which a row's 128 dims lie in shared memory, and the
// K' / V tile producer.
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

// D (16x8 fp32) += A (16x16) * B (16x8), fp16 and bf16.  Not volatile: a pure
// function of registers, which the compiler may move between other work.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
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

__device__ __forceinline__ float2 cmul(float2 x, float2 y) {
  return make_float2(x.x * y.x - x.y * y.y, x.x * y.y + x.y * y.x);
}

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
__device__ __forceinline__ void st_shared4(uint32_t at, const uint32_t* x) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3])
               : "memory");
}
__device__ __forceinline__ void ld_shared4(uint32_t at, uint32_t (&x)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(at));
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

// k' / ck of one row, fp16, in rope order into row r of `tile`; w_* are this
// lane's weights divided by ck, rot its pair's rotation at the row's position.
__device__ __forceinline__ void store_k_row(uint8_t* tile, int r, const KRow& x, int lane,
                                            float w_lo, float w_hi, float4 w_rest, float2 rot,
                                            float eps) {
  const float lo = bf16_f32(x.lo), hi = bf16_f32(x.hi);
  const float a0 = bf16_lo(x.rest.x), a1 = bf16_hi(x.rest.x);
  const float a2 = bf16_lo(x.rest.y), a3 = bf16_hi(x.rest.y);
  float ss = lo * lo + hi * hi + a0 * a0 + a1 * a1 + a2 * a2 + a3 * a3;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float rinv = rsqrtf(ss * (1.0f / kHeadDim) + eps);
  if (lane < kMaxPairs) {
    const float u = lo * rinv * w_lo, v = hi * rinv * w_hi;
    const int kk = lane >> 3, m = lane & 7;
    *reinterpret_cast<__half*>(tile + row_off(r, 2 * kk) + 2 * m) =
        __float2half_rn(u * rot.x - v * rot.y);
    *reinterpret_cast<__half*>(tile + row_off(r, 2 * kk + 1) + 2 * m) =
        __float2half_rn(v * rot.x + u * rot.y);
  }
  if (lane < 20) {
    int c0, by;
    rest_pos(lane, &c0, &by);
    *reinterpret_cast<uint32_t*>(tile + row_off(r, c0) + by) =
        pack_f16x2(a0 * rinv * w_rest.x, a1 * rinv * w_rest.y);
    *reinterpret_cast<uint32_t*>(tile + row_off(r, c0 + 1) + by) =
        pack_f16x2(a2 * rinv * w_rest.z, a3 * rinv * w_rest.w);
  }
}

// 16-byte chunk c (dims 8 c .. 8 c + 7) of V row r into split order.
__device__ __forceinline__ void store_v_chunk(uint8_t* tile, int r, int c, uint4 x) {
  const int m = c >> 2, by = 4 * (c & 3);
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m) + by) = x.x;
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m + 1) + by) = x.y;
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m + 2) + by) = x.z;
  *reinterpret_cast<uint32_t*>(tile + row_off(r, 4 * m + 3) + by) = x.w;
}

}  // namespace snk
}  // namespace swa
