// sink_bwd.cu -- backward of the gated sliding-window attention with sink
// tokens, for sm_100a.
//
// With s = sigmoid(g), A the attention output before the gate, P_ij the
// probabilities and x . y a sum over the 128 dims:
//   dg_i  = dO_i A_i s (1 - s) = dO_i o_i (1 - s)
//   dA_i  = dO_i s,      D_i = dA_i . A_i = sum_j P_ij dP_ij
//   P_ij  = exp(scale q'_i . k'_j - lse_i),   dP_ij = dA_i . v_j
//   dS_ij = P_ij (dP_ij - D_i)
//   dq'_i = scale sum_j dS_ij k'_j,  dk'_j = scale sum_i dS_ij q'_i,
//   dv_j  = sum_i P_ij dA_i
// and from dx' (x = q or k) back through RoPE and the norm, with u = x / rms:
//   du = w RoPE^-1(dx'),  dx = (du - u mean(du u)) / rms,  dw = sum RoPE^-1(dx') u.
// o is the forward's bf16 output: it gives dg without a second P V, at the price of its
// rounding beside dg's own (2.4e-3 in the 2-norm, 1.7e-3 from a recomputed A).  D could
// come from o too, but dP - D cancels where a row's probability sits on few keys (a
// sequence's first tokens), and o's rounding would remain.
//
// Kernels, each waiting for the one before it on the stream:
//   sink_bwd_kv_kernel    k' and v as fp16 operand rows; the table of rotations.
//   sink_bwd_rows_kernel  q' and dA as operand rows, and dg.
//   sink_bwd_q_kernel     query-major: 16 queries of one head per warp step, nine
//                         band blocks and the sinks: S, dP, D, dQ.  Writes dq and D.
//   sink_bwd_sink_kernel  the sinks' dk' and dv: every query contributes to the same
//                         16 keys, so chunks of tokens make partial sums, and
//   sink_bwd_sum_kernel   adds them up in a fixed order.
//   sink_bwd_k_kernel     key-major: 16 keys per warp against the nine blocks of
//                         queries that see them, all heads of the group: S^T, dP^T,
//                         dV, dK.  Adds the sinks' sums to the keys that are sinks.
//   sink_bwd_w_kernel     adds up the CTAs' dwq and dwk in a fixed order.
// No sum is made by atomics, so results do not depend on the order of CTAs.
//
// What bounds it.  The seven products of 160 keys per query take 39 us each for
// 16,384 tokens of 32 / 8 heads at the 550 TFLOP/s that mma.sync reaches, with about
// as many shared-memory cycles for their operands; memory needs 0.19 ms.  Warp tiles
// of 16 x 16 waste little of the 128-key band (1.1 of 1), where tcgen05's 128 rows
// of two heads would compute 1.6 times the products and hand S, dP, P and dS through
// TMEM; the two passes instead of one with atomics cost two products, since a band
// keeps dK and dV of 192 keys live, too many for registers.  Neither pass is bound by the
// products (below), so that count does not speak against tcgen05, on which these two
// passes were not built: the window backward, built there, takes 770 us at this shape.
//
// Measured there (us): kv 44, rows 192, q 354, sinks 65 + 5, k 336, w 6; the
// key-major pass reads its operands from shared memory at 66 % of the pipe's rate
// with the tensor pipe at 44 %, and the query-major pass is its S - P - dS chain.
//
// Numbers.  All products have fp16 operands and fp32 sums.  q' and k' are divided
// by a power of two not below the norm weights (at most sqrt(128) then); a row
// of dA is scaled by 2^b and one of v by 2^a so that its largest entry lies in
// [1, 4): gradients and values of any magnitude keep fp16's 2^-11 rounding.  The
// scales leave a product where its row or column index carries them; where an
// index is summed over, the least exponent of the rows at hand takes their place,
// and only entries far below the largest lose bits.  |dS| 2^(a + b) <= 2 x 128 x 2 x 4.
//
// Values that are not finite.  A masked pair has P = dS = 0, but 0 * inf and 0 * NaN are
// NaN in a product of tiles: the operand rows hold zeros in such places, and the query's
// lse (from the forward for q and k, here for dA) or the key's exponent (v) is NaN, which
// reaches P or dP of exactly the pairs that are visible.
#include <atomic>

#include "launch.cuh"
#include "sink_common.cuh"

namespace swa {
namespace snk {

constexpr float kNoScale = 126.0f;  // exponent of an all-zero row: takes part in no minimum

// Exponent that brings m into [1, 2), or [2, 4) from 2^127 on, so that the factor is a
// normal fp32 number; below 2 from 2^-126 down.
__device__ __forceinline__ float scale_exp(float m) {
  if (!(m > 0.0f)) return kNoScale;
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 255u) - 127;
  return static_cast<float>(max(-126, min(126, -e)));
}
// 2^(am - e - up) for a key whose row has exponent e; NaN for a row that is not finite, whose
// dP is NaN then for every query that sees it.
__device__ __forceinline__ float key_factor(float am, float e, float up) {
  return e == e ? pow2i(fmaxf(fminf(am - e, 0.0f) - up, -126.0f)) : e;
}
// The larger of two numbers; NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// v 2^x for whole x in [-252, 252], in two steps
__device__ __forceinline__ float scale2(float v, float x) {
  const float h = truncf(0.5f * x);
  return v * pow2i(h) * pow2i(x - h);
}

// Factors f that make acc into acc v 2^x, for rows r and r + 8 of a fragment.  Beyond 2^100
// (values and gradients both near the end of their range, though the sums need not be
// large) a part of it is taken here, since the factor would leave fp32.
__device__ __forceinline__ void split_scale(float (&acc)[16][4], float v, const float (&x)[2],
                                            float (&f)[2]) {
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const float at = x[rr], over = fmaxf(at - 100.0f, 0.0f);
    if (__any_sync(0xffffffffu, over > 0.0f)) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        acc[n][2 * rr] = scale2(acc[n][2 * rr], over);
        acc[n][2 * rr + 1] = scale2(acc[n][2 * rr + 1], over);
      }
    }
    f[rr] = scale2(v, at - over);
  }
}

// ------------------------------------------------------------- operand rows

// One warp per token: its rotation, and k' and v of every KV head.
__global__ void __launch_bounds__(256) sink_bwd_kv_kernel(const SinkBwdArgs a) {
  // operand rows are put together here and leave in 16-byte pieces
  __shared__ __align__(16) uint8_t stage[8][2][4 * kRowBytes];
  pdl_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = static_cast<long long>(blockIdx.x) * 8 + warp;
  if (gw >= static_cast<long long>(a.B) * a.Tp) return;
  const int b = static_cast<int>(gw / a.Tp);
  const int t = static_cast<int>(gw - static_cast<long long>(b) * a.Tp);
  const int P = a.half_rot;
  float2 rot = make_float2(1.0f, 0.0f);
  if (lane < P) rope_cos_sin(static_cast<double>(t), a.inv_freq[lane], &rot.x, &rot.y);
  if (b == 0 && lane < kMaxPairs) a.rot[static_cast<long long>(t) * kMaxPairs + lane] = rot;
  const float ick = 1.0f / pow2_ceil(warp_absmax(a.wk, lane));
  const int dlo = lane < kMaxPairs ? pair_lo(lane, P) : 0;
  const int dhi = lane < kMaxPairs ? pair_hi(lane, P) : 0;
  const float w_lo = __ldg(a.wk + dlo) * ick, w_hi = __ldg(a.wk + dhi) * ick;
  float4 w_rest = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < 20) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(a.wk + kRopeDims + 4 * lane));
    w_rest = make_float4(w.x * ick, w.y * ick, w.z * ick, w.w * ick);
  }
  const bool real = t < a.T;
  constexpr int kN = 4;  // heads at a time (their rows lie next to each other)
  for (int h0 = 0; h0 < a.Hkv; h0 += kN) {
    KRow x[kN][1];
    uint2 v[kN];
    float m[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const bool have = real && h0 + e < a.Hkv;
      const long long src = ((static_cast<long long>(b) * a.T + t) * a.Hkv + h0 + e) * kHeadDim;
      x[e][0] = load_k_row(have ? a.k + src : nullptr, lane, dlo, dhi);
      v[e] = have ? __ldg(reinterpret_cast<const uint2*>(a.v + src + 4 * lane))
                  : make_uint2(0u, 0u);
    }
    v_absmax<kN>(v, m);
    const float2 rot1[1] = {rot};
    const float eps1[1] = {real ? a.eps : 1.0f};
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      // a row's chunks lie as row t & 7 of a tile
      uint8_t* kt = stage[warp][0] + (e - (t & 7)) * kRowBytes;
      uint8_t* vt = stage[warp][1] + (e - (t & 7)) * kRowBytes;
      store_k_rows<1>(kt, t & 7, x[e], lane, w_lo, w_hi, w_rest, rot1, eps1);
      // a row that is not finite: zeros, and NaN for its exponent
      const bool bad = m[e] == INFINITY;
      const float ex = bad ? NAN : scale_exp(m[e]);
      store_v_row(vt, t & 7, bad ? make_uint2(0u, 0u) : v[e], lane, bad ? 1.0f : pow2i(ex));
      if (lane == 0 && h0 + e < a.Hkv)
        a.va[(static_cast<long long>(b) * a.Hkv + h0 + e) * a.Tp + t] = ex;
    }
    __syncwarp();
#pragma unroll
    for (int y = 0; y < kN / 2; ++y) {
      const int e = 2 * y + (lane >> 4), at = e * kRowBytes + 16 * (lane & 15);
      if (h0 + e >= a.Hkv) continue;
      const long long dst =
          ((static_cast<long long>(b) * a.Hkv + h0 + e) * a.Tp + t) * kRowBytes + 16 * (lane & 15);
      *reinterpret_cast<uint4*>(a.kr + dst) = *reinterpret_cast<const uint4*>(stage[warp][0] + at);
      *reinterpret_cast<uint4*>(a.vr + dst) = *reinterpret_cast<const uint4*>(stage[warp][1] + at);
    }
    __syncwarp();
  }
}

// One warp per 16 tokens of a query head, two rows at a time and four dims per lane:
// q' and dA as operand rows, dg, and the rows' lse and exponent b.  Bound by memory:
// 1 KiB read and 768 bytes written per row.  The next two rows are on their way to
// shared memory while a pair is worked on: 170 us for 16,384 tokens of 32 heads against
// 241 with plain loads and as many warps, and 192 us with D's estimate and the checks for
// rows that are not finite (issue slots 81 %, DRAM 59 %).
__global__ void __launch_bounds__(256, 4) sink_bwd_rows_kernel(const SinkBwdArgs a) {
  constexpr int kN = 2;
  __shared__ __align__(16) uint8_t in[8][2][4][kN * kRowBytes];  // q, g, dO, o as they are
  // operand rows are put together here and leave in 16-byte pieces
  __shared__ __align__(16) uint8_t stage[8][2][kN * kRowBytes];
  pdl_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, P = a.half_rot;
  const long long gw = static_cast<long long>(blockIdx.x) * 8 + warp;
  // heads of one token group are neighbours: their rows lie next to each other
  const long long grp = gw / a.Hq;
  const int hq = static_cast<int>(gw - grp * a.Hq);
  const int per = a.Tp >> 4, b = static_cast<int>(grp / per);
  if (b >= a.B) return;
  const int t0 = static_cast<int>(grp - static_cast<long long>(b) * per) * 16;
  const uint16_t* src[4] = {a.q, a.g, a.dO, a.o};
  const auto fetch = [&](int i, int buf) {
    const int t = t0 + i + (lane >> 4);
    const long long at = ((static_cast<long long>(b) * a.T + min(t, a.T - 1)) * a.Hq + hq) *
                             kHeadDim + 8 * (lane & 15);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      cp_async16(smem_u32(in[warp][buf][x]) + 16 * lane, src[x] + at, t < a.T);
    cp_async_commit();
  };
  const float* lse = a.lse + (static_cast<long long>(b) * a.Hq + hq) * a.T;
  float2 rot[kN];
  float l2[kN];
  const auto fetch_row = [&](int i) {  // rotations and lse, held in registers
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int t = t0 + i + e;
      rot[e] = lane < kMaxPairs ? a.rot[static_cast<long long>(t) * kMaxPairs + lane]
                                : make_float2(1.f, 0.f);
      l2[e] = t < a.T ? __ldg(lse + t) * 1.4426950408889634f : 0.f;
    }
  };
  fetch(0, 0);
  fetch_row(0);
  const float icq = 1.0f / pow2_ceil(warp_absmax(a.wq, lane));
  const int dlo = lane < kMaxPairs ? pair_lo(lane, P) : 0;
  const int dhi = lane < kMaxPairs ? pair_hi(lane, P) : 0;
  const float w_lo = __ldg(a.wq + dlo) * icq, w_hi = __ldg(a.wq + dhi) * icq;
  float4 w_rest = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < 20) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(a.wq + kRopeDims + 4 * lane));
    w_rest = make_float4(w.x * icq, w.y * icq, w.z * icq, w.w * icq);
  }
  const long long out = (static_cast<long long>(b) * a.Hq + hq) * a.Tp + t0;
  float bm = kNoScale;
#pragma unroll 1
  for (int i = 0; i < 16; i += kN) {
    const int buf = (i / kN) & 1;
    if (i + kN < 16) {
      fetch(i + kN, buf ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncwarp();  // the rows have landed, and the stage has been read out
    float2 u0[kN], u1[kN];
    float m[kN], eps[kN], D[kN];
    KRow x[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const uint8_t* row = &in[warp][buf][0][0] + e * kRowBytes;
      constexpr int kTensor = kN * kRowBytes;
      const uint16_t* qrow = reinterpret_cast<const uint16_t*>(row);
      x[e].lo = x[e].hi = 0;
      x[e].rest = make_uint2(0u, 0u);
      if (lane < kMaxPairs) {
        x[e].lo = qrow[dlo];
        x[e].hi = qrow[dhi];
      }
      if (lane < 20) x[e].rest = *reinterpret_cast<const uint2*>(qrow + kRopeDims + 4 * lane);
      const uint2 g2 = *reinterpret_cast<const uint2*>(row + kTensor + 8 * lane);
      const uint2 d2 = *reinterpret_cast<const uint2*>(row + 2 * kTensor + 8 * lane);
      const uint2 o2 = *reinterpret_cast<const uint2*>(row + 3 * kTensor + 8 * lane);
      float2 n0, n1;
      const float2 s0 = sigmoid_both(make_float2(bf16_lo(g2.x), bf16_hi(g2.x)), &n0);
      const float2 s1 = sigmoid_both(make_float2(bf16_lo(g2.y), bf16_hi(g2.y)), &n1);
      const float2 d0 = make_float2(bf16_lo(d2.x), bf16_hi(d2.x));
      const float2 d1 = make_float2(bf16_lo(d2.y), bf16_hi(d2.y));
      const float2 q0 = make_float2(bf16_lo(o2.x), bf16_hi(o2.x));
      const float2 q1 = make_float2(bf16_lo(o2.y), bf16_hi(o2.y));
      u0[e] = __fmul2_rn(d0, s0);
      u1[e] = __fmul2_rn(d1, s1);
      const float2 x0 = __fmul2_rn(d0, q0), x1 = __fmul2_rn(d1, q1);
      D[e] = (x0.x + x0.y) + (x1.x + x1.y);
      const float2 y0 = __fmul2_rn(x0, n0), y1 = __fmul2_rn(x1, n1);
      const int t = t0 + i + e;
      eps[e] = t < a.T ? a.eps : 1.0f;
      if (t < a.T)
        *reinterpret_cast<uint2*>(
            a.dg + ((static_cast<long long>(b) * a.T + t) * a.Hq + hq) * kHeadDim + 4 * lane) =
            make_uint2(pack_bf16x2(y0.x, y0.y), pack_bf16x2(y1.x, y1.y));
      const float mx = max_nan(max_nan(fabsf(u0[e].x), fabsf(u0[e].y)),
                               max_nan(fabsf(u1[e].x), fabsf(u1[e].y)));
      // magnitudes order as their bits do, NaN above all
      m[e] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    }
    // the two rows' sums, row 0's in lanes below 16 and row 1's above
    const bool up = lane & 16;
    float Ds = (up ? D[1] : D[0]) + __shfl_xor_sync(0xffffffffu, up ? D[0] : D[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) Ds += __shfl_xor_sync(0xffffffffu, Ds, o);
    // the stage holds rows i & 7 .. of an eight-row tile
    uint8_t* qt = stage[warp][0] - (i & 7) * kRowBytes;
    uint8_t* dt = stage[warp][1] - (i & 7) * kRowBytes;
    store_k_rows<kN>(qt, i & 7, x, lane, w_lo, w_hi, w_rest, rot, eps);
    const int md = lane >> 3, c = (lane & 7) >> 1, q = 2 * (lane & 1);
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const bool bad = !(m[e] < INFINITY);  // a row that is not finite: zeros, lse NaN
      const float be = bad ? kNoScale : scale_exp(m[e]), f = pow2i(be);
      bm = fminf(bm, be);
      const int r = (i & 7) + e;
      *reinterpret_cast<uint32_t*>(dt + row_off(r, 4 * md + q) + 4 * c) =
          bad ? 0u : pack_f16x2(u0[e].x * f, u0[e].y * f);
      *reinterpret_cast<uint32_t*>(dt + row_off(r, 4 * md + q + 1) + 4 * c) =
          bad ? 0u : pack_f16x2(u1[e].x * f, u1[e].y * f);
      if (lane == 16 * e)
        a.row[out + i + e] =
            make_float4(bad ? NAN : l2[e], be, fabsf(Ds) < INFINITY ? Ds : 0.f, 0.f);
    }
    if (i + kN < 16) fetch_row(i + kN);
    __syncwarp();
    const long long at = (out + i) * kRowBytes + 16 * lane;
    *reinterpret_cast<uint4*>(a.qr + at) =
        *reinterpret_cast<const uint4*>(stage[warp][0] + 16 * lane);
    *reinterpret_cast<uint4*>(a.dr + at) =
        *reinterpret_cast<const uint4*>(stage[warp][1] + 16 * lane);
  }
  if (lane == 0) a.bmin[out >> 4] = bm;
}

// ------------------------------------------- back through RoPE and the norm

// The rotated dims of a warp's 16 rows pass through shared memory (rows of 96
// bytes), because a fragment's thread holds them two bytes at a time: 16-byte
// accesses to global memory on one side, 2-byte ones to shared memory on the other.
constexpr int kRopeRow = kRopeDims * 2;
constexpr int kRopeBytes = 16 * kRopeRow;

// Start the copy of dims 0 .. 47 of rows 0 .. rows - 1 (row x at src + x * stride)
// into the warp's buffer; rows past them become zeros.
__device__ __forceinline__ void rope_fetch(uint8_t* buf, const uint16_t* src, long long stride,
                                           int rows, int lane) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int x = lane + 32 * i, row = x / 6, ch = x - 6 * row;
    cp_async16(smem_u32(buf) + row * kRopeRow + 16 * ch,
               src + (row < rows ? row * stride : 0) + 8 * ch, row < rows);
  }
  cp_async_commit();
}

// dx of a fragment's 16 rows whose accumulators hold dx' in rope order times a
// factor that f undoes for the thread's rows r and r + 8.  src, dst: row 0 of x and
// dx; rot: the rows' rotations, row 0 of the table.  rope_fetch has been called
// for the same rows.  dw[d] gains the rows' share of the weight gradient (one
// warp's own array).
__device__ __forceinline__ void norm_rope_back(const float (&acc)[16][4], const float (&f)[2],
                                               uint8_t* buf, const uint16_t* src, uint16_t* dst,
                                               long long stride, int rows, const float2* rot,
                                               const float* w, float* dw, int lane, int P,
                                               float eps) {
  const int c = lane & 3, r = lane >> 2;
  float dws[32];  // by i: 0..5 first and 6..11 second dims of the pairs, then the rest
#pragma unroll
  for (int i = 0; i < 32; ++i) dws[i] = 0.f;
  uint32_t rest[2][10];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int row = r + 8 * rr;
    uint2 r3 = make_uint2(0u, 0u);
    uint4 r4 = make_uint4(0u, 0u, 0u, 0u), r6 = r4;
    if (row < rows) {
      const uint16_t* p = src + row * stride;
      r3 = __ldg(reinterpret_cast<const uint2*>(p + 48 + 4 * c));
      r4 = __ldg(reinterpret_cast<const uint4*>(p + 64 + 8 * c));
      r6 = __ldg(reinterpret_cast<const uint4*>(p + 96 + 8 * c));
    }
    const uint32_t x[10] = {r3.x, r3.y, r4.x, r4.y, r4.z, r4.w, r6.x, r6.y, r6.z, r6.w};
#pragma unroll
    for (int i = 0; i < 10; ++i) rest[rr][i] = x[i];
  }
  cp_async_wait<0>();
  __syncwarp();
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int row = r + 8 * rr;
    uint16_t* rp = reinterpret_cast<uint16_t*>(buf + row * kRopeRow);
    RawRow x;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int j = 8 * (i >> 1) + 2 * c + (i & 1);
      x.lo[i] = bf16_f32(rp[pair_lo(j, P)]);
      x.hi[i] = bf16_f32(rp[pair_hi(j, P)]);
    }
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      x.rest[2 * i] = bf16_lo(rest[rr][i]);
      x.rest[2 * i + 1] = bf16_hi(rest[rr][i]);
    }
    const float rinv = raw_rinv(x, row < rows ? eps : 1.0f);  // zeros past them: not 0 inf
    float dot = 0.f;
    float yl[6], yh[6], yr[20];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int j = 8 * (i >> 1) + 2 * c + (i & 1);
      const float2 cs = rot[row * kMaxPairs + j];
      const float u = acc[2 * (i >> 1)][2 * rr + (i & 1)] * f[rr];
      const float v = acc[2 * (i >> 1) + 1][2 * rr + (i & 1)] * f[rr];
      const float al = u * cs.x + v * cs.y, ah = v * cs.x - u * cs.y;
      x.lo[i] *= rinv;
      x.hi[i] *= rinv;
      dws[i] += al * x.lo[i];
      dws[6 + i] += ah * x.hi[i];
      yl[i] = al * __ldg(w + pair_lo(j, P));
      yh[i] = ah * __ldg(w + pair_hi(j, P));
      dot += yl[i] * x.lo[i] + yh[i] * x.hi[i];
    }
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const float2 ww = __ldg(reinterpret_cast<const float2*>(w + rest_dim(2 * i, c)));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 2 * i + e;
        const float al = acc[6 + i][2 * rr + e] * f[rr];
        x.rest[k] *= rinv;
        dws[12 + k] += al * x.rest[k];
        yr[k] = al * (e ? ww.y : ww.x);
        dot += yr[k] * x.rest[k];
      }
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    const float mean = dot * (1.0f / kHeadDim);
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int j = 8 * (i >> 1) + 2 * c + (i & 1);
      const uint32_t y = pack_bf16x2(rinv * (yl[i] - x.lo[i] * mean),
                                     rinv * (yh[i] - x.hi[i] * mean));
      rp[pair_lo(j, P)] = static_cast<uint16_t>(y);
      rp[pair_hi(j, P)] = static_cast<uint16_t>(y >> 16);
    }
    if (row < rows) {
      uint32_t o[10];
#pragma unroll
      for (int i = 0; i < 10; ++i)
        o[i] = pack_bf16x2(rinv * (yr[2 * i] - x.rest[2 * i] * mean),
                           rinv * (yr[2 * i + 1] - x.rest[2 * i + 1] * mean));
      uint16_t* p = dst + row * stride;
      *reinterpret_cast<uint2*>(p + 48 + 4 * c) = make_uint2(o[0], o[1]);
      *reinterpret_cast<uint4*>(p + 64 + 8 * c) = make_uint4(o[2], o[3], o[4], o[5]);
      *reinterpret_cast<uint4*>(p + 96 + 8 * c) = make_uint4(o[6], o[7], o[8], o[9]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int x = lane + 32 * i, row = x / 6, ch = x - 6 * row;
    if (row < rows)
      *reinterpret_cast<uint4*>(dst + row * stride + 8 * ch) =
          *reinterpret_cast<const uint4*>(buf + row * kRopeRow + 16 * ch);
  }
  __syncwarp();  // the buffer may take the next rows
  // Sums over the fragment's rows: the eight lanes of one c each end up with four
  // of the 32 values (a lane hands over the half that its partner keeps).
  float h16[16], h8[8], h4[4];
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    h16[i] = (b4 ? dws[16 + i] : dws[i]) +
             __shfl_xor_sync(0xffffffffu, b4 ? dws[i] : dws[16 + i], 16);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    h8[i] = (b3 ? h16[8 + i] : h16[i]) +
            __shfl_xor_sync(0xffffffffu, b3 ? h16[i] : h16[8 + i], 8);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h4[i] = (b2 ? h8[4 + i] : h8[i]) + __shfl_xor_sync(0xffffffffu, b2 ? h8[i] : h8[4 + i], 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = (b4 ? 16 : 0) + (b3 ? 8 : 0) + (b2 ? 4 : 0) + i;
    const int p = k < 6 ? k : k - 6, j = 8 * (p >> 1) + 2 * c + (p & 1);
    const int d = k < 6 ? pair_lo(j, P) : (k < 12 ? pair_hi(j, P) : rest_dim(k - 12, c));
    dw[d] += h4[i];
  }
}

// ---------------------------------------------------------- query-major pass

constexpr int kQThreads = 128;
constexpr int kBand = 3 * kSinkTile;  // key rows a tile's queries may see: 192

struct alignas(1024) QSmem {
  uint8_t k[kBand * kRowBytes];
  uint8_t v[kBand * kRowBytes];
  uint8_t ks[kSinkBytes], vs[kSinkBytes];
  float vf[kBand + kMaxSink];  // 2^(amin - a) of each key row
  float dw[4][kHeadDim];
  uint8_t rope[4][kRopeBytes];
  uint64_t full, never;
  int abort;
};

static_assert(sizeof(QSmem) <= 115712, "two CTAs per SM");

enum BwdSite { kSiteBForced = 0xF0, kSiteBFull, kSiteBEmpty, kSiteBTile };

// One CTA per (batch row, KV head, 64 queries), or per part of the head's query heads
// where those are too few for the SMs (sink_head_parts).
__global__ void __launch_bounds__(kQThreads, 2) sink_bwd_q_kernel(const SinkBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  QSmem& sm = *reinterpret_cast<QSmem*>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3, P = a.half_rot;
  const int part = static_cast<int>(blockIdx.x % a.head_parts);
  const long long unit = blockIdx.x / a.head_parts;
  const int tile = static_cast<int>(unit % a.tiles);
  const long long chain = unit / a.tiles;
  const int b = static_cast<int>(chain / a.Hkv), kvh = static_cast<int>(chain % a.Hkv);
  const int h0 = a.G * part / a.head_parts, h1 = a.G * (part + 1) / a.head_parts;
  const int t0 = tile * kSinkTile;
  const int s0 = max(0, t0 - kWindow);      // first key row in shared memory
  const int shift = s0 - (t0 - kWindow);    // rows of the band before the sequence
  if (tid == 0) {
    mbar_init(&sm.full, 1);
    mbar_init(&sm.never, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < 4 * kHeadDim; i += kQThreads) (&sm.dw[0][0])[i] = 0.f;
  __syncthreads();
  pdl_start();
  const bool sinks = a.n_sink > 0 && t0 >= kWindow;
  if (tid == 0) {
    const uint32_t n = static_cast<uint32_t>(t0 + kSinkTile - s0) * kRowBytes;
    mbar_arrive_expect_tx(&sm.full, 2 * n + (sinks ? 2 * kSinkBytes : 0));
    const long long at = (chain * a.Tp + s0) * kRowBytes;
    bulk_load(sm.k + shift * kRowBytes, a.kr + at, n, &sm.full);
    bulk_load(sm.v + shift * kRowBytes, a.vr + at, n, &sm.full);
    if (sinks) {
      bulk_load(sm.ks, a.kr + chain * a.Tp * kRowBytes, kSinkBytes, &sm.full);
      bulk_load(sm.vs, a.vr + chain * a.Tp * kRowBytes, kSinkBytes, &sm.full);
    }
  }
  // the least exponent of the keys at hand, and each key's distance from it
  float am = kNoScale;
  for (int i = lane; i < kBand; i += 32)
    if (i >= shift) am = fminf(am, a.va[chain * a.Tp + t0 - kWindow + i]);
  if (sinks && lane < kMaxSink && lane < a.n_sink) am = fminf(am, a.va[chain * a.Tp + lane]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = fminf(am, __shfl_xor_sync(0xffffffffu, am, o));
  for (int i = tid; i < kBand + kMaxSink; i += kQThreads) {
    float e = am;
    if (i < kBand && i >= shift) e = a.va[chain * a.Tp + t0 - kWindow + i];
    if (i >= kBand && sinks) e = a.va[chain * a.Tp + i - kBand];
    sm.vf[i] = key_factor(am, e, 0.0f);
  }
  if (tid == 0 && part == 0) a.amin[chain * a.tiles + tile] = am;
  const float cq = pow2_ceil(warp_absmax(a.wq, lane)), ck = pow2_ceil(warp_absmax(a.wk, lane));
  const float sc = a.scale_log2 * cq * ck;
  volatile int* abort = &sm.abort;
  __syncthreads();
  bool ok = true;
  if (a.flags & SWA_FLAG_FORCE_TIMEOUT) ok = mbar_wait(&sm.never, 0, abort, a.err, kSiteBForced);
  ok = __all_sync(0xffffffffu, ok && mbar_wait(&sm.full, 0, abort, a.err, kSiteBFull));
  if (!ok) {  // copies in flight land before the CTA ends
    if (tid == 0) mbar_wait_drain(&sm.full, 0);
    __syncthreads();  // the one at the end, for warps whose wait did not run out
    return;
  }

  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  const int i0 = t0 + 16 * w;
  const int lo = max(0, 8 - (i0 >> 4));
  const bool sink = a.n_sink > 0 && i0 >= kWindow;
  const long long stride = static_cast<long long>(a.Hq) * kHeadDim;
  const int rows = min(16, a.T - i0);  // none or fewer past the sequence's end
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const int hq = kvh * a.G + h;
    const long long hrow = (static_cast<long long>(b) * a.Hq + hq) * a.Tp + i0;
    // ---- q' and dA as A fragments: words c of the rows' chunks
    uint32_t qf[8][4], df[8][4];
    float L2[2], fs[2], Dn[2], mid[2];
    const long long raw = ((static_cast<long long>(b) * a.T + min(i0, a.T - 1)) * a.Hq + hq) *
                          kHeadDim;
    rope_fetch(sm.rope[w], a.q + raw, stride, rows, lane);
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const uint8_t* qrow = a.qr + hrow * kRowBytes + 4 * c;
      const uint8_t* drow = a.dr + hrow * kRowBytes + 4 * c;
      const float4 rec = a.row[hrow + r + 8 * rr];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          qf[kk][2 * hf + rr] =
              *reinterpret_cast<const uint32_t*>(qrow + row_off(r + 8 * rr, 2 * kk + hf));
          df[kk][2 * hf + rr] =
              *reinterpret_cast<const uint32_t*>(drow + row_off(r + 8 * rr, 2 * kk + hf));
        }
      L2[rr] = rec.x;
      fs[rr] = -(rec.y + am);
      mid[rr] = scale2(rec.z, rec.y + am);
    }
    // the next head's rows, and this one's raw q for the end, towards L2
    {
      const long long nx =
          (hrow + (h + 1 < h1 ? static_cast<long long>(a.Tp) : 0)) * kRowBytes;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.qr + nx + 128 * lane));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.dr + nx + 128 * lane));
      const int t = min(i0 + (lane >> 1), a.T - 1);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          a.q + ((static_cast<long long>(b) * a.T + t) * a.Hq + hq) * kHeadDim + 64 * (lane & 1)));
    }
    // ---- S and dP of all blocks; P and dP - mid stay in registers (fp16) until D - mid, the
    // sum of their products, is known.  mid is D from the forward's o, as exact as its
    // rounding allows: where a row's probability sits on few keys their dP is near D, and dP
    // itself in fp16 would leave 2^-11 of it in the difference.
    uint32_t pf[10][4], gf[10][4];
    Dn[0] = Dn[1] = 0.f;
#pragma unroll
    for (int x = 0; x < 10; ++x) {
      if (x == 9 ? sink : x >= lo) {
        const uint32_t kt = x == 9 ? smem_u32(sm.ks) : smem_u32(sm.k) + 16 * (w + x) * kRowBytes;
        const uint32_t vt = x == 9 ? smem_u32(sm.vs) : smem_u32(sm.v) + 16 * (w + x) * kRowBytes;
        const float* vf = x == 9 ? sm.vf + kBand : sm.vf + 16 * (w + x);
        float s[2][4], dp[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
          dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.f;
        }
        uint32_t kf[2][4], vg[2][4];
        ldsm_x4(kt + k_lane, kf[0]);
        ldsm_x4(vt + k_lane, vg[0]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if (kk < 7) {
            ldsm_x4((kt + k_lane) ^ ((kk + 1) << 5), kf[(kk + 1) & 1]);
            ldsm_x4((vt + k_lane) ^ ((kk + 1) << 5), vg[(kk + 1) & 1]);
          }
          mma_f16(s[0], qf[kk], kf[kk & 1][0], kf[kk & 1][1]);
          mma_f16(s[1], qf[kk], kf[kk & 1][2], kf[kk & 1][3]);
          mma_f16(dp[0], df[kk], vg[kk & 1][0], vg[kk & 1][1]);
          mma_f16(dp[1], df[kk], vg[kk & 1][2], vg[kk & 1][3]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float2 f2 = *reinterpret_cast<const float2*>(vf + 8 * n + 2 * c);
          float p[4], y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = e >> 1, row = r + 8 * rr, col = 8 * n + 2 * c + (e & 1);
            p[e] = ex2_approx(fmaf(s[n][e], sc, -L2[rr]));
            y[e] = fmaf(dp[n][e], (e & 1) ? f2.y : f2.x, -mid[rr]);
            bool hide = false;
            if (x == 0) hide = col <= row;
            if (x == 8) hide = col > row;
            if (x == 9) hide = col >= a.n_sink || col > i0 + row - kWindow;
            if (hide) p[e] = y[e] = 0.f;
          }
          pf[x][2 * n] = pack_f16x2(p[0], p[1]);
          pf[x][2 * n + 1] = pack_f16x2(p[2], p[3]);
          gf[x][2 * n] = pack_f16x2(y[0], y[1]);
          gf[x][2 * n + 1] = pack_f16x2(y[2], y[3]);
          Dn[0] += p[0] * y[0] + p[1] * y[1];
          Dn[1] += p[2] * y[2] + p[3] * y[3];
        }
      } else {
        pf[x][0] = pf[x][1] = pf[x][2] = pf[x][3] = 0u;
        gf[x][0] = gf[x][1] = gf[x][2] = gf[x][3] = 0u;
      }
    }
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      Dn[rr] += __shfl_xor_sync(0xffffffffu, Dn[rr], 1);
      Dn[rr] += __shfl_xor_sync(0xffffffffu, Dn[rr], 2);
      if (c == 0)
        reinterpret_cast<float2*>(a.row + hrow + r + 8 * rr)[1] = make_float2(Dn[rr] + mid[rr], am);
    }
    // ---- dQ = dS K', dS = P (dP - D)
    float dq[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) dq[n][0] = dq[n][1] = dq[n][2] = dq[n][3] = 0.f;
#pragma unroll
    for (int x = 0; x < 10; ++x) {
      if (!(x == 9 ? sink : x >= lo)) continue;
      const uint32_t kt = x == 9 ? smem_u32(sm.ks) : smem_u32(sm.k) + 16 * (w + x) * kRowBytes;
      uint32_t ds[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&pf[x][i]));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&gf[x][i]));
        ds[i] = pack_f16x2(p.x * (y.x - Dn[i & 1]), p.y * (y.y - Dn[i & 1]));
      }
      uint32_t kf[2][4];
      ldsm_x4_trans(kt + t_lane, kf[0]);
#pragma unroll
      for (int nd = 0; nd < 16; nd += 2) {
        if (nd < 14) ldsm_x4_trans((kt + t_lane) ^ ((nd + 2) << 4), kf[((nd >> 1) + 1) & 1]);
        mma_f16(dq[nd], ds, kf[(nd >> 1) & 1][0], kf[(nd >> 1) & 1][1]);
        mma_f16(dq[nd + 1], ds, kf[(nd >> 1) & 1][2], kf[(nd >> 1) & 1][3]);
      }
    }
    split_scale(dq, a.scale * ck, fs, fs);
    norm_rope_back(dq, fs, sm.rope[w], a.q + raw, a.dq + raw, stride, rows,
                   a.rot + static_cast<long long>(i0) * kMaxPairs, a.wq, sm.dw[w], lane, P, a.eps);
  }
  __syncthreads();
  for (int d = tid; d < kHeadDim; d += kQThreads)
    a.dwq_part[static_cast<long long>(blockIdx.x) * kHeadDim + d] =
        (sm.dw[0][d] + sm.dw[1][d]) + (sm.dw[2][d] + sm.dw[3][d]);
}

// ------------------------------------------------------------ key-major block

// P enters dV as 2^14 P: fp16 then keeps probabilities down to 2^-28 normal.
constexpr float kPUp = 14.0f;

// One block of 16 queries against a warp's 16 keys: P^T and dS^T, added into dv
// and dk.  q' and dA rows of the block start at qt and dt, its row records at
// `row`; fj and D carry 2^-kPUp, and dv 2^kPUp.  hide(key row, query column) masks,
// where `masked` says that any is.
template <typename Hide, typename VFrag>
__device__ __forceinline__ void key_block(float (&dk)[16][4], float (&dv)[16][4],
                                          const uint32_t (&kf)[8][4], VFrag vfrag, uint32_t qt,
                                          uint32_t dt, const float4* row, float sc, float bm,
                                          float am, const float (&fj)[2], uint32_t k_lane,
                                          uint32_t t_lane, int lane, bool masked, Hide hide) {
  const int r = lane >> 2, c = lane & 3;
  float s[2][4], dp[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.f;
  }
  uint32_t qg[2][4], dg[2][4], vg[2][4];  // the next k-step's operands load under this one's
  ldsm_x4(qt + k_lane, qg[0]);
  ldsm_x4(dt + k_lane, dg[0]);
  vfrag(0, vg[0]);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const int x = kk & 1;
    if (kk < 7) {
      ldsm_x4((qt + k_lane) ^ ((kk + 1) << 5), qg[x ^ 1]);
      ldsm_x4((dt + k_lane) ^ ((kk + 1) << 5), dg[x ^ 1]);
      vfrag(kk + 1, vg[x ^ 1]);
    }
    mma_f16(s[0], kf[kk], qg[x][0], qg[x][1]);
    mma_f16(s[1], kf[kk], qg[x][2], qg[x][3]);
    mma_f16(dp[0], vg[x], dg[x][0], dg[x][1]);
    mma_f16(dp[1], vg[x], dg[x][2], dg[x][3]);
  }
  uint32_t pf[4], ds[4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float p[4], y[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * n + 2 * c + e;
      const float4 x = row[col];  // lse log2(e), b, D 2^(b + a) and its a, at least am
      // whole exponents: exact
      const float ei = ex2_approx(bm - x.y + kPUp), Dn = x.z * ex2_approx(am - x.w - kPUp);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int i = 2 * rr + e;
        p[i] = ex2_approx(fmaf(s[n][i], sc, -x.x)) * ei;
        y[i] = p[i] * fmaf(dp[n][i], fj[rr], -Dn);
        if (masked && hide(r + 8 * rr, col)) p[i] = y[i] = 0.f;
      }
    }
    pf[2 * n] = pack_f16x2(p[0], p[1]);
    pf[2 * n + 1] = pack_f16x2(p[2], p[3]);
    ds[2 * n] = pack_f16x2(y[0], y[1]);
    ds[2 * n + 1] = pack_f16x2(y[2], y[3]);
  }
  ldsm_x4_trans(dt + t_lane, dg[0]);
  ldsm_x4_trans(qt + t_lane, qg[0]);
#pragma unroll
  for (int nd = 0; nd < 16; nd += 2) {
    const int x = (nd >> 1) & 1;
    if (nd < 14) {
      ldsm_x4_trans((dt + t_lane) ^ ((nd + 2) << 4), dg[x ^ 1]);
      ldsm_x4_trans((qt + t_lane) ^ ((nd + 2) << 4), qg[x ^ 1]);
    }
    mma_f16(dv[nd], pf, dg[x][0], dg[x][1]);
    mma_f16(dv[nd + 1], pf, dg[x][2], dg[x][3]);
    mma_f16(dk[nd], ds, qg[x][0], qg[x][1]);
    mma_f16(dk[nd + 1], ds, qg[x][2], qg[x][3]);
  }
}

// Least b and a over the rows of tiles [ta, tb) and all heads of the group.
__device__ __forceinline__ void tile_scales(const SinkBwdArgs& a, int b, int kvh, int ta, int tb,
                                            int lane, float* bm, float* am) {
  float x = kNoScale, y = kNoScale;
  const int per = 4 * (tb - ta);
  for (int i = lane; i < per * a.G; i += 32) {
    const int h = i / per, t = i - h * per;
    x = fminf(x, a.bmin[((static_cast<long long>(b) * a.Hq + kvh * a.G + h) * a.Tp >> 4) +
                        4 * ta + t]);
  }
  for (int t = ta + lane; t < tb; t += 32)
    y = fminf(y, a.amin[(static_cast<long long>(b) * a.Hkv + kvh) * a.tiles + t]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x = fminf(x, __shfl_xor_sync(0xffffffffu, x, o));
    y = fminf(y, __shfl_xor_sync(0xffffffffu, y, o));
  }
  *bm = x;
  *am = y;
}

// ---------------------------------------------------------------- sinks' pass

constexpr int kSWarps = 8;
constexpr int kSBlockBytes = 16 * kRowBytes;

struct alignas(1024) SSmem {
  uint8_t ks[kSinkBytes], vs[kSinkBytes];
  uint8_t q[kSWarps][2][kSBlockBytes];  // two blocks in flight per warp
  uint8_t d[kSWarps][2][kSBlockBytes];
  float4 row[kSWarps][2][16];
};
static_assert(sizeof(SSmem) >= kSWarps / 2 * kMaxSink * kHeadDim * 2 * 4, "partial sums");

// One CTA per (batch row, KV head, chunk of a.chunk tokens); its warps take the
// 16-query blocks of all heads in turn and are added up at the end.
__global__ void __launch_bounds__(32 * kSWarps, 1) sink_bwd_sink_kernel(const SinkBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SSmem& sm = *reinterpret_cast<SSmem*>(smem_raw);
  pdl_start();
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  const long long chain = blockIdx.x / a.chunks;
  const int b = static_cast<int>(chain / a.Hkv), kvh = static_cast<int>(chain % a.Hkv);
  const int ta = chunk * a.chunk, tb = min(a.Tp, ta + a.chunk);
  for (int i = tid; i < 2 * kSinkBytes / 16; i += 32 * kSWarps) {
    const int at = i & (kSinkBytes / 16 - 1);
    const uint8_t* src = (i < kSinkBytes / 16 ? a.kr : a.vr) + chain * a.Tp * kRowBytes;
    *reinterpret_cast<uint4*>((i < kSinkBytes / 16 ? sm.ks : sm.vs) + 16 * at) =
        *reinterpret_cast<const uint4*>(src + 16 * at);
  }
  float bm, am;
  tile_scales(a, b, kvh, ta / kSinkTile, tb / kSinkTile, lane, &bm, &am);
  const float cq = pow2_ceil(warp_absmax(a.wq, lane)), ck = pow2_ceil(warp_absmax(a.wk, lane));
  const float sc = a.scale_log2 * cq * ck;
  __syncthreads();
  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  uint32_t kf[8][4];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) ldsm_x4((smem_u32(sm.ks) + t_lane) ^ (kk << 5), kf[kk]);
  const uint32_t va = smem_u32(sm.vs) + t_lane;
  auto vfrag = [&](int kk, uint32_t (&f)[4]) { ldsm_x4(va ^ (kk << 5), f); };
  float fj[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) fj[rr] = key_factor(am, a.va[chain * a.Tp + r + 8 * rr], kPUp);
  float dk[16][4], dv[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    dk[n][0] = dk[n][1] = dk[n][2] = dk[n][3] = 0.f;
    dv[n][0] = dv[n][1] = dv[n][2] = dv[n][3] = 0.f;
  }
  const int first = max(ta, kWindow);  // queries that see a sink outside their window
  const int per = max(0, (tb - first) >> 4), total = per * a.G;
  auto fetch = [&](int u, int buf) {
    if (u < total) {
      const int h = u / per, i0 = first + 16 * (u - h * per);
      const long long at =
          (static_cast<long long>(b) * a.Hq + kvh * a.G + h) * a.Tp + i0;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int o = 16 * (lane + 32 * it);
        cp_async16(smem_u32(sm.q[w][buf]) + o, a.qr + at * kRowBytes + o, true);
        cp_async16(smem_u32(sm.d[w][buf]) + o, a.dr + at * kRowBytes + o, true);
      }
      if (lane < 16) cp_async16(smem_u32(&sm.row[w][buf][lane]), a.row + at + lane, true);
    }
    cp_async_commit();
  };
  fetch(w, 0);
  int buf = 0;
#pragma unroll 1
  for (int u = w; u < total; u += kSWarps, buf ^= 1) {
    fetch(u + kSWarps, buf ^ 1);
    cp_async_wait<1>();
    __syncwarp();
    const int i0 = first + 16 * (u % per);
    key_block(dk, dv, kf, vfrag, smem_u32(sm.q[w][buf]), smem_u32(sm.d[w][buf]), sm.row[w][buf], sc,
              bm, am, fj, k_lane, t_lane, lane, true, [&](int key, int col) {
                return key >= a.n_sink || key > i0 + col - kWindow;
              });
    __syncwarp();
  }
  cp_async_wait<0>();
  // the eight warps' sums, in a fixed order: four halves in shared memory, added up
  // by the warps that wrote none, then by one of them
  float* part = reinterpret_cast<float*>(smem_raw);
  constexpr int kN = kMaxSink * kHeadDim;
  const float xk[2] = {-(bm + am), -(bm + am)}, fv = scale2(1.0f, -bm - kPUp);
  float fk[2];
  split_scale(dk, a.scale * cq, xk, fk);
#pragma unroll 1
  for (int half = kSWarps / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (w >= half && w < 2 * half) {
      float* p = part + (w - half) * 2 * kN;
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int at = (r + 8 * rr) * kHeadDim + 8 * n + 2 * (lane & 3);
          *reinterpret_cast<float2*>(p + at) = make_float2(dk[n][2 * rr], dk[n][2 * rr + 1]);
          *reinterpret_cast<float2*>(p + kN + at) = make_float2(dv[n][2 * rr], dv[n][2 * rr + 1]);
        }
    }
    __syncthreads();
    if (w < half) {
      const float* p = part + w * 2 * kN;
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int at = (r + 8 * rr) * kHeadDim + 8 * n + 2 * (lane & 3);
          const float2 x = *reinterpret_cast<const float2*>(p + at);
          const float2 y = *reinterpret_cast<const float2*>(p + kN + at);
          dk[n][2 * rr] += x.x;
          dk[n][2 * rr + 1] += x.y;
          dv[n][2 * rr] += y.x;
          dv[n][2 * rr + 1] += y.y;
        }
    }
  }
  if (w == 0) {
    float* out = a.sink_part + static_cast<long long>(blockIdx.x) * 2 * kN;
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int at = (r + 8 * rr) * kHeadDim + 8 * n + 2 * (lane & 3);
        *reinterpret_cast<float2*>(out + at) =
            make_float2(dk[n][2 * rr] * fk[rr], dk[n][2 * rr + 1] * fk[rr]);
        *reinterpret_cast<float2*>(out + kN + at) =
            make_float2(dv[n][2 * rr] * fv, dv[n][2 * rr + 1] * fv);
      }
  }
}

__global__ void __launch_bounds__(256) sink_bwd_sum_kernel(const SinkBwdArgs a) {
  pdl_start();
  constexpr int kN = 2 * kMaxSink * kHeadDim;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<long long>(a.B) * a.Hkv * kN) return;
  const long long chain = i / kN;
  const int e = static_cast<int>(i - chain * kN);
  float s = 0.f;
#pragma unroll 8
  for (int c = 0; c < a.chunks; ++c) s += a.sink_part[(chain * a.chunks + c) * kN + e];
  a.sink_sum[i] = s;
}

// ------------------------------------------------------------ key-major pass

constexpr int kKThreads = 128;
constexpr int kKStages = 5;
constexpr int kStageRows = 32;
constexpr int kStageBytes = kStageRows * kRowBytes;

struct alignas(1024) KSmem {
  uint8_t v[kTileBytes];
  uint8_t q[kKStages][kStageBytes];
  uint8_t d[kKStages][kStageBytes];
  float4 row[kKStages][kStageRows];
  float dw[4][kHeadDim];
  uint8_t rope[4][kRopeBytes];
  uint64_t full[kKStages], empty[kKStages], tile, never;
  int abort;
};
static_assert(sizeof(KSmem) <= 115712, "two CTAs per SM");

// One CTA per (batch row, KV head, 64 keys), a warp per 16 keys.  The rows of the
// 192 queries that may see them stream through a ring of stages, 32 queries of one
// head at a time, by bulk copies that one lane issues.
__global__ void __launch_bounds__(kKThreads, 2) sink_bwd_k_kernel(const SinkBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  KSmem& sm = *reinterpret_cast<KSmem*>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int tile = static_cast<int>(blockIdx.x % a.tiles);
  const long long chain = blockIdx.x / a.tiles;
  const int b = static_cast<int>(chain / a.Hkv), kvh = static_cast<int>(chain % a.Hkv);
  const int t0 = tile * kSinkTile;
  const int steps = (min(a.Tp, t0 + kBand) - t0) / kStageRows;  // stages per head
  const int total = steps * a.G;
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 4);
    }
    mbar_init(&sm.tile, 1);
    mbar_init(&sm.never, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < 4 * kHeadDim; i += kKThreads) (&sm.dw[0][0])[i] = 0.f;
  __syncthreads();
  pdl_start();
  volatile int* abort = &sm.abort;
  auto issue = [&](int i) {  // stage i: head i / steps, queries t0 + 32 (i % steps) ..
    const int h = i / steps, s = i % kKStages;
    const long long at = (static_cast<long long>(b) * a.Hq + kvh * a.G + h) * a.Tp + t0 +
                         kStageRows * (i - h * steps);
    mbar_arrive_expect_tx(&sm.full[s], 2 * kStageBytes + kStageRows * 16);
    bulk_load(sm.q[s], a.qr + at * kRowBytes, kStageBytes, &sm.full[s]);
    bulk_load(sm.d[s], a.dr + at * kRowBytes, kStageBytes, &sm.full[s]);
    bulk_load(sm.row[s], a.row + at, kStageRows * 16, &sm.full[s]);
  };
  int issued = 0;
  if (tid == 0) {
    // K' passes through the last stage's q' buffer on its way to registers
    mbar_arrive_expect_tx(&sm.tile, 2 * kTileBytes);
    const long long at = (chain * a.Tp + t0) * kRowBytes;
    bulk_load(sm.v, a.vr + at, kTileBytes, &sm.tile);
    bulk_load(sm.q[kKStages - 2], a.kr + at, kTileBytes, &sm.tile);
    for (; issued < min(total, kKStages - 2); ++issued) issue(issued);
  }
  float bm, am;
  tile_scales(a, b, kvh, tile, min(a.tiles, tile + 3), lane, &bm, &am);
  const float cq = pow2_ceil(warp_absmax(a.wq, lane)), ck = pow2_ceil(warp_absmax(a.wk, lane));
  const float sc = a.scale_log2 * cq * ck;
  const int j0 = t0 + 16 * w;
  float fj[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr)
    fj[rr] = key_factor(am, a.va[chain * a.Tp + j0 + r + 8 * rr], kPUp);
  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  bool ok = true;
  if (a.flags & SWA_FLAG_FORCE_TIMEOUT) ok = mbar_wait(&sm.never, 0, abort, a.err, kSiteBForced);
  ok = __all_sync(0xffffffffu, ok && mbar_wait(&sm.tile, 0, abort, a.err, kSiteBTile));
  uint32_t kf[8][4];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    ldsm_x4((smem_u32(sm.q[kKStages - 2]) + 16 * w * kRowBytes + t_lane) ^ (kk << 5), kf[kk]);
  __syncthreads();
  if (tid == 0 && ok)
    for (; issued < min(total, kKStages); ++issued) issue(issued);
  const uint32_t va = smem_u32(sm.v) + 16 * w * kRowBytes + t_lane;
  auto vfrag = [&](int kk, uint32_t (&f)[4]) { ldsm_x4(va ^ (kk << 5), f); };
  float dk[16][4], dv[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    dk[n][0] = dk[n][1] = dk[n][2] = dk[n][3] = 0.f;
    dv[n][0] = dv[n][1] = dv[n][2] = dv[n][3] = 0.f;
  }
#pragma unroll 1
  for (int i = 0; ok && i < total; ++i) {
    const int s = i % kKStages;
    ok = __all_sync(0xffffffffu,
                    mbar_wait(&sm.full[s], (i / kKStages) & 1, abort, a.err, kSiteBFull));
    if (!ok) break;
    const int q0 = kStageRows * (i % steps);  // of the stage's first query, from t0
#pragma unroll 1
    for (int x = 0; x < kStageRows / 16; ++x) {
      const int dist = (q0 >> 4) + x - w;  // blocks from this warp's keys to the queries
      if (dist < 0 || dist > 8) continue;
      key_block(dk, dv, kf, vfrag, smem_u32(sm.q[s]) + 16 * x * kRowBytes,
                smem_u32(sm.d[s]) + 16 * x * kRowBytes, sm.row[s] + 16 * x, sc, bm, am, fj, k_lane,
                t_lane, lane, dist == 0 || dist == 8, [&](int key, int col) {
                  return (dist == 0 && col < key) || (dist == 8 && col >= key);
                });
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[s]);
    if (tid == 0 && issued < total) {  // refill the stage this CTA left last
      if (mbar_wait(&sm.empty[issued % kKStages], ((issued / kKStages) - 1) & 1, abort, a.err,
                    kSiteBEmpty)) {
        issue(issued);
        ++issued;
      }
    }
    __syncwarp();
  }
  if (!ok) {  // copies in flight land before the CTA ends
    if (tid == 0) {
      mbar_wait_drain(&sm.tile, 0);
      for (int s = 0; s < kKStages; ++s) {
        const int n = (issued - s + kKStages - 1) / kKStages;
        if (n > 0) mbar_wait_drain(&sm.full[s], (n - 1) & 1);
      }
    }
    __syncthreads();  // the one at the end, for warps whose waits did not run out
    return;
  }
  const long long raw = ((static_cast<long long>(b) * a.T + min(j0, a.T - 1)) * a.Hkv + kvh) *
                        kHeadDim;
  const long long stride = static_cast<long long>(a.Hkv) * kHeadDim;
  const int rows = min(16, a.T - j0);
  rope_fetch(sm.rope[w], a.k + raw, stride, rows, lane);
  // ---- true scale; the sinks' sums from the queries beyond the window
  const float xk[2] = {-(bm + am), -(bm + am)}, fv = scale2(1.0f, -bm - kPUp);
  float fk[2];
  split_scale(dk, a.scale * cq, xk, fk);
  const bool add = a.n_sink > 0 && tile == 0 && w == 0;
  const float* sk = a.sink_sum + chain * 2 * kMaxSink * kHeadDim;
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      float2 x = make_float2(0.f, 0.f), y = x;
      if (add) {
        const int at = (r + 8 * rr) * kHeadDim + 8 * n + 2 * c;
        x = *reinterpret_cast<const float2*>(sk + at);
        y = *reinterpret_cast<const float2*>(sk + kMaxSink * kHeadDim + at);
      }
      dk[n][2 * rr] = fmaf(dk[n][2 * rr], fk[rr], x.x);
      dk[n][2 * rr + 1] = fmaf(dk[n][2 * rr + 1], fk[rr], x.y);
      dv[n][2 * rr] = fmaf(dv[n][2 * rr], fv, y.x);
      dv[n][2 * rr + 1] = fmaf(dv[n][2 * rr + 1], fv, y.y);
    }
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int t = j0 + r + 8 * rr;
    const long long at = ((static_cast<long long>(b) * a.T + t) * a.Hkv + kvh) * kHeadDim;
    if (t < a.T)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        *reinterpret_cast<uint4*>(a.dv + at + 32 * m + 8 * c) =
            make_uint4(pack_bf16x2(dv[4 * m][2 * rr], dv[4 * m][2 * rr + 1]),
                       pack_bf16x2(dv[4 * m + 1][2 * rr], dv[4 * m + 1][2 * rr + 1]),
                       pack_bf16x2(dv[4 * m + 2][2 * rr], dv[4 * m + 2][2 * rr + 1]),
                       pack_bf16x2(dv[4 * m + 3][2 * rr], dv[4 * m + 3][2 * rr + 1]));
  }
  const float one[2] = {1.0f, 1.0f};
  norm_rope_back(dk, one, sm.rope[w], a.k + raw, a.dk + raw, stride, rows,
                 a.rot + static_cast<long long>(j0) * kMaxPairs, a.wk, sm.dw[w], lane, a.half_rot,
                 a.eps);
  __syncthreads();
  for (int d = tid; d < kHeadDim; d += kKThreads)
    a.dwk_part[static_cast<long long>(blockIdx.x) * kHeadDim + d] =
        (sm.dw[0][d] + sm.dw[1][d]) + (sm.dw[2][d] + sm.dw[3][d]);
}

// dwq (blockIdx.y 0) and dwk (1): 16 dims per block, 64 slices of the CTAs' partial
// sums each, then the slices in order.
__global__ void __launch_bounds__(1024) sink_bwd_w_kernel(const SinkBwdArgs a) {
  __shared__ float part[64][17];
  pdl_start();
  const int d = threadIdx.x & 15, s = threadIdx.x >> 4, dim = 16 * blockIdx.x + d;
  const float* src = blockIdx.y == 0 ? a.dwq_part : a.dwk_part;
  const long long n = static_cast<long long>(a.B) * a.Hkv * a.tiles *
                      (blockIdx.y == 0 ? a.head_parts : 1);
  float x = 0.f;
#pragma unroll 8
  for (long long i = s; i < n; i += 64) x += src[i * kHeadDim + dim];
  part[s][d] = x;
  __syncthreads();
  if (s == 0) {
    float y = 0.f;
    for (int i = 0; i < 64; ++i) y += part[i][d];
    float* out = blockIdx.y == 0 ? a.dwq : a.dwk;
    out[dim] += y;
  }
}

}  // namespace snk

int launch_sink_bwd(const SinkBwdArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  static std::atomic<int> configured[64];  // per device
  if (!configured[di.device].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(snk::sink_bwd_q_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(sizeof(snk::QSmem)));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(snk::sink_bwd_sink_kernel,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(sizeof(snk::SSmem)));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(snk::sink_bwd_k_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(sizeof(snk::KSmem)));
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long tokens = static_cast<long long>(a.B) * a.Tp;
  const long long tiles = static_cast<long long>(a.B) * a.Hkv * a.tiles;
  const long long chains = static_cast<long long>(a.B) * a.Hkv;
  const long long row_warps = tokens / 16 * a.Hq;
  if (row_warps / 8 > 0x7fffffffLL || tokens / 8 > 0x7fffffffLL ||
      tiles * a.head_parts > 0x7fffffffLL || chains * 16 > 0x7fffffffLL ||
      chains * a.chunks > 0x7fffffffLL)
    return SWA_ERR_UNSUPPORTED;
  const auto grid = [](long long n) { return static_cast<unsigned>(n); };
  rc = launch_dependent(snk::sink_bwd_kv_kernel, grid((tokens + 7) / 8), 256, 0, stream, a);
  if (rc == SWA_OK)
    rc = launch_dependent(snk::sink_bwd_rows_kernel, grid((row_warps + 7) / 8), 256, 0, stream, a);
  if (rc == SWA_OK)
    rc = launch_dependent(snk::sink_bwd_q_kernel, grid(tiles * a.head_parts), snk::kQThreads,
                          sizeof(snk::QSmem), stream, a);
  if (rc == SWA_OK && a.n_sink > 0) {
    rc = launch_dependent(snk::sink_bwd_sink_kernel, grid(chains * a.chunks), 32 * snk::kSWarps,
                          sizeof(snk::SSmem), stream, a);
    if (rc == SWA_OK)
      rc = launch_dependent(snk::sink_bwd_sum_kernel, grid(chains * 16), 256, 0, stream, a);
  }
  if (rc == SWA_OK)
    rc = launch_dependent(snk::sink_bwd_k_kernel, grid(tiles), snk::kKThreads, sizeof(snk::KSmem),
                          stream, a);
  if (rc != SWA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kHeadDim / 16, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return map_cuda_error(cudaLaunchKernelEx(&cfg, snk::sink_bwd_w_kernel, a));
}

}  // namespace swa
