// sink_bwd.cu -- backward of the gated sliding-window attention with sink
// tokens, for sm_100a.
//
// With s = sigmoid(g), A the attention output before the gate, P_ij the
// probabilities and x . y a sum over the 128 dims:
//   dg_i  = dO_i A_i s (1 - s) = dO_i o_i (1 - s)
//   dA_i  = dO_i s,      D_i = dA_i . A_i = dO_i . o_i
//   P_ij  = exp(scale q'_i . k'_j - lse_i),   dP_ij = dA_i . v_j
//   dS_ij = P_ij (dP_ij - D_i)
//   dq'_i = scale sum_j dS_ij k'_j,  dk'_j = scale sum_i dS_ij q'_i,
//   dv_j  = sum_i P_ij dA_i
// and from dx' (x = q or k) back through RoPE and the norm, with u = x / rms:
//   du = w RoPE^-1(dx'),  dx = (du - u mean(du u)) / rms,  dw = sum RoPE^-1(dx') u.
// o is the forward's bf16 output: it gives dg and D without a second P V.
//
// Kernels, each waiting for the one before it on the stream:
//   sink_bwd_kv_kernel    k' and v as fp16 operand rows; the table of rotations.
//   sink_bwd_q_kernel     query-major: 16 queries of one head per warp step, nine
//                         band blocks and the sinks: S, dP, dQ.  Writes dq, dg and
//                         the operand rows q' and dA for the next two.
//   sink_bwd_sink_kernel  the sinks' dk' and dv: every query contributes to the same
//                         16 keys, so chunks of 512 tokens make partial sums, and
//   sink_bwd_sum_kernel   adds them up in a fixed order.
//   sink_bwd_k_kernel     key-major: 16 keys per warp against the nine blocks of
//                         queries that see them, all heads of the group: S^T, dP^T,
//                         dV, dK.  Adds the sinks' sums to the keys that are sinks.
//   sink_bwd_w_kernel     adds up the CTAs' dwq and dwk in a fixed order.
// No sum is made by atomics, so results do not depend on the order of CTAs.
//
// What bounds it: the seven products of 160 keys per query on mma.sync (see
// sink_fwd.cu on why not tcgen05), 39 us each for 16,384 tokens of 32 heads at
// 550 TFLOP/s, with as many shared-memory cycles for their operands; memory
// needs about 0.19 ms.  The two passes instead of one with atomics cost two
// products; a band keeps dK and dV of 192 keys live, too many for registers.
//
// Numbers.  All products have fp16 operands and fp32 sums.  q' and k' are divided
// by a power of two not below the norm weights (at most sqrt(128) then); a row
// of dA is scaled by 2^b and one of v by 2^a so that its largest entry lies in
// [1, 2): gradients and values of any magnitude keep fp16's 2^-12 rounding.  The
// scales leave a product where its row or column index carries them; where an
// index is summed over, the least exponent of the rows at hand takes their place,
// and only entries far below the largest lose bits.  |dS| 2^(a + b) <= 1024.
#include <atomic>

#include "launch.cuh"
#include "sink_common.cuh"

namespace swa {
namespace snk {

constexpr float kNoScale = 100.0f;  // exponent of an all-zero row: takes part in no minimum

// Exponent that brings m into [1, 2), within what two fp32 factors carry.
__device__ __forceinline__ float scale_exp(float m) {
  if (!(m > 0.0f)) return kNoScale;
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 255u) - 127;
  return static_cast<float>(max(-100, min(100, -e)));
}
// 2^x for a whole x in [-126, 127]
__device__ __forceinline__ float pow2i(float x) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<int>(x) + 127) << 23);
}
// v 2^x for whole x in [-252, 254], in two steps
__device__ __forceinline__ float scale2(float v, float x) {
  const float h = truncf(0.5f * x);
  return v * pow2i(h) * pow2i(x - h);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
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

// ------------------------------------------------------------- operand rows

// One warp per token: its rotation, and k' and v of every KV head.
__global__ void __launch_bounds__(256) sink_bwd_kv_kernel(const SinkBwdArgs a) {
  pdl_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = static_cast<long long>(blockIdx.x) * 8 + warp;
  if (gw >= static_cast<long long>(a.B) * a.Tp) return;
  const int b = static_cast<int>(gw / a.Tp), t = static_cast<int>(gw - static_cast<long long>(b) * a.Tp);
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
  for (int h = 0; h < a.Hkv; ++h) {
    const long long src = ((static_cast<long long>(b) * a.T + t) * a.Hkv + h) * kHeadDim;
    const long long dst = (static_cast<long long>(b) * a.Hkv + h) * a.Tp + t;
    const KRow x = load_k_row(real ? a.k + src : nullptr, lane, dlo, dhi);
    // row index t & 7 selects the chunk swizzle; the row itself starts at dst
    store_k_row(a.kr + (dst - (t & 7)) * kRowBytes, t & 7, x, lane, w_lo, w_hi, w_rest, rot, a.eps);
    uint2 vv = make_uint2(0u, 0u);
    if (real) vv = __ldg(reinterpret_cast<const uint2*>(a.v + src + 4 * lane));
    const float v0 = bf16_lo(vv.x), v1 = bf16_hi(vv.x), v2 = bf16_lo(vv.y), v3 = bf16_hi(vv.y);
    float m = fmaxf(fmaxf(fabsf(v0), fabsf(v1)), fmaxf(fabsf(v2), fabsf(v3)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float e = scale_exp(m), f = pow2i(e);
    // dims 4 lane .. + 3 = 32 m + 8 c + 2 q (q = 0 or 2): words q and q + 1
    const int md = lane >> 3, c = (lane & 7) >> 1, q = 2 * (lane & 1);
    uint8_t* row = a.vr + (dst - (t & 7)) * kRowBytes;
    *reinterpret_cast<uint32_t*>(row + row_off(t & 7, 4 * md + q) + 4 * c) =
        pack_f16x2(v0 * f, v1 * f);
    *reinterpret_cast<uint32_t*>(row + row_off(t & 7, 4 * md + q + 1) + 4 * c) =
        pack_f16x2(v2 * f, v3 * f);
    if (lane == 0) a.va[dst] = e;
  }
}

// ------------------------------------------- back through RoPE and the norm

// The raw row of x that a fragment's thread c covers: pairs 8 kk + 2 c + e and
// dims 48 + 4 c .., 64 + 8 c .., 96 + 8 c ...
struct RawRow {
  float lo[6], hi[6], rest[20];
};
__device__ __forceinline__ void load_raw(RawRow& x, const uint16_t* row, int c, int P) {
  if (row == nullptr) {
#pragma unroll
    for (int i = 0; i < 6; ++i) x.lo[i] = x.hi[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 20; ++i) x.rest[i] = 0.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int j = 8 * (i >> 1) + 2 * c + (i & 1);
    x.lo[i] = bf16_f32(__ldg(row + pair_lo(j, P)));
    x.hi[i] = bf16_f32(__ldg(row + pair_hi(j, P)));
  }
  const uint2 r3 = __ldg(reinterpret_cast<const uint2*>(row + 48 + 4 * c));
  const uint4 r4 = __ldg(reinterpret_cast<const uint4*>(row + 64 + 8 * c));
  const uint4 r6 = __ldg(reinterpret_cast<const uint4*>(row + 96 + 8 * c));
  const uint32_t w[10] = {r3.x, r3.y, r4.x, r4.y, r4.z, r4.w, r6.x, r6.y, r6.z, r6.w};
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    x.rest[2 * i] = bf16_lo(w[i]);
    x.rest[2 * i + 1] = bf16_hi(w[i]);
  }
}
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

// dx of the two rows (r, r + 8) of a fragment whose accumulators hold dx' in rope
// order times a factor undone by `f`; dw gets the rows' share by dim (one warp's
// own shared array).  A null row writes nothing.
__device__ __forceinline__ void norm_rope_back(const float (&acc)[16][4], const float (&f)[2],
                                               const uint16_t* const (&src)[2],
                                               uint16_t* const (&dst)[2],
                                               const float2* const (&rot)[2], const float* w,
                                               float* dw, int lane, int P, float eps) {
  const int c = lane & 3;
  float dwl[6], dwh[6], dwr[20];
#pragma unroll
  for (int i = 0; i < 6; ++i) dwl[i] = dwh[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 20; ++i) dwr[i] = 0.f;
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    RawRow x;
    load_raw(x, src[rr], c, P);
    const float rinv = raw_rinv(x, eps);
    float dot = 0.f;
    float yl[6], yh[6], yr[20];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int j = 8 * (i >> 1) + 2 * c + (i & 1);
      const float2 cs = rot[rr] != nullptr ? __ldg(rot[rr] + j) : make_float2(1.f, 0.f);
      const float u = acc[2 * (i >> 1)][2 * rr + (i & 1)] * f[rr];
      const float v = acc[2 * (i >> 1) + 1][2 * rr + (i & 1)] * f[rr];
      const float al = u * cs.x + v * cs.y, ah = v * cs.x - u * cs.y;
      x.lo[i] *= rinv;
      x.hi[i] *= rinv;
      dwl[i] += al * x.lo[i];
      dwh[i] += ah * x.hi[i];
      yl[i] = al * __ldg(w + pair_lo(j, P));
      yh[i] = ah * __ldg(w + pair_hi(j, P));
      dot += yl[i] * x.lo[i] + yh[i] * x.hi[i];
    }
#pragma unroll
    for (int i = 0; i < 20; ++i) {
      const float al = acc[6 + (i >> 1)][2 * rr + (i & 1)] * f[rr];
      x.rest[i] *= rinv;
      dwr[i] += al * x.rest[i];
      yr[i] = al * __ldg(w + rest_dim(i, c));
      dot += yr[i] * x.rest[i];
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    const float mean = dot * (1.0f / kHeadDim);
    if (dst[rr] != nullptr) {
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const int j = 8 * (i >> 1) + 2 * c + (i & 1);
        *reinterpret_cast<__nv_bfloat16*>(dst[rr] + pair_lo(j, P)) =
            __float2bfloat16_rn(rinv * (yl[i] - x.lo[i] * mean));
        *reinterpret_cast<__nv_bfloat16*>(dst[rr] + pair_hi(j, P)) =
            __float2bfloat16_rn(rinv * (yh[i] - x.hi[i] * mean));
      }
      uint32_t o[10];
#pragma unroll
      for (int i = 0; i < 10; ++i)
        o[i] = pack_bf16x2(rinv * (yr[2 * i] - x.rest[2 * i] * mean),
                           rinv * (yr[2 * i + 1] - x.rest[2 * i + 1] * mean));
      *reinterpret_cast<uint2*>(dst[rr] + 48 + 4 * c) = make_uint2(o[0], o[1]);
      *reinterpret_cast<uint4*>(dst[rr] + 64 + 8 * c) = make_uint4(o[2], o[3], o[4], o[5]);
      *reinterpret_cast<uint4*>(dst[rr] + 96 + 8 * c) = make_uint4(o[6], o[7], o[8], o[9]);
    }
  }
  // sums over the fragment's rows: lanes of one c
  auto add = [&](float x, int d) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    if (lane < 4) dw[d] += x;
  };
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int j = 8 * (i >> 1) + 2 * c + (i & 1);
    add(dwl[i], pair_lo(j, P));
    add(dwh[i], pair_hi(j, P));
  }
#pragma unroll
  for (int i = 0; i < 20; ++i) add(dwr[i], rest_dim(i, c));
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
  uint64_t full;
  int abort;
};

enum BwdSite { kSiteBQ = 0xF0, kSiteBFull, kSiteBEmpty, kSiteBTile };

__global__ void __launch_bounds__(kQThreads, 2) sink_bwd_q_kernel(const SinkBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  QSmem& sm = *reinterpret_cast<QSmem*>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3, P = a.half_rot;
  const int tile = static_cast<int>(blockIdx.x % a.tiles);
  const long long chain = blockIdx.x / a.tiles;
  const int b = static_cast<int>(chain / a.Hkv), kvh = static_cast<int>(chain % a.Hkv);
  const int t0 = tile * kSinkTile;
  const int s0 = max(0, t0 - kWindow);      // first key row in shared memory
  const int shift = s0 - (t0 - kWindow);    // rows of the band before the sequence
  if (tid == 0) {
    mbar_init(&sm.full, 1);
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
    sm.vf[i] = pow2i(fmaxf(fminf(am - e, 0.0f), -126.0f));
  }
  if (tid == 0) a.amin[chain * a.tiles + tile] = am;
  const float cq = pow2_ceil(warp_absmax(a.wq, lane)), ck = pow2_ceil(warp_absmax(a.wk, lane));
  const float icq = 1.0f / cq, sc = a.scale_log2 * cq * ck;
  volatile int* abort = &sm.abort;
  __syncthreads();
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.full, 0, abort, a.err, kSiteBFull));
  if (!ok) return;

  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  const int i0 = t0 + 16 * w;
  const int lo = max(0, 8 - (i0 >> 4));
  const bool sink = a.n_sink > 0 && i0 >= kWindow;
  const float2* rot[2];
  bool real[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int t = i0 + r + 8 * rr;
    real[rr] = t < a.T;
    rot[rr] = a.rot + static_cast<long long>(t) * kMaxPairs;
  }
#pragma unroll 1
  for (int h = 0; h < a.G; ++h) {
    const int hq = kvh * a.G + h;
    const long long hrow = (static_cast<long long>(b) * a.Hq + hq) * a.Tp;
    uint32_t qf[8][4], df[8][4];
    float L2[2], Dn[2], fs[2], bexp[2];
    const uint16_t* qsrc[2];
    uint16_t* qdst[2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int t = i0 + r + 8 * rr;
      const long long at = ((static_cast<long long>(b) * a.T + t) * a.Hq + hq) * kHeadDim;
      qsrc[rr] = real[rr] ? a.q + at : nullptr;
      qdst[rr] = real[rr] ? a.dq + at : nullptr;
      // ---- q'
      {
        RawRow x;
        load_raw(x, qsrc[rr], c, P);
        const float rinv = raw_rinv(x, a.eps) * icq;
#pragma unroll
        for (int kk = 0; kk < 3; ++kk) {
          float ul[2], uh[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * kk + 2 * c + e;
            const float2 cs = __ldg(rot[rr] + j);
            const float u = x.lo[2 * kk + e] * rinv * __ldg(a.wq + pair_lo(j, P));
            const float v = x.hi[2 * kk + e] * rinv * __ldg(a.wq + pair_hi(j, P));
            ul[e] = u * cs.x - v * cs.y;
            uh[e] = v * cs.x + u * cs.y;
          }
          qf[kk][rr] = pack_f16x2(ul[0], ul[1]);
          qf[kk][2 + rr] = pack_f16x2(uh[0], uh[1]);
        }
#pragma unroll
        for (int i = 0; i < 10; ++i)
          qf[3 + (i >> 1)][2 * (i & 1) + rr] =
              pack_f16x2(x.rest[2 * i] * rinv * __ldg(a.wq + rest_dim(2 * i, c)),
                         x.rest[2 * i + 1] * rinv * __ldg(a.wq + rest_dim(2 * i + 1, c)));
      }
      // ---- dg, dA, D
      {
        float da[32];
        float D = 0.f, m = 0.f;
#pragma unroll
        for (int md = 0; md < 4; ++md) {
          uint4 g4 = make_uint4(0u, 0u, 0u, 0u), d4 = g4, o4 = g4;
          if (real[rr]) {
            g4 = __ldg(reinterpret_cast<const uint4*>(a.g + at + 32 * md + 8 * c));
            d4 = __ldg(reinterpret_cast<const uint4*>(a.dO + at + 32 * md + 8 * c));
            o4 = __ldg(reinterpret_cast<const uint4*>(a.o + at + 32 * md + 8 * c));
          }
          const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, dw4[4] = {d4.x, d4.y, d4.z, d4.w},
                         ow[4] = {o4.x, o4.y, o4.z, o4.w};
          uint32_t y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 gx = make_float2(bf16_lo(gw[x]), bf16_hi(gw[x]));
            const float2 dx = make_float2(bf16_lo(dw4[x]), bf16_hi(dw4[x]));
            const float2 ox = make_float2(bf16_lo(ow[x]), bf16_hi(ow[x]));
            const float2 s = sigmoid2(gx), n = sigmoid2(make_float2(-gx.x, -gx.y));
            const float2 p = __fmul2_rn(dx, ox), t2 = __fmul2_rn(p, n), u = __fmul2_rn(dx, s);
            D += p.x + p.y;
            y[x] = pack_bf16x2(t2.x, t2.y);
            da[8 * md + 2 * x] = u.x;
            da[8 * md + 2 * x + 1] = u.y;
            m = fmaxf(m, fmaxf(fabsf(u.x), fabsf(u.y)));
          }
          if (real[rr])
            *reinterpret_cast<uint4*>(a.dg + at + 32 * md + 8 * c) =
                make_uint4(y[0], y[1], y[2], y[3]);
        }
        D += __shfl_xor_sync(0xffffffffu, D, 1);
        D += __shfl_xor_sync(0xffffffffu, D, 2);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float be = scale_exp(m), f = pow2i(be);
#pragma unroll
        for (int md = 0; md < 4; ++md)
#pragma unroll
          for (int x = 0; x < 4; ++x)  // word x of the group: k-step 2 md + x / 2, half x & 1
            df[2 * md + (x >> 1)][2 * (x & 1) + rr] =
                pack_f16x2(da[8 * md + 2 * x] * f, da[8 * md + 2 * x + 1] * f);
        const float l2 =
            real[rr] ? __ldg(a.lse + (static_cast<long long>(b) * a.Hq + hq) * a.T + t) *
                           1.4426950408889634f
                     : 0.0f;
        bexp[rr] = be;
        L2[rr] = l2;
        const float Db = D * f;
        Dn[rr] = Db * pow2i(am);
        fs[rr] = scale2(a.scale * ck, -(be + am));
        if (c == 0) a.row[hrow + t] = make_float4(l2, Db, be, 0.f);
      }
      // ---- the operand rows of the key-major passes
      uint8_t* qrow = a.qr + (hrow + t - (t & 7)) * kRowBytes;
      uint8_t* drow = a.dr + (hrow + t - (t & 7)) * kRowBytes;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          *reinterpret_cast<uint32_t*>(qrow + row_off(t & 7, 2 * kk + hf) + 4 * c) =
              qf[kk][2 * hf + rr];
          *reinterpret_cast<uint32_t*>(drow + row_off(t & 7, 2 * kk + hf) + 4 * c) =
              df[kk][2 * hf + rr];
        }
    }
    {
      float bm = fminf(bexp[0], bexp[1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) bm = fminf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
      if (lane == 0) a.bmin[(hrow + i0) >> 4] = bm;
    }
    // ---- the blocks: S, dP, dS, dQ
    float dq[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) dq[n][0] = dq[n][1] = dq[n][2] = dq[n][3] = 0.f;
#pragma unroll 1
    for (int x = lo; x < (sink ? 10 : 9); ++x) {
      const uint32_t kt = x == 9 ? smem_u32(sm.ks) : smem_u32(sm.k) + 16 * (w + x) * kRowBytes;
      const uint32_t vt = x == 9 ? smem_u32(sm.vs) : smem_u32(sm.v) + 16 * (w + x) * kRowBytes;
      const float* vf = x == 9 ? sm.vf + kBand : sm.vf + 16 * (w + x);
      float s[2][4], dp[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.f;
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t kf[4], vg[4];
        ldsm_x4((kt + k_lane) ^ (kk << 5), kf);
        ldsm_x4((vt + k_lane) ^ (kk << 5), vg);
        mma_f16(s[0], qf[kk], kf[0], kf[1]);
        mma_f16(s[1], qf[kk], kf[2], kf[3]);
        mma_f16(dp[0], df[kk], vg[0], vg[1]);
        mma_f16(dp[1], df[kk], vg[2], vg[3]);
      }
      uint32_t ds[4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 f2 = *reinterpret_cast<const float2*>(vf + 8 * n + 2 * c);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = e >> 1, row = r + 8 * rr, col = 8 * n + 2 * c + (e & 1);
          const float p = ex2_approx(fmaf(s[n][e], sc, -L2[rr]));
          y[e] = p * fmaf(dp[n][e], (e & 1) ? f2.y : f2.x, -Dn[rr]);
          if (x == 0 && col <= row) y[e] = 0.f;
          if (x == 8 && col > row) y[e] = 0.f;
          if (x == 9 && (col >= a.n_sink || col > i0 + row - kWindow)) y[e] = 0.f;
        }
        ds[2 * n] = pack_f16x2(y[0], y[1]);
        ds[2 * n + 1] = pack_f16x2(y[2], y[3]);
      }
#pragma unroll
      for (int nd = 0; nd < 16; nd += 2) {
        uint32_t kf[4];
        ldsm_x4_trans((kt + t_lane) ^ (nd << 4), kf);
        mma_f16(dq[nd], ds, kf[0], kf[1]);
        mma_f16(dq[nd + 1], ds, kf[2], kf[3]);
      }
    }
    norm_rope_back(dq, fs, qsrc, qdst, rot, a.wq, sm.dw[w], lane, P, a.eps);
  }
  __syncthreads();
  for (int d = tid; d < kHeadDim; d += kQThreads)
    a.dwq_part[static_cast<long long>(blockIdx.x) * kHeadDim + d] =
        (sm.dw[0][d] + sm.dw[1][d]) + (sm.dw[2][d] + sm.dw[3][d]);
}

// ------------------------------------------------------------ key-major block

// One block of 16 queries against a warp's 16 keys: P^T and dS^T, added into dv
// and dk.  q' and dA rows of the block start at qt and dt, its row records at
// `row`.  hide(key row, query column) masks.
template <typename Hide, typename VFrag>
__device__ __forceinline__ void key_block(float (&dk)[16][4], float (&dv)[16][4],
                                          const uint32_t (&kf)[8][4], VFrag vfrag, uint32_t qt,
                                          uint32_t dt, const float4* row, float sc, float bm,
                                          float am2, const float (&fj)[2], uint32_t k_lane,
                                          uint32_t t_lane, int lane, Hide hide) {
  const int r = lane >> 2, c = lane & 3;
  float s[2][4], dp[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.f;
  }
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t qg[4], dg[4], vg[4];
    ldsm_x4((qt + k_lane) ^ (kk << 5), qg);
    ldsm_x4((dt + k_lane) ^ (kk << 5), dg);
    vfrag(kk, vg);
    mma_f16(s[0], kf[kk], qg[0], qg[1]);
    mma_f16(s[1], kf[kk], qg[2], qg[3]);
    mma_f16(dp[0], vg, dg[0], dg[1]);
    mma_f16(dp[1], vg, dg[2], dg[3]);
  }
  uint32_t pf[4], ds[4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float p[4], y[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * n + 2 * c + e;
      const float4 x = row[col];  // lse log2(e), D 2^b, b
      const float ei = pow2i(fmaxf(bm - x.z, -126.0f)), Dn = x.y * am2;
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int i = 2 * rr + e;
        float pe = ex2_approx(fmaf(s[n][i], sc, -x.x)) * ei;
        float ye = pe * fmaf(dp[n][i], fj[rr], -Dn);
        if (hide(r + 8 * rr, col)) pe = ye = 0.f;
        p[i] = pe;
        y[i] = ye;
      }
    }
    pf[2 * n] = pack_f16x2(p[0], p[1]);
    pf[2 * n + 1] = pack_f16x2(p[2], p[3]);
    ds[2 * n] = pack_f16x2(y[0], y[1]);
    ds[2 * n + 1] = pack_f16x2(y[2], y[3]);
  }
#pragma unroll
  for (int nd = 0; nd < 16; nd += 2) {
    uint32_t dg[4], qg[4];
    ldsm_x4_trans((dt + t_lane) ^ (nd << 4), dg);
    ldsm_x4_trans((qt + t_lane) ^ (nd << 4), qg);
    mma_f16(dv[nd], pf, dg[0], dg[1]);
    mma_f16(dv[nd + 1], pf, dg[2], dg[3]);
    mma_f16(dk[nd], ds, qg[0], qg[1]);
    mma_f16(dk[nd + 1], ds, qg[2], qg[3]);
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

// One CTA per (batch row, KV head, chunk of kSinkChunk tokens); its warps take the
// 16-query blocks of all heads in turn and are added up at the end.
__global__ void __launch_bounds__(32 * kSWarps, 1) sink_bwd_sink_kernel(const SinkBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SSmem& sm = *reinterpret_cast<SSmem*>(smem_raw);
  pdl_start();
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  const long long chain = blockIdx.x / a.chunks;
  const int b = static_cast<int>(chain / a.Hkv), kvh = static_cast<int>(chain % a.Hkv);
  const int ta = chunk * kSinkChunk, tb = min(a.Tp, ta + kSinkChunk);
  for (int i = tid; i < 2 * kSinkBytes / 16; i += 32 * kSWarps) {
    const int at = i & (kSinkBytes / 16 - 1);
    const uint8_t* src = (i < kSinkBytes / 16 ? a.kr : a.vr) + chain * a.Tp * kRowBytes;
    *reinterpret_cast<uint4*>((i < kSinkBytes / 16 ? sm.ks : sm.vs) + 16 * at) =
        __ldg(reinterpret_cast<const uint4*>(src + 16 * at));
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
  for (int rr = 0; rr < 2; ++rr)
    fj[rr] = pow2i(fmaxf(fminf(am - a.va[chain * a.Tp + r + 8 * rr], 0.0f), -126.0f));
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
              bm, pow2i(am), fj, k_lane, t_lane, lane, [&](int key, int col) {
                return key >= a.n_sink || key > i0 + col - kWindow;
              });
    __syncwarp();
  }
  cp_async_wait<0>();
  // the eight warps' sums, in a fixed order: four halves in shared memory, added up
  // by the warps that wrote none, then by one of them
  float* part = reinterpret_cast<float*>(smem_raw);
  constexpr int kN = kMaxSink * kHeadDim;
  const float fk = scale2(a.scale * cq, -(bm + am)), fv = scale2(1.0f, -bm);
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
            make_float2(dk[n][2 * rr] * fk, dk[n][2 * rr + 1] * fk);
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
  uint64_t full[kKStages], empty[kKStages], tile;
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
    fj[rr] = pow2i(fmaxf(fminf(am - a.va[chain * a.Tp + j0 + r + 8 * rr], 0.0f), -126.0f));
  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.tile, 0, abort, a.err, kSiteBTile));
  uint32_t kf[8][4];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    ldsm_x4((smem_u32(sm.q[kKStages - 2]) + 16 * w * kRowBytes + t_lane) ^ (kk << 5), kf[kk]);
  __syncthreads();
  if (tid == 0 && ok)
    for (; issued < min(total, kKStages); ++issued) issue(issued);
  const uint32_t va = smem_u32(sm.v) + 16 * w * kRowBytes + t_lane;
  auto vfrag = [&](int kk, uint32_t (&f)[4]) { ldsm_x4(va ^ (kk << 5), f); };
  const float am2 = pow2i(am);
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
                smem_u32(sm.d[s]) + 16 * x * kRowBytes, sm.row[s] + 16 * x, sc, bm, am2, fj, k_lane,
                t_lane, lane, [&](int key, int col) {
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
    if (tid == 0)
      for (int s = 0; s < kKStages; ++s) {
        const int n = (issued - s + kKStages - 1) / kKStages;
        if (n > 0) mbar_wait_drain(&sm.full[s], (n - 1) & 1);
      }
    return;
  }
  // ---- true scale; the sinks' sums from the queries beyond the window
  const float fk = scale2(a.scale * cq, -(bm + am)), fv = scale2(1.0f, -bm);
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
      dk[n][2 * rr] = fmaf(dk[n][2 * rr], fk, x.x);
      dk[n][2 * rr + 1] = fmaf(dk[n][2 * rr + 1], fk, x.y);
      dv[n][2 * rr] = fmaf(dv[n][2 * rr], fv, y.x);
      dv[n][2 * rr + 1] = fmaf(dv[n][2 * rr + 1], fv, y.y);
    }
  const uint16_t* ksrc[2];
  uint16_t* kdst[2];
  const float2* rot[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int t = j0 + r + 8 * rr;
    const long long at = ((static_cast<long long>(b) * a.T + t) * a.Hkv + kvh) * kHeadDim;
    ksrc[rr] = t < a.T ? a.k + at : nullptr;
    kdst[rr] = t < a.T ? a.dk + at : nullptr;
    rot[rr] = a.rot + static_cast<long long>(t) * kMaxPairs;
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
  norm_rope_back(dk, one, ksrc, kdst, rot, a.wk, sm.dw[w], lane, a.half_rot, a.eps);
  __syncthreads();
  for (int d = tid; d < kHeadDim; d += kKThreads)
    a.dwk_part[static_cast<long long>(blockIdx.x) * kHeadDim + d] =
        (sm.dw[0][d] + sm.dw[1][d]) + (sm.dw[2][d] + sm.dw[3][d]);
}

// dwq (blockIdx.y 0) and dwk (1): 16 dims per block, 16 slices of the CTAs' partial
// sums each, then the slices in order.
__global__ void __launch_bounds__(256) sink_bwd_w_kernel(const SinkBwdArgs a) {
  __shared__ float part[16][17];
  pdl_start();
  const int d = threadIdx.x & 15, s = threadIdx.x >> 4, dim = 16 * blockIdx.x + d;
  const float* src = blockIdx.y == 0 ? a.dwq_part : a.dwk_part;
  const long long n = static_cast<long long>(a.B) * a.Hkv * a.tiles;
  float x = 0.f;
#pragma unroll 8
  for (long long i = s; i < n; i += 16) x += src[i * kHeadDim + dim];
  part[s][d] = x;
  __syncthreads();
  if (s == 0) {
    float y = 0.f;
    for (int i = 0; i < 16; ++i) y += part[i][d];
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
  if (tokens / 8 > 0x7fffffffLL || tiles > 0x7fffffffLL || chains * 16 > 0x7fffffffLL)
    return SWA_ERR_UNSUPPORTED;
  const auto grid = [](long long n) { return static_cast<unsigned>(n); };
  rc = launch_dependent(snk::sink_bwd_kv_kernel, grid((tokens + 7) / 8), 256, 0, stream, a);
  if (rc == SWA_OK)
    rc = launch_dependent(snk::sink_bwd_q_kernel, grid(tiles), snk::kQThreads, sizeof(snk::QSmem),
                          stream, a);
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
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return map_cuda_error(cudaLaunchKernelEx(&cfg, snk::sink_bwd_w_kernel, a));
}

}  // namespace swa
