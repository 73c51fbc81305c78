// sink_fwd.cu -- forward of the gated sliding-window attention with sink
// tokens, for sm_100a.
//
//   q' = RoPE(RMSNorm(q; wq)),  k' = RoPE(RMSNorm(k; wk))
//   query i sees key j  iff  j <= i and (i - j < W or j < n_sink)
//   O_i = softmax_j(scale q'_i . k'_j) V (*) sigmoid(g_i)
//
// Work.  A tile is 64 tokens of one (batch row, KV head) chain.  A CTA walks a
// contiguous run of tiles and keeps the K' and V of three (192 keys) and of the
// sinks in shared memory; its four warps take 16 tokens each, MH query heads at a
// time (two where the group's head count is even: each K' and V fragment then
// serves two heads, else one).  A warp's keys are nine 16-key blocks, i0-128 ..
// i0+15, and one block of sinks: 160 keys per query for the 128 + n_sink it sees.
//
// Why warp MMAs (m16n8k16).  The path is bound by memory, not by arithmetic
// (28 KiB and 2.4 MFLOP per token of 32 query heads), and a band of 144 keys is
// narrow for tcgen05's 128-row tiles: the dense two-tile band is 1.6 times the
// products, sinks need an operand and TMEM columns of their own, and S, P and O
// travel through TMEM.  Here they stay in registers.  mma.sync runs at 550
// TFLOP/s on this part, 78 us for 16,384 tokens of 32 heads against 72 us of
// memory time.  Two CTAs of four warps with 255 registers a thread share an SM,
// so one's loads, norms and gate run under the other's products.
//
// Numbers.  All products have fp16 operands and fp32 sums.  q' and k' are divided
// by a power of two not below the norm weights, so they are at most sqrt(128).  A V
// row whose largest entry lies in [2^-6, 2^15) is taken as it is; any other is
// scaled by 2^a into [1, 2), and P carries 2^(a_min - a) then.  P is not divided by
// its row sum before the product; it is relative to a reference score per row, the
// row's maximum over the diagonal block, raised (with O and the row sum rescaled)
// when a later P would pass 2^14, so that P keeps fp16's precision.
//
// Values that are not finite.  A masked key has P = 0, but 0 * inf and 0 * NaN
// are NaN in a product of tiles.  A warp whose O is not finite sums it once more
// in scalar code that skips every key with P = 0.
#include <atomic>

#include "launch.cuh"
#include "sink_common.cuh"

namespace swa {
namespace snk {

constexpr int kFwdThreads = 128;
constexpr int kSlots = 3;

struct alignas(1024) FwdSmem {
  uint8_t k[kSlots][kTileBytes];
  uint8_t v[kSlots][kTileBytes];
  uint8_t ks[kSinkBytes], vs[kSinkBytes];
  float2 tab[16][kMaxPairs];               // rot(t w_j), t = 0 .. 15
  float2 base[4][kMaxPairs];               // rot((64 tile + 16 x) w_j) of the current tile
  float va[kSlots * kSinkTile + kMaxSink]; // a of each V row: v 2^a is stored
  int scaled[kSlots + 1];                  // a row of the slot (or a sink) has a != 0
};
static_assert(sizeof(FwdSmem) <= 115712, "two CTAs per SM");

template <int MH>
__global__ void __launch_bounds__(kFwdThreads, 2) sink_fwd_kernel(const SinkFwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int P = a.half_rot;
  const long long u0 = a.total_tiles * blockIdx.x / gridDim.x;
  const int n_tiles = static_cast<int>(a.total_tiles * (blockIdx.x + 1) / gridDim.x - u0);
  for (int i = tid; i < 16 * kMaxPairs; i += kFwdThreads) {
    const int t = i / kMaxPairs, j = i - t * kMaxPairs;
    float2 x = make_float2(1.0f, 0.0f);
    if (j < P) rope_cos_sin(static_cast<double>(t), a.inv_freq[j], &x.x, &x.y);
    sm.tab[t][j] = x;
  }
  pdl_start();
  const float cq = pow2_ceil(warp_absmax(a.wq, lane)), ck = pow2_ceil(warp_absmax(a.wk, lane));
  const float icq = 1.0f / cq, ick = 1.0f / ck;
  const float sc = a.scale_log2 * cq * ck;
  const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t t_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                          (((lane >> 4) ^ (lane & 7)) << 4);
  const int pairs = (a.G + MH - 1) / MH;

  // Rows r0 .. r0 + n - 1 (this warp's) of the tile at token t0 into kt, vt: K'
  // rotated by base and tab, V with its exponents at va.  Returns
  // whether any row is scaled.
  auto load_rows = [&](uint8_t* kt, uint8_t* vt, float* va, int b, int kvh, int t0, int r0, int n,
                       int limit, float2 base) {
    const int dlo = lane < kMaxPairs ? pair_lo(lane, P) : 0;
    const int dhi = lane < kMaxPairs ? pair_hi(lane, P) : 0;
    const float w_lo = __ldg(a.wk + dlo) * ick, w_hi = __ldg(a.wk + dhi) * ick;
    float4 w_rest = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane < 20) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.wk + kRopeDims + 4 * lane));
      w_rest = make_float4(x.x * ick, x.y * ick, x.z * ick, x.w * ick);
    }
    const long long at = ((static_cast<long long>(b) * a.T + t0) * a.Hkv + kvh) * kHeadDim;
    const long long rs = static_cast<long long>(a.Hkv) * kHeadDim;
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {
      KRow x[4];
      uint2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = r0 + i + e;
        x[e] = load_k_row(row < limit ? a.k + at + row * rs : nullptr, lane, dlo, dhi);
        v[e] = row < limit ? __ldg(reinterpret_cast<const uint2*>(a.v + at + row * rs + 4 * lane))
                           : make_uint2(0u, 0u);
      }
      float2 rot[4];
      float m[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rot[e] = make_float2(1.0f, 0.0f);
        if (lane < kMaxPairs) rot[e] = cmul(base, sm.tab[(r0 + i + e) & 15][lane]);
      }
      v_absmax<4>(v, m);
      store_k_rows<4>(kt, r0 + i, x, lane, w_lo, w_hi, w_rest, rot, a.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = r0 + i + e;
        const float ex = v_exp(m[e]);
        store_v_row(vt, row, v[e], lane, pow2i(ex));
        if (lane == 0) va[row] = ex;
        any = any || ex != 0.0f;
      }
    }
    return any;
  };

  int seen = -1;  // chain of the tiles in shared memory
  for (int ut = 0; ut < n_tiles; ++ut) {
    const long long u = u0 + ut;
    const int chain = static_cast<int>(u / a.tiles), t = static_cast<int>(u - static_cast<long long>(chain) * a.tiles);
    const int b = chain / a.Hkv, kvh = chain - b * a.Hkv;
    __syncthreads();  // the tile before is done with its slots
    if (tid < kSlots + 1 && (chain != seen || tid == t % kSlots)) {
      sm.scaled[tid] = 0;
    }
    // this warp's rows of the new tile(s): 16 tokens from 64 tt + 16 w
    __syncthreads();
    for (int tt = chain == seen ? t : max(0, t - 2); tt <= t; ++tt) {
      float2 base = make_float2(1.0f, 0.0f);
      if (lane < P)
        rope_cos_sin(static_cast<double>(tt) * kSinkTile + 16 * w, a.inv_freq[lane], &base.x,
                     &base.y);
      if (tt == t && lane < kMaxPairs) sm.base[w][lane] = base;
      const int s = tt % kSlots;
      if (load_rows(sm.k[s], sm.v[s], sm.va + s * kSinkTile, b, kvh, tt * kSinkTile, 16 * w, 16,
                    min(kSinkTile, a.T - tt * kSinkTile), base) &&
          lane == 0)
        sm.scaled[s] = 1;
    }
    if (a.n_sink > 0 && t >= 2 && (chain != seen || t == 2)) {
      if (load_rows(sm.ks, sm.vs, sm.va + kSlots * kSinkTile, b, kvh, 0, 4 * w, 4,
                    min(a.T, a.n_sink), make_float2(1.0f, 0.0f)) &&
          lane == 0)
        sm.scaled[kSlots] = 1;
    }
    seen = chain;
    __syncthreads();
    const bool sinks = a.n_sink > 0 && t >= 2;
    // Least exponent of the keys at hand; almost always 0 with no row scaled.
    bool scaled = sinks && sm.scaled[kSlots];
    for (int s = 0; s < kSlots; ++s) scaled = scaled || (t >= s && sm.scaled[(t - s) % kSlots]);
    float am = 0.0f;
    if (scaled) {
      am = 100.0f;
      for (int s = 0; s < kSlots; ++s)
        if (t >= s)
          for (int i = lane; i < kSinkTile; i += 32)
            am = fminf(am, sm.va[((t - s) % kSlots) * kSinkTile + i]);
      if (sinks && lane < a.n_sink) am = fminf(am, sm.va[kSlots * kSinkTile + lane]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) am = fminf(am, __shfl_xor_sync(0xffffffffu, am, o));
    }
    // the next tile's K and V towards L2
    if (t + 1 < a.tiles && ut + 1 < n_tiles) {
      const int row = min((t + 1) * kSinkTile + (tid >> 1), a.T - 1);
      const long long at =
          ((static_cast<long long>(b) * a.T + row) * a.Hkv + kvh) * kHeadDim + 64 * (tid & 1);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.k + at));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.v + at));
    }

    const int i0 = t * kSinkTile + 16 * w;
    const int first = a.n_sink > 0 && i0 >= kWindow ? -1 : 0;
    const int kb0 = max(0, (i0 >> 4) - 8), nb = (i0 >> 4) - kb0 + 1;
    const bool edge = i0 >= kWindow;
#pragma unroll 1
    for (int hp = 0; hp < pairs; ++hp) {
      const int h0 = kvh * a.G + hp * MH;
      long long row[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int tok = i0 + r + 8 * rr;
        row[rr] = tok < a.T ? ((static_cast<long long>(b) * a.T + tok) * a.Hq + h0) * kHeadDim : -1;
      }
      // ---- q' as A fragments; the gate and the next heads' q towards L2
      uint32_t qf[MH][8][4];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float2 rot[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const int j = 8 * (i >> 1) + 2 * c + (i & 1);
          rot[i] = cmul(sm.base[w][j], sm.tab[r + 8 * rr][j]);
        }
#pragma unroll
        for (int h = 0; h < MH; ++h) {
          RawRow x;
          load_raw(x, row[rr] >= 0 ? a.q + row[rr] + h * kHeadDim : nullptr, c, P);
          q_fragment(qf[h], x, rr, a.eps, icq, a.wq, c, P, [&](int i) { return rot[i]; });
        }
      }
      if (i0 + (lane >> 1) < a.T) {
        const long long at =
            ((static_cast<long long>(b) * a.T + i0 + (lane >> 1)) * a.Hq + h0) * kHeadDim +
            64 * (lane & 1);
#pragma unroll
        for (int h = 0; h < MH; ++h) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.g + at + h * kHeadDim));
          if (hp + 1 < pairs)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + at + (MH + h) * kHeadDim));
          else if (i0 + kSinkTile + (lane >> 1) < a.T)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                a.q + at + (static_cast<long long>(kSinkTile) * a.Hq + MH + h - a.G) * kHeadDim));
        }
      }

      float o[MH][16][4], l[MH][2], ms[MH][2];
      // Passes over the blocks: the products (1), and the sum key by key (2, only
      // after an O that is not finite).  One loop body, so that the code stays small.
      int pass = 1;
      while (true) {
#pragma unroll
        for (int h = 0; h < MH; ++h) {
#pragma unroll
          for (int nd = 0; nd < 16; ++nd)
            o[h][nd][0] = o[h][nd][1] = o[h][nd][2] = o[h][nd][3] = 0.f;
          l[h][0] = l[h][1] = 0.f;
        }
#pragma unroll 1
        for (int i = nb - 1; i >= first; --i) {
          const int at = (kb0 + i) % (4 * kSlots);  // block of the ring
          const uint32_t kt =
              i < 0 ? smem_u32(sm.ks) : smem_u32(sm.k) + at * 16 * kRowBytes;
          const uint32_t vt = kt + (i < 0 ? kSinkBytes : kSlots * kTileBytes);
          float s[MH][2][4];
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
          uint32_t kf[2][4];
          ldsm_x4(kt + k_lane, kf[0]);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk < 7) ldsm_x4((kt + k_lane) ^ ((kk + 1) << 5), kf[(kk + 1) & 1]);
#pragma unroll
            for (int h = 0; h < MH; ++h) {
              mma_f16(s[h][0], qf[h][kk], kf[kk & 1][0], kf[kk & 1][1]);
              mma_f16(s[h][1], qf[h][kk], kf[kk & 1][2], kf[kk & 1][3]);
            }
          }
          // masked: the sinks, the block at the window's edge and the diagonal
          if (i < 0 || i == nb - 1 || (i == 0 && edge)) {
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int tok = r + 8 * e2;
              const int lo = i == 0 && edge ? tok + 1 : 0;
              const int hi = i < 0 ? min(a.n_sink - 1, i0 + tok - kWindow) : (i == nb - 1 ? tok : 15);
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int col = 8 * n + 2 * c + e;
#pragma unroll
                  for (int h = 0; h < MH; ++h)
                    if (col < lo || col > hi) s[h][n][2 * e2 + e] = -INFINITY;
                }
            }
          }
          if (i == nb - 1) {  // the row sees at least its own token here
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2) {
                float m = fmaxf(fmaxf(s[h][0][2 * e2], s[h][0][2 * e2 + 1]),
                                fmaxf(s[h][1][2 * e2], s[h][1][2 * e2 + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                ms[h][e2] = m == -INFINITY ? 0.0f : m * sc;  // all NaN: any reference
              }
          }
          float top = 0.0f;
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[h][n][e] = fmaf(s[h][n][e], sc, -ms[h][e >> 1]);
                top = fmaxf(top, s[h][n][e]);
              }
          if (__any_sync(0xffffffffu, top > 14.0f)) {  // raise the references
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2) {
                float m = fmaxf(fmaxf(s[h][0][2 * e2], s[h][0][2 * e2 + 1]),
                                fmaxf(s[h][1][2 * e2], s[h][1][2 * e2 + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2)), 0.0f);
                const float f = ex2_approx(-m);
                ms[h][e2] += m;
                l[h][e2] *= f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  s[h][n][2 * e2] -= m;
                  s[h][n][2 * e2 + 1] -= m;
                }
#pragma unroll
                for (int nd = 0; nd < 16; ++nd) {
                  o[h][nd][2 * e2] *= f;
                  o[h][nd][2 * e2 + 1] *= f;
                }
              }
          }
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[h][n][e] = ex2_approx(s[h][n][e]);
#pragma unroll
          for (int h = 0; h < MH; ++h) {
            l[h][0] += (s[h][0][0] + s[h][0][1]) + (s[h][1][0] + s[h][1][1]);
            l[h][1] += (s[h][0][2] + s[h][0][3]) + (s[h][1][2] + s[h][1][3]);
          }
          if (pass == 1) {
            if (scaled) {
              const float* va = sm.va + (i < 0 ? kSlots * kSinkTile : at * 16);
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float f =
                      pow2i(fmaxf(fminf(am - va[8 * n + 2 * c + e], 0.0f), -126.0f));
#pragma unroll
                  for (int h = 0; h < MH; ++h) {
                    s[h][n][e] *= f;
                    s[h][n][2 + e] *= f;
                  }
                }
            }
            uint32_t pf[MH][4];
#pragma unroll
            for (int h = 0; h < MH; ++h) {
              pf[h][0] = pack_f16x2(s[h][0][0], s[h][0][1]);
              pf[h][1] = pack_f16x2(s[h][0][2], s[h][0][3]);
              pf[h][2] = pack_f16x2(s[h][1][0], s[h][1][1]);
              pf[h][3] = pack_f16x2(s[h][1][2], s[h][1][3]);
            }
            uint32_t vf[2][4];
            ldsm_x4_trans(vt + t_lane, vf[0]);
#pragma unroll
            for (int nd = 0; nd < 16; nd += 2) {
              if (nd < 14) ldsm_x4_trans((vt + t_lane) ^ ((nd + 2) << 4), vf[((nd >> 1) + 1) & 1]);
              const uint32_t(&x)[4] = vf[(nd >> 1) & 1];
#pragma unroll
              for (int h = 0; h < MH; ++h) {
                mma_f16(o[h][nd], pf[h], x[0], x[1]);
                mma_f16(o[h][nd + 1], pf[h], x[2], x[3]);
              }
            }
          } else {
            const int key0 = i < 0 ? 0 : (kb0 + i) * 16;
#pragma unroll
            for (int x = 0; x < 4; ++x) {  // column 8 (x >> 1) + 2 cc + (x & 1)
#pragma unroll 1
              for (int cc = 0; cc < 4; ++cc) {
                const int key = key0 + 8 * (x >> 1) + 2 * cc + (x & 1);
                if (key >= a.T) continue;
                const uint16_t* vr =
                    a.v + ((static_cast<long long>(b) * a.T + key) * a.Hkv + kvh) * kHeadDim;
#pragma unroll
                for (int h = 0; h < MH; ++h)
#pragma unroll
                  for (int e2 = 0; e2 < 2; ++e2) {
                    const float pv = __shfl_sync(0xffffffffu, s[h][x >> 1][2 * e2 + (x & 1)],
                                                 (lane & ~3) | cc);
                    if (pv == 0.0f) continue;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                      const uint4 y = __ldg(reinterpret_cast<const uint4*>(vr + 32 * m + 8 * c));
                      const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                      for (int q4 = 0; q4 < 4; ++q4) {
                        float* ov = &o[h][4 * m + q4][2 * e2];
                        ov[0] = fmaf(pv, bf16_lo(yw[q4]), ov[0]);
                        ov[1] = fmaf(pv, bf16_hi(yw[q4]), ov[1]);
                      }
                    }
                  }
              }
            }
          }
        }
        if (pass == 2) break;
        float2 z = make_float2(0.f, 0.f);
        const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < MH; ++h)
#pragma unroll
          for (int nd = 0; nd < 16; ++nd) {
            z = __ffma2_rn(make_float2(o[h][nd][0], o[h][nd][1]), zero, z);
            z = __ffma2_rn(make_float2(o[h][nd][2], o[h][nd][3]), zero, z);
          }
        if (!__any_sync(0xffffffffu, !(z.x + z.y == 0.0f))) break;
        pass = 2;
      }

      // ---- o = O / l * sigmoid(g)
      const float unscale = pass == 2 ? 1.0f : pow2i(-am);
#pragma unroll
      for (int h = 0; h < MH; ++h)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          uint4 gw[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            gw[m] = row[rr] >= 0 ? __ldg(reinterpret_cast<const uint4*>(
                                       a.g + row[rr] + h * kHeadDim + 32 * m + 8 * c))
                                 : make_uint4(0u, 0u, 0u, 0u);
          float ls = l[h][rr];
          ls += __shfl_xor_sync(0xffffffffu, ls, 1);
          ls += __shfl_xor_sync(0xffffffffu, ls, 2);
          if (a.lse != nullptr && row[rr] >= 0 && c == 0)
            a.lse[(static_cast<long long>(b) * a.Hq + h0 + h) * a.T + i0 + r + 8 * rr] =
                (ms[h][rr] + log2f(ls)) * 0.6931471805599453f;
          const float il = 1.0f / ls * unscale;
          const float2 il2 = make_float2(il, il);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t gx[4] = {gw[m].x, gw[m].y, gw[m].z, gw[m].w};
            uint32_t ow[4];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const float2 sg = sigmoid2(make_float2(bf16_lo(gx[q4]), bf16_hi(gx[q4])));
              const float2 y = __fmul2_rn(
                  __fmul2_rn(make_float2(o[h][4 * m + q4][2 * rr], o[h][4 * m + q4][2 * rr + 1]),
                             il2),
                  sg);
              ow[q4] = pack_bf16x2(y.x, y.y);
            }
            if (row[rr] >= 0)
              *reinterpret_cast<uint4*>(a.o + row[rr] + h * kHeadDim + 32 * m + 8 * c) =
                  make_uint4(ow[0], ow[1], ow[2], ow[3]);
          }
        }
    }
  }
}

template <int MH>
int launch_fwd_impl(const SinkFwdArgs& a, const DeviceInfo& di, cudaStream_t stream) {
  static std::atomic<int> configured[64];  // per device: 0 not yet, 1 ready
  if (!configured[di.device].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(sink_fwd_kernel<MH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(FwdSmem)));
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long most = 2ll * di.num_sms;
  const long long grid = a.total_tiles < most ? a.total_tiles : most;
  return launch_dependent(sink_fwd_kernel<MH>, static_cast<unsigned>(grid), kFwdThreads,
                          sizeof(FwdSmem), stream, a);
}

}  // namespace snk

int launch_sink_fwd(const SinkFwdArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  return a.G % 2 == 0 ? snk::launch_fwd_impl<2>(a, di, stream)
                      : snk::launch_fwd_impl<1>(a, di, stream);
}

}  // namespace swa
