// sink_fwd.cu -- forward of the gated sliding-window attention with sink
// tokens, for sm_100a.
//
//   q' = RoPE(RMSNorm(q; wq)),  k' = RoPE(RMSNorm(k; wk))
//   query i sees key j  iff  j <= i and (i - j < W or j < n_sink)
//   O_i = softmax_j(scale q'_i . k'_j) V (*) sigmoid(g_i)
//
// Work.  A tile is 64 tokens of one (batch row, KV head) chain.  A CTA walks a
// contiguous run of tiles; a warp's job is 16 tokens of MH = 1 query head, its
// keys nine 16-key blocks, i0-128 .. i0+15, plus one block of sinks: 160 keys per
// query for the 128 + n_sink it sees.
//
// Why warp MMAs (m16n8k16).  The path is bound by memory, not by arithmetic
// (28 KiB and 2.4 MFLOP per token of 32 query heads), and a band of 144 keys is
// narrow for tcgen05's 128-row tiles: the dense two-tile band is 1.6 times the
// products, sinks need an operand and TMEM columns of their own, and S, P and O
// travel through TMEM.  Here they stay in registers.  mma.sync runs at 550
// TFLOP/s on this part, 78 us for 16,384 tokens of 32 heads against 72 us of
// memory time.
//
// Roles.  Warps 0-3 produce: K rows are normalised, rotated and rounded to fp16,
// V rows copied, into a ring of four tiles (three live, one ahead).  Warps 4-19
// consume, each at its own pace: a slot is free again when all of them have left
// the tile two after it.  Q of a warp's next job arrives in its own buffer by
// cp.async while the current one computes; g is read straight into the layout of
// the product's fragment (see the order of the dims in sink_common.cuh).
//
// Numbers.  q' and k' are fp16 (divided by a power of two not below the norm
// weights, so at most sqrt(128)): 2^-12 relative rounding of the scores' terms,
// an eighth of bf16's.  P is rounded to bf16 because V is used as it is: fp16
// would narrow V's range.  Sums, row sums and O are fp32.  The softmax subtracts
// the bound scale D max|wq| max|wk| instead of a running maximum, where that
// cannot underflow, and each row's maximum (one more pass of scores) where it
// could.
//
// Values that are not finite.  A masked key has P = 0, but 0 * inf and 0 * NaN
// are NaN in a product of tiles.  A job whose O is not finite is therefore
// summed once more in scalar code that skips every key with P = 0.
#include <atomic>
#include <type_traits>

#include "launch.cuh"
#include "sink_common.cuh"

namespace swa {
namespace snk {

constexpr int kFwdThreads = 640;
constexpr int kConsumers = 16;
constexpr int kSlots = 4;
constexpr int kBlocks = 10;  // a job's key blocks: nine of the band, then the sinks
constexpr int kFwdRegsLaunch = 96, kFwdRegsProducer = 56, kFwdRegsConsumer = 104;
static_assert(kFwdRegsProducer + 4 * kFwdRegsConsumer <= 5 * kFwdRegsLaunch, "register split");

struct alignas(1024) FwdSmem {
  uint8_t k[kSlots][kTileBytes];
  uint8_t v[kSlots][kTileBytes];
  uint8_t ks[kSinkBytes], vs[kSinkBytes];
  uint8_t q[kConsumers][16 * kRowBytes];  // each consumer's next Q rows
  float2 tab[kSinkTile][kMaxPairs];           // rot(t w_j), t = 0 .. 63
  float2 base[kSlots][kMaxPairs];             // rot(64 tile w_j) of the tile in each slot
  float wq[kHeadDim];                         // wq / cq in rope order
  uint64_t full[kSlots], empty[kSlots], sink_full, sink_empty, never;
  int abort;
};
static_assert(sizeof(FwdSmem) <= 232448, "shared memory over the 227 KiB per-CTA limit");

enum FwdSite { kSiteSFull = 0xC0, kSiteSEmpty, kSiteSSink, kSiteSSinkEmpty, kSiteSForced };

// Swizzle of a Q buffer row: both the 2-byte reads of eight rows and the 16-byte
// reads of two rows are free of bank conflicts.
__device__ __forceinline__ uint32_t q_off(int row, int chunk) {
  const int f = ((row & 1) << 2) | ((row >> 1) & 3);
  return static_cast<uint32_t>(row * kRowBytes + ((chunk ^ f) << 4));
}

// The walk of a CTA over its tiles.
struct Walk {
  int chain, t;       // (batch row, KV head) and tile of the chain
  int ln;             // index of tile t among the tiles the CTA loads
  __device__ Walk(const SinkFwdArgs& a, long long u0)
      : chain(static_cast<int>(u0 / a.tiles)), t(static_cast<int>(u0 % a.tiles)) {
    ln = min(2, t);
  }
  __device__ void next(const SinkFwdArgs& a) {
    ++ln;
    if (++t == a.tiles) {
      t = 0;
      ++chain;
    }
  }
};

template <int MH>
__device__ __forceinline__ void prefetch_q(const SinkFwdArgs& a, long long u0, int n_tiles, int jpt,
                                           int job, uint32_t buf, int lane) {
  if (job < n_tiles * jpt) {
    const int ut = job / jpt, j = job - ut * jpt;
    const long long u = u0 + ut;
    const int chain = static_cast<int>(u / a.tiles), t = static_cast<int>(u % a.tiles);
    const int b = chain / a.Hkv, kvh = chain - b * a.Hkv;
    const int i0 = t * kSinkTile + (j & 3) * 16, h0 = kvh * a.G + (j >> 2) * MH;
#pragma unroll
    for (int it = 0; it < 8 * MH; ++it) {
      const int row = 2 * (it & 7) + (lane >> 4), h = it >> 3;
      const long long tok = i0 + row;
      const bool real = tok < a.T;
      const uint16_t* src = a.q +
                            ((static_cast<long long>(b) * a.T + (real ? tok : 0)) * a.Hq + h0 + h) *
                                kHeadDim +
                            8 * (lane & 15);
      cp_async16(buf + h * 16 * kRowBytes + q_off(row, lane & 15), src, real);
    }
  }
  cp_async_commit();
}

template <int MH>
__global__ void __launch_bounds__(kFwdThreads, 1) sink_fwd_kernel(const SinkFwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.half_rot;
  const long long u0 = a.total_tiles * blockIdx.x / gridDim.x;
  const int n_tiles = static_cast<int>(a.total_tiles * (blockIdx.x + 1) / gridDim.x - u0);
  const int jpt = 4 * ((a.G + MH - 1) / MH);  // jobs per tile

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], kConsumers);
    }
    mbar_init(&sm.sink_full, 4);
    mbar_init(&sm.sink_empty, kConsumers);
    mbar_init(&sm.never, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < kSinkTile * kMaxPairs; i += kFwdThreads) {
    const int t = i / kMaxPairs, j = i - t * kMaxPairs;
    float2 r = make_float2(1.0f, 0.0f);
    if (j < P) rope_cos_sin(static_cast<double>(t), a.inv_freq[j], &r.x, &r.y);
    sm.tab[t][j] = r;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Bounds of the norm weights: every warp reduces them for itself.
  float wmq = 0.f, wmk = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wmq = fmaxf(wmq, fabsf(a.wq[lane + 32 * i]));
    wmk = fmaxf(wmk, fabsf(a.wk[lane + 32 * i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    wmq = fmaxf(wmq, __shfl_xor_sync(0xffffffffu, wmq, o));
    wmk = fmaxf(wmk, __shfl_xor_sync(0xffffffffu, wmk, o));
  }
  const float cq = pow2_ceil(wmq), ck = pow2_ceil(wmk);
  if (tid < kHeadDim) {  // wq / cq by position
    const int kk = tid >> 4, m = tid & 15;
    int d;
    if (kk < 3) {
      d = m < 8 ? pair_lo(8 * kk + m, P) : pair_hi(8 * kk + m - 8, P);
    } else if (kk == 3) {
      d = 48 + 4 * ((m & 7) >> 1) + 2 * (m >> 3) + (m & 1);
    } else {
      d = 64 + 32 * ((kk - 4) >> 1) + 8 * ((m & 7) >> 1) + 4 * (kk & 1) + 2 * (m >> 3) + (m & 1);
    }
    sm.wq[tid] = a.wq[d] / cq;
  }
  __syncthreads();
  volatile int* abort = &sm.abort;

  if (warp < 4) {
    // ------------------------------------------------------------ producer
    regs_dec<kFwdRegsProducer>();
    const int dlo = lane < kMaxPairs ? pair_lo(lane, P) : 0;
    const int dhi = lane < kMaxPairs ? pair_hi(lane, P) : 0;
    const float ick = 1.0f / ck;
    const float w_lo = a.wk[dlo] * ick, w_hi = a.wk[dhi] * ick;
    float4 w_rest = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane < 20) {
      w_rest = *reinterpret_cast<const float4*>(a.wk + kRopeDims + 4 * lane);
      w_rest = make_float4(w_rest.x * ick, w_rest.y * ick, w_rest.z * ick, w_rest.w * ick);
    }
    // Rows r0 .. r0 + n - 1 (n even) of the tile that starts at token t0.  The raw
    // rows land in the tile by cp.async and are rewritten in place, a row (of V:
    // two) per warp step: all lanes have read it before any writes.
    auto rows = [&](uint8_t* kt, uint8_t* vt, int b, int kvh, int t0, int r0, int n, int limit,
                    float2 base) {
      const int rs = a.Hkv * kHeadDim, ch = lane & 15;
      const long long at = ((static_cast<long long>(b) * a.T + t0) * a.Hkv + kvh) * kHeadDim;
#pragma unroll 1
      for (int i = 0; i < n; i += 2) {
        const int row = r0 + i + (lane >> 4);
        const bool real = row < limit;
        const long long src = at + (real ? static_cast<long long>(row) * rs : 0) + 8 * ch;
        cp_async16(smem_u32(kt) + row_off(row, ch), a.k + src, real);
        cp_async16(smem_u32(vt) + row_off(row, ch), a.v + src, real);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll 2
      for (int i = 0; i < n; ++i) {
        const int row = r0 + i;
        KRow x;
        x.lo = x.hi = 0;
        x.rest = make_uint2(0u, 0u);
        float2 rot = make_float2(1.0f, 0.0f);
        if (lane < kMaxPairs) {
          x.lo = *reinterpret_cast<const uint16_t*>(kt + row_off(row, dlo >> 3) + 2 * (dlo & 7));
          x.hi = *reinterpret_cast<const uint16_t*>(kt + row_off(row, dhi >> 3) + 2 * (dhi & 7));
          rot = cmul(base, sm.tab[row][lane]);
        }
        if (lane < 20)
          x.rest = *reinterpret_cast<const uint2*>(kt + row_off(row, 6 + (lane >> 1)) +
                                                   8 * (lane & 1));
        store_k_row(kt, row, x, lane, w_lo, w_hi, w_rest, rot, a.eps);
      }
#pragma unroll 2
      for (int i = 0; i < n; i += 2) {
        const int row = r0 + i + (lane >> 4);
        const uint4 y = *reinterpret_cast<const uint4*>(vt + row_off(row, ch));
        __syncwarp();
        store_v_chunk(vt, row, ch, y);
      }
    };
    bool ok = true;
    int ln = 0, seg = 0;
    for (long long u = u0; ok && u < u0 + n_tiles; ++seg) {
      const int chain = static_cast<int>(u / a.tiles), t0 = static_cast<int>(u % a.tiles);
      const int t1 = static_cast<int>(min(static_cast<long long>(a.tiles), t0 + (u0 + n_tiles - u)));
      const int b = chain / a.Hkv, kvh = chain - b * a.Hkv;
      const int first = max(0, t0 - 2);
      for (int t = first; ok && t < t1; ++t, ++ln) {
        const int s = ln & (kSlots - 1);
        if (ln >= kSlots)
          ok = __all_sync(0xffffffffu, mbar_wait_inl(&sm.empty[s], ((ln >> 2) - 1) & 1, abort, a.err,
                                                     kSiteSEmpty));
        if (!ok) break;
        float2 base = make_float2(1.0f, 0.0f);
        if (lane < P)
          rope_cos_sin(static_cast<double>(t) * kSinkTile, a.inv_freq[lane], &base.x, &base.y);
        if (warp == 0 && lane < kMaxPairs) sm.base[s][lane] = base;
        const int left = a.T - t * kSinkTile;  // real rows of the tile
        rows(sm.k[s], sm.v[s], b, kvh, t * kSinkTile, 16 * warp, 16, min(left, kSinkTile), base);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
        if (t == first) {  // the chain's sinks, behind its first tile
          if (seg > 0)
            ok = __all_sync(0xffffffffu, mbar_wait_inl(&sm.sink_empty, (seg - 1) & 1, abort, a.err,
                                                       kSiteSSinkEmpty));
          if (!ok) break;
          rows(sm.ks, sm.vs, b, kvh, 0, 4 * warp, 4, min(a.T, a.n_sink), make_float2(1.0f, 0.0f));
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sink_full);
        }
      }
      u += t1 - t0;
    }
  } else {
    // ------------------------------------------------------------ consumers
    regs_inc<kFwdRegsConsumer>();
    const int cw = warp - 4, r = lane >> 2, c = lane & 3;
    const uint32_t qbuf = smem_u32(sm.q[cw]);
    const uint8_t* qp = sm.q[cw];
    const float sc = a.scale_log2 * cq * ck;
    const float bound = a.scale_log2 * kHeadDim * wmq * wmk * (1.0f + 1.0f / 64.0f);
    const bool exact = !(2.0f * bound <= 120.0f);
    // ldmatrix addresses inside a 16-key block: K' rows (keys 0-7, 8-15; two
    // chunks of a k-step) and V rows transposed (two chunks of dims)
    const uint32_t k_lane = (lane & 7) * kRowBytes + (lane >> 4) * 8 * kRowBytes +
                            ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
    const uint32_t v_lane = (lane & 7) * kRowBytes + ((lane >> 3) & 1) * 8 * kRowBytes +
                            (((lane >> 4) ^ (lane & 7)) << 4);
    bool ok = true;
    if (a.flags & SWA_FLAG_FORCE_TIMEOUT)
      ok = __all_sync(0xffffffffu, mbar_wait_inl(&sm.never, 0, abort, a.err, kSiteSForced));
    int job = cw;
    if (ok) prefetch_q<MH>(a, u0, n_tiles, jpt, job, qbuf, lane);
    Walk w(a, u0);
    int seg = 0;
    for (int ut = 0; ok && ut < n_tiles; ++ut) {
      const int b = w.chain / a.Hkv, kvh = w.chain - b * a.Hkv;
      if (ut == 0)  // the tiles before the run's first one
        for (int i = 0; i < w.ln; ++i)
          ok = ok && __all_sync(0xffffffffu,
                                mbar_wait_inl(&sm.full[i], 0, abort, a.err, kSiteSFull));
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inl(&sm.full[w.ln & (kSlots - 1)],
                                                       (w.ln >> 2) & 1, abort, a.err, kSiteSFull));
      if (ok && a.n_sink > 0 && w.t >= 2)
        ok = __all_sync(0xffffffffu,
                        mbar_wait_inl(&sm.sink_full, seg & 1, abort, a.err, kSiteSSink));
      if (!ok) break;

      for (; job < (ut + 1) * jpt; job += kConsumers) {
        const int j = job - ut * jpt;
        const int toff = (j & 3) * 16;
        const int i0 = w.t * kSinkTile + toff, h0 = kvh * a.G + (j >> 2) * MH;

        // ---- Q: normalised, rotated, fp16, as A fragments
        cp_async_wait<0>();
        __syncwarp();
        uint32_t qf[MH][8][4];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int tok = r + 8 * rr;
          float2 rot[6];
#pragma unroll
          for (int kk = 0; kk < 3; ++kk) {
            const int jp = 8 * kk + 2 * c;
            const float4 tb = *reinterpret_cast<const float4*>(&sm.tab[toff + tok][jp]);
            const float4 bs =
                *reinterpret_cast<const float4*>(&sm.base[w.ln & (kSlots - 1)][jp]);
            rot[2 * kk] = cmul(make_float2(bs.x, bs.y), make_float2(tb.x, tb.y));
            rot[2 * kk + 1] = cmul(make_float2(bs.z, bs.w), make_float2(tb.z, tb.w));
          }
#pragma unroll
          for (int h = 0; h < MH; ++h) {
            const uint8_t* qh = qp + h * 16 * kRowBytes;
            float lo[6], hi[6];
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 6; ++i) {
              const int jp = 8 * (i >> 1) + 2 * c + (i & 1);
              const int d0 = pair_lo(jp, P), d1 = pair_hi(jp, P);
              lo[i] = bf16_f32(*reinterpret_cast<const uint16_t*>(qh + q_off(tok, d0 >> 3) +
                                                                  2 * (d0 & 7)));
              hi[i] = bf16_f32(*reinterpret_cast<const uint16_t*>(qh + q_off(tok, d1 >> 3) +
                                                                  2 * (d1 & 7)));
              const float2 f = make_float2(lo[i], hi[i]);
              ss = __ffma2_rn(f, f, ss);
            }
            const uint2 x3 = *reinterpret_cast<const uint2*>(qh + q_off(tok, 6 + (c >> 1)) +
                                                             8 * (c & 1));
            const uint4 x4 = *reinterpret_cast<const uint4*>(qh + q_off(tok, 8 + c));
            const uint4 x6 = *reinterpret_cast<const uint4*>(qh + q_off(tok, 12 + c));
            const uint32_t x[10] = {x3.x, x3.y, x4.x, x4.y, x4.z, x4.w, x6.x, x6.y, x6.z, x6.w};
#pragma unroll
            for (int i = 0; i < 10; ++i) {
              const float2 f = make_float2(bf16_lo(x[i]), bf16_hi(x[i]));
              ss = __ffma2_rn(f, f, ss);
            }
            float s1 = ss.x + ss.y;
            s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
            s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
            const float rinv = rsqrtf(s1 * (1.0f / kHeadDim) + a.eps);
#pragma unroll
            for (int kk = 0; kk < 3; ++kk) {
              const float2 wl = *reinterpret_cast<const float2*>(&sm.wq[16 * kk + 2 * c]);
              const float2 wh = *reinterpret_cast<const float2*>(&sm.wq[16 * kk + 8 + 2 * c]);
              const float u0f = lo[2 * kk] * rinv * wl.x, v0f = hi[2 * kk] * rinv * wh.x;
              const float u1f = lo[2 * kk + 1] * rinv * wl.y, v1f = hi[2 * kk + 1] * rinv * wh.y;
              const float2 c0 = rot[2 * kk], c1 = rot[2 * kk + 1];
              qf[h][kk][rr] = pack_f16x2(u0f * c0.x - v0f * c0.y, u1f * c1.x - v1f * c1.y);
              qf[h][kk][2 + rr] = pack_f16x2(v0f * c0.x + u0f * c0.y, v1f * c1.x + u1f * c1.y);
            }
            const float2 rv = make_float2(rinv, rinv);
#pragma unroll
            for (int i = 0; i < 10; ++i) {
              const int kk = 3 + (i >> 1), hf = i & 1;
              const float2 ww = *reinterpret_cast<const float2*>(&sm.wq[16 * kk + 8 * hf + 2 * c]);
              const float2 y =
                  __fmul2_rn(__fmul2_rn(make_float2(bf16_lo(x[i]), bf16_hi(x[i])), rv), ww);
              qf[h][kk][2 * hf + rr] = pack_f16x2(y.x, y.y);
            }
          }
        }
        __syncwarp();
        prefetch_q<MH>(a, u0, n_tiles, jpt, job + kConsumers, qbuf, lane);
        // the gate's rows towards L2 while the products run
#pragma unroll
        for (int h = 0; h < MH; ++h)
          if (i0 + (lane >> 1) < a.T)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                a.g + ((static_cast<long long>(b) * a.T + i0 + (lane >> 1)) * a.Hq + h0 + h) *
                          kHeadDim + 64 * (lane & 1)));

        // ---- the key blocks: block x < 9 of the band is the 16 rows at ring position
        // (ring + x) mod 16, block 9 the sinks.  A job near the sequence's start lacks
        // the blocks before lo.
        const int ring = 4 * (w.ln - w.t) + (i0 >> 4) - 8;
        const int lo = max(0, 8 - (i0 >> 4));
        const bool sink = a.n_sink > 0 && i0 >= kWindow;
        auto k_block = [&](int x) {
          return x == 9 ? smem_u32(sm.ks) : smem_u32(sm.k) + (((ring + x) & 15) << 12);
        };
        auto v_block = [&](int x) {
          return x == 9 ? smem_u32(sm.vs) : smem_u32(sm.v) + (((ring + x) & 15) << 12);
        };
        // is column col of block x hidden from token row `row` of the job
        auto hidden = [&](int x, int row, int col) {
          if (x == 0) return col <= row;                       // the window's edge
          if (x == 8) return col > row;                        // the diagonal
          if (x == 9) return col >= a.n_sink || col > i0 + row - kWindow;
          return false;
        };
        auto scores = [&](int x, float (&s)[MH][2][4]) {
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
          const uint32_t kt = k_block(x) + k_lane;
          uint32_t kf[2][4];
          ldsm_x4(kt, kf[0]);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk < 7) ldsm_x4(kt ^ ((kk + 1) << 5), kf[(kk + 1) & 1]);
#pragma unroll
            for (int h = 0; h < MH; ++h) {
              mma_f16(s[h][0], qf[h][kk], kf[kk & 1][0], kf[kk & 1][1]);
              mma_f16(s[h][1], qf[h][kk], kf[kk & 1][2], kf[kk & 1][3]);
            }
          }
        };
        float ms[MH][2];  // subtracted from a row's scores
#pragma unroll
        for (int h = 0; h < MH; ++h) ms[h][0] = ms[h][1] = bound;
        if (exact) {  // the row maxima first
#pragma unroll
          for (int h = 0; h < MH; ++h) ms[h][0] = ms[h][1] = -INFINITY;
#pragma unroll 1
          for (int x = lo; x < (sink ? 10 : 9); ++x) {
            float s[MH][2][4];
            scores(x, s);
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!hidden(x, r + 8 * (e >> 1), 8 * n + 2 * c + (e & 1)))
                    ms[h][e >> 1] = fmaxf(ms[h][e >> 1], s[h][n][e]);
          }
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = ms[h][e];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              ms[h][e] = m * sc;
            }
        }
        // The blocks are unrolled: all of P stays in registers (as bf16), q' dies before
        // O begins, and O is made and written 32 dims at a time.
        auto attend = [&](auto all_blocks) {
          constexpr bool kAll = decltype(all_blocks)::value;
          auto have = [&](int x) { return kAll || (x == 9 ? sink : x >= lo); };
          uint32_t pf[kBlocks][MH][4];
          float l[MH][2];
#pragma unroll
          for (int h = 0; h < MH; ++h) l[h][0] = l[h][1] = 0.f;
#pragma unroll
          for (int x = 0; x < kBlocks; ++x) {
            if (have(x)) {
              float s[MH][2][4];
              scores(x, s);
#pragma unroll
              for (int h = 0; h < MH; ++h) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float p = ex2_approx(fmaf(s[h][n][e], sc, -ms[h][e >> 1]));
                    s[h][n][e] = hidden(x, r + 8 * (e >> 1), 8 * n + 2 * c + (e & 1)) ? 0.0f : p;
                  }
                l[h][0] += (s[h][0][0] + s[h][0][1]) + (s[h][1][0] + s[h][1][1]);
                l[h][1] += (s[h][0][2] + s[h][0][3]) + (s[h][1][2] + s[h][1][3]);
                pf[x][h][0] = pack_bf16x2(s[h][0][0], s[h][0][1]);
                pf[x][h][1] = pack_bf16x2(s[h][0][2], s[h][0][3]);
                pf[x][h][2] = pack_bf16x2(s[h][1][0], s[h][1][1]);
                pf[x][h][3] = pack_bf16x2(s[h][1][2], s[h][1][3]);
              }
            } else {
#pragma unroll
              for (int h = 0; h < MH; ++h)
                pf[x][h][0] = pf[x][h][1] = pf[x][h][2] = pf[x][h][3] = 0u;
            }
          }
          float il[MH][2];
          long long row[MH][2];
#pragma unroll
          for (int h = 0; h < MH; ++h)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              const long long tok = i0 + r + 8 * rr;
              const bool real = tok < a.T;
              float ls = l[h][rr];
              ls += __shfl_xor_sync(0xffffffffu, ls, 1);
              ls += __shfl_xor_sync(0xffffffffu, ls, 2);
              if (a.lse != nullptr && real && c == 0)
                a.lse[(static_cast<long long>(b) * a.Hq + h0 + h) * a.T + tok] =
                    (ms[h][rr] + log2f(ls)) * 0.6931471805599453f;
              il[h][rr] = 1.0f / ls;
              row[h][rr] = real ? ((static_cast<long long>(b) * a.T + tok) * a.Hq + h0 + h) *
                                          kHeadDim + 8 * c
                                : -1;
            }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint4 gw[MH][2];
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int rr = 0; rr < 2; ++rr)
                gw[h][rr] = row[h][rr] >= 0
                                ? __ldg(reinterpret_cast<const uint4*>(a.g + row[h][rr] + 32 * m))
                                : make_uint4(0u, 0u, 0u, 0u);
            float o[MH][4][4];
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int n = 0; n < 4; ++n) o[h][n][0] = o[h][n][1] = o[h][n][2] = o[h][n][3] = 0.f;
#pragma unroll
            for (int x = 0; x < kBlocks; ++x) {
              if (!have(x)) continue;
              const uint32_t vt = v_block(x) + v_lane;
              uint32_t vf[2][4];
              ldsm_x4_trans(vt ^ ((4 * m) << 4), vf[0]);
              ldsm_x4_trans(vt ^ ((4 * m + 2) << 4), vf[1]);
#pragma unroll
              for (int h = 0; h < MH; ++h)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                  mma_bf16(o[h][n], pf[x][h], vf[n >> 1][2 * (n & 1)], vf[n >> 1][2 * (n & 1) + 1]);
            }
            // not finite: these dims again, key by key, without the keys of P = 0
            float2 z = make_float2(0.f, 0.f);
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                z = __ffma2_rn(make_float2(o[h][n][0], o[h][n][1]), make_float2(0.f, 0.f), z);
                z = __ffma2_rn(make_float2(o[h][n][2], o[h][n][3]), make_float2(0.f, 0.f), z);
              }
            if (__any_sync(0xffffffffu, !(z.x + z.y == 0.0f))) {
#pragma unroll
              for (int h = 0; h < MH; ++h)
#pragma unroll
                for (int n = 0; n < 4; ++n) o[h][n][0] = o[h][n][1] = o[h][n][2] = o[h][n][3] = 0.f;
#pragma unroll
              for (int x = 0; x < kBlocks; ++x) {
                const int key0 = x == 9 ? 0 : i0 - kWindow + 16 * x;
#pragma unroll 1
                for (int y = 0; y < 16; ++y) {  // column y: thread (y & 7) / 2 of the row holds P
                  const int key = key0 + y;
                  if (!have(x) || key >= a.T) continue;
                  const uint4 vv = __ldg(reinterpret_cast<const uint4*>(
                      a.v + ((static_cast<long long>(b) * a.T + key) * a.Hkv + kvh) * kHeadDim +
                      32 * m + 8 * c));
                  const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                  for (int h = 0; h < MH; ++h)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                      const uint32_t pw = __shfl_sync(
                          0xffffffffu, y < 8 ? pf[x][h][rr] : pf[x][h][2 + rr],
                          (lane & ~3) | ((y & 7) >> 1));
                      const float p = (y & 1) ? bf16_hi(pw) : bf16_lo(pw);
                      if (p != 0.0f) {
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                          o[h][n][2 * rr] = fmaf(p, bf16_lo(vw[n]), o[h][n][2 * rr]);
                          o[h][n][2 * rr + 1] = fmaf(p, bf16_hi(vw[n]), o[h][n][2 * rr + 1]);
                        }
                      }
                    }
                }
              }
            }
            // o = O / l * sigmoid(g)
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
              for (int rr = 0; rr < 2; ++rr) {
                const uint32_t gx[4] = {gw[h][rr].x, gw[h][rr].y, gw[h][rr].z, gw[h][rr].w};
                const float2 il2 = make_float2(il[h][rr], il[h][rr]);
                uint32_t ow[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  const float2 sg = sigmoid2(make_float2(bf16_lo(gx[n]), bf16_hi(gx[n])));
                  const float2 y = __fmul2_rn(
                      __fmul2_rn(make_float2(o[h][n][2 * rr], o[h][n][2 * rr + 1]), il2), sg);
                  ow[n] = pack_bf16x2(y.x, y.y);
                }
                if (row[h][rr] >= 0)
                  *reinterpret_cast<uint4*>(a.o + row[h][rr] + 32 * m) =
                      make_uint4(ow[0], ow[1], ow[2], ow[3]);
              }
          }
        };
        if (lo == 0 && sink) attend(std::true_type{});
        else attend(std::false_type{});
      }
      // ---- leave the tile: the slot two back is free, all of them at a chain's end
      __syncwarp();
      const bool seg_end = w.t == a.tiles - 1 || ut == n_tiles - 1;
      if (lane == 0) {
        if (w.t >= 2) mbar_arrive(&sm.empty[(w.ln - 2) & (kSlots - 1)]);
        if (seg_end) {
          if (w.t >= 1) mbar_arrive(&sm.empty[(w.ln - 1) & (kSlots - 1)]);
          mbar_arrive(&sm.empty[w.ln & (kSlots - 1)]);
          mbar_arrive(&sm.sink_empty);
        }
      }
      if (seg_end) ++seg;
      w.next(a);
    }
    cp_async_wait<0>();  // nothing of this warp's is in flight when the CTA ends
  }
}

template <int MH>
int launch_fwd_impl(const SinkFwdArgs& a, const DeviceInfo& di, cudaStream_t stream) {
  static std::atomic<int> configured[64];  // per device: 0 not yet, 1 ready
  if (!configured[di.device].load(std::memory_order_acquire)) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, sink_fwd_kernel<MH>);
    if (e != cudaSuccess) return map_cuda_error(e);
    if (attr.numRegs != kFwdRegsLaunch) return SWA_ERR_UNSUPPORTED;
    e = cudaFuncSetAttribute(sink_fwd_kernel<MH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(FwdSmem)));
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long grid = a.total_tiles < di.num_sms ? a.total_tiles : di.num_sms;
  return launch_dependent(sink_fwd_kernel<MH>, static_cast<unsigned>(grid), kFwdThreads,
                          sizeof(FwdSmem), stream, a);
}

}  // namespace snk

int launch_sink_fwd(const SinkFwdArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  return snk::launch_fwd_impl<1>(a, di, stream);
}

}  // namespace swa
