// sink_decode.cu -- one decode step of the gated sliding-window attention with
// sink tokens, and the prefill -> sink cache handoff, for sm_100a.
//
// A sequence keeps a 128-slot ring of its last tokens and a cache of its first
// n_sink tokens' k' and v.  The new token at position p attends over the ring
// (slot s holds position p - ((p - s) mod W), ignored when negative) and over
// the sinks s <= p - W, which have left the ring.  A token with p < n_sink is a
// sink itself and is written to both.
//
// What bounds it: memory.  A unit is one (sequence, KV head): 64 KiB of ring,
// 512 bytes per sink and 2.5 KiB of new rows.  As in the plain decode step a
// persistent CTA streams its units: a producer warp keeps the next ones in
// flight by TMA (128-byte swizzle) and two groups take alternate units.  A group is
// five warps: warp w < 4 attends over slots 32 w .. 32 w + 31, the fifth over the
// sinks, and the five partial results are joined by their maxima and sums.  A unit's
// rows (q, the new k and v, position) land on a barrier of their own, so q' and k'
// are worked out while its rings are still on their way.
//
// Measured, 256 sequences x 32 / 8 heads, 4 sinks, 146 MB a step (20 steps over four
// caches in a graph): 27.7 us, 5.3 TB/s.  Sinks on one of the four ring warps, in
// loops behind the ring's: 31.4 us; inside the ring's loops, where the branch keeps
// loads and products from overlapping, and with two units in flight: 39.5 us.  With
// 16 sinks two units fit: 33.8 us.
//
// Two bf16 terms at no cost.  The tensor core's A operand has 16 rows and a
// group at most eight heads, so rows 0-7 carry the bf16 of q' and rows 8-15
// what that rounding left over, and likewise for P; the two halves of a product
// are added.  q' and P so enter with 16 bits of mantissa, and only the caches'
// own bf16 and the output's rounding remain.
#include <atomic>

#include "decode_internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "rowops.cuh"
#include "sink_internal.h"
#include "warp_mma.cuh"

namespace swa {
namespace snd {

constexpr int kGroups = 2;
constexpr int kGroupWarps = 5;           // four for the ring, one for the sinks
constexpr int kThreads = 32 * (1 + kGroupWarps * kGroups);
constexpr int kMaxStages = 3;
constexpr int kHalf = kWindow * 64 * 2;  // 128 slots x 64 dims (one TMA box)
constexpr int kQStride = 68;             // words per packed q' row
constexpr int kOStride = 136;            // floats per partial-O row

struct Group {
  float scratch[kGroupWarps][kHeadDim];
  float mw[kGroupWarps][kDecMaxGroup], lw[kGroupWarps][kDecMaxGroup];
  uint2 k_row[32], v_row[32];  // the new token's k' and v, four dims each
};
struct Control {
  Group grp[kGroups];
  // rows: q, the new k and v, rotation, position; full: rings, sinks, g
  uint64_t rows[kMaxStages], full[kMaxStages], empty[kMaxStages], never;
  int abort;
};
static_assert(kGroupWarps * kDecMaxGroup * kOStride * 4 <= 2 * kHalf,
              "partial O does not fit the K ring");

// Behind Control, for each group: q' as bf16 pairs, [2 G][kQStride] words (the heads,
// then their remainders).
__host__ __device__ inline int qa_bytes(int G) { return 2 * G * kQStride * 4; }

// A stage: K ring, V ring (two 64-dim halves each), K and V sinks (two halves
// of s8 rows each), q and g rows, the new k and v, the rotation, the position.
struct Stage {
  uint8_t* p;
  int s8, G;
  __device__ uint8_t* k() const { return p; }
  __device__ uint8_t* v() const { return p + 2 * kHalf; }
  __device__ uint8_t* ks() const { return p + 4 * kHalf; }
  __device__ uint8_t* vs() const { return p + 4 * kHalf + s8 * 256; }
  __device__ uint16_t* q() const { return reinterpret_cast<uint16_t*>(p + 4 * kHalf + s8 * 512); }
  __device__ uint16_t* g() const { return q() + G * kHeadDim; }
  __device__ uint16_t* kn() const { return g() + G * kHeadDim; }
  __device__ uint16_t* vn() const { return kn() + kHeadDim; }
  __device__ float2* rot() const { return reinterpret_cast<float2*>(vn() + kHeadDim); }
  __device__ long long* pos() const { return reinterpret_cast<long long*>(rot() + kMaxPairs); }
};
inline int stage_size(int s8, int G) {
  const int n = 4 * kHalf + s8 * 512 + 2 * G * kHeadDim * 2 + 2 * kHeadDim * 2 + kMaxPairs * 8 + 8;
  return (n + 1023) & ~1023;
}

enum Site { kSiteFull = 0xD8, kSiteEmpty, kSiteForced, kSiteRows };

// Byte offset of 16-byte chunk c (0..15) of row s in a [half][row][64] tile with
// 128-byte swizzle; `half` is the bytes of one half.
__device__ __forceinline__ uint32_t tile_off(int s, int c, int half) {
  return static_cast<uint32_t>((c >> 3) * half + s * 128 + (((c & 7) ^ (s & 7)) << 4));
}

// Barrier over a group's 160 threads that also ANDs v across them.
__device__ __forceinline__ bool group_and(bool v, int id) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 160, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return r != 0;
}

// bf16 pair of (x, y) and of what the rounding left over.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}

// One warp's share of a unit: S = q' K^T over NT n-tiles of 8 keys, the softmax of its
// own keys in log2 units (maximum m, sum l of head row grp), and the partial O = P V.
// krow + kstep j is the K row of n-tile j that this lane fetches, vrow its V row.  Keys
// that valid(key) refuses are masked; their V rows are finite.
template <int NT, typename Valid>
__device__ __forceinline__ void attend(uint32_t kbase, uint32_t vbase, int half, int krow,
                                       int kstep, int vrow, const uint32_t* qh, const uint32_t* ql,
                                       bool row_ok, float scale_log2, int lane, Valid&& valid,
                                       float& m, float& l, float (&oacc)[16][4]) {
  const int tig = lane & 3;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
#pragma unroll
  for (int kp2 = 0; kp2 < 4; ++kp2) {
    uint32_t q0[2], q1[2], q2[2], q3[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int kk = 2 * kp2 + e;
      q0[e] = row_ok ? qh[8 * kk] : 0u;
      q1[e] = row_ok ? ql[8 * kk] : 0u;
      q2[e] = row_ok ? qh[8 * kk + 4] : 0u;
      q3[e] = row_ok ? ql[8 * kk + 4] : 0u;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t b[4];
      ldsm_x4(kbase + tile_off(krow + kstep * j, 4 * kp2 + (lane >> 3), half), b);
      mma_16816(acc[j], q0[0], q1[0], q2[0], q3[0], b[0], b[1]);
      mma_16816(acc[j], q0[1], q1[1], q2[1], q3[1], b[2], b[3]);
    }
  }
  m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      acc[j][e] =
          valid(8 * j + 2 * tig + e) ? (acc[j][e] + acc[j][e + 2]) * scale_log2 : -INFINITY;
      m = fmaxf(m, acc[j][e]);
    }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float mu = m == -INFINITY ? 0.0f : m;
  l = 0.0f;
  uint32_t ph[NT], pl[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const float p0 = ex2_approx(acc[j][0] - mu), p1 = ex2_approx(acc[j][1] - mu);
    l += p0 + p1;
    split2(p0, p1, ph[j], pl[j]);
    if (!row_ok) ph[j] = pl[j] = 0u;
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
#pragma unroll
  for (int nd = 0; nd < 16; ++nd)
    oacc[nd][0] = oacc[nd][1] = oacc[nd][2] = oacc[nd][3] = 0.0f;
  if constexpr (NT == 4) {  // lane: V row of keys 0 .. 31, one n-tile of dims at a time
#pragma unroll
    for (int nd = 0; nd < 16; ++nd) {
      uint32_t b[4];
      ldsm_x4_trans(vbase + tile_off(vrow, nd, half), b);
      mma_16816(oacc[nd], ph[0], pl[0], ph[1], pl[1], b[0], b[1]);
      mma_16816(oacc[nd], ph[2], pl[2], ph[3], pl[3], b[2], b[3]);
    }
  } else {  // lane: V row of keys 0 .. 15, two n-tiles of dims at a time
#pragma unroll
    for (int nd = 0; nd < 16; nd += 2) {
      uint32_t b[4];
      ldsm_x4_trans(vbase + tile_off(vrow, nd + (lane >> 4), half), b);
      mma_16816(oacc[nd], ph[0], pl[0], ph[1], pl[1], b[0], b[1]);
      mma_16816(oacc[nd + 1], ph[0], pl[0], ph[1], pl[1], b[2], b[3]);
    }
  }
}

// One unit by one group of five warps.  q' (warps 0-3) and the new k' (warp 4) depend
// on the rows alone, which land first: they are worked out while the rings are still
// on their way.  Then warps 0-3 take 32 ring slots each and warp 4 the sinks.  False
// where a wait ran out.
__device__ __forceinline__ bool process_unit(const Stage& st, Group& gp, uint32_t* qa,
                                             const SinkDecArgs& a, int n, int kvh, int gi, int lw,
                                             int lane, uint64_t* rows, uint64_t* full,
                                             uint32_t phase, volatile int* abort) {
  const int bar_id = 1 + gi;
  if (!group_and(mbar_wait(rows, phase, abort, a.err, kSiteRows), bar_id)) return false;
  const long long p = *st.pos();
  const bool bad = p < 0;  // the same value for the whole group
  if (bad && lw == 0 && lane == 0) atomicCAS(a.err, 0, kDevErrBadPosition);
  const int s0 = static_cast<int>(p & (kWindow - 1));
  // sinks outside the window (0: none, and warp 4 has no part)
  const int seen =
      p - kWindow >= a.n_sink ? a.n_sink : max(0, static_cast<int>(p - kWindow) + 1);
  const int parts = seen > 0 ? 5 : 4;

  float cs = 1.0f, sn = 0.0f;
  if (lane < a.half_rot) {
    const float2 r = st.rot()[lane];
    cs = r.x;
    sn = r.y;
  }
  if (lw < 4) {
    for (int h = lw; h < a.G; h += 4) {
      float x[4];
      load4(st.q() + h * kHeadDim + 4 * lane, x);
      norm_rope_row(x, a.wq, a.eps, gp.scratch[lw], lane, a.half_rot, cs, sn);
      uint32_t hi, lo;
      split2(x[0], x[1], hi, lo);
      qa[h * kQStride + 2 * lane] = hi;
      qa[(a.G + h) * kQStride + 2 * lane] = lo;
      split2(x[2], x[3], hi, lo);
      qa[h * kQStride + 2 * lane + 1] = hi;
      qa[(a.G + h) * kQStride + 2 * lane + 1] = lo;
    }
  } else {
    float x[4];
    load4(st.kn() + 4 * lane, x);
    norm_rope_row(x, a.wk, a.eps, gp.scratch[lw], lane, a.half_rot, cs, sn);
    gp.k_row[lane] = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    gp.v_row[lane] = *reinterpret_cast<const uint2*>(st.vn() + 4 * lane);
  }
  // the rings have landed, and q' and the new row are visible to the group
  if (!group_and(mbar_wait(full, phase, abort, a.err, kSiteFull), bar_id)) return false;
  if (bad) return true;
  // Each warp reads its own slots only, so what it changes there needs no barrier.
  // Slots that hold no token of the sequence may hold anything: their V rows become
  // zeros, since P = 0 does not hide an infinity or a NaN.
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  if (lw < 4) {
    const int s = 32 * lw + lane;
    if (p - ((p - s) & (kWindow - 1)) < 0) {
#pragma unroll
      for (int c = 0; c < 16; ++c) *reinterpret_cast<uint4*>(st.v() + tile_off(s, c, kHalf)) = z;
    }
    if (lw == s0 >> 5) {  // the new token's row, into its slot and the caches
      const uint2 kp = gp.k_row[lane], vp = gp.v_row[lane];
      const uint32_t off = tile_off(s0, lane >> 1, kHalf) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>(st.k() + off) = kp;
      *reinterpret_cast<uint2*>(st.v() + off) = vp;
      const long long unit = static_cast<long long>(n) * a.Hkv + kvh;
      const long long row = (unit * kWindow + s0) * kHeadDim + 4 * lane;
      *reinterpret_cast<uint2*>(a.k_cache + row) = kp;
      *reinterpret_cast<uint2*>(a.v_cache + row) = vp;
      if (p < a.n_sink) {
        const long long srow = (unit * a.n_sink + p) * kHeadDim + 4 * lane;
        *reinterpret_cast<uint2*>(a.k_sink + srow) = kp;
        *reinterpret_cast<uint2*>(a.v_sink + srow) = vp;
      }
    }
  } else if (lane >= seen && lane < a.s8) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      *reinterpret_cast<uint4*>(st.vs() + tile_off(lane, c, a.s8 * 128)) = z;
  }
  __syncwarp();

  const int grp = lane >> 2, tig = lane & 3;
  const bool row_ok = grp < a.G;
  const uint32_t *qh = qa + grp * kQStride + tig, *ql = qh + a.G * kQStride;
  float m = -INFINITY, l = 0.0f, oacc[16][4];
  if (lw < 4) {
    attend<4>(smem_u32(st.k()), smem_u32(st.v()), kHalf, 32 * lw + (lane & 7), 8, 32 * lw + lane,
              qh, ql, row_ok, a.scale_log2, lane,
              [&](int key) { return p - ((p - (32 * lw + key)) & (kWindow - 1)) >= 0; }, m, l,
              oacc);
  } else if (seen > 0) {
    // an 8-row cache has no keys 8 .. 15: rows 0 .. 7 again, masked
    const bool wide = a.s8 == 16;
    attend<2>(smem_u32(st.ks()), smem_u32(st.vs()), a.s8 * 128, lane & 7, wide ? 8 : 0,
              lane & (wide ? 15 : 7), qh, ql, row_ok, a.scale_log2, lane,
              [&](int key) { return key < seen; }, m, l, oacc);
  }
  group_and(true, bar_id);  // every warp is done with the K ring: reuse it
  float* part = reinterpret_cast<float*>(st.k());  // [parts][kDecMaxGroup][kOStride]
  if (row_ok && lw < parts) {
    float* dst = part + (lw * kDecMaxGroup + grp) * kOStride + 2 * tig;
#pragma unroll
    for (int nd = 0; nd < 16; ++nd)
      *reinterpret_cast<float2*>(dst + 8 * nd) =
          make_float2(oacc[nd][0] + oacc[nd][2], oacc[nd][1] + oacc[nd][3]);
    if (tig == 0) {
      gp.mw[lw][grp] = m;
      gp.lw[lw][grp] = l;
    }
  }
  fence_proxy_async_smem();  // this thread's writes before a later copy into the stage
  group_and(true, bar_id);

  // ---- o = (sum_w O_w 2^(m_w - m)) / (sum_w l_w 2^(m_w - m)) * sigmoid(g)
  for (int h = lw; h < a.G; h += kGroupWarps) {
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w)
      if (w < parts) mx = fmaxf(mx, gp.mw[w][h]);
    float lsum = 0.0f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) {
      if (w >= parts) continue;
      const float f = gp.mw[w][h] == -INFINITY ? 0.0f : ex2_approx(gp.mw[w][h] - mx);
      lsum += f * gp.lw[w][h];
      const float4 v4 =
          *reinterpret_cast<const float4*>(part + (w * kDecMaxGroup + h) * kOStride + 4 * lane);
      y[0] += f * v4.x;
      y[1] += f * v4.y;
      y[2] += f * v4.z;
      y[3] += f * v4.w;
    }
    const float inv_l = 1.0f / lsum;
    float gx[4];
    load4(st.g() + h * kHeadDim + 4 * lane, gx);
    float ov[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ov[e] = y[e] * inv_l / (1.0f + __expf(-gx[e]));
    *reinterpret_cast<uint2*>(a.o + (static_cast<long long>(n) * a.Hq + kvh * a.G + h) * kHeadDim +
                              4 * lane) =
        make_uint2(pack_bf16x2(ov[0], ov[1]), pack_bf16x2(ov[2], ov[3]));
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    sink_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_ks,
                       const __grid_constant__ CUtensorMap tm_vs, const SinkDecArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Control& sm = *reinterpret_cast<Control*>(base + a.stages * a.stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long units = static_cast<long long>(a.N) * a.Hkv;
  const long long u0 = units * blockIdx.x / gridDim.x;
  const int n_units = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - u0);

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sm.rows[s], 2);  // the copies' expect_tx arrive + the position
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.never, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort = &sm.abort;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    const uint32_t row_bytes = kHeadDim * 2;
    const uint32_t bytes = 4 * kHalf + a.s8 * 512 + a.G * row_bytes;
    int issued = 0;
    long long seq = -1, p = 0;
    float2 rot = make_float2(1.0f, 0.0f);
    int s = 0, round = 0;
    for (int i = 0; i < n_units; ++i) {
      bool w = true;
      if (lane == 0 && round > 0)
        w = mbar_wait(&sm.empty[s], (round - 1) & 1, abort, a.err, kSiteEmpty);
      if (!__shfl_sync(0xffffffffu, w ? 1 : 0, 0)) break;
      const long long u = u0 + i;
      const int n = static_cast<int>(u / a.Hkv), kvh = static_cast<int>(u - u / a.Hkv * a.Hkv);
      const Stage st{base + s * a.stage_bytes, a.s8, a.G};
      if (lane == 0) {
        uint64_t *rows = &sm.rows[s], *full = &sm.full[s];
        const long long qrow = (static_cast<long long>(n) * a.Hq + kvh * a.G) * kHeadDim;
        const long long kvrow = (static_cast<long long>(n) * a.Hkv + kvh) * kHeadDim;
        mbar_arrive_expect_tx(rows, (a.G + 2) * row_bytes);
        bulk_load(st.q(), a.q + qrow, a.G * row_bytes, rows);
        bulk_load(st.kn(), a.k_new + kvrow, row_bytes, rows);
        bulk_load(st.vn(), a.v_new + kvrow, row_bytes, rows);
        mbar_arrive_expect_tx(full, bytes);
        tma_load_4d(st.k(), &tm_k, full, 0, 0, kvh, n);
        tma_load_4d(st.k() + kHalf, &tm_k, full, 64, 0, kvh, n);
        tma_load_4d(st.v(), &tm_v, full, 0, 0, kvh, n);
        tma_load_4d(st.v() + kHalf, &tm_v, full, 64, 0, kvh, n);
        if (a.s8 > 0) {
          tma_load_4d(st.ks(), &tm_ks, full, 0, 0, kvh, n);
          tma_load_4d(st.ks() + a.s8 * 128, &tm_ks, full, 64, 0, kvh, n);
          tma_load_4d(st.vs(), &tm_vs, full, 0, 0, kvh, n);
          tma_load_4d(st.vs() + a.s8 * 128, &tm_vs, full, 64, 0, kvh, n);
        }
        bulk_load(st.g(), a.g + qrow, a.G * row_bytes, full);
        issued = i + 1;
      }
      if (n != seq) {
        seq = n;
        p = a.pos[n];
        if (lane < a.half_rot)
          rope_cos_sin(static_cast<double>(p), a.inv_freq[lane], &rot.x, &rot.y);
      }
      if (lane == 0) *st.pos() = p;
      if (lane < a.half_rot) st.rot()[lane] = rot;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rows[s]);
      if (++s == a.stages) {
        s = 0;
        ++round;
      }
    }
    // no copy is in flight when the CTA ends, whatever the consumers did
    if (lane == 0) {
      for (int i = max(0, issued - a.stages); i < issued; ++i) {
        mbar_wait_drain(&sm.rows[i % a.stages], (i / a.stages) & 1);
        mbar_wait_drain(&sm.full[i % a.stages], (i / a.stages) & 1);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- consumer group
    const int gi = (warp - 1) / kGroupWarps, lw = (warp - 1) % kGroupWarps;
    uint32_t* qa = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(&sm + 1) +
                                               gi * qa_bytes(a.G));
    bool live = true;
    if (a.flags & SWA_FLAG_FORCE_TIMEOUT)
      live = group_and(mbar_wait(&sm.never, 0, abort, a.err, kSiteForced), 1 + gi);
    for (int i = gi; live && i < n_units; i += kGroups) {
      const int s = i % a.stages;
      const long long u = u0 + i;
      const int n = static_cast<int>(u / a.Hkv), kvh = static_cast<int>(u - u / a.Hkv * a.Hkv);
      if (!process_unit(Stage{base + s * a.stage_bytes, a.s8, a.G}, sm.grp[gi], qa, a, n, kvh, gi,
                        lw, lane, &sm.rows[s], &sm.full[s], (i / a.stages) & 1, abort))
        break;
      group_and(true, 1 + gi);
      if (lw == 0 && lane == 0) mbar_arrive(&sm.empty[s]);
    }
  }
  __syncthreads();
}

// Prefill -> sink caches: one warp per (sequence, sink) writes k' (rounded as a
// decode step rounds it) and v of the token at position s, for every KV head;
// sinks that the sequence's tokens do not reach keep their contents.
__global__ void __launch_bounds__(128) sink_fill_kernel(const SinkFillArgs a) {
  __shared__ __align__(16) float scratch[4][kHeadDim];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = static_cast<long long>(blockIdx.x) * 4 + warp;
  const long long b = gw / a.n_sink;
  const int s = static_cast<int>(gw - b * a.n_sink);
  if (b >= a.B) return;
  long long first = b * a.T, len = a.T, p0 = 0;
  if (a.lens != nullptr) {
    first = a.starts[b];
    len = a.lens[b];
    p0 = a.pos0 != nullptr ? a.pos0[b] : 0;
    if (first < 0 || len < 0 || p0 < 0 || len > a.T || first > a.T - len) {
      if (s == 0 && lane == 0) atomicCAS(a.err, 0, kDevErrBadPosition);
      return;
    }
  }
  if (s < p0 || s - p0 >= len) return;
  float cs = 1.0f, sn = 0.0f;
  if (lane < a.half_rot) rope_cos_sin(static_cast<double>(s), a.inv_freq[lane], &cs, &sn);
  for (int h = 0; h < a.Hkv; ++h) {
    const long long row = ((first + (s - p0)) * a.Hkv + h) * kHeadDim;
    float x[4];
    load4(a.k + row + 4 * lane, x);
    const uint2 vv = *reinterpret_cast<const uint2*>(a.v + row + 4 * lane);
    norm_rope_row(x, a.wk, a.eps, scratch[warp], lane, a.half_rot, cs, sn);
    const long long dst = ((b * a.Hkv + h) * a.n_sink + s) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(a.k_sink + dst) =
        make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    *reinterpret_cast<uint2*>(a.v_sink + dst) = vv;
  }
}

}  // namespace snd

int launch_sink_decode(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tks,
                       const CUtensorMap& tvs, SinkDecArgs a, cudaStream_t stream) {
  DeviceInfo di;
  int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  constexpr int kLimit = 232448;
  const int fixed =
      static_cast<int>(sizeof(snd::Control)) + snd::kGroups * snd::qa_bytes(a.G) + 1024;
  a.stage_bytes = snd::stage_size(a.s8, a.G);
  // Three units in flight where they fit (no sinks, or up to 8 and at most four heads per KV
  // head), else two.
  a.stages = 3 * a.stage_bytes + fixed <= kLimit ? 3 : 2;
  static std::atomic<int> configured[64];
  if (!configured[di.device].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(snd::sink_decode_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kLimit);
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long units = static_cast<long long>(a.N) * a.Hkv;
  const long long grid = units < di.num_sms ? units : di.num_sms;
  return launch_dependent(snd::sink_decode_kernel, static_cast<unsigned>(grid), snd::kThreads,
                          static_cast<size_t>(a.stages) * a.stage_bytes + fixed, stream, tk, tv,
                          tks, tvs, a);
}

int launch_sink_fill(const SinkFillArgs& a, cudaStream_t stream) {
  const long long grid = (static_cast<long long>(a.B) * a.n_sink + 3) / 4;
  if (grid > 0x7fffffffLL) return SWA_ERR_UNSUPPORTED;
  return launch_dependent(snd::sink_fill_kernel, static_cast<unsigned>(grid), 128, 0, stream, a);
}

}  // namespace swa
