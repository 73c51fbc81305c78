// sink_fwd.cu -- forward of the gated sliding-window attention with sink
// tokens, for sm_100a.
//
//   q' = RoPE(RMSNorm(q; wq)),  k' = RoPE(RMSNorm(k; wk))
//   query i sees key j  iff  j <= i and (i - j < W or j < n_sink)
//   O_i = softmax_j(scale q'_i . k'_j) V (*) sigmoid(g_i)
//
// The tile.  M = 128 rows are 64 tokens of two heads (row = 2 token + head), because
// then the keys that a tile can see fit the accumulator: the 64 tokens' own tile
// and the two before it (192 keys) and one block of 16 sinks are N = 208 columns, P
// over their first 104, O in 128 more, two such regions in the 512 columns of TMEM.
// With 128 tokens of one head the band alone is 256 columns.  One N = 208 MMA per
// k-step reads the three K' tiles and the sinks, which lie one after the other in
// shared memory; the products are 208 keys per query for the 128 + n_sink it sees.
// A group with an odd number of heads leaves its last tile's second head unused.
//
// Roles as in the plain forward (fwd.cu): warp 0 loads K and Q, warp 3 V, one thread
// of warp 1 issues the MMAs, and two region warpgroups, a thread per row, take
// alternate head pairs: Q' in place, softmax, epilogue.  The region that owns a
// tile's first pair also turns its K into K' and its V into fp16.  K arrives in a
// staging tile one ahead, so its copy does not wait for the ring.
//
// Numbers.  All products have fp16 operands and fp32 sums.  q' and k' are divided
// by a power of two not below the norm weights, so they are at most sqrt(128).  A V row is
// scaled by 2^a: by 2^8 where its largest entry lies in [2^-6, 2^7), else to bring that into
// [2^8, 2^9), and P carries 2^(a_min - a) then.  P is relative to its
// row's maximum, where it is 2^14 (one pass of TMEM loads; relative to the fixed bound
// scale D max|wq| max|wk| of the plain forward it would leave fp16's range), and not
// divided by its row sum before the product.  o is within 1.7e-3 (relative, 2-norm) of
// the 64-bit value, of which bf16's rounding of o alone is 1.66e-3.
//
// Values that are not finite.  A masked key has P = 0, but 0 * inf and 0 * NaN are NaN
// in a product of tiles: a V row that is not finite enters the tile as zeros and takes no
// part in the scales of the others, and the queries that see it are summed again key by
// key.  A K row that is not finite makes P of those that see it NaN.  Sequences of 4096
// whose last 100 tokens are NaN cost 252 us below (940 when rows were summed again wherever
// O was not finite).
//
// What bounds it: the regions' chain per unit (64 tokens of two heads), about 27,000
// cycles of which the MMAs are 1,700: Q' 2.4k, K' 3.5k and V 2k of the owner, maximum
// 2k, P 4.9k, gate and store 7.5k, waits for S and O 3.5k.  4 x 4096 tokens of 32 heads:
// 220 us, 33 % of the measured copy rate (the plain forward: 143 us, without the
// maximum, with 128-token tiles and bf16 operands).  A run starts with its first K tiles
// loaded straight into the ring and shared by the regions, and the tokens' rotations
// evaluated once per CTA: 1 x 256 tokens of 4 / 1 heads 28.5 -> 26.3 us cold (24 us back to
// back).  Measured instead:
//   - warp MMAs (m16n8k16) on 16 tokens x 2 heads per warp, S, P and O in registers,
//     eight warps per SM: 320 us (their operands' shared-memory reads and latency);
//     with 16 warps and one head each, bf16 P and spills: 252 us.
//   - K' and V by a helper warp in the background: 336 us, one warp is too slow.
//   - work moved from the region of a tile's first pair to the other, whose chain is
//     shorter: V 246 us, the next tile's K' 258 us (against 232 in the same minutes;
//     why was not found);
//   - a run's first V tiles by the second region before its first S: 24.5 us at 1 x 256,
//     but 240 us here, for the second copy of that code.
#include <atomic>

#include "launch.cuh"
#include "sink_common.cuh"

namespace swa {
namespace snk {
namespace fwd {

constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168, kRegsControl = 56, kRegsRegion = 224;
static_assert(kRegsControl + 2 * kRegsRegion <= 3 * kRegsLaunch, "register split");
constexpr int kTok = 64;                       // tokens per tile
constexpr int kSlots = 3;
constexpr int kRing = kSlots * kTok + kMaxSink;  // operand rows: 208
constexpr int kRingHalf = kRing * 128;           // one 64-dim half of the ring
constexpr int kTileHalf = kTok * 128;            // one half of a 64-row tile (a TMA box)
constexpr int kQHalf = 128 * 128;
constexpr int kQBytes = 2 * kQHalf;

struct alignas(1024) Smem {
  uint8_t k[2][kRingHalf];
  uint8_t v[2][kRingHalf];
  uint8_t q[3][kQBytes];            // head pair n uses slot n % 3: Q, then g, then o
  uint8_t stage[2][kTileHalf];      // the next tile's raw K
  // rot(64 t w_p) of the tile of K load n in table n % 4: not by slot, since a chain's
  // tile 0 may be loaded while Q rows of the last chain's tile in that slot are due.
  float2 rot_tile[4][kMaxPairs];
  float wq[kHeadDim], wk[kHeadDim];    // divided by cq, ck
  float va[kRing];                     // a of each V row (v 2^a is stored)
  int scaled[kSlots + 1];              // some row of the slot (or a sink) has a != kVExp
  float cc;                            // cq ck
  uint64_t rotfull[4], runfull, stgfull, stgempty, kready[3], kempty[3];
  uint64_t vfull[3], vready[3], vempty[3];
  uint64_t skfull, skready, skempty, svfull, svready, svempty;  // the sinks' K and V
  uint64_t qfull[3], qready[2], sfull[2], pfull[2], ofull[2], tfree[2];
  uint64_t gfull[3], ostore[2], slotfree[3], drain, never;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) <= 232448, "shared memory over the 227 KiB per-CTA limit");

enum Site {
  kSiteStgEmpty = 0xC0, kSiteStgFull, kSiteRot, kSiteKReady, kSiteKEmpty, kSiteVFull, kSiteVReady,
  kSiteVEmpty, kSiteSink, kSiteQFull, kSiteQReady, kSiteSFull, kSitePFull, kSiteOFull, kSiteTFree,
  kSiteGFull, kSiteOStore, kSiteSlotFree, kSiteForced, kSiteAlign
};

struct Cursor {
  int b, kvh, t, h, u;  // h: head pair of the group; u: tiles since the run's start
};
__device__ __forceinline__ Cursor cursor_at(const SinkFwdArgs& a, long long u0) {
  Cursor c;
  const int chain = static_cast<int>(u0 / a.tiles);
  c.t = static_cast<int>(u0 - static_cast<long long>(chain) * a.tiles);
  c.b = chain / a.Hkv;
  c.kvh = chain - c.b * a.Hkv;
  c.h = 0;
  c.u = 0;
  return c;
}
__device__ __forceinline__ void next_tile(Cursor& c, const SinkFwdArgs& a) {
  ++c.u;
  if (++c.t == a.tiles) {
    c.t = 0;
    if (++c.kvh == a.Hkv) {
      c.kvh = 0;
      ++c.b;
    }
  }
}
__device__ __forceinline__ void next_pair(Cursor& c, const SinkFwdArgs& a) {
  if (++c.h == (a.G + 1) / 2) {
    c.h = 0;
    next_tile(c, a);
  }
}
// First tile to load at this tile: the two before it at the start of a run.
__device__ __forceinline__ int first_load(const Cursor& c) {
  return c.u == 0 ? max(0, c.t - 2) : c.t;
}
__device__ __forceinline__ bool seg_first(const Cursor& c) { return c.u == 0 || c.t == 0; }
__device__ __forceinline__ bool seg_last(const Cursor& c, const SinkFwdArgs& a, int n_tiles) {
  return c.u == n_tiles - 1 || c.t == a.tiles - 1;
}

__device__ __forceinline__ uint32_t sw_off(int row, int chunk16) {
  return static_cast<uint32_t>(row * 128 + ((chunk16 ^ (row & 7)) << 4));
}
// Phases of a ring of three slots, as their loads are counted in order.
struct Ring {
  uint32_t par = 0, used = 0;
  __device__ __forceinline__ uint32_t parity(int s) const { return (par >> s) & 1u; }
  __device__ __forceinline__ bool was_used(int s) const { return (used >> s) & 1u; }
  __device__ __forceinline__ void advance(int s) {
    par ^= 1u << s;
    used |= 1u << s;
  }
};
__device__ __forceinline__ float2 cmul(float2 x, float2 y) {
  return make_float2(x.x * y.x - x.y * y.y, x.x * y.y + x.y * y.x);
}
template <int kPairs>
struct RowRot {
  float2 r[kPairs > 0 ? kPairs : 1];
};
__device__ __forceinline__ float2 unpack2(uint32_t u) { return make_float2(bf16_lo(u), bf16_hi(u)); }

// Sum of squares of the 64 dims in a half row's eight chunks.
__device__ __forceinline__ float half_sumsq(const uint4 (&x)[8]) {
  float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float2 a = unpack2(x[c].x), b = unpack2(x[c].y), d = unpack2(x[c].z), e = unpack2(x[c].w);
    s0 = __ffma2_rn(a, a, s0);
    s1 = __ffma2_rn(b, b, s1);
    s0 = __ffma2_rn(d, d, s0);
    s1 = __ffma2_rn(e, e, s1);
  }
  return (s0.x + s0.y) + (s1.x + s1.y);
}
// Chunk of eight dims times s w, as fp16.
__device__ __forceinline__ uint4 scale_chunk(const uint4& x, float s, const float* w) {
  const float4 a = *reinterpret_cast<const float4*>(w), b = *reinterpret_cast<const float4*>(w + 4);
  const float2 s2 = make_float2(s, s);
  const float2 y0 = __fmul2_rn(__fmul2_rn(unpack2(x.x), make_float2(a.x, a.y)), s2);
  const float2 y1 = __fmul2_rn(__fmul2_rn(unpack2(x.y), make_float2(a.z, a.w)), s2);
  const float2 y2 = __fmul2_rn(__fmul2_rn(unpack2(x.z), make_float2(b.x, b.y)), s2);
  const float2 y3 = __fmul2_rn(__fmul2_rn(unpack2(x.w), make_float2(b.z, b.w)), s2);
  return make_uint4(pack_f16x2(y0.x, y0.y), pack_f16x2(y1.x, y1.y), pack_f16x2(y2.x, y2.y),
                    pack_f16x2(y3.x, y3.y));
}
// Chunks 0 .. n-1 (n = the rotated chunks) of a row: s w x, pairs (p, p + kPairs)
// turned by base rr.  x may be changed; out receives the fp16 chunks.
template <int kPairs>
__device__ __forceinline__ void rope_head(const uint4* in, uint4* out, float s, const float* w,
                                          const float2* base, const RowRot<kPairs>& rr) {
  constexpr int kN = (2 * kPairs + 7) / 8;
  if constexpr (kN > 0) {
    float x[kN * 8];
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const uint32_t u[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * c + 2 * e] = bf16_lo(u[e]) * s * w[8 * c + 2 * e];
        x[8 * c + 2 * e + 1] = bf16_hi(u[e]) * s * w[8 * c + 2 * e + 1];
      }
    }
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const float2 t = base != nullptr ? cmul(base[p], rr.r[p]) : rr.r[p];
      const float u = x[p], v = x[p + kPairs];
      x[p] = u * t.x - v * t.y;
      x[p + kPairs] = v * t.x + u * t.y;
    }
#pragma unroll
    for (int c = 0; c < kN; ++c)
      out[c] = make_uint4(pack_f16x2(x[8 * c], x[8 * c + 1]), pack_f16x2(x[8 * c + 2], x[8 * c + 3]),
                          pack_f16x2(x[8 * c + 4], x[8 * c + 5]),
                          pack_f16x2(x[8 * c + 6], x[8 * c + 7]));
  }
}

// A K row (two 64-dim halves at src) to k' at dst, by two neighbouring threads:
// thread hf takes rotated pairs 12 hf .. 12 hf + 11 (of 24: those past kPairs are dims
// that are not rotated) and five of the ten chunks of dims 48 .. 127, so neither waits
// for the other's kind of work.
template <int kPairs>
__device__ __forceinline__ void k_row_pair(const uint8_t* s0, const uint8_t* s1, int srow,
                                           uint8_t* d0, uint8_t* d1, int drow, int hf,
                                           const float* wk, const float2* base,
                                           const RowRot<kPairs>& rr, float eps) {
  float lo[12], hi[12];
  float2 ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 12; ++i) {
    const int p = i + 12 * hf, a = pair_lo(p, kPairs), b = pair_hi(p, kPairs);
    lo[i] = bf16_f32(
        *reinterpret_cast<const uint16_t*>(s0 + sw_off(srow, a >> 3) + 2 * (a & 7)));
    hi[i] = bf16_f32(
        *reinterpret_cast<const uint16_t*>(s0 + sw_off(srow, b >> 3) + 2 * (b & 7)));
    const float2 f = make_float2(lo[i], hi[i]);
    ss = __ffma2_rn(f, f, ss);
  }
  uint4 x[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int c = 6 + 5 * hf + i;  // chunks 6 .. 15 of the row
    x[i] = *reinterpret_cast<const uint4*>((c < 8 ? s0 : s1) + sw_off(srow, c & 7));
    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack2(u[e]);
      ss = __ffma2_rn(f, f, ss);
    }
  }
  float s = ss.x + ss.y;
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  const float rinv = rsqrtf(s * (1.0f / kHeadDim) + eps);
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int c = 6 + 5 * hf + i;
    *reinterpret_cast<uint4*>((c < 8 ? d0 : d1) + sw_off(drow, c & 7)) =
        scale_chunk(x[i], rinv, wk + 8 * c);
  }
#pragma unroll
  for (int i = 0; i < 12; ++i) {
    const int p = i + 12 * hf, a = pair_lo(p, kPairs), b = pair_hi(p, kPairs);
    float2 t = make_float2(1.0f, 0.0f);
    if (kPairs > 0) {
      const float2 r0 = i < kPairs ? rr.r[i < kPairs ? i : 0] : t;
      const float2 r1 = i + 12 < kPairs ? rr.r[i + 12 < kPairs ? i + 12 : 0] : t;
      const float2 r = hf ? r1 : r0;
      t = base != nullptr && p < kPairs ? cmul(base[p], r) : r;
    }
    const float u = lo[i] * rinv * wk[a], v = hi[i] * rinv * wk[b];
    const uint32_t y = pack_f16x2(u * t.x - v * t.y, v * t.x + u * t.y);
    *reinterpret_cast<uint16_t*>(d0 + sw_off(drow, a >> 3) + 2 * (a & 7)) = static_cast<uint16_t>(y);
    *reinterpret_cast<uint16_t*>(d0 + sw_off(drow, b >> 3) + 2 * (b & 7)) =
        static_cast<uint16_t>(y >> 16);
  }
}

// Half a V row from bf16 to fp16 in place; returns the row's exponent a.  A row that is
// not finite becomes zeros, and so does one that `keep` refuses (a sink past n_sink).
__device__ __forceinline__ float v_half_row(uint8_t* half, int row, bool keep) {
  uint4 x[8];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    x[c] = *reinterpret_cast<const uint4*>(half + sw_off(row, c));
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu),
                             __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
  }
  m = max(m & 0xffffu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const float e = keep ? v_exp(__uint_as_float(min(m, 0x7f80u) << 16)) : kZeroRow;
  const float f = pow2i(fmaxf(e, -126.0f));
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (keep && e != kBadRow) {
      const float2 s2 = make_float2(f, f);
      const float2 a = __fmul2_rn(unpack2(x[c].x), s2), b = __fmul2_rn(unpack2(x[c].y), s2);
      const float2 d = __fmul2_rn(unpack2(x[c].z), s2), g = __fmul2_rn(unpack2(x[c].w), s2);
      y = make_uint4(pack_f16x2(a.x, a.y), pack_f16x2(b.x, b.y), pack_f16x2(d.x, d.y),
                     pack_f16x2(g.x, g.y));
    }
    *reinterpret_cast<uint4*>(half + sw_off(row, c)) = y;
  }
  return e;
}

// A Q row (both halves of a 128-row slot) in place: q' / cq, fp16.
template <int kPairs>
__device__ __forceinline__ void q_row(uint8_t* tile, int row, const float* wq, const float2* base,
                                      const RowRot<kPairs>& rr, float eps) {
  float ss = 0.f;
  uint4 x[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = *reinterpret_cast<const uint4*>(tile + kQHalf + sw_off(row, c));
  ss = half_sumsq(x);
  uint4 y[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) y[c] = *reinterpret_cast<const uint4*>(tile + sw_off(row, c));
  ss += half_sumsq(y);
  const float rinv = rsqrtf(ss * (1.0f / kHeadDim) + eps);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(tile + kQHalf + sw_off(row, c)) = scale_chunk(x[c], rinv, wq + 64 + 8 * c);
  constexpr int kN = (2 * kPairs + 7) / 8;
#pragma unroll
  for (int c = kN; c < 8; ++c)
    *reinterpret_cast<uint4*>(tile + sw_off(row, c)) = scale_chunk(y[c], rinv, wq + 8 * c);
  if constexpr (kN > 0) {
    uint4 z[kN];
    rope_head<kPairs>(y, z, rinv, wq, base, rr);
#pragma unroll
    for (int c = 0; c < kN; ++c) *reinterpret_cast<uint4*>(tile + sw_off(row, c)) = z[c];
  }
}

// fp16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kIdescQK = idesc_f16(128, kRing, false);
constexpr uint32_t kIdescPV = idesc_f16(128, 128, true);

template <int kPairs>
__global__ void __launch_bounds__(kThreads, 1)
    sink_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_g,
                       const __grid_constant__ CUtensorMap tm_o,
                       const __grid_constant__ CUtensorMap tm_ks,
                       const __grid_constant__ CUtensorMap tm_vs, const SinkFwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem_raw) & 1023u) {
    if (tid == 0) atomicCAS(a.err, 0, kDevErrTimeoutBase + kSiteAlign);
    return;
  }
  const long long u0 = a.total_tiles * blockIdx.x / gridDim.x;
  const int n_tiles = static_cast<int>(a.total_tiles * (blockIdx.x + 1) / gridDim.x - u0);
  const int pairs = (a.G + 1) / 2, n_units = n_tiles * pairs;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&sm.rotfull[i], 1);
    mbar_init(&sm.runfull, 1);  // the run's first K tiles
    mbar_init(&sm.stgfull, 1);
    mbar_init(&sm.stgempty, 128);
    mbar_init(&sm.skfull, 1);
    mbar_init(&sm.skready, 128);
    mbar_init(&sm.skempty, 1);
    mbar_init(&sm.svfull, 1);
    mbar_init(&sm.svready, 128);
    mbar_init(&sm.svempty, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sm.kready[i], 128);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], 1);
      mbar_init(&sm.vready[i], 128);
      mbar_init(&sm.vempty[i], 1);
      mbar_init(&sm.qfull[i], 1);
      mbar_init(&sm.gfull[i], 1);
      mbar_init(&sm.slotfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qready[i], 128);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i], 128);
      mbar_init(&sm.ofull[i], 1);
      mbar_init(&sm.tfree[i], 128);
      mbar_init(&sm.ostore[i], 128);
    }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.never, 1);
    for (int i = 0; i <= kSlots; ++i) sm.scaled[i] = 0;
    sm.abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    prefetch_tensormap(&tm_g);
    prefetch_tensormap(&tm_o);
    prefetch_tensormap(&tm_ks);
    prefetch_tensormap(&tm_vs);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  // rot(tok w_p) of the tile's 64 tokens, evaluated once for all threads, in a Q slot
  // that no copy uses before the second barrier below
  float2* tok_rot = reinterpret_cast<float2*>(sm.q[2]);
  for (int i = tid; i < kPairs * kTok; i += kThreads) {
    float cv, sv;
    rope_cos_sin(static_cast<double>(i & (kTok - 1)), a.inv_freq[i / kTok], &cv, &sv);
    tok_rot[i] = make_float2(cv, sv);
  }
  fence_proxy_async_smem();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  {
    const float cq = pow2_ceil(warp_absmax(a.wq, lane));
    const float ck = pow2_ceil(warp_absmax(a.wk, lane));
    if (tid < kHeadDim) {
      sm.wq[tid] = a.wq[tid] / cq;
      sm.wk[tid] = a.wk[tid] / ck;
    }
    if (tid == 0) sm.cc = cq * ck;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const bool sinks = a.n_sink > 0;
  const int pre = min(2, cursor_at(a, u0).t);  // tiles loaded before the run's first
  RowRot<kPairs> rr;  // of a region thread's rows of Q, K and V, which are one token's
  if (warp >= 4) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) rr.r[p] = tok_rot[p * kTok + (((tid - 128) & 127) >> 1)];
  }
  __syncthreads();

  if (warp < 4) {
    regs_dec<kRegsControl>();
    if (warp == 0) {
      // -------------------------------------------------------- K and Q producer
      bool ok = true;
      auto wait0 = [&](uint64_t* bar, uint32_t par, int site) -> bool {
        bool w = true;
        if (lane == 0) w = mbar_wait_inl(bar, par, abort, a.err, site);
        return __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
      };
      int nk = 0, nq = 0, ns = 0;  // K tiles, Q slots and sink blocks loaded
      Cursor c = cursor_at(a, u0);
      auto load_q = [&](const Cursor& x, int h) -> bool {
        const int qs = nq % 3;
        if (nq >= 3 && !wait0(&sm.slotfree[qs], ((nq / 3) - 1) & 1, kSiteSlotFree)) return false;
        if (lane == 0) {
          const int hq = x.kvh * a.G + 2 * h;
          mbar_arrive_expect_tx(&sm.qfull[qs], kQBytes);
          tma_load_4d(sm.q[qs], &tm_q, &sm.qfull[qs], 0, hq, x.t * kTok, x.b);
          tma_load_4d(sm.q[qs] + kQHalf, &tm_q, &sm.qfull[qs], 64, hq, x.t * kTok, x.b);
          tma_prefetch_4d(&tm_g, 0, hq, x.t * kTok, x.b);
          tma_prefetch_4d(&tm_g, 64, hq, x.t * kTok, x.b);
        }
        ++nq;
        return true;
      };
      ok = load_q(c, 0);  // the first rows do not wait for the run's K tiles
      for (int it = 0; it < n_tiles && ok; ++it, next_tile(c, a)) {
        // Tile it's load follows that of tile it - 1 out of the staging tile (tile 0's do
        // not use it).
        if (it >= 2 && !(ok = wait0(&sm.stgempty, it & 1, kSiteStgEmpty))) break;
        // The tables of this tile's loads.  Table n % 4 is free: the loads before n are
        // done with theirs, and load n - 1 was transformed into a slot that Q K^T of load
        // n - 4's tile or a later one freed, so that tile's Q rows are too.
        for (int j = first_load(c); j <= c.t; ++j) {
          const int n = nk + j - first_load(c);
          if (lane < kPairs) {
            float cv, sv;
            rope_cos_sin(static_cast<double>(j) * kTok, a.inv_freq[lane], &cv, &sv);
            sm.rot_tile[n & 3][lane] = make_float2(cv, sv);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.rotfull[n & 3]);
        }
        if (it == 0) {  // the run's first tiles at once, straight into the ring
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.runfull, (pre + 1) * 2 * kTileHalf);
            for (int j = c.t - pre; j <= c.t; ++j) {
              const int s = j % kSlots;
              tma_load_4d(sm.k[0] + s * kTileHalf, &tm_k, &sm.runfull, 0, c.kvh, j * kTok, c.b);
              tma_load_4d(sm.k[1] + s * kTileHalf, &tm_k, &sm.runfull, 64, c.kvh, j * kTok, c.b);
            }
          }
          nk = pre + 1;
        } else {
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.stgfull, 2 * kTileHalf);
            tma_load_4d(sm.stage[0], &tm_k, &sm.stgfull, 0, c.kvh, c.t * kTok, c.b);
            tma_load_4d(sm.stage[1], &tm_k, &sm.stgfull, 64, c.kvh, c.t * kTok, c.b);
          }
          ++nk;
        }
        if (ok && sinks && seg_first(c)) {
          if (ns > 0) ok = wait0(&sm.skempty, (ns - 1) & 1, kSiteSink);
          if (ok) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&sm.skfull, 2 * kMaxSink * 128);
              tma_load_4d(sm.k[0] + kSlots * kTileHalf, &tm_ks, &sm.skfull, 0, c.kvh, 0, c.b);
              tma_load_4d(sm.k[1] + kSlots * kTileHalf, &tm_ks, &sm.skfull, 64, c.kvh, 0, c.b);
            }
            ++ns;
          }
        }
        for (int h = it == 0 ? 1 : 0; h < pairs && ok; ++h) ok = load_q(c, h);
      }
      if (!ok && lane == 0) {  // copies in flight land before the CTA's memory is released
        if (nk > 0) mbar_wait_drain(&sm.runfull, 0);
        if (nk > pre + 1) mbar_wait_drain(&sm.stgfull, (nk - pre) & 1);
        if (ns > 0) mbar_wait_drain(&sm.skfull, (ns - 1) & 1);
        for (int s = 0; s < 3; ++s) {
          const int n = (nq - s + 2) / 3;
          if (n > 0) mbar_wait_drain(&sm.qfull[s], static_cast<uint32_t>(n - 1) & 1);
        }
      }
    } else if (warp == 3 && lane == 0) {
      // ------------------------------------------------------------ V producer
      Ring vr;
      int ns = 0;
      bool ok = true;
      Cursor c = cursor_at(a, u0);
      for (int it = 0; it < n_tiles && ok; ++it, next_tile(c, a)) {
        for (int j = first_load(c); j <= c.t && ok; ++j) {
          const int s = j % kSlots;
          if (vr.was_used(s) && !(ok = mbar_wait_inl(&sm.vempty[s], vr.parity(s) ^ 1u, abort, a.err,
                                                     kSiteVEmpty)))
            break;
          mbar_arrive_expect_tx(&sm.vfull[s], 2 * kTileHalf);
          tma_load_4d(sm.v[0] + s * kTileHalf, &tm_v, &sm.vfull[s], 0, c.kvh, j * kTok, c.b);
          tma_load_4d(sm.v[1] + s * kTileHalf, &tm_v, &sm.vfull[s], 64, c.kvh, j * kTok, c.b);
          vr.advance(s);
        }
        if (ok && sinks && seg_first(c)) {
          if (ns > 0) ok = mbar_wait_inl(&sm.svempty, (ns - 1) & 1, abort, a.err, kSiteSink);
          if (ok) {
            mbar_arrive_expect_tx(&sm.svfull, 2 * kMaxSink * 128);
            tma_load_4d(sm.v[0] + kSlots * kTileHalf, &tm_vs, &sm.svfull, 0, c.kvh, 0, c.b);
            tma_load_4d(sm.v[1] + kSlots * kTileHalf, &tm_vs, &sm.svfull, 64, c.kvh, 0, c.b);
            ++ns;
          }
        }
      }
      if (!ok) {
        for (int s = 0; s < kSlots; ++s)
          if (vr.was_used(s)) mbar_wait_drain(&sm.vfull[s], vr.parity(s) ^ 1u);
        if (ns > 0) mbar_wait_drain(&sm.svfull, (ns - 1) & 1);
      }
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      Ring kr, vr;
      bool ok = true;
      if (a.flags & SWA_FLAG_FORCE_TIMEOUT)
        ok = mbar_wait_inl(&sm.never, 0, abort, a.err, kSiteForced);
      auto W = [&](uint64_t* bar, uint32_t par, int site) {
        if (ok) ok = mbar_wait_inl(bar, par, abort, a.err, site);
        return ok;
      };
      int seg_q = 0, seg_p = 0;  // segments whose sinks were waited for
      Cursor cq = cursor_at(a, u0), cp = cq;
      for (int n = 0; n < n_units && ok; n += 2) {
        for (int i = 0; i < 2 && n + i < n_units && ok; ++i, next_pair(cq, a)) {
          const int m = n + i, r = m & 1;
          const uint32_t cnt = static_cast<uint32_t>(m >> 1);
          if (cq.h == 0) {
            for (int j = first_load(cq); j <= cq.t && ok; ++j) {
              const int s = j % kSlots;
              W(&sm.kready[s], kr.parity(s), kSiteKReady);
              kr.advance(s);
            }
            if (sinks && seg_first(cq)) {
              W(&sm.skready, seg_q & 1, kSiteSink);
              ++seg_q;
            }
          }
          if (!W(&sm.qready[r], cnt & 1, kSiteQReady)) break;
          if (cnt > 0 && !W(&sm.tfree[r], (cnt - 1) & 1, kSiteTFree)) break;
          tc_fence_after();
          const uint64_t qd = make_desc_sw128(smem_u32(sm.q[m % 3]), 16, 1024);
          const uint64_t kd = make_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem + r * 256, desc_advance(qd, (kk >> 2) * kQHalf + (kk & 3) * 32),
                   desc_advance(kd, (kk >> 2) * kRingHalf + (kk & 3) * 32), kIdescQK, kk > 0);
          mma_commit(&sm.sfull[r]);
          if (cq.h == pairs - 1) {
            if (cq.t >= 2) mma_commit(&sm.kempty[(cq.t - 2) % kSlots]);
            if (seg_last(cq, a, n_tiles)) {
              if (cq.t >= 1) mma_commit(&sm.kempty[(cq.t - 1) % kSlots]);
              mma_commit(&sm.kempty[cq.t % kSlots]);
              if (sinks) mma_commit(&sm.skempty);
            }
          }
        }
        for (int i = 0; i < 2 && n + i < n_units && ok; ++i, next_pair(cp, a)) {
          const int m = n + i, r = m & 1;
          const uint32_t cnt = static_cast<uint32_t>(m >> 1);
          if (cp.h == 0) {
            for (int j = first_load(cp); j <= cp.t && ok; ++j) {
              const int s = j % kSlots;
              W(&sm.vready[s], vr.parity(s), kSiteVReady);
              vr.advance(s);
            }
            if (sinks && seg_first(cp)) {
              W(&sm.svready, seg_p & 1, kSiteSink);
              ++seg_p;
            }
          }
          if (!W(&sm.pfull[r], cnt & 1, kSitePFull)) break;
          tc_fence_after();
          const uint32_t base = tmem + r * 256;
          const uint64_t vd = make_desc_sw128(smem_u32(sm.v[0]), kRingHalf, 1024);
          uint32_t acc = 0;
          for (int d = min(2, cp.t); d >= 0; --d) {  // the tiles that exist
            const int s = (cp.t - d) % kSlots;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              mma_ts(base + 128, base + s * 32 + kk * 8, desc_advance(vd, s * kTileHalf + kk * 2048),
                     kIdescPV, acc);
              acc = 1;
            }
          }
          if (sinks && cp.t >= 2)
            mma_ts(base + 128, base + kSlots * 32, desc_advance(vd, kSlots * kTileHalf), kIdescPV, 1);
          mma_commit(&sm.ofull[r]);
          if (cp.h == pairs - 1) {
            if (cp.t >= 2) mma_commit(&sm.vempty[(cp.t - 2) % kSlots]);
            if (seg_last(cp, a, n_tiles)) {
              if (cp.t >= 1) mma_commit(&sm.vempty[(cp.t - 1) % kSlots]);
              mma_commit(&sm.vempty[cp.t % kSlots]);
              if (sinks) mma_commit(&sm.svempty);
            }
          }
        }
      }
      if (!ok) {
        mma_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0);
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- regions
    regs_inc<kRegsRegion>();
    const int r = (warp - 4) >> 2, wq4 = warp & 3;
    const int row = wq4 * 32 + lane, tok = row >> 1, head = row & 1;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(wq4 * 32) << 16) + r * 256;
    const float sc = a.scale_log2 * sm.cc;
    const bool elected = row == 0;
    bool ok = true;
    // Every wait's outcome is the same for the whole warp: the TMEM accesses and
    // shuffles behind it are warp-wide.
    auto W = [&](uint64_t* bar, uint32_t par, int site) {
      ok = __all_sync(0xffffffffu, mbar_wait_inl(bar, par, abort, a.err, site));
      return ok;
    };
    // The loads in order, for the phases of their slots (both regions count all).  A
    // wait by parity tells a phase from the one before it only: where the other
    // region may have taken the loads in between, its readiness is waited for first.
    Ring kr, vr;
    int nk = 0, last_s = 0, last_v = -1, seg_k = 0, seg_v = 0;
    Cursor kc = cursor_at(a, u0), vc = kc;
    int kacct = 0, vacct = 0;  // tiles accounted so far
    int g_issued[3] = {0, 0, 0};
    uint32_t last_g_phase[3] = {0u, 0u, 0u};

    Cursor c = cursor_at(a, u0);
    if (r == 1) next_pair(c, a);
    for (int n = r; n < n_units && ok; n += 2) {
      const uint32_t cnt = static_cast<uint32_t>(n >> 1);
      const int qs = n % 3;
      const uint32_t qph = static_cast<uint32_t>(n / 3) & 1;
      const int hq = c.kvh * a.G + 2 * c.h;
      const int i0 = c.t * kTok;
      const bool whole = 2 * c.h + 1 < a.G;     // both heads are the group's
      const bool real = whole || head == 0;     // this row's is
      const bool owner = c.h == 0;

      // ---- Q'
      const int load = pre + c.u;  // the tile's place among the run's K loads
      if (!W(&sm.rotfull[load & 3], (load >> 2) & 1, kSiteRot)) break;
      if (!W(&sm.qfull[qs], qph, kSiteQFull)) break;
      q_row<kPairs>(sm.q[qs], row, sm.wq, sm.rot_tile[load & 3], rr, a.eps);
      fence_proxy_async_smem();
      mbar_arrive(&sm.qready[r]);

      // ---- K of the tile (and of those before it at a run's start)
      for (; ok && kacct <= c.u; ++kacct, next_tile(kc, a)) {
        const bool mine = owner && kacct == c.u;
        for (int j = first_load(kc); j <= kc.t && ok; ++j, ++nk) {
          const int s = j % kSlots;
          // the run's first tiles in place, by both regions where both start with them
          const bool first = kacct == 0;
          if (first ? (pairs > 1 ? ((kc.t - j) & 1) == r : r == 0) : mine) {
            if (first) {
              if (!W(&sm.rotfull[nk & 3], 0, kSiteRot)) break;
              if (!W(&sm.runfull, 0, kSiteStgFull)) break;
            } else {
              if (!W(&sm.kready[last_s], kr.parity(last_s) ^ 1u, kSiteKReady)) break;
              if (!W(&sm.stgfull, (nk - pre - 1) & 1, kSiteStgFull)) break;
              if (kr.was_used(s) && !W(&sm.kempty[s], kr.parity(s) ^ 1u, kSiteKEmpty)) break;
            }
            const int at = s * kTok + tok;
            k_row_pair<kPairs>(first ? sm.k[0] : sm.stage[0], first ? sm.k[1] : sm.stage[1],
                               first ? at : tok, sm.k[0], sm.k[1], at, head, sm.wk,
                               sm.rot_tile[nk & 3], rr, a.eps);
            fence_proxy_async_smem();
            mbar_arrive(&sm.kready[s]);
            if (!first) mbar_arrive(&sm.stgempty);
          }
          kr.advance(s);
          last_s = s;
        }
        if (ok && sinks && seg_first(kc)) {
          if (mine) {
            if (seg_k > 0 && !W(&sm.skready, (seg_k - 1) & 1, kSiteSink)) break;
            if (!W(&sm.skfull, seg_k & 1, kSiteSink)) break;
            if (wq4 == 0) {  // 16 rows, two threads each
              const int at = kSlots * kTok + tok;
              k_row_pair<kPairs>(sm.k[0], sm.k[1], at, sm.k[0], sm.k[1], at, head, sm.wk, nullptr,
                                 rr, a.eps);
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.skready);
          }
          ++seg_k;
        }
      }
      if (!ok) break;

      // ---- softmax
      if (!W(&sm.sfull[r], cnt & 1, kSiteSFull)) break;
      tc_fence_after();
      if (elected) {  // Q K^T has read Q: the slot takes the gate tile now
        mbar_arrive_expect_tx(&sm.gfull[qs], kQBytes);
        tma_load_4d(sm.q[qs], &tm_g, &sm.gfull[qs], 0, hq, i0, c.b);
        tma_load_4d(sm.q[qs] + kQHalf, &tm_g, &sm.gfull[qs], 64, hq, i0, c.b);
        ++g_issued[qs];
        last_g_phase[qs] = qph;
      }
      __syncwarp();
      const int tm3 = c.t % kSlots;
      const bool see_sinks = sinks && c.t >= 2;
      // How slot s relates to this tile: 0 its own keys, 1 the tile before, 2 the one
      // before that, -1 none.  Chunk ch (32 keys) of it, for this warp's 16 tokens:
      // none of it visible, all, or some.
      auto dist = [&](int s) {
        const int d = tm3 >= s ? tm3 - s : tm3 + kSlots - s;
        return d <= c.t ? d : -1;
      };
      auto none = [&](int d, int ch) {
        return (d == 0 && ch == 1 && wq4 < 2) || (d == 2 && ch == 0 && wq4 >= 2);
      };
      auto full = [&](int d, int ch) {
        return d == 1 || (d == 0 && ch == 0 && wq4 >= 2) || (d == 2 && ch == 1 && wq4 < 2);
      };
      const int sink_hi = min(a.n_sink - 1, i0 + tok - kWindow);  // last visible sink
      // the row's maximum
      float mx = -INFINITY;
#pragma unroll 1
      for (int x = 0; x < 2 * kSlots; ++x) {
        const int s = x >> 1, ch = x & 1, d = dist(s);
        if (d < 0 || none(d, ch)) continue;
        uint32_t v[32];
        tmem_ld32(t_row + s * 64 + ch * 32, v);
        tmem_wait_ld();
        if (full(d, ch)) {
          float m1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            mx = fmaxf(mx, __uint_as_float(v[i]));
            m1 = fmaxf(m1, __uint_as_float(v[i + 1]));
          }
          mx = fmaxf(mx, m1);
        } else {
          const int edge = tok - 32 * ch;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (d == 0 ? i <= edge : i > edge) mx = fmaxf(mx, __uint_as_float(v[i]));
        }
      }
      if (see_sinks) {
        uint32_t v[16];
        tmem_ld16(t_row + kSlots * 64, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i <= sink_hi) mx = fmaxf(mx, __uint_as_float(v[i]));
      }
      // ---- V of the tile: as late as its scales allow, for its slot was freed last
      for (; ok && vacct <= c.u; ++vacct, next_tile(vc, a)) {
        for (int j = first_load(vc); j <= vc.t && ok; ++j) {
          const int s = j % kSlots;
          if (owner && vacct == c.u) {
            // the load before this one first (its scales are read below, and it may have
            // been the other region's)
            if (last_v >= 0 && !W(&sm.vready[last_v], vr.parity(last_v) ^ 1u, kSiteVReady)) break;
            if (!W(&sm.vfull[s], vr.parity(s), kSiteVFull)) break;
            const float e = v_half_row(sm.v[head], s * kTok + tok, true);
            if (head == 0) sm.va[s * kTok + tok] = e;
            // the slot's flag: set by any of the four warps, cleared by none but the first
            const bool any = __any_sync(0xffffffffu, e != kVExp && e != kZeroRow);
            if (lane == 0) {
              if (any) atomicOr(&sm.scaled[s], 1 << wq4);
              else atomicAnd(&sm.scaled[s], ~(1 << wq4));
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.vready[s]);
          } else if (vacct == c.u && j == vc.t) {
            if (!W(&sm.vready[s], vr.parity(s), kSiteVReady)) break;
          }
          vr.advance(s);
          last_v = s;
        }
        if (ok && sinks && seg_first(vc)) {
          if (owner && vacct == c.u) {
            if (seg_v > 0 && !W(&sm.svready, (seg_v - 1) & 1, kSiteSink)) break;
            if (!W(&sm.svfull, seg_v & 1, kSiteSink)) break;
            if (wq4 == 0) {  // rows past n_sink become zeros
              const int at = kSlots * kTok + tok;
              const float e = v_half_row(sm.v[head], at, tok < a.n_sink);
              const bool any = __any_sync(0xffffffffu, e != kVExp && e != kZeroRow);
              if (head == 0) sm.va[at] = e;
              if (lane == 0) sm.scaled[kSlots] = any;
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.svready);
          }
          ++seg_v;
        }
      }
      if (ok && see_sinks) W(&sm.svready, (seg_v - 1) & 1, kSiteSink);
      if (!ok) break;

      // P is 2^14 at the row's maximum, so that fp16 keeps P down to 2^-28 of it normal.
      const float ms = mx == -INFINITY ? 0.0f : mx * sc - 14.0f;  // all NaN: any reference
      // Least exponent of the V rows that this row sees (what a masked one holds must
      // not matter).  With V near 1 it is kVExp for all.
      bool scaled = see_sinks && sm.scaled[kSlots] != 0;
      for (int s = 0; s < kSlots; ++s) scaled = scaled || (dist(s) >= 0 && sm.scaled[s] != 0);
      scaled = __any_sync(0xffffffffu, scaled);  // TMEM loads below: one way for the warp
      float am = kVExp;
      bool sees_bad = false;
      if (scaled) {
        am = 126.0f;
#pragma unroll 1
        for (int s = 0; s < kSlots; ++s) {
          const int d = dist(s);
          if (d < 0) continue;
#pragma unroll 4
          for (int j = 0; j < kTok; j += 4) {
            const float4 e = *reinterpret_cast<const float4*>(&sm.va[s * kTok + j]);
            const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (d == 0 ? j + i <= tok : (d == 1 || j + i > tok)) {
                sees_bad = sees_bad || ev[i] == kBadRow;
                am = fminf(am, ev[i] == kBadRow ? am : ev[i]);
              }
          }
        }
        if (see_sinks)
          for (int i = 0; i < kMaxSink; ++i)
            if (i <= sink_hi) {
              const float ev = sm.va[kSlots * kTok + i];
              sees_bad = sees_bad || ev == kBadRow;
              am = fminf(am, ev == kBadRow ? am : ev);
            }
        __syncwarp();
      }
      // P = 2^(s sc - ms) as fp16 over the region's first columns, slot by slot: P of
      // slot s goes to columns 32 s .., which slots 0 .. s have been read out of.
      float2 l2 = make_float2(0.f, 0.f);
      const float2 sc2 = make_float2(sc, sc), nms2 = make_float2(-ms, -ms);
#pragma unroll 1
      for (int x = 0; x < 2 * kSlots; ++x) {
        const int s = x >> 1, ch = x & 1, d = dist(s);
        if (d < 0) continue;
        uint32_t pk[16];
        if (none(d, ch)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          uint32_t v[32];
          tmem_ld32(t_row + s * 64 + ch * 32, v);
          tmem_wait_ld();
          float2 p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 z = __ffma2_rn(
                make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc2, nms2);
            p[e] = make_float2(ex2_approx(z.x), ex2_approx(z.y));
          }
          if (!full(d, ch)) {
            const int edge = tok - 32 * ch;  // this tile's keys up to it, or the oldest's past it
            const bool up = d == 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              p[e].x = (2 * e <= edge) == up ? p[e].x : 0.f;
              p[e].y = (2 * e + 1 <= edge) == up ? p[e].y : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) l2 = __fadd2_rn(l2, p[e]);
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = pack_f16x2(p[e].x, p[e].y);
        }
        tmem_st16(t_row + s * 32 + ch * 16, pk);
      }
      if (see_sinks) {
        uint32_t v[16], pk[8];
        tmem_ld16(t_row + kSlots * 64, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 z = __ffma2_rn(
              make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc2, nms2);
          float2 p = make_float2(2 * e <= sink_hi ? ex2_approx(z.x) : 0.f,
                                 2 * e + 1 <= sink_hi ? ex2_approx(z.y) : 0.f);
          l2 = __fadd2_rn(l2, p);
          pk[e] = pack_f16x2(p.x, p.y);
        }
        tmem_st8(t_row + kSlots * 32, pk);
      }
      const float l = l2.x + l2.y;
      tmem_wait_st();
      if (scaled) {  // P carries 2^(am - a) of its key's V
#pragma unroll 1
        for (int x = 0; x < kRing / 16; ++x) {
          if ((x >> 2) < kSlots ? dist(x >> 2) < 0 : !see_sinks) continue;
          uint32_t pw[8];
          tmem_ld8(t_row + 8 * x, pw);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&pw[e]));
            const float2 va = *reinterpret_cast<const float2*>(&sm.va[16 * x + 2 * e]);
            pw[e] = pack_f16x2(p.x * pow2i(fmaxf(fminf(am - va.x, 0.0f), -126.0f)),
                               p.y * pow2i(fmaxf(fminf(am - va.y, 0.0f), -126.0f)));
          }
          tmem_st8(t_row + 8 * x, pw);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&sm.pfull[r]);
      const long long pos = static_cast<long long>(i0) + tok;
      if (a.lse != nullptr && pos < a.T && real)
        a.lse[(static_cast<long long>(c.b) * a.Hq + hq + head) * a.T + pos] =
            (ms + log2f(l)) * 0.6931471805599453f;

      // ---- epilogue: o = O / l * sigmoid(g) over g, 32 dims at a time
      if (!W(&sm.ofull[r], cnt & 1, kSiteOFull)) break;
      if (!W(&sm.gfull[qs], qph, kSiteGFull)) break;
      tc_fence_after();
      // V of all keys below 2^-64: the result's factor in two steps, both normal
      const float split = am > 64.0f ? 64.0f : 0.0f;
      const float il = 1.0f / l * pow2i(split - am);
      const bool in_two = __any_sync(0xffffffffu, split != 0.0f);  // one way for the warp
      // (a row sum of NaN makes O NaN by itself)
      const bool again = __any_sync(0xffffffffu, sees_bad && l == l);
      const float ilc = again ? 1.0f : il;
#pragma unroll 1
      for (int ch = 0; ch < kHeadDim / 32; ++ch) {
        uint32_t ov[32];
        tmem_ld32(t_row + 128 + ch * 32, ov);
        tmem_wait_ld();
        if (again) {
          // These dims again, key by key, from the P in TMEM and V in memory, with the
          // row's factor on P: beside an infinity V may hold any number.
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 1
          for (int x = 0; x < kRing / 16; ++x) {  // 16 keys: 8 columns of P
            const int s = x >> 2, d = s < kSlots ? dist(s) : (see_sinks ? 0 : -1);
            if (d < 0) continue;
            const int key0 = s < kSlots ? (c.t - d) * kTok + 16 * (x & 3) : 0;
            uint32_t pw[8];
            tmem_ld8(t_row + 8 * x, pw);
            tmem_wait_ld();
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              uint32_t word = pw[0];
#pragma unroll
              for (int k = 1; k < 8; ++k) word = (e >> 1) == k ? pw[k] : word;
              const float2 p2 = __half22float2(*reinterpret_cast<const __half2*>(&word));
              const float p = (e & 1) ? p2.y : p2.x;
              if (p == 0.0f || key0 + e >= a.T) continue;
              const uint16_t* vrow =
                  a.v + ((static_cast<long long>(c.b) * a.T + key0 + e) * a.Hkv + c.kvh) * kHeadDim;
              // the key's own a (the ring's record may have moved on); a bad row's P was not
              // scaled
              uint32_t m = 0;
#pragma unroll 4
              for (int i = 0; i < kHeadDim / 8; ++i) {
                const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(vrow) + i);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(w4.x & 0x7fff7fffu, w4.y & 0x7fff7fffu),
                                         __vmaxu2(w4.z & 0x7fff7fffu, w4.w & 0x7fff7fffu)));
              }
              m = max(m & 0xffffu, m >> 16);
              const float ek = v_exp(__uint_as_float(min(m, 0x7f80u) << 16));
              const float f = pow2i(ek == kBadRow ? am : ek);
              const float wt = p * il * f * pow2i(-split);
              const uint4* vr4 = reinterpret_cast<const uint4*>(vrow + 32 * ch);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint4 w4 = __ldg(vr4 + y);
                const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  o[8 * y + 2 * q] = fmaf(wt, bf16_lo(ww[q]), o[8 * y + 2 * q]);
                  o[8 * y + 2 * q + 1] = fmaf(wt, bf16_hi(ww[q]), o[8 * y + 2 * q + 1]);
                }
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(o[i]);
        }
        if (in_two && !again) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ov[i] = __float_as_uint(__uint_as_float(ov[i]) * pow2i(-split));
        }
        if (ch + 1 == kHeadDim / 32) {
          tc_fence_before();
          mbar_arrive(&sm.tfree[r]);  // the region may take the next Q K^T
        }
        const float2 il2 = make_float2(ilc, ilc);
        uint8_t* half = sm.q[qs] + (ch >> 1) * kQHalf;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* gp = reinterpret_cast<uint4*>(half + sw_off(row, (ch & 1) * 4 + i));
          const uint4 gv = *gp;
          const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
          uint32_t ow[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 sg = sigmoid2(unpack2(gw[e]));
            const float2 y =
                __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(ov[8 * i + 2 * e]),
                                                  __uint_as_float(ov[8 * i + 2 * e + 1])),
                                      il2),
                           sg);
            ow[e] = pack_bf16x2(y.x, y.y);
          }
          *gp = make_uint4(ow[0], ow[1], ow[2], ow[3]);
        }
      }
      if (!whole && real && pos < a.T) {  // the copy below would write the other head too
        uint16_t* dst =
            a.o + ((static_cast<long long>(c.b) * a.T + pos) * a.Hq + hq) * kHeadDim;
#pragma unroll 4
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<uint4*>(dst + 8 * i) = *reinterpret_cast<const uint4*>(
              sm.q[qs] + (i >> 3) * kQHalf + sw_off(row, i & 7));
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.ostore[r]);
      if (elected) {
        const bool w = mbar_wait_inl(&sm.ostore[r], cnt & 1, abort, a.err, kSiteOStore);
        if (w) {
          if (whole) {
            tma_store_4d(&tm_o, sm.q[qs], 0, hq, i0, c.b);
            tma_store_4d(&tm_o, sm.q[qs] + kQHalf, 64, hq, i0, c.b);
            bulk_commit();
            bulk_wait_read<0>();
          }
          mbar_arrive(&sm.slotfree[qs]);
        }
      }
      __syncwarp();
      next_pair(c, a);
      next_pair(c, a);
    }
    if (elected) {
      if (!ok) {
        for (int s = 0; s < 3; ++s)
          if (g_issued[s] > 0) mbar_wait_drain(&sm.gfull[s], last_g_phase[s]);
      }
      bulk_wait_all();
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kPairs>
int launch_impl(const SinkFwdMaps& m, const SinkFwdArgs& a, const DeviceInfo& di,
                cudaStream_t stream) {
  static std::atomic<int> configured[64];  // per device
  if (!configured[di.device].load(std::memory_order_acquire)) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, sink_fwd_kernel<kPairs>);
    if (e != cudaSuccess) return map_cuda_error(e);
    if (attr.numRegs != kRegsLaunch) return SWA_ERR_UNSUPPORTED;  // the register split's budget
    e = cudaFuncSetAttribute(sink_fwd_kernel<kPairs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(Smem)));
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long grid = a.total_tiles < di.num_sms ? a.total_tiles : di.num_sms;
  return launch_dependent(sink_fwd_kernel<kPairs>, static_cast<unsigned>(grid), kThreads,
                          sizeof(Smem), stream, m.q, m.k, m.v, m.g, m.o, m.ks, m.vs, a);
}

}  // namespace fwd
}  // namespace snk

int launch_sink_fwd(const SinkFwdMaps& m, const SinkFwdArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  switch (a.half_rot) {
    case 0: return snk::fwd::launch_impl<0>(m, a, di, stream);
    case 16: return snk::fwd::launch_impl<16>(m, a, di, stream);
    case 21: return snk::fwd::launch_impl<21>(m, a, di, stream);
    case 24: return snk::fwd::launch_impl<24>(m, a, di, stream);
    default: return SWA_ERR_UNSUPPORTED;
  }
}

}  // namespace swa
