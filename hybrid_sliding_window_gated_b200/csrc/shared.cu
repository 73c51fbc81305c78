// shared.cu -- decode step of a global layer for sequences that share a prefix,
// for sm_100a: the prefix's K' and V are read once for all of them.
//
//   o_n = softmax over [prefix keys 0 .. L-1 ; own keys L .. pos_n] of q'_n . k'
//
// Split at the prefix's end, the two parts are separate softmaxes joined by
// their maxima and sums.  Three kernels:
//   global_decode_kernel  (global.cu) the sequences' own keys, split over chunks; it
//                         also writes the new tokens' k' and v to the caches and q'
//                         to the workspace.
//   prefix_attn_kernel    (here) the prefix part.
//   global_combine_kernel (global.cu) the join.
//
// The prefix part.  For one KV head the N G query rows are a matrix Q' (rows x
// 128) against K' and V (L x 128): 4 x 128 operations per row and key, 512 bytes
// per key.  Up to about 256 rows it is bound by reading K' and V, above by the
// tensor core, so it runs on tcgen05 with 128-row tiles: S = Q' K_j^T in TMEM,
// P as packed bf16 over S, O += P V_j.  A CTA takes a range of 128-key tiles of
// one KV head; the ranges are cut so that the CTAs come out near a multiple of
// 148 (shared_ws).  Two region warpgroups keep the tensor core busy in turn:
//   - more than 128 rows: region r holds row tile 2 pair + r, both read the same
//     key tiles;
//   - up to 128 rows: both regions hold the same rows and take alternate key
//     tiles, each with a partial result of its own.
//
// Numbers.  The caches are bf16, so the operands of a product are too.  q' enters
// as two bf16 terms (its value and what the rounding left over: 16 bits of
// mantissa, half as many products again in all); one term alone adds 1.7e-3
// relative error to o, which already carries P's and the output's rounding.  P enters as
// one bf16 term (o 2.0 to 2.4e-3 off, 1.7e-3 by its own rounding alone): the own-keys
// kernel has spare MMA rows for a second, here it would be 8 more MMAs on the 24 per pair
// of tiles that bound the kernel.
// S, row sums and O are fp32.  The cache's keys are the caller's, so the softmax
// assumes no bound on them: each row keeps a reference maximum, and only when a
// tile exceeds it by 2^8 are the row's O and sum rescaled (P <= 2^8 meanwhile,
// which bf16 and fp32 hold without loss).
#include <atomic>

#include "global_internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace swa {
namespace shr {

constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168, kRegsControl = 96, kRegsRegion = 200;
static_assert(kRegsControl + 2 * kRegsRegion <= 3 * kRegsLaunch, "register split");
constexpr int kHalfBytes = kTile * 64 * 2;
constexpr int kTileBytes = 2 * kHalfBytes;  // a 128 x 128 bf16 tile
constexpr int kTiles = 7;                   // tiles in shared memory: Q' (2 or 4) and the ring
constexpr int kMaxSlots = 5;
constexpr float kSlack = 8.0f;              // log2 units a tile may exceed the reference

struct alignas(1024) Smem {
  uint8_t tile[kTiles][kTileBytes];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t qfull, sfull[2], pfull[2], odone[2], drain, never;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) <= 232448, "shared memory over the 227 KiB per-CTA limit");

enum Site {
  kSiteEmpty = 0xE0, kSiteFull, kSiteQ, kSiteS, kSiteP, kSiteO, kSiteForced, kSiteAlign
};

__device__ __forceinline__ uint64_t desc_k(const uint8_t* tile, int kk) {
  return desc_advance(make_desc_sw128(smem_u32(tile), 16, 1024),
                      (kk >> 2) * kHalfBytes + (kk & 3) * 32);
}
__device__ __forceinline__ uint64_t desc_v(const uint8_t* tile, int kk) {
  return desc_advance(make_desc_sw128(smem_u32(tile), kHalfBytes, 1024), kk * 2048);
}
constexpr uint32_t kIdescQK = make_idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescPV = make_idesc_bf16(128, 128, false, true);

__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PrefixArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem_raw) & 1023u) {
    if (tid == 0) atomicCAS(a.err, 0, kDevErrTimeoutBase + kSiteAlign);
    return;
  }
  // CTAs that read the same keys are neighbours, so the second reads hit L2.
  const int pair = static_cast<int>(blockIdx.x) % a.pairs;
  const int rest = static_cast<int>(blockIdx.x) / a.pairs;
  const int split = rest % a.ctas_per_head, kvh = rest / a.ctas_per_head;
  const int j0 = static_cast<int>(static_cast<long long>(a.key_tiles) * split / a.ctas_per_head);
  const int nt = static_cast<int>(static_cast<long long>(a.key_tiles) * (split + 1) /
                                  a.ctas_per_head) - j0;  // key tiles of this CTA (>= 1)
  const int row_tiles = a.two ? min(2, (a.rows + kTile - 1) / kTile - 2 * pair) : 1;
  const int n_q = a.two ? 4 : 2;      // Q' tiles: value and remainder of each row tile
  const int n_slots = kTiles - n_q;
  uint8_t(*ring)[kTileBytes] = sm.tile + n_q;

  if (tid == 0) {
    for (int i = 0; i < n_slots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.qfull, 1);
    for (int r = 0; r < 2; ++r) {
      mbar_init(&sm.sfull[r], 1);
      mbar_init(&sm.pfull[r], 128);
      mbar_init(&sm.odone[r], 1);
    }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.never, 1);
    sm.abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;

  if (warp < 4) {
    regs_dec<kRegsControl>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------- K and V, in the order of use
      int cnt = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int j) {
        const int s = cnt % n_slots;
        if (cnt >= n_slots)
          ok = mbar_wait_inl(&sm.empty[s], ((cnt / n_slots) - 1) & 1, abort, a.err, kSiteEmpty);
        if (!ok) return;
        mbar_arrive_expect_tx(&sm.full[s], kTileBytes);
        tma_load_4d(ring[s], map, &sm.full[s], 0, (j0 + j) * kTile, kvh, 0);
        tma_load_4d(ring[s] + kHalfBytes, map, &sm.full[s], 64, (j0 + j) * kTile, kvh, 0);
        ++cnt;
      };
      const int ahead = a.two ? 1 : 2;  // K tiles issued before the first V
      for (int j = 0; ok && j < min(ahead, nt); ++j) load(&tm_k, j);
      for (int j = 0; ok && j < nt; ++j) {
        load(&tm_v, j);
        if (ok && j + ahead < nt) load(&tm_k, j + ahead);
      }
      if (!ok) {
        for (int s = 0; s < n_slots; ++s) {
          const int issued = (cnt - s + n_slots - 1) / n_slots;
          if (issued > 0) mbar_wait_drain(&sm.full[s], (issued - 1) & 1);
        }
      }
    } else if (warp == 2 && lane == 0) {
      // ------------------------------------------------------------------- Q'
      mbar_arrive_expect_tx(&sm.qfull, row_tiles * 2 * kTileBytes);
      for (int r = 0; r < row_tiles; ++r)
        for (int x = 0; x < 2; ++x) {
          const int row = (2 * pair + r) * kTile;
          tma_load_4d(sm.tile[2 * r + x], &tm_q, &sm.qfull, 0, row, kvh, x);
          tma_load_4d(sm.tile[2 * r + x] + kHalfBytes, &tm_q, &sm.qfull, 64, row, kvh, x);
        }
      mbar_wait_drain(&sm.qfull, 0);  // landed before this CTA can end
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      bool ok = true;
      if (a.flags & SWA_FLAG_FORCE_TIMEOUT)
        ok = mbar_wait_inl(&sm.never, 0, abort, a.err, kSiteForced);
      int cnt = 0, pc[2] = {0, 0};
      auto W = [&](uint64_t* bar, uint32_t par, int site) {
        if (ok) ok = mbar_wait_inl(bar, par, abort, a.err, site);
        return ok;
      };
      auto item = [&](int i) { return W(&sm.full[i % n_slots], (i / n_slots) & 1, kSiteFull); };
      auto qk = [&](int r, int i) {  // S_r = Q'_r K^T, both terms of Q'
        const uint8_t* kt = ring[i % n_slots];
        const uint8_t* qt = sm.tile[a.two ? 2 * r : 0];
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem + r * 256, desc_k(qt, kk), desc_k(kt, kk), kIdescQK, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem + r * 256, desc_k(qt + kTileBytes, kk), desc_k(kt, kk), kIdescQK, 1);
        mma_commit(&sm.sfull[r]);
      };
      auto pv = [&](int r, int i) {
        const uint8_t* vt = ring[i % n_slots];
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + r * 256 + 128, tmem + r * 256 + kk * 8, desc_v(vt, kk), kIdescPV,
                 (pc[r] > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&sm.odone[r]);
      };
      W(&sm.qfull, 0, kSiteQ);
      if (a.two) {
        if (item(0)) {
          tc_fence_after();
          for (int r = 0; r < row_tiles; ++r) qk(r, 0);
          mma_commit(&sm.empty[0]);
          ++cnt;
        }
        for (int j = 0; ok && j < nt; ++j) {
          const int vi = cnt++, ki = j + 1 < nt ? cnt++ : -1;
          for (int r = 0; ok && r < row_tiles; ++r) {
            if (!W(&sm.pfull[r], pc[r] & 1, kSiteP)) break;
            if (r == 0 && !item(vi)) break;
            tc_fence_after();
            pv(r, vi);
            ++pc[r];
            if (ki >= 0) {
              if (r == 0 && !item(ki)) break;
              tc_fence_after();
              qk(r, ki);
            }
          }
          if (!ok) break;
          mma_commit(&sm.empty[vi % n_slots]);
          if (ki >= 0) mma_commit(&sm.empty[ki % n_slots]);
        }
      } else {
        for (int j = 0; ok && j < min(2, nt); ++j) {
          if (!item(cnt)) break;
          tc_fence_after();
          qk(j, cnt);
          mma_commit(&sm.empty[cnt % n_slots]);
          ++cnt;
        }
        for (int j = 0; ok && j < nt; ++j) {
          const int r = j & 1;
          if (!W(&sm.pfull[r], pc[r] & 1, kSiteP) || !item(cnt)) break;
          tc_fence_after();
          pv(r, cnt);
          ++pc[r];
          mma_commit(&sm.empty[cnt % n_slots]);
          ++cnt;
          if (j + 2 < nt) {
            if (!item(cnt)) break;
            tc_fence_after();
            qk(r, cnt);
            mma_commit(&sm.empty[cnt % n_slots]);
            ++cnt;
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
    // ------------------------------------------------------------- regions
    regs_inc<kRegsRegion>();
    const int r = (warp - 4) >> 2, wq4 = warp & 3;
    const int row = wq4 * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(wq4 * 32) << 16) + r * 256;
    const int mine = a.two ? (r < row_tiles ? nt : 0) : (nt + 1 - r) >> 1;
    const float sl2 = a.scale_log2;
    float ref = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f);
    bool ok = true;
    for (int t = 0; t < mine; ++t) {
      const int j = j0 + (a.two ? t : 2 * t + r);
      const int valid = min(kTile, a.len - j * kTile);  // keys of the tile
      ok = __all_sync(0xffffffffu,
                      mbar_wait_inl(&sm.sfull[r], t & 1, abort, a.err, kSiteS));
      if (!ok) break;
      tc_fence_after();
      // the tile's row maximum
      float mx = -INFINITY;
#pragma unroll 1
      for (int pc = 0; pc < 4; ++pc) {
        uint32_t v[32];
        tmem_ld32(t_row + pc * 32, v);
        tmem_wait_ld();
        if (valid < kTile) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (pc * 32 + i < valid) mx = fmaxf(mx, __uint_as_float(v[i]));
        } else {
          float m1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            mx = fmaxf(mx, __uint_as_float(v[i]));
            m1 = fmaxf(m1, __uint_as_float(v[i + 1]));
          }
          mx = fmaxf(mx, m1);
        }
      }
      mx *= sl2;
      if (mx == -INFINITY) mx = 0.0f;  // scores that are all NaN
      if (t == 0) {
        ref = mx;
      } else {
        const bool grow = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          // O of the tiles before is complete; the next P V waits for this P
          ok = mbar_wait_inl(&sm.odone[r], (t - 1) & 1, abort, a.err, kSiteO);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const float f = grow ? ex2_approx(ref - mx) : 1.0f;
          const float2 f2 = make_float2(f, f);
          if (grow) ref = mx;
          l2 = __fmul2_rn(l2, f2);
#pragma unroll 1
          for (int pc = 0; pc < 8; ++pc) {
            uint32_t v[16];
            tmem_ld16(t_row + 128 + pc * 16, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st16(t_row + 128 + pc * 16, v);
          }
          tmem_wait_st();
        }
      }
      const float2 sc2 = make_float2(sl2, sl2), nr2 = make_float2(-ref, -ref);
#pragma unroll 1
      for (int pc = 0; pc < 4; ++pc) {
        uint32_t v[32], pk[16];
        tmem_ld32(t_row + pc * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 z = __ffma2_rn(
              make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc2, nr2);
          float2 p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
          if (valid < kTile) {
            const int c0 = pc * 32 + 2 * e;
            p = make_float2(c0 < valid ? p.x : 0.f, c0 + 1 < valid ? p.y : 0.f);
          }
          l2 = __fadd2_rn(l2, p);
          pk[e] = pack_bf16x2(p.x, p.y);
        }
        // P over S's first 64 columns: this thread has read columns below 32 (pc + 1)
        tmem_st16(t_row + pc * 16, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.pfull[r]);
    }
    // ---- the partial result of this region's keys
    const int grow_row = (a.two ? (2 * pair + r) * kTile : 0) + row;
    const int part = a.two ? split : 2 * split + r;
    const long long slot =
        (static_cast<long long>(kvh) * a.splits + part) * a.rows_pad + grow_row;
    if (ok && mine > 0) {
      ok = mbar_wait_inl(&sm.odone[r], (mine - 1) & 1, abort, a.err, kSiteO);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int pc = 0; pc < 4; ++pc) {
          uint32_t v[32];
          tmem_ld32(t_row + 128 + pc * 32, v);
          tmem_wait_ld();
          if (grow_row < a.rows) {
            float* dst = a.part_o + slot * kHeadDim + pc * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(dst + 4 * i) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      }
    }
    if ((!a.two || r < row_tiles) && grow_row < a.rows)
      *reinterpret_cast<float2*>(a.part_ml + slot * 2) =
          make_float2(ok && mine > 0 ? ref : -INFINITY, l2.x + l2.y);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace shr

// The split of the prefix over CTAs: the count per KV head (and row pair) whose
// longest chain of tiles is shortest when the CTAs run 148 at a time; a CTA's
// start and end cost about three tiles.
SharedWs shared_ws(long long N, int Hkv, int G, long long prefix, long long cap) {
  SharedWs w{};
  const long long rows = N * G;
  w.rows_pad = static_cast<int>((rows + kTile - 1) / kTile * kTile);
  w.two = rows > kTile ? 1 : 0;
  w.pairs = w.two ? (w.rows_pad / kTile + 1) / 2 : 1;
  w.key_tiles = static_cast<int>((prefix + kTile - 1) / kTile);
  w.ctas_per_head = 0;
  if (w.key_tiles > 0) {
    const long long units = static_cast<long long>(Hkv) * w.pairs;
    long long best = -1;
    for (int c = 1; c <= w.key_tiles && c <= 148; ++c) {
      const long long waves = (units * c + 147) / 148;
      const long long cost = waves * ((w.key_tiles + c - 1) / c + 3);
      if (best < 0 || cost < best) {
        best = cost;
        w.ctas_per_head = c;
      }
    }
  }
  w.splits = w.two ? w.ctas_per_head : 2 * w.ctas_per_head;
  const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const long long chunks = (cap + kGlobalChunk - 1) / kGlobalChunk;
  const size_t pre_rows = static_cast<size_t>(Hkv) * w.splits * w.rows_pad;
  const size_t own_rows = static_cast<size_t>(N) * Hkv * chunks * G;
  w.qs = 0;
  w.pre_o = up(static_cast<size_t>(2) * Hkv * w.rows_pad * kHeadDim * 2);
  w.pre_ml = w.pre_o + up(pre_rows * kHeadDim * 4);
  w.part_o = w.pre_ml + up(pre_rows * 8);
  w.part_ml = w.part_o + up(own_rows * kHeadDim * 4);
  w.total = w.part_ml + up(own_rows * 8);
  return w;
}

int launch_prefix(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                  const PrefixArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != SWA_OK) return rc;
  static std::atomic<int> configured[64];  // per device
  if (!configured[di.device].load(std::memory_order_acquire)) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, shr::prefix_attn_kernel);
    if (e != cudaSuccess) return map_cuda_error(e);
    if (attr.numRegs != shr::kRegsLaunch) return SWA_ERR_UNSUPPORTED;
    e = cudaFuncSetAttribute(shr::prefix_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(shr::Smem)));
    if (e != cudaSuccess) return map_cuda_error(e);
    configured[di.device].store(1, std::memory_order_release);
  }
  const long long grid = static_cast<long long>(a.Hkv) * a.ctas_per_head * a.pairs;
  if (grid > 0x7fffffffLL) return SWA_ERR_UNSUPPORTED;
  return launch_dependent(shr::prefix_attn_kernel, static_cast<unsigned>(grid), shr::kThreads,
                          sizeof(shr::Smem), stream, tq, tk, tv, a);
}

}  // namespace swa
