// sink_internal.h -- arguments of the sink-attention kernels (host and device):
// the window layers' attention with the first n_sink tokens of every sequence
// visible to all later ones.
#pragma once
#include "swa_internal.h"

namespace swa {

constexpr int kMaxSink = 16;     // sink tokens: one 16-key block of the tensor-core loops
constexpr int kSinkTile = 64;    // tokens per tile of the prefill and backward kernels

struct SinkFwdArgs {
  int B, T, Hq, Hkv, G;
  int n_sink;
  int half_rot;              // rot_dim / 2 rotated pairs
  int tiles;                 // kSinkTile-token tiles per sequence
  long long total_tiles;     // tiles * B * Hkv
  float scale_log2;          // softmax scale * log2(e)
  float eps;
  int flags;
  const uint16_t* v;         // [B, T, Hkv, D], for rows that are summed key by key
  const float* wq;
  const float* wk;
  uint16_t* o;               // [B, T, Hq, D]
  float* lse;                // [B, Hq, T] or null
  int* err;
  double inv_freq[kMaxPairs];
};

// One decode step over the rings and the sink caches.
struct SinkDecArgs {
  int N, Hq, Hkv, G;
  int n_sink;
  int s8;            // sink rows per stage: n_sink rounded up to 8
  int stages;        // units in flight per CTA (2 or 3, what fits in shared memory)
  int stage_bytes;
  int half_rot;
  int flags;
  float scale_log2;
  float eps;
  const int64_t* pos;
  const uint16_t* q;      // [N, Hq, D]
  const uint16_t* k_new;  // [N, Hkv, D]
  const uint16_t* v_new;
  const uint16_t* g;
  const float* wq;
  const float* wk;
  uint16_t* k_cache;      // [N, Hkv, W, D]
  uint16_t* v_cache;
  uint16_t* k_sink;       // [N, Hkv, n_sink, D]
  uint16_t* v_sink;
  uint16_t* o;            // [N, Hq, D]
  int* err;
  double inv_freq[kMaxPairs];
};

// Prefill -> sink caches: tokens at positions 0 .. n_sink - 1.
struct SinkFillArgs {
  int B, T, Hkv, n_sink, half_rot;
  float eps;
  const uint16_t* k;  // [B, T, Hkv, D], or [T, Hkv, D] rows with starts / lens
  const uint16_t* v;
  const float* wk;
  uint16_t* k_sink;   // [B, Hkv, n_sink, D]
  uint16_t* v_sink;
  const int64_t* starts;
  const int64_t* lens;
  const int64_t* pos0;
  int* err;
  double inv_freq[kMaxPairs];
};

int launch_sink_decode(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tks,
                       const CUtensorMap& tvs, SinkDecArgs a, cudaStream_t stream);
int launch_sink_fill(const SinkFillArgs& a, cudaStream_t stream);

// Backward.  Everything in `ws` is scratch, laid out by sink_bwd_ws; Tp is T
// rounded up to a whole tile, and rows past T hold zeros.
struct SinkBwdArgs {
  int B, T, Tp, Hq, Hkv, G;
  int n_sink;
  int half_rot;
  int tiles;              // kSinkTile-token tiles per sequence
  int flags;
  int chunk, chunks;      // the sinks' pass: tokens per CTA, CTAs per (batch row, KV head)
  int head_parts;         // CTAs of the query-major pass per (KV head, tile)
  float scale, scale_log2, eps;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* g;
  const uint16_t* o;
  const uint16_t* dO;
  const float* lse;       // [B, Hq, T]
  const float* wq;
  const float* wk;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  uint16_t* dg;
  float* dwq;
  float* dwk;
  // Operand rows are 256 bytes of fp16 whose 16-byte chunk c lies at c ^ (t & 7).
  float2* rot;            // [Tp, kMaxPairs]: rot(t w_j)
  uint8_t* kr;            // [B, Hkv, Tp] rows k' / ck, rope order
  uint8_t* vr;            // [B, Hkv, Tp] rows v 2^a, split order
  float* va;              // [B, Hkv, Tp]: a, the exponent that brings max|v| to 1 .. 4 (NaN: not finite)
  uint8_t* qr;            // [B, Hq, Tp] rows q' / cq, rope order
  uint8_t* dr;            // [B, Hq, Tp] rows dA 2^b, split order
  float4* row;            // [B, Hq, Tp]: lse log2(e), b, then D (from o; later D 2^(b + a), a)
  float* bmin;            // [B, Hq, Tp / 16]: least b of 16 rows
  float* amin;            // [B, Hkv, tiles]: least a of the keys the tile's queries may see
  float* dwq_part;        // [B Hkv tiles head_parts, D]
  float* dwk_part;        // [B Hkv tiles, D]
  float* sink_part;       // [B, Hkv, chunks, 2, kMaxSink, D]: dk' (rope order), dv (split order)
  float* sink_sum;        // [B, Hkv, 2, kMaxSink, D]
  int* err;
  double inv_freq[kMaxPairs];
};

// Tokens per CTA of the sinks' pass: fewer where a sequence is short, since a CTA
// takes about 4 us + 3 us per 64 tokens of 4 heads.  The length alone decides, so a
// sequence's gradients are the same bits in every batch.  2 x 1001 tokens of 8 / 2
// heads: 28 us with 512 tokens per CTA, 16 us with 128; 16,384 tokens of 32 / 8: 62 us.
inline int sink_chunk(long long T) { return T <= 4096 ? 128 : 512; }
// Parts of a KV head's G query heads in the query-major pass: as many as keep its CTAs
// to two per SM of 148 (each reads the tile's keys again).  2 x 1001 tokens of 8 / 2
// heads, 64 tiles: 39 us in one part, 19 us in four.
inline int sink_head_parts(long long units, int G) {
  const long long n = 296 / units;
  return static_cast<int>(n < 1 ? 1 : (n > G ? G : n));
}

struct SinkBwdWs {
  size_t rot, kr, vr, va, qr, dr, row, bmin, amin, dwq, dwk, part, sum, total;
};
inline SinkBwdWs sink_bwd_ws(long long B, long long T, int Hq, int Hkv, int n_sink) {
  const size_t Tp = static_cast<size_t>((T + kSinkTile - 1) / kSinkTile) * kSinkTile;
  const size_t tiles = Tp / kSinkTile, hk = static_cast<size_t>(B) * Hkv;
  const size_t hq = static_cast<size_t>(B) * Hq;
  const size_t chunks = n_sink > 0 ? (Tp + sink_chunk(T) - 1) / sink_chunk(T) : 0;
  const size_t parts = hk == 0 || tiles == 0 ? 1 : sink_head_parts(hk * tiles, Hq / Hkv);
  SinkBwdWs w{};
  size_t at = 0;
  const auto take = [&at](size_t n) {
    const size_t r = at;
    at = (at + n + 255) & ~static_cast<size_t>(255);
    return r;
  };
  w.rot = take(Tp * kMaxPairs * 8);
  w.kr = take(hk * Tp * 256);
  w.vr = take(hk * Tp * 256);
  w.va = take(hk * Tp * 4);
  w.qr = take(hq * Tp * 256);
  w.dr = take(hq * Tp * 256);
  w.row = take(hq * Tp * 16);
  w.bmin = take(hq * Tp / 16 * 4);
  w.amin = take(hk * tiles * 4);
  w.dwq = take(hk * tiles * parts * kHeadDim * 4);
  w.dwk = take(hk * tiles * kHeadDim * 4);
  w.part = take(hk * chunks * 2 * kMaxSink * kHeadDim * 4);
  w.sum = take(n_sink > 0 ? hk * 2 * kMaxSink * kHeadDim * 4 : 0);
  w.total = at;
  return w;
}

int launch_sink_bwd(const SinkBwdArgs& a, cudaStream_t stream);

// Tensor maps of the forward: q, g, o in boxes of 64 tokens x 2 heads x 64
// dims, k and v of 64 tokens x 64 dims, and of the first 16 tokens.
struct SinkFwdMaps {
  CUtensorMap q, k, v, g, o, ks, vs;
};
int launch_sink_fwd(const SinkFwdMaps& m, const SinkFwdArgs& a, cudaStream_t stream);

}  // namespace swa
