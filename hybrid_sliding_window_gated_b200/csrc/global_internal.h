// global_internal.h -- arguments of the global causal GQA layer's kernels
// (host and device): the full-length KV-cache writer, the causal prefill
// attention and the decode step over the cache.
#pragma once
#include "swa_internal.h"

namespace swa {

// Write k' = RoPE_p(RMSNorm(k)) (rounded to bf16) and v into slot p of the
// full-length caches.  Prefill: rows (b, t) of k, v [B, T, Hkv, D] at p = t.
// Decode: rows n of k, v [N, Hkv, D] at p = pos[n].
struct GlobalKvArgs {
  int B, T, Hkv;
  int half_rot;
  float eps;
  long long cap;          // cache slots per (sequence, KV head)
  const int64_t* pos;     // decode: [N] positions; prefill: null
  const uint16_t* k;
  const uint16_t* v;
  const float* wk;
  uint16_t* k_cache;      // [B, Hkv, cap, D]
  uint16_t* v_cache;
  int* err;
  double inv_freq[kMaxPairs];
};

struct GlobalFwdArgs {
  int B, T, Hq, Hkv, G;
  int tiles;            // query (and key) tiles per sequence
  int pairs;            // head pairs per KV head: ceil(G / 2)
  long long units;      // tiles * B * Hkv * pairs
  float scale_log2;
  float eps;
  int flags;
  const float* wq;
  const float* wk;
  float* lse;           // [B, Hq, T] or null
  int* err;
  double inv_freq[kMaxPairs];
};

// Decode: each work item is (sequence, KV head, chunk of kGlobalChunk keys);
// its partial result goes to the workspace and a second kernel combines them.
constexpr int kGlobalChunk = 2048;
constexpr int kGlobalMaxGroup = 8;

struct GlobalDecArgs {
  int N, Hq, Hkv, G;
  int half_rot;
  int chunks;           // chunk slots per (sequence, KV head) in the workspace
  int flags;
  float scale_log2;
  float eps;
  long long cap;
  const int64_t* pos;
  const uint16_t* q;    // [N, Hq, D]
  const float* wq;
  float* part_o;        // [N, Hkv, chunks, G, D] fp32
  float* part_ml;       // [N, Hkv, chunks, G, 2] fp32: row maximum (log2 units), row sum
  uint16_t* o;          // [N, Hq, D]
  int* err;
  // Shared prefix (swa_global_decode_shared): the caches hold positions base,
  // base + 1, ..; the prefix's partial results come from prefix_attn_kernel.
  long long base;
  int splits;             // prefix partials per query row (0: no prefix)
  int rows_pad;           // query rows per KV head, rounded up to 128
  const float* pre_o;     // [Hkv, splits, rows_pad, D] fp32
  const float* pre_ml;    // [Hkv, splits, rows_pad, 2] fp32
  const uint16_t* k_new;  // [N, Hkv, D]
  const uint16_t* v_new;
  const float* wk;
  uint16_t* k_cache;      // [N, Hkv, cap, D]
  uint16_t* v_cache;
  uint16_t* qs;           // [2, Hkv, rows_pad, D]: q' as bf16, and what that left over
  double inv_freq[kMaxPairs];
};

struct PrefixArgs {
  int Hkv, rows, rows_pad;
  int pairs;              // 256-row pairs of row tiles (two = 1), or 1 row tile (two = 0)
  int two;                // 1: the two regions hold different rows; 0: different keys
  int splits;             // partial results per row
  int ctas_per_head;      // splits of the key tiles over CTAs
  int key_tiles;          // 128-key tiles of the prefix
  int len;                // prefix length
  float scale_log2;
  int flags;
  float* part_o;
  float* part_ml;
  int* err;
};

// Workspace of the shared-prefix step, in bytes from its start.
struct SharedWs {
  int rows_pad, two, pairs, ctas_per_head, splits, key_tiles;
  size_t qs, pre_o, pre_ml, part_o, part_ml, total;
};
SharedWs shared_ws(long long N, int Hkv, int G, long long prefix, long long cap);

int launch_prefix(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                  const PrefixArgs& a, cudaStream_t stream);
int launch_shared_own(const CUtensorMap& tk, const CUtensorMap& tv, const GlobalDecArgs& a,
                      cudaStream_t stream);
int launch_shared_combine(const GlobalDecArgs& a, cudaStream_t stream);

inline size_t global_decode_ws_bytes(long long N, int Hkv, int G, long long cap) {
  const long long chunks = (cap + kGlobalChunk - 1) / kGlobalChunk;
  const size_t po = static_cast<size_t>(N) * Hkv * chunks * G * kHeadDim * 4;
  const size_t pm = static_cast<size_t>(N) * Hkv * chunks * G * 2 * 4;
  return ((po + 255) & ~static_cast<size_t>(255)) + ((pm + 255) & ~static_cast<size_t>(255));
}

int launch_global_kv(const GlobalKvArgs& a, long long rows, cudaStream_t stream);
int launch_global_fwd(int rot_dim, const CUtensorMap& tq, const CUtensorMap& tk,
                      const CUtensorMap& tv, const CUtensorMap& to, const GlobalFwdArgs& a,
                      cudaStream_t stream);
int launch_global_decode(const CUtensorMap& tk, const CUtensorMap& tv, const GlobalDecArgs& a,
                         cudaStream_t stream);

}  // namespace swa
