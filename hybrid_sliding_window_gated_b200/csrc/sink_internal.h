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
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* g;
  const float* wq;
  const float* wk;
  uint16_t* o;
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

int launch_sink_fwd(const SinkFwdArgs& a, cudaStream_t stream);

}  // namespace swa
