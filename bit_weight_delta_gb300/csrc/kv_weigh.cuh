// kv_weigh.cuh — what the two kernels of bitdelta_kv_weigh share: runs of query
// rows over keys, the batch's checks, and the parts of key sums that several CTAs
// of the tile kernel leave.
#pragma once

#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {

constexpr float kWeighLog2e = 1.4426950408889634f;
// Rows (query tokens times query heads per key head) up to which a run is the
// short kernel's.
constexpr int kWeighShortRows = 16;
constexpr int kWeighBlockKeys = 256;  // keys of a block of the tile kernel

// A block of keys that several CTAs share: the sums of CTA c's tiles are in
// parts[2c] (of the block that it began in) or parts[2c + 1] (that it ended in), and
// what they are is in records[2c], [2c + 1].
constexpr uint32_t kWeighPart = 1, kWeighBegins = 2, kWeighEnds = 4;  // the block's first tiles, its last
// Where a key's sum goes, beside a part that begins a block: its row in the tables, to be
// added to; ~row for a slot of the step's own tokens, to be set; or kWeighNowhere.
constexpr int32_t kWeighNowhere = INT32_MIN;

struct WeighArgs {
  bd_attention_batch b;
  const uint16_t* q;
  const float* lse;
  const uint16_t* k_pages;
  float scale_log2;
  int32_t window;
  const int32_t* pos_offset;
  float* weights;
  int32_t* positions;
  int32_t tile_ctas;      // of the tile kernel; 0 where it is not launched
  uint32_t* records;      // [2·tile_ctas]
  float* parts;           // [2·tile_ctas][kWeighBlockKeys]
  int32_t* rows;          // the same
  DevCtx ctx;
};

struct WeighMaps {
  CUtensorMap q, k;
};
cudaError_t launch_weigh_tile(const WeighArgs& p, const WeighMaps& maps, cudaStream_t s);
int weigh_tile_tokens(int heads_per_key_head);  // query tokens of a row tile

#ifdef __CUDACC__

// Query rows and the keys that they look at: a sequence's window of query tokens
// over its own keys, or all of a group's over their shared prefix.
struct WeighRun {
  int seq;         // whose page-table row is read
  int k0, k1;      // slots; none where k1 <= k0
  int tok0, tok1;  // query tokens
  int causal;      // token t sees slots up to t + causal
  int fresh;       // first slot of the step's own tokens
};
constexpr int kWeighSeesAll = 1 << 30;  // causal of a prefix

// The prefix of sequence s (0 outside of every group); the groups are sorted.
__device__ __forceinline__ int weigh_prefix(const bd_attention_batch& b, int s) {
  int lo = 0, hi = b.n_group;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.group_offsets[mid + 1] <= s)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo < b.n_group && b.group_offsets[lo] <= s ? b.prefix_len[lo] : 0;
}

// Run r: the sequences' own, then the groups'.  A run whose entries break the batch's
// bounds is empty and sets *bad.
__device__ __forceinline__ WeighRun weigh_run(const WeighArgs& p, int r, bool* bad) {
  const bd_attention_batch& b = p.b;
  WeighRun x{};
  if (r < b.n_seq) {
    const int lo = b.seq_offsets[r], hi = b.seq_offsets[r + 1], kv = b.kv_len[r];
    const int prefix = b.n_group > 0 ? weigh_prefix(b, r) : 0;
    if (lo < 0 || hi < lo || hi > b.n_tokens || hi - lo > b.max_q_len || kv < 0 ||
        kv > b.max_kv_len || kv > b.table_stride * b.page_size ||
        (prefix > 0 && hi > lo && kv - (hi - lo) < prefix)) {
      *bad = true;
      return x;
    }
    x.seq = r;
    x.k0 = prefix;
    x.k1 = kv;
    x.tok0 = p.window > 0 && hi - lo > p.window ? hi - p.window : lo;
    x.tok1 = hi;
    x.causal = kv - hi;
    x.fresh = kv - (hi - lo);
  } else {
    const int g = r - b.n_seq, a = b.group_offsets[g], e = b.group_offsets[g + 1];
    const int len = b.prefix_len[g];
    if (a < 0 || e < a || e > b.n_seq || len < 0 || len > b.max_kv_len ||
        len % b.page_size != 0) {
      *bad = true;
      return x;
    }
    if (e == a) return x;
    x.seq = a;
    x.k1 = len;
    x.tok0 = b.seq_offsets[a];
    x.tok1 = b.seq_offsets[e];
    x.causal = kWeighSeesAll;
    x.fresh = INT32_MAX;
    // (the sequences check their own offsets; here only what the group's work is cut by)
    if (x.tok0 < 0 || x.tok1 < x.tok0 || x.tok1 > b.n_tokens) {
      *bad = true;
      return WeighRun{};
    }
  }
  if (x.tok1 <= x.tok0) x.k1 = x.k0;
  return x;
}

// Whether token t counts in the window of its sequence, one of [s0, s1).
__device__ __forceinline__ bool weigh_in_window(const WeighArgs& p, int t, int s0, int s1) {
  while (s1 - s0 > 1) {
    const int mid = (s0 + s1) >> 1;
    if (p.b.seq_offsets[mid] <= t)
      s0 = mid;
    else
      s1 = mid;
  }
  return p.b.seq_offsets[s0 + 1] - t <= p.window;
}

#endif  // __CUDACC__

}  // namespace bd
