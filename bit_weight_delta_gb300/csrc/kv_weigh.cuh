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
// parts[2c] (of the block that it began in) or parts[2c + 1] (that it ended in).
struct WeighRecord {
  int32_t used;        // 0: no part
  int32_t run, head, block;
  int32_t begins, ends;  // the block's first tiles, its last ones
  int32_t pad0, pad1;
};

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
  WeighRecord* records;   // [2·tile_ctas]
  float* parts;           // [2·tile_ctas][kWeighBlockKeys]
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

// Run r: the sequences' own, then the groups'.
__device__ __forceinline__ WeighRun weigh_run(const WeighArgs& p, int r) {
  const bd_attention_batch& b = p.b;
  WeighRun x{};
  if (r < b.n_seq) {
    const int lo = b.seq_offsets[r], hi = b.seq_offsets[r + 1], kv = b.kv_len[r];
    x.seq = r;
    x.k0 = b.n_group > 0 ? weigh_prefix(b, r) : 0;
    x.k1 = kv;
    x.tok0 = p.window > 0 && hi - lo > p.window ? hi - p.window : lo;
    x.tok1 = hi;
    x.causal = kv - hi;
    x.fresh = kv - (hi - lo);
  } else {
    const int g = r - b.n_seq, a = b.group_offsets[g], e = b.group_offsets[g + 1];
    x.seq = a;
    x.k1 = e > a ? b.prefix_len[g] : 0;
    x.tok0 = e > a ? b.seq_offsets[a] : 0;
    x.tok1 = e > a ? b.seq_offsets[e] : 0;
    x.causal = kWeighSeesAll;
    x.fresh = INT32_MAX;
  }
  if (x.tok1 <= x.tok0) x.k1 = x.k0;
  return x;
}

// Whether the batch's tables break their bounds (this thread's share of them).
__device__ __forceinline__ bool weigh_breaks_bounds(const WeighArgs& p) {
  const bd_attention_batch& b = p.b;
  const int step = static_cast<int>(blockDim.x);
  bool bad = false;
  for (int g = threadIdx.x; g < b.n_group; g += step) {
    const int a = b.group_offsets[g], e = b.group_offsets[g + 1], len = b.prefix_len[g];
    bad |= a < 0 || e < a || e > b.n_seq || len < 0 || len % b.page_size != 0;
  }
  for (int s = threadIdx.x; s < b.n_seq; s += step) {
    const int lo = b.seq_offsets[s], hi = b.seq_offsets[s + 1], kv = b.kv_len[s];
    bad |= lo < 0 || hi < lo || hi > b.n_tokens || hi - lo > b.max_q_len || kv < 0 ||
           kv > b.max_kv_len || kv > b.table_stride * b.page_size;
    if (b.n_group > 0) {
      const int prefix = weigh_prefix(b, s);
      bad |= prefix > 0 && static_cast<int64_t>(kv) - (hi - lo) < prefix;
    }
  }
  return bad;
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

// The row of slot `key` and head h in the tables beside the cache, or −1.
__device__ __forceinline__ int64_t weigh_row(const bd_attention_batch& b, int seq, int key, int h) {
  const int page = b.page_table[static_cast<int64_t>(seq) * b.table_stride + key / b.page_size];
  if (page < 0 || page >= b.n_pages) return -1;
  return (static_cast<int64_t>(page) * b.n_kv_heads + h) * b.page_size + key % b.page_size;
}

// A key's sum to the table.
__device__ __forceinline__ void weigh_add(const WeighArgs& p, const WeighRun& x, int key,
                                          int64_t row, float a) {
  if (key >= x.fresh) {
    p.weights[row] = a;
    p.positions[row] = key + (p.pos_offset != nullptr ? p.pos_offset[x.seq] : 0);
  } else {
    p.weights[row] += a;
  }
}

#endif  // __CUDACC__

}  // namespace bd
