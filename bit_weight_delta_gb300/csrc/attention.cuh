// attention.cuh — what the attention's kernels share: the plan's layout, the
// partial results' layout and the launchers.
//
// A batch's work falls in two kinds of run.  Short runs (a sequence with at
// most d_rows query rows per key head, i.e. query tokens x query heads per key
// head) are the decode role's, whose time is reading the cache.  Long runs are
// the tile role's, on the tensor cores: sequences with more rows, over their
// own keys, and groups of sequences, over their shared prefix.  A batch that
// can only hold short runs runs the decode kernel; any other the tile kernel,
// some of whose CTAs take the decode role, as many as the plan finds that the
// two kinds of work end together.  Rows whose keys
// are spread over several pieces (a key range cut over CTAs, a prefix and an
// own part) are joined by the combine kernel from partial results
//   o = Σ 2^(s − m)·v,  l = Σ 2^(s − m),  m      (s in units of log2)
// as Σ 2^(m_i − M)·o_i / Σ 2^(m_i − M)·l_i with M = max m_i.
#pragma once

#include <cstdint>

#include "bitdelta_block.h"
#include "kernels.h"

namespace bd {

constexpr int kTileKeys = 128;   // keys per block of the tile kernel
constexpr int kHalfRows = 128;   // rows per half of its 256-row tile (tensor-memory lanes)
constexpr int kUnitKeys = 16;    // keys per unit of the decode role's split
constexpr int kDecodeWarps = 4;      // warps per CTA of the decode kernel
constexpr int kTileDecodeWarps = 8;  // of the tile kernel's decode role
constexpr int kMinUnits = 4;     // units per warp at least: a part costs a row's sums

struct PlanHeader {
  int32_t d_units;    // units of the decode role, all sequences and key heads
  int32_t d_per;      // units per warp
  int32_t d_warps;    // warps per CTA
  int32_t t_entries;  // pieces of the tile kernel (each once per key head)
  int32_t t_ctas;     // CTAs of its launch that take pieces; the others take units
  int32_t n_comb;     // tokens whose rows the combine kernel writes
  int32_t next_piece; // the tile kernel's dealing: t_ctas between calls
};

// The decode role's parts of a run of units [u0, u1), out of `total` units cut
// into `per` per warp and `w` warps per CTA.  A CTA whose whole range lies in
// one run works on it with all its warps and leaves one part; elsewhere each
// warp has a range, and parts, of its own.  A run's parts are thus those of the
// warps of its first CTA, one of each CTA in between, and those of the warps of
// its last CTA.  A part's slot is 2·warp, plus one where the run begins inside
// the range of its warp (a warp has at most one part that began earlier and one
// that goes on).
struct DecodeParts {
  int g0;            // first warp (or first warp of the first CTA)
  int mid0;          // first warp of the CTAs in between
  int last0;         // first warp of the last parts
  int na, nb, nc;    // parts of the first CTA, in between, of the last CTA
  int w, first_odd;  // warps per CTA; 1 where the first part's slot is the odd one
  __host__ __device__ int count() const { return na + nb + nc; }
  __host__ __device__ int slot(int i) const {
    if (i < na) return 2 * (g0 + i) + (i == 0 ? first_odd : 0);
    if (i < na + nb) return 2 * (mid0 + (i - na) * w);
    return 2 * (last0 + (i - na - nb));
  }
};
// (Units are counted in 31 bits, which the plan checks: 64-bit divisions took
// most of a microsecond here.)
__host__ __device__ inline DecodeParts decode_parts(uint32_t u0, uint32_t u1, uint32_t total,
                                                    uint32_t per, uint32_t w) {
  DecodeParts d{};
  const uint32_t w0 = u0 / per, w1 = (u1 - 1) / per, c0 = w0 / w, c1 = w1 / w;
  const uint32_t span = per * w;
  const uint32_t end0 = (c0 + 1) * span < total ? (c0 + 1) * span : total;
  const uint32_t end1 = (c1 + 1) * span < total ? (c1 + 1) * span : total;
  d.w = static_cast<int>(w);
  if (u0 <= c0 * span && u1 >= end0) {  // all of the first CTA
    d.g0 = static_cast<int>(c0 * w);
    d.na = 1;
  } else {
    d.g0 = static_cast<int>(w0);
    d.na = static_cast<int>((c0 == c1 ? w1 : (c0 + 1) * w - 1) - w0) + 1;
    d.first_odd = 1;
  }
  if (c1 > c0) {
    d.mid0 = static_cast<int>((c0 + 1) * w);
    d.nb = static_cast<int>(c1 - c0 - 1);
    d.last0 = static_cast<int>(c1 * w);
    d.nc = u1 >= end1 ? 1 : static_cast<int>(w1 - c1 * w) + 1;
  }
  return d;
}

// One sequence, as the decode role and the combine kernel see it.
struct SeqRec {
  int32_t unit0;      // first of its decode units (key head h: + h · units per head)
  int32_t units;      // decode units per key head (0: none, or a tile-role run)
  int32_t tok0, q_len, kv_len;
  int32_t k0;         // first own key (the shared prefix ends there)
  int32_t group;      // group whose prefix it reads, or −1
  int32_t pad;
};

// Where a warp of the decode role begins: its units [lo, hi) and the sequence
// that holds lo.  One load, so that its first page ids are one step away.
struct DecodeStart {
  SeqRec r;
  int32_t lo, hi;
  int32_t seq;
};

// A token whose rows the combine kernel writes, and where its parts lie.  Own
// part: tile slots own_slot .. (own_ns of them, rows from own_row), or decode
// units (units > 0: rows from own_row, the slots following from the head's
// units).  Prefix part: pre_ns tile slots.
struct CombItem {
  int32_t unit0, units;
  int32_t tok;
  int32_t own_slot, own_ns, own_row;
  int32_t pre_slot, pre_ns, pre_row;
};

// One piece of the tile kernel's work: a tile of query tokens by a range of
// 128-key blocks.
struct TileEntry {
  int32_t tok0, n_tok;   // query tokens
  int32_t seq;           // whose page-table row is read
  int32_t k_lo, k_hi;    // keys of the tile; block b starts at k_lo + 128·b
  int32_t causal;        // token t sees keys below min(k_hi, t + causal)
  int32_t b0, b1;        // blocks of this piece
  int32_t slot;          // partial slot (times n_kv_heads plus head), or −1: final
  int32_t tail;          // values past k_hi in its 16-key step may hold anything
  int32_t pad0, pad1;
};

// Sizes that the host fixes for a batch, and where everything lies.
struct AttnLayout {
  int32_t g;             // query heads per key head
  int32_t half_tok;      // tokens per half tile
  int32_t d_rows;        // rows up to which a run is short
  int32_t d_ctas;        // CTAs of the decode kernel
  int32_t d_warps;       // warps that take the decode role in either kernel, at most
  int32_t t_ctas;        // CTAs of the tile kernel
  bool use_tile;
  int64_t max_tiles, max_entries, t_slots;
  // plan
  size_t o_tok_seq, o_seq, o_start, o_group, o_run, o_tile_slot, o_tile_ns, o_entry, o_comb;
  size_t plan_bytes;
  // workspace: O then (m, l) of each
  size_t w_d_o, w_d_ml, w_r_o, w_r_ml, w_t_o, w_t_ml;
  size_t ws_bytes;
};
AttnLayout attn_layout(const bd_attention_batch& b, int num_sms);

struct AttnArgs {
  bd_attention_batch b;
  AttnLayout L;
  uint8_t* plan;
  uint8_t* ws;
  const uint16_t *q, *k_pages, *v_pages;
  float scale_log2;
  uint16_t* out;
  float* lse;
  DevCtx ctx;

  __host__ __device__ const PlanHeader* header() const {
    return reinterpret_cast<const PlanHeader*>(plan);
  }
  __device__ int* piece_counter() const {
    return &reinterpret_cast<PlanHeader*>(plan)->next_piece;
  }
  __host__ __device__ const SeqRec* seqs() const {
    return reinterpret_cast<const SeqRec*>(plan + L.o_seq);
  }
  __host__ __device__ const DecodeStart* starts() const {
    return reinterpret_cast<const DecodeStart*>(plan + L.o_start);
  }
  __host__ __device__ const TileEntry* entries() const {
    return reinterpret_cast<const TileEntry*>(plan + L.o_entry);
  }
  __host__ __device__ const CombItem* comb() const {
    return reinterpret_cast<const CombItem*>(plan + L.o_comb);
  }
};

// Partial results.  A slot of R rows holds o as [D/4][R] float4 (four
// neighbouring elements of a row together, neighbouring rows next to them) and
// (m, l) as [R] float2.
__device__ __forceinline__ float4* part_o(uint8_t* base, int64_t slot, int rows, int dim) {
  return reinterpret_cast<float4*>(base) + slot * rows * (dim / 4);
}
__device__ __forceinline__ float2* part_ml(uint8_t* base, int64_t slot, int rows) {
  return reinterpret_cast<float2*>(base) + slot * rows;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLn2 = 0.69314718055994531f;

// The running reference m of a row's softmax follows its maximum only in steps
// of more than this (log2 units).  Any reference within the exponents' range
// gives the same relative precision (weights are fp32 and bf16, sums fp32): a
// row's weights are at most 2^40 and 2^30 of them, times |v|, stay inside fp32,
// and the sums are seldom rescaled.
constexpr float kRescale = 40.f;

cudaError_t launch_attn_decode(const AttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s);
// Tensor maps of the query rows, of the cache in boxes of a page's panel (tile
// role) and in boxes of 16 keys (decode role).
struct TileMaps {
  CUtensorMap q, k, v, dk, dv;
};
cudaError_t launch_attn_tile(const AttnArgs& a, const TileMaps& maps, cudaStream_t s);

// Tensor map of up to 3 dimensions of 16-bit elements in the 128-byte swizzle;
// strides in bytes of dimensions 1 and 2.
bool encode_tmap_bf16_3d(CUtensorMap* map, const void* base, const uint64_t (&dims)[3],
                         const uint64_t (&strides)[2], const uint32_t (&box)[3]);

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace bd
