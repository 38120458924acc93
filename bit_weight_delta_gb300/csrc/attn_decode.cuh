// attn_decode.cuh — attention of short query runs (a decode step's single
// tokens, or a few tokens) over the paged cache.
//
// A run has at most 16·RT rows per key head (query tokens x query heads per
// key head), so each key and value byte feeds few products and the kernel's
// floor is reading the cache once.  The batch's keys, in units of 16, key head
// by key head and sequence by sequence, are cut evenly over the warps; a run
// cut between them leaves partial results that the combine kernel joins.
//
// Where a CTA's whole range lies in one run its warps (W of them) take the
// run's 16-key tiles in turn; elsewhere each walks its own range.  A warp has its own
// ring of stages that it fills itself by TMA (one box of 16 keys for K, one
// for V, in the 128-byte swizzle), so warps never wait for one another but at
// the end of a run.  Scores are mma.sync m16n8k16 products of the rows with 16
// keys; the softmax statistics and the output stay in registers; at the end of
// a run the warps' results are joined in shared memory.
//
// Measured (64 query and 8 key heads of 128, in the decode kernel): 64 tokens
// over 500 to 8000 keys each, 1.12 GB of cache, 175 us, 6.4 TB/s; one token
// over 131071 keys, 537 MB, 87.2 us, 6.2 TB/s, of which the launch, the first
// pages' latency and the join are about 8; 8 tokens over 120 to 1000 keys, 10.7
// us, bound by that latency.  Taking two tiles at a time won 2.5% on the one long
// context and lost as much on the 8 tokens.
#pragma once

#include <cstdint>

#include "attention.cuh"

namespace bd {
namespace attn_decode {

template <int D, int RT, int W>
struct Cfg {
  static constexpr int kRows = 16 * RT;
  static constexpr int kKv = 16 * D * 2;  // K (or V) bytes of a stage
  static constexpr int kStage = 2 * kKv;
  // 24 KB of ring per warp (16 KB for 32 rows, whose join needs more)
  static constexpr int kStages = (RT == 1 ? 24576 : 16384) / kStage;
  static constexpr int kMerge = kRows * D * 4;  // one warp's o
  static constexpr int kOffMerge = W * kStages * kStage;
  static constexpr int kOffM = kOffMerge + W / 2 * kMerge;  // [warps][rows] m
  static constexpr int kOffL = kOffM + W * kRows * 4;       // [warps / 2][rows] l
  static constexpr int kOffBar = kOffL + W / 2 * kRows * 4;
  static constexpr int kSmem = kOffBar + W * kStages * 8 + 16;
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A walk over the runs in a CTA's range of units.
struct Walk {
  SeqRec r;
  int seq, h;          // current run
  int at, end;         // next unit, end of the range
  int t0, t1;          // the run's 16-key tiles in the range
  int u0;              // the run's first unit
  bool whole;          // the range holds all of the run
};

// The run at w.at; false at the end of the range.
__device__ __forceinline__ bool next_run(const AttnArgs& p, Walk& w) {
  if (w.at >= w.end) return false;
  while (true) {  // units beyond the current sequence belong to a later one
    const int rel = w.at - w.r.unit0;
    if (rel < w.r.units * p.b.n_kv_heads) {
      w.h = static_cast<int>(static_cast<uint32_t>(rel) / static_cast<uint32_t>(w.r.units));
      break;
    }
    if (++w.seq >= p.b.n_seq) return false;
    w.r = p.seqs()[w.seq];
  }
  w.u0 = w.r.unit0 + w.h * w.r.units;
  const int stop = w.u0 + w.r.units < w.end ? w.u0 + w.r.units : w.end;
  w.whole = w.at == w.u0 && stop == w.u0 + w.r.units;
  static_assert(kUnitKeys == 16, "a unit is a tile");
  w.t0 = w.at - w.u0;
  w.t1 = stop - w.u0;
  w.at = stop;
  return true;
}

template <int W>
__device__ __forceinline__ void sync_warps() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
}

// The work of one CTA's warps 0 .. W − 1: the plan's decode range `cta`.
// `smem` is 1024-byte aligned; warp 0's lane 0 must have set `*abort` to 0 and
// every warp initialised its barriers (init) before a CTA-wide barrier.
template <int D, int RT, int W>
__device__ __forceinline__ void init(uint8_t* smem, int warp, int lane) {
  using C = Cfg<D, RT, W>;
  if (warp < W && lane == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 1);
    if (warp == 0) *reinterpret_cast<volatile int*>(smem + C::kOffBar + W * C::kStages * 8) = 0;
  }
  fence_mbar_init();
}

template <int D, int RT, int W>
__device__ __forceinline__ void run(const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                                    const AttnArgs& p, uint8_t* smem, int warp, int lane,
                                    int cta) {
  using C = Cfg<D, RT, W>;
  constexpr int kKSteps = D / 16;
  const bd_attention_batch& b = p.b;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffBar + W * C::kStages * 8);
  uint8_t* ring = smem + warp * C::kStages * C::kStage;
  float* s_m = reinterpret_cast<float*>(smem + C::kOffM);
  float* s_l = reinterpret_cast<float*>(smem + C::kOffL);

  // A CTA whose whole range lies in one run works on it with all its warps
  // (tiles in turn, joined at the end); elsewhere each warp walks its own range
  // and writes its own rows and parts, with no exchange.
  const PlanHeader hd = *p.header();
  const DecodeStart st0 = p.starts()[cta * W], mine = p.starts()[cta * W + warp];
  if (st0.lo >= st0.hi) return;
  const int span = hd.d_per * W;
  const int cta_hi = st0.lo < hd.d_units - span ? st0.lo + span : hd.d_units;
  const uint32_t units = static_cast<uint32_t>(st0.r.units);
  const uint32_t run0 = static_cast<uint32_t>(st0.lo - st0.r.unit0) / units * units;
  const bool together = st0.r.unit0 + run0 + units >= static_cast<uint32_t>(cta_hi);
  if (!together && mine.lo >= mine.hi) return;
  const int step = together ? W : 1, skew = together ? warp : 0;
  const int lo = together ? st0.lo : mine.lo;
  Walk cons{};
  cons.seq = together ? st0.seq : mine.seq;
  cons.r = together ? st0.r : mine.r;
  cons.at = lo;
  cons.end = together ? cta_hi : mine.hi;
  Walk prod = cons;
  const int g = p.L.g;
  const int page_shift = 31 - __clz(b.page_size);
  const int64_t cache_rows = b.n_pages * b.n_kv_heads * b.page_size;

  // ---- producer: the warp's tiles of every run in turn
  int p_tile = 0, p_end = 0, p_page = 0, p_have = 0;
  int p_stage = 0;
  const auto issue = [&]() {
    while (p_tile >= p_end) {
      if (!next_run(p, prod)) return;
      p_tile = prod.t0 + skew;
      p_end = prod.t1;
      p_have = 32;
    }
    if (p_have == 32) {  // page ids of the next 32 tiles, one per lane
      const int tile = p_tile + step * lane;
      p_page = -1;
      if (tile < p_end) {
        p_page = b.page_table[static_cast<int64_t>(prod.seq) * b.table_stride +
                              ((prod.r.k0 + 16 * tile) >> page_shift)];
        if (p_page < 0 || p_page >= b.n_pages) {
          record_error(p.ctx, kErrBounds);
          p_page = -1;
        }
      }
      p_have = 0;
    }
    const int page = __shfl_sync(0xFFFFFFFFu, p_page, p_have);
    if (lane == 0) {
      const int key = prod.r.k0 + 16 * p_tile;
      // a page outside the cache reads as zeros (rows past the tensor)
      const int64_t row =
          page < 0 ? cache_rows
                   : (static_cast<int64_t>(page) * b.n_kv_heads + prod.h) * b.page_size +
                         (key & (b.page_size - 1));
      uint8_t* dst = ring + p_stage * C::kStage;
      mbar_arrive_expect_tx(&bars[p_stage], C::kStage);
      tma_load_3d(dst, &tmap_k, &bars[p_stage], 0, static_cast<int32_t>(row), 0);
      tma_load_3d(dst + C::kKv, &tmap_v, &bars[p_stage], 0, static_cast<int32_t>(row), 0);
    }
    ++p_have;
    p_tile += step;
    p_stage = p_stage + 1 == C::kStages ? 0 : p_stage + 1;
  };
  for (int s = 0; s < C::kStages; ++s) issue();

  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  while (next_run(p, cons)) {
    const SeqRec r = cons.r;
    const int rows = r.q_len * g;
    const int pos0 = r.kv_len - r.q_len;  // the first token's position
    uint32_t qf[RT][kKSteps][4];
    int limit[RT][2];                     // keys below it are seen by rows g8, g8 + 8
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      const uint16_t* src[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * m + 8 * e + g8;
        limit[m][e] = row < rows ? pos0 + row / g + 1 : 0;
        src[e] = row < rows ? p.q + (static_cast<int64_t>(r.tok0 + row / g) * b.n_q_heads +
                                     cons.h * g + row % g) * D + 2 * t4
                            : nullptr;
      }
#pragma unroll
      for (int k = 0; k < kKSteps; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint16_t* s = src[x & 1];
          qf[m][k][x] =
              s ? __ldg(reinterpret_cast<const uint32_t*>(s + 16 * k + 8 * (x >> 1))) : 0u;
        }
    }
    float o[RT][D / 8][4], mref[RT][2], l[RT][2];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[m][n][x] = 0.f;
      mref[m][0] = mref[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }

    for (int tile = cons.t0 + skew; tile < cons.t1; tile += step) {
      ok = ok && mbar_wait(&bars[stage], phase, p.ctx, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const uint32_t kb = smem_addr(ring + stage * C::kStage);
      const uint32_t vb = kb + C::kKv;
      const int key0 = r.k0 + 16 * tile;
      // two chains of products per score, each half as long (the two row tiles of
      // 32 rows are two chains already)
      constexpr int kChains = RT == 1 ? 2 : 1;
      float s[RT][2][4], part[kChains][RT][2][4];
#pragma unroll
      for (int c = 0; c < kChains; ++c)
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) part[c][m][n][x] = 0.f;
      {
        const int tok = (lane & 7) + ((lane & 16) ? 8 : 0), sel = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < kKSteps; ++k) {
          uint32_t kf[4];
          ldsm_x4(kf, kb + (k >> 2) * 2048 + tok * 128 +
                          (((((k & 3) << 1) + sel) ^ (tok & 7)) << 4));
#pragma unroll
          for (int m = 0; m < RT; ++m) {
            mma16816(part[k % kChains][m][0], qf[m][k], kf[0], kf[1]);
            mma16816(part[k % kChains][m][1], qf[m][k], kf[2], kf[3]);
          }
        }
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              s[m][n][x] = kChains == 2 ? part[0][m][n][x] + part[kChains - 1][m][n][x]
                                        : part[0][m][n][x];
      }
      const bool edge = key0 + 16 > pos0 + 1;  // some row does not see all 16 keys
      if (edge) {
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (key0 + 8 * n + 2 * t4 + (x & 1) >= limit[m][x >> 1]) s[m][n][x] = -INFINITY;
      }
      uint32_t pf[RT][4];
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(fmaxf(s[m][0][2 * e], s[m][0][2 * e + 1]),
                         fmaxf(s[m][1][2 * e], s[m][1][2 * e + 1])) * p.scale_log2;
        }
        // each lane looks at its own scores; the row's maximum is exchanged only
        // where one of them moves the reference
        const bool move = top[0] > mref[m][0] + kRescale || top[1] > mref[m][1] + kRescale;
        if (__any_sync(0xFFFFFFFFu, move)) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 2));
            const float mn = fmaxf(mref[m][e], top[e]);
            f[e] = mn == -INFINITY ? 1.f : ex2(mref[m][e] - mn);
            mref[m][e] = mn;
            l[m][e] *= f[e];
          }
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[m][n][x] *= f[x >> 1];
        }
        float w[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float ref = mref[m][x >> 1] == -INFINITY ? 0.f : mref[m][x >> 1];
            w[n][x] = ex2(fmaf(s[m][n][x], p.scale_log2, -ref));
            l[m][x >> 1] += w[n][x];
          }
        // the weights as the A operand of the product with V, rounded to bf16:
        // the tensor core's operand type, 2^-9 of each weight
        pf[m][0] = pack_bf16x2_rn(w[0][0], w[0][1]);
        pf[m][1] = pack_bf16x2_rn(w[0][2], w[0][3]);
        pf[m][2] = pack_bf16x2_rn(w[1][0], w[1][1]);
        pf[m][3] = pack_bf16x2_rn(w[1][2], w[1][3]);
      }
      {
        const int tok = lane & 15, sel = lane >> 4;
        // values past kv_len may be anything and must not meet a zero weight
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        const bool tail = key0 + 16 > r.kv_len;
        if (tail) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = key0 + 8 * e + 2 * t4;
            keep[e] = (k < r.kv_len ? 0xFFFFu : 0u) | (k + 1 < r.kv_len ? 0xFFFF0000u : 0u);
          }
        }
#pragma unroll
        for (int d = 0; d < kKSteps; ++d) {
          uint32_t vf[4];
          ldsm_x4_t(vf, vb + (d >> 2) * 2048 + tok * 128 +
                            (((((d & 3) << 1) + sel) ^ (tok & 7)) << 4));
          if (tail) {
            vf[0] &= keep[0];
            vf[1] &= keep[1];
            vf[2] &= keep[0];
            vf[3] &= keep[1];
          }
#pragma unroll
          for (int m = 0; m < RT; ++m) {
            mma16816(o[m][2 * d], pf[m], vf[0], vf[1]);
            mma16816(o[m][2 * d + 1], pf[m], vf[2], vf[3]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      issue();
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[m][e] += __shfl_xor_sync(0xFFFFFFFFu, l[m][e], 1);
        l[m][e] += __shfl_xor_sync(0xFFFFFFFFu, l[m][e], 2);
        if (together && t4 == 0) s_m[warp * C::kRows + 16 * m + 8 * e + g8] = mref[m][e];
      }
    if (together) {
      // ---- join the warps: m, then o and l relative to the common m
      sync_warps<W>();
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * m + 8 * e + g8;
          float top = s_m[row];
#pragma unroll
          for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w * C::kRows + row]);
          f[e] = top == -INFINITY ? 1.f : ex2(mref[m][e] - top);
          mref[m][e] = top;
          l[m][e] *= f[e];
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[m][n][x] *= f[x >> 1];
      }
      const auto put = [&](int slot) {
        float4* d = reinterpret_cast<float4*>(smem + C::kOffMerge + slot * C::kMerge) + lane;
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            d[(m * (D / 8) + n) * 32] = make_float4(o[m][n][0], o[m][n][1], o[m][n][2], o[m][n][3]);
        if (t4 == 0)
#pragma unroll
          for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) s_l[slot * C::kRows + 16 * m + 8 * e + g8] = l[m][e];
      };
      const auto add = [&](int slot) {
        const float4* d =
            reinterpret_cast<const float4*>(smem + C::kOffMerge + slot * C::kMerge) + lane;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const float4 v = d[(m * (D / 8) + n) * 32];
            o[m][n][0] += v.x;
            o[m][n][1] += v.y;
            o[m][n][2] += v.z;
            o[m][n][3] += v.w;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) l[m][e] += s_l[slot * C::kRows + 16 * m + 8 * e + g8];
        }
      };
      // halves of the remaining warps, one onto the other; a warp's slot is one
      // that nobody but itself has still to read
#pragma unroll
      for (int half = W / 2; half >= 1; half /= 2) {
        const int first = half == W / 2 ? W / 2 : 0;
        if (warp >= half && warp < 2 * half) put(warp - first);
        sync_warps<W>();
        if (warp < half) add(warp + half - first);
      }
      if (warp != 0) continue;
    }

    // ---- final rows, or a partial result
    const bool last = cons.whole && r.group < 0;
    uint8_t *po, *pml;
    int64_t slot;
    int part_rows;
    if (cons.whole) {
      po = p.ws + p.L.w_r_o;
      pml = p.ws + p.L.w_r_ml;
      part_rows = g;
    } else {
      // a cut run is the warp's last one (it begins there) or its first
      slot = 2 * (static_cast<int64_t>(cta) * W + (together ? 0 : warp)) +
             (!together && cons.u0 >= lo ? 1 : 0);
      po = p.ws + p.L.w_d_o;
      pml = p.ws + p.L.w_d_ml;
      part_rows = p.L.d_rows;
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * m + 8 * e + g8;
        if (row >= rows) continue;
        const int64_t tok = r.tok0 + row / g;
        const int64_t at = tok * b.n_q_heads + cons.h * g + row % g;
        if (last) {
          const float inv = l[m][e] != 0.f ? 1.f / l[m][e] : 0.f;  // (a NaN goes through)
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D) + t4;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            dst[4 * n] = pack_bf16x2_rn(o[m][n][2 * e] * inv, o[m][n][2 * e + 1] * inv);
          if (t4 == 0 && p.lse != nullptr)
            p.lse[at] = l[m][e] != 0.f ? (mref[m][e] + log2f(l[m][e])) * kLn2 : -INFINITY;
          continue;
        }
        int part_row = row;
        if (cons.whole) {
          slot = tok * b.n_kv_heads + cons.h;
          part_row = row % g;
        }
        float2* dst = reinterpret_cast<float2*>(part_o(po, slot, part_rows, D));
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          const int d = 8 * n + 2 * t4;
          dst[(static_cast<int64_t>(d >> 2) * part_rows + part_row) * 2 + ((d >> 1) & 1)] =
              make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
        }
        if (t4 == 0)
          part_ml(pml, slot, part_rows)[part_row] = make_float2(mref[m][e], l[m][e]);
      }
  }
  // After a wait that gave up, loads may still be in flight: see them land.
  if (!ok)
    for (int s = 0; s < C::kStages; ++s) {
      const int i = (stage + s) % C::kStages;
      mbar_wait(&bars[i], phase ^ (stage + s >= C::kStages ? 1u : 0u), p.ctx, nullptr);
    }
}

}  // namespace attn_decode
}  // namespace bd
