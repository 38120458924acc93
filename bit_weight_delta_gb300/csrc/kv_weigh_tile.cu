// kv_weigh_tile.cu — attention weights of cached keys for runs of many query rows
// (prompts, chunks, the rows of a whole group over its prefix), on the tensor cores.
//
// With the keys as the product's M rows,
//   Sᵀ = K·Qᵀ   (128 keys x 128 query rows, fp32, in tensor memory),
// a thread of the epilogue owns a key, and its sum over the query rows
//   a = Σ 2^(scale·S − lse)   (log2 units)
// needs no exchange between threads.  A block is 256 keys of a run and key head,
// resident in shared memory while its tiles of 128 query rows pass, each used for
// both halves of the block.  The work is counted in tiles: block after block, and
// every CTA takes an even share of all of them.  A block whose tiles lie in
// several CTAs' shares is summed from their parts, in their order, by the kernel
// that follows.
//
// Warps: 0-3 and 4-7 the epilogues of the block's halves, 8 the MMA issuer, 9 the
// TMA producer of K and Q, 10 loads the rows' lse.  Tensor memory: tile buffer b,
// half h at column 256·b + 128·h.
#include <cstdint>

#include "attention.cuh"
#include "kv_weigh.cuh"
#include "tc_tile.cuh"

namespace bd {
namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kLseWarp = 10;
constexpr int kRows = 128;          // query rows of a tile
constexpr int kPanel = 128 * 128;   // 128 rows x 128 bytes
constexpr int kLseStages = 4;
constexpr uint32_t kTmemCols = 512;

// The rows of a tile: what is subtracted from a score (−lse in log2 units) and the
// last slot that a row sees (−1: a row that does not count), with the least and the
// largest of each 32 of them.
struct Rows {
  float minus[kRows];
  int sees[kRows];
  int least[4], most[4];
};

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kHalfBytes = kPanels * kPanel;  // 128 rows
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kOffQ = 4 * kHalfBytes;  // two blocks of keys before it
  static constexpr int kOffRows = kOffQ + kQStages * kHalfBytes;
  static constexpr int kOffBar = kOffRows + kLseStages * static_cast<int>(sizeof(Rows));
  // k_full[2], k_empty[2], s_full[2], s_empty[2], lse_full[], lse_empty[], q_full[],
  // q_empty[], drain
  static constexpr int kBars = 8 + 2 * kLseStages + 2 * kQStages + 1;
  static constexpr int kOffMisc = (kOffBar + 8 * kBars + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 16 + 1024;  // with slack for alignment
};

// A run as this kernel's work: its blocks, and the tiles of each.
struct TileRun {
  WeighRun x;
  bool group;
  int blocks;
  int n_full, m_full;  // the first m_full blocks are seen from the first token on
  int64_t per_head;    // tiles
  // first token that sees block i
  __device__ __forceinline__ int first_token(int i) const {
    return i < m_full ? x.tok0 : x.k0 + kWeighBlockKeys * i - x.causal;
  }
  __device__ __forceinline__ int tiles(int i, int tok) const {
    return i < m_full ? n_full : (x.tok1 - first_token(i) + tok - 1) / tok;
  }
};

__device__ TileRun tile_run(const WeighArgs& p, int r, int tok) {
  TileRun t{};
  t.x = weigh_run(p, r);
  t.group = r >= p.b.n_seq;
  const int g = p.b.n_q_heads / p.b.n_kv_heads;
  const int n_tok = t.x.tok1 - t.x.tok0;
  if (t.x.k1 <= t.x.k0 || static_cast<int64_t>(n_tok) * g <= kWeighShortRows) return t;
  t.blocks = (t.x.k1 - t.x.k0 + kWeighBlockKeys - 1) / kWeighBlockKeys;
  t.n_full = (n_tok + tok - 1) / tok;
  const int64_t ahead = static_cast<int64_t>(t.x.tok0) + t.x.causal - t.x.k0;
  t.m_full = t.group ? t.blocks
                     : static_cast<int>(ahead < 0 ? 0 : ahead / kWeighBlockKeys + 1);
  if (t.m_full > t.blocks) t.m_full = t.blocks;
  t.per_head = static_cast<int64_t>(t.m_full) * t.n_full;
  for (int i = t.m_full; i < t.blocks; ++i) t.per_head += t.tiles(i, tok);
  return t;
}

// Tiles [j0, j1) of a block.
struct Item {
  int h, i;
  int key0;       // the block's first slot
  int first;      // token of tile 0
  int j0, j1, n;  // n: tiles of the block
};

// A CTA's share, item after item; every role walks it for itself.
struct Walk {
  TileRun t;
  int64_t left;
  int run, h, i, j;

  __device__ __forceinline__ bool next(const WeighArgs& p, int tok, Item& it) {
    if (left <= 0) return false;
    while (h == p.b.n_kv_heads) {  // (there is a further run: left counts its tiles)
      t = tile_run(p, ++run, tok);
      if (t.per_head > 0) h = 0;
    }
    it.h = h;
    it.i = i;
    it.key0 = t.x.k0 + kWeighBlockKeys * i;
    it.first = t.first_token(i);
    it.n = t.tiles(i, tok);
    it.j0 = j;
    it.j1 = left < it.n - j ? j + static_cast<int>(left) : it.n;
    left -= it.j1 - it.j0;
    j = it.j1;
    // `t` stays this item's run until the next call
    if (j == it.n) {
      j = 0;
      if (++i == t.blocks) {
        i = 0;
        ++h;
      }
    }
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tile_kernel(const __grid_constant__ WeighMaps maps, const WeighArgs p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_sum[kWarps], s_at;
  __shared__ int s_run;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + 2;
  uint64_t* s_full = k_full + 4;
  uint64_t* s_empty = k_full + 6;
  uint64_t* lse_full = k_full + 8;
  uint64_t* lse_empty = lse_full + kLseStages;
  uint64_t* q_full = lse_empty + kLseStages;
  uint64_t* q_empty = q_full + C::kQStages;
  uint64_t* drain = q_empty + C::kQStages;
  Rows* rows = reinterpret_cast<Rows*>(smem + C::kOffRows);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const bd_attention_batch& b = p.b;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31, tid = threadIdx.x;
  const int G = b.n_q_heads / b.n_kv_heads, tok = kRows / G;
  const int n_run = b.n_seq + b.n_group;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    for (int i = 0; i < kLseStages; ++i) {
      mbar_init(&lse_full[i], 1);
      mbar_init(&lse_empty[i], 8);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    mbar_init(drain, 1);
    *abort = 0;
    s_run = 0;
    s_at = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's share of all tiles, and where it begins
  const bool bad = __syncthreads_or(weigh_breaks_bounds(p));
  int64_t total = 0;
  if (!bad) {
    int64_t mine = 0;
    for (int r = tid; r < n_run; r += kThreads) mine += tile_run(p, r, tok).per_head;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, off);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) total += s_sum[i];
    total *= b.n_kv_heads;
  } else if (tid == 0 && blockIdx.x == 0) {
    record_error(p.ctx, kErrBounds);
  }
  const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  if (hi > lo) {
    int64_t before = 0;
    for (int base = 0; base < n_run && before <= lo; base += kThreads) {
      const int64_t n =
          base + tid < n_run ? tile_run(p, base + tid, tok).per_head * b.n_kv_heads : 0;
      int64_t inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
        if (lane >= off) inc += o;
      }
      __syncthreads();  // the sums before have been read
      if (lane == 31) s_sum[warp] = inc;
      __syncthreads();
      int64_t at = before;
      for (int i = 0; i < kWarps; ++i) {
        if (i == warp) inc += at;
        at += s_sum[i];
      }
      if (inc - n <= lo && lo < inc) {
        s_run = base + tid;
        s_at = lo - (inc - n);
      }
      before = at;
    }
  }
  if (tid < 2) {
    WeighRecord none{};
    p.records[2 * blockIdx.x + tid] = none;
  }
  __syncthreads();
  Walk walk{};
  walk.left = hi - lo;
  walk.run = s_run;
  if (walk.left > 0) {
    walk.t = tile_run(p, walk.run, tok);
    walk.h = static_cast<int>(s_at / walk.t.per_head);
    int64_t at = s_at - walk.h * walk.t.per_head;
    const int64_t full = static_cast<int64_t>(walk.t.m_full) * walk.t.n_full;
    if (at < full) {
      walk.i = static_cast<int>(at / walk.t.n_full);
      at -= static_cast<int64_t>(walk.i) * walk.t.n_full;
    } else {
      at -= full;
      for (walk.i = walk.t.m_full; at >= walk.t.tiles(walk.i, tok); ++walk.i)
        at -= walk.t.tiles(walk.i, tok);
    }
    walk.j = static_cast<int>(at);
  }
  Item it;
  bool ok = true;

  if (warp < 8) {
    // ============================================================ sums
    const int half = warp >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128u * half;
    const int mine = 128 * half + 32 * (warp & 3) + lane;  // key of the block
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    uint32_t s_phase = 0, l_phase = 0;
    int buf = 0, ls = 0;
    bool started = false;  // an item before this one
    while (ok && walk.next(p, tok, it)) {
      const WeighRun& x = walk.t.x;
      const int key = it.key0 + mine;
      const int key_lo = it.key0 + 128 * half;  // the half's
      const int key_hi = key_lo + 127 < x.k1 - 1 ? key_lo + 127 : x.k1 - 1;
      uint64_t sum[2] = {0u, 0u};
      for (int j = it.j0; j < it.j1; ++j) {
        ok = warp_wait(&lse_full[ls], l_phase, p.ctx, abort) &&
             warp_wait(&s_full[buf], s_phase, p.ctx, abort);
        if (!ok) break;
        tc_fence_after();
        const Rows& rw = rows[ls];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (rw.most[c] < key_lo || key_lo >= x.k1) continue;
          uint32_t s[32];
          tmem_ld_32x32b_x32(t_lane + 256u * buf + 32u * c, s);
          tmem_ld_wait();
          const ulonglong2* m2 = reinterpret_cast<const ulonglong2*>(rw.minus + 32 * c);
          if (rw.least[c] >= key_hi) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const ulonglong2 m = m2[v];
              float e0, e1, e2, e3;
              unpack2(fma2(pack2(__uint_as_float(s[4 * v]), __uint_as_float(s[4 * v + 1])), scale2,
                           m.x), e0, e1);
              unpack2(fma2(pack2(__uint_as_float(s[4 * v + 2]), __uint_as_float(s[4 * v + 3])),
                           scale2, m.y), e2, e3);
              sum[0] = add2(sum[0], pack2(ex2(e0), ex2(e1)));
              sum[1] = add2(sum[1], pack2(ex2(e2), ex2(e3)));
            }
          } else {
            const int4* sees = reinterpret_cast<const int4*>(rw.sees + 32 * c);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const ulonglong2 m = m2[v];
              const int4 z = sees[v];
              float e0, e1, e2, e3;
              unpack2(fma2(pack2(__uint_as_float(s[4 * v]), __uint_as_float(s[4 * v + 1])), scale2,
                           m.x), e0, e1);
              unpack2(fma2(pack2(__uint_as_float(s[4 * v + 2]), __uint_as_float(s[4 * v + 3])),
                           scale2, m.y), e2, e3);
              // (selected, not multiplied: a row that does not count may hold anything)
              sum[0] = add2(sum[0], pack2(key <= z.x ? ex2(e0) : 0.f, key <= z.y ? ex2(e1) : 0.f));
              sum[1] = add2(sum[1], pack2(key <= z.z ? ex2(e2) : 0.f, key <= z.w ? ex2(e3) : 0.f));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_empty[buf]);
          mbar_arrive(&lse_empty[ls]);
        }
        if ((buf ^= 1) == 0) s_phase ^= 1u;
        if (++ls == kLseStages) {
          ls = 0;
          l_phase ^= 1u;
        }
      }
      if (!ok) break;
      float a0, a1;
      unpack2(add2(sum[0], sum[1]), a0, a1);
      const float a = a0 + a1;
      if (it.j0 == 0 && it.j1 == it.n) {
        if (key < x.k1) {
          const int64_t row = weigh_row(b, x.seq, key, it.h);
          if (row >= 0) weigh_add(p, x, key, row, a);
        }
      } else {
        const int slot = 2 * static_cast<int>(blockIdx.x) + (started ? 1 : 0);
        p.parts[static_cast<int64_t>(slot) * kWeighBlockKeys + mine] = a;
        if (tid == 0)
          p.records[slot] = WeighRecord{1, walk.run, it.h, it.i, it.j0 == 0, it.j1 == it.n, 0, 0};
      }
      started = true;
    }
  } else if (warp == kMmaWarp) {
    // ============================================================ MMA issuer
    const bool lead = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(128, kRows);
    const uint32_t base = smem_addr(smem);
    int kb = 0, qs = 0, buf = 0;
    uint32_t k_phase = 0, q_phase = 0, s_phase = 1;
    bool issued = false;
    while (ok && walk.next(p, tok, it)) {
      ok = warp_wait(&k_full[kb], k_phase, p.ctx, abort);
      const bool both = it.key0 + 128 < walk.t.x.k1;  // keys in the second half
      for (int j = it.j0; ok && j < it.j1; ++j) {
        ok = warp_wait(&q_full[qs], q_phase, p.ctx, abort) &&
             warp_wait(&s_empty[buf], s_phase, p.ctx, abort);
        if (!ok) break;
        tc_fence_after();
        issued = true;
        if (lead) {
          const uint64_t qd = sdesc_k_sw128(base + C::kOffQ + qs * C::kHalfBytes);
          for (int h = 0; h < (both ? 2 : 1); ++h) {
            const uint64_t kd = sdesc_k_sw128(base + (2 * kb + h) * C::kHalfBytes);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t step = static_cast<uint64_t>((k >> 2) * (kPanel >> 4) + 2 * (k & 3));
              mma_ss(tmem + 256u * buf + 128u * h, kd + step, qd + step, idesc, k > 0 ? 1u : 0u);
            }
          }
          mma_commit(&s_full[buf]);
          mma_commit(&q_empty[qs]);
          if (j == it.j1 - 1) mma_commit(&k_empty[kb]);
        }
        __syncwarp();
        if ((buf ^= 1) == 0) s_phase ^= 1u;
        if (++qs == C::kQStages) {
          qs = 0;
          q_phase ^= 1u;
        }
      }
      if ((kb ^= 1) == 0) k_phase ^= 1u;
    }
    if (issued) {
      if (lead) mma_commit(drain);
      mbar_wait(drain, 0, p.ctx, nullptr);
    }
    __syncwarp();
  } else if (warp == kTmaWarp) {
    // ============================================================ TMA producer
    const int page_shift = 31 - __clz(b.page_size);
    int kb = 0, qs = 0, k_fill = 0, q_fill = 0;
    uint32_t k_phase = 1, q_phase = 1;
    while (ok && walk.next(p, tok, it)) {
      const WeighRun& x = walk.t.x;
      const int keys = x.k1 - it.key0 < kWeighBlockKeys ? x.k1 - it.key0 : kWeighBlockKeys;
      const int n_pg = (keys + b.page_size - 1) >> page_shift;  // at most 16
      int page = -1;
      if (lane < n_pg) {
        page = b.page_table[static_cast<int64_t>(x.seq) * b.table_stride +
                            ((it.key0 >> page_shift) + lane)];
        if (page >= b.n_pages) page = -1;
        if (page < 0) record_error(p.ctx, kErrBounds);  // its sums go nowhere
      }
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, page >= 0);
      if (!(ok = warp_wait(&k_empty[kb], k_phase, p.ctx, abort))) break;
      if (lane == 0)
        mbar_arrive_expect_tx(&k_full[kb], static_cast<uint32_t>(__popc(live) * b.page_size * 128 *
                                                                 C::kPanels));
      __syncwarp();
      if (page >= 0) {
        const int at = lane << page_shift;  // key of the block
        uint8_t* dst = smem + (2 * kb + (at >> 7)) * C::kHalfBytes + (at & 127) * 128;
#pragma unroll
        for (int c = 0; c < C::kPanels; ++c)
          tma_load_3d(dst + c * kPanel, &maps.k, &k_full[kb], 0,
                      (page * b.n_kv_heads + it.h) << page_shift, c);
      }
      __syncwarp();
      ++k_fill;
      if ((kb ^= 1) == 0) k_phase ^= 1u;
      for (int j = it.j0; j < it.j1; ++j) {
        if (!(ok = warp_wait(&q_empty[qs], q_phase, p.ctx, abort))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[qs], static_cast<uint32_t>(C::kPanels * tok * G * 128));
#pragma unroll
          for (int c = 0; c < C::kPanels; ++c)
            tma_load_3d(smem + C::kOffQ + qs * C::kHalfBytes + c * kPanel, &maps.q, &q_full[qs],
                        64 * c, it.h * G, it.first + j * tok);
        }
        __syncwarp();
        ++q_fill;
        if (++qs == C::kQStages) {
          qs = 0;
          q_phase ^= 1u;
        }
      }
    }
    // See every issued load land (bounded, also after an abort).
    if (lane == 0) {
      for (int f = k_fill > 2 ? k_fill - 2 : 0; f < k_fill; ++f)
        mbar_wait(&k_full[f & 1], static_cast<uint32_t>(f >> 1 & 1), p.ctx, nullptr);
      for (int f = q_fill > C::kQStages ? q_fill - C::kQStages : 0; f < q_fill; ++f)
        mbar_wait(&q_full[f % C::kQStages], static_cast<uint32_t>(f / C::kQStages & 1), p.ctx,
                  nullptr);
    }
    __syncwarp();
  } else if (warp == kLseWarp) {
    // ============================================================ the rows' lse
    const bool windowed = p.window > 0 && p.window < b.max_q_len;
    int ls = 0;
    uint32_t phase = 1;
    while (ok && walk.next(p, tok, it)) {
      const WeighRun& x = walk.t.x;
      const int s1 = walk.t.group ? b.group_offsets[walk.run - b.n_seq + 1] : 0;
      for (int j = it.j0; j < it.j1; ++j) {
        float minus[4];
        int sees[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = 32 * c + lane;
          const int t = it.first + j * tok + row / G;
          minus[c] = 0.f;
          sees[c] = -1;
          if (row < tok * G && t < x.tok1) {
            const float l = p.lse[static_cast<int64_t>(t) * b.n_q_heads + it.h * G + row % G];
            if (isfinite(l) && (!walk.t.group || !windowed || weigh_in_window(p, t, x.seq, s1))) {
              minus[c] = -l * kWeighLog2e;
              sees[c] = walk.t.group ? INT32_MAX : t + x.causal;
            }
          }
        }
        if (!(ok = warp_wait(&lse_empty[ls], phase, p.ctx, abort))) break;
        Rows& rw = rows[ls];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          rw.minus[32 * c + lane] = minus[c];
          rw.sees[32 * c + lane] = sees[c];
          const int least = __reduce_min_sync(0xFFFFFFFFu, sees[c]);
          const int most = __reduce_max_sync(0xFFFFFFFFu, sees[c]);
          if (lane == 0) {
            rw.least[c] = least;
            rw.most[c] = most;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lse_full[ls]);
        if (++ls == kLseStages) {
          ls = 0;
          phase ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch(const WeighArgs& p, const WeighMaps& maps, cudaStream_t s) {
  static_assert(Cfg<D>::kSmem <= 226 * 1024, "shared memory of one CTA");
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(weigh_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Cfg<D>::kSmem);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  return launch_pdl(weigh_tile_kernel<D>, dim3(static_cast<unsigned>(p.tile_ctas)), dim3(kThreads),
                    Cfg<D>::kSmem, s, maps, p);
}

}  // namespace

int weigh_tile_tokens(int heads_per_key_head) { return kRows / heads_per_key_head; }

cudaError_t launch_weigh_tile(const WeighArgs& p, const WeighMaps& maps, cudaStream_t s) {
  return p.b.head_dim == 128 ? launch<128>(p, maps, s) : launch<64>(p, maps, s);
}

}  // namespace bd
