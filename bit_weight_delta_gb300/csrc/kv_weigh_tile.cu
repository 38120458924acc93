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
// The subtraction of lse is a product as well: three more columns, ones in K and
// −lse/scale in three bf16 parts in Q.  (Read by the epilogue from shared memory it
// took a quarter of a tile's time.)
//
// The keys are the product's A operand from tensor memory, where the epilogue's warps
// put a block once: with both operands in shared memory the two halves' products read
// it at its full rate (128 bytes a clock), and the loads of Q and the epilogue's of
// lse came on top (1650 cycles a tile).
//
// Warps: 0-15 the epilogue, of which a warp has 32 keys of one of the block's halves
// and 64 of a tile's 128 rows (eight warps with all rows took 59 us where these took
// 49); 16 and 17 the halves' MMA issuers (one's waits are then the time of the other's
// products); 18 the TMA producer of K and Q, which also walks through the CTA's share
// and puts its items in a ring for the other roles; 19 loads the rows' lse.
// Tensor memory: the block's halves in columns 0-127, three buffers of 128 columns
// behind them that the halves' products go to in turn.
//
// A block and a tile of 128-element heads are 8.4 MFLOP of products, 1024 cycles of the
// tensor pipe and an eighth more for lse, and 32768 exponentials, 1024 cycles of the
// SM's special function units: the two bound it.  Measured (152 SMs, 64 query and 8 key
// heads of 128): a prompt of 2048 tokens 43.7 us, the tensor pipe 38% and the special
// function units 31% busy; it is a tile's chain of wait, load from tensor memory, sum
// and release, about 2200 cycles, that the three buffers do not hide in full.  The last
// 64 tokens of a prompt over its 8192 keys take 19.6 us, of which the start of a CTA
// (lengths, share, page) is 4, its first block and product 3 and the join by the kernel
// that follows 3.
#include <cstdint>

#include "attention.cuh"
#include "kv_weigh.cuh"
#include "tc_tile.cuh"

namespace bd {
namespace {

constexpr int kSumWarps = 16;
constexpr int kMmaWarp = 16, kTmaWarp = 18, kLseWarp = 19;  // MMA: 16 and 17, a half each
constexpr int kWarps = 20;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 128;          // query rows of a tile
constexpr int kPanel = 128 * 128;   // 128 rows x 128 bytes
constexpr int kLseStages = 4;
constexpr int kSumStages = 4;
constexpr int kBuffers = 3;  // of a half's product
// The products ("units") are numbered in the order of tiles and halves; unit u goes to
// buffer u % 3.  It has barriers u % 6 of its own: one that two units of different
// halves took in turn would let a half that is ahead pass for a phase too early.
constexpr int kUnits = 2 * kBuffers;
struct Unit {
  int u = 0;  // modulo 12
  __device__ __forceinline__ void skip(int n) { u = u + n >= 2 * kUnits ? u + n - 2 * kUnits : u + n; }
  __device__ __forceinline__ int bar() const { return u >= kUnits ? u - kUnits : u; }
  __device__ __forceinline__ uint32_t phase() const { return u >= kUnits ? 1u : 0u; }
  __device__ __forceinline__ uint32_t column() const {
    return 128u + 128u * (bar() >= kBuffers ? bar() - kBuffers : bar());
  }
  __device__ __forceinline__ Unit plus(int n) const {
    Unit x = *this;
    x.skip(n);
    return x;
  }
};
constexpr uint32_t kTmemCols = 512;

// The last slot that each row of a tile sees (−1: a row that does not count), with
// the least and the largest of each 32 of them.
struct Rows {
  int sees[kRows];
  int least[4], most[4];
};
constexpr int kLseBytes = kRows * 64;  // the rows' −lse/scale as operand columns

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kHalfBytes = kPanels * kPanel;  // 128 rows
  static constexpr int kQStages = D == 128 ? 3 : 4;
  static constexpr int kOffQ = 2 * kHalfBytes;  // a block of keys before it
  static constexpr int kOffLse = kOffQ + kQStages * kHalfBytes;
  static constexpr int kOffOnes = kOffLse + kLseStages * kLseBytes;
  static constexpr int kOffRows = kOffOnes + kLseBytes;
  static constexpr int kOffItem = kOffRows + kLseStages * static_cast<int>(sizeof(Rows));
  static constexpr int kOffSum = kOffItem + 4 * 48;  // items
  static constexpr int kOffBar = kOffSum + kSumStages * kWeighBlockKeys * 4;
  // k_full, k_empty, k_ready[2], s_full[], s_empty[], lse_full[], lse_empty[], q_full[],
  // q_empty[], item_full[], item_empty[], sum_full[],
  // drain[2]
  static constexpr int kBars = 4 + 4 * kBuffers + 2 * kLseStages + 2 * kQStages + 2 * 4 + kSumStages + 2;
  static constexpr int kOffMisc = (kOffBar + 8 * kBars + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 16 + 1024;  // with slack for alignment
};

// The row of slot `key` and head h in the tables beside the cache, or −1.
__device__ __forceinline__ int64_t weigh_row(const bd_attention_batch& b, int seq, int key, int h) {
  const int page = b.page_table[static_cast<int64_t>(seq) * b.table_stride + key / b.page_size];
  if (page < 0 || page >= b.n_pages) return -1;
  return (static_cast<int64_t>(page) * b.n_kv_heads + h) * b.page_size + key % b.page_size;
}

// a / b of numbers that are not negative, in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// A run as this kernel's work: its blocks, and the tiles of each.
struct TileRun {
  WeighRun x;
  bool group;
  int blocks;
  int n_full, m_full;  // the first m_full blocks are seen from the first token on
  int step;            // of the others each has so many tiles fewer than the one before it
                       // (0: it depends)
  int64_t per_head;    // tiles
  // first token that sees block i
  __device__ __forceinline__ int first_token(int i) const {
    return i < m_full ? x.tok0 : x.k0 + kWeighBlockKeys * i - x.causal;
  }
  __device__ __forceinline__ int tiles(int i, int tok) const {
    return i < m_full ? n_full : (x.tok1 - first_token(i) + tok - 1) / tok;
  }
};

__device__ __forceinline__ TileRun tile_run(const WeighArgs& p, int r, int tok, bool* bad) {
  TileRun t{};
  t.x = weigh_run(p, r, bad);
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
  t.step = kWeighBlockKeys % tok == 0 ? kWeighBlockKeys / tok : 0;
  const int64_t n = t.blocks - t.m_full;
  if (n > 0 && t.step > 0)
    t.per_head += n * t.tiles(t.m_full, tok) - t.step * (n * (n - 1) / 2);
  else
    for (int i = t.m_full; i < t.blocks; ++i) t.per_head += t.tiles(i, tok);
  return t;
}

// The same where it is seldom needed.
__device__ __noinline__ TileRun further_run(const WeighArgs& p, int r, int tok, bool* bad) {
  return tile_run(p, r, tok, bad);
}

// Lane src's, in every lane.
__device__ __forceinline__ TileRun run_of_lane(TileRun t, int src) {
  for (int* f : {&t.x.seq, &t.x.k0, &t.x.k1, &t.x.tok0, &t.x.tok1, &t.x.causal, &t.x.fresh,
                 &t.blocks, &t.n_full, &t.m_full, &t.step})
    *f = __shfl_sync(0xFFFFFFFFu, *f, src);
  t.group = __shfl_sync(0xFFFFFFFFu, static_cast<int>(t.group), src) != 0;
  t.per_head = __shfl_sync(0xFFFFFFFFu, t.per_head, src);
  return t;
}

// Tiles [j0, j1) of a block, as the roles read it from shared memory; h < 0 ends the
// work.
struct Item {
  int h;
  int key0;       // the block's first slot
  int first;      // token of tile 0
  int j0, j1, n;  // n: tiles of the block
  int seq, k1, tok1, causal, fresh;  // the run's
  int s1;         // a group's end, 0 for a sequence
};
static_assert(sizeof(Item) == 48, "as the ring's place in shared memory has it");
constexpr int kItemStages = 4;
constexpr int kItemReaders = kSumWarps + 3;  // the MMA issuers and the loader of lse

// A CTA's share, item after item.
struct Walk {
  TileRun t;
  int64_t left;
  int run, h, i, j;

  // To tile `at` of the run.
  __device__ __forceinline__ void seek(int64_t at, int tok) {
    h = static_cast<int>(quotient(at, t.per_head));
    at -= h * t.per_head;
    const int64_t full = static_cast<int64_t>(t.m_full) * t.n_full;
    if (at < full) {
      i = static_cast<int>(quotient(at, t.n_full));
      at -= static_cast<int64_t>(i) * t.n_full;
    } else {
      at -= full;
      i = t.m_full;
      for (int n = t.tiles(i, tok); at >= n; n = t.step > 0 ? n - t.step : t.tiles(i, tok)) {
        at -= n;
        ++i;
      }
    }
    j = static_cast<int>(at);
  }

  // To the next run that has tiles (there is one: left counts them), by a whole warp: a
  // run per lane.  (One after the other, at 0.5 us a run and 1.25 with groups, two prompts of
  // 2000 with 100 single tokens between them took 77 us and with 1000 of them 548, now 26 and
  // 50, side by side 25 and 33; with some 10^6 the other roles' waits could run out.)
  __device__ __forceinline__ bool next_run(const WeighArgs& p, int tok) {
    const int lane = threadIdx.x & 31, n_run = p.b.n_seq + p.b.n_group;
    for (++run; run < n_run; run += 32) {
      TileRun r{};
      bool bad = false;
      if (run + lane < n_run) r = further_run(p, run + lane, tok, &bad);
      const uint32_t with = __ballot_sync(0xFFFFFFFFu, r.per_head > 0);
      if (with == 0) continue;
      const int src = __ffs(with) - 1;
      t = run_of_lane(r, src);
      run += src;
      h = 0;
      return true;
    }
    return false;
  }

  __device__ __forceinline__ void next(const WeighArgs& p, int tok, Item& it) {
    it.h = -1;
    if (left <= 0 || (h == p.b.n_kv_heads && !next_run(p, tok))) return;
    it.h = h;
    it.key0 = t.x.k0 + kWeighBlockKeys * i;
    it.first = t.first_token(i);
    it.n = t.tiles(i, tok);
    it.j0 = j;
    it.j1 = left < it.n - j ? j + static_cast<int>(left) : it.n;
    it.seq = t.x.seq;
    it.k1 = t.x.k1;
    it.tok1 = t.x.tok1;
    it.causal = t.x.causal;
    it.fresh = t.x.fresh;
    it.s1 = t.group ? p.b.group_offsets[run - p.b.n_seq + 1] : 0;
    left -= it.j1 - it.j0;
    j = it.j1;
    if (j == it.n) {
      j = 0;
      if (++i == t.blocks) {
        i = 0;
        ++h;
      }
    }
  }
};

// The CTA's items in turn, which the TMA producer puts and the other roles take.
struct Items {
  const Item* slots;
  uint64_t *full, *empty;
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ bool take(Item& it, const DevCtx& ctx, volatile int* abort) {
    if (!warp_wait(&full[at], phase, ctx, abort)) return false;
    it = slots[at];
    // (a value from lane 0 is known to be the same in all lanes: what it decides stays
    // in uniform registers, which the tensor instructions take)
    for (int* f : {&it.h, &it.key0, &it.first, &it.j0, &it.j1, &it.n, &it.seq, &it.k1, &it.tok1,
                   &it.causal, &it.fresh, &it.s1})
      *f = __shfl_sync(0xFFFFFFFFu, *f, 0);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[at]);
    if (++at == kItemStages) {
      at = 0;
      phase ^= 1u;
    }
    return it.h >= 0;
  }
  // The next item's first slot and its run's end, before it is taken; false where
  // there is none.
  __device__ __forceinline__ bool peek(int& key0, int& k1, bool& ok, const DevCtx& ctx,
                                       volatile int* abort) {
    if (!(ok = warp_wait(&full[at], phase, ctx, abort))) return false;
    const int h = __shfl_sync(0xFFFFFFFFu, slots[at].h, 0);
    key0 = __shfl_sync(0xFFFFFFFFu, slots[at].key0, 0);
    k1 = __shfl_sync(0xFFFFFFFFu, slots[at].k1, 0);
    return h >= 0;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tile_kernel(const __grid_constant__ WeighMaps maps,
                      const __grid_constant__ WeighArgs p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_sum[kWarps], s_more[kWarps];
  __shared__ Walk s_walk;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + 1;
  uint64_t* k_ready = k_full + 2;
  uint64_t* s_full = k_full + 4;
  uint64_t* s_empty = s_full + kUnits;
  uint64_t* lse_full = s_empty + kUnits;
  uint64_t* lse_empty = lse_full + kLseStages;
  uint64_t* q_full = lse_empty + kLseStages;
  uint64_t* q_empty = q_full + C::kQStages;
  uint64_t* item_full = q_empty + C::kQStages;
  uint64_t* item_empty = item_full + kItemStages;
  uint64_t* sum_full = item_empty + kItemStages;
  uint64_t* drain = sum_full + kSumStages;
  Item* item_slots = reinterpret_cast<Item*>(smem + C::kOffItem);
  Rows* rows = reinterpret_cast<Rows*>(smem + C::kOffRows);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const bd_attention_batch& b = p.b;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31, tid = threadIdx.x;
  const int G = b.n_q_heads / b.n_kv_heads, tok = kRows / G;
  const int n_run = b.n_seq + b.n_group;

  if (tid == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, kSumWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&k_ready[i], kSumWarps / 2);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps / 2);
    }
    for (int i = 0; i < kLseStages; ++i) {
      mbar_init(&lse_full[i], 1);
      mbar_init(&lse_empty[i], kSumWarps);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
    }
    for (int i = 0; i < kItemStages; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kItemReaders);
    }
    for (int i = 0; i < kSumStages; ++i) mbar_init(&sum_full[i], kSumWarps / 2);
    for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
    *abort = 0;
    fence_mbar_init();
  }
  // Rows of 64 bytes in the 64-byte swizzle, of which a product step reads the first
  // 16 columns: three ones, and three places for a row's −lse/scale.
  for (int i = tid; i < (kLseStages + 1) * kLseBytes / 16; i += kThreads) {
    const int row = i >> 2 & (kRows - 1), chunk = i & 3 ^ (row >> 1 & 3);
    const bool ones = i >= kLseStages * kLseBytes / 16 && chunk == 0;
    *reinterpret_cast<uint4*>(smem + C::kOffLse + 16 * i) =
        make_uint4(ones ? 0x3F803F80u : 0u, ones ? 0x3F80u : 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
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

  // ---- this CTA's share of all tiles, and where it begins: a run per thread, and
  // further rounds of them where there are more runs
  bool bad = false;
  TileRun mine{};
  if (tid < n_run) mine = tile_run(p, tid, tok, &bad);
  int64_t more = 0;
  for (int r = tid + kThreads; r < n_run; r += kThreads)
    more += further_run(p, r, tok, &bad).per_head;
  // inclusive sums over the lanes
  const auto scan = [&](int64_t n) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, n, off);
      if (lane >= off) n += o;
    }
    return n;
  };
  // the sum of all warps' n, and of those before this one
  const auto of_warps = [&](const int64_t* n, int64_t& before) {
    const int64_t mine = lane < kWarps ? n[lane] : 0, inc = scan(mine);
    before = __shfl_sync(0xFFFFFFFFu, inc - mine, warp);
    return __shfl_sync(0xFFFFFFFFu, inc, 31);
  };
  int64_t inc = scan(mine.per_head);
  if (lane == 31) s_sum[warp] = inc;
  if (n_run > kThreads) {
    more = scan(more);
    if (lane == 31) s_more[warp] = more;
  }
  bad = __syncthreads_or(bad);
  int64_t others;
  int64_t round = of_warps(s_sum, others);  // over the round's runs
  inc += others;
  int64_t total = n_run > kThreads ? of_warps(s_more, others) : 0;
  total = bad ? 0 : (total + round) * b.n_kv_heads;
  if (bad && tid == 0 && blockIdx.x == 0) record_error(p.ctx, kErrBounds);
  const int64_t each = quotient(total, gridDim.x), extra = total - each * gridDim.x;
  const int64_t lo = each * blockIdx.x + (blockIdx.x < extra ? blockIdx.x : extra);
  const int64_t hi = lo + each + (blockIdx.x < extra ? 1 : 0);
  if (hi > lo) {
    int64_t before = 0;
    for (int base = 0; base < n_run && before <= lo; base += kThreads) {
      if (base > 0) {
        mine = TileRun{};
        if (base + tid < n_run) mine = further_run(p, base + tid, tok, &bad);
        inc = scan(mine.per_head);
        __syncthreads();  // the sums before have been read
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        round = of_warps(s_sum, others);
        inc += others;
      }
      const int64_t first = before + (inc - mine.per_head) * b.n_kv_heads;
      if (first <= lo && lo < before + inc * b.n_kv_heads) {
        Walk w{};
        w.t = mine;
        w.left = hi - lo;
        w.run = base + tid;
        w.seek(lo - first, tok);
        s_walk = w;
      }
      before += round * b.n_kv_heads;
    }
  }
  if (tid < 2) {
    p.records[2 * blockIdx.x + tid] = 0;
  }
  __syncthreads();
  Items items{item_slots, item_full, item_empty};
  Item it;
  bool ok = true;

  if (warp < kSumWarps) {
    // ============================================================ sums
    const int half = warp >> 2 & 1;
    const int c0 = warp >> 3 << 1;  // of the tile's four groups of 32 rows
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int row_of_half = 32 * (warp & 3) + lane;
    const int mine = 128 * half + row_of_half;  // key of the block
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    uint32_t l_phase = 0, k_phase = 0;
    int ls = 0;
    Unit unit;  // the tile's first
    bool started = false;  // an item before this one
    // Sums over a tile's later 64 rows, for the warps of the first ones.  Four of these need
    // no wait to be written: an item's keys arrive when all warps have staged those of the
    // one before it, which they do at the end of the item before that one at the earliest.
    // So a warp that sums item n has all others behind the end of item n − 3.  (The products'
    // buffers alone would not bound it: the warps of a half without keys wait for none.)
    float* others = reinterpret_cast<float*>(smem + C::kOffSum);
    int ss = 0;
    uint32_t sum_phase = 0;
    // A block's keys to tensor memory: this warp's 32 rows, half of their columns.  The
    // products that read the block before have completed: the last of them has been
    // waited for.
    const auto stage = [&](int key0, int k1) {
      if (!warp_wait(k_full, k_phase, p.ctx, abort)) return false;
      k_phase ^= 1u;
      const bool live = half == 0 || key0 + 128 < k1;
      if (live) {
        constexpr int kChunks = D / 16;  // 16-byte pieces of a row's half
        const int x0 = (c0 >> 1) * kChunks;
        const uint8_t* src = smem + half * C::kHalfBytes + row_of_half * 128;
#pragma unroll
        for (int y = 0; y < kChunks; y += 4) {
          uint32_t w[16];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int chunk = x0 + y + z;
            const uint4 v = *reinterpret_cast<const uint4*>(
                src + (chunk >> 3) * kPanel + (((chunk & 7) ^ (lane & 7)) << 4));
            w[4 * z] = v.x;
            w[4 * z + 1] = v.y;
            w[4 * z + 2] = v.z;
            w[4 * z + 3] = v.w;
          }
          tmem_st_x16(t_lane + static_cast<uint32_t>(half * (D / 2) + 4 * (x0 + y)), w);
        }
        tmem_st_done();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_empty);
        if (live) mbar_arrive(&k_ready[half]);
      }
      return true;
    };
    bool staged = false;  // the item's keys, while the one before was summed
    while (ok && items.take(it, p.ctx, abort)) {
      const int key = it.key0 + mine;
      const int key_lo = it.key0 + 128 * half + 32 * (warp & 3);  // the warp's
      const int key_hi = key_lo + 31 < it.k1 - 1 ? key_lo + 31 : it.k1 - 1;
      const bool both = it.key0 + 128 < it.k1;  // keys in the second half
      const bool idle = half != 0 && !both;
      if (!staged && !(ok = stage(it.key0, it.k1))) break;
      staged = false;
      // the key's place and what it has, on their way while its sum is formed
      int row = -1;
      float old = 0.f;
      if (c0 == 0 && key < it.k1 && it.j0 == 0) {
        row = static_cast<int>(weigh_row(b, it.seq, key, it.h));  // below 2^31
        if (row >= 0 && key < it.fresh && it.j1 == it.n) old = p.weights[row];
      }
      uint64_t sum[2] = {0u, 0u};
      for (int j = it.j0; j < it.j1; ++j) {
        const Unit u = unit.plus(half);
        ok = warp_wait(&lse_full[ls], l_phase, p.ctx, abort) &&
             (idle || warp_wait(&s_full[u.bar()], u.phase(), p.ctx, abort));
        if (!ok) break;
        tc_fence_after();
        // The half's last product with this block: the next block's keys go to tensor
        // memory now, and its products run while this tile is summed.  (Taken up after
        // that, an item of two tiles took 8200 cycles.)
        if (j == it.j1 - 1) {
          int key0, k1;
          if (items.peek(key0, k1, ok, p.ctx, abort)) staged = ok = stage(key0, k1);
          if (!ok) break;
        }
        const Rows& rw = rows[ls];
        const uint32_t t_s = t_lane + u.column();
        if (!idle) {
          // 32 rows at a time; the buffer goes back to the MMA issuer before the last of
          // them are summed.
#pragma unroll
          for (int c = c0; c < c0 + 2; ++c) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(t_s + 32u * c, s);
            tmem_ld_wait();
            if (c == c0 + 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_empty[u.bar()]);
            }
            if (rw.least[c] >= key_hi) {  // all of them see all of the warp's keys
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                float e0, e1;
                unpack2(mul2(pack2(__uint_as_float(s[2 * v]), __uint_as_float(s[2 * v + 1])),
                             scale2), e0, e1);
                sum[v & 1] = add2(sum[v & 1], pack2(ex2(e0), ex2(e1)));
              }
            } else if (rw.most[c] >= key_lo) {
              const int2* z2 = reinterpret_cast<const int2*>(rw.sees + 32 * c);
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                const int2 z = z2[v];
                float e0, e1;
                unpack2(mul2(pack2(__uint_as_float(s[2 * v]), __uint_as_float(s[2 * v + 1])),
                             scale2), e0, e1);
                // (selected, not multiplied: a row that does not count may hold anything)
                sum[v & 1] = add2(sum[v & 1],
                                  pack2(key <= z.x ? ex2(e0) : 0.f, key <= z.y ? ex2(e1) : 0.f));
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lse_empty[ls]);
        unit.skip(both ? 2 : 1);
        if (++ls == kLseStages) {
          ls = 0;
          l_phase ^= 1u;
        }
      }
      if (!ok) break;
      float a0, a1;
      unpack2(add2(sum[0], sum[1]), a0, a1);
      float a = a0 + a1;
      if (c0 != 0) {
        others[ss * kWeighBlockKeys + mine] = a;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sum_full[ss]);
      } else {
        if (!(ok = warp_wait(&sum_full[ss], sum_phase, p.ctx, abort))) break;
        a += others[ss * kWeighBlockKeys + mine];
      }
      if (++ss == kSumStages) {
        ss = 0;
        sum_phase ^= 1u;
      }
      const bool first_item = !started;
      started = true;
      if (c0 != 0) continue;
      if (row >= 0 && key >= it.fresh)
        p.positions[row] = key + (p.pos_offset != nullptr ? p.pos_offset[it.seq] : 0);
      if (it.j0 == 0 && it.j1 == it.n) {
        if (row >= 0) p.weights[row] = old + a;
      } else {
        const int slot = 2 * static_cast<int>(blockIdx.x) + (first_item ? 0 : 1);
        const int64_t at = static_cast<int64_t>(slot) * kWeighBlockKeys + mine;
        p.parts[at] = a;
        if (it.j0 == 0) p.rows[at] = row < 0 ? kWeighNowhere : key < it.fresh ? row : ~row;
        if (tid == 0)
          p.records[slot] = kWeighPart | (it.j0 == 0 ? kWeighBegins : 0) |
                            (it.j1 == it.n ? kWeighEnds : 0);
      }
    }
  } else if (warp < kTmaWarp) {
    // ============================================================ MMA issuers
    const int half = warp - kMmaWarp;
    const bool lead = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(128, kRows);
    const uint32_t base = smem_addr(smem);
    const uint32_t t_k = tmem + static_cast<uint32_t>(half * (D / 2));
    int qs = 0, ls = 0;
    Unit unit;
    uint32_t k_phase = 0, q_phase = 0, l_phase = 0;
    const uint64_t ones = sdesc_k_sw64(base + C::kOffOnes);
    bool issued = false;
    while (ok && items.take(it, p.ctx, abort)) {
      const bool both = it.key0 + 128 < it.k1;
      const bool idle = half != 0 && !both;
      if (!idle) {
        if (!(ok = warp_wait(&k_ready[half], k_phase, p.ctx, abort))) break;
        k_phase ^= 1u;
      }
      for (int j = it.j0; j < it.j1; ++j) {
        const Unit u = unit.plus(half);
        const Unit last = u.plus(2 * kUnits - kBuffers);  // in this buffer, three units ago
        // (one that is idle takes no part in the lse ring, which does not wait for it)
        ok = (idle || (warp_wait(&s_empty[last.bar()], last.phase(), p.ctx, abort) &&
                       warp_wait(&lse_full[ls], l_phase, p.ctx, abort))) &&
             warp_wait(&q_full[qs], q_phase, p.ctx, abort);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          if (idle) {
            mbar_arrive(&q_empty[qs]);
          } else {
            const uint64_t qd = sdesc_k_sw128(base + C::kOffQ + qs * C::kHalfBytes);
            const uint64_t ld = sdesc_k_sw64(base + C::kOffLse + ls * kLseBytes);
            const uint32_t t_s = tmem + u.column();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ts(t_s, t_k + 8u * k,
                     qd + static_cast<uint64_t>((k >> 2) * (kPanel >> 4) + 2 * (k & 3)), idesc,
                     k > 0 ? 1u : 0u);
            // (last: −lse/scale is the largest of the terms, and where it comes first all
            // later sums are rounded at its size: the weights of a prompt of 2048 were off by
            // 1.4e-6 of the largest, now by 2.4e-7)
            mma_ss(t_s, ones, ld, idesc, 1u);
            mma_commit(&s_full[u.bar()]);
            mma_commit(&q_empty[qs]);
          }
        }
        issued = issued || !idle;
        __syncwarp();
        unit.skip(both ? 2 : 1);
        if (++qs == C::kQStages) {
          qs = 0;
          q_phase ^= 1u;
        }
        if (++ls == kLseStages) {
          ls = 0;
          l_phase ^= 1u;
        }
      }
    }
    if (issued) {
      if (lead) mma_commit(&drain[half]);
      mbar_wait(&drain[half], 0, p.ctx, nullptr);
    }
    __syncwarp();
  } else if (warp == kTmaWarp) {
    // ============================================================ TMA producer
    const int page_shift = 31 - __clz(b.page_size);
    int qs = 0, k_fill = 0, q_fill = 0;
    uint32_t k_phase = 1, q_phase = 1;
    Walk walk{};
    if (hi > lo) walk = s_walk;
    int put = 0;
    uint32_t put_phase = 1;
    while (ok) {
      walk.next(p, tok, it);
      if (!(ok = warp_wait(&item_empty[put], put_phase, p.ctx, abort))) break;
      if (lane == 0) {
        item_slots[put] = it;
        mbar_arrive(&item_full[put]);
      }
      __syncwarp();
      if (++put == kItemStages) {
        put = 0;
        put_phase ^= 1u;
      }
      if (it.h < 0) break;
      const int keys = it.k1 - it.key0 < kWeighBlockKeys ? it.k1 - it.key0 : kWeighBlockKeys;
      const int n_pg = (keys + b.page_size - 1) >> page_shift;  // at most 16
      int page = -1;
      if (lane < n_pg) {
        page = b.page_table[static_cast<int64_t>(it.seq) * b.table_stride +
                            ((it.key0 >> page_shift) + lane)];
        if (page >= b.n_pages) page = -1;
        if (page < 0) record_error(p.ctx, kErrBounds);  // its sums go nowhere
      }
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, page >= 0);
      if (!(ok = warp_wait(k_empty, k_phase, p.ctx, abort))) break;
      k_phase ^= 1u;
      if (lane == 0)
        mbar_arrive_expect_tx(k_full, static_cast<uint32_t>(__popc(live) * b.page_size * 128 *
                                                            C::kPanels));
      __syncwarp();
      if (page >= 0) {
        const int at = lane << page_shift;  // key of the block
        uint8_t* dst = smem + (at >> 7) * C::kHalfBytes + (at & 127) * 128;
#pragma unroll
        for (int c = 0; c < C::kPanels; ++c)
          tma_load_3d(dst + c * kPanel, &maps.k, k_full, 0,
                      (page * b.n_kv_heads + it.h) << page_shift, c);
      }
      __syncwarp();
      ++k_fill;
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
      if (k_fill > 0) mbar_wait(k_full, static_cast<uint32_t>(k_fill - 1 & 1), p.ctx, nullptr);
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
    // −lse/scale as the sum of three bf16 numbers (24 bits), to be added by the product
    const float to_score = -kWeighLog2e / p.scale_log2;
    const auto put = [&](int stage, int row, float v) {
      const uint32_t hi = pack_bf16x2_rn(v, 0.f);
      const float r = v - bf16lo_to_f32(hi);
      const uint32_t mid = pack_bf16x2_rn(r, 0.f);
      const uint32_t lo = pack_bf16x2_rn(r - bf16lo_to_f32(mid), 0.f);
      *reinterpret_cast<uint2*>(smem + C::kOffLse + stage * kLseBytes + row * 64 +
                                ((row >> 1 & 3) << 4)) = make_uint2(hi | mid << 16, lo);
    };
    int row_tok[4], row_head[4];  // of the lane's four rows; the token −1: no row
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = 32 * c + lane;
      row_tok[c] = row < tok * G ? row / G : -1;
      row_head[c] = row % G;
    }
    while (ok && items.take(it, p.ctx, abort)) {
      const float* lse = p.lse + it.h * G;
      float l[4];  // of the next tile, on their way while this one waits
      const auto load = [&](int j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = it.first + j * tok + row_tok[c];
          l[c] = row_tok[c] >= 0 && t < it.tok1
                     ? lse[static_cast<int64_t>(t) * b.n_q_heads + row_head[c]]
                     : INFINITY;
        }
      };
      load(it.j0);
      for (int j = it.j0; j < it.j1; ++j) {
        float x[4];
        int sees[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = it.first + j * tok + row_tok[c];
          x[c] = 0.f;
          sees[c] = -1;
          if (isfinite(l[c]) &&
              (it.s1 == 0 || !windowed || weigh_in_window(p, t, it.seq, it.s1))) {
            x[c] = fminf(fmaxf(l[c] * to_score, -3e38f), 3e38f);
            sees[c] = it.s1 > 0 ? INT32_MAX : t + it.causal;
          }
        }
        if (j + 1 < it.j1) load(j + 1);
        if (!(ok = warp_wait(&lse_empty[ls], phase, p.ctx, abort))) break;
        Rows& rw = rows[ls];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          put(ls, 32 * c + lane, x[c]);
          rw.sees[32 * c + lane] = sees[c];
          const int least = __reduce_min_sync(0xFFFFFFFFu, sees[c]);
          const int most = __reduce_max_sync(0xFFFFFFFFu, sees[c]);
          if (lane == 0) {
            rw.least[c] = least;
            rw.most[c] = most;
          }
        }
        fence_proxy_async_smem();
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
