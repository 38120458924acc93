// attention.cu — causal attention of ragged query runs over the paged cache:
// the C entry points, the plan kernel and the combine kernel.  attention.cuh
// says how the work is divided; attn_decode.cu and attn_tile.cu do it.
#include <climits>
#include <cmath>
#include <cstdint>

#include "attention.cuh"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);

namespace {
size_t pad256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }
}  // namespace

AttnLayout attn_layout(const bd_attention_batch& b, int num_sms) {
  AttnLayout L{};
  L.g = b.n_q_heads / b.n_kv_heads;
  L.half_tok = kHalfRows / L.g;
  const int64_t tile_tok = 2 * L.half_tok;
  // Short runs have at most 16 rows, one mma.sync row tile.  Longer ones are the
  // tile role's: at 128-element heads its 256-row tile takes a few rows faster
  // than two row tiles per warp did (8 sequences of 4 tokens, 8 query heads per key
  // head, 20.4 -> 14.5 us; 256 of them 75 -> 53; 64 single tokens of 32 query heads
  // per key head 64 -> 60).  At 64 a block's softmax takes twice its loads, and
  // two row tiles win (64 sequences of 4 tokens over 500 to 8000 keys, 109
  // against 177 us; 256 single tokens of 20 query heads per key head, 23 against
  // 30), so runs have up to 32 rows where a single token already has more than
  // 16, or no sequence has more than 32.
  const int64_t max_rows = static_cast<int64_t>(b.max_q_len) * L.g;
  L.d_rows = b.head_dim == 64 && (L.g > 16 || (max_rows > 16 && max_rows <= 32)) ? 32 : 16;
  L.use_tile = max_rows > L.d_rows || b.n_group > 0;
  L.d_ctas = 2 * num_sms;
  L.d_warps = 8 * num_sms;
  L.t_ctas = num_sms;
  const int64_t T = b.n_tokens;
  int64_t long_seqs = 0;  // at most
  if (max_rows > L.d_rows) {
    long_seqs = T * L.g / (L.d_rows + 1);
    long_seqs = long_seqs < b.n_seq ? long_seqs : b.n_seq;
  }
  L.max_tiles = 0;
  if (max_rows > L.d_rows) L.max_tiles += T / tile_tok + long_seqs;
  const int64_t prefix_tiles = b.n_group > 0 ? T / tile_tok + b.n_group : 0;
  L.max_tiles += prefix_tiles;
  // pieces: at most one per tile plus two per CTA of the launch (the plan cuts
  // tiles longer than the CTAs' even share, into shares or half shares)
  L.max_entries = L.use_tile ? L.max_tiles + 2 * L.t_ctas : 0;
  // slots: the pieces of cut tiles (a tile of more than one piece has at most
  // twice its blocks' worth of them, so four per CTA), with groups every prefix
  // piece and every own piece of a member
  L.t_slots = L.use_tile ? 4 * L.t_ctas + (b.n_group > 0 ? L.max_tiles * b.n_kv_heads : 0) : 0;
  size_t o = pad256(sizeof(PlanHeader));
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += pad256(bytes);
    return at;
  };
  L.o_tok_seq = take(4 * static_cast<size_t>(T));
  L.o_seq = take(sizeof(SeqRec) * static_cast<size_t>(b.n_seq));
  L.o_start = take(sizeof(DecodeStart) * static_cast<size_t>(L.d_warps));
  L.o_group = take(4 * static_cast<size_t>(b.n_group));
  L.o_run = take(4 * (static_cast<size_t>(b.n_seq) + b.n_group + 1));
  L.o_tile_slot = take(4 * static_cast<size_t>(L.max_tiles));
  L.o_tile_ns = take(4 * static_cast<size_t>(L.max_tiles));
  L.o_entry = take(sizeof(TileEntry) * static_cast<size_t>(L.max_entries));
  L.o_comb = take(sizeof(CombItem) * static_cast<size_t>(T));
  L.plan_bytes = o;
  o = 0;
  const size_t d_rows = static_cast<size_t>(L.d_warps) * 2 * L.d_rows;
  L.w_d_o = take(d_rows * b.head_dim * 4);
  L.w_d_ml = take(d_rows * 8);
  const size_t r_rows = b.n_group > 0 ? static_cast<size_t>(T) * b.n_q_heads : 0;
  L.w_r_o = take(r_rows * b.head_dim * 4);
  L.w_r_ml = take(r_rows * 8);
  const size_t t_rows = static_cast<size_t>(L.t_slots) * 2 * kHalfRows;
  L.w_t_o = take(t_rows * b.head_dim * 4);
  L.w_t_ml = take(t_rows * 8);
  L.ws_bytes = o;
  return L;
}

namespace {

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kLenBuckets = 1024;

// Exclusive prefix sum over the CTA; *total receives the sum.
__device__ int64_t block_scan(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
    if (lane >= off) inc += o;
  }
  __syncthreads();  // s_warp of an earlier call has been read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, w, off);
      if (lane >= off) w += o;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return inc - v + (warp > 0 ? s_warp[warp - 1] : 0);
}

// One CTA.  Every phase walks sequences, runs or tiles with all threads; what
// later kernels read is a function of the lengths alone (the order of equally
// long pieces is not, and decides only which CTA runs them).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttnArgs p) {
  __shared__ int64_t s_warp[32];
  __shared__ int s_hist[kLenBuckets];
  __shared__ unsigned long long s_blocks;
  __shared__ int s_comb, s_longest;
  const bd_attention_batch& b = p.b;
  const AttnLayout& L = p.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kPlanThreads / 32;
  PlanHeader* hd = reinterpret_cast<PlanHeader*>(p.plan);
  int32_t* tok_seq = reinterpret_cast<int32_t*>(p.plan + L.o_tok_seq);
  SeqRec* seqs = reinterpret_cast<SeqRec*>(p.plan + L.o_seq);
  DecodeStart* starts = reinterpret_cast<DecodeStart*>(p.plan + L.o_start);
  int32_t* prefix = reinterpret_cast<int32_t*>(p.plan + L.o_group);
  int32_t* run_tile0 = reinterpret_cast<int32_t*>(p.plan + L.o_run);
  int32_t* tile_slot = reinterpret_cast<int32_t*>(p.plan + L.o_tile_slot);
  int32_t* tile_ns = reinterpret_cast<int32_t*>(p.plan + L.o_tile_ns);
  TileEntry* entries = reinterpret_cast<TileEntry*>(p.plan + L.o_entry);
  CombItem* comb = reinterpret_cast<CombItem*>(p.plan + L.o_comb);
  const int tile_tok = 2 * L.half_tok;
  const int n_run = L.use_tile ? b.n_seq + b.n_group : 0;
  griddep_wait();
  if (tid == 0) {
    s_blocks = 0;
    s_comb = 0;
    s_longest = 0;
  }
  for (int i = tid; i < kLenBuckets; i += kPlanThreads) s_hist[i] = 0;

  // The tables' bounds.  A table that breaks them plans no work: every row is
  // then written as a row without keys.
  int bad = 0;
  for (int s = tid; s < b.n_seq; s += kPlanThreads) {
    const int a = b.seq_offsets[s], e = b.seq_offsets[s + 1], kv = b.kv_len[s];
    bad |= a < 0 || e < a || e > b.n_tokens || e - a > b.max_q_len || kv < 0 ||
           kv > b.max_kv_len || kv > b.table_stride * b.page_size ||
           static_cast<int64_t>(kv) * b.n_kv_heads > INT32_MAX;
  }
  for (int g = tid; g < b.n_group; g += kPlanThreads) {
    const int a = b.group_offsets[g], e = b.group_offsets[g + 1];
    bad |= a < 0 || e < a || e > b.n_seq || b.prefix_len[g] < 0;
  }
  bad = __syncthreads_or(bad);
  for (int64_t t = tid; t < b.n_tokens; t += kPlanThreads) {
    tok_seq[t] = -1;
    if (bad) {
      CombItem it{};
      it.tok = static_cast<int32_t>(t);
      comb[t] = it;
    }
  }
  if (bad) {
    for (int c = tid; c < L.d_warps; c += kPlanThreads) starts[c].lo = starts[c].hi = 0;
    if (tid == 0) {
      record_error(p.ctx, kErrBounds);
      *hd = PlanHeader{0, 1, 1, 0, 0, static_cast<int32_t>(b.n_tokens), 0};
    }
    return;
  }
  for (int s = tid; s < b.n_seq; s += kPlanThreads) {
    SeqRec r{};
    r.tok0 = b.seq_offsets[s];
    r.q_len = b.seq_offsets[s + 1] - r.tok0;
    r.kv_len = b.kv_len[s];
    r.group = -1;
    seqs[s] = r;
  }
  __syncthreads();
  for (int s = warp; s < b.n_seq; s += kWarps)
    for (int t = lane; t < seqs[s].q_len; t += 32) tok_seq[seqs[s].tok0 + t] = s;

  // A group's prefix, cut to what every member has before its first query
  // token and to whole pages.  Two or three sequences of few rows read it by
  // themselves: the decode kernel is then as fast as the join.
  for (int g = warp; g < b.n_group; g += kWarps) {
    const int a = b.group_offsets[g], e = b.group_offsets[g + 1];
    int len = b.prefix_len[g];
    for (int s = a + lane; s < e; s += 32) {
      const int before = seqs[s].kv_len - seqs[s].q_len;
      len = before < len ? before : len;
    }
    len = __reduce_min_sync(0xFFFFFFFFu, len);
    len = len > 0 ? len / b.page_size * b.page_size : 0;
    const int64_t rows =
        e > a ? static_cast<int64_t>(b.seq_offsets[e] - b.seq_offsets[a]) * L.g : 0;
    if (e - a < 2 || (e - a < 4 && rows <= 32)) len = 0;
    if (lane == 0) prefix[g] = len;
    if (len > 0)
      for (int s = a + lane; s < e; s += 32) {
        seqs[s].k0 = len;
        seqs[s].group = g;
      }
  }
  __syncthreads();

  // Decode units: every 16 own keys of a short run, once per key head.
  int64_t carry = 0;
  for (int base = 0; base < b.n_seq; base += kPlanThreads) {
    const int s = base + tid;
    int64_t n = 0;
    if (s < b.n_seq) {
      const SeqRec r = seqs[s];
      const int rows = r.q_len * L.g;
      if (rows > 0 && rows <= L.d_rows) n = (r.kv_len - r.k0 + kUnitKeys - 1) / kUnitKeys;
    }
    int64_t sum;
    const int64_t at = carry + block_scan(n * b.n_kv_heads, s_warp, &sum);
    if (s < b.n_seq) {
      seqs[s].unit0 = static_cast<int32_t>(at);
      seqs[s].units = static_cast<int32_t>(n);
    }
    carry += sum;
  }
  // Units are counted in 31 bits; more (2^35 keys times key heads) plan nothing.
  if (carry > INT32_MAX) {
    for (int64_t t = tid; t < b.n_tokens; t += kPlanThreads) {
      CombItem it{};
      it.tok = static_cast<int32_t>(t);
      comb[t] = it;
    }
    for (int c = tid; c < L.d_warps; c += kPlanThreads) starts[c].lo = starts[c].hi = 0;
    if (tid == 0) {
      record_error(p.ctx, kErrBounds);
      *hd = PlanHeader{0, 1, 1, 0, 0, static_cast<int32_t>(b.n_tokens), 0};
    }
    return;
  }
  const int64_t d_units = carry;
  __syncthreads();

  // Tiles of the long runs: sequences, then groups.
  carry = 0;
  for (int base = 0; base < n_run; base += kPlanThreads) {
    const int r = base + tid;
    int64_t n = 0;
    if (r < b.n_seq) {
      const SeqRec q = seqs[r];
      if (q.q_len * static_cast<int64_t>(L.g) > L.d_rows)
        n = (q.q_len + tile_tok - 1) / tile_tok;
    } else if (r < n_run && prefix[r - b.n_seq] > 0) {
      const int g = r - b.n_seq;
      const int toks =
          b.seq_offsets[b.group_offsets[g + 1]] - b.seq_offsets[b.group_offsets[g]];
      n = (toks + tile_tok - 1) / tile_tok;
    }
    int64_t sum;
    const int64_t at = carry + block_scan(n, s_warp, &sum);
    if (r < n_run) run_tile0[r] = static_cast<int32_t>(at);
    carry += sum;
  }
  const int n_tiles = static_cast<int>(carry);
  if (tid == 0 && n_run > 0) run_tile0[n_run] = n_tiles;
  __syncthreads();

  // Tile i of run r without its piece: what it covers and its blocks.
  const auto tile_of = [&](int r, int i, int* blocks) {
    TileEntry e{};
    int first, toks;
    if (r < b.n_seq) {
      const SeqRec q = seqs[r];
      first = q.tok0;
      toks = q.q_len;
      e.seq = r;
      e.k_lo = q.k0;
      e.causal = q.kv_len - (q.tok0 + q.q_len) + 1;
    } else {
      const int g = r - b.n_seq, s0 = b.group_offsets[g];
      first = seqs[s0].tok0;
      toks = b.seq_offsets[b.group_offsets[g + 1]] - first;
      e.seq = s0;
      e.causal = 1 << 30;
    }
    e.tok0 = first + i * tile_tok;
    e.n_tok = toks - i * tile_tok < tile_tok ? toks - i * tile_tok : tile_tok;
    if (r < b.n_seq) {
      const int kv = seqs[r].kv_len;
      e.k_hi = e.tok0 + e.n_tok - 1 + e.causal;  // what the tile's last token sees
      e.tail = (e.k_hi + 15) / 16 * 16 > kv;
    } else {
      e.k_hi = prefix[r - b.n_seq];
    }
    *blocks = e.k_hi > e.k_lo ? (e.k_hi - e.k_lo + kTileKeys - 1) / kTileKeys : 0;
    return e;
  };
  for (int r = warp; r < n_run; r += kWarps) {
    const int t0 = run_tile0[r], t1 = run_tile0[r + 1];
    for (int i = t0 + lane; i < t1; i += 32) {
      int nb;
      tile_of(r, i - t0, &nb);
      atomicAdd(&s_blocks, static_cast<unsigned long long>(nb));
      atomicMax(&s_longest, nb);
    }
  }
  __syncthreads();
  // CTAs per role, so that both end at about the same time: a block of 256 rows
  // takes about 1.4 µs of an SM (1 at 64-element heads) and a piece 5 µs on
  // top, a CTA reads keys and values at about 80 bytes per ns.  A batch of 64
  // ragged decode rows and four 512-token chunks took 117 µs with the two kinds
  // of work one after the other.
  const int64_t t_blocks = static_cast<int64_t>(s_blocks) * b.n_kv_heads;
  int n_tile = 0, n_dec = L.d_ctas;
  if (L.use_tile) {
    const float t_cost = static_cast<float>(t_blocks) * (b.head_dim == 128 ? 1.4f : 1.f) +
                         5.f * static_cast<float>(n_tiles) * b.n_kv_heads;
    const float d_cost = static_cast<float>(d_units) * (kUnitKeys * 4.f / 80e3f) * b.head_dim;
    // (the quotient may round to a little above its bound: both ends are cut)
    n_dec = d_units == 0 ? 0
                         : static_cast<int>(ceilf(L.t_ctas * d_cost / (t_cost + d_cost)));
    const int least = d_units > 0 ? 1 : 0, most = L.t_ctas - (t_blocks > 0 ? 1 : 0);
    n_dec = n_dec < least ? least : (n_dec > most ? most : n_dec);
    n_tile = L.t_ctas - n_dec;
  }
  const int warps = L.use_tile ? kTileDecodeWarps : kDecodeWarps;
  int64_t d_per = n_dec > 0 ? (d_units + n_dec * warps - 1) / (n_dec * warps) : 1;
  d_per = d_per > kMinUnits ? d_per : kMinUnits;
  // Where each decode warp's units begin.
  for (int s = tid; s < b.n_seq; s += kPlanThreads) {
    DecodeStart st{};
    st.r = seqs[s];
    st.seq = s;
    const int64_t end = st.r.unit0 + static_cast<int64_t>(st.r.units) * b.n_kv_heads;
    for (int64_t c = (st.r.unit0 + d_per - 1) / d_per; c * d_per < end; ++c) {
      st.lo = static_cast<int32_t>(c * d_per);
      st.hi = static_cast<int32_t>(st.lo + d_per < d_units ? st.lo + d_per : d_units);
      starts[c] = st;
    }
  }
  for (int64_t c = (d_units + d_per - 1) / d_per + tid; c < L.d_warps; c += kPlanThreads)
    starts[c].lo = starts[c].hi = 0;

  // Where the longest tile exceeds the CTAs' even share by more than a quarter
  // and by more than 4 blocks, tiles longer than the share are cut into pieces
  // of that share.  Below that the join of the pieces costs more than the
  // uneven end: 256 tiles of up to 20 blocks with a share of 17 took 55 µs and
  // 32 µs more for the join when cut.
  int64_t share = n_tile == 0 ? 0 : (t_blocks + n_tile - 1) / n_tile;
  const bool cut = s_longest > share + (share / 4 > 4 ? share / 4 : 4);
  if (!cut) share = s_longest;
  int piece = static_cast<int>(share < 2 ? 2 : share);
  if (cut && static_cast<int64_t>(n_tiles) * b.n_kv_heads <= n_tile) {
    // Few tiles: the shortest pieces that are one per CTA, so that none takes a
    // remainder on top of a full piece (each thread tries one length).  Where that
    // is far above the share (about as many uneven tiles as CTAs), pieces of half
    // a share, several per CTA: 128 tiles of 4 to 63 blocks, 90 us with one piece
    // per CTA, 60 so.
    __syncthreads();
    if (tid == 0) s_longest = INT_MAX;
    for (int r = warp; r < n_run; r += kWarps)
      for (int i = run_tile0[r] + lane; i < run_tile0[r + 1]; i += 32) {
        int nb;
        tile_of(r, i - run_tile0[r], &nb);
        tile_ns[i] = nb;
      }
    __syncthreads();
    int64_t pieces = 0;
    for (int i = 0; i < n_tiles; ++i) pieces += (tile_ns[i] + piece + tid - 1) / (piece + tid);
    if (pieces * b.n_kv_heads <= n_tile) atomicMin(&s_longest, piece + tid);
    __syncthreads();
    const int most = static_cast<int>(share + (share / 4 > 4 ? share / 4 : 4));
    piece = s_longest <= most ? s_longest : (piece + 1) / 2;
  }
  // slots first (a scan over tiles, which belong to runs: by tile index)
  for (int r = warp; r < n_run; r += kWarps) {
    const int t0 = run_tile0[r], t1 = run_tile0[r + 1];
    const bool parts = r >= b.n_seq || (t1 > t0 && seqs[r].group >= 0);
    for (int i = t0 + lane; i < t1; i += 32) {
      int nb;
      tile_of(r, i - t0, &nb);
      const int ns = (nb + piece - 1) / piece;
      tile_ns[i] = ns;
      tile_slot[i] = ns > 1 || (parts && ns > 0) ? 0 : -1;
      for (int j = 0; j < ns; ++j) {
        const int len = j + 1 < ns ? piece : nb - j * piece;
        atomicAdd(&s_hist[len < kLenBuckets ? len : kLenBuckets - 1], 1);
      }
    }
  }
  __syncthreads();
  carry = 0;
  for (int base = 0; base < n_tiles; base += kPlanThreads) {
    const int i = base + tid;
    const int64_t n = i < n_tiles && tile_slot[i] >= 0 ? tile_ns[i] : 0;
    int64_t sum;
    const int64_t at = carry + block_scan(n, s_warp, &sum);
    if (n > 0) tile_slot[i] = static_cast<int32_t>(at);
    carry += sum;
  }
  const bool over = carry * b.n_kv_heads > L.t_slots;  // attn_layout's bound: cannot happen
  // The longest pieces first: bucket offsets in descending order of length.
  {
    const int len = kLenBuckets - 1 - tid;
    int64_t sum;
    const int64_t at = block_scan(s_hist[len], s_warp, &sum);
    carry = sum;
    __syncthreads();
    s_hist[len] = static_cast<int>(at);
  }
  const int n_entries = static_cast<int>(carry);
  const bool fits = !over && n_entries <= L.max_entries;
  __syncthreads();
  for (int r = warp; r < n_run && fits; r += kWarps) {
    const int t0 = run_tile0[r], t1 = run_tile0[r + 1];
    for (int i = t0 + lane; i < t1; i += 32) {
      int nb;
      TileEntry e = tile_of(r, i - t0, &nb);
      const int ns = tile_ns[i], slot = tile_slot[i];
      for (int j = 0; j < ns; ++j) {
        e.b0 = j * piece;
        e.b1 = j + 1 < ns ? e.b0 + piece : nb;
        e.slot = slot < 0 ? -1 : slot + j;
        const int len = e.b1 - e.b0;
        entries[atomicAdd(&s_hist[len < kLenBuckets ? len : kLenBuckets - 1], 1)] = e;
      }
    }
  }

  // Tokens whose rows are joined, or have no keys at all.
  for (int64_t t = tid; t < b.n_tokens; t += kPlanThreads) {
    const int s = tok_seq[t];
    bool join = true;
    CombItem it{};
    it.tok = static_cast<int32_t>(t);
    if (s >= 0) {
      const SeqRec r = seqs[s];
      const int x = it.tok - r.tok0;
      if (r.q_len * static_cast<int64_t>(L.g) > L.d_rows) {
        const int i = run_tile0[s] + x / tile_tok, y = x % tile_tok;
        join = tile_slot[i] >= 0 || tile_ns[i] == 0;
        it.own_slot = tile_slot[i];
        it.own_ns = tile_ns[i];
        it.own_row = y / L.half_tok * kHalfRows + y % L.half_tok * L.g;
      } else if (r.units > 0) {
        it.unit0 = r.unit0;
        it.units = r.units;
        it.own_row = x * L.g;
        join = r.group >= 0;  // else final where no head's units are cut
        for (int h = 0; h < b.n_kv_heads && !join; ++h) {
          const uint32_t u0 = r.unit0 + h * r.units;
          join = decode_parts(u0, u0 + r.units, d_units, d_per, warps).count() > 1;
        }
      }
      if (r.group >= 0) {
        const int z = it.tok - seqs[b.group_offsets[r.group]].tok0;
        const int i = run_tile0[b.n_seq + r.group] + z / tile_tok, y = z % tile_tok;
        it.pre_slot = tile_slot[i];
        it.pre_ns = tile_ns[i];
        it.pre_row = y / L.half_tok * kHalfRows + y % L.half_tok * L.g;
      }
    }
    if (join) comb[atomicAdd(&s_comb, 1)] = it;
  }
  __syncthreads();
  if (tid == 0) {
    if (!fits) record_error(p.ctx, kErrBounds);
    *hd = PlanHeader{static_cast<int32_t>(d_units), static_cast<int32_t>(d_per), warps,
                     fits ? n_entries : 0, n_tile, s_comb, n_tile};
  }
}

// ------------------------------------------------------------------ combine

constexpr int kCombThreads = 128;
constexpr int kCombCtas = 8;   // per SM, and in the launch: one round, no second wave
constexpr int kCombBatch = 4;  // parts that a thread has in flight

// One CTA per (token, key head) of the plan's list, or per slice of its columns
// where there are few.  A row's parts are dealt to the thread groups of
// the CTA, which join them in a fixed order with a running maximum and meet in
// shared memory: the join is one load of the item and about parts / (groups ·
// 4) rounds of independent loads.  Neighbouring threads read neighbouring rows
// of a slot.  Bound by the latency of those loads from L2: 64 tokens of 64 heads
// behind two shared prefixes, 6 to 8 parts a row, 10.2 us by itself on a cold
// cache.  With 256 threads of 80 registers the CTAs ran in several waves.
__global__ void __launch_bounds__(kCombThreads, kCombCtas) combine_kernel(const AttnArgs p) {
  __shared__ float4 s_o[kCombThreads];
  __shared__ float2 s_ml[kCombThreads];
  const bd_attention_batch& b = p.b;
  const AttnLayout& L = p.L;
  const int g = L.g, D = b.head_dim, H = b.n_kv_heads;
  // The plan is older than the kernel that this one waits for, which has itself
  // waited for it before it let this one start: its header and this CTA's first
  // item are fetched while that kernel ends.
  const PlanHeader hd = *p.header();
  // As many column slices as one round of CTAs takes, at least what fits a CTA;
  // and, where few items leave SMs idle, fewer rows for each CTA, so that more
  // thread groups share the parts (one token of 32 query heads on one key head,
  // 65536 keys, 57 -> 21 us).
  const int64_t items = static_cast<int64_t>(hd.n_comb) * H;
  int slice_bits = D == 128 ? 3 : 2, row_bits = 0;
  while (slice_bits > 0 && g * (D / 4) * 2 <= kCombThreads << slice_bits &&
         items << slice_bits > gridDim.x)
    --slice_bits;
  while (4 << row_bits < g && items << (slice_bits + row_bits + 1) <= L.d_ctas) ++row_bits;
  const int cut_bits = slice_bits + row_bits;     // 2^cut_bits CTAs per item
  const int g_cta = (g + (1 << row_bits) - 1) >> row_bits;
  const int cols = (D / 4) >> slice_bits;         // float4 columns per CTA
  const int groups = kCombThreads / (cols * g_cta);
  const int q = threadIdx.x / g_cta;
  const int col = q % cols, grp = q / cols, row_in = threadIdx.x % g_cta;
  const int n_work = static_cast<int>(items << cut_bits);
  // An item's own parts: tile slots own_slot .. (times heads plus head), decode
  // parts, or the one part of a run that a warp or CTA did alone; none to join
  // where that part is final already (another head of the token is cut).
  struct Work {
    CombItem it;
    DecodeParts dp;
    int64_t first;
    int kvh, d4, row, n_own, rows, own_row;
    bool cut, skip;
    uint8_t *o, *ml;
  };
  const auto prepare = [&](const CombItem& it, int w) {
    Work k;
    k.it = it;
    k.kvh = static_cast<int>((static_cast<uint32_t>(w) >> cut_bits) % static_cast<uint32_t>(H));
    k.d4 = (w & ((1 << slice_bits) - 1)) * cols + col;
    k.row = (w >> slice_bits & ((1 << row_bits) - 1)) * g_cta + row_in;
    k.first = static_cast<int64_t>(it.own_slot) * H + k.kvh;
    k.n_own = it.own_ns;
    k.rows = 2 * kHalfRows;
    k.own_row = it.own_row;
    k.o = p.ws + L.w_t_o;
    k.ml = p.ws + L.w_t_ml;
    k.cut = k.skip = false;
    if (it.units > 0) {
      const uint32_t u0 = it.unit0 + k.kvh * it.units;
      k.dp = decode_parts(u0, u0 + it.units, hd.d_units, hd.d_per, hd.d_warps);
      k.n_own = k.dp.count();
      k.cut = k.n_own > 1;
      k.skip = !k.cut && it.pre_ns == 0;
      if (!k.cut) {
        k.first = static_cast<int64_t>(it.tok) * H + k.kvh;
        k.own_row = 0;
      }
      k.rows = k.cut ? L.d_rows : g;
      k.o = p.ws + (k.cut ? L.w_d_o : L.w_r_o);
      k.ml = p.ws + (k.cut ? L.w_d_ml : L.w_r_ml);
    }
    return k;
  };
  const auto item_of = [&](int w) {
    return p.comb()[(static_cast<uint32_t>(w) >> cut_bits) / static_cast<uint32_t>(H)];
  };
  const int stride = static_cast<int>(gridDim.x);
  int w = static_cast<int>(blockIdx.x);
  Work k{};
  CombItem ahead{};
  if (w < n_work) k = prepare(item_of(w), w);
  if (w + stride < n_work) ahead = item_of(w + stride);
  griddep_wait();
  griddep_launch_dependents();
  // the tile kernel has dealt its pieces: its counter for the next call
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.piece_counter() = hd.t_ctas;
  for (; w < n_work; w += stride) {
    if (w != static_cast<int>(blockIdx.x)) {
      k = prepare(ahead, w);
      if (w + stride < n_work) ahead = item_of(w + stride);
    }
    if (k.skip) continue;
    const CombItem& it = k.it;
    const int kvh = k.kvh, d4 = k.d4, row = k.row, n_own = k.n_own, rows = k.rows, own_row = k.own_row;
    const int n = n_own + it.pre_ns;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp < groups && row < g) {
      for (int i0 = grp; i0 < n; i0 += groups * kCombBatch) {
        float2 ml[kCombBatch];
        float4 v[kCombBatch];
#pragma unroll
        for (int x = 0; x < kCombBatch; ++x) {
          const int i = i0 + x * groups;
          ml[x] = make_float2(-INFINITY, 0.f);
          v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n_own) {
            const int64_t slot = k.cut ? k.dp.slot(i) : k.first + static_cast<int64_t>(i) * H;
            ml[x] = part_ml(k.ml, slot, rows)[own_row + row];
            v[x] = part_o(k.o, slot, rows, D)[static_cast<int64_t>(d4) * rows + own_row + row];
          } else if (i < n) {
            const int64_t slot = static_cast<int64_t>(it.pre_slot + (i - n_own)) * H + kvh;
            ml[x] = part_ml(p.ws + L.w_t_ml, slot, 2 * kHalfRows)[it.pre_row + row];
            v[x] = part_o(p.ws + L.w_t_o, slot, 2 * kHalfRows,
                          D)[static_cast<int64_t>(d4) * 2 * kHalfRows + it.pre_row + row];
          }
        }
        float top = m;
#pragma unroll
        for (int x = 0; x < kCombBatch; ++x) top = fmaxf(top, ml[x].x);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = ex2(m - ref);
        l *= f;
        o.x *= f;
        o.y *= f;
        o.z *= f;
        o.w *= f;
#pragma unroll
        for (int x = 0; x < kCombBatch; ++x) {
          const float s = ex2(ml[x].x - ref);
          l = fmaf(ml[x].y, s, l);
          o.x = fmaf(v[x].x, s, o.x);
          o.y = fmaf(v[x].y, s, o.y);
          o.z = fmaf(v[x].z, s, o.z);
          o.w = fmaf(v[x].w, s, o.w);
        }
        m = top;
      }
    }
    if (groups > 1) {
      __syncthreads();  // the last item's values have been read
      s_o[threadIdx.x] = o;
      s_ml[threadIdx.x] = make_float2(m, l);
      __syncthreads();
    }
    if (grp != 0 || row >= g) continue;
    const int span = g_cta * cols, most = groups < n ? groups : n;
    float top = m;
    for (int k = 1; k < most; ++k) top = fmaxf(top, s_ml[threadIdx.x + k * span].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - ref);
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
    for (int k = 1; k < most; ++k) {
      const float2 ml = s_ml[threadIdx.x + k * span];
      const float4 v = s_o[threadIdx.x + k * span];
      const float s = ex2(ml.x - ref);
      l = fmaf(ml.y, s, l);
      o.x = fmaf(v.x, s, o.x);
      o.y = fmaf(v.y, s, o.y);
      o.z = fmaf(v.z, s, o.z);
      o.w = fmaf(v.w, s, o.w);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN goes through)
    const int64_t at = static_cast<int64_t>(it.tok) * b.n_q_heads + kvh * g + row;
    reinterpret_cast<uint2*>(p.out + at * D)[d4] =
        make_uint2(pack_bf16x2_rn(o.x * inv, o.y * inv), pack_bf16x2_rn(o.z * inv, o.w * inv));
    if (d4 == 0 && p.lse != nullptr)
      p.lse[at] = l != 0.f ? (ref + log2f(l)) * kLn2 : -INFINITY;
  }
}

int fill_args(const bd_attention_batch* batch, AttnArgs* p) {
  int sms = 0;
  const int st = current_device_context(&p->ctx, &sms);
  if (st != BD_OK) return st;
  p->b = *batch;
  p->L = attn_layout(*batch, sms);
  return BD_OK;
}

// Plan and workspace sizes need the device's SM count; without a device they
// are those of a GB300.
AttnLayout sized_layout(const bd_attention_batch* batch) {
  DevCtx ctx;
  int sms = 0;
  if (current_device_context(&ctx, &sms) != BD_OK) sms = 152;
  return attn_layout(*batch, sms);
}

bd_status run_attention(AttnArgs& p, cudaStream_t s) {
  const bd_attention_batch& b = p.b;
  const uint64_t D = static_cast<uint64_t>(b.head_dim), H = static_cast<uint64_t>(b.n_q_heads);
  const uint64_t rows =
      static_cast<uint64_t>(b.n_pages) * b.n_kv_heads * static_cast<uint64_t>(b.page_size);
  const uint64_t kdims[3] = {64, rows, D / 64};
  const uint64_t kstr[2] = {2 * D, 128};
  const uint32_t box16[3] = {64, 16, static_cast<uint32_t>(D / 64)};
  TileMaps m;
  if (!encode_tmap_bf16_3d(&m.dk, p.k_pages, kdims, kstr, box16) ||
      !encode_tmap_bf16_3d(&m.dv, p.v_pages, kdims, kstr, box16))
    return BD_ERR_CUDA;
  if (p.L.use_tile) {
    const uint32_t box[3] = {64, static_cast<uint32_t>(b.page_size), 1};
    const uint64_t qdims[3] = {D, H, static_cast<uint64_t>(b.n_tokens)};
    const uint64_t qstr[2] = {2 * D, 2 * D * H};
    const uint32_t qbox[3] = {64, static_cast<uint32_t>(p.L.g),
                              static_cast<uint32_t>(p.L.half_tok)};
    if (!encode_tmap_bf16_3d(&m.k, p.k_pages, kdims, kstr, box) ||
        !encode_tmap_bf16_3d(&m.v, p.v_pages, kdims, kstr, box) ||
        !encode_tmap_bf16_3d(&m.q, p.q, qdims, qstr, qbox))
      return BD_ERR_CUDA;
    if (launch_attn_tile(p, m, s) != cudaSuccess) return BD_ERR_CUDA;
  } else if (launch_attn_decode(p, m.dk, m.dv, s) != cudaSuccess) {
    return BD_ERR_CUDA;
  }
  const int64_t items = b.n_tokens * b.n_kv_heads * (b.head_dim / 16);
  const int64_t few = p.L.d_ctas, most = kCombCtas * static_cast<int64_t>(p.L.t_ctas);
  const dim3 grid(static_cast<unsigned>(items < few ? few : (items < most ? items : most)));
  const cudaError_t e = launch_pdl(combine_kernel, grid, dim3(kCombThreads), 0, s, p);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

}  // namespace
}  // namespace bd

extern "C" {

size_t bitdelta_attention_plan_bytes(const bd_attention_batch* batch) {
  if (bd::check_attention_batch(batch) != BD_OK) return 0;
  return bd::sized_layout(batch).plan_bytes;
}

bd_status bitdelta_attention_plan(const bd_attention_batch* batch, void* plan, size_t plan_bytes,
                                  bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (batch->n_tokens == 0) return BD_OK;
  if (!plan) return BD_ERR_WORKSPACE;
  if (bd::off(plan, 256)) return BD_ERR_MISALIGNED;
  bd::AttnArgs p{};
  if ((st = bd::fill_args(batch, &p)) != BD_OK) return static_cast<bd_status>(st);
  if (plan_bytes < p.L.plan_bytes) return BD_ERR_WORKSPACE;
  p.plan = static_cast<uint8_t*>(plan);
  const cudaError_t e = bd::launch_pdl(bd::plan_kernel, dim3(1), dim3(bd::kPlanThreads), 0,
                                       reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

size_t bitdelta_attention_workspace_bytes(const bd_attention_batch* batch) {
  if (bd::check_attention_batch(batch) != BD_OK) return 0;
  return bd::sized_layout(batch).ws_bytes;
}

bd_status bitdelta_attention(const bd_attention_batch* batch, void* plan, size_t plan_bytes,
                             const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                             float scale, uint16_t* out, float* lse, void* workspace,
                             size_t workspace_bytes, bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || std::isinf(scale_log2)) return BD_ERR_INVALID_ARG;
  if (batch->n_tokens == 0) return BD_OK;
  if (!q || !k_pages || !v_pages || !out || batch->n_pages < 1) return BD_ERR_INVALID_ARG;
  if (!plan || !workspace) return BD_ERR_WORKSPACE;
  if (bd::off(q, 16) || bd::off(k_pages, 16) || bd::off(v_pages, 16) || bd::off(out, 16) ||
      bd::off(lse, 4) || bd::off(plan, 256) || bd::off(workspace, 256))
    return BD_ERR_MISALIGNED;
  const size_t tables = sizeof(bd::PlanHeader);  // no plan is smaller
  if (plan_bytes < tables) return BD_ERR_WORKSPACE;
  bd::AttnArgs p{};
  if ((st = bd::fill_args(batch, &p)) != BD_OK) return static_cast<bd_status>(st);
  if (plan_bytes < p.L.plan_bytes || workspace_bytes < p.L.ws_bytes) return BD_ERR_WORKSPACE;
  p.plan = static_cast<uint8_t*>(plan);
  p.ws = static_cast<uint8_t*>(workspace);
  p.q = q;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.scale_log2 = scale_log2;
  p.out = out;
  p.lse = lse;
  return bd::run_attention(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
