// kv_evict.cu — a paged cache held to a budget (bitdelta_kv_evict,
// bitdelta_kv_evict_lengths).
//
// Per sequence and key head: of m slots the K that rank highest stay (protected
// ones, then by weight, equal ones by the lowest slot).  Attention does not depend
// on the order of the keys, so only the ones that stay in slots from K on move,
// each into a slot below K that came free: no row is read and written by the same
// eviction, and a step over the budget moves as few rows as it drops.
//
// A cluster of CTAs holds the ranks of one sequence and key head in shared memory
// as 32-bit keys in the order of the choice.  The K-th largest key is found digit
// by digit (11, 11 and 10 bits) from counts that every CTA reads of the whole
// cluster.  The free slots and the ones that move into them are numbered by
// prefix sums and exchanged over distributed shared memory, so that each CTA moves
// an even share.
//
// Bound by the weights' bytes and the moves at best; with few of either by the chain of
// phases between barriers.  Measured (152 SMs, 8 key heads of 128): 64 sequences of 4097
// to 4160 keys to 4096 21.0 us; four of 8192 to 1024 14.8 us; one of 131071 to 65536
// 83 us, of which 52 are 270 MB of moves (70% of the copy rate in rows of 256 bytes).
#include <cooperative_groups.h>

#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);

namespace {

namespace cg = cooperative_groups;

struct EvictArgs {
  bd_attention_batch b;
  const int32_t* keep;
  int32_t recent, sink;
  const int32_t* pos_offset;
  uint16_t *k_pages, *v_pages;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int32_t cap;  // keys of a CTA, a multiple of 128
  DevCtx ctx;
};

constexpr int kDigits = 2048;
constexpr int kMaxKeys = 43008;  // of a CTA
constexpr int kMaxLen = 8 * kMaxKeys;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

struct alignas(16) Shared {  // what follows it is read 16 bytes at a time
  uint32_t digits[3][kDigits];  // counts of the three passes
  uint32_t warp_n[2][32];
  uint32_t found, above;         // a pass' digit, and the keys above it
  uint32_t equal;                // keys that equal the threshold
  uint32_t n_list, n_few;        // keys with the threshold's digits so far: of this CTA, of all
  uint32_t holes, movers;        // of this CTA
  int bad, prefix;
  // then keys[cap + 256], once they are no longer needed the lists of holes' and movers'
  // rows, (cap + 256) / 2 each; a byte for four slots: holes, movers; and in a cluster
  // total[kDigits], a pass' counts in all of it
};

// Whether a length lies within the batch's bounds, and a page within the cache.  A sequence
// of which one of them does not (of the pages, those that are chosen from) is refused, by
// the eviction and by the update of the lengths alike.
__device__ __forceinline__ bool length_fits(const bd_attention_batch& b, int kv) {
  return kv >= 0 && kv <= b.max_kv_len && kv <= b.table_stride * b.page_size;
}
__device__ __forceinline__ bool page_fits(const bd_attention_batch& b, int page) {
  return page >= 0 && page < b.n_pages;
}
// New length of a sequence of kv keys whose first `prefix` are shared.
__device__ __forceinline__ int evicted_length(int kv, int keep, int prefix) {
  if (keep < 0 || keep >= kv) return kv;
  return keep > prefix ? keep : prefix;
}
// The whole pages of a group's prefix, at most kv keys.
__device__ __forceinline__ int prefix_keys(const bd_attention_batch& b, int len, int kv) {
  len = len > 0 ? len / b.page_size * b.page_size : 0;
  return len < kv ? len : kv;
}

__device__ __forceinline__ uint32_t key_of(float w, int position, int late, int sink) {
  if (position >= late || position < sink) return kProtected;
  if (isnan(w)) return 0u;
  const uint32_t bits = __float_as_uint(w + 0.f);  // −0 as 0
  return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

template <typename T>
__device__ __forceinline__ T warp_inclusive(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T o = __shfl_up_sync(0xFFFFFFFFu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// T threads: 256, 512 or 1024, and four, two or one CTA an SM.
template <int C, int T>
__global__ void __launch_bounds__(T, 1024 / T) kv_evict_kernel(const EvictArgs p) {
  constexpr int kWarps = T / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  uint8_t* stay = reinterpret_cast<uint8_t*>(keys + p.cap + 256);  // two bits a slot
  uint32_t* total = reinterpret_cast<uint32_t*>(stay + p.cap / 4);
  const bd_attention_batch& b = p.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const uint32_t item = blockIdx.x / C;
  const int s = static_cast<int>(item / static_cast<uint32_t>(b.n_kv_heads));
  const int h = static_cast<int>(item - static_cast<uint32_t>(s) * b.n_kv_heads);
  const auto meet = [&] {
    if constexpr (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  const auto peer = [&](int r) { return C == 1 ? &sh : cluster.map_shared_rank(&sh, r); };

  for (int i = tid; i < 3 * kDigits; i += T) (&sh.digits[0][0])[i] = 0u;
  if (tid == 0) {
    sh.bad = 0;
    sh.prefix = 0;
    sh.n_list = 0;
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  for (int g = tid; g < b.n_group; g += T)
    if (b.group_offsets[g] <= s && s < b.group_offsets[g + 1])
      atomicMax(&sh.prefix, b.prefix_len[g]);
  const int kv = b.kv_len[s], keep = p.keep[s];
  const int shift = p.pos_offset != nullptr ? p.pos_offset[s] : 0;
  if (!length_fits(b, kv)) {
    if (tid == 0) record_error(p.ctx, kErrBounds);
    return;  // every CTA of the cluster
  }
  __syncthreads();
  const int prefix = prefix_keys(b, sh.prefix, kv);
  const int len = evicted_length(kv, keep, prefix);
  const int32_t* table = b.page_table + static_cast<int64_t>(s) * b.table_stride;
  const int page_shift = 31 - __clz(b.page_size);
  // a slot's row (of this head) in the cache, or −1
  const auto row_of = [&](int slot) {
    const int page = table[slot >> page_shift];
    if (!page_fits(b, page)) return -1;
    return ((page * b.n_kv_heads + h) << page_shift) + (slot & (b.page_size - 1));
  };
  const bool apart = p.weights_out != p.weights || p.positions_out != p.positions;
  // Four neighbouring slots of a thread, which lie in one page (slots are counted from a
  // page's start, pages hold 16 and more), and kBatch of these at a time, T apart.
  constexpr int kBatch = 2;
  struct Entries {
    int row[kBatch];  // of the first slot (below 2^31), −1: no such page, −2: past the end
    float4 w[kBatch];
    int4 pos[kBatch];
  };
  const auto fetch = [&](Entries& e, int slot, int end) {
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      e.row[x] = slot + 4 * x * T < end ? row_of(slot + 4 * x * T) : -2;
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      if (e.row[x] >= 0) {
        e.w[x] = *reinterpret_cast<const float4*>(p.weights + e.row[x]);
        e.pos[x] = *reinterpret_cast<const int4*>(p.positions + e.row[x]);
      }
  };
  // the first `live` of four
  const auto put = [&](int row, int live, const float4& w, const int4& pos) {
    if (live >= 4) {
      *reinterpret_cast<float4*>(p.weights_out + row) = w;
      *reinterpret_cast<int4*>(p.positions_out + row) = pos;
      return;
    }
    const float ws[3] = {w.x, w.y, w.z};
    const int ps[3] = {pos.x, pos.y, pos.z};
#pragma unroll
    for (int y = 0; y < 3; ++y)
      if (y < live) {
        p.weights_out[row + y] = ws[y];
        p.positions_out[row + y] = ps[y];
      }
  };
  bool bad = false;
  if (apart) {  // what is not chosen from
    const int end = len == kv ? kv : prefix;
    for (int slot = 4 * (rank * T * kBatch + tid); slot < end; slot += 4 * C * T * kBatch) {
      Entries e;
      fetch(e, slot, end);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (e.row[x] >= 0) put(e.row[x], end - slot - 4 * x * T, e.w[x], e.pos[x]);
        bad |= e.row[x] == -1;
      }
    }
    if (bad) record_error(p.ctx, kErrBounds);
    bad = false;
  }
  if (len == kv) return;

  // ---- the keys of slots prefix + [i0, i1)
  const int m = kv - prefix, K = len - prefix;
  const int per = ((m + C - 1) / C + 127) & ~127;
  const int i0 = rank * per < m ? rank * per : m;
  const int n = (i0 + per < m ? i0 + per : m) - i0;
  const int64_t late64 = static_cast<int64_t>(kv) + shift - p.recent;
  const int late = static_cast<int>(late64 > INT32_MAX   ? INT32_MAX
                                    : late64 < INT32_MIN ? INT32_MIN
                                                         : late64);
  for (int i = 4 * tid; i < n; i += 4 * T * kBatch) {
    Entries e;
    fetch(e, prefix + i0 + i, prefix + i0 + n);
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      if (e.row[x] == -2) break;
      const int at = i + 4 * x * T;
      uint32_t key[4] = {0u, 0u, 0u, 0u};
      if (e.row[x] < 0) {
        bad = true;
      } else {
        const float w[4] = {e.w[x].x, e.w[x].y, e.w[x].z, e.w[x].w};
        const int pos[4] = {e.pos[x].x, e.pos[x].y, e.pos[x].z, e.pos[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (at + y >= n) continue;
          key[y] = key_of(w[y], pos[y], late, p.sink);
          atomicAdd(&sh.digits[0][key[y] >> 21], 1u);
        }
        // (all slots that go on; the movers' weights overwrite the freed ones' below)
        if (apart && i0 + at < K) put(e.row[x], K - i0 - at, e.w[x], e.pos[x]);
      }
      *reinterpret_cast<uint4*>(keys + at) = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  if (bad) sh.bad = 1;
  meet();
  bool any_bad = false;
#pragma unroll
  for (int r = 0; r < C; ++r) any_bad |= peer(r)->bad != 0;
  if (any_bad) {
    if (tid == 0) record_error(p.ctx, kErrBounds);
    meet();  // the flags have been read
    return;
  }

  // the sum of what the warps before this one have
  const auto before = [&](const uint32_t* n) {
    return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? n[lane] : 0u);
  };
  // ---- the K-th largest key, and how many of its equals stay (K = 0: none of them), by
  // digits from the top.  (Rolled: this runs once, and its instructions are fetched for it.)
  // Where the keys that have the digits so far are few, every CTA of a cluster takes them
  // all, and the passes that are left need nothing of the others.  (Over all keys two passes
  // took 10600 cycles by a cluster of four, so 4700, and four prompts 19.1 -> 15.0 us.  A
  // CTA by itself passes over 4160 keys in 2300, and making the list took it 3700.)
  constexpr int kFew = 1024, kPer = kFew / T;
  uint32_t threshold = 0u, left = static_cast<uint32_t>(K), equals = 0u;
  bool few = false;
  uint32_t cand[kPer];
#pragma unroll 1
  for (int pass = 0; pass < 3 && K > 0; ++pass) {
    const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int up = pass == 1 ? 21 : 10;  // of the pass before
    uint32_t* digits = sh.digits[pass];
    if (few) {
#pragma unroll
      for (int x = 0; x < kPer; ++x)
        if (static_cast<uint32_t>(tid + x * T) < sh.n_few && cand[x] >> up == threshold >> up)
          atomicAdd(&digits[cand[x] >> down & 0x7FFu], 1u);
      __syncthreads();
    } else if (pass > 0) {
#pragma unroll 2
      for (int i = 4 * tid; i < n; i += 4 * T) {
        const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (i + y < n && key[y] >> up == threshold >> up)
            atomicAdd(&digits[key[y] >> down & 0x7FFu], 1u);
      }
      meet();
    }
    // The cluster's counts: every CTA adds up a share of the digits and gives it to all.
    // (All digits of all CTAs read by each took 64 KB of the others' memory a pass, 13 us
    // of three passes by eight CTAs.)
    if (C > 1 && !few) {
      constexpr int kShare = kDigits / C;
      for (int d = rank * kShare + tid; d < (rank + 1) * kShare; d += T) {
        uint32_t count = 0u;
#pragma unroll
        for (int r = 0; r < C; ++r) count += peer(r)->digits[pass][d];
#pragma unroll
        for (int r = 0; r < C; ++r) cluster.map_shared_rank(total, r)[d] = count;
      }
      meet();
    }
    // an even share of the digits per thread, from the top
    constexpr int kEach = kDigits / T;
    uint32_t c[kEach];
    {
      const uint2* d = reinterpret_cast<const uint2*>((C > 1 && !few ? total : digits) + kDigits -
                                                      kEach * (tid + 1));
#pragma unroll
      for (int x = 0; x < kEach / 2; ++x) {
        const uint2 v = d[x];
        c[kEach - 1 - 2 * x] = v.x;
        c[kEach - 2 - 2 * x] = v.y;
      }
    }
    uint32_t sum = 0u;
#pragma unroll
    for (int x = 0; x < kEach; ++x) sum += c[x];
    const uint32_t inc = warp_inclusive(sum);
    if (lane == 31) sh.warp_n[0][warp] = inc;
    __syncthreads();
    uint32_t above = inc - sum + before(sh.warp_n[0]);
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      if (above < left && left <= above + c[x]) {
        sh.found = static_cast<uint32_t>(kDigits - 1 - kEach * tid - x);
        sh.above = above;
        sh.equal = c[x];
      }
      above += c[x];
    }
    __syncthreads();
    threshold |= sh.found << down;
    left -= sh.above;
    equals = sh.equal;
    if (C == 1 || few || pass == 2 || equals > kFew) continue;
    few = true;
    // this CTA's in place of the pass' digits, which all have read
    for (int i = 4 * tid; i - 4 * lane < n; i += 4 * T) {
      uint32_t key[4] = {0u, 0u, 0u, 0u}, hit = 0u;
      if (i < n) {
        const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
        key[0] = v.x, key[1] = v.y, key[2] = v.z, key[3] = v.w;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          hit |= (i + y < n && key[y] >> down == threshold >> down ? 1u : 0u) << y;
      }
      if (!__any_sync(0xFFFFFFFFu, hit != 0)) continue;
      const uint32_t inc = warp_inclusive(static_cast<uint32_t>(__popc(hit)));
      uint32_t at = lane == 31 ? atomicAdd(&sh.n_list, inc) : 0u;
      at = __shfl_sync(0xFFFFFFFFu, at, 31) + inc - __popc(hit);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (hit >> y & 1u) digits[at++] = key[y];
    }
    if (tid == 0) sh.n_few = equals;
    meet();
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      uint32_t at = tid + x * T;  // of all CTAs' lists
      cand[x] = 0u;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const uint32_t n_list = peer(r)->n_list;
        if (at < n_list) cand[x] = peer(r)->digits[pass][at];
        at = at < n_list ? UINT32_MAX : at - n_list;
      }
    }
  }
  const bool split = left < equals;  // not all of the threshold's equals stay

  // ---- which slots stay: a warp owns a run of them, a lane four neighbours
  const int w_per = ((n + kWarps - 1) / kWarps + 127) & ~127;
  const int w0 = warp * w_per < n ? warp * w_per : n;
  const int w1 = w0 + w_per < n ? w0 + w_per : n;
  uint32_t equal_at = 0u;  // equals before this warp's slots
  if (split) {
    uint32_t e = 0u;
    for (int i = w0 + 4 * lane; i < w1; i += 128) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) e += i + y < w1 && key[y] == threshold;
    }
    e = __reduce_add_sync(0xFFFFFFFFu, e);
    if (lane == 0) sh.warp_n[0][warp] = e;
    __syncthreads();
    equal_at = before(sh.warp_n[0]);
    if (tid == T - 1) sh.equal = equal_at + e;
    meet();
#pragma unroll
    for (int r = 0; r < C; ++r)
      if (r < rank) equal_at += peer(r)->equal;
  }
  // of four slots from i on, those that lie below K
  const auto below = [&](int i) {
    const int d = K - (i0 + i);
    return d >= 4 ? 15u : d <= 0 ? 0u : (1u << d) - 1u;
  };
  uint32_t holes = 0u, movers = 0u;
  for (int i = w0 + 4 * lane; i - 4 * lane < w1; i += 128) {
    uint32_t key[4] = {0u, 0u, 0u, 0u}, lives = 0u, same = 0u, kept = 0u;
    if (i < w1) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      key[0] = v.x, key[1] = v.y, key[2] = v.z, key[3] = v.w;
      lives = w1 - i >= 4 ? 15u : (1u << (w1 - i)) - 1u;
    }
    if (K > 0) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        kept |= (key[y] > threshold ? 1u : 0u) << y;
        same |= (key[y] == threshold ? 1u : 0u) << y;
      }
      same &= lives;
      if (!split) {
        kept |= same;
      } else {
        const uint32_t inc = warp_inclusive(static_cast<uint32_t>(__popc(same)));
        uint32_t at = equal_at + inc - __popc(same);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (same >> y & 1u) kept |= (at++ < left ? 1u : 0u) << y;
        equal_at += __shfl_sync(0xFFFFFFFFu, inc, 31);
      }
      kept &= lives;
    }
    const uint32_t low = below(i);
    const uint32_t hole = lives & ~kept & low, mover = kept & ~low;
    if (i < w1) stay[i >> 2] = static_cast<uint8_t>(hole | mover << 4);
    holes += __popc(hole);
    movers += __popc(mover);
  }
  holes = __reduce_add_sync(0xFFFFFFFFu, holes);
  movers = __reduce_add_sync(0xFFFFFFFFu, movers);
  __syncthreads();  // the sums of equals have been read
  if (lane == 0) {
    sh.warp_n[0][warp] = holes;
    sh.warp_n[1][warp] = movers;
  }
  __syncthreads();
  uint32_t hole_at = before(sh.warp_n[0]), mover_at = before(sh.warp_n[1]);
  if (tid == T - 1) {
    sh.holes = hole_at + holes;
    sh.movers = mover_at + movers;
  }
  meet();  // and all keys have been read
  uint32_t moves = 0u;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const Shared* o = peer(r);
    if (r < rank) {
      hole_at += o->holes;
      mover_at += o->movers;
    }
    moves += o->movers;
  }

  // ---- their rows: entry e of both lists lies in CTA e / share
  const uint32_t share = (moves + C - 1) / C;
  const int half = (p.cap + 256) / 2;
  const auto note = [&](int list, uint32_t e, int row) {
    const uint32_t r = C == 1 ? 0u : e / share;
    uint32_t* to = C == 1 ? keys : cluster.map_shared_rank(keys, r);
    to[list * half + (e - r * share)] = static_cast<uint32_t>(row);
  };
  for (int i = w0 + 4 * lane; i - 4 * lane < w1; i += 128) {
    const uint32_t bits = i < w1 ? stay[i >> 2] : 0u;
    if (__ballot_sync(0xFFFFFFFFu, bits != 0) == 0) continue;
    const uint32_t hole = bits & 15u, mover = bits >> 4;
    // both numbers in one sum
    const uint32_t mine = __popc(hole) | __popc(mover) << 16;
    const uint32_t inc = warp_inclusive(mine);
    uint32_t e = hole_at + ((inc - mine) & 0xFFFFu), f = mover_at + ((inc - mine) >> 16);
    if (bits != 0) {
      const int row = row_of(prefix + i0 + i);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (hole >> y & 1u) note(0, e++, row + y);
        if (mover >> y & 1u) note(1, f++, row + y);
      }
    }
    const uint32_t all = __shfl_sync(0xFFFFFFFFu, inc, 31);
    hole_at += all & 0xFFFFu;
    mover_at += all >> 16;
  }
  meet();

  // ---- the moves: a row of 16-byte pieces per group of lanes
  const uint32_t first = rank * share;
  const int mine = first < moves ? static_cast<int>(moves - first < share ? moves - first : share) : 0;
  const int lanes = b.head_dim >> 3;  // per row
  const int rows = 32 / lanes;        // rows a warp moves at once, of keys or values
  const int sub = lane / lanes, at = lane - sub * lanes;
  constexpr int kMoves = 4;
  for (int e0 = warp * rows; e0 < mine; e0 += kMoves * kWarps * rows) {
    uint4 k[kMoves], v[kMoves];
    int64_t to[kMoves];
    float w[kMoves];
    int pos[kMoves];
#pragma unroll
    for (int x = 0; x < kMoves; ++x) {
      const int e = e0 + x * kWarps * rows + sub;
      to[x] = -1;
      if (e < mine) {
        to[x] = keys[e];
        const int64_t from = keys[half + e];
        k[x] = reinterpret_cast<const uint4*>(p.k_pages + from * b.head_dim)[at];
        v[x] = reinterpret_cast<const uint4*>(p.v_pages + from * b.head_dim)[at];
        w[x] = p.weights[from];
        pos[x] = p.positions[from];
      }
    }
#pragma unroll
    for (int x = 0; x < kMoves; ++x) {
      if (to[x] < 0) continue;
      reinterpret_cast<uint4*>(p.k_pages + to[x] * b.head_dim)[at] = k[x];
      reinterpret_cast<uint4*>(p.v_pages + to[x] * b.head_dim)[at] = v[x];
      if (at == 0) {
        p.weights_out[to[x]] = w[x];
        p.positions_out[to[x]] = pos[x];
      }
    }
  }
}

constexpr int kLengthThreads = 128;

// A CTA per sequence, as the page-table row of one that is cut has to be read (a thread per
// sequence without that took 2.3 us for 64 sequences, this 2.4; one of 131071 keys in pages
// of 16 takes 4.8).
__global__ void __launch_bounds__(kLengthThreads)
    evict_lengths_kernel(const bd_attention_batch b, const int32_t* keep, int32_t* kv_len_out,
                         int32_t* pos_offset, DevCtx ctx) {
  __shared__ int s_prefix;
  const int s = static_cast<int>(blockIdx.x), tid = threadIdx.x;
  if (tid == 0) s_prefix = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  for (int g = tid; g < b.n_group; g += kLengthThreads)
    if (b.group_offsets[g] <= s && s < b.group_offsets[g + 1])
      atomicMax(&s_prefix, b.prefix_len[g]);
  const int kv = b.kv_len[s], keeps = keep[s];
  __syncthreads();
  bool fits = length_fits(b, kv);
  const int prefix = fits ? prefix_keys(b, s_prefix, kv) : 0;
  const int len = fits ? evicted_length(kv, keeps, prefix) : kv;
  if (len != kv && b.page_table != nullptr && b.n_pages > 0) {
    const int32_t* table = b.page_table + static_cast<int64_t>(s) * b.table_stride;
    const int page_shift = 31 - __clz(b.page_size);
    for (int i = (prefix >> page_shift) + tid; i <= (kv - 1) >> page_shift; i += kLengthThreads)
      fits &= page_fits(b, table[i]);
  }
  fits = __syncthreads_and(fits);  // and kv_len[s], which may be kv_len_out[s], has been read
  if (tid != 0) return;
  if (!fits) record_error(ctx, kErrBounds);
  kv_len_out[s] = fits ? len : kv;
  if (fits) pos_offset[s] += kv - len;
}

constexpr size_t smem_bytes(int cap, int c) {
  return sizeof(Shared) + 4 * (static_cast<size_t>(cap) + 256) + static_cast<size_t>(cap) / 4 +
         (c > 1 ? 4 * kDigits : 0);
}

template <int C, int T>
cudaError_t launch(const EvictArgs& p, cudaStream_t s) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(kv_evict_kernel<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem_bytes(kMaxKeys, C)));
      if (e == cudaSuccess && C > 8)
        e = cudaFuncSetAttribute(kv_evict_kernel<C, T>,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  static_assert(smem_bytes(kMaxKeys, C) <= 227 * 1024, "shared memory of one CTA");
  const unsigned grid = static_cast<unsigned>(p.b.n_seq) * p.b.n_kv_heads * C;
  return launch_pdl_cluster(kv_evict_kernel<C, T>, dim3(grid), dim3(T), C, smem_bytes(p.cap, C), s, p);
}

// Clusters of 16 that the device holds at once with the most shared memory that the
// choice below gives them (half of the keys of the longest); 0 where it holds none.
int large_clusters() {
  static int known[64] = {};  // plus one
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(host_cache_mutex());
  int& n = known[dev & 63];
  if (n == 0) {
    const size_t bytes = smem_bytes(kMaxLen / 16, 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    const auto kernel = kv_evict_kernel<16, 1024>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes)) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      count = 0;
    }
    n = count + 1;
  }
  return n - 1;
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// The batch as far as an eviction looks at it.
int check_batch(const bd_attention_batch* b, const int32_t* keep) {
  const int st = check_attention_batch(b);
  if (st != BD_OK) return st;
  if (b->max_kv_len > kMaxLen || static_cast<int64_t>(b->n_seq) * b->n_kv_heads > (1 << 27))
    return BD_ERR_UNSUPPORTED_SHAPE;
  if (b->n_seq == 0) return BD_OK;
  if (!b->kv_len || !keep) return BD_ERR_INVALID_ARG;
  if (b->n_group > 0 && (!b->group_offsets || !b->prefix_len)) return BD_ERR_INVALID_ARG;
  if (off(b->kv_len, 4) || off(keep, 4) || off(b->group_offsets, 4) || off(b->prefix_len, 4))
    return BD_ERR_MISALIGNED;
  return BD_OK;
}

}  // namespace
}  // namespace bd

extern "C" {

bd_status bitdelta_kv_evict(const bd_attention_batch* batch, const int32_t* keep, int32_t recent,
                            int32_t sink, const int32_t* pos_offset, uint16_t* k_pages,
                            uint16_t* v_pages, const float* weights, const int32_t* positions,
                            float* weights_out, int32_t* positions_out, bd_stream_t stream) {
  int st = bd::check_batch(batch, keep);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (recent < 0 || sink < 0) return BD_ERR_INVALID_ARG;
  if (batch->n_seq == 0) return BD_OK;
  if (!batch->page_table || !k_pages || !v_pages || !weights || !positions || !weights_out ||
      !positions_out)
    return BD_ERR_INVALID_ARG;
  if (bd::off(batch->page_table, 4) || bd::off(pos_offset, 4) || bd::off(k_pages, 16) ||
      bd::off(v_pages, 16) || bd::off(weights, 16) || bd::off(positions, 16) ||
      bd::off(weights_out, 16) || bd::off(positions_out, 16))
    return BD_ERR_MISALIGNED;
  bd::EvictArgs p{};
  int sms = 0;
  if ((st = bd::current_device_context(&p.ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  p.b = *batch;
  p.keep = keep;
  p.recent = recent;
  p.sink = sink;
  p.pos_offset = pos_offset;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.weights = weights;
  p.positions = positions;
  p.weights_out = weights_out;
  p.positions_out = positions_out;
  // CTAs per sequence and key head: as many as the keys need, and more while the device
  // has SMs left for them (clusters fill 0.85 of it) and each still has 2048.  Threads:
  // where each SM has a CTA, as many as its keys keep busy; where there are more CTAs, few,
  // so that several share an SM, whose phases wait for one another.  Over 164 sizes (8 to
  // 1024 items of 300 to 32768 keys) the choice costs 2.3% more than the best of 1 to 8
  // CTAs of 256, 512 and 1024 threads.  (us, keys x items to 98%, CTAs of threads: 4160 x
  // 512 29.3 by 1 of 256, 33.4 of 512, 45.7 of 1024; 16384 x 512 103, 83 and 97; 8192 x 64
  // 27.3, 21.2 and 19.1; 32768 x 16 25.2 by 4 of 1024, 43.6 by 8, of which not all run at
  // once.)
  const int64_t items = static_cast<int64_t>(batch->n_seq) * batch->n_kv_heads;
  const int len = batch->max_kv_len;
  int c = 1;
  while (c < 8 && (len > bd::kMaxKeys * c || (items * 2 * c <= 0.85 * sms && len > 2048 * c)))
    c *= 2;
  if (c == 8 && items * 16 <= sms && len > 2048 * 8 && bd::large_clusters() >= items) c = 16;
  p.cap = ((len + c - 1) / c + 127) / 128 * 128;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int few = items <= sms ? 512 : 4608, some = items <= sms ? 2048 : 16384;
  const bool half = p.cap <= 4096;
  cudaError_t e;
  switch (c) {
    case 1:
      e = len <= few    ? bd::launch<1, 256>(p, s)
          : len <= some ? bd::launch<1, 512>(p, s)
                        : bd::launch<1, 1024>(p, s);
      break;
    case 2: e = half ? bd::launch<2, 512>(p, s) : bd::launch<2, 1024>(p, s); break;
    case 4: e = half ? bd::launch<4, 512>(p, s) : bd::launch<4, 1024>(p, s); break;
    case 8: e = half ? bd::launch<8, 512>(p, s) : bd::launch<8, 1024>(p, s); break;
    default: e = bd::launch<16, 1024>(p, s); break;
  }
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

bd_status bitdelta_kv_evict_lengths(const bd_attention_batch* batch, const int32_t* keep,
                                    int32_t* kv_len_out, int32_t* pos_offset,
                                    bd_stream_t stream) {
  int st = bd::check_batch(batch, keep);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (batch->n_seq == 0) return BD_OK;
  if (!kv_len_out || !pos_offset) return BD_ERR_INVALID_ARG;
  if (bd::off(batch->page_table, 4) || bd::off(kv_len_out, 4) || bd::off(pos_offset, 4))
    return BD_ERR_MISALIGNED;
  bd::DevCtx ctx;
  int sms = 0;
  if ((st = bd::current_device_context(&ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  const cudaError_t e =
      bd::launch_pdl(bd::evict_lengths_kernel, dim3(static_cast<unsigned>(batch->n_seq)),
                     dim3(bd::kLengthThreads), 0, reinterpret_cast<cudaStream_t>(stream), *batch,
                     keep, kv_len_out, pos_offset, ctx);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

}  // extern "C"
