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
  int32_t cap;  // keys of a CTA, a multiple of 32
  DevCtx ctx;
};

constexpr int kDigits = 2048;
constexpr int kMaxKeys = 49152;  // of a CTA
constexpr int kMaxLen = 8 * kMaxKeys;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

struct Shared {
  uint32_t digits[3][kDigits];  // counts of the three passes
  uint32_t warp_n[2][32];
  uint32_t found, above;         // a pass' digit, and the keys above it
  uint32_t equal;                // keys that equal the threshold
  uint32_t holes, movers;        // of this CTA
  int bad, prefix;
  // then keys[cap + 64], once they are no longer needed the lists of holes and movers,
  // (cap + 64) / 2 each; and a bit for each key that stays
};

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

// T threads: 256 for few keys, four CTAs an SM, and 1024 for many.
template <int C, int T>
__global__ void __launch_bounds__(T, T == 256 ? 4 : 1) kv_evict_kernel(const EvictArgs p) {
  constexpr int kWarps = T / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  uint32_t* stay = keys + p.cap + 64;  // bits
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
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  for (int g = tid; g < b.n_group; g += T)
    if (b.group_offsets[g] <= s && s < b.group_offsets[g + 1])
      atomicMax(&sh.prefix, b.prefix_len[g]);
  const int kv = b.kv_len[s], keep = p.keep[s];
  const int shift = p.pos_offset != nullptr ? p.pos_offset[s] : 0;
  if (kv < 0 || kv > b.max_kv_len || kv > b.table_stride * b.page_size) {
    if (tid == 0) record_error(p.ctx, kErrBounds);
    return;  // every CTA of the cluster
  }
  __syncthreads();
  const int prefix = prefix_keys(b, sh.prefix, kv);
  const int len = evicted_length(kv, keep, prefix);
  const int32_t* table = b.page_table + static_cast<int64_t>(s) * b.table_stride;
  const int page_shift = 31 - __clz(b.page_size);
  // a slot's row (of this head) in the cache, or −1
  const auto row_of = [&](int slot) -> int64_t {
    const int page = table[slot >> page_shift];
    if (page < 0 || page >= b.n_pages) return -1;
    return ((static_cast<int64_t>(page) * b.n_kv_heads + h) << page_shift) +
           (slot & (b.page_size - 1));
  };
  const bool apart = p.weights_out != p.weights || p.positions_out != p.positions;
  // kBatch slots of a thread at a time, T apart: their rows, weights and positions
  constexpr int kBatch = 8;
  struct Entries {
    int64_t row[kBatch];
    float w[kBatch];
    int pos[kBatch];
  };
  const auto fetch = [&](Entries& e, int slot, int end) {
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      e.row[x] = slot + x * T < end ? row_of(slot + x * T) : -2;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      e.w[x] = e.row[x] >= 0 ? p.weights[e.row[x]] : 0.f;
      e.pos[x] = e.row[x] >= 0 ? p.positions[e.row[x]] : 0;
    }
  };
  bool bad = false;
  if (apart) {  // what is not chosen from
    const int end = len == kv ? kv : prefix;
    for (int slot = rank * T * kBatch + tid; slot < end; slot += C * T * kBatch) {
      Entries e;
      fetch(e, slot, end);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (e.row[x] >= 0) {
          p.weights_out[e.row[x]] = e.w[x];
          p.positions_out[e.row[x]] = e.pos[x];
        }
        bad |= e.row[x] == -1;
      }
    }
    if (bad) record_error(p.ctx, kErrBounds);
    bad = false;
  }
  if (len == kv) return;

  // ---- the keys of slots prefix + [i0, i1)
  const int m = kv - prefix, K = len - prefix;
  const int per = ((m + C - 1) / C + 31) & ~31;
  const int i0 = rank * per < m ? rank * per : m;
  const int n = (i0 + per < m ? i0 + per : m) - i0;
  const int64_t late64 = static_cast<int64_t>(kv) + shift - p.recent;
  const int late = static_cast<int>(late64 > INT32_MAX   ? INT32_MAX
                                    : late64 < INT32_MIN ? INT32_MIN
                                                         : late64);
  for (int i = tid; i < n; i += T * kBatch) {
    Entries e;
    fetch(e, prefix + i0 + i, prefix + i0 + n);
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      if (e.row[x] == -2) break;
      uint32_t key = 0u;
      if (e.row[x] < 0) {
        bad = true;
      } else {
        key = key_of(e.w[x], e.pos[x], late, p.sink);
        atomicAdd(&sh.digits[0][key >> 21], 1u);
        // (all slots that go on; the movers' weights overwrite the freed ones' below)
        if (apart && i0 + i + x * T < K) {
          p.weights_out[e.row[x]] = e.w[x];
          p.positions_out[e.row[x]] = e.pos[x];
        }
      }
      keys[i + x * T] = key;
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

  // ---- the K-th largest key, and how many of its equals stay
  uint32_t threshold = 0u, left = static_cast<uint32_t>(K);
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0};
    const int down = kShift[pass];
    if (pass > 0) {
      const int up = kShift[pass - 1];
      for (int i = tid; i < n; i += T) {
        const uint32_t key = keys[i];
        if (key >> up == threshold >> up) atomicAdd(&sh.digits[pass][key >> down & 0x7FFu], 1u);
      }
      meet();
    }
    // an even share of the digits per thread, from the top
    constexpr int kEach = kDigits / T;
    uint32_t c[kEach];
#pragma unroll
    for (int x = 0; x < kEach; ++x) c[x] = 0u;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint2* d = reinterpret_cast<const uint2*>(peer(r)->digits[pass] + kDigits - kEach * (tid + 1));
#pragma unroll
      for (int x = 0; x < kEach / 2; ++x) {
        const uint2 v = d[x];
        c[kEach - 1 - 2 * x] += v.x;
        c[kEach - 2 - 2 * x] += v.y;
      }
    }
    uint32_t sum = 0u;
#pragma unroll
    for (int x = 0; x < kEach; ++x) sum += c[x];
    const uint32_t inc = warp_inclusive(sum);
    if (lane == 31) sh.warp_n[0][warp] = inc;
    __syncthreads();
    uint32_t above = inc - sum;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) above += i < warp ? sh.warp_n[0][i] : 0u;
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
    if (K > 0) {
      threshold |= sh.found << down;
      left -= sh.above;
    }
  }
  // (K = 0: nothing of the candidates stays)
  const uint32_t equals = K > 0 ? sh.equal : 0u;
  const bool split = left < equals;  // not all of the threshold's equals stay

  // ---- which slots stay: a warp owns a run of them
  const int w_per = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = warp * w_per < n ? warp * w_per : n;
  const int w1 = w0 + w_per < n ? w0 + w_per : n;
  uint32_t equal_at = 0u;  // equals before this warp's slots
  if (split) {
    uint32_t e = 0u;
    for (int i = w0; i < w1; i += 32)
      e += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < w1 && keys[i + lane] == threshold));
    if (lane == 0) sh.warp_n[0][warp] = e;
    __syncthreads();
    if (tid == 0) {
      uint32_t all = 0u;
      for (int i = 0; i < kWarps; ++i) all += sh.warp_n[0][i];
      sh.equal = all;
    }
    for (int i = 0; i < warp; ++i) equal_at += sh.warp_n[0][i];
    meet();
#pragma unroll
    for (int r = 0; r < C; ++r)
      if (r < rank) equal_at += peer(r)->equal;
  }
  uint32_t holes = 0u, movers = 0u;
  // bits of the 32 slots from i on that lie below K
  const auto below = [&](int i) {
    const int d = K - (i0 + i);
    return d >= 32 ? 0xFFFFFFFFu : d <= 0 ? 0u : (1u << d) - 1u;
  };
  for (int i = w0; i < w1; i += 32) {
    const bool live = i + lane < w1;
    const uint32_t key = live ? keys[i + lane] : 0u;
    const uint32_t lives = __ballot_sync(0xFFFFFFFFu, live);
    const uint32_t same = __ballot_sync(0xFFFFFFFFu, live && K > 0 && key == threshold);
    bool stays = live && K > 0 && key > threshold;
    if (same >> lane & 1u)
      stays = !split || equal_at + __popc(same & ((1u << lane) - 1u)) < left;
    equal_at += __popc(same);
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, stays);
    if (lane == 0) stay[i >> 5] = kept;
    holes += __popc(lives & ~kept & below(i));
    movers += __popc(kept & ~below(i));
  }
  __syncthreads();  // the sums of equals have been read
  if (lane == 0) {
    sh.warp_n[0][warp] = holes;
    sh.warp_n[1][warp] = movers;
  }
  __syncthreads();
  uint32_t hole_at = 0u, mover_at = 0u, all_holes = 0u, all_movers = 0u;
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) {
      hole_at = all_holes;
      mover_at = all_movers;
    }
    all_holes += sh.warp_n[0][i];
    all_movers += sh.warp_n[1][i];
  }
  if (tid == 0) {
    sh.holes = all_holes;
    sh.movers = all_movers;
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

  // ---- their numbers: entry e of both lists lies in CTA e / share
  const uint32_t share = (moves + C - 1) / C;
  const int half = (p.cap + 64) / 2;
  const auto put = [&](int list, uint32_t e, int slot) {
    const uint32_t r = C == 1 ? 0u : e / share;
    uint32_t* to = C == 1 ? keys : cluster.map_shared_rank(keys, r);
    to[list * half + (e - r * share)] = static_cast<uint32_t>(slot);
  };
  for (int i = w0; i < w1; i += 32) {
    const uint32_t lives = w1 - i >= 32 ? 0xFFFFFFFFu : (1u << (w1 - i)) - 1u;
    const uint32_t kept = stay[i >> 5], low = below(i);
    const uint32_t hole = lives & ~kept & low, mover = kept & ~low;
    const uint32_t before = (1u << lane) - 1u;
    if (hole >> lane & 1u) put(0, hole_at + __popc(hole & before), prefix + i0 + i + lane);
    if (mover >> lane & 1u) put(1, mover_at + __popc(mover & before), prefix + i0 + i + lane);
    hole_at += __popc(hole);
    mover_at += __popc(mover);
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
        to[x] = row_of(static_cast<int>(keys[e]));
        const int64_t from = row_of(static_cast<int>(keys[half + e]));
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

__global__ void __launch_bounds__(256)
    evict_lengths_kernel(const bd_attention_batch b, const int32_t* keep, int32_t* kv_len_out,
                         int32_t* pos_offset, DevCtx ctx) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= b.n_seq) return;
  const int kv = b.kv_len[s];
  if (kv < 0 || kv > b.max_kv_len) {
    record_error(ctx, kErrBounds);
    return;
  }
  int prefix = 0;
  for (int g = 0; g < b.n_group; ++g)
    if (b.group_offsets[g] <= s && s < b.group_offsets[g + 1] && b.prefix_len[g] > prefix)
      prefix = b.prefix_len[g];
  const int len = evicted_length(kv, keep[s], prefix_keys(b, prefix, kv));
  kv_len_out[s] = len;
  pos_offset[s] += kv - len;
}

size_t smem_bytes(int cap) {
  return sizeof(Shared) + 4 * (static_cast<size_t>(cap) + 64) + static_cast<size_t>(cap) / 8;
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
                               static_cast<int>(smem_bytes(kMaxKeys)));
      if (e == cudaSuccess && C > 8)
        e = cudaFuncSetAttribute(kv_evict_kernel<C, T>,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  static_assert(sizeof(Shared) + 4 * (kMaxKeys + 64) + kMaxKeys / 8 <= 227 * 1024,
                "shared memory of one CTA");
  const unsigned grid = static_cast<unsigned>(p.b.n_seq) * p.b.n_kv_heads * C;
  return launch_pdl_cluster(kv_evict_kernel<C, T>, dim3(grid), dim3(T), C, smem_bytes(p.cap), s, p);
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
    const size_t bytes = smem_bytes(kMaxLen / 16);
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
  if (batch->max_kv_len > bd::kMaxLen) return BD_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<int64_t>(batch->n_seq) * batch->n_kv_heads > (1 << 27))
    return BD_ERR_UNSUPPORTED_SHAPE;
  if (batch->n_seq == 0) return BD_OK;
  if (!batch->page_table || !k_pages || !v_pages || !weights || !positions || !weights_out ||
      !positions_out)
    return BD_ERR_INVALID_ARG;
  if (bd::off(batch->page_table, 4) || bd::off(pos_offset, 4) || bd::off(k_pages, 16) ||
      bd::off(v_pages, 16) || bd::off(weights, 4) || bd::off(positions, 4) ||
      bd::off(weights_out, 4) || bd::off(positions_out, 4))
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
  // has SMs left for them and each still has 2048.  Where there are more CTAs than SMs,
  // and few keys each, they have 256 threads, which leaves an SM four of them: their
  // phases wait for one another.
  const int64_t items = static_cast<int64_t>(batch->n_seq) * batch->n_kv_heads;
  const int len = batch->max_kv_len;
  int c = 1;
  while (c < 8 && (len > bd::kMaxKeys * c || (items * 2 * c <= sms && len > 2048 * c))) c *= 2;
  if (c == 8 && items * 16 <= sms && len > 2048 * 8 && bd::large_clusters() >= items) c = 16;
  p.cap = ((len + c - 1) / c + 31) / 32 * 32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool few = p.cap <= 8192 && items * c > sms;
  cudaError_t e;
  switch (c) {
    case 1: e = few ? bd::launch<1, 256>(p, s) : bd::launch<1, 1024>(p, s); break;
    case 2: e = few ? bd::launch<2, 256>(p, s) : bd::launch<2, 1024>(p, s); break;
    case 4: e = few ? bd::launch<4, 256>(p, s) : bd::launch<4, 1024>(p, s); break;
    case 8: e = few ? bd::launch<8, 256>(p, s) : bd::launch<8, 1024>(p, s); break;
    default: e = few ? bd::launch<16, 256>(p, s) : bd::launch<16, 1024>(p, s); break;
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
  if (bd::off(kv_len_out, 4) || bd::off(pos_offset, 4)) return BD_ERR_MISALIGNED;
  bd::DevCtx ctx;
  int sms = 0;
  if ((st = bd::current_device_context(&ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  const unsigned grid = (static_cast<unsigned>(batch->n_seq) + 255) / 256;
  const cudaError_t e =
      bd::launch_pdl(bd::evict_lengths_kernel, dim3(grid), dim3(256), 0,
                     reinterpret_cast<cudaStream_t>(stream), *batch, keep, kv_len_out, pos_offset,
                     ctx);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

}  // extern "C"
