// kv_weigh.cu — the attention weight that each cached key got from a step's
// queries, added to a table beside the cache (bitdelta_kv_weigh).
//
//   a[p] = Σ over rows (query token, query head) of exp(scale·q·k_p − lse)
//
// The attention has left each row's lse, so a weight needs no second pass: the
// keys are read once and the values not at all.
//
// Runs of at most 16 rows (single tokens, as a rule) are this file's, whose time is
// reading the keys; longer ones are kv_weigh_tile.cu's, on the tensor cores, whose
// parts of blocks are joined here.
//
// A unit is 16 keys of a run and key head; every warp has an even share of all units,
// in the order of runs, heads and keys.  The keys are the rows of mma.sync tiles (16
// keys by 8 query rows by 16 elements), so that a key's sum stays in its four lanes,
// and are loaded straight from memory to registers, 16 bytes a lane: which of a row's
// elements a lane holds is the same for keys and queries, and a product's sum does not
// care about their order.  Scores, powers and sums are fp32; keys and queries are the
// cache's bf16.
//
// Bound by the keys' bytes.  Measured (152 SMs, 64 query and 8 key heads of 128):
// 64 tokens over 500 to 8000 keys 93.5 us, 575 MB at 91% of the copy rate; one over
// 131071 keys 46.6 us, 88%; 8 over 120 to 1000 keys 7.0 us, most of it five accesses
// in a row (lengths, page, key, product, store).
#include <cmath>
#include <cstdint>

#include "attention.cuh"
#include "kv_weigh.cuh"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitKeys = 16;
static_assert(kThreads == kWeighBlockKeys, "the join takes a key per thread");

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Units per key head of a run: none where the tile kernel has it.
__device__ __forceinline__ int units_of(const WeighArgs& p, const WeighRun& x) {
  const int64_t rows =
      static_cast<int64_t>(x.tok1 - x.tok0) * (p.b.n_q_heads / p.b.n_kv_heads);
  return rows <= kWeighShortRows && x.k1 > x.k0 ? (x.k1 - x.k0 + kUnitKeys - 1) / kUnitKeys : 0;
}

// The blocks that several CTAs of the tile kernel share: their parts in their order.
// (As a rule two, of neighbouring CTAs, in the next place or the one behind it: these are
// loaded before it is known which.)
__device__ void join_parts(const WeighArgs& p) {
  const int n = 2 * p.tile_ctas;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    constexpr int kAhead = 3;
    uint32_t f[kAhead];
    float v[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      f[x] = i + x < n ? p.records[i + x] : 0u;
      v[x] = i + x < n ? p.parts[static_cast<int64_t>(i + x) * kWeighBlockKeys + threadIdx.x] : 0.f;
    }
    const int32_t to = p.rows[static_cast<int64_t>(i) * kWeighBlockKeys + threadIdx.x];
    if ((f[0] & kWeighBegins) == 0) continue;
    const float old = to >= 0 ? p.weights[to] : 0.f;
    float a = v[0];
    bool more = (f[0] & kWeighEnds) == 0;
#pragma unroll
    for (int x = 1; x < kAhead; ++x)
      if (more && f[x] != 0) {
        a += v[x];
        more = (f[x] & kWeighEnds) == 0;
      }
    for (int j = i + kAhead; more && j < n; ++j) {
      const uint32_t o = p.records[j];
      if (o == 0) continue;
      a += p.parts[static_cast<int64_t>(j) * kWeighBlockKeys + threadIdx.x];
      more = (o & kWeighEnds) == 0;
    }
    if (to != kWeighNowhere) p.weights[to >= 0 ? to : ~to] = old + a;
  }
}

// A unit on its way: its rows g8 and g8 + 8, 8 elements of every 32 per lane, where it
// lies in the cache (−1: nowhere) and what the lane's key had.
template <int D>
struct Tile {
  uint4 k[2][D / 32];
  int row;
  float old;
};

// CTAs per SM, by the registers that the keys and queries take.
template <int D, int NT>
constexpr int kCtas = NT == 1 ? (D == 128 ? 3 : 4) : (D == 128 ? 2 : 3);

// NT: query rows in tiles of 8, at most.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtas<D, NT>) kv_weigh_kernel(const WeighArgs p) {
  __shared__ int64_t s_sum[kWarps];
  __shared__ WeighRun s_run[kThreads];
  __shared__ int64_t s_before[kThreads + 1];  // units before each run of the round
  const bd_attention_batch& b = p.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = b.n_kv_heads;
  const int G = b.n_q_heads / H;
  const int n_run = b.n_seq + b.n_group;
  // The tile kernel ahead, where there is one, lets this one start only when it has
  // seen all before it complete: the units here need nothing of it, and run while
  // its last CTAs do.
  if (p.tile_ctas == 0) griddep_wait();
  griddep_launch_dependents();
  // ---- an even share of all units for each warp; the first runs, a run per thread
  bool bad = false;
  WeighRun mine{};
  int units = 0;
  if (tid < n_run) {
    mine = weigh_run(p, tid, &bad);
    units = units_of(p, mine);
  }
  int64_t all = units;
  for (int r = tid + kThreads; r < n_run; r += kThreads) all += units_of(p, weigh_run(p, r, &bad));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
  if (lane == 0) s_sum[warp] = all;
  bad = __syncthreads_or(bad);
  int64_t total = 0;
  for (int i = 0; i < kWarps; ++i) total += s_sum[i];
  total = bad ? 0 : total * H;
  if (bad && tid == 0 && blockIdx.x == 0) record_error(p.ctx, kErrBounds);
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t each = (total + n_warps - 1) / n_warps;
  int64_t u = each * gw < total ? each * gw : total;
  const int64_t u1 = u + each < total ? u + each : total;
  const int64_t cta_end = each * kWarps * (blockIdx.x + 1) < total
                              ? each * kWarps * (blockIdx.x + 1) : total;

  const int g8 = lane >> 2, quad = lane & 3;
  const int page_shift = 31 - __clz(b.page_size);
  const bool windowed = p.window > 0 && p.window < b.max_q_len;
  int64_t before = 0;
  for (int base = 0; base < n_run && before < cta_end; base += kThreads) {
    if (base > 0) {
      mine = WeighRun{};
      units = 0;
      if (base + tid < n_run) {
        mine = weigh_run(p, base + tid, &bad);
        units = units_of(p, mine);
      }
    }
    int64_t inc = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
      if (lane >= off) inc += o;
    }
    __syncthreads();  // sums and the round before have been read
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += s_sum[i];
    s_run[tid] = mine;
    s_before[tid + 1] = before + inc * H;
    if (tid == 0) s_before[0] = before;
    __syncthreads();
    before = s_before[kThreads];
    // the run that holds the warp's first unit: the last that begins at or before it
    int r = -1;
    if (u < u1 && u < before) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        r += __popc(__ballot_sync(0xFFFFFFFFu, s_before[32 * i + lane] <= u));
    }
    while (u < u1 && u < before) {
      while (s_before[r + 1] <= u) ++r;  // runs without units
      const WeighRun x = s_run[r];
      const bool group = base + r >= b.n_seq;
      const int per_head = (x.k1 - x.k0 + kUnitKeys - 1) / kUnitKeys;
      const int64_t at = u - s_before[r];
      const int h = static_cast<int>(at < (1ll << 31) ? static_cast<uint32_t>(at) / per_head
                                                      : at / per_head);
      const int blk0 = static_cast<int>(at - static_cast<int64_t>(h) * per_head);
      const int blk1 = u1 - u < per_head - blk0 ? blk0 + static_cast<int>(u1 - u) : per_head;
      u += blk1 - blk0;

      // ---- the units blk0 .. blk1 of run x and head h
      const int32_t* table = b.page_table + static_cast<int64_t>(x.seq) * b.table_stride;
      const auto page_of = [&](int blk) {
        return blk < blk1 ? table[(x.k0 + blk * kUnitKeys) >> page_shift] : 0;
      };
      const auto fetch = [&](Tile<D>& t, int blk, int page) {
        const int key = x.k0 + blk * kUnitKeys;
        t.row = -1;
        t.old = 0.f;
        if (blk < blk1) {
          if (page >= 0 && page < b.n_pages)
            t.row = ((page * H + h) << page_shift) + (key & (b.page_size - 1));  // below 2^31
          else
            record_error(p.ctx, kErrBounds);
        }
        const uint16_t* src = p.k_pages + static_cast<int64_t>(t.row + g8) * D + 8 * quad;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            t.k[y][j] = make_uint4(0u, 0u, 0u, 0u);
            if (t.row >= 0 && key + g8 + 8 * y < x.k1)
              t.k[y][j] = ldg_stream_v4(src + y * (8 * D) + 32 * j);
          }
        if (t.row >= 0 && quad < 2 && key + g8 + 8 * quad < x.k1)
          t.old = p.weights[t.row + g8 + 8 * quad];
      };
      int page = page_of(blk0);
      // The query rows, as the products' other operand, and their lse: on their way before
      // the first unit's page is known.
      const int rows = (x.tok1 - x.tok0) * G;  // at most 8·NT
      uint4 q[NT][D / 32];
      float lse[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = 8 * i + g8;
        const uint16_t* src = p.q +
            (static_cast<int64_t>(x.tok0 + row / G) * b.n_q_heads + h * G + row % G) * D + 8 * quad;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          q[i][j] = row < rows ? ldg_v4(src + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int c = 8 * i + 2 * quad + y;
          lse[i][y] = c < rows ? p.lse[static_cast<int64_t>(x.tok0 + c / G) * b.n_q_heads + h * G +
                                       c % G]
                               : INFINITY;
        }
      }
      Tile<D> t;
      fetch(t, blk0, page);
      page = page_of(blk0 + 1);
      float minus[NT][2];
      int sees[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int tok = x.tok0 + (8 * i + 2 * quad + y) / G;
          const bool counts =
              isfinite(lse[i][y]) &&
              (!group || !windowed ||
               weigh_in_window(p, tok, x.seq, b.group_offsets[base + r - b.n_seq + 1]));
          minus[i][y] = counts ? -lse[i][y] * kWeighLog2e : 0.f;
          sees[i][y] = counts ? (group ? INT32_MAX : tok + x.causal) : -1;
        }
      const auto weigh = [&](const Tile<D>& t, int blk) {
        const int key = x.k0 + blk * kUnitKeys + g8;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            mma_16816(c, t.k[0][j].x, t.k[1][j].x, t.k[0][j].y, t.k[1][j].y, q[i][j].x, q[i][j].y);
            mma_16816(d, t.k[0][j].z, t.k[1][j].z, t.k[0][j].w, t.k[1][j].w, q[i][j].z, q[i][j].w);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float w = ex2(fmaf(c[y] + d[y], p.scale_log2, minus[i][y & 1]));
            // (selected, not multiplied: a row that does not count may hold anything)
            sum[y >> 1] += key + 8 * (y >> 1) <= sees[i][y & 1] ? w : 0.f;
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          sum[y] += __shfl_xor_sync(0xFFFFFFFFu, sum[y], 1);
          sum[y] += __shfl_xor_sync(0xFFFFFFFFu, sum[y], 2);
        }
        const int mine_key = key + 8 * quad;  // of the first two lanes of four
        if (t.row >= 0 && quad < 2 && mine_key < x.k1) {
          const int row = t.row + g8 + 8 * quad;
          const float a = quad == 0 ? sum[0] : sum[1];
          if (mine_key >= x.fresh) {
            p.weights[row] = a;
            p.positions[row] = mine_key + (p.pos_offset != nullptr ? p.pos_offset[x.seq] : 0);
          } else {
            p.weights[row] = t.old + a;
          }
        }
      };
#pragma unroll 1
      for (int blk = blk0; blk < blk1; ++blk) {
        weigh(t, blk);
        fetch(t, blk + 1, page);
        page = page_of(blk + 2);
      }
    }
  }
  if (p.tile_ctas > 0) {
    griddep_wait();
    join_parts(p);
  }
}

// CTAs of the short runs' kernel.  Behind the tile kernel, and where the batch may have many
// units, as many as the SMs hold; for few of them fewer, which start sooner and ask less
// often for the same lengths.  (us, 8 key heads of 128, one CTA for two SMs, one an SM, two
// and three: 1 token over 1000 keys 4.2 4.3 5.4 5.7; 8 over 500 7.5 5.8 6.7 6.8; 1 over
// 8000 10.7 8.1 8.4 8.6; 64 over 300 20.2 14.0 13.5 12.1.  Of 64, where four fit: 64 over
// 300 17.9 12.0 9.7, 10.6 by four; 64 over 2000 88 48 32, 27.5 by four.)
template <int D>
unsigned short_ctas(const WeighArgs& p, int sms, int most) {
  if (p.tile_ctas > 0) return static_cast<unsigned>(most * sms);
  const int64_t units = static_cast<int64_t>(p.b.n_seq) * p.b.n_kv_heads *
                        ((p.b.max_kv_len + kUnitKeys - 1) / kUnitKeys);
  if (units <= 4ll * sms) return static_cast<unsigned>((sms + 1) / 2);
  if (units <= (D == 128 ? 32ll : 16ll) * sms) return static_cast<unsigned>(sms);
  if (D == 64 && units <= 80ll * sms) return static_cast<unsigned>(2 * sms);
  return static_cast<unsigned>(most * sms);
}

template <int D>
cudaError_t launch_short(const WeighArgs& p, int sms, cudaStream_t s) {
  const dim3 block(kThreads);
  const int64_t rows = static_cast<int64_t>(p.b.max_q_len) * (p.b.n_q_heads / p.b.n_kv_heads);
  // (a group of few members has up to 16 rows of single tokens)
  return rows <= 8 && p.b.n_group == 0
             ? launch_pdl(kv_weigh_kernel<D, 1>, dim3(short_ctas<D>(p, sms, kCtas<D, 1>)), block, 0, s, p)
             : launch_pdl(kv_weigh_kernel<D, 2>, dim3(short_ctas<D>(p, sms, kCtas<D, 2>)), block, 0, s, p);
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Whether a batch may hold runs of the tile kernel.
bool may_tile(const bd_attention_batch& b) {
  return b.n_group > 0 ||
         static_cast<int64_t>(b.max_q_len) * (b.n_q_heads / b.n_kv_heads) > kWeighShortRows;
}
size_t records_bytes(int ctas) {
  return (sizeof(uint32_t) * 2 * static_cast<size_t>(ctas) + 255) / 256 * 256;
}
size_t parts_bytes(int ctas) {
  return sizeof(float) * 2 * static_cast<size_t>(ctas) * kWeighBlockKeys;
}
size_t workspace_bytes(int ctas) { return records_bytes(ctas) + 2 * parts_bytes(ctas); }

bd_status run_weigh(WeighArgs& p, int sms, cudaStream_t s) {
  const bd_attention_batch& b = p.b;
  if (p.tile_ctas > 0) {
    const uint64_t D = static_cast<uint64_t>(b.head_dim), H = static_cast<uint64_t>(b.n_q_heads);
    const int g = b.n_q_heads / b.n_kv_heads;
    const uint64_t rows =
        static_cast<uint64_t>(b.n_pages) * b.n_kv_heads * static_cast<uint64_t>(b.page_size);
    const uint64_t kdims[3] = {64, rows, D / 64}, kstr[2] = {2 * D, 128};
    const uint32_t kbox[3] = {64, static_cast<uint32_t>(b.page_size), 1};
    const uint64_t qdims[3] = {D, H, static_cast<uint64_t>(b.n_tokens)};
    const uint64_t qstr[2] = {2 * D, 2 * D * H};
    const uint32_t qbox[3] = {64, static_cast<uint32_t>(g),
                              static_cast<uint32_t>(weigh_tile_tokens(g))};
    WeighMaps m;
    if (!encode_tmap_bf16_3d(&m.k, p.k_pages, kdims, kstr, kbox) ||
        !encode_tmap_bf16_3d(&m.q, p.q, qdims, qstr, qbox))
      return BD_ERR_CUDA;
    if (launch_weigh_tile(p, m, s) != cudaSuccess) return BD_ERR_CUDA;
  }
  const cudaError_t e = b.head_dim == 128 ? launch_short<128>(p, sms, s)
                                          : launch_short<64>(p, sms, s);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

}  // namespace
}  // namespace bd

extern "C" {

size_t bitdelta_kv_weigh_workspace_bytes(const bd_attention_batch* batch) {
  if (bd::check_attention_batch(batch) != BD_OK) return 0;
  bd::DevCtx ctx;
  int sms = 0;
  if (bd::current_device_context(&ctx, &sms) != BD_OK) sms = 152;
  return bd::workspace_bytes(sms);
}

bd_status bitdelta_kv_weigh(const bd_attention_batch* batch, const uint16_t* q, const float* lse,
                            const uint16_t* k_pages, float scale, int32_t window,
                            const int32_t* pos_offset, float* weights, int32_t* positions,
                            void* workspace, size_t workspace_bytes, bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  const float scale_log2 = scale * bd::kWeighLog2e;
  // (the tile kernel divides lse by the scale)
  if (!(scale >= 0x1p-100f) || std::isinf(scale_log2) || window < 0) return BD_ERR_INVALID_ARG;
  if (batch->n_tokens == 0 || batch->n_seq == 0) return BD_OK;
  if (!q || !lse || !k_pages || !weights || !positions || batch->n_pages < 1)
    return BD_ERR_INVALID_ARG;
  if (!workspace) return BD_ERR_WORKSPACE;
  if (bd::off(q, 16) || bd::off(lse, 4) || bd::off(k_pages, 16) || bd::off(pos_offset, 4) ||
      bd::off(weights, 4) || bd::off(positions, 4) || bd::off(workspace, 256))
    return BD_ERR_MISALIGNED;
  if (workspace_bytes < 256) return BD_ERR_WORKSPACE;  // no workspace is smaller
  bd::WeighArgs p{};
  int sms = 0;
  if ((st = bd::current_device_context(&p.ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  if (workspace_bytes < bd::workspace_bytes(sms)) return BD_ERR_WORKSPACE;
  p.b = *batch;
  p.q = q;
  p.lse = lse;
  p.k_pages = k_pages;
  p.scale_log2 = scale_log2;
  p.window = window;
  p.pos_offset = pos_offset;
  p.weights = weights;
  p.positions = positions;
  p.tile_ctas = bd::may_tile(*batch) ? sms : 0;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  p.records = reinterpret_cast<uint32_t*>(at);
  p.parts = reinterpret_cast<float*>(at += bd::records_bytes(sms));
  p.rows = reinterpret_cast<int32_t*>(at + bd::parts_bytes(sms));
  return bd::run_weigh(p, sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
