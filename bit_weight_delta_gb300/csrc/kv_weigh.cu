// kv_weigh.cu — the attention weight that each cached key got from a step's
// queries, added to a table beside the cache (bitdelta_kv_weigh).
//
//   a[p] = Σ over rows (query token, query head) of exp(scale·q·k_p − lse)
//
// The attention has left each row's lse, so a weight needs no second pass: the
// keys are read once and the values not at all.
//
// A run is a set of rows with the keys that they look at: a sequence's window of
// query tokens over its own keys, or all of a group's over their shared prefix.
// A unit is 32 keys of a run and key head, worked on by one warp: the keys are the
// rows of mma.sync tiles (16 keys by 8 query rows by 16 elements) and stay in
// registers while the query rows pass, 8 at a time, so that a key's sum stays
// in its lanes.  Both operands are loaded straight from memory, 16 bytes a lane:
// which of a row's elements a lane holds is the same for both, and a product's
// sum does not care about their order.
#include <cmath>
#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);

namespace {

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
  DevCtx ctx;
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitKeys = 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Run {
  int seq;       // whose page-table row is read
  int k0, k1;    // slots
  int tok0, tok1;  // query tokens whose rows look at them
  int causal;    // token t sees slots up to t + causal
  int fresh;     // first slot of the step's own tokens
  int units;     // per key head
};

// The prefix of sequence s (0 outside of every group); the groups are sorted.
__device__ __forceinline__ int prefix_of(const bd_attention_batch& b, int s) {
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
__device__ Run run_of(const WeighArgs& p, int r) {
  const bd_attention_batch& b = p.b;
  Run x{};
  if (r < b.n_seq) {
    const int lo = b.seq_offsets[r], hi = b.seq_offsets[r + 1], kv = b.kv_len[r];
    x.seq = r;
    x.k0 = b.n_group > 0 ? prefix_of(b, r) : 0;
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
    x.causal = 1 << 30;
    x.fresh = INT32_MAX;
  }
  x.units = x.tok1 > x.tok0 && x.k1 > x.k0 ? (x.k1 - x.k0 + kUnitKeys - 1) / kUnitKeys : 0;
  return x;
}

// Whether the batch's tables break their bounds (this thread's share of them).
__device__ bool breaks_bounds(const WeighArgs& p) {
  const bd_attention_batch& b = p.b;
  bool bad = false;
  for (int g = threadIdx.x; g < b.n_group; g += kThreads) {
    const int a = b.group_offsets[g], e = b.group_offsets[g + 1], len = b.prefix_len[g];
    bad |= a < 0 || e < a || e > b.n_seq || len < 0 || len % b.page_size != 0;
  }
  for (int s = threadIdx.x; s < b.n_seq; s += kThreads) {
    const int lo = b.seq_offsets[s], hi = b.seq_offsets[s + 1], kv = b.kv_len[s];
    bad |= lo < 0 || hi < lo || hi > b.n_tokens || hi - lo > b.max_q_len || kv < 0 ||
           kv > b.max_kv_len || kv > b.table_stride * b.page_size ||
           (b.n_group > 0 && static_cast<int64_t>(kv) - (hi - lo) < prefix_of(b, s) &&
            prefix_of(b, s) > 0);
  }
  return bad;
}

// Whether token t counts in the window of its sequence, one of [s0, s1).
__device__ bool in_window(const WeighArgs& p, int t, int s0, int s1) {
  while (s1 - s0 > 1) {
    const int mid = (s0 + s1) >> 1;
    if (p.b.seq_offsets[mid] <= t)
      s0 = mid;
    else
      s1 = mid;
  }
  return p.b.seq_offsets[s0 + 1] - t <= p.window;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_weigh_kernel(const WeighArgs p) {
  __shared__ int64_t s_sum[kWarps];
  const bd_attention_batch& b = p.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = b.n_kv_heads;
  const uint32_t G = b.n_q_heads / H;
  const int n_run = b.n_seq + b.n_group;
  griddep_wait();
  griddep_launch_dependents();
  if (__syncthreads_or(breaks_bounds(p))) {
    if (tid == 0 && blockIdx.x == 0) record_error(p.ctx, kErrBounds);
    return;
  }
  // ---- an even share of all units for each warp
  int64_t mine = 0;
  for (int r = tid; r < n_run; r += kThreads) mine += run_of(p, r).units;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, off);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int i = 0; i < kWarps; ++i) total += s_sum[i];
  total *= H;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t u0 = total * gw / n_warps, u1 = total * (gw + 1) / n_warps;

  const int g8 = lane >> 2, quad = lane & 3;
  const int page_shift = 31 - __clz(b.page_size);
  const bool windowed = p.window > 0 && p.window < b.max_q_len;
  // 32 runs at a time: a lane holds one of them and the units before it
  int64_t before = 0;
  int64_t u = u0;
  for (int r0 = 0; r0 < n_run && u < u1; r0 += 32) {
    Run own{};
    if (r0 + lane < n_run) own = run_of(p, r0 + lane);
    int64_t inc = static_cast<int64_t>(own.units) * H;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
      if (lane >= off) inc += o;
    }
    const int64_t end = before + __shfl_sync(0xFFFFFFFFu, inc, 31);
    for (; u < u1 && u < end; ++u) {
      const int src = __ffs(__ballot_sync(0xFFFFFFFFu, before + inc > u)) - 1;
      Run x;
      x.seq = __shfl_sync(0xFFFFFFFFu, own.seq, src);
      x.k0 = __shfl_sync(0xFFFFFFFFu, own.k0, src);
      x.k1 = __shfl_sync(0xFFFFFFFFu, own.k1, src);
      x.tok0 = __shfl_sync(0xFFFFFFFFu, own.tok0, src);
      x.tok1 = __shfl_sync(0xFFFFFFFFu, own.tok1, src);
      x.causal = __shfl_sync(0xFFFFFFFFu, own.causal, src);
      x.fresh = __shfl_sync(0xFFFFFFFFu, own.fresh, src);
      x.units = __shfl_sync(0xFFFFFFFFu, own.units, src);
      const bool group = r0 + src >= b.n_seq;
      const int64_t first = __shfl_sync(0xFFFFFFFFu, before + inc - static_cast<int64_t>(own.units) * H, src);
      const int at = static_cast<int>(u - first);
      const int h = at / x.units;
      const int key0 = x.k0 + (at - h * x.units) * kUnitKeys;

      // ---- the unit's keys: tiles of 16, each within a page
      const int32_t* table = b.page_table + static_cast<int64_t>(x.seq) * b.table_stride;
      uint4 k[2][2][D / 32];
      int64_t tile_row[2];  // of the tile's first key in the cache, or −1
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = key0 + 16 * i;
        tile_row[i] = -1;
        if (key < x.k1) {
          const int page = table[key >> page_shift];
          if (page >= 0 && page < b.n_pages)
            tile_row[i] = ((static_cast<int64_t>(page) * H + h) << page_shift) +
                          (key & (b.page_size - 1));
          else
            record_error(p.ctx, kErrBounds);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            k[i][y][j] = make_uint4(0u, 0u, 0u, 0u);
            if (tile_row[i] >= 0 && key + g8 + 8 * y < x.k1)
              k[i][y][j] = ldg_stream_v4(p.k_pages + (tile_row[i] + g8 + 8 * y) * D + 32 * j + 8 * quad);
          }
      }
      // ---- the query rows, 8 at a time
      float sum[2][2] = {};
      const uint32_t rows = static_cast<uint32_t>(x.tok1 - x.tok0) * G;
      // rows before the first that sees a key of the unit are left out
      const int t_lo = group ? x.tok0 : max(x.tok0, key0 - x.causal);
      for (uint32_t r = static_cast<uint32_t>(t_lo - x.tok0) * G & ~7u; r < rows; r += 8) {
        uint4 q[D / 32];
        {
          const uint32_t row = r + g8;
          const int t = x.tok0 + row / G;
          const uint16_t* src_q =
              p.q + (static_cast<int64_t>(t) * b.n_q_heads + h * G + row % G) * D + 8 * quad;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            q[j] = row < rows ? ldg_v4(src_q + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
        float lse[2];
        int sees[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t row = r + 2 * quad + y;
          lse[y] = INFINITY;
          sees[y] = -1;
          if (row < rows) {
            const int t = x.tok0 + row / G;
            const float l = p.lse[static_cast<int64_t>(t) * b.n_q_heads + h * G + row % G];
            const bool counts =
                !group || !windowed ||
                in_window(p, t, x.seq, b.group_offsets[r0 + src - b.n_seq + 1]);
            if (isfinite(l) && counts) {
              lse[y] = l * kLog2e;
              sees[y] = group ? INT32_MAX : t + x.causal;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            mma_16816(c, k[i][0][j].x, k[i][1][j].x, k[i][0][j].y, k[i][1][j].y, q[j].x, q[j].y);
            mma_16816(c, k[i][0][j].z, k[i][1][j].z, k[i][0][j].w, k[i][1][j].w, q[j].z, q[j].w);
          }
          const int key = key0 + 16 * i + g8;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float w = ex2(fmaf(c[y], p.scale_log2, -lse[y & 1]));
            if (key + 8 * (y >> 1) <= sees[y & 1]) sum[i][y >> 1] += w;
          }
        }
      }
      // ---- a key's four lanes together; each then writes one key
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          sum[i][y] += __shfl_xor_sync(0xFFFFFFFFu, sum[i][y], 1);
          sum[i][y] += __shfl_xor_sync(0xFFFFFFFFu, sum[i][y], 2);
        }
      const int i = quad >> 1, y = quad & 1;
      const float a = i == 0 ? (y == 0 ? sum[0][0] : sum[0][1]) : (y == 0 ? sum[1][0] : sum[1][1]);
      const int key = key0 + 16 * i + 8 * y + g8;
      const int64_t tile = i == 0 ? tile_row[0] : tile_row[1];
      if (key < x.k1 && tile >= 0) {
        const int64_t row = tile + 8 * y + g8;
        if (key >= x.fresh) {
          p.weights[row] = a;
          p.positions[row] = key + (p.pos_offset != nullptr ? p.pos_offset[x.seq] : 0);
        } else {
          p.weights[row] += a;
        }
      }
    }
    before = end;
  }
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace
}  // namespace bd

extern "C" bd_status bitdelta_kv_weigh(const bd_attention_batch* batch, const uint16_t* q,
                                       const float* lse, const uint16_t* k_pages, float scale,
                                       int32_t window, const int32_t* pos_offset, float* weights,
                                       int32_t* positions, bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  const float scale_log2 = scale * bd::kLog2e;
  if (!(scale > 0.f) || std::isinf(scale_log2) || window < 0) return BD_ERR_INVALID_ARG;
  if (batch->n_tokens == 0 || batch->n_seq == 0) return BD_OK;
  if (!q || !lse || !k_pages || !weights || !positions) return BD_ERR_INVALID_ARG;
  if (bd::off(q, 16) || bd::off(lse, 4) || bd::off(k_pages, 16) || bd::off(pos_offset, 4) ||
      bd::off(weights, 4) || bd::off(positions, 4))
    return BD_ERR_MISALIGNED;
  bd::WeighArgs p{};
  int sms = 0;
  if ((st = bd::current_device_context(&p.ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  p.b = *batch;
  p.q = q;
  p.lse = lse;
  p.k_pages = k_pages;
  p.scale_log2 = scale_log2;
  p.window = window;
  p.pos_offset = pos_offset;
  p.weights = weights;
  p.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(2 * sms), block(bd::kThreads);
  const cudaError_t e = batch->head_dim == 128
                            ? bd::launch_pdl(bd::kv_weigh_kernel<128>, grid, block, 0, s, p)
                            : bd::launch_pdl(bd::kv_weigh_kernel<64>, grid, block, 0, s, p);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}
