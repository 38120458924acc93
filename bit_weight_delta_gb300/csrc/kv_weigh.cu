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
// A unit is 32 keys of a run and key head, worked on by one warp: the keys are the
// rows of mma.sync tiles (16 keys by 8 query rows by 16 elements) and stay in
// registers while the query rows pass, 8 at a time, so that a key's sum stays
// in its lanes.  Both operands are loaded straight from memory, 16 bytes a lane:
// which of a row's elements a lane holds is the same for both, and a product's
// sum does not care about their order.
#include <cmath>
#include <cstdint>

#include "attention.cuh"
#include "kv_weigh.cuh"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitKeys = 32;
static_assert(kThreads == kWeighBlockKeys, "the join takes a key per thread");

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A run with its units per key head: none where the tile kernel has it.
struct Run : WeighRun {
  int units;
};
__device__ __forceinline__ Run run_of(const WeighArgs& p, int r, bool* bad) {
  Run x{};
  static_cast<WeighRun&>(x) = weigh_run(p, r, bad);
  const int64_t rows =
      static_cast<int64_t>(x.tok1 - x.tok0) * (p.b.n_q_heads / p.b.n_kv_heads);
  x.units = rows <= kWeighShortRows && x.k1 > x.k0 ? (x.k1 - x.k0 + kUnitKeys - 1) / kUnitKeys : 0;
  return x;
}

// The blocks that several CTAs of the tile kernel share: their parts in their
// order.
__device__ void join_parts(const WeighArgs& p) {
  const int n = 2 * p.tile_ctas;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const WeighRecord r = p.records[i];
    if (!r.used || !r.begins) continue;
    float a = p.parts[static_cast<int64_t>(i) * kWeighBlockKeys + threadIdx.x];
    bool more = !r.ends;
    for (int j = i + 1; more && j < n; ++j) {
      const WeighRecord o = p.records[j];
      if (!o.used) continue;
      a += p.parts[static_cast<int64_t>(j) * kWeighBlockKeys + threadIdx.x];
      more = !o.ends;
    }
    bool bad = false;  // (the kernel that left the parts has looked)
    const WeighRun x = weigh_run(p, r.run, &bad);
    const int key = x.k0 + r.block * kWeighBlockKeys + static_cast<int>(threadIdx.x);
    if (key < x.k1) {
      const int64_t row = weigh_row(p.b, x.seq, key, r.head);
      if (row >= 0) weigh_add(p, x.seq, x.fresh, key, row, a);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_weigh_kernel(const WeighArgs p) {
  __shared__ int64_t s_sum[kWarps];
  const bd_attention_batch& b = p.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = b.n_kv_heads;
  const uint32_t G = b.n_q_heads / H;
  const int n_run = b.n_seq + b.n_group;
  // The tile kernel ahead, where there is one, lets this one start only when it has
  // seen all before it complete: the units here need nothing of it, and run while
  // its last CTAs do.
  if (p.tile_ctas == 0) griddep_wait();
  griddep_launch_dependents();
  // ---- an even share of all units for each warp
  bool bad = false;
  int64_t mine = 0;
  for (int r = tid; r < n_run; r += kThreads) mine += run_of(p, r, &bad).units;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, off);
  if (lane == 0) s_sum[warp] = mine;
  bad = __syncthreads_or(bad);
  int64_t total = 0;
  for (int i = 0; i < kWarps; ++i) total += s_sum[i];
  total = bad ? 0 : total * H;
  if (bad && tid == 0 && blockIdx.x == 0) record_error(p.ctx, kErrBounds);
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
    if (r0 + lane < n_run) own = run_of(p, r0 + lane, &bad);
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
                weigh_in_window(p, t, x.seq, b.group_offsets[r0 + src - b.n_seq + 1]);
            if (isfinite(l) && counts) {
              lse[y] = l * kWeighLog2e;
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
        weigh_add(p, x.seq, x.fresh, key, tile + 8 * y + g8, a);
      }
    }
    before = end;
  }
  if (p.tile_ctas > 0) {
    griddep_wait();
    join_parts(p);
  }
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Whether a batch may hold runs of the tile kernel.
bool may_tile(const bd_attention_batch& b) {
  return b.n_group > 0 ||
         static_cast<int64_t>(b.max_q_len) * (b.n_q_heads / b.n_kv_heads) > kWeighShortRows;
}
size_t records_bytes(int ctas) {
  return (sizeof(WeighRecord) * 2 * static_cast<size_t>(ctas) + 255) / 256 * 256;
}
size_t workspace_bytes(int ctas) {
  return records_bytes(ctas) + sizeof(float) * 2 * static_cast<size_t>(ctas) * kWeighBlockKeys;
}

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
  const dim3 grid(2 * sms), block(kThreads);
  const cudaError_t e = b.head_dim == 128
                            ? launch_pdl(kv_weigh_kernel<128>, grid, block, 0, s, p)
                            : launch_pdl(kv_weigh_kernel<64>, grid, block, 0, s, p);
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
  if (!(scale > 0.f) || std::isinf(scale_log2) || window < 0) return BD_ERR_INVALID_ARG;
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
  p.records = static_cast<bd::WeighRecord*>(workspace);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + bd::records_bytes(sms));
  return bd::run_weigh(p, sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
