// kv_append.cu — rotary positions on a QKV row and the append of its keys and
// values to the paged cache (bitdelta_kv_append, bitdelta_kv_append_at).
//
// One CTA per token.  Every element moves once (QKV in, q and the cache rows
// out), so the floor is those bytes over the HBM bandwidth; a decode step's
// few tokens are bound by the chain of dependent loads lengths -> page ->
// store instead.  A thread owns one 16-element unit of a head (the
// two 8-element halves that rotate together, or 16 neighbours), keeps its
// angle's cosines and sines in registers and walks over the heads with it.
//
// Measured: 4 prompts of 2048 tokens, 64 query and 8 key heads of 128 (340 MB)
// 51.8 us, 6.57 TB/s; 64 single tokens and four chunks of 512, 32 query heads
// (52 MB) 11.9 us: 2.8 rounds of CTAs, whose QKV loads come behind that chain;
// 8 single tokens 2.7 us (3.6 a call from the host).
#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {
namespace {

struct AppendArgs {
  bd_attention_batch b;
  const uint16_t* qkv;
  const float* rope;
  int64_t rope_rows;
  int32_t rot_dim;
  uint16_t *k_pages, *v_pages, *q_out;
  const int32_t* pos_offset;  // or null
  int32_t ahead;  // tokens
  DevCtx ctx;
};

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  lo = bf16lo_to_f32(w);
  hi = bf16hi_to_f32(w);
}

// (a, b) -> (a·cos − b·sin, b·cos + a·sin)
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = fmaf(x, c, -(y * s));
  b = fmaf(y, c, x * s);
}

template <bool kPairs>
__device__ __forceinline__ void rotate_unit(uint4& lo, uint4& hi, const float (&cs)[8],
                                            const float (&sn)[8]) {
  uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a0, a1, b0, b1;
    unpack2(l[j], a0, a1);
    unpack2(h[j], b0, b1);
    if constexpr (kPairs) {
      rotate(a0, a1, cs[j], sn[j]);
      rotate(b0, b1, cs[4 + j], sn[4 + j]);
    } else {
      rotate(a0, b0, cs[2 * j], sn[2 * j]);
      rotate(a1, b1, cs[2 * j + 1], sn[2 * j + 1]);
    }
    l[j] = pack_bf16x2_rn(a0, a1);
    h[j] = pack_bf16x2_rn(b0, b1);
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
}

// kAhead: each CTA also fetches into L2 the row of a token that one of the next
// CTAs will take.
template <bool kPairs, bool kAhead>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs p) {
  __shared__ int s_seq, s_pos;
  const bd_attention_batch& b = p.b;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int units = b.head_dim >> 4;     // 16-element units per head
  const int u = tid % units;
  const int rot_units = p.rot_dim >> 4;  // the first ones rotate
  const int n_heads = b.n_q_heads + 2 * b.n_kv_heads;
  // the unit's two 8-element pieces within a head
  const int half = p.rot_dim >> 1;
  const int e0 = u < rot_units && !kPairs ? 8 * u : 16 * u;
  const int e1 = u < rot_units && !kPairs ? half + 8 * u : e0 + 8;

  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_seq = -1;
  if constexpr (kAhead) {
    if (tid == 128 && t + p.ahead < b.n_tokens)
      prefetch_l2(p.qkv + (t + p.ahead) * n_heads * b.head_dim, 2 * n_heads * b.head_dim);
  }
  __syncthreads();
  // The token's sequence, by the thread that holds its offset, and the table's
  // bounds: a table that breaks them appends nothing (in the same round of
  // loads, which has the position as well).
  int bad = 0;
  for (int s = tid; s < b.n_seq; s += kAppendThreads) {
    const int lo = b.seq_offsets[s], hi = b.seq_offsets[s + 1], kv = b.kv_len[s];
    bad |= lo < 0 || hi < lo || hi > b.n_tokens || hi - lo > b.max_q_len || kv < 0 ||
           kv > b.max_kv_len;
    if (lo <= t && t < hi) {
      s_seq = s;
      s_pos = kv - (hi - static_cast<int>(t));
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) record_error(p.ctx, kErrBounds);
  const int seq = s_seq;
  const int64_t pos = seq >= 0 && !bad ? s_pos : -1;
  bool ok = pos >= 0;
  // the position that the angle goes by
  const int64_t at = pos + (ok && p.pos_offset != nullptr ? p.pos_offset[seq] : 0);
  int64_t row0 = 0;  // the token's first cache row (head 0) in rows of head_dim
  if (ok) {
    const int64_t pg = pos / b.page_size;
    int64_t page = -1;
    if (pg < b.table_stride && (p.rot_dim == 0 || (at >= 0 && at < p.rope_rows)))
      page = b.page_table[static_cast<int64_t>(seq) * b.table_stride + pg];
    if (page < 0 || page >= b.n_pages) {
      if (tid == 0) record_error(p.ctx, kErrBounds);
      ok = false;
    } else {
      row0 = page * b.n_kv_heads * b.page_size + pos % b.page_size;
    }
  }
  float cs[8], sn[8];
  if (ok && u < rot_units) {
    const float* r = p.rope + at * p.rot_dim + 8 * u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 c = reinterpret_cast<const float4*>(r)[j];
      const float4 s = reinterpret_cast<const float4*>(r + half)[j];
      cs[4 * j] = c.x, cs[4 * j + 1] = c.y, cs[4 * j + 2] = c.z, cs[4 * j + 3] = c.w;
      sn[4 * j] = s.x, sn[4 * j + 1] = s.y, sn[4 * j + 2] = s.z, sn[4 * j + 3] = s.w;
    }
  }
  const uint16_t* src = p.qkv + t * n_heads * b.head_dim;
  uint16_t* q = p.q_out + t * b.n_q_heads * b.head_dim;
  const int stride = kAppendThreads / units;
  for (int h = tid / units; h < n_heads; h += stride) {
    uint4 lo = ldg_stream_v4(src + h * b.head_dim + e0);
    uint4 hi = ldg_stream_v4(src + h * b.head_dim + e1);
    uint16_t* dst;
    if (h < b.n_q_heads) {
      dst = q + h * b.head_dim;
      if (!ok) lo = hi = make_uint4(0u, 0u, 0u, 0u);
    } else {
      if (!ok) continue;
      const int kh = h - b.n_q_heads;
      const int head = kh < b.n_kv_heads ? kh : kh - b.n_kv_heads;
      dst = (kh < b.n_kv_heads ? p.k_pages : p.v_pages) +
            (row0 + static_cast<int64_t>(head) * b.page_size) * b.head_dim;
    }
    if (ok && u < rot_units && h < b.n_q_heads + b.n_kv_heads)
      rotate_unit<kPairs>(lo, hi, cs, sn);
    *reinterpret_cast<uint4*>(dst + e0) = lo;
    *reinterpret_cast<uint4*>(dst + e1) = hi;
  }
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace

int check_attention_batch(const bd_attention_batch* b) {
  if (!b) return BD_ERR_INVALID_ARG;
  if (b->n_tokens < 0 || b->n_seq < 0 || b->max_q_len < 0 || b->max_kv_len < 0 ||
      b->n_group < 0 || b->n_pages < 0 || b->table_stride < 0 || b->n_q_heads < 1 ||
      b->n_kv_heads < 1)
    return BD_ERR_INVALID_ARG;
  if (b->n_q_heads % b->n_kv_heads != 0 || b->n_q_heads / b->n_kv_heads > 32 ||
      b->n_q_heads > 1024 || (b->head_dim != 64 && b->head_dim != 128) ||
      (b->page_size != 16 && b->page_size != 32 && b->page_size != 64 && b->page_size != 128) ||
      b->n_tokens > (1 << 26) || b->n_tokens * b->n_kv_heads > (1 << 28) ||
      b->n_seq > (1 << 20) || b->n_group > b->n_seq ||
      b->n_pages > 0x7FFFFFFF / b->n_kv_heads / b->page_size || b->table_stride > 0x7FFFFFFF ||
      b->max_kv_len > (1 << 30))
    return BD_ERR_UNSUPPORTED_SHAPE;
  if (b->n_tokens > 0 && b->n_seq > 0) {
    if (!b->seq_offsets || !b->kv_len || !b->page_table) return BD_ERR_INVALID_ARG;
    if (b->n_group > 0 && (!b->group_offsets || !b->prefix_len)) return BD_ERR_INVALID_ARG;
    if (off(b->seq_offsets, 4) || off(b->kv_len, 4) || off(b->page_table, 4) ||
        off(b->group_offsets, 4) || off(b->prefix_len, 4))
      return BD_ERR_MISALIGNED;
  }
  return BD_OK;
}

}  // namespace bd

extern "C" bd_status bitdelta_kv_append(const bd_attention_batch* batch, const uint16_t* qkv,
                                        const float* rope, int64_t rope_rows, int32_t rot_dim,
                                        bd_rope_style style, uint16_t* k_pages,
                                        uint16_t* v_pages, uint16_t* q_out, bd_stream_t stream) {
  return bitdelta_kv_append_at(batch, nullptr, qkv, rope, rope_rows, rot_dim, style, k_pages,
                               v_pages, q_out, stream);
}

extern "C" bd_status bitdelta_kv_append_at(const bd_attention_batch* batch,
                                           const int32_t* pos_offset, const uint16_t* qkv,
                                           const float* rope, int64_t rope_rows, int32_t rot_dim,
                                           bd_rope_style style, uint16_t* k_pages,
                                           uint16_t* v_pages, uint16_t* q_out,
                                           bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (style != BD_ROPE_HALVES && style != BD_ROPE_PAIRS) return BD_ERR_INVALID_ARG;
  if (rope_rows < 0 || rot_dim < 0) return BD_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > batch->head_dim) return BD_ERR_UNSUPPORTED_SHAPE;
  if (batch->n_tokens == 0) return BD_OK;
  if (!qkv || !q_out || !k_pages || !v_pages || (rot_dim > 0 && !rope)) return BD_ERR_INVALID_ARG;
  if (bd::off(qkv, 16) || bd::off(q_out, 16) || bd::off(k_pages, 16) || bd::off(v_pages, 16) ||
      bd::off(rope, 16) || bd::off(pos_offset, 4))
    return BD_ERR_MISALIGNED;
  bd::AppendArgs p{};
  int sms = 0;
  if ((st = bd::current_device_context(&p.ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  p.b = *batch;
  p.pos_offset = pos_offset;
  p.qkv = qkv;
  p.rope = rope;
  p.rope_rows = rope_rows;
  p.rot_dim = rot_dim;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.q_out = q_out;
  // Five CTAs of 48 registers a thread per SM.  From two rounds of them on, the
  // fetch ahead keeps reads in flight while CTAs search, wait and store (in a
  // graph, 4 x 2048 tokens of 80 heads 57.6 -> 51.5 us, 2 x 1024 of 48 heads 10.4
  // -> 9.9); below it gives little (512 tokens 5.90 -> 5.84 us) or costs its
  // instructions (8 tokens 2.65 -> 2.74).  Distances of one, three and five CTAs
  // per SM: 51.6, 51.5 and 52.3 us.
  p.ahead = sms * 2;
  const bool ahead = batch->n_tokens >= 2 * 5 * static_cast<int64_t>(sms);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(batch->n_tokens)), block(bd::kAppendThreads);
  const auto launch = [&](auto kernel) {
    return bd::launch_pdl(kernel, grid, block, 0, s, p);
  };
  const cudaError_t e =
      style == BD_ROPE_PAIRS
          ? launch(ahead ? bd::kv_append_kernel<true, true> : bd::kv_append_kernel<true, false>)
          : launch(ahead ? bd::kv_append_kernel<false, true> : bd::kv_append_kernel<false, false>);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}
