// attention.cu — causal attention of ragged query runs over the paged cache
// (bitdelta_attention) and its plan (bitdelta_attention_plan).
//
//   out[t, h] = Σ_{p ≤ pos(t)} softmax_p(scale · q[t, h]·k_p) · v_p
//
// One warp per token and query head: its lanes hold the head's elements, a
// score is one warp reduction, and the running maximum m, denominator l and
// sum o of the softmax are rescaled by 2^(m_old − m_new) as m grows, so every
// key is visited once.
#include <climits>
#include <cmath>
#include <cstdint>

#include "bitdelta_block.h"
#include "kernels.h"

namespace bd {
int check_attention_batch(const bd_attention_batch* b);
namespace {

struct AttnArgs {
  bd_attention_batch b;
  const int32_t* tok_seq;
  const uint16_t *q, *k_pages, *v_pages;
  float scale_log2;
  uint16_t* out;
  float* lse;
  DevCtx ctx;
};

size_t plan_bytes_of(const bd_attention_batch& b) {
  return (static_cast<size_t>(b.n_tokens) * 4 + 255) & ~static_cast<size_t>(255);
}

// tok_seq[t]: the sequence of token t, −1 for a token of none.
__global__ void plan_kernel(bd_attention_batch b, int32_t* tok_seq, DevCtx ctx) {
  griddep_wait();
  int bad = 0;
  for (int s = threadIdx.x; s < b.n_seq; s += blockDim.x) {
    const int a = b.seq_offsets[s], e = b.seq_offsets[s + 1], kv = b.kv_len[s];
    bad |= a < 0 || e < a || e > b.n_tokens || e - a > b.max_q_len || kv < 0 ||
           kv > b.max_kv_len || kv > b.table_stride * b.page_size;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) record_error(ctx, kErrBounds);
  for (int64_t t = threadIdx.x; t < b.n_tokens; t += blockDim.x) tok_seq[t] = -1;
  __syncthreads();
  if (bad) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < b.n_seq; s += blockDim.x >> 5)
    for (int t = b.seq_offsets[s] + lane; t < b.seq_offsets[s + 1]; t += 32) tok_seq[t] = s;
}

template <int D>
__global__ void __launch_bounds__(128) attention_rows_kernel(const AttnArgs p) {
  constexpr int E = D / 32;
  const bd_attention_batch& b = p.b;
  griddep_wait();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= b.n_tokens * b.n_q_heads) return;
  const int64_t t = r / b.n_q_heads;
  const int h = static_cast<int>(r % b.n_q_heads);
  const int kvh = h / (b.n_q_heads / b.n_kv_heads);
  const int seq = p.tok_seq[t];
  int64_t keys = 0;
  if (seq >= 0) keys = static_cast<int64_t>(b.kv_len[seq]) - (b.seq_offsets[seq + 1] - t) + 1;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float(static_cast<uint32_t>(p.q[r * D + e * 32 + lane]) << 16);
    o[e] = 0.f;
  }
  for (int64_t k = 0; k < keys; ++k) {
    int64_t page = b.page_table[static_cast<int64_t>(seq) * b.table_stride + k / b.page_size];
    if (page < 0 || page >= b.n_pages) {
      if (lane == 0) record_error(p.ctx, kErrBounds);
      break;
    }
    const int64_t row = (page * b.n_kv_heads + kvh) * b.page_size + k % b.page_size;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s = fmaf(q[e],
               __uint_as_float(static_cast<uint32_t>(p.k_pages[row * D + e * 32 + lane]) << 16),
               s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float f = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(o[e], f,
                  w * __uint_as_float(static_cast<uint32_t>(p.v_pages[row * D + e * 32 + lane])
                                      << 16));
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[r * D + e * 32 + lane] =
        static_cast<uint16_t>(pack_bf16x2_rn(o[e] * inv, 0.f) & 0xFFFFu);
  if (p.lse != nullptr && lane == 0)
    p.lse[r] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace
}  // namespace bd

extern "C" {

size_t bitdelta_attention_plan_bytes(const bd_attention_batch* batch) {
  if (bd::check_attention_batch(batch) != BD_OK) return 0;
  return bd::plan_bytes_of(*batch);
}

bd_status bitdelta_attention_plan(const bd_attention_batch* batch, void* plan, size_t plan_bytes,
                                  bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (batch->n_tokens == 0 || batch->n_seq == 0) return BD_OK;
  if (!plan || plan_bytes < bd::plan_bytes_of(*batch)) return BD_ERR_WORKSPACE;
  if (bd::off(plan, 256)) return BD_ERR_MISALIGNED;
  bd::DevCtx ctx;
  int sms = 0;
  if ((st = bd::current_device_context(&ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  const cudaError_t e =
      bd::launch_pdl(bd::plan_kernel, dim3(1), dim3(1024), 0,
                     reinterpret_cast<cudaStream_t>(stream), *batch,
                     static_cast<int32_t*>(plan), ctx);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

size_t bitdelta_attention_workspace_bytes(const bd_attention_batch* batch) {
  (void)batch;
  return 0;
}

bd_status bitdelta_attention(const bd_attention_batch* batch, const void* plan, size_t plan_bytes,
                             const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                             float scale, uint16_t* out, float* lse, void* workspace,
                             size_t workspace_bytes, bd_stream_t stream) {
  int st = bd::check_attention_batch(batch);
  if (st != BD_OK) return static_cast<bd_status>(st);
  if (!(scale > 0.f) || std::isinf(scale)) return BD_ERR_INVALID_ARG;
  if (batch->n_tokens == 0 || batch->n_seq == 0) return BD_OK;
  if (!q || !k_pages || !v_pages || !out) return BD_ERR_INVALID_ARG;
  if (!plan || plan_bytes < bd::plan_bytes_of(*batch)) return BD_ERR_WORKSPACE;
  const size_t need = bitdelta_attention_workspace_bytes(batch);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BD_ERR_WORKSPACE;
  if (bd::off(q, 16) || bd::off(k_pages, 16) || bd::off(v_pages, 16) || bd::off(out, 16) ||
      bd::off(lse, 4) || bd::off(plan, 256) || bd::off(workspace, 256))
    return BD_ERR_MISALIGNED;
  bd::AttnArgs p{};
  int sms = 0;
  if ((st = bd::current_device_context(&p.ctx, &sms)) != BD_OK) return static_cast<bd_status>(st);
  p.b = *batch;
  p.tok_seq = static_cast<const int32_t*>(plan);
  p.q = q;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  const int64_t rows = batch->n_tokens * batch->n_q_heads;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      batch->head_dim == 128
          ? bd::launch_pdl(bd::attention_rows_kernel<128>, grid, dim3(128), 0, s, p)
          : bd::launch_pdl(bd::attention_rows_kernel<64>, grid, dim3(128), 0, s, p);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}

}  // extern "C"
