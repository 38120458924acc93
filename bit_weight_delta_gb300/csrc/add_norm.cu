// add_norm.cu — residual addition with the RMS norms after and before a
// decoder sub-block (bitdelta_add_norm).
//
//   b = y or RMSNorm(y; w_post),  h = residual + scale·gate·b,
//   x = RMSNorm(h; w_pre)
//
// One CTA per row, the row in registers as fp32 from the first load to the
// last store, so every input is read once and every output written once:
// the floor is those bytes over the HBM bandwidth.  (Above 16384 elements a
// little of the row, above 32768 about half of it, goes through local memory: a
// thread has 64 registers.)  The two sums of squares are each one warp-shuffle
// reduction and one exchange through shared memory.
//
// Measured: 2112 rows x 4096 with both norms, a gate and an fp32 residual (104
// MB, 15.6 us at the copy rate) 17.7 us on repeated inputs and 22.2 us on
// inputs that change (4.7 TB/s): behind its loads a row waits for its segment, the
// segment's variant, that one's two table entries and, after the first sum, the
// weights, with no other loads in flight, and 2112 rows are 3.5 rounds of CTAs.
// 2048 bf16 rows of 8192 22.1 us (6.1 TB/s); 512 of 16384, 32768 and 65536 14.4,
// 26.7 and 98.7 us (4.7, 5.0 and 2.7 TB/s; the last stores and loads another
// 0.8 MB of local memory a row, more than the row's own 0.5).
// 8 rows x 8192: 2.9 us on the GPU, bound by a row's chain.  Rows streamed
// through a ring in shared memory by one persistent CTA per SM were slower at
// every size.
#include <cstdint>

#include "bitdelta_block.h"
#include "kernels.h"

namespace bd {
namespace {

struct NormArgs {
  const uint16_t* y;
  const void* residual;
  void* residual_out;
  const uint16_t* gate;
  int64_t gate_stride;
  float scale, eps;
  const uint16_t* const* pre_table;
  const uint16_t* const* post_table;
  int32_t n_tab;
  const int32_t* seg_offsets;
  const int32_t* seg_variant;
  int32_t n_seg;
  uint16_t* x_out;
  int64_t M;
  int32_t d;
  int32_t ahead;  // rows
  DevCtx ctx;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16lo_to_f32(v.x);
  f[1] = bf16hi_to_f32(v.x);
  f[2] = bf16lo_to_f32(v.y);
  f[3] = bf16hi_to_f32(v.y);
  f[4] = bf16lo_to_f32(v.z);
  f[5] = bf16hi_to_f32(v.z);
  f[6] = bf16lo_to_f32(v.w);
  f[7] = bf16hi_to_f32(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                    pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
}

// Sum over the CTA; `s_part` holds one value per warp and is private to this
// call.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = static_cast<int>(threadIdx.x & 31) < warps ? s_part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// The weights of a row's variant: table[slot], or null (ones) for an entry
// that cannot be read.
__device__ __forceinline__ const uint16_t* weights_of(const uint16_t* const* table, int slot,
                                                      const DevCtx& ctx) {
  const uint16_t* w = table[slot];
  if (w == nullptr || (reinterpret_cast<uintptr_t>(w) & 15) != 0) {
    if (threadIdx.x == 0) record_error(ctx, kErrBounds);
    return nullptr;
  }
  return w;
}

// C chunks of 8 elements per thread.
// (32 registers where they do, so that rows of 8192 stay two to an SM; the
// weights are fetched late for that.)
// kAhead: each CTA also fetches into L2 a row that one of the next CTAs will take.
template <int C, bool kF32, bool kAhead>
__global__ void __launch_bounds__(1024, C == 1 ? 2 : 1) add_norm_kernel(const NormArgs p) {
  __shared__ float s_post[32], s_pre[32];
  __shared__ int s_seg, s_bad;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int n8 = p.d >> 3;
  griddep_wait();
  griddep_launch_dependents();

  if constexpr (kAhead) {
    if (tid == 0 && row + p.ahead < p.M) {
      const int64_t next = (row + p.ahead) * p.d;
      prefetch_l2(p.y + next, 2 * p.d);
      if (p.residual != nullptr)
        prefetch_l2(static_cast<const uint16_t*>(p.residual) + next, 2 * p.d);
    }
  }

  uint4 yv[C], gv[C], ra[C], rb[C];
  const uint4* y8 = reinterpret_cast<const uint4*>(p.y + row * p.d);
  const uint4* g8 = reinterpret_cast<const uint4*>(p.gate + row * p.gate_stride);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + tid;
    yv[c] = gv[c] = ra[c] = rb[c] = make_uint4(0u, 0u, 0u, 0u);
    if (i < n8) {
      yv[c] = ldg_stream_v4(y8 + i);
      if (p.residual != nullptr) {
        if constexpr (kF32) {
          const uint4* r4 = reinterpret_cast<const uint4*>(
              static_cast<const float*>(p.residual) + row * p.d);
          // plain loads: residual_out may be the same buffer
          ra[c] = r4[2 * i];
          rb[c] = r4[2 * i + 1];
        } else {
          ra[c] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) +
                                                 row * p.d)[i];
        }
      }
      if (p.gate != nullptr) gv[c] = ldg_v4(g8 + i);
    }
  }

  // The row's segment, by the thread that holds its offset: one round of
  // loads instead of a search of dependent ones.
  int slot = 0;
  if (p.seg_offsets != nullptr) {
    if (tid == 0) {
      s_seg = -1;
      s_bad = 0;
    }
    __syncthreads();
    const int at = static_cast<int>(row), rows = static_cast<int>(p.M);
    for (int s = tid; s < p.n_seg; s += blockDim.x) {
      const int lo = p.seg_offsets[s], hi = p.seg_offsets[s + 1];
      if (lo <= at && at < hi) s_seg = s;
      if (lo < 0 || hi < lo || hi > rows) s_bad = 1;  // overlapping ones have no one variant
    }
    __syncthreads();
    if (s_bad != 0) {
      if (tid == 0) record_error(p.ctx, kErrBounds);
      return;
    }
    if (s_seg < 0) return;  // a row of no segment
    slot = p.seg_variant[s_seg];
    if (slot < 0 || slot >= p.n_tab) {
      if (tid == 0) record_error(p.ctx, kErrBounds);
      slot = 0;
    }
  }
  const uint16_t* w_pre = p.pre_table ? weights_of(p.pre_table, slot, p.ctx) : nullptr;

  float inv_post = 1.f;
  const uint16_t* w_post = nullptr;
  if (p.post_table != nullptr) {
    w_post = weights_of(p.post_table, slot, p.ctx);
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8];
      unpack8(yv[c], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
    }
    inv_post = rsqrtf(block_sum(ss, s_post) / static_cast<float>(p.d) + p.eps);
  }

  float h[C][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + tid;
    float f[8], r[8];
    unpack8(yv[c], f);
    if constexpr (kF32) {
      const uint32_t u[8] = {ra[c].x, ra[c].y, ra[c].z, ra[c].w,
                             rb[c].x, rb[c].y, rb[c].z, rb[c].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = __uint_as_float(u[e]);
    } else {
      unpack8(ra[c], r);
    }
    if (w_post != nullptr && i < n8) {
      float w[8];
      unpack8(ldg_v4(reinterpret_cast<const uint4*>(w_post) + i), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= w[e];
    }
    if (p.gate != nullptr) {
      float g[8];
      unpack8(gv[c], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= g[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[c][e] = fmaf(f[e], p.scale * inv_post, r[e]);
      ss = fmaf(h[c][e], h[c][e], ss);
    }
    if (i < n8 && p.residual_out != nullptr) {
      if constexpr (kF32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + row * p.d);
        o[2 * i] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
        o[2 * i + 1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
      } else {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + row * p.d)[i] =
            pack8(h[c]);
      }
    }
  }
  if (p.x_out == nullptr) return;
  uint4 wv[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + tid;
    // 0x3F80 is one
    wv[c] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (i < n8 && w_pre != nullptr) wv[c] = ldg_v4(reinterpret_cast<const uint4*>(w_pre) + i);
  }
  const float inv = rsqrtf(block_sum(ss, s_pre) / static_cast<float>(p.d) + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + tid;
    float w[8];
    unpack8(wv[c], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= h[c][e] * inv;
    if (i < n8) reinterpret_cast<uint4*>(p.x_out + row * p.d)[i] = pack8(w);
  }
}

template <int C>
cudaError_t launch_c(NormArgs p, int sms, bool f32, int threads, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.M)), block(threads);
  if (f32) return launch_pdl(add_norm_kernel<C, true, false>, grid, block, 0, s, p);
  // Where an SM holds at most two CTAs, their loads stop together while they sum:
  // with two rounds of CTAs or more, half a round is fetched ahead (2048 rows of
  // 8192, bf16, 23.9 -> 21.9 us; 1024 of 16384 34.3 -> 30.9; of 6144 21.3 -> 20.7).
  // More, smaller CTAs cover one another (8192 rows of 1024 16.0 -> 16.4 us, 2048
  // of 5120 unchanged), fewer rounds leave little to fetch (500 rows of 8192 7.6
  // -> 7.9), and rows with an fp32 residual lose by it (4096 of 8192 74.3 -> 78.4).
  const int resident = (C == 1 ? 2048 : 1024) / threads;
  if (resident > 2 || p.M < 2 * static_cast<int64_t>(sms) * resident)
    return launch_pdl(add_norm_kernel<C, false, false>, grid, block, 0, s, p);
  p.ahead = sms * resident / 2;
  return launch_pdl(add_norm_kernel<C, false, true>, grid, block, 0, s, p);
}

cudaError_t launch_add_norm(const NormArgs& p, int sms, bool f32, cudaStream_t s) {
  const int n8 = p.d / 8;
  const auto threads = [&](int c) { return ((n8 + c - 1) / c + 31) / 32 * 32; };
  if (n8 <= 1024) return launch_c<1>(p, sms, f32, threads(1), s);
  if (n8 <= 2048) return launch_c<2>(p, sms, f32, threads(2), s);
  if (n8 <= 4096) return launch_c<4>(p, sms, f32, threads(4), s);
  return launch_c<8>(p, sms, f32, threads(8), s);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace
}  // namespace bd

extern "C" bd_status bitdelta_add_norm(const uint16_t* y, int64_t M, int64_t d,
                                       const void* residual, void* residual_out,
                                       bd_residual_type rtype, const uint16_t* gate,
                                       int64_t gate_stride, float scale, float eps,
                                       const uint16_t* const* pre_table,
                                       const uint16_t* const* post_table, int32_t n_tab,
                                       const int32_t* seg_offsets, const int32_t* seg_variant,
                                       int32_t n_seg, uint16_t* x_out, bd_stream_t stream) {
  if (M < 0 || d < 1 || n_seg < 0 || n_tab < 0) return BD_ERR_INVALID_ARG;
  if (rtype != BD_RESIDUAL_BF16 && rtype != BD_RESIDUAL_F32) return BD_ERR_INVALID_ARG;
  if (gate != nullptr && gate_stride != 0 && gate_stride != d) return BD_ERR_INVALID_ARG;
  if ((seg_offsets == nullptr) != (seg_variant == nullptr)) return BD_ERR_INVALID_ARG;
  if (seg_offsets == nullptr && n_seg != 0) return BD_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 65536) return BD_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || (seg_offsets != nullptr && n_seg == 0)) return BD_OK;
  if (M > 0x7FFFFFFF) return BD_ERR_UNSUPPORTED_SHAPE;
  if (!y || (!x_out && !residual_out)) return BD_ERR_INVALID_ARG;
  if ((x_out && !pre_table) || ((pre_table || post_table) && n_tab < 1))
    return BD_ERR_INVALID_ARG;
  if (bd::off16(y) || bd::off16(residual) || bd::off16(residual_out) || bd::off16(gate) ||
      bd::off16(x_out) || bd::off(pre_table, 8) || bd::off(post_table, 8) ||
      bd::off(seg_offsets, 4) || bd::off(seg_variant, 4))
    return BD_ERR_MISALIGNED;
  bd::NormArgs p{};
  int sms = 0;
  const int st = bd::current_device_context(&p.ctx, &sms);
  if (st != BD_OK) return static_cast<bd_status>(st);
  p.y = y;
  p.residual = residual;
  p.residual_out = residual_out;
  p.gate = gate;
  p.gate_stride = gate_stride;
  p.scale = scale;
  p.eps = eps;
  p.pre_table = x_out ? pre_table : nullptr;
  p.post_table = post_table;
  p.n_tab = n_tab;
  p.seg_offsets = seg_offsets;
  p.seg_variant = seg_variant;
  p.n_seg = n_seg;
  p.x_out = x_out;
  p.M = M;
  p.d = static_cast<int32_t>(d);
  const cudaError_t e = bd::launch_add_norm(p, sms, rtype == BD_RESIDUAL_F32,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}
