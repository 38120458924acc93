// attn_decode.cu — the decode kernel: two CTAs of four warps per SM over a batch
// of short runs alone (attn_decode.cuh).
#include "attn_decode.cuh"

namespace bd {
namespace {

constexpr int kWarps = kDecodeWarps;

template <int D, int RT>
__global__ void __launch_bounds__(32 * kWarps, 2)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const AttnArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  attn_decode::init<D, RT, kWarps>(smem, warp, lane);
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  attn_decode::run<D, RT, kWarps>(tmap_k, tmap_v, p, smem, warp, lane,
                                  static_cast<int>(blockIdx.x));
}

template <int D, int RT>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                   cudaStream_t s) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(attn_decode_kernel<D, RT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               attn_decode::Cfg<D, RT, kWarps>::kSmem);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  return launch_pdl(attn_decode_kernel<D, RT>, dim3(a.L.d_ctas), dim3(32 * kWarps),
                    attn_decode::Cfg<D, RT, kWarps>::kSmem, s, tk, tv, a);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
  if (a.b.head_dim == 128)
    return launch<128, 1>(a, tk, tv, s);
  return a.L.d_rows == 16 ? launch<64, 1>(a, tk, tv, s) : launch<64, 2>(a, tk, tv, s);
}

}  // namespace bd
