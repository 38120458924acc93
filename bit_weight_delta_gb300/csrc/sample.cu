// sample.cu — a token per row of logits (bitdelta_sample).
//
// A bf16 row has fewer than 2^16 different values, so all that the cuts and the
// choice need of it is how often each value occurs: one pass over the row counts
// its values in shared memory, 16 bits a value.  A value's weight
//   w = exp((v − largest)/T)
// is then formed once per value instead of once per token, to about 2^-40 and as
// a whole number of 2^-44 steps, and every cut is a prefix of the order (largest value
// first, equal ones by index): top_k a count, top_p a sum, min_p a weight.  Sums of
// whole numbers do not depend on the order of the work, so the choice is the same
// however a row is spread.  The chosen value and its number r among its equals
// give the token: a second look at one CTA's part of the row finds the r-th.
//
// A row is shared by a cluster of CTAs, each with counts of its own part, which
// are added where they are read (distributed shared memory).  Values lie in the
// order of the bins: bin = 0x7FFF − bits for positive ones and bits for
// negative ones, a bin's count in half of a 32-bit word (bin & 0x7FFF): the low
// half for positive values.  Segments are 32 bins; most are empty.
#include <cooperative_groups.h>

#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {
namespace {

namespace cg = cooperative_groups;

struct SampleArgs {
  const uint16_t* logits;
  int64_t V, stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* prob;
  DevCtx ctx;
};

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kWords = 32768;   // counts, two bins each
constexpr int kSegs = 2048;     // of 32 bins
constexpr int kMaxCluster = 8;
constexpr int kMaxChunks = 8190;  // 8-element chunks of a CTA: counts stay below 2^16
constexpr int kOneBits = 44;      // a weight of 1 is 2^44; 2^19 of them stay below 2^63
constexpr int kBinFirst = 0x7F;   // +inf; NaN lies below
constexpr int kBinLast = 0xFF7F;  // −inf and NaN lie above
constexpr int kZeroBin = 0x7FFF;

// 2^(j/64) to 48 bits, from the exponential's series.
constexpr double exp_series(double x) {
  double sum = 1.0, term = 1.0;
  for (int i = 1; i < 30; ++i) {
    term *= x / i;
    sum += term;
  }
  return sum;
}
struct Pow2Table {
  float hi[64], lo[64];
};
constexpr Pow2Table make_pow2_table() {
  Pow2Table t{};
  for (int j = 0; j < 64; ++j) {
    const double v = exp_series(0.69314718055994530942 * j / 64);
    t.hi[j] = static_cast<float>(v);
    t.lo[j] = static_cast<float>(v - static_cast<double>(t.hi[j]));
  }
  return t;
}
__device__ constexpr Pow2Table kPow2 = make_pow2_table();

struct Shared {
  uint32_t counts[kWords];
  uint64_t mass[kSegs];     // rank 0: sums before each listed segment
  uint32_t number[kSegs];
  uint16_t list[kSegs];     // segments that are not empty, in order
  uint32_t occupied[kSegs / 32];   // this CTA's
  float pow2_hi[64], pow2_lo[64];
  uint64_t scan_mass[kWarps];
  uint32_t scan_number[kWarps];
  float c_hi, c_lo;         // 2·log2(e)/T
  int first;                // the largest value's bin, of this CTA's part
  int all_first;
  int n_list;
  int find_bin;             // the token's value, or −1: not in this CTA's part
  uint32_t find_rank;       // its number among this CTA's tokens of that value
  float find_prob;
  uint32_t warp_hits[kWarps];
};

__device__ __forceinline__ float value_of(int bin) {
  const uint32_t b = bin < 0x8000 ? 0x7FFF - bin : bin;
  return __uint_as_float(b << 16);
}

// The weight of a value relative to the largest, in 2^-44: 2^y with y =
// (v − max)·log2(e)/T held in two floats (half the difference, so that it stays
// finite; 2·log2(e)/T for it).  2^y = 2^n · 2^(j/64) · e^t with |t| < 0.0055, where
// e^t − 1 = t + t²/2 + … needs only its first term in two floats.
__device__ uint64_t weight_of(const Shared& sh, int bin, int first) {
  if (bin == first) return uint64_t{1} << kOneBits;
  if (first == kBinFirst) return 0;  // +inf takes all
  const float a = 0.5f * value_of(bin), b = -0.5f * value_of(first);
  const float dh = __fadd_rn(a, b);
  const float bb = __fsub_rn(dh, a);
  const float dl = __fadd_rn(__fsub_rn(a, __fsub_rn(dh, bb)), __fsub_rn(b, bb));
  const float yh = __fmul_rn(dh, sh.c_hi);
  if (!(yh > -46.f)) return 0;
  const float ye = __fmaf_rn(dh, sh.c_hi, -yh);
  const float yl = __fmaf_rn(dh, sh.c_lo, __fmaf_rn(dl, sh.c_hi, ye));
  const float k = rintf(yh * 64.f);
  const float r = __fmaf_rn(k, -1.f / 64.f, yh);  // exact
  constexpr double ln2 = 0.69314718055994530942;
  constexpr float l2h = static_cast<float>(ln2);
  constexpr float l2l = static_cast<float>(ln2 - static_cast<double>(l2h));
  const float p = __fmul_rn(r, l2h);
  const float q = __fmaf_rn(r, l2h, -p) + __fmaf_rn(r, l2l, yl * l2h);
  const float th = __fadd_rn(p, q);
  const float tl = __fsub_rn(q, __fsub_rn(th, p));
  const float series = 0.5f + th * (1.f / 6.f + th * (1.f / 24.f + th * (1.f / 120.f)));
  const float w = __fmaf_rn(th * th, series, __fmaf_rn(th, tl, tl));
  const int ki = static_cast<int>(k);
  const float hi = sh.pow2_hi[ki & 63], lo = sh.pow2_lo[ki & 63];
  const float ph = __fmul_rn(hi, th);
  const float pe = __fmaf_rn(hi, th, -ph);
  const float s = __fadd_rn(hi, ph);
  const float e = __fsub_rn(ph, __fsub_rn(s, hi));
  const float rest = e + (pe + (__fmaf_rn(hi, w, lo) + lo * th));
  const float unit = __int_as_float((127 + kOneBits + (ki >> 6)) << 23);
  return static_cast<uint64_t>(__float2ll_rn(s * unit) + __float2ll_rn(rest * unit));
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

// Eight logits from a 16-byte boundary on; those outside the row are NaN.
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int64_t V, int mis, int chunk) {
  const int64_t i0 = static_cast<int64_t>(chunk) * 8 - mis;
  if (i0 >= 0 && i0 + 8 <= V) return ldg_stream_v4(row + i0);
  uint32_t w[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int64_t i = i0 + 2 * x;
    const uint32_t lo = i >= 0 && i < V ? row[i] : 0x7FFFu;
    const uint32_t hi = i + 1 >= 0 && i + 1 < V ? row[i + 1] : 0x7FFFu;
    w[x] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The bins of two logits.
__device__ __forceinline__ uint32_t bins_of(uint32_t w) {
  uint32_t negative;  // 0xFFFF where the sign is set: bytes 1 and 3's signs, twice each
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(w));
  return w ^ (0x7FFF7FFFu & ~negative);
}

__device__ __forceinline__ void count(uint32_t* counts, uint32_t bin) {
  atomicAdd(counts + (bin & 0x7FFFu), bin & 0x8000u ? 0x10000u : 1u);
}

// What a position in the order needs: the bin that holds it and what lies before.
struct Place {
  int bin;
  uint32_t number;   // tokens before the bin
  uint64_t mass;     // their weight
  uint64_t weight;   // of one of the bin's tokens
  uint32_t count;    // of them
};

// Tokens of `bin` in the whole row.
__device__ __forceinline__ uint32_t count_of(const uint32_t* const (&counts)[kMaxCluster],
                                             int ranks, int bin) {
  const int shift = bin & 0x8000 ? 16 : 0;
  uint32_t n = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < ranks) n += counts[r][bin & 0x7FFF] >> shift & 0xFFFFu;
  return n;
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const int64_t m = blockIdx.x / C;
  const uint16_t* row = p.logits + m * p.stride;
  const auto meet = [&] {
    if constexpr (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };

  for (int i = tid; i < kWords / 4; i += kThreads)
    reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < 64) {
    sh.pow2_hi[tid] = kPow2.hi[tid];
    sh.pow2_lo[tid] = kPow2.lo[tid];
    sh.occupied[tid] = 0u;
  }
  if (tid == 0) sh.first = kBinLast + 1;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) {
    const double c = 2.8853900817779268 /  // 2·log2(e)
                     static_cast<double>(p.temperature != nullptr ? p.temperature[m] : 1.f);
    sh.c_hi = static_cast<float>(c);
    sh.c_lo = isinf(sh.c_hi) ? 0.f : static_cast<float>(c - static_cast<double>(sh.c_hi));
  }
  __syncthreads();

  // ---- counts of this CTA's part
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 7);
  const int chunks = static_cast<int>((p.V + mis + 7) >> 3);
  const int per = (chunks + C - 1) / C;
  const int c0 = rank * per < chunks ? rank * per : chunks;
  const int c1 = c0 + per < chunks ? c0 + per : chunks;
  constexpr int kUnroll = 4;
  for (int c = c0 + tid; c < c1; c += kUnroll * kThreads) {
    uint4 v[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x)
      if (c + x * kThreads < c1) v[x] = load_chunk(row, p.V, mis, c + x * kThreads);
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      if (c + x * kThreads >= c1) break;
      const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t b = bins_of(w[y]);
        count(sh.counts, b & 0xFFFFu);
        count(sh.counts, b >> 16);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {  // −0 counts as 0
    const uint32_t minus = sh.counts[0] >> 16;  // bin 0x8000
    sh.counts[0] &= 0xFFFFu;
    sh.counts[kZeroBin] += minus;
  }
  __syncthreads();

  // ---- which segments hold anything
  for (int s = warp; s < kSegs / 2; s += kWarps) {
    const uint32_t w = sh.counts[32 * s + lane];
    const uint32_t pos = __ballot_sync(0xFFFFFFFFu, (w & 0xFFFFu) != 0 && 32 * s + lane >= kBinFirst);
    const uint32_t neg =
        __ballot_sync(0xFFFFFFFFu, (w >> 16) != 0 && 0x8000 + 32 * s + lane <= kBinLast);
    if (lane == 0) {
      if (pos != 0) {
        atomicOr(&sh.occupied[s >> 5], 1u << (s & 31));
        atomicMin(&sh.first, 32 * s + __ffs(pos) - 1);
      }
      if (neg != 0) {
        atomicOr(&sh.occupied[32 + (s >> 5)], 1u << (s & 31));
        atomicMin(&sh.first, 0x8000 + 32 * s + __ffs(neg) - 1);
      }
    }
  }
  meet();
  const uint32_t* counts[kMaxCluster];
#pragma unroll
  for (int r = 0; r < C; ++r)
    counts[r] = C == 1 ? sh.counts : cluster.map_shared_rank(sh.counts, r);
  if (warp == 0) {
    int first = kBinLast + 1;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const Shared* o = C == 1 ? &sh : cluster.map_shared_rank(&sh, r);
      first = o->first < first ? o->first : first;
      w[0] |= o->occupied[lane];
      w[1] |= o->occupied[32 + lane];
    }
    int at = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int inc = warp_inclusive(__popc(w[x]));
      int to = at + inc - __popc(w[x]);
      for (uint32_t bits = w[x]; bits != 0; bits &= bits - 1)
        sh.list[to++] = static_cast<uint16_t>(1024 * x + 32 * lane + __ffs(bits) - 1);
      at += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) {
      sh.n_list = at;
      sh.all_first = first;
      sh.find_bin = -1;
    }
  }
  __syncthreads();
  const int n_list = sh.n_list, first = sh.all_first;

  // ---- the segments' numbers of tokens and weights, to the first CTA
  Shared* lead = C == 1 ? &sh : cluster.map_shared_rank(&sh, 0);
  for (int j = rank * kWarps + warp; j < n_list; j += C * kWarps) {
    const int bin = 32 * sh.list[j] + lane;
    uint32_t n = bin >= kBinFirst && bin <= kBinLast ? count_of(counts, C, bin) : 0u;
    uint64_t w = n != 0 ? n * weight_of(sh, bin, first) : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
      w += __shfl_xor_sync(0xFFFFFFFFu, w, off);
    }
    if (lane == 0) {
      lead->number[j] = n;
      lead->mass[j] = w;
    }
  }
  meet();

  if (rank == 0) {
    // exclusive sums over the listed segments, two per thread
    uint32_t n[2];
    uint64_t w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      n[x] = 2 * tid + x < n_list ? sh.number[2 * tid + x] : 0u;
      w[x] = 2 * tid + x < n_list ? sh.mass[2 * tid + x] : 0u;
    }
    const uint32_t ni = warp_inclusive(n[0] + n[1]);
    const uint64_t wi = warp_inclusive(w[0] + w[1]);
    if (lane == 31) {
      sh.scan_number[warp] = ni;
      sh.scan_mass[warp] = wi;
    }
    __syncthreads();
    if (warp == 0) {
      const uint32_t a = sh.scan_number[lane];
      const uint64_t b = sh.scan_mass[lane];
      sh.scan_number[lane] = warp_inclusive(a) - a;
      sh.scan_mass[lane] = warp_inclusive(b) - b;
    }
    __syncthreads();
    uint32_t nb = sh.scan_number[warp] + ni - n[0] - n[1];
    uint64_t wb = sh.scan_mass[warp] + wi - w[0] - w[1];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (2 * tid + x < n_list) {
        sh.number[2 * tid + x] = nb;
        sh.mass[2 * tid + x] = wb;
      }
      nb += n[x];
      wb += w[x];
    }
    if (tid == kThreads - 1) {
      sh.scan_number[0] = nb;  // the whole row
      sh.scan_mass[0] = wb;
    }
    __syncthreads();

    if (warp == 0) {
      const uint32_t all = sh.scan_number[0];
      const uint64_t all_mass = sh.scan_mass[0];
      float u = p.u[m];
      const float t = p.temperature != nullptr ? p.temperature[m] : 1.f;
      const int k = p.top_k != nullptr ? p.top_k[m] : 0;
      const float top_p = p.top_p != nullptr ? p.top_p[m] : 1.f;
      const float min_p = p.min_p != nullptr ? p.min_p[m] : 0.f;
      const bool bad = !(t >= 0.f) || isnan(u) || isnan(top_p) || isnan(min_p);
      if (bad || all == 0) {
        if (lane == 0) {
          if (bad) record_error(p.ctx, kErrBounds);
          p.tokens[m] = -1;
          if (p.prob != nullptr) p.prob[m] = 0.f;
        }
      } else {
        // The last listed segment for which `before` holds (it holds for the
        // first, and for all before one that it holds for).
        const auto search = [&](auto before) {
          int lo = 0, hi = n_list;
          while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
            const uint32_t yes = __ballot_sync(0xFFFFFFFFu, at < hi && (lane == 0 || before(at)));
            const int top = 31 - __clz(yes);
            lo += top * step;
            hi = lo + step < hi ? lo + step : hi;
          }
          return lo;
        };
        // The bin of segment j in which `inside` first holds of a lane's bin's sums
        // before and after; all lanes receive it.
        const auto bin_in = [&](int j, auto inside) {
          const int bin = 32 * sh.list[j] + lane;
          Place pl;
          pl.bin = bin;
          pl.count = bin >= kBinFirst && bin <= kBinLast ? count_of(counts, C, bin) : 0u;
          pl.weight = pl.count != 0 ? weight_of(sh, bin, first) : 0;
          const uint64_t w_all = pl.count * pl.weight;
          pl.number = sh.number[j] + warp_inclusive(pl.count) - pl.count;
          pl.mass = sh.mass[j] + warp_inclusive(w_all) - w_all;
          const uint32_t yes = __ballot_sync(0xFFFFFFFFu, pl.count != 0 && inside(pl));
          const int src = yes != 0 ? __ffs(yes) - 1 : 0;
          pl.bin = __shfl_sync(0xFFFFFFFFu, pl.bin, src);
          pl.number = __shfl_sync(0xFFFFFFFFu, pl.number, src);
          pl.mass = __shfl_sync(0xFFFFFFFFu, pl.mass, src);
          pl.weight = __shfl_sync(0xFFFFFFFFu, pl.weight, src);
          pl.count = __shfl_sync(0xFFFFFFFFu, pl.count, src);
          return pl;
        };
        // The weight of the first n tokens, 1 <= n <= all.
        const auto mass_of = [&](uint32_t n) {
          if (n == all) return all_mass;
          const int j = search([&](int i) { return sh.number[i] < n; });
          const Place pl = bin_in(j, [&](const Place& x) { return x.number + x.count >= n; });
          return pl.mass + (n - pl.number) * pl.weight;
        };
        // floor(w·f), and whether that is all of it; f in [0, 1).
        const auto share = [](uint64_t w, float f, bool* exact) {
          const uint64_t fixed = __float2ull_rz(f * 18446744073709551616.f);
          *exact = w * fixed == 0;
          return __umul64hi(w, fixed);
        };
        uint32_t n = all;
        uint64_t kept = all_mass;
        bool exact;
        if (k > 0 && static_cast<uint32_t>(k) < all) {
          n = static_cast<uint32_t>(k);
          kept = mass_of(n);
        }
        if (t == 0.f) n = 1;
        uint32_t cut = n;
        if (cut > 1 && top_p < 1.f) {
          const uint64_t down = share(kept, top_p > 0.f ? top_p : 0.f, &exact);
          const uint64_t want = down + (exact ? 0 : 1);
          if (want == 0) {
            cut = 1;
          } else {
            const int j = search([&](int i) { return sh.mass[i] < want; });
            const Place pl = bin_in(j, [&](const Place& x) {
              return x.mass + x.count * x.weight >= want;
            });
            const uint32_t at =
                pl.number + static_cast<uint32_t>((want - pl.mass + pl.weight - 1) / pl.weight);
            cut = at < cut ? at : cut;
          }
        }
        if (cut > 1 && min_p > 0.f) {
          const uint64_t least =
              min_p >= 1.f ? uint64_t{1} << kOneBits
                           : static_cast<uint64_t>(ceilf(min_p * static_cast<float>(uint64_t{1} << kOneBits)));
          const int j = search([&](int i) {
            const int bin = 32 * sh.list[i];
            return weight_of(sh, bin < first ? first : bin, first) >= least;
          });
          // (a bin below the weight, or none in this segment)
          const int bin = 32 * sh.list[j] + lane;
          const uint32_t c = bin >= kBinFirst && bin <= kBinLast ? count_of(counts, C, bin) : 0u;
          uint32_t with = c != 0 && weight_of(sh, bin, first) >= least ? c : 0u;
          with = __reduce_add_sync(0xFFFFFFFFu, with);
          const uint32_t at = sh.number[j] + with;
          cut = at < cut ? (at > 0 ? at : 1) : cut;
        }
        if (cut != n || t == 0.f) kept = mass_of(cut);
        u = u > 0.f ? u : 0.f;
        uint64_t target = u < 1.f ? share(kept, u, &exact) : kept - 1;
        const int j = search([&](int i) { return sh.mass[i] <= target; });
        const Place pl = bin_in(j, [&](const Place& x) {
          return x.mass + x.count * x.weight > target;
        });
        uint32_t r = static_cast<uint32_t>((target - pl.mass) / pl.weight);
        // whose part holds the r-th token of that value
        int owner = 0;
        const int shift = pl.bin & 0x8000 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < C - 1; ++i) {
          const uint32_t c = counts[i][pl.bin & 0x7FFF] >> shift & 0xFFFFu;
          if (owner == i && r >= c) {
            r -= c;
            ++owner;
          }
        }
        if (lane == 0) {
          Shared* o = C == 1 ? &sh : cluster.map_shared_rank(&sh, owner);
          o->find_bin = pl.bin;
          o->find_rank = r;
          o->find_prob = static_cast<float>(static_cast<double>(pl.weight) /
                                            static_cast<double>(kept));
        }
      }
    }
  }
  meet();
  const int bin = sh.find_bin;
  if (bin < 0) return;

  // ---- the r-th token of that value in this CTA's part: each warp looks through
  // a range of it, and the one that holds the token through its own once more
  const uint32_t bits = bin < 0x8000 ? 0x7FFFu - bin : static_cast<uint32_t>(bin);
  const uint32_t mask = bin == kZeroBin ? 0x7FFF7FFFu : 0xFFFFFFFFu;
  const uint32_t pattern = bits | bits << 16;
  const int w_per = (c1 - c0 + kWarps - 1) / kWarps;
  const int w0 = c0 + warp * w_per < c1 ? c0 + warp * w_per : c1;
  const int w1 = w0 + w_per < c1 ? w0 + w_per : c1;
  const auto hits_of = [&](int c) {  // two bits per pair of logits
    const uint4 v = load_chunk(row, p.V, mis, c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint32_t x = (w[y] & mask) ^ pattern;
      h |= ((x & 0xFFFFu) == 0 ? 1u : 0u) << (2 * y) | (x >> 16 == 0 ? 2u : 0u) << (2 * y);
    }
    return h;
  };
  uint32_t hits = 0;
#pragma unroll 4
  for (int c = w0 + lane; c < w1; c += 32) hits += __popc(hits_of(c));
  hits = __reduce_add_sync(0xFFFFFFFFu, hits);
  if (lane == 0) sh.warp_hits[warp] = hits;
  __syncthreads();
  uint32_t before = 0;
  for (int i = 0; i < warp; ++i) before += sh.warp_hits[i];
  const uint32_t r = sh.find_rank;
  if (r < before || r >= before + hits) return;
  for (int c = w0; c < w1; c += 32) {
    const uint32_t h = c + lane < w1 ? hits_of(c + lane) : 0u;
    const uint32_t inc = before + warp_inclusive(static_cast<uint32_t>(__popc(h)));
    if (r < inc && r >= inc - __popc(h)) {
      uint32_t left = r - (inc - __popc(h)), x = h;
      for (; left > 0; --left) x &= x - 1;
      p.tokens[m] = static_cast<int32_t>(static_cast<int64_t>(c + lane) * 8 - mis + __ffs(x) - 1);
      if (p.prob != nullptr) p.prob[m] = sh.find_prob;
    }
    before = __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
}

template <int C>
cudaError_t launch(const SampleArgs& p, int64_t M, cudaStream_t s) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(sample_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(sizeof(Shared)));
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  return launch_pdl_cluster(sample_kernel<C>, dim3(static_cast<unsigned>(M * C)), dim3(kThreads),
                            C, sizeof(Shared), s, p);
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace
}  // namespace bd

extern "C" bd_status bitdelta_sample(const uint16_t* logits, int64_t M, int64_t V,
                                     int64_t row_stride, const float* u,
                                     const float* temperature, const int32_t* top_k,
                                     const float* top_p, const float* min_p, int32_t* tokens,
                                     float* prob, bd_stream_t stream) {
  if (M < 0 || V < 1 || row_stride < V) return BD_ERR_INVALID_ARG;
  if (V > 524032 || M > (1 << 26) || row_stride > (int64_t{1} << 32))
    return BD_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return BD_OK;
  if (!logits || !u || !tokens) return BD_ERR_INVALID_ARG;
  if (bd::off(logits, 2) || bd::off(u, 4) || bd::off(temperature, 4) || bd::off(top_k, 4) ||
      bd::off(top_p, 4) || bd::off(min_p, 4) || bd::off(tokens, 4) || bd::off(prob, 4))
    return BD_ERR_MISALIGNED;
  bd::SampleArgs p{};
  int sms = 0;
  const int st = bd::current_device_context(&p.ctx, &sms);
  if (st != BD_OK) return static_cast<bd_status>(st);
  p.logits = logits;
  p.V = V;
  p.stride = row_stride;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.tokens = tokens;
  p.prob = prob;
  // CTAs per row: as many as the counts' 16 bits need, and more while all rows'
  // still fit the device at once.
  const int64_t chunks = (V + 14) / 8;
  int c = 1;
  while (c < bd::kMaxCluster &&
         (chunks > static_cast<int64_t>(bd::kMaxChunks) * c || M * 2 * c <= sms))
    c *= 2;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c == 1   ? bd::launch<1>(p, M, s)
                        : c == 2 ? bd::launch<2>(p, M, s)
                        : c == 4 ? bd::launch<4>(p, M, s)
                                 : bd::launch<8>(p, M, s);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}
