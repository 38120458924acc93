// sample.cu — a token per row of logits (bitdelta_sample).
//
// A bf16 row has fewer than 2^16 different values, so all that the cuts and the
// choice need of it is how often each value occurs: one pass over the row counts
// its values in shared memory.  A value's weight
//   w = exp((v − largest)/T)
// is then formed once per value instead of once per token, to about 2^-40 and as
// a whole number of 2^-44 steps, and every cut is a prefix of the order (largest value
// first, equal ones by index): top_k a count, top_p a sum, min_p a weight.  Sums of
// whole numbers do not depend on the order of the work, so the choice is the same
// however a row is spread.  The chosen value and its number r among its equals
// give the token: a second look at one CTA's part of the row finds the r-th.
//
// Values are numbered by their bin: 0x7FFF − bits for positive ones and bits for
// negative ones, the largest value first.  Counted are the values from 2^-40 to 2^16 in
// size, and zero: two tables of 7168 counters, of 32 bits, with one more at either end
// for what lies outside.  (All bins' would fill an SM's shared memory with 16-bit ones,
// and their phases of few threads would stand alone: 500 rows of 99991 took 161 us.)
// Additions of 1 to one address are merged by the hardware (17 a clock, and 8 to different
// ones), so that a masked row costs no more than another.  A row with a value outside
// that may be taken goes through all bins in several passes, by one CTA.
//
// A row is shared by a cluster of CTAs, each with counts of its own part, which
// are added where they are read (distributed shared memory); a cluster takes row
// after row.  Segments are 32 bins, a lane each; most are empty.
//
// Bound by the counters' additions where rows are many (500 of 99991 80.2 us, where their
// bytes are 15), and by the chain of short phases where they are few (one of 32000
// 16.0 us, 64 of 128000 26.0).
#include <cooperative_groups.h>

#include <cstdint>

#include "bitdelta_decode.h"
#include "kernels.h"

namespace bd {
namespace {

namespace cg = cooperative_groups;

struct SampleArgs {
  const uint16_t* logits;
  int64_t M, V, stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* prob;
  DevCtx ctx;
};

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 2;          // per SM
constexpr int kMaxCluster = 8;
constexpr int kOneBits = 44;      // a weight of 1 is 2^44; 2^19 of them stay below 2^63
constexpr int kBinFirst = 0x7F;   // +inf; NaN lies below
constexpr int kBinLast = 0xFF7F;  // −inf and NaN lie above
constexpr int kZeroBin = 0x7FFF;
constexpr int kSegs = 2048;       // of 32 bins, of all bins

// The counters: of either sign kSpan bins, behind one for the bins before them and with
// one for those that follow.  Behind the positive ones (and before the
// negative) lie zero and what is smaller than the counted values.
constexpr int kSpan = 56 * 128;
constexpr int kPosBin = 0x8000 - ((127 + 16) << 7) - 1;  // 2^16, of slot 0
constexpr int kNegShift = 0x8000 + ((127 - 40) << 7) - 1 - kPosBin;  // to the negative bins
constexpr int kNegSlot = kSpan + 64;
constexpr int kSlots = 2 * kNegSlot;
constexpr int kZeroSlot = kSpan + 1;
constexpr int kFarSlot = kNegSlot + kSpan + 1;  // −2^16 and below, −inf, −NaN
static_assert(kSlots % 128 == 0, "four segments at a time");
constexpr int kSlotSegs = kSlots / 32;
constexpr int kMasks = (kSlotSegs + 31) / 32;
// The least size that is counted, as a bf16 number's bits.
constexpr uint32_t kLeastBits = (127 - 40) << 7;

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
  uint32_t counts[kSlots];
  uint64_t mass[kSegs];            // rank 0: sums before each listed segment
  uint32_t number[kSegs];
  uint16_t list[kSegs];            // segments that are not empty, in order
  uint32_t seg_counts[32];         // one segment's, where all bins are gone through
  alignas(8) uint8_t flags[8 * kMasks];  // of four segments each: not empty (0 behind them)
  uint32_t occupied[kMasks];       // this CTA's
  float pow2_hi[64], pow2_lo[64];
  float half, c_hi, c_lo;          // 1/2 and 2·log2(e)/T (2^-65 and 2^64 of it for large T)
  int first, all_first;            // the largest value's bin, of this part and of the row
  int wide, all_wide;              // values outside of the counted ones
  int far;                         // logits of −2^16 and below
  int n_list;
  int asked;                       // the segment that the CTA is to count, or −1
  int find_bin;                    // the token's value, or −1: not in this CTA's part
  uint32_t find_rank;              // its number among this CTA's tokens of that value
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
__device__ __forceinline__ uint64_t weigh(const Shared& sh, int bin, int first) {
  if (bin == first) return uint64_t{1} << kOneBits;
  if (first == kBinFirst) return 0;  // +inf takes all
  const float a = sh.half * value_of(bin), b = -sh.half * value_of(first);
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
__device__ __noinline__ uint64_t weight_of(const Shared& sh, int bin, int first) {
  return weigh(sh, bin, first);
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

// Eight logits from a 16-byte boundary on; those outside the row are −NaN.
__device__ __noinline__ uint4 edge_chunk(const uint16_t* row, int64_t V, int64_t i0) {
  uint32_t w[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int64_t i = i0 + 2 * x;
    const uint32_t lo = i >= 0 && i < V ? row[i] : 0xFFFFu;
    const uint32_t hi = i + 1 >= 0 && i + 1 < V ? row[i + 1] : 0xFFFFu;
    w[x] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int64_t V, int mis, int chunk) {
  const int64_t i0 = static_cast<int64_t>(chunk) * 8 - mis;
  if (i0 >= 0 && i0 + 8 <= V) return ldg_stream_v4(row + i0);
  return edge_chunk(row, V, i0);
}

// The bins of two logits.
__device__ __forceinline__ uint32_t bins_of(uint32_t w) {
  uint32_t negative;  // 0xFFFF where the sign is set: bytes 1 and 3's signs, twice each
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(w));
  return w ^ (0x7FFF7FFFu & ~negative);
}

// The bin of a slot of the counters (any, where a slot has none).
__device__ __forceinline__ int bin_of_slot(int slot) {
  return slot < kZeroSlot ? slot + kPosBin
                          : slot < kNegSlot ? kZeroBin : slot - kNegSlot + kPosBin + kNegShift;
}

// Counts two logits.  least: the smallest size of a logit that is not zero, of each half
// (as a negative number: bits − 0x8001; zero is 0x7FFF).
__device__ __forceinline__ void count2(uint32_t* counts, uint32_t w, uint32_t& least) {
  constexpr uint32_t two = 0x10001u;
  least = __vmins2(least, (w | 0x8000u * two) - two);
  uint32_t negative;  // 0xFFFF where the sign is set: bytes 1 and 3's signs, twice each
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(w));
  const uint32_t bin = w ^ (0x7FFF7FFFu & ~negative);
  uint32_t e = bin - (negative & kNegShift * two);
  e = __vminu2(__vmaxu2(e, kPosBin * two), (kPosBin + kSpan + 1) * two) - kPosBin * two;
  const uint32_t at = 4 * e + (negative & 4 * kNegSlot * two);  // bytes, below 2^16
  uint8_t* base = reinterpret_cast<uint8_t*>(counts);
  atomicAdd(reinterpret_cast<uint32_t*>(base + (at & 0xFFFFu)), 1u);
  atomicAdd(reinterpret_cast<uint32_t*>(base + (at >> 16)), 1u);
}

// a / b, below 2^20; 0 where b is.
__device__ __forceinline__ uint32_t quotient(uint64_t a, uint64_t b) {
  if (b == 0) return 0;
  uint32_t q = static_cast<uint32_t>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  while (static_cast<uint64_t>(q) * b > a) --q;
  while ((static_cast<uint64_t>(q) + 1) * b <= a) ++q;
  return q;
}

// What a position in the order needs: the bin that holds it and what lies before.
struct Place {
  int bin;
  uint32_t number;   // tokens before the bin
  uint64_t mass;     // their weight
  uint64_t weight;   // of one of the bin's tokens
  uint32_t count;    // of them
};

// ---- where the counts of a listed segment come from

// The cluster's counters.
template <int C>
struct Counters {
  const uint32_t* counts[C];
  // of the lane
  __device__ __forceinline__ int bin(int seg, int i) const { return bin_of_slot(32 * seg + i); }
  __device__ __forceinline__ uint32_t get(int seg) const {
    uint32_t n = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) n += counts[r][32 * seg + (threadIdx.x & 31)];
    return n;
  }
};

__device__ __forceinline__ void cta_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// Tokens of the bins [base, base + n) in the whole row; a barrier lies before and
// behind it.
__device__ void count_range(const SampleArgs& p, const uint16_t* row, int mis, int base, int n,
                            uint32_t* counts) {
  const int chunks = static_cast<int>((p.V + mis + 7) >> 3);
  for (int c = threadIdx.x; c < chunks; c += kThreads) {
    const uint4 v = load_chunk(row, p.V, mis, c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const uint32_t b = bins_of(w[y >> 1]);
      int bin = static_cast<int>(y & 1 ? b >> 16 : b & 0xFFFFu);
      if (bin == kZeroBin + 1) bin = kZeroBin;
      if (bin >= base && bin < base + n && bin >= kBinFirst && bin <= kBinLast)
        atomicAdd(counts + (bin - base), 1u);
    }
  }
}

// A segment of all bins, counted by the whole CTA when it is asked for.
struct Recount {
  const SampleArgs& p;
  Shared& sh;
  const uint16_t* row;
  int mis;
  __device__ __forceinline__ int bin(int seg, int i) const { return 32 * seg + i; }
  __device__ void count() const {  // every thread
    count_range(p, row, mis, 32 * sh.asked, 32, sh.seg_counts);
    cta_barrier();
  }
  __device__ __forceinline__ uint32_t get(int seg) const {  // the first warp
    const int lane = threadIdx.x & 31;
    sh.seg_counts[lane] = 0;
    if (lane == 0) sh.asked = seg;
    cta_barrier();
    count();
    const uint32_t n = sh.seg_counts[lane];
    __syncwarp();
    return n;
  }
  // the other warps, until the first has what it needs
  __device__ void serve() const {
    while (true) {
      cta_barrier();
      if (sh.asked < 0) return;
      count();
    }
  }
  __device__ void done() const {
    if ((threadIdx.x & 31) == 0) sh.asked = -1;
    cta_barrier();
  }
};

// Exclusive sums over the listed segments, in place; returns those of all.  One warp,
// neighbouring segments to a lane: one scan over the lanes, whatever their number.
__device__ void sum_list(Shared& sh, int n_list, uint32_t& all, uint64_t& all_mass) {
  const int lane = threadIdx.x & 31;
  const int per = (n_list + 31) >> 5;
  const int i0 = lane * per < n_list ? lane * per : n_list;
  const int i1 = i0 + per < n_list ? i0 + per : n_list;
  uint32_t n = 0;
  uint64_t w = 0;
  for (int i = i0; i < i1; ++i) {
    n += sh.number[i];
    w += sh.mass[i];
  }
  uint32_t n_at = warp_inclusive(n);
  uint64_t w_at = warp_inclusive(w);
  all = __shfl_sync(0xFFFFFFFFu, n_at, 31);
  all_mass = __shfl_sync(0xFFFFFFFFu, w_at, 31);
  n_at -= n;
  w_at -= w;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = sh.number[i];
    const uint64_t y = sh.mass[i];
    sh.number[i] = n_at;
    sh.mass[i] = w_at;
    n_at += x;
    w_at += y;
  }
  __syncwarp();
}

// Sums over a warp's lanes, in pieces of 25, 25 and 14 bits (32 of each fit 32 bits).  Any w
// will do whose sum over the lanes fits 64: a row's is below 2^63.
__device__ __forceinline__ void warp_sums(uint32_t& n, uint64_t& w) {
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  const uint32_t a = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(w) & 0x1FFFFFFu);
  const uint32_t b = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(w >> 25) & 0x1FFFFFFu);
  const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(w >> 50));
  w = a + (static_cast<uint64_t>(b) << 25) + (static_cast<uint64_t>(c) << 50);
}

struct Settings {
  float u, t, top_p, min_p;
  int k;
};

// The cuts and the choice, by one warp: the value of the row's token, its number among
// its equals and its probability.  False where there is none.
//
// All of it are questions for the place in the order at which something is reached: a
// number of tokens, a sum, or a weight below `goal`.  One loop asks them: this runs
// once a row, and its instructions are fetched from memory for that.
template <class Source>
__device__ __noinline__ bool choose(const SampleArgs& p, Shared& sh, const Source& source,
                                    const Settings& set, int n_list, int first, int* bin_out,
                                    uint32_t* rank_out, float* prob_out) {
  const int lane = threadIdx.x & 31;
  uint32_t all;
  uint64_t kept;  // the weight of the first `cut` tokens, once it is known
  sum_list(sh, n_list, all, kept);
  const bool bad = !(set.t >= 0.f) || isnan(set.u) || isnan(set.top_p) || isnan(set.min_p);
  if (bad || all == 0) {
    if (bad && lane == 0) record_error(p.ctx, kErrBounds);
    return false;
  }
  constexpr uint64_t one = uint64_t{1} << kOneBits;
  uint32_t cut = set.k > 0 && static_cast<uint32_t>(set.k) < all ? static_cast<uint32_t>(set.k) : all;
  if (set.t == 0.f) cut = 1;
  if (cut != all) kept = cut == 1 ? one : 0;  // 0: to be asked for
  // floor(w·f); f in [0, 1)
  const auto share = [](uint64_t w, float f, bool* exact) {
    const uint64_t fixed = __float2ull_rz(f * 18446744073709551616.f);
    *exact = w * fixed == 0;
    return __umul64hi(w, fixed);
  };
  enum Step { kTopP, kMinP, kChoose };
  enum Kind { kNumber, kMass, kWeight };
  int have = -1;  // the segment that was last looked at: the lane's bin of it
  Place mine{};
  uint64_t target = 0;
#pragma unroll 1
  for (int step = kTopP; step <= kChoose;) {
    // ---- the next question
    Kind kind = kMass;
    uint64_t goal;
    bool exact;
    if (step == kMinP) {
      if (cut == 1 || !(set.min_p > 0.f)) {
        ++step;
        continue;
      }
      kind = kWeight;
      goal = set.min_p >= 1.f
                 ? one : static_cast<uint64_t>(ceilf(set.min_p * static_cast<float>(one)));
    } else {
      if (step == kTopP && (cut == 1 || !(set.top_p < 1.f))) {
        ++step;
        continue;
      }
      if (kept == 0) {
        kind = kNumber;
        goal = cut;
      } else if (step == kTopP) {
        goal = share(kept, set.top_p > 0.f ? set.top_p : 0.f, &exact);
        if (!exact) ++goal;
        if (goal == 0) goal = 1;
      } else {
        const float u = set.u > 0.f ? set.u : 0.f;
        target = u < 1.f ? share(kept, u, &exact) : kept - 1;
        goal = target + 1;
      }
    }
    // ---- the last listed segment before it: that holds for the first, and for all before
    // one that it holds for
    int lo = 0, hi = n_list;
#pragma unroll 1
    while (hi - lo > 1) {
      const int width = (hi - lo + 31) >> 5, at = lo + lane * width;
      bool before = at < hi;
      if (before && lane > 0) {
        if (kind == kNumber) {
          before = sh.number[at] < goal;
        } else if (kind == kMass) {
          before = sh.mass[at] < goal;
        } else {
          const int bin = source.bin(sh.list[at], 0);
          before = weight_of(sh, bin < first ? first : bin, first) >= goal;
        }
      }
      const int top = 31 - __clz(__ballot_sync(0xFFFFFFFFu, before));
      lo += top * width;
      hi = lo + width < hi ? lo + width : hi;
    }
    // ---- its bins, a lane each, and the first that reaches it
    if (lo != have) {
      have = lo;
      const int seg = sh.list[lo];
      mine.count = source.get(seg);
      mine.bin = source.bin(seg, lane);
      mine.weight = weight_of(sh, mine.bin, first);
      const uint64_t w = mine.count * mine.weight;
      mine.number = sh.number[lo] + warp_inclusive(mine.count) - mine.count;
      mine.mass = sh.mass[lo] + warp_inclusive(w) - w;
    }
    if (kind == kWeight) {
      const uint32_t with = __reduce_add_sync(
          0xFFFFFFFFu, mine.weight >= goal ? mine.count : 0u);
      uint32_t at = sh.number[lo] + with;
      at = at > 0 ? at : 1;
      if (at < cut) {
        cut = at;
        kept = cut == 1 ? one : 0;
      }
      ++step;
      continue;
    }
    const bool reaches = kind == kNumber ? mine.number + mine.count >= goal
                                         : mine.mass + mine.count * mine.weight >= goal;
    const uint32_t yes = __ballot_sync(0xFFFFFFFFu, mine.count != 0 && reaches);
    const int src = yes != 0 ? __ffs(yes) - 1 : 0;
    const int bin = __shfl_sync(0xFFFFFFFFu, mine.bin, src);
    const uint32_t number = __shfl_sync(0xFFFFFFFFu, mine.number, src);
    const uint64_t mass = __shfl_sync(0xFFFFFFFFu, mine.mass, src);
    const uint64_t weight = __shfl_sync(0xFFFFFFFFu, mine.weight, src);
    if (kind == kNumber) {
      kept = mass + (goal - number) * weight;
    } else if (step == kTopP) {
      const uint32_t at = number + quotient(goal - mass + weight - 1, weight);
      if (at < cut) {
        cut = at;
        kept = cut == 1 ? one : 0;
      }
      ++step;
    } else {
      *bin_out = bin;
      *rank_out = quotient(target - mass, weight);
      *prob_out = static_cast<float>(weight) / static_cast<float>(kept);
      ++step;
    }
  }
  return true;
}

// The r-th token of the chosen value among the chunks [c0, c1): each warp looks through
// a range of them, in batches, and the one that holds the token at its batch once more.
__device__ __noinline__ void find(const SampleArgs& p, Shared& sh, const uint16_t* row, int64_t m,
                                  int mis, int c0, int c1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bin = sh.find_bin;
  const uint32_t bits = bin < 0x8000 ? 0x7FFFu - bin : static_cast<uint32_t>(bin);
  const uint32_t mask = bin == kZeroBin ? 0x7FFF7FFFu : 0xFFFFFFFFu;
  const uint32_t pattern = bits | bits << 16;
  constexpr int kBatch = 8;  // chunks of a lane, 32 apart
  const int batches = (c1 - c0 + 32 * kBatch - 1) / (32 * kBatch);
  const int per = (batches + kWarps - 1) / kWarps;
  const int b0 = warp * per < batches ? warp * per : batches;
  const int b1 = b0 + per < batches ? b0 + per : batches;
  // the top bit of each half of a chunk's word that is the value
  const auto hit = [&](uint32_t w) {
    const uint32_t d = (w & mask) ^ pattern;
    return ~(((d & 0x7FFF7FFFu) + 0x7FFF7FFFu) | d | 0x7FFF7FFFu);
  };
  const uint32_t r = sh.find_rank;
  uint32_t before = 0;          // of the token, in the part
  uint32_t counts = 0;          // the lane's hits in the last batch, four bits a chunk
  int b = b0, end = b1, last = b0;  // the batch of `counts`
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t hits = 0, mine = 0;  // of the warp; of batch b0 + lane
#pragma unroll 1
    for (; b < end; ++b) {
      const int c = c0 + 32 * kBatch * b + lane;
      uint4 v[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
        v[x] = c + 32 * x < c1 ? load_chunk(row, p.V, mis, c + 32 * x)
                               : make_uint4(~0u, ~0u, ~0u, ~0u);
      counts = 0;
      uint32_t n = 0;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const uint32_t k = (hit(v[x].x) >> 15) + (hit(v[x].y) >> 15) + (hit(v[x].z) >> 15) +
                           (hit(v[x].w) >> 15);
        const uint32_t both = (k + (k >> 16)) & 0xFu;  // up to eight
        counts |= both << (4 * x);
        n += both;
      }
      n = __reduce_add_sync(0xFFFFFFFFu, n);
      hits += n;
      last = b;
      if (b - b0 == lane) mine = n;
    }
    if (pass == 1) break;
    if (lane == 0) sh.warp_hits[warp] = hits;
    __syncthreads();
    const uint32_t theirs = lane < kWarps ? sh.warp_hits[lane] : 0u;
    before = __shfl_sync(0xFFFFFFFFu, warp_inclusive(theirs) - theirs, warp);
    if (r < before || r >= before + hits) return;
    // the batch (of the first 32 of the warp, which are all of a part below 1 M logits)
    const uint32_t inc = before + warp_inclusive(mine);
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, inc > r)) - 1;
    before = __shfl_sync(0xFFFFFFFFu, inc - mine, at);
    b = b0 + at;
    end = last == b ? b : b + 1;
  }
#pragma unroll 1
  for (int x = 0; x < kBatch; ++x) {
    const uint32_t k = counts >> (4 * x) & 0xFu;
    const uint32_t to = before + warp_inclusive(k);
    if (r < to && r >= to - k) {
      const int c = c0 + 32 * (kBatch * last + x) + lane;
      const int64_t i0 = static_cast<int64_t>(c) * 8 - mis;
      uint32_t left = r - (to - k);
      for (int64_t i = i0 < 0 ? 0 : i0; i < i0 + 8 && i < p.V; ++i)
        if ((row[i] & (mask & 0xFFFFu)) == bits && left-- == 0) {
          p.tokens[m] = static_cast<int32_t>(i);
          if (p.prob != nullptr) p.prob[m] = sh.find_prob;
        }
    }
    before = __shfl_sync(0xFFFFFFFFu, to, 31);
    if (before > r) return;
  }
}

// A row through all bins, by one CTA.  Leaves the counters zero.
__device__ __noinline__ void all_bins(const SampleArgs& p, Shared& sh, const uint16_t* row,
                                      int64_t m, int mis, const Settings& set) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kStep = kSlotSegs;  // segments at a time
  if (tid == 0) sh.all_first = kBinLast + 1;
  for (int s0 = 0; s0 < kSegs; s0 += kStep) {
    for (int i = tid; i < kSlots / 4; i += kThreads)
      reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    count_range(p, row, mis, 32 * s0, kSlots, sh.counts);
    __syncthreads();
    int first = kBinLast + 1;
    for (int i = kSlots - 1 - tid; i >= 0; i -= kThreads)
      if (sh.counts[i] != 0) first = 32 * s0 + i;
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    if (lane == 0) atomicMin(&sh.all_first, first);
    __syncthreads();
    for (int s = warp; s < kStep && s0 + s < kSegs; s += kWarps) {
      uint32_t n = sh.counts[32 * s + lane];
      uint64_t w = n != 0 ? n * weight_of(sh, 32 * (s0 + s) + lane, sh.all_first) : 0;
      warp_sums(n, w);
      if (lane == 0) {
        sh.number[s0 + s] = n;
        sh.mass[s0 + s] = w;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < kSlots / 4; i += kThreads)
    reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
  // the segments that are not empty, closed up
  if (warp == 0) {
    int at = 0;
    for (int s = lane; s < kSegs; s += 32) {
      const uint32_t n = sh.number[s];
      const uint64_t w = sh.mass[s];
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, n != 0);
      if (n != 0) {
        const int to = at + __popc(live & ((1u << lane) - 1u));
        sh.number[to] = n;
        sh.mass[to] = w;
        sh.list[to] = static_cast<uint16_t>(s);
      }
      at += __popc(live);
      __syncwarp();
    }
    if (lane == 0) {
      sh.n_list = at;
      sh.find_bin = -1;
    }
  }
  __syncthreads();
  const Recount source{p, sh, row, mis};
  if (warp == 0) {
    int bin;
    uint32_t rank;
    float prob;
    const bool any =
        choose(p, sh, source, set, sh.n_list, sh.all_first, &bin, &rank, &prob);
    if (lane == 0) {
      if (any) {
        sh.find_bin = bin;
        sh.find_rank = rank;
        sh.find_prob = prob;
      } else {
        p.tokens[m] = -1;
        if (p.prob != nullptr) p.prob[m] = 0.f;
      }
    }
    source.done();
  } else {
    source.serve();
  }
  __syncthreads();
  if (sh.find_bin >= 0) find(p, sh, row, m, mis, 0, static_cast<int>((p.V + mis + 7) >> 3));
  __syncthreads();
}

template <int C>
__global__ void __launch_bounds__(kThreads, kCtas) sample_kernel(const SampleArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const auto meet = [&] {
    if constexpr (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  const auto peer = [&](int r) { return C == 1 ? &sh : cluster.map_shared_rank(&sh, r); };

  for (int i = tid; i < kSlots / 4; i += kThreads)
    reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = tid; i < 8 * kMasks; i += kThreads) sh.flags[i] = 0;
  if (tid < 64) {
    sh.pow2_hi[tid] = kPow2.hi[tid];
    sh.pow2_lo[tid] = kPow2.lo[tid];
  }
  griddep_wait();
  griddep_launch_dependents();
  Counters<C> source;
#pragma unroll
  for (int r = 0; r < C; ++r) source.counts[r] = peer(r)->counts;

  for (int64_t m = blockIdx.x / C; m < p.M; m += gridDim.x / C) {
    const uint16_t* row = p.logits + m * p.stride;
    Settings set;
    set.t = p.temperature != nullptr ? p.temperature[m] : 1.f;
    set.u = p.u[m];
    set.k = p.top_k != nullptr ? p.top_k[m] : 0;
    set.top_p = p.top_p != nullptr ? p.top_p[m] : 1.f;
    set.min_p = p.min_p != nullptr ? p.min_p[m] : 0.f;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 7);
    const int chunks = static_cast<int>((p.V + mis + 7) >> 3);
    const int per = (chunks + C - 1) / C;
    const int c0 = rank * per < chunks ? rank * per : chunks;
    const int c1 = c0 + per < chunks ? c0 + per : chunks;
    constexpr int kUnroll = 4;
    uint4 v[kUnroll];
    const auto load = [&](int c) {
#pragma unroll
      for (int x = 0; x < kUnroll; ++x)
        v[x] = c + x * kThreads < c1 ? load_chunk(row, p.V, mis, c + x * kThreads)
                                     : make_uint4(~0u, ~0u, ~0u, ~0u);
    };
    load(c0 + tid);
    if (tid == 0) {
      sh.wide = 0;
      // the cluster's next row on its way to the L2 cache
      const int64_t next = m + gridDim.x / C;
      if (next < p.M && c1 - c0 > 2)
        prefetch_l2(reinterpret_cast<const void*>(
                        (reinterpret_cast<uintptr_t>(p.logits + next * p.stride) & ~15ull) +
                        16 * static_cast<int64_t>(c0 + 1)),
                    16u * static_cast<uint32_t>(c1 - c0 - 2));
    } else if (tid == 32) {  // 2·log2(e)/T, and what its rounding left
      constexpr double a = 2.8853900817779268;
      constexpr float ah = static_cast<float>(a), al = static_cast<float>(a - static_cast<double>(ah));
      const bool hot = set.t > 0x1p64f;  // both sides smaller, or the quotient has no bits left
      const float t = hot ? set.t * 0x1p-64f : set.t;
      const float hi = ah / t;
      sh.half = hot ? 0x1p-65f : 0.5f;
      sh.c_hi = hi;
      sh.c_lo = isinf(hi) || hi == 0.f ? 0.f : (__fmaf_rn(-hi, t, ah) + al) / t;
    }
    __syncthreads();  // the counts are zero, too

    // ---- counts of this CTA's part
    uint32_t least = 0x7FFF7FFFu;
    for (int c = c0 + tid; c - tid < c1; c += kUnroll * kThreads) {
      uint4 now[kUnroll];
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) now[x] = v[x];
      if (c - tid + kUnroll * kThreads < c1) load(c + kUnroll * kThreads);
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        count2(sh.counts, now[x].x, least);
        count2(sh.counts, now[x].y, least);
        count2(sh.counts, now[x].z, least);
        count2(sh.counts, now[x].w, least);
      }
    }
    {
      // (bits − 0x8001 below 0: a size, and one that is not counted)
      const int lo = static_cast<int16_t>(least & 0xFFFFu), hi = static_cast<int16_t>(least >> 16);
      const int bound = static_cast<int>(kLeastBits) - 0x8001;
      if (lo < bound || hi < bound) sh.wide = 1;
    }
    __syncthreads();
    if (tid == 0) {
      // −0 is 0; larger values than the counted ones, and NaN, are another matter
      sh.counts[kZeroSlot] += sh.counts[kNegSlot];
      if (sh.counts[0] != 0) sh.wide = 1;
      sh.far = sh.counts[kFarSlot] != 0;
      sh.counts[kNegSlot] = sh.counts[0] = sh.counts[kFarSlot] = 0;
    }
    __syncthreads();
    // ---- which segments hold anything: four at a time, eight lanes each
    for (int s = warp; s < kSlots / 128; s += kWarps) {
      const uint4 n = reinterpret_cast<const uint4*>(sh.counts)[s * 32 + lane];
      const uint32_t any = __ballot_sync(0xFFFFFFFFu, (n.x | n.y | n.z | n.w) != 0);
      if (lane == 0)
        sh.flags[s] = static_cast<uint8_t>((any & 0xFFu ? 1 : 0) | (any & 0xFF00u ? 2 : 0) |
                                           (any & 0xFF0000u ? 4 : 0) | (any >> 24 ? 8 : 0));
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t bits = 0;
      if (lane < kMasks) {
        const uint32_t* f = reinterpret_cast<const uint32_t*>(sh.flags) + 2 * lane;
        // a nibble of each byte
        const auto pack = [](uint32_t x) {
          x = (x | x >> 4) & 0x00FF00FFu;
          return (x | x >> 8) & 0xFFFFu;
        };
        bits = pack(f[0]) | pack(f[1]) << 16;
        sh.occupied[lane] = bits;
      }
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, bits != 0);
      int slot = kSlots;  // of the largest value of this part
      if (live != 0) {
        const int at = __ffs(live) - 1;
        const int seg = 32 * at + __ffs(__shfl_sync(0xFFFFFFFFu, bits, at)) - 1;
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, sh.counts[32 * seg + lane] != 0);
        slot = 32 * seg + __ffs(some) - 1;
      }
      if (lane == 0) sh.first = slot < kSlots ? bin_of_slot(slot) : kBinLast + 1;
    }
    meet();
    if (warp == 0) {
      int first = kBinLast + 1, any_wide = 0, any_far = 0;
      uint32_t w = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const Shared* o = peer(r);
        first = o->first < first ? o->first : first;
        any_wide |= o->wide;
        any_far |= o->far;
        if (lane < kMasks) w |= o->occupied[lane];
      }
      int n_list = 0;
#pragma unroll
      for (int i = 0; i < kMasks; ++i) {
        const uint32_t bits = __shfl_sync(0xFFFFFFFFu, w, i);
        if (bits >> lane & 1u)
          sh.list[n_list + __popc(bits & ((1u << lane) - 1u))] =
              static_cast<uint16_t>(32 * i + lane);
        n_list += __popc(bits);
      }
      __syncwarp();
      if (lane == 0) {
        sh.n_list = n_list;
        sh.all_first = first;
        // logits of −2^16 and below have no weight next to one 33·T above that
        sh.all_wide = any_wide != 0 ||
                      (any_far != 0 && !(first <= kBinLast && value_of(first) > 33.f * set.t - 65536.f));
        sh.find_bin = -1;
      }
    }
    __syncthreads();
    const int n_list = sh.n_list, first = sh.all_first;
    if (sh.all_wide != 0) {
      meet();  // the others' flags have been read
      if (rank == 0) all_bins(p, sh, row, m, mis, set);
      else
        for (int i = tid; i < kSlots / 4; i += kThreads)
          reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      continue;
    }

    // ---- the segments' numbers of tokens and weights, to the first CTA
    for (int j = rank * kWarps + warp; j < n_list; j += C * kWarps) {
      const int seg = sh.list[j];
      uint32_t n = source.get(seg);
      uint64_t w = n * weigh(sh, source.bin(seg, lane), first);
      warp_sums(n, w);
      if (lane == 0) {
        peer(0)->number[j] = n;
        peer(0)->mass[j] = w;
      }
    }
    meet();
    if (rank == 0 && warp == 0) {
      {
        int bin;
        uint32_t r;
        float prob;
        if (choose(p, sh, source, set, n_list, first, &bin, &r, &prob)) {
          // whose part holds the r-th token of that value
          const int slot = bin <= kPosBin + kSpan ? bin - kPosBin
                           : bin < 0x8000         ? kZeroSlot
                                                  : bin - kPosBin - kNegShift + kNegSlot;
          int owner = 0;
#pragma unroll
          for (int i = 0; i < C - 1; ++i) {
            const uint32_t c = source.counts[i][slot];
            if (owner == i && r >= c) {
              r -= c;
              ++owner;
            }
          }
          if (lane == 0) {
            Shared* o = peer(owner);
            o->find_bin = bin;
            o->find_rank = r;
            o->find_prob = prob;
          }
        } else if (lane == 0) {
          p.tokens[m] = -1;
          if (p.prob != nullptr) p.prob[m] = 0.f;
        }
      }
    }
    meet();
    for (int i = tid; i < kSlots / 4; i += kThreads)
      reinterpret_cast<uint4*>(sh.counts)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (sh.find_bin >= 0) find(p, sh, row, m, mis, c0, c1);
    __syncthreads();
  }
}

template <int C>
cudaError_t launch(const SampleArgs& p, int sms, cudaStream_t s) {
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
  const int64_t most = sms * kCtas >= C ? sms * kCtas / C : 1;
  const int64_t clusters = p.M < most ? p.M : most;
  return launch_pdl_cluster(sample_kernel<C>, dim3(static_cast<unsigned>(clusters * C)),
                            dim3(kThreads), C, sizeof(Shared), s, p);
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
  p.M = M;
  p.V = V;
  p.stride = row_stride;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.tokens = tokens;
  p.prob = prob;
  // CTAs per row: the number with which all rounds of rows take least.  A round takes about
  // 8 us, 3 more in clusters, 2 more where two CTAs share an SM, and 1 us for each 8000
  // logits of an SM (10000 in clusters: of their parts the second look takes one).  Clusters
  // do not fill the device: 0.85 of it, 0.75 with one CTA an SM.  Over 94 sizes (1 to 1000
  // rows of 5000 to 262144) the choice costs 0.9% more than the best number.  (us with 1, 2,
  // 4 and 8: 1 row of 128000 28.7 23.7 18.8 17.2; 38 of 32000 18.4 18.8 20.1 33.6; 64 of
  // 128000 31.0 27.1 25.8 40.9; 152 of 128000 33.3 35.2 79.1 135.4.)
  int c = 1;
  double best = 0;
  for (int n = 1; n <= bd::kMaxCluster; n *= 2) {
    const bool alone = n == 1;
    const int64_t room = static_cast<int64_t>((alone ? 1.0 : 0.85) * bd::kCtas * sms / n);
    const int64_t at_once = room > 1 ? room : 1;
    const int64_t rows = M < at_once ? M : at_once;
    const int share = rows * n <= (alone ? 1.0 : 0.75) * sms ? 1 : bd::kCtas;  // of an SM
    const double logits = static_cast<double>(share) * static_cast<double>(V) / n;
    const double time = static_cast<double>((M + at_once - 1) / at_once) *
                        (8.0 + (alone ? 0.0 : 3.0) + (share > 1 ? 2.0 : 0.0) +
                         logits / (alone ? 8e3 : 10e3));
    if (n == 1 || time < best) {
      c = n;
      best = time;
    }
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c == 1   ? bd::launch<1>(p, sms, s)
                        : c == 2 ? bd::launch<2>(p, sms, s)
                        : c == 4 ? bd::launch<4>(p, sms, s)
                                 : bd::launch<8>(p, sms, s);
  return e == cudaSuccess ? BD_OK : BD_ERR_CUDA;
}
