// attn_tile.cu — attention of long query runs (prompts, and the rows of a
// whole group of sequences over their shared prefix) on the tensor cores.
//
// A tile is 256 query rows of one key head: two halves of 128 rows, each row a
// (token, query head) pair, so all query heads that share a key head use the
// same key block.  Per 128-key block and half, tcgen05.mma forms
//   S = Q·Kᵀ   (128 x 128, fp32, in tensor memory)
// a warpgroup turns it into weights P = 2^(scale·S − m), one row per thread
// (row maximum and sum need no exchange between threads), rounds them to bf16
// over S's tensor memory, and a second product adds
//   O += P·V   (128 x D, fp32, in tensor memory; P from tensor memory).
// The two halves take turns: while one half's warpgroup works on its weights,
// the tensor core runs the other half's products.  O is rescaled only when a
// row's maximum has grown by more than 2^8 since the last time.
//
// Tensor memory (512 columns): S/P of half h at 128·h, O of half h at 256 +
// 128·h.  Warps: 0-3 and 4-7 the halves' softmax and epilogue, 8 the MMA
// issuer, 9 the TMA producer (10, 11 idle).  Q, K and V lie in shared memory in
// the 128-byte swizzle, 64 columns (128 bytes) of 128 rows per 16 KB panel; K
// is the K-major B operand, V (keys x D as stored) the MN-major one.
//
// Pieces (plan.entries, longest first) are dealt to the CTAs back and forth,
// which evens out their lengths without a counter.
#include <cstdint>

#include "attention.cuh"

namespace bd {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kTmaWarp = 9;
constexpr int kPanel = kTileKeys * 128;  // 128 rows x 128 bytes
// 384 threads launch with 168 registers each; the two softmax warpgroups take
// 208 and leave 88 for the third: 2·208 + 88 = 3·168.
constexpr int kSoftmaxRegs = 208;
constexpr int kOtherRegs = 88;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kStageBytes = kPanels * kPanel;  // a K or V block
  static constexpr int kQBytes = 2 * kPanels * kPanel;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffKv = kQBytes;
  static constexpr int kOffBar = kOffKv + kStages * kStageBytes;
  // q_full, q_empty, s_full[2], p_full[2][2], o_full[2], tail, drain, kv_full[],
  // kv_empty[]
  static constexpr int kBars = 12 + 2 * kStages;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;  // with slack for alignment
};

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
// D (+)= A·Bᵀ with A and B in shared memory, and with A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_done() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Descriptor of a [keys][64] panel pair read as the MN-major operand (N = D
// along the 128-byte rows, K = keys): 64-element row groups one panel apart
// (leading offset), 8-key groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kPanel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kIdescB_MN = 1u << 16;  // instruction descriptor: B is MN-major

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 values in one 64-bit register and the paired operations on them.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
               : "=r"(p));
  return p != 0;
}
// Bounded wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                          volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ctx, abort));
}

// The pieces of one CTA in turn, each fetched while the one before it runs.
struct Pieces {
  const AttnArgs& p;
  int64_t n, k;
  TileEntry next;
  int next_h;
  bool has;
  __device__ __forceinline__ explicit Pieces(const AttnArgs& a)
      : p(a), n(static_cast<int64_t>(a.header()->t_entries) * a.b.n_kv_heads), k(0) {
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    const int64_t c = blockIdx.x, w = gridDim.x;
    const int64_t i = k * w + ((k & 1) ? w - 1 - c : c);
    has = i < n;
    if (has) {
      const int4* src = reinterpret_cast<const int4*>(p.entries() + i / p.b.n_kv_heads);
      const int4 x = __ldg(src), y = __ldg(src + 1), z = __ldg(src + 2);
      next = TileEntry{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, 0, 0};
      next_h = static_cast<int>(i % p.b.n_kv_heads);
    }
    ++k;
  }
  __device__ __forceinline__ bool take(TileEntry& e, int& h) {
    // later rounds hold shorter rows of pieces: once one is missing in an
    // even round none follows; a missing odd-round piece likewise
    if (!has) return false;
    e = next;
    h = next_h;
    fetch();
    return true;
  }
};

// Blocks of half h in a piece: [b0, end), empty when end <= b0.
__device__ __forceinline__ int half_end(const TileEntry& e, int h, int half_tok) {
  const int last = (h + 1) * half_tok < e.n_tok ? (h + 1) * half_tok : e.n_tok;
  if (last <= h * half_tok) return e.b0;
  const int sees = e.causal < (1 << 30) ? e.tok0 + last - 1 + e.causal : e.k_hi;
  const int keys = (sees < e.k_hi ? sees : e.k_hi) - e.k_lo;
  const int nb = keys > 0 ? (keys + kTileKeys - 1) / kTileKeys : 0;
  return nb < e.b1 ? nb : e.b1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmap_q,
                     const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const AttnArgs p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = q_full + 4;
  uint64_t* o_full = q_full + 8;
  uint64_t* tail_bar = q_full + 10;
  uint64_t* drain_bar = q_full + 11;
  uint64_t* kv_full = q_full + 12;
  uint64_t* kv_empty = kv_full + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const bd_attention_batch& b = p.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half_tok = p.L.half_tok, g = p.L.g;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[2 * h], 4);
      mbar_init(&p_full[2 * h + 1], 4);
      mbar_init(&o_full[h], 1);
    }
    mbar_init(tail_bar, 1);
    mbar_init(drain_bar, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp < 8) {
    // ============================================================ softmax
    reg_inc<kSoftmaxRegs>();
    const int h = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the half, and tensor-memory lane
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + 128u * h;
    const uint32_t t_o = tmem + lanes + 256u + 128u * h;
    const int row_tok = r / g, row_head = r - row_tok * g;
    uint32_t s_phase = 0, o_phase = 0;
    Pieces pieces(p);
    TileEntry e;
    int kvh;
    bool ok = true;
    while (ok && pieces.take(e, kvh)) {
      const int end = half_end(e, h, half_tok);
      const int i = h * half_tok + row_tok;                      // token of the tile
      const bool live = row_tok < half_tok && i < e.n_tok;       // a row that exists
      int limit = 0;                                             // keys of the tile it sees
      if (live) {
        const int sees = e.causal < (1 << 30) ? e.tok0 + i + e.causal : e.k_hi;
        limit = (sees < e.k_hi ? sees : e.k_hi) - e.k_lo;
      }
      float mref = -INFINITY, l = 0.f;
      for (int j = e.b0; j < end; ++j) {
        ok = warp_wait(&s_full[h], s_phase, p.ctx, abort);
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32u * c, s[c]);
        tmem_ld_wait();
        const int seen = limit - j * kTileKeys;
        if (__any_sync(0xFFFFFFFFu, seen < kTileKeys)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (32 * c + x >= seen) s[c][x] = 0xFF800000u;  // −inf
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
          for (int x = 2; x < 32; x += 2)
            top[c] = max3(top[c], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
        if (__any_sync(0xFFFFFFFFu, mx > mref + kRescale)) {
          const float mn = fmaxf(mref, mx);
          const float f = mn == -INFINITY ? 1.f : ex2(mref - mn);
          mref = mn;
          l *= f;
          if (j > e.b0) {
            // the product of block j − 1 is complete: S of block j was issued
            // after it by the same thread, and its commit has arrived
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_x16(t_o + 16u * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st_x16(t_o + 16u * c, o);
            }
          }
        }
        const float ref = mref == -INFINITY ? 0.f : mref;
        // weights two at a time: the row maximum and the sum are then half the
        // instructions of the scalar form
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), ref2 = pack2(-ref, -ref);
        uint64_t sum[2] = {0u, 0u};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float a, z;
            unpack2(fma2(pack2(__uint_as_float(s[c][2 * x]), __uint_as_float(s[c][2 * x + 1])),
                         scale2, ref2), a, z);
            a = ex2(a);
            z = ex2(z);
            sum[x & 1] = add2(sum[x & 1], pack2(a, z));
            // rounded to bf16, the tensor core's operand type: 2^-9 of each
            // weight, while l sums them unrounded
            w[x] = pack_bf16x2_rn(a, z);
          }
          tmem_st_x16(t_s + 16u * c, w);
          if (c & 1) {  // 64 keys' weights are written: their product may start
            tmem_st_done();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * h + (c >> 1)]);
          }
        }
        float l0, l1;
        unpack2(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
      }
      if (!ok) break;
      // ---- epilogue: the half's rows, final or as a partial result
      const bool any = end > e.b0;
      if (any) {
        ok = warp_wait(&o_full[h], o_phase, p.ctx, abort);
        if (!ok) break;
        o_phase ^= 1u;
        tc_fence_after();
      }
      const int64_t at = (static_cast<int64_t>(e.tok0) + i) * b.n_q_heads + kvh * g + row_head;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t slot = static_cast<int64_t>(e.slot) * b.n_kv_heads + kvh;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (any) {
          tmem_ld_32x32b_x32(t_o + 32u * c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0u;
        }
        if (live && e.slot < 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D) + 4 * c;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              v[y] = pack_bf16x2_rn(__uint_as_float(o[8 * x + 2 * y]) * inv,
                                    __uint_as_float(o[8 * x + 2 * y + 1]) * inv);
            dst[x] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        } else if (live) {
          float4* dst = part_o(p.ws + p.L.w_t_o, slot, 2 * kHalfRows, D) + h * kHalfRows + r;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            dst[(8 * c + x) * 2 * kHalfRows] =
                make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                            __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
        }
        __syncwarp();
      }
      if (live) {
        if (e.slot >= 0)
          part_ml(p.ws + p.L.w_t_ml, slot, 2 * kHalfRows)[h * kHalfRows + r] = make_float2(mref, l);
        else if (p.lse != nullptr)
          p.lse[at] = l > 0.f ? (mref + log2f(l)) * kLn2 : -INFINITY;
      }
      tc_fence_before();  // O has been read before the next piece's first P is signalled
    }
  } else {
    reg_dec<kOtherRegs>();
    if (warp == kMmaWarp) {
      // ========================================================== MMA issuer
      // The whole warp walks the pieces, so that descriptors and addresses stay
      // in uniform registers, and one elected lane issues: with a single-lane
      // walk each product took about 100 cycles to issue, against 64 to run.
      const bool lead = elect_one();
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTileKeys);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescB_MN;
      const uint32_t q_base = smem_addr(smem);
      const uint32_t kv_base = smem_addr(smem + C::kOffKv);
      uint32_t q_phase = 0, p_phase[2] = {0, 0};
      int64_t fill = 0;  // ring position of the current block's K
      bool ok = true, issued = false;
      const auto wait_fill = [&](int64_t f) {
        return warp_wait(&kv_full[f % C::kStages],
                         static_cast<uint32_t>((f / C::kStages) & 1), p.ctx, abort);
      };
      Pieces pieces(p);
      TileEntry e;
      int kvh;
      while (ok && pieces.take(e, kvh)) {
        const int end[2] = {half_end(e, 0, half_tok), half_end(e, 1, half_tok)};
        ok = warp_wait(q_full, q_phase, p.ctx, abort);
        q_phase ^= 1u;
        for (int j = e.b0; ok && j <= e.b1; ++j) {
          bool have_v = false, have_k = false;
          for (int h = 0; h < 2 && ok; ++h) {
            if (j > e.b0 && j - 1 < end[h]) {  // O += P·V of block j − 1
              if (!have_v) ok = wait_fill(fill - 1);
              have_v = true;
              ok = ok && warp_wait(&p_full[2 * h], p_phase[h], p.ctx, abort);
              if (!ok) break;
              tc_fence_after();
              const uint64_t vd =
                  sdesc_mn_sw128(kv_base + static_cast<uint32_t>((fill - 1) % C::kStages) *
                                               C::kStageBytes);
              const int left = e.k_hi - e.k_lo - (j - 1) * kTileKeys;
              const int steps = left >= kTileKeys ? kTileKeys / 16 : (left + 15) / 16;
              const uint32_t t_o = tmem + 256u + 128u * h, t_p = tmem + 128u * h;
              const uint32_t acc = j - 1 > e.b0 ? 1u : 0u;
              // the weights of the block's first 64 keys, then of the others
              if (lead) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (k < steps)
                    mma_ts(t_o, t_p + 8u * k, vd + 128u * k, idesc_o, k > 0 ? 1u : acc);
              }
              issued = true;
              ok = warp_wait(&p_full[2 * h + 1], p_phase[h], p.ctx, abort);
              if (!ok) break;
              p_phase[h] ^= 1u;
              tc_fence_after();
              if (lead) {
#pragma unroll
                for (int k = 4; k < 8; ++k)
                  if (k < steps) mma_ts(t_o, t_p + 8u * k, vd + 128u * k, idesc_o, 1u);
                if (j == end[h]) mma_commit(&o_full[h]);
              }
            }
            if (j < e.b1 && j < end[h]) {  // S = Q·Kᵀ of block j
              if (!have_k) ok = wait_fill(fill);
              have_k = true;
              if (!ok) break;
              tc_fence_after();
              const uint64_t qd = sdesc_k_sw128(q_base + static_cast<uint32_t>(h) * C::kStageBytes);
              const uint64_t kd = sdesc_k_sw128(
                  kv_base + static_cast<uint32_t>(fill % C::kStages) * C::kStageBytes);
              if (lead) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint64_t step =
                      static_cast<uint64_t>((k >> 2) * (kPanel >> 4) + 2 * (k & 3));
                  mma_ss(tmem + 128u * h, qd + step, kd + step, idesc_s, k > 0 ? 1u : 0u);
                }
              }
              issued = true;
              if (lead) mma_commit(&s_full[h]);
            }
          }
          if (!ok) break;
          if (lead) {
            if (j > e.b0) mma_commit(&kv_empty[(fill - 1) % C::kStages]);
            if (j < e.b1) mma_commit(&kv_empty[fill % C::kStages]);
            if (j == e.b1 - 1) mma_commit(q_empty);
          }
          if (j < e.b1) fill += 2;
        }
      }
      if (issued) {
        if (lead) mma_commit(drain_bar);
        mbar_wait(drain_bar, 0, p.ctx, nullptr);
      }
      __syncwarp();
    } else if (warp == kTmaWarp) {
      // ========================================================== TMA producer
      const int page_shift = 31 - __clz(b.page_size);
      const int64_t cache_rows = b.n_pages * b.n_kv_heads * b.page_size;
      int64_t fill = 0;
      uint32_t q_phase = 1, tail_phase = 0;
      int64_t q_loads = 0;
      bool ok = true;
      // One K or V block into the next stage: lanes 0 .. panels·pages − 1 load
      // a page's panel each.
      const auto load_block = [&](const CUtensorMap* map, int page, int n_pg, int kvh, int zero0) {
        const int s = static_cast<int>(fill % C::kStages);
        const uint32_t ph = static_cast<uint32_t>((fill / C::kStages) & 1);
        ok = warp_wait(&kv_empty[s], ph ^ 1u, p.ctx, abort);
        if (!ok) return;
        uint8_t* dst = smem + C::kOffKv + s * C::kStageBytes;
        uint64_t* bar = zero0 >= 0 ? tail_bar : &kv_full[s];
        if (lane == 0)
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n_pg * b.page_size * 128 * C::kPanels));
        __syncwarp();
        const int pg = lane / C::kPanels, panel = lane % C::kPanels;
        const int id = __shfl_sync(0xFFFFFFFFu, page, pg & 7);
        if (pg < n_pg) {
          const int64_t row =
              id < 0 ? cache_rows
                     : (static_cast<int64_t>(id) * b.n_kv_heads + kvh) * b.page_size;
          tma_load_3d(dst + panel * kPanel + pg * b.page_size * 128, map, bar, 0,
                      static_cast<int32_t>(row), panel);
        }
        if (zero0 >= 0) {
          // Values past the last key may be anything, and zero weights do not
          // cancel a NaN: clear them up to the end of their 16-key step.
          ok = warp_wait(tail_bar, tail_phase, p.ctx, abort);
          tail_phase ^= 1u;
          const int n = ((zero0 + 15) / 16 * 16 - zero0) * 8;
          for (int x = lane; x < n * C::kPanels; x += 32)
            *reinterpret_cast<uint4*>(dst + x / n * kPanel + zero0 * 128 + x % n * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[s]);
        }
        ++fill;
      };
      Pieces pieces(p);
      TileEntry e;
      int kvh;
      while (ok && pieces.take(e, kvh)) {
        const int32_t* table = b.page_table + static_cast<int64_t>(e.seq) * b.table_stride;
        const int per = kTileKeys >> page_shift;  // pages per block, at most 8
        const auto page_of = [&](int j) {
          const int key = e.k_lo + j * kTileKeys + ((lane & 7) << page_shift);
          int id = -1;
          if ((lane & 7) < per && key < e.k_hi && j < e.b1) {
            id = table[key >> page_shift];
            if (id < 0 || id >= b.n_pages) {
              record_error(p.ctx, kErrBounds);
              id = -1;
            }
          }
          return id;
        };
        int page = page_of(e.b0);
        ok = warp_wait(q_empty, q_phase, p.ctx, abort);
        q_phase ^= 1u;
        if (!ok) break;
        const int halves = e.n_tok > half_tok ? 2 : 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full,
                                static_cast<uint32_t>(halves * C::kPanels * half_tok * g * 128));
          for (int h = 0; h < halves; ++h)
            for (int c = 0; c < C::kPanels; ++c)
              tma_load_3d(smem + (h * C::kPanels + c) * kPanel, &tmap_q, q_full, 64 * c, kvh * g,
                          e.tok0 + h * half_tok);
        }
        ++q_loads;
        __syncwarp();
        for (int j = e.b0; j < e.b1 && ok; ++j) {
          const int left = e.k_hi - e.k_lo - j * kTileKeys;
          const int n_pg = left >= kTileKeys ? per : (left + b.page_size - 1) >> page_shift;
          const int next = page_of(j + 1);
          load_block(&tmap_k, page, n_pg, kvh, -1);
          if (!ok) break;
          load_block(&tmap_v, page, n_pg, kvh,
                     e.tail && left <= kTileKeys && left % 16 != 0 ? left : -1);
          page = next;
        }
      }
      // See every issued load land (bounded, also after an abort).
      if (lane == 0) {
        for (int64_t f = fill > C::kStages ? fill - C::kStages : 0; f < fill; ++f)
          mbar_wait(&kv_full[f % C::kStages], static_cast<uint32_t>((f / C::kStages) & 1), p.ctx,
                    nullptr);
        if (q_loads > 0)
          mbar_wait(q_full, static_cast<uint32_t>((q_loads - 1) & 1), p.ctx, nullptr);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tv, cudaStream_t s) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(attn_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Cfg<D>::kSmem);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  return launch_pdl(attn_tile_kernel<D>, dim3(a.L.t_ctas), dim3(kThreads), Cfg<D>::kSmem, s, tq,
                    tk, tv, a);
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t s) {
  return a.b.head_dim == 128 ? launch<128>(a, tq, tk, tv, s) : launch<64>(a, tq, tk, tv, s);
}

}  // namespace bd
