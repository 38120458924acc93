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
// row's maximum has left the reference's range (kRescale).
//
// Tensor memory (512 columns): S/P of half h at 128·h, O of half h at 256 +
// 128·h.  Warps: 0-3 and 4-7 the halves' softmax and epilogue, 8 and 9 their
// MMA issuers, 10 and 11 the TMA producers of Q and K, and of V.  Q, K and V
// lie in shared memory in the 128-byte swizzle, 64 columns (128 bytes) of 128
// rows per 16 KB panel; K is the K-major B operand, V (keys x D as stored) the
// MN-major one.
//
// Pieces (the plan's list, longest first) are dealt to the CTAs as they come: a
// batch of 256 pieces of 1 to 20 blocks ended within 3% on all CTAs, where a
// fixed deal back and forth left a tail of 9%.
//
// Measured (64 query and 8 key heads of 128): a prompt of 8192 tokens 690 us,
// 1.59 PFLOP/s of the products that the mask leaves, with the tensor pipe busy
// 74% of the time and the SM clock held down by power; one of 2048 tokens 54.7
// us on repeated inputs, 59.7 on inputs that change, 1.26 and 1.15 PFLOP/s: 512 pieces of 1 to 16 blocks leave a CTA three
// or four changes of piece, a start of about 5 us and an uneven end.  A half's
// 128·128 powers take the multifunction units half as long as its products take
// the tensor core; the maximum, the scaling, the rounding and the moves to and
// from tensor memory fill most of the rest, which the other half's products
// cover.
#include <cstdint>

#include "attn_decode.cuh"

namespace bd {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;  // and the next one: a half each
constexpr int kTmaWarp = 10;  // K and Q; the next one V
constexpr int kPanel = kTileKeys * 128;  // 128 rows x 128 bytes
// 384 threads launch with 168 registers each; the two softmax warpgroups take
// 208 and leave 88 for the third: 2·208 + 88 = 3·168.
constexpr int kSoftmaxRegs = 208;
constexpr int kOtherRegs = 88;
// CTAs of the decode role: eight warps of 232, 2·232 + 40 = 3·168.
constexpr int kDecodeRegs = 232;
constexpr int kIdleRegs = 40;
constexpr uint32_t kTmemCols = 512;
constexpr int kPieceBytes = 64;

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kStageBytes = kPanels * kPanel;  // a K or V block
  static constexpr int kQBytes = 2 * kPanels * kPanel;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffKv = kQBytes;
  static constexpr int kOffOut = kOffKv + kStages * kStageBytes;  // 4 KB per softmax warp
  static constexpr int kOffBar = kOffOut + 8 * 4096;
  // q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], tail, drain[2],
  // turn[2], piece_full[2], piece_empty[2], kv_full[], kv_empty[]
  static constexpr int kBars = 21 + 2 * kStages;
  static constexpr int kOffMisc = (kOffBar + kBars * 8 + 15) / 16 * 16;
  static constexpr int kOffPiece = kOffMisc + 16;
  static constexpr int kSmem = kOffPiece + 2 * kPieceBytes + 1024;  // with slack for alignment
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack2_bf16(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2_rn(lo, hi);
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

// A piece as the roles read it from shared memory: kvh < 0 ends the work.
struct Piece {
  TileEntry e;
  int kvh, pad[3];
};
static_assert(sizeof(Piece) == kPieceBytes, "four 16-byte words");

// The CTA's pieces in turn, two slots of shared memory that the K producer
// fills (one piece ahead) and every other warp of the tile role empties.
struct Pieces {
  const Piece* slots;
  uint64_t *full, *empty;
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ bool take(TileEntry& e, int& kvh, const DevCtx& ctx,
                                       volatile int* abort) {
    if (!warp_wait(&full[slot], phase, ctx, abort)) return false;
    const int4* src = reinterpret_cast<const int4*>(slots + slot);
    const int4 x = src[0], y = src[1], z = src[2];
    e = TileEntry{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, 0, 0};
    kvh = slots[slot].kvh;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[slot]);
    if (++slot == 2) {
      slot = 0;
      phase ^= 1u;
    }
    return kvh >= 0;
  }
};
constexpr int kPieceReaders = 11;  // 8 softmax warps, 2 issuers, the V producer

// Blocks of half h in a piece: [b0, end), empty when end <= b0.
__device__ __forceinline__ int half_end(const TileEntry& e, int h, int half_tok) {
  const int last = (h + 1) * half_tok < e.n_tok ? (h + 1) * half_tok : e.n_tok;
  if (last <= h * half_tok) return e.b0;
  const int sees = e.causal < (1 << 30) ? e.tok0 + last - 1 + e.causal : e.k_hi;
  const int keys = (sees < e.k_hi ? sees : e.k_hi) - e.k_lo;
  const int nb = keys > 0 ? (keys + kTileKeys - 1) / kTileKeys : 0;
  return nb < e.b1 ? nb : e.b1;
}

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ TileMaps maps, const AttnArgs p) {
  using C = Cfg<D>;
  const CUtensorMap &tmap_q = maps.q, &tmap_k = maps.k, &tmap_v = maps.v;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* p_full = q_full + 6;
  uint64_t* o_full = q_full + 10;
  uint64_t* tail_bar = q_full + 12;
  uint64_t* drain_bar = q_full + 13;
  uint64_t* turn = q_full + 15;
  uint64_t* piece_full = q_full + 17;
  uint64_t* piece_empty = q_full + 19;
  uint64_t* kv_full = q_full + 21;
  Piece* piece_slots = reinterpret_cast<Piece*>(smem + C::kOffPiece);
  uint64_t* kv_empty = kv_full + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const bd_attention_batch& b = p.b;
  // (a value from lane 0 is known to be the same in all lanes)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int half_tok = p.L.half_tok, g = p.L.g;

  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&q_full[h], 1);
      mbar_init(&q_empty[h], 1);
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[2 * h], 4);
      mbar_init(&p_full[2 * h + 1], 4);
      mbar_init(&o_full[h], 1);
      mbar_init(&turn[h], 1);
      mbar_init(&piece_full[h], 1);
      mbar_init(&piece_empty[h], kPieceReaders);
    }
    mbar_init(tail_bar, 1);
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
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
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  griddep_wait();
  griddep_launch_dependents();

  const int n_tile = p.header()->t_ctas;
  if (static_cast<int>(blockIdx.x) >= n_tile) {
    // ============================================================ decode role
    __syncthreads();  // everyone has read the tensor-memory address
    attn_decode::init<D, RT, kTileDecodeWarps>(smem, warp, lane);
    __syncthreads();
    if (warp < kTileDecodeWarps) {
      reg_inc<kDecodeRegs>();
      attn_decode::run<D, RT, kTileDecodeWarps>(maps.dk, maps.dv, p, smem, warp, lane,
                                            static_cast<int>(blockIdx.x) - n_tile);
    } else {
      reg_dec<kIdleRegs>();
    }
  } else if (warp < 8) {
    // ============================================================ softmax
    reg_inc<kSoftmaxRegs>();
    const int h = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the half, and tensor-memory lane
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + 128u * h;
    const uint32_t t_o = tmem + lanes + 256u + 128u * h;
    const int row_tok = r / g, row_head = r - row_tok * g;
    uint32_t s_phase = 0, o_phase = 0;
    Pieces pieces{piece_slots, piece_full, piece_empty};
    TileEntry e;
    int kvh;
    bool ok = true;
    while (ok && pieces.take(e, kvh, p.ctx, abort)) {
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
        // Weights two at a time (paired fp32 operations: half the instructions),
        // relative to a reference that follows the row's maximum lazily.
        // (Forming the first weights with the reference as it stands, before the
        // block's maximum is known, and again where it moves, measured no faster
        // on long prompts and 3-5% slower on batches of short pieces.)
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
        uint64_t sum[2] = {0u, 0u};
        const auto weigh = [&](int c, uint64_t ref2) {
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
        };
        const auto done = [&](int part) {  // 64 keys' weights are written
          tmem_st_done();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * h + part]);
        };
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
        const uint64_t ref2 = pack2(-ref, -ref);
        weigh(0, ref2);
        weigh(1, ref2);
        done(0);
        weigh(2, ref2);
        weigh(3, ref2);
        done(1);
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
      const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN goes through)
      const uint64_t inv2 = pack2(inv, inv);
      const int row_at = i * b.n_q_heads + row_head;  // the row's head in the tile's tokens
      const int64_t tile_at = static_cast<int64_t>(e.tok0) * b.n_q_heads + kvh * g;
      const int64_t slot = static_cast<int64_t>(e.slot) * b.n_kv_heads + kvh;
      // (Code that runs once a piece: rolled to 64 columns for the instruction
      // cache, which are all read before the first is used; 16 at a time took 1.6%
      // longer on a 2048-token prompt, 2.5% on eight of 512.)
      uint8_t* mine = smem + C::kOffOut + warp * 4096;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[4][16];
        if (any) {
#pragma unroll
          for (int x = 0; x < 4; ++x) tmem_ld_x16(t_o + 64u * c + 16u * x, o[x]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 16; ++y) o[x][y] = 0u;
        }
        if (e.slot < 0) {
          // Through shared memory (swizzled), so that a store instruction covers
          // whole 128-byte lines of four rows: with a row per lane the 32 lines
          // of each store took 3 µs a piece.
#pragma unroll
          for (int x = 0; x < 8; ++x) {  // 8 columns
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int at = 8 * (x & 1) + 2 * y;
              w[y] = pack2_bf16(mul2(pack2(__uint_as_float(o[x >> 1][at]),
                                           __uint_as_float(o[x >> 1][at + 1])), inv2));
            }
            *reinterpret_cast<uint4*>(mine + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (live) {
          float4* dst = part_o(p.ws + p.L.w_t_o, slot, 2 * kHalfRows, D) + h * kHalfRows + r +
                        16 * c * 2 * kHalfRows;
#pragma unroll
          for (int x = 0; x < 16; ++x)
            dst[x * 2 * kHalfRows] = make_float4(
                __uint_as_float(o[x >> 2][4 * (x & 3)]), __uint_as_float(o[x >> 2][4 * (x & 3) + 1]),
                __uint_as_float(o[x >> 2][4 * (x & 3) + 2]), __uint_as_float(o[x >> 2][4 * (x & 3) + 3]));
        }
        __syncwarp();
        if (e.slot >= 0) continue;
        int at[8];
        uint4 v[8];
        const int chunk = lane & 7;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int row = 4 * x + (lane >> 3);
          at[x] = __shfl_sync(0xFFFFFFFFu, live ? row_at : -1, row);
          v[x] = *reinterpret_cast<const uint4*>(mine + row * 128 + ((chunk ^ (row & 7)) << 4));
        }
        uint16_t* dst = p.out + tile_at * D + 64 * c + 8 * chunk;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (at[x] >= 0) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(at[x]) * D) = v[x];
        __syncwarp();
      }
      if (live) {
        if (e.slot >= 0)
          part_ml(p.ws + p.L.w_t_ml, slot, 2 * kHalfRows)[h * kHalfRows + r] = make_float2(mref, l);
        else if (p.lse != nullptr)
          p.lse[tile_at + row_at] = l != 0.f ? (mref + log2f(l)) * kLn2 : -INFINITY;
      }
      tc_fence_before();  // O has been read before the next piece's first P is signalled
    }
  } else {
    reg_dec<kOtherRegs>();
    if (warp < kTmaWarp) {
      // ========================================================== MMA issuers
      // A warp per half, so that one half's waits do not hold up the other's
      // products, and a turn that they pass to and fro with each block's two
      // products.  Without it the halves' products interleave, their softmaxes
      // then run side by side on the same schedulers, and a block takes a
      // quarter longer (3450 cycles against 2810).  The whole warp walks the
      // pieces, which keeps descriptors and addresses in uniform registers, and
      // one elected lane issues: with a single-lane walk a product took about
      // 100 cycles to issue, against 64 to run.
      const int h = warp - kMmaWarp;
      const bool lead = elect_one();
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTileKeys);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescB_MN;
      const uint32_t kv_base = smem_addr(smem + C::kOffKv);
      const uint32_t t_s = tmem + 128u * h, t_o = tmem + 256u + 128u * h;
      const uint64_t qd =
          sdesc_k_sw128(smem_addr(smem) + static_cast<uint32_t>(h) * C::kStageBytes);
      uint32_t q_phase = 0, p_phase = 0, my_turn = h == 0 ? 1u : 0u;
      int stage = 0, v_stage = 1;      // of the current K, of the last block's V
      uint32_t phase = 0, v_phase = 0;
      bool ok = true, issued = false;
      Pieces pieces{piece_slots, piece_full, piece_empty};
      TileEntry e;
      int kvh;
      while (ok && pieces.take(e, kvh, p.ctx, abort)) {
        const int b0 = __shfl_sync(0xFFFFFFFFu, e.b0, 0), b1 = __shfl_sync(0xFFFFFFFFu, e.b1, 0);
        const int end = __shfl_sync(0xFFFFFFFFu, half_end(e, h, half_tok), 0);
        // keys from the last block on
        int left = __shfl_sync(0xFFFFFFFFu, e.k_hi - e.k_lo, 0) - b0 * kTileKeys + kTileKeys;
        if (end > b0) {
          ok = warp_wait(&q_full[h], q_phase, p.ctx, abort);
          q_phase ^= 1u;
        }
        for (int j = b0; ok; ++j) {
          const bool more = j < b1, back = j > b0;
          if (more) ok = warp_wait(&kv_full[stage], phase, p.ctx, abort);
          if (back) ok = ok && warp_wait(&kv_full[v_stage], v_phase, p.ctx, abort);
          if (back && j <= end) ok = ok && warp_wait(&p_full[2 * h], p_phase, p.ctx, abort);
          ok = ok && warp_wait(&turn[h], my_turn, p.ctx, abort);
          if (!ok) break;
          my_turn ^= 1u;
          if (back && j <= end) {  // O += P·V of block j − 1
            const uint64_t vd =
                sdesc_mn_sw128(kv_base + static_cast<uint32_t>(v_stage) * C::kStageBytes);
            const int steps = left >= kTileKeys ? kTileKeys / 16 : (left + 15) / 16;
            const uint32_t acc = j > b0 + 1 ? 1u : 0u;
            // the weights of the block's first 64 keys, then of the others
            tc_fence_after();
            issued = true;
            if (lead) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < steps)
                  mma_ts(t_o, t_s + 8u * k, vd + 128u * k, idesc_o, k > 0 ? 1u : acc);
            }
            if (!(ok = warp_wait(&p_full[2 * h + 1], p_phase, p.ctx, abort))) break;
            p_phase ^= 1u;
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int k = 4; k < 8; ++k)
                if (k < steps) mma_ts(t_o, t_s + 8u * k, vd + 128u * k, idesc_o, 1u);
              if (j == end) mma_commit(&o_full[h]);
            }
          }
          if (more && j < end) {  // S = Q·Kᵀ of block j
            const uint64_t kd =
                sdesc_k_sw128(kv_base + static_cast<uint32_t>(stage) * C::kStageBytes);
            tc_fence_after();
            issued = true;
            if (lead) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint64_t step = static_cast<uint64_t>((k >> 2) * (kPanel >> 4) + 2 * (k & 3));
                mma_ss(t_s, qd + step, kd + step, idesc_s, k > 0 ? 1u : 0u);
              }
              mma_commit(&s_full[h]);
              if (j == end - 1) mma_commit(&q_empty[h]);
            }
          }
          if (lead) {
            mbar_arrive(&turn[h ^ 1]);
            if (back) mma_commit(&kv_empty[v_stage]);
            if (more) mma_commit(&kv_empty[stage]);
          }
          if (!more) break;
          left -= kTileKeys;
          v_stage = stage + 1;
          v_phase = phase;
          stage += 2;
          if (stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (issued) {
        if (lead) mma_commit(&drain_bar[h]);
        mbar_wait(&drain_bar[h], 0, p.ctx, nullptr);
      }
      __syncwarp();
    } else {
      // ========================================================== TMA producers
      // K blocks (and the pieces' Q rows) go to the ring's even stages, V blocks
      // to the odd ones, by a warp each: with 16-token pages a block is 16
      // copies, and one warp for both took longer than the products.
      const bool is_v = warp != kTmaWarp;
      const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
      const int page_shift = 31 - __clz(b.page_size);
      // rows of the cache's tensor map fit 31 bits (checked on the host)
      const int cache_rows = static_cast<int>(b.n_pages * b.n_kv_heads * b.page_size);
      const int per = kTileKeys >> page_shift;  // pages per block, at most 8
      int fill = 0, stage = is_v ? 1 : 0;
      uint32_t phase = 1, q_phase[2] = {1, 1}, tail_phase = 0;
      bool ok = true;
      // The K producer also deals the pieces: the first by the CTA's index, then
      // the next of the list (longest first) once it has loaded all of the
      // current one, about two blocks before that ends.  (Drawn earlier, a CTA
      // with a long piece takes another long one.)  The counter starts at the
      // number of CTAs, set by the plan and again by the kernel that joins the
      // parts.
      const int n_pieces = p.header()->t_entries * b.n_kv_heads;
      int* counter = p.piece_counter();
      int put_slot = 0;
      uint32_t put_phase = 1;
      const auto read_piece = [&](int i, TileEntry& e, int& kvh) {
        kvh = -1;
        if (i >= n_pieces) return;
        const int q = static_cast<int>(static_cast<unsigned>(i) /
                                       static_cast<unsigned>(b.n_kv_heads));
        const int4* src = reinterpret_cast<const int4*>(p.entries() + q);
        const int4 x = __ldg(src), y = __ldg(src + 1), z = __ldg(src + 2);
        e = TileEntry{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, 0, 0};
        kvh = i - q * b.n_kv_heads;
      };
      const auto put = [&](const TileEntry& e, int kvh) {
        if (!warp_wait(&piece_empty[put_slot], put_phase, p.ctx, abort)) return false;
        if (lane == 0) {
          int4* dst = reinterpret_cast<int4*>(piece_slots + put_slot);
          dst[0] = make_int4(e.tok0, e.n_tok, e.seq, e.k_lo);
          dst[1] = make_int4(e.k_hi, e.causal, e.b0, e.b1);
          dst[2] = make_int4(e.slot, e.tail, 0, 0);
          piece_slots[put_slot].kvh = kvh;
          mbar_arrive(&piece_full[put_slot]);
        }
        __syncwarp();
        if (++put_slot == 2) {
          put_slot = 0;
          put_phase ^= 1u;
        }
        return true;
      };
      Pieces pieces{piece_slots, piece_full, piece_empty};
      TileEntry e, next_e;
      int kvh, next_kvh = -1;
      if (!is_v) {
        read_piece(static_cast<int>(blockIdx.x), next_e, next_kvh);
        ok = put(next_e, next_kvh);
      }
      while (ok) {
        if (is_v) {
          if (!pieces.take(e, kvh, p.ctx, abort)) break;
        } else {
          e = next_e;
          kvh = next_kvh;
          if (kvh < 0) break;
        }
        const int32_t* table = b.page_table + static_cast<int64_t>(e.seq) * b.table_stride;
        const auto page_of = [&](int j) {
          const int key = e.k_lo + j * kTileKeys + ((lane & 7) << page_shift);
          // not looked at before its block is loaded, a block later
          return (lane & 7) < per && key < e.k_hi && j < e.b1 ? table[key >> page_shift] : -1;
        };
        int page = page_of(e.b0);
        for (int j = e.b0; j < e.b1; ++j) {
          const int left = e.k_hi - e.k_lo - j * kTileKeys;
          const int n_pg = left >= kTileKeys ? per : (left + b.page_size - 1) >> page_shift;
          // keys of the block from which on values may be anything, or −1
          const int zero0 = is_v && e.tail && left <= kTileKeys && left % 16 != 0 ? left : -1;
          const int next = page_of(j + 1);
          if (!(ok = warp_wait(&kv_empty[stage], phase, p.ctx, abort))) break;
          uint8_t* dst = smem + C::kOffKv + stage * C::kStageBytes;
          uint64_t* bar = zero0 >= 0 ? tail_bar : &kv_full[stage];
          if (lane == 0)
            mbar_arrive_expect_tx(
                bar, static_cast<uint32_t>(n_pg * b.page_size * 128 * C::kPanels));
          __syncwarp();
          // lanes 0 .. panels · pages − 1 load a page's panel each
          const int pg = lane / C::kPanels, panel = lane % C::kPanels;
          const int id = __shfl_sync(0xFFFFFFFFu, page, pg & 7);
          if (pg < n_pg) {
            // a page outside the cache reads as zeros (rows past the tensor)
            const bool in = id >= 0 && id < b.n_pages;
            if (!in) record_error(p.ctx, kErrBounds);
            tma_load_3d(dst + panel * kPanel + pg * b.page_size * 128, map, bar, 0,
                        in ? (id * b.n_kv_heads + kvh) << page_shift : cache_rows, panel);
          }
          __syncwarp();
          if (zero0 >= 0) {
            // Zero weights do not cancel a NaN: the values past the last key
            // are cleared up to the end of their 16-key step.
            ok = warp_wait(tail_bar, tail_phase, p.ctx, abort);
            tail_phase ^= 1u;
            const int n = ((zero0 + 15) / 16 * 16 - zero0) * 8;
            for (int x = lane; x < n * C::kPanels; x += 32)
              *reinterpret_cast<uint4*>(dst + x / n * kPanel + zero0 * 128 + x % n * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[stage]);
          }
          ++fill;
          stage += 2;
          if (stage >= C::kStages) {
            stage -= C::kStages;
            phase ^= 1u;
          }
          if (!ok) break;
          if (j == e.b0) {
            // the halves' rows, each as soon as its last product has read it
            for (int h = 0; h < 2 && ok && !is_v; ++h) {
              if (half_end(e, h, half_tok) <= e.b0) continue;
              if (!(ok = warp_wait(&q_empty[h], q_phase[h], p.ctx, abort))) break;
              q_phase[h] ^= 1u;
              if (lane == 0) {
                mbar_arrive_expect_tx(&q_full[h],
                                      static_cast<uint32_t>(C::kPanels * half_tok * g * 128));
                for (int c = 0; c < C::kPanels; ++c)
                  tma_load_3d(smem + (h * C::kPanels + c) * kPanel, &tmap_q, &q_full[h], 64 * c,
                              kvh * g, e.tok0 + h * half_tok);
              }
              __syncwarp();
            }
            if (!ok) break;
          }
          page = next;
        }
        if (ok && !is_v) {
          int drawn = 0;
          if (lane == 0) drawn = atomicAdd(counter, 1);
          read_piece(__shfl_sync(0xFFFFFFFFu, drawn, 0), next_e, next_kvh);
          ok = put(next_e, next_kvh);
        }
      }
      // See every issued load land (bounded, also after an abort).
      if (lane == 0) {
        constexpr int kMine = C::kStages / 2;
        for (int f = fill > kMine ? fill - kMine : 0; f < fill; ++f)
          mbar_wait(&kv_full[2 * (f % kMine) + (is_v ? 1 : 0)],
                    static_cast<uint32_t>((f / kMine) & 1), p.ctx, nullptr);
        // q_phase[h] == 1: no load yet, or an even number; the last one's phase
        // is q_phase[h] in either case
        for (int h = 0; h < 2 && !is_v; ++h) mbar_wait(&q_full[h], q_phase[h], p.ctx, nullptr);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int RT>
cudaError_t launch(const AttnArgs& a, const TileMaps& maps, cudaStream_t s) {
  constexpr int kDecodeSmem = attn_decode::Cfg<D, RT, kTileDecodeWarps>::kSmem + 1024;
  constexpr int kSmem = Cfg<D>::kSmem > kDecodeSmem ? Cfg<D>::kSmem : kDecodeSmem;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(host_cache_mutex());
    if (!done[dev & 63]) {
      e = cudaFuncSetAttribute(attn_tile_kernel<D, RT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  return launch_pdl(attn_tile_kernel<D, RT>, dim3(a.L.t_ctas), dim3(kThreads), kSmem, s, maps, a);
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, const TileMaps& maps, cudaStream_t s) {
  if (a.b.head_dim == 128)
    return launch<128, 1>(a, maps, s);
  return a.L.d_rows == 16 ? launch<64, 1>(a, maps, s) : launch<64, 2>(a, maps, s);
}

}  // namespace bd
