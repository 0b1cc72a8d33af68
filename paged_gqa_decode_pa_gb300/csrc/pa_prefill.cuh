// pa_prefill.cuh -- attention of a chunk of new tokens over the paged cache
// (pa_prefill) on the fifth-generation tensor cores.
//
// For query row i of a sequence (its token, one head), the keys t < lim_i:
//   x_t = scale * q . K_t,  out = sum_t 2^(y_t - m) V_t / sum_t 2^(y_t - m),
//   lse = ln sum_t e^(x_t),  with y = x * log2(e) and m a running maximum.
//
// Rows.  The n tokens and G heads of one kv head are packed token-major into
// tiles of 128 rows (floor(128 / G) tokens), so a K/V tile read once feeds all
// heads that share it.  An item is one kv head's tile pair (d <= 128) or tile
// (d = 256, where one accumulator fills half the tensor memory).
//
// Products.  Per step of 64 keys S[128 rows x 64 keys] = Q . K^T with Q and K
// K-major in shared memory (d = 256: Q in tensor memory); O[128 x d] += P . V
// with P in tensor memory, written over S in 16 bits by the softmax, and V as an
// MN-major operand straight from its TMA copy.  Every tile has two S buffers, so
// that the next step's scores run while this one's softmax does.  Warps 0-3 and
// 4-7 are the softmax of the two tiles, a thread per row: no reduction crosses
// threads.  Where an item's rows fill one tile only (d <= 128: single tokens,
// drafts, a chunk's last rows), the two warpgroups take its steps in turn, each
// with a maximum, a sum and an accumulator of its own, and join them at the
// piece's end, half of the dims each.
//
// Split.  The keys of all items are laid end to end, with a charge per item,
// and every CTA of the persistent grid takes an equal share
// (pa_prefill_sched.cuh).  An item cut by a share's end leaves fp32 partial
// states that pa_prefill_merge_kernel joins in a fixed order.
//
// Rounding.  Scores, maxima, sums and O stay in fp32; P is rounded to the
// storage type for the product (by at most 2^-8 or 2^-11 of a weight, the size
// of the output's own rounding; in fp16 a weight below 2^-14 by up to 2^-25, with
// the largest at 1 or more) while the sum takes the unrounded values.  The tensor
// core aligns the addends to the accumulator and cuts what lies below its last
// bit: a product below 2^-24 of it is lost in either type.  (So weights lifted by
// 2^7 in fp16, to keep small ones from rounding to 0, gave no better an output
// behind a first key of 2^25 times the others' weight, 3.4 10^-3 off for 131,072
// keys on one CTA, and prompts took 277 us for 269.)
//
// Measured on a GB300 (cuBLAS bf16 1911 TFLOP/s, copy 6768 GB/s): 4096 rows of
// 24 heads over 32,768 keys, d = 256, bf16: 2.4 ms, 1270 TFLOP/s (products at
// their rate, the copies of K and V from L2 bound it; long runs are also
// power-capped, cuBLAS then gives 1730).  Prompts of 2000 tokens, 64 heads, d =
// 128, fp16: 273 us, 960 TFLOP/s, tensor pipe 46% active, issue slots 43%: the
// hand-overs between scores, softmax and products bound it, and the pieces' starts
// and ends.  Steps of 128 keys, with one S buffer a tile and the tiles' products
// in turn, took 258 us there (265 with 64 then; looking V over for what is hidden
// took 8 more), but 158 us for decode rows beside chunks (152, and 6 for V), 47.5 for
// rows that all see 700 to 2500 keys at d = 64 (44) and 20.4 for single tokens
// (17.3).  Also slower: half of Q in tensor memory, with one S buffer and P
// beside it (276 us, and 167 for decode rows beside chunks); the next scores
// loaded before this step's weights are handed over (281, 160); all products
// issued by one warp (378: its waits and commits, about 700 cycles a step, bound
// it).  Drafts of a few tokens over contexts of up to 8192, 1.16 GB: 192 us, 6.0
// TB/s (ring of 8 units for 10: 201 us).
#pragma once

#include <type_traits>

#include "pa_kernels.cuh"
#include "pa_prefill_sched.cuh"
#include "pa_ptx.cuh"
#include "pagedgqa.h"

namespace pa {

constexpr int kPfThreads = 384;  // two softmax warpgroups; one with the TMA warp and an MMA warp per tile
// Registers: a softmax thread holds 64 scores of its row, their weights and its
// share of O's way out.  The block starts with 168 a thread (64,512); the split
// below sums to 63,488.
constexpr int kPfRegsSoftmax = 208, kPfRegsRest = 80;
static_assert(256 * kPfRegsSoftmax + 128 * kPfRegsRest <= kPfThreads * 168, "the split waits for registers forever");
constexpr uint32_t kPfChunk = 128u * 128u;  // [128 rows][64 dims], 128-byte swizzled
constexpr uint64_t kPfWaitNs = 2000000000ull;  // every wait is for a step or two of another role ...
// ... but the schedule's, which is for a whole piece: up to 2^30 keys, 2^24 steps of
// about a microsecond.  (It ends at once where another wait has given up.)
constexpr uint64_t kPfPieceWaitNs = 100000000000ull;
// The running maximum m need not be the maximum: any m gives the same output as
// long as no weight 2^(y - m) leaves its type's range.  Raising m rescales O, a
// round trip to tensor memory and a wait for the products under way.
//
// bf16, whose range is fp32's: the weights of 64 keys are computed with the m
// at hand, and only where their sum is above kPfLimit is m raised to the
// maximum and the weights computed again; no maximum stands between the scores
// and the weights (an exp-sum of 2^30 such sums stays finite).
//
// fp16, largest value 2^16: raises are frequent, so the step's maximum is taken
// first and m raised where it is passed by more than kPfSlack, once for all the
// step's keys (as in bf16, 4 prompts of 2000 tokens took 336 us for 260).
// (Setting m above the maximum, for more slack, rounds small weights among the
// subnormals: the error then passes the weights' half step.)
template <typename T>
constexpr bool kPfTracksMax = std::is_same<T, __half>::value;
constexpr float kPfSlack = 14.f;
constexpr float kPfLimit = 0x1p40f;

template <int D>
struct PfShape {
  static constexpr int kTiles = D == 256 ? 1 : 2;          // 128-row tiles of an item
  // Where Q lies.  At d = 256 in tensor memory: in shared memory its 64 KB leave
  // room for two and a half steps of K and V, and the score products read more
  // from there (Q again for every 64 keys) than it delivers; 4096 rows over
  // 32,768 keys took 2.6 ms.
  static constexpr bool kQInTmem = D == 256;
  // Keys of a step: with 64, two S buffers a tile fit beside O (and Q at d = 256),
  // and copies run ahead by several steps.
  static constexpr int kKeys = 64;
  // A ring unit is the K (or V) of a step: [8-row groups][64-dim chunks][8
  // rows][128 bytes], swizzled by 128 bytes.  One copy per page brings all
  // chunks, and the groups of a chunk lie at one stride, as the descriptors
  // want.
  static constexpr uint32_t kChunks = D / 64;
  static constexpr uint32_t kUnitBytes = 2u * kKeys * D;
  static constexpr int kRing = D == 64 ? 12 : (D == 128 ? 10 : 7);
  static constexpr uint32_t kTileBytes = 256u * D;         // Q of one tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kRingOff = kQInTmem ? 0 : kTiles * kTileBytes;
  static constexpr uint32_t kBars = kRingOff + kRing * kUnitBytes;
  static constexpr uint32_t kScan = kBars + 512;           // the prologue's scan and start; then the pieces' slots
  static constexpr uint32_t kPair = kScan + 256;            // (max, sum) of a row's two halves
  static constexpr uint32_t kSmem = kPair + (kTiles == 2 ? 1024 : 0) + 1024;    // and room to align the base
  static constexpr PA_HD uint32_t kS(int y, int x) { return (uint32_t)(kKeys * (2 * y + x)); }
  static constexpr uint32_t kQCols = 128;  // (d = 256) Q's columns, 16-bit dims two to a column
  static constexpr uint32_t kO(int y) { return 256u + (uint32_t)(D * y); }
};

// The steps of a piece (whose tiles are of 128 keys).
template <int D>
__device__ __forceinline__ int pf_steps(const PfPiece& pc) {
  constexpr int kKeys = PfShape<D>::kKeys;
  if (pc.t0 == pc.t1) return 0;
  return (min(pc.keys, pc.t1 * 128) - pc.t0 * 128 + kKeys - 1) / kKeys;
}

// Barrier offsets.
struct PfBars {
  static PA_HD uint32_t full(uint32_t s) { return 8u * s; }
  static PA_HD uint32_t empty(uint32_t s) { return 128u + 8u * s; }
  // Tile y's S buffer x is ready / holds P.
  static PA_HD uint32_t s_full(int y, int x) { return 256u + 8u * (2 * y + x); }
  static PA_HD uint32_t p_full(int y, int x) { return 288u + 8u * (2 * y + x); }
  // Tile y's product with V of a step is done.  A waiter at step i knows that
  // product i - 2 is done, S(i) having been issued after it, so i - 1's phase is
  // not mistaken.
  static PA_HD uint32_t pv_done(int y) { return 320u + 8u * y; }
  // All products of a piece's tile y are done (one phase a piece).
  static PA_HD uint32_t o_full(int y) { return 336u + 8u * y; }
  static constexpr uint32_t kQFull = 352, kQEmpty = 360, kDrain = 368;
  static constexpr uint32_t kTmem = 376, kAbort = 380;
  // (One-tile pieces) warpgroup y's (max, sum) is in shared memory, its products
  // done; it has read both accumulators.
  static PA_HD uint32_t pair_ready(int y) { return 384u + 8u * y; }
  static PA_HD uint32_t pair_read(int y) { return 400u + 8u * y; }
  // Not a barrier: see pf_softmax (what a later row alone sees).
  static constexpr uint32_t kMark = 488;
  // Piece slots: filled by the scheduling warp, read by all others.
  static PA_HD uint32_t piece_full(uint32_t s) { return 416u + 8u * s; }
  static PA_HD uint32_t piece_empty(uint32_t s) { return 448u + 8u * s; }
};

// The CTA's pieces, handed to every warp through slots in shared memory: one
// warp walks the schedule, whose divisions and 64-bit sums would otherwise stand
// in every role's code and registers.
constexpr uint32_t kPfSlots = 4;
static_assert(kPfSlots * sizeof(PfPiece) <= 256, "the pieces' slots take the prologue's scratch");

template <int D>
struct PfPieces {
  uint32_t bars, at;  // barriers, slots
  volatile int* abort;
  uint32_t n = 0;

  __device__ __forceinline__ PfPieces(uint32_t base, volatile int* flag)
      : bars(base + PfShape<D>::kBars), at(base + PfShape<D>::kScan), abort(flag) {}

  // The scheduling lane: the next piece, or b = -1 behind the last one.
  __device__ __forceinline__ bool put(const PfPiece& p) {
    const uint32_t s = n % kPfSlots;
    if (n >= kPfSlots &&
        !mbar_wait_bounded(bars + PfBars::piece_empty(s), (n / kPfSlots - 1) & 1u, abort, kPfPieceWaitNs))
      return false;
    const int32_t* src = reinterpret_cast<const int32_t*>(&p);
#pragma unroll
    for (uint32_t k = 0; k < sizeof(PfPiece) / 4; ++k) sts32(at + s * sizeof(PfPiece) + 4 * k, (uint32_t)src[k]);
    mbar_arrive(bars + PfBars::piece_full(s));
    ++n;
    return true;
  }
  // Every other warp (converged): the next piece, false behind the last one.
  __device__ __forceinline__ bool next(PfPiece& p) {
    const uint32_t s = n % kPfSlots;
    const bool ok = mbar_wait_bounded(bars + PfBars::piece_full(s), (n / kPfSlots) & 1u, abort, kPfWaitNs);
    if (!__all_sync(0xffffffffu, ok)) return false;
    int32_t* dst = reinterpret_cast<int32_t*>(&p);
#pragma unroll
    for (uint32_t k = 0; k < sizeof(PfPiece) / 4; ++k) dst[k] = (int32_t)lds32(at + s * sizeof(PfPiece) + 4 * k);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars + PfBars::piece_empty(s));
    ++n;
    return p.b >= 0;
  }
};

// Groups of products of one K range, issued by one elected thread of a
// converged warp (the same one every time): per 16-wide k-step one MMA, the
// descriptors' address fields stepping as the operands' layouts do.  The whole
// warp runs the code, so that descriptors stay in uniform registers: one
// thread of a diverged warp took about 120 cycles to issue an MMA that runs
// for 64.

// D (+)= A[smem] . B[smem], both K-major: 4 k-steps of 32 bytes per 64-wide
// chunk, kPfChunk bytes between chunks.
#define PA_MMA_SS(step, pred) "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " pred ";\n\t" step
#define PA_STEP_SS(n) "add.s64 a, a, " n "; add.s64 b, b, " n ";\n\t"
__device__ __forceinline__ void umma_ss_4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 a, %1;\n\tmov.b64 b, %2;\n\t" PA_MMA_SS(PA_STEP_SS("2"), "p") PA_MMA_SS(PA_STEP_SS("2"), "t")
          PA_MMA_SS(PA_STEP_SS("2"), "t") PA_MMA_SS("", "t") "}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc));
}

// D (+)= A[tmem] . B[smem], 64 keys: A's rows are the lanes, its 16-bit
// elements packed two to a column (8 columns a step); B is MN-major, kStep
// 16-byte units a step.
#define PA_MMA_TS(step, pred) "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, " pred ";\n\t" step
#define PA_STEP_TS "add.u32 a, a, 8; add.s64 b, b, %5;\n\t"
template <int kStep>
__device__ __forceinline__ void umma_ts_4(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b32 a, %1;\n\tmov.b64 b, %2;\n\t" PA_MMA_TS(PA_STEP_TS, "p") PA_MMA_TS(PA_STEP_TS, "t")
          PA_MMA_TS(PA_STEP_TS, "t") PA_MMA_TS("", "t") "}" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(acc), "n"(kStep));
}

// An arrival by the thread that issues the products, after what it issued.
__device__ __forceinline__ void arrive_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// The elected thread's products so far arrive on `bar` when they are done.
__device__ __forceinline__ void umma_commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d_keep(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

#define PA_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define PA_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])

// 32 consecutive columns of this thread's lane; complete after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : PA_R4(r, 0), PA_R4(r, 4), PA_R4(r, 8), PA_R4(r, 12), PA_R4(r, 16), PA_R4(r, 20), PA_R4(r, 24), PA_R4(r, 28)
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::PA_W4(r, 0),
      PA_W4(r, 4), PA_W4(r, 8), PA_W4(r, 12), PA_W4(r, 16), PA_W4(r, 20), PA_W4(r, 24), PA_W4(r, 28), "r"(taddr)
      : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ TMA warp

// Walks the CTA's pieces: the Q tiles of each, then K and V of its key tiles,
// unit by unit into the ring, a lane per page.  (One copy per page and 64-dim
// chunk was as slow as the tensor cores allow at 16 rows a page.)  Pages past
// the item's keys, and table entries that are no block, are fetched from
// beyond the pool: the copy fills zeros, and the expected bytes stay the same.
template <int D>
__device__ __forceinline__ void pf_producer(const PfArgs& a, PfPieces<D> it, const CUtensorMap* tmq, const CUtensorMap* tmk,
                                            const CUtensorMap* tmv, uint32_t base, volatile int* abort) {
  using S = PfShape<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t bars = base + S::kBars;
  const int bpt = S::kKeys / a.bs;  // pages of a step, a lane each
  const bool copies = lane < bpt;
  uint32_t u = 0, piece = 0;
  bool ok = true;
  PfPiece pc;
  // Table entries are read 32 at a time, a lane each, a batch ahead: one by one,
  // every step waited for one from memory.
  const int per = 32 / bpt;  // steps of a batch
  auto pages = [&](int batch) {
    const int32_t col = (pc.t0 * 128 + batch * per * S::kKeys) / a.bs + lane;
    if (col * a.bs >= min(pc.keys, pc.t1 * 128)) return a.P;  // none: one past the pool
    const int32_t phys = __ldg(a.table + (int64_t)pc.b * a.maxblk + col);
    return phys < 0 || phys >= a.P ? INT32_MAX : phys;
  };
  // the K or V of one step of kv head pc.j into the ring
  auto fetch = [&](const CUtensorMap* map, int32_t phys) {
    const uint32_t s = u % S::kRing;
    if (u >= (uint32_t)S::kRing &&
        !__all_sync(0xffffffffu,
                    mbar_wait_bounded(bars + PfBars::empty(s), ((u / S::kRing) - 1) & 1u, abort, kPfWaitNs)))
      return false;
    ++u;
    const uint32_t full = bars + PfBars::full(s);
    if (lane == 0) mbar_arrive_expect_tx(full, S::kUnitBytes);
    __syncwarp();
    if (copies)
      tma_load_5d_keep(base + S::kRingOff + s * S::kUnitBytes + (uint32_t)(lane * a.bs) * 128u * S::kChunks, map, full,
                       0, 0, 0, 0, phys * a.bs * a.Hkv + pc.j);
    return true;
  };
  while (ok && it.next(pc)) {
    const int n = pf_steps<D>(pc);
    if (n == 0) continue;
    const int tiles = pc.rows > 128 ? 2 : 1;
    int32_t batch = pages(0), ahead = per < n ? pages(1) : a.P;
    for (int i = 0, in = 0; i < n && ok; ++i, ++in) {
      if (in == per) {
        in = 0;
        batch = ahead;
        ahead = i + per < n ? pages(i / per + 1) : a.P;
      }
      int32_t phys = __shfl_sync(0xffffffffu, batch, (in * bpt + lane) & 31);
      if (!copies) phys = a.P;
      if (phys == INT32_MAX) {
        atomicOr(a.status, PA_STATUS_BAD_BLOCK);
        phys = a.P;
      }
      ok = fetch(tmk, phys);
      if (!S::kQInTmem && i == 0) {
        // Q after the first K: its buffer is free only when the last piece's
        // scores are done, the ring sooner
        if (ok && piece > 0)
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(bars + PfBars::kQEmpty, (piece - 1) & 1u, abort, kPfWaitNs));
        if (!ok) break;
        ++piece;
        if (lane == 0) {
          const uint32_t box = (uint32_t)(a.G * a.tt) * 128u;
          mbar_arrive_expect_tx(bars + PfBars::kQFull, (uint32_t)tiles * (D / 64) * box);
          for (int y = 0; y < tiles; ++y)
            for (int c = 0; c < D / 64; ++c)
              tma_load_5d_keep(base + S::kQ + y * S::kTileBytes + c * kPfChunk, tmq, bars + PfBars::kQFull, 0, c, 0,
                               pc.j, pc.q0 + pc.tok0 + y * a.tt);
        }
        __syncwarp();
      }
      ok = ok && fetch(tmv, phys);
    }
  }
  // after a timeout, the copies in flight must land before the CTA leaves
  if (lane == 0) {
    volatile int never = 0;
    for (uint32_t k = u > (uint32_t)S::kRing ? u - S::kRing : 0; k < u; ++k)
      mbar_wait_bounded(bars + PfBars::full(k % S::kRing), (k / S::kRing) & 1u, &never, kPfWaitNs / 4);
    if (piece) mbar_wait_bounded(bars + PfBars::kQFull, (piece - 1) & 1u, &never, kPfWaitNs / 4);  // (0 without TMA's Q)
  }
}

// ------------------------------------------------------------------ MMA warps

// A warp per tile: one warp's chain of waits and issues for both tiles took
// longer than the products themselves.  A warp issues S of its next step, then
// P . V of the current one.  The tensor pipe runs one thread's products in the
// order of issue, so S may be written over P as soon as that P's product has been
// issued.  A ring unit is free when both warps say so.
template <typename T, int D>
struct PfMma {
  using S = PfShape<D>;
  static constexpr int bf = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  static constexpr uint32_t kIdS = idesc_f16(bf, 0, 0, 128, S::kKeys);
  static constexpr uint32_t kIdO = idesc_f16(bf, 0, 1, 128, D);  // V: dims run along N

  uint32_t base, bars, tmem;
  volatile int* abort;
  int y, qy;  // accumulator and S buffers; Q
  uint32_t id_s;

  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bars + bar, parity, abort, kPfWaitNs));
  }
  // The K or V in ring unit u has landed.
  __device__ __forceinline__ bool landed(uint32_t u) { return wait(PfBars::full(u % S::kRing), (u / S::kRing) & 1u); }
  // S[x] = Q[y] . K^T, K (landed) in ring unit u
  __device__ __forceinline__ void scores(int x, uint32_t u) {
    tc_fence_after();
    const uint32_t s = u % S::kRing;
    const uint64_t qd = sdesc_sw128(base + S::kQ + qy * S::kTileBytes, 16, 1024);
    const uint64_t kd = sdesc_sw128(base + S::kRingOff + s * S::kUnitBytes, 16, S::kChunks * 1024);
#pragma unroll
    for (uint32_t c = 0; c < S::kChunks; ++c) {
      if (S::kQInTmem)
        umma_ts_4<2>(tmem + S::kS(y, x), tmem + S::kQCols + 32 * c, kd + c * (1024 >> 4), id_s, c > 0);
      else
        umma_ss_4(tmem + S::kS(y, x), qd + c * (kPfChunk >> 4), kd + c * (1024 >> 4), id_s, c > 0);
    }
    umma_commit_elected(bars + PfBars::s_full(y, x));
    umma_commit_elected(bars + PfBars::empty(s));
  }
  // O[y] (+)= P[x] . V, V (landed) in ring unit u
  __device__ __forceinline__ void values(int x, uint32_t u, bool first) {
    tc_fence_after();
    const uint32_t s = u % S::kRing;
    const uint64_t vd = sdesc_sw128(base + S::kRingOff + s * S::kUnitBytes, 1024, S::kChunks * 1024);
    umma_ts_4<2 * S::kChunks * 1024 / 16>(tmem + S::kO(y), tmem + S::kS(y, x), vd, kIdO, !first);
    umma_commit_elected(bars + PfBars::empty(s));
    umma_commit_elected(bars + PfBars::pv_done(y));
  }
};

template <typename T, int D>
__device__ __forceinline__ void pf_mma(const PfArgs& a, PfPieces<D> it, int warp_y, uint32_t base, uint32_t tmem,
                                       volatile int* abort) {
  using S = PfShape<D>;
  PfMma<T, D> m;
  const int y = __reduce_max_sync(0xffffffffu, warp_y);
  m.y = y;
  m.id_s = PfMma<T, D>::kIdS | (a.negate ? 1u << 13 : 0u);  // negated Q: scale < 0
  m.base = base;
  m.bars = base + S::kBars;
  m.tmem = __reduce_max_sync(0xffffffffu, tmem);
  m.abort = abort;
  // the next piece that has keys (a reduction's result is known to be the same
  // in all lanes, so what follows from it can stay in uniform registers)
  int n = 0;
  bool two = false;
  auto fetch = [&]() {
    PfPiece pc;
    for (n = 0; n == 0;) {
      if (!it.next(pc)) return;
      n = __reduce_max_sync(0xffffffffu, pf_steps<D>(pc));
      two = __reduce_max_sync(0xffffffffu, pc.rows) > 128;
    }
  };
  uint32_t u = 0, piece = 0;
  uint32_t np0 = 0, np1 = 0;  // P's taken from the two buffers
  bool ok = true;
  fetch();
  while (ok && n > 0) {
    // step i's K is in ring unit u + 2 i, its V in the next
    auto ku = [&](int i) { return u + 2u * (uint32_t)i; };
    const bool split = S::kTiles == 2 && !two;
    m.qy = split ? 0 : y;
    // The other warp's step.  Waited for and released all the same: a warp that
    // left units out would lose count of their barriers' phases, which it tells
    // only modulo two.
    auto pass = [&](int i) {
      if (!m.landed(ku(i)) || !m.landed(ku(i) + 1)) return false;
      arrive_elected(m.bars + PfBars::empty(ku(i) % S::kRing));
      arrive_elected(m.bars + PfBars::empty((ku(i) + 1) % S::kRing));
      return true;
    };
    const int first = split ? y : 0, stride = split ? 2 : 1;
    ok = m.wait(PfBars::kQFull, piece & 1u) && (first == 0 || pass(0));
    if (ok && first < n) {
      ok = m.landed(ku(first));
      if (!ok) break;
      m.scores(0, ku(first));
      if (first + stride >= n) umma_commit_elected(m.bars + PfBars::kQEmpty);
      int x = 0;
      for (int i = first; i < n; i += stride, x ^= 1) {
        const int next = i + stride;
        if (split && i + 1 < n) ok = pass(i + 1);
        if (ok && next < n) {
          ok = m.landed(ku(next));
          if (!ok) break;
          m.scores(x ^ 1, ku(next));
          if (next + stride >= n) umma_commit_elected(m.bars + PfBars::kQEmpty);
        }
        const uint32_t v = ku(i) + 1, np = x ? np1++ : np0++;
        ok = ok && m.landed(v) && m.wait(PfBars::p_full(y, x), np & 1u);
        if (!ok) break;
        m.values(x, v, i == first);
        if (next >= n) umma_commit_elected(m.bars + PfBars::o_full(y));
      }
    } else if (ok) {
      arrive_elected(m.bars + PfBars::kQEmpty);
    }
    ++piece;
    u += 2u * (uint32_t)n;
    fetch();
  }
  // every product issued has completed before the tensor memory is released
  umma_commit_elected(m.bars + PfBars::kDrain);
  volatile int never = 0;
  mbar_wait_bounded(m.bars + PfBars::kDrain, 0, &never, kPfWaitNs / 4);
}

// ------------------------------------------------------------------ softmax

// The first key of the piece whose block is none (rows that see it are NaN), or
// past every key; the warp reads the piece's table entries together.
__device__ __forceinline__ int32_t pf_first_bad(const PfArgs& a, const PfPiece& pc) {
  const int32_t* row = a.table + (int64_t)pc.b * a.maxblk;
  const int32_t c0 = pc.t0 * (128 / a.bs), c1 = (min(pc.keys, pc.t1 * 128) + a.bs - 1) / a.bs;
  int32_t first = 0x7fffffff;
#pragma unroll 4
  for (int32_t col = c0 + (threadIdx.x & 31); col < c1; col += 32) {
    const int32_t phys = __ldg(row + col);
    if (phys < 0 || phys >= a.P) first = min(first, col * a.bs);
  }
  return __reduce_min_sync(0xffffffffu, first);
}

// All bits of those of two 16-bit values that are NaN or infinite.
template <typename T>
__device__ __forceinline__ uint32_t no_number(uint32_t x) {
  const uint32_t e = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpeq2(x & e, e);
}

// Warpgroup y, thread = row.
template <typename T, int D>
__device__ __forceinline__ void pf_softmax(const PfArgs& a, PfPieces<D> it, int y, uint32_t base, uint32_t tmem,
                                           volatile int* abort) {
  using S = PfShape<D>;
  constexpr int kKeys = S::kKeys;
  const int r = threadIdx.x & 127, warp = r >> 5, lane = r & 31;
  const uint32_t bars = base + S::kBars;
  const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
  const int rt = r / a.G, rg = r - rt * a.G;  // this row's token and head in its tile
  const float c = a.qscale;                   // |scale| log2(e), above 0 (Q's sign is turned in the product)
  const uint64_t c2 = pack2(c, c);
  uint32_t ns0 = 0, ns1 = 0, npv = 0, u = 0, done = 0, pieces = 0, pairs = 0;  // S's read so far from the two buffers; products
  PfPiece pc;
  while (it.next(pc)) {
    const bool two = pc.rows > 128;
    const int n = pf_steps<D>(pc);
    // one tile of rows: the warpgroups take its steps in turn, each with a
    // maximum, a sum and an accumulator of its own, joined at the end
    const bool split = S::kTiles == 2 && !two, pair = split && n > 1;
    const int first = split ? y : 0, stride = split ? 2 : 1;
    if (split && y == 1 && !pair) {  // nothing to do
      u += 2u * (uint32_t)n;
      continue;
    }
    const int tok = pc.tok0 + (two ? y * a.tt : 0) + rt;
    const bool row = rt < a.tt && tok < pc.nq;
    const int32_t lim = !row ? 0 : (a.causal ? max(0, min(pc.len, pc.len - pc.nq + tok + 1)) : pc.len);
    // Keys from here on are hidden from the item's first row, if from any.  A NaN or
    // an infinity that V holds there is turned to 0 before the product, where 0 * it
    // would reach the rows that do not see it, and added at the end to the rows that
    // do; kMark holds the last piece where one was found (maybe by the other
    // warpgroup).  V's ring unit serves both tiles, so both clear from the same key
    // on: were the second tile's warpgroup to leave the keys that all of its rows see,
    // the first one's stores would race with the second tile's product, and a weight
    // of 0 there give NaN or not by timing.
    const int32_t lim0 = a.causal ? max(0, min(pc.len, pc.len - pc.nq + pc.tok0 + 1)) : pc.len;
    const uint32_t mark = u + 2u;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (S::kQInTmem && n > 0) {
      // this thread's row of Q, once the last piece's scores are done
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (int64_t)(pc.q0 + tok) * a.q_stride +
                                                        ((int64_t)pc.j * a.G + rg) * D);
      if (pieces > 0) ok = mbar_wait_bounded(bars + PfBars::kQEmpty, (pieces - 1) & 1u, abort, kPfWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint4 v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = row ? __ldg(src + 16 * z + k) : make_uint4(0u, 0u, 0u, 0u);
        tmem_st32(lanes + S::kQCols + 64 * z, reinterpret_cast<const uint32_t*>(v));
        tmem_st32(lanes + S::kQCols + 64 * z + 32, reinterpret_cast<const uint32_t*>(v + 8));
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + PfBars::kQFull);
      ++pieces;
    }
#pragma unroll 1
    for (int i = first, x = 0; i < n; i += stride, x ^= 1) {
      const int32_t k0 = pc.t0 * 128 + i * kKeys;
      const uint32_t seen_s = x ? ns1++ : ns0++;
      ok = mbar_wait_bounded(bars + PfBars::s_full(y, x), seen_s & 1u, abort, kPfWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // rows past the keys inside the last block: 0 * (what lies there) must
      // be 0, so V is cleared there before the product reads it
      if (k0 + kKeys > lim0) {  // (lim0 <= pc.keys)
        const int h0 = max(lim0 - k0, 0), v0 = min(kKeys, pc.keys - k0);
        const int v1 = min(kKeys, (v0 + a.bs - 1) / a.bs * a.bs);
        if (h0 < v1) {
          // (V's ring unit was full and read before K's landed, so its barrier's
          // phase is not mistaken)
          const uint32_t vu = u + 2u * (uint32_t)i + 1u;
          if (!mbar_wait_bounded(bars + PfBars::full(vu % S::kRing), (vu / S::kRing) & 1u, abort, kPfWaitNs)) ok = false;
          const uint32_t at = base + S::kRingOff + (vu % S::kRing) * S::kUnitBytes;
          if (ok)
#pragma unroll 1  // (4: 284 us for 265 for prompts: code in the way of the loop's)
            for (int z = r; z < (v1 - h0) * (D / 8); z += 128) {
              const uint32_t k = h0 + z / (D / 8), w = z % (D / 8);  // key, 16 bytes of its row
              const uint32_t to = at + ((k >> 3) * S::kChunks + (w >> 3)) * 1024u + (k & 7) * 128u + (w & 7) * 16u;
              uint4 x = make_uint4(0u, 0u, 0u, 0u);
              if ((int)k < v0) {
                x = lds128(to);
                const uint32_t none = no_number<T>(x.x) | no_number<T>(x.y) | no_number<T>(x.z) | no_number<T>(x.w);
                if (!none) continue;
                asm volatile("red.relaxed.cta.shared::cta.max.u32 [%0], %1;" ::"r"(bars + PfBars::kMark), "r"(mark) : "memory");
                __threadfence_block();
                x.x &= ~no_number<T>(x.x);
                x.y &= ~no_number<T>(x.y);
                x.z &= ~no_number<T>(x.z);
                x.w &= ~no_number<T>(x.w);
              }
              sts128(to, x);
            }
          fence_proxy_async_smem();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
      }
      tc_fence_after();
      const bool some_hidden = !__all_sync(0xffffffffu, lim >= k0 + kKeys);
      // this row's scores, -infinity for keys that it does not see
      float s[64];
      tmem_ld32(lanes + S::kS(y, x), reinterpret_cast<uint32_t*>(s));
      tmem_ld32(lanes + S::kS(y, x) + 32, reinterpret_cast<uint32_t*>(s + 32));
      tmem_ld_wait();
      if (some_hidden) {
        const int32_t seen = lim - k0;
#pragma unroll
        for (int k = 0; k < 64; ++k) s[k] = k < seen ? s[k] : -INFINITY;
      }
      auto largest = [&]() {
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int k = 4; k < 60; k += 8) {
#pragma unroll
          for (int z = 0; z < 4; ++z) mx[z] = max3(mx[z], s[k + z], s[k + 4 + z]);
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) mx[z] = fmaxf(mx[z], s[60 + z]);
        return c * fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      };
      // m to mx where that is larger; O and the sum follow, O once the products
      // of the steps before are done
      auto raise_m = [&](float mx) {
        const float to = fmaxf(m, mx), al = to == -INFINITY ? 1.f : ex2(m - to);
        l *= al;
        m = to;
        if (i == first) return;
        if (!mbar_wait_bounded(bars + PfBars::pv_done(y), (npv - 1) & 1u, abort, kPfWaitNs)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        // (fp16, where it happens more often: 16, 32, 64 columns 267, 264, 269 us for
        // prompts)
        constexpr int kCols = kPfTracksMax<T> ? 32 : 16;
#pragma unroll 1
        for (int q = 0; q < D / kCols; ++q) {
          float o[kCols];
#pragma unroll
          for (int k = 0; k < kCols; k += 16) tmem_ld16(lanes + S::kO(y) + kCols * q + k, *reinterpret_cast<float(*)[16]>(o + k));
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < kCols; ++k) o[k] *= al;
#pragma unroll
          for (int k = 0; k < kCols; k += 16) tmem_st16(lanes + S::kO(y) + kCols * q + k, *reinterpret_cast<float(*)[16]>(o + k));
        }
      };
      uint32_t p[32];
      float sum;
      const float mx = kPfTracksMax<T> ? largest() : 0.f;
      // (bf16) a row's first keys set m
      bool raise = kPfTracksMax<T> ? __any_sync(0xffffffffu, mx > m + kPfSlack)
                                   : __any_sync(0xffffffffu, m == -INFINITY && lim > k0);
#pragma unroll 1
      for (bool checked = kPfTracksMax<T>;; checked = true) {
        if (raise) {
          raise_m(kPfTracksMax<T> ? mx : largest());
          if (!ok) break;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        const uint64_t nms2 = pack2(-ms, -ms);
        uint64_t l2[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float y0, y1;
          unpack2(fma2(pack2(s[2 * k], s[2 * k + 1]), c2, nms2), y0, y1);
          const float p0 = ex2(y0), p1 = ex2(y1);
          l2[k & 1] = add2(l2[k & 1], pack2(p0, p1));
          p[k] = Cvt<T>::pack(p0, p1);
        }
        float la, lb;
        unpack2(add2(l2[0], l2[1]), la, lb);
        sum = la + lb;
        raise = !checked && __any_sync(0xffffffffu, sum > kPfLimit);
        if (!raise) break;
      }
      if (!ok) break;
      l += sum;
      tmem_st32(lanes + S::kS(y, x), p);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + PfBars::p_full(y, x));
      ++npv;
    }
    u += 2u * (uint32_t)n;
    // the accumulated row (the pages are looked over while its product runs)
    const bool poison = pc.bad || lim > pf_first_bad(a, pc);
    if (ok && first < n) {
      ok = mbar_wait_bounded(bars + PfBars::o_full(y), done++ & 1u, abort, kPfWaitNs);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) return;
    tc_fence_after();
    if (poison) l = __int_as_float(0x7fc00000);
    float own = 1.f, others = 0.f;  // weights of this warpgroup's accumulator and the other's
    if (pair) {
      const uint32_t at = base + S::kPair + 8u * (uint32_t)r;
      // 1's through shared memory, then 0's in its place
      float mo = 0.f, lo = 0.f;
#pragma unroll
      for (int turn = 1; turn >= 0; --turn) {
        if (turn == y) {
          sts32(at, __float_as_uint(m));
          sts32(at + 4u, __float_as_uint(l));
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + PfBars::pair_ready(y));
        } else {
          ok = mbar_wait_bounded(bars + PfBars::pair_ready(1 - y), pairs & 1u, abort, kPfWaitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return;
          tc_fence_after();
          mo = __uint_as_float(lds32(at));
          lo = __uint_as_float(lds32(at + 4u));
        }
      }
      const float to = fmaxf(m, mo), ms = to == -INFINITY ? 0.f : to;
      own = ex2(m - ms);
      others = ex2(mo - ms);
      l = l * own + lo * others;
      m = to;
    }
    // a warpgroup writes its rows, or (pair) half of their dims
    const int q0 = pair ? y * (D / 64) : 0, q1 = pair ? q0 + D / 64 : D / 32;
    auto dims = [&](int q, float(&o)[32]) {
      tmem_ld32(lanes + S::kO(y) + 32 * q, reinterpret_cast<uint32_t*>(o));
      if (S::kTiles == 2 && pair) {
        float z[32];
        tmem_ld32(lanes + S::kO(1 - y) + 32 * q, reinterpret_cast<uint32_t*>(z));
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = o[k] * own + z[k] * others;
      } else {
        tmem_ld_wait();
      }
    };
    const int64_t orow = (int64_t)(pc.q0 + tok) * a.H + (int64_t)pc.j * a.G + rg;
    if (pc.slot < 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that saw nothing is 0
      // A thread holds 64 bytes of its row at a time; four lanes trade pieces
      // so that they store 64 bytes of one row together (16 bytes of 32 rows
      // per store took four times the cycles of the store unit).
      const int sub = lane & 3;
      int64_t drow[4];  // where the rows of this lane's group of four go, or -1
#pragma unroll
      for (int k = 0; k < 4; ++k) drow[k] = __shfl_sync(0xffffffffu, row ? orow : -1, (lane & ~3) + k);
#pragma unroll 1
      for (int q = q0; q < q1; ++q) {
        float o[32];
        if (n > 0) {
          dims(q, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        uint32_t p[4][4];
#pragma unroll
        for (int k = 0; k < 16; ++k) p[k >> 2][k & 3] = Cvt<T>::pack(o[2 * k] * inv, o[2 * k + 1] * inv);
        // after the two exchanges p[k] is piece `sub` of the group's row k
#pragma unroll
        for (int z = 0; z < 4; ++z) {
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, sub & 1 ? p[k][z] : p[k + 1][z], 1);
            if (sub & 1)
              p[k][z] = got;
            else
              p[k + 1][z] = got;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, sub & 2 ? p[k][z] : p[k + 2][z], 2);
            if (sub & 2)
              p[k][z] = got;
            else
              p[k + 2][z] = got;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (drow[k] >= 0)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + drow[k] * D + 32 * q + 8 * sub) =
                make_uint4(p[k][0], p[k][1], p[k][2], p[k][3]);
      }
      if (row && a.lse && q0 == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
    } else {
      // partial state, [d / 4][rows] so that a warp's stores are dense
      constexpr int kRows = 128 * S::kTiles;
      const int at = (two ? y * 128 : 0) + r;
      float4* acc = reinterpret_cast<float4*>(a.ws_acc) + (int64_t)pc.slot * (D / 4) * kRows + at;
#pragma unroll 1
      for (int q = q0; q < q1; ++q) {
        float o[32];
        dims(q, o);
        if (row) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            acc[(int64_t)(8 * q + k) * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (row && q0 == 0) reinterpret_cast<float2*>(a.ws_ml)[(int64_t)pc.slot * kRows + at] = make_float2(m, l);
    }
    tc_fence_before();
    uint32_t marked;
    asm volatile("ld.volatile.shared::cta.u32 %0, [%1];" : "=r"(marked) : "r"(bars + PfBars::kMark) : "memory");
    if (lim0 < pc.keys && marked >= mark) {
      // what was turned to 0, added to what was just written (loops rolled up: more
      // code here slows down all of the kernel)
      __syncwarp();
      const int32_t end = min(lim, min(pc.keys, pc.t1 * 128));
#pragma unroll 1
      for (int32_t t = max(lim0, pc.t0 * 128); t < end; ++t) {
        const int32_t phys = __ldg(a.table + (int64_t)pc.b * a.maxblk + t / a.bs);
        if (phys < 0 || phys >= a.P) continue;
        const uint16_t* v = static_cast<const uint16_t*>(a.v) + (((int64_t)phys * a.bs + t % a.bs) * a.Hkv + pc.j) * D;
#pragma unroll 1
        for (int e = 32 * q0; e < 32 * q1; ++e) {
          const uint16_t h = __ldg(v + e);
          if (!no_number<T>(h)) continue;
          const float x = Cvt<T>::widen(h);
          if (pc.slot < 0) {
            uint16_t* o = static_cast<uint16_t*>(a.out) + orow * D + e;
            *o = (uint16_t)Cvt<T>::pack(Cvt<T>::widen(*o) + x, 0.f);
          } else {
            a.ws_acc[(((int64_t)pc.slot * (D / 4) + e / 4) * (128 * S::kTiles) + (two ? y * 128 : 0) + r) * 4 + e % 4] += x;
          }
        }
      }
    }
    if (pair) {  // the next piece's products may be written over both accumulators
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + PfBars::pair_read(y));
      ok = mbar_wait_bounded(bars + PfBars::pair_read(1 - y), pairs++ & 1u, abort, kPfWaitNs);
      if (!__all_sync(0xffffffffu, ok)) return;
    }
  }
}

// ------------------------------------------------------------------ schedule

// One lane: the CTA's pieces in order, and what the merge must join.
template <int D>
__device__ __forceinline__ void pf_schedule(const PfArgs& a, PfIter walk, PfPieces<D> out) {
  int4 cut = make_int4(-1, 0, 0, 0), rows = cut;
  const int64_t share = walk.end - walk.at;  // a share that an item runs out of is whole
  PfPiece p;
  while (walk.next(a, p)) {
    if (p.slot == 2 * walk.cta + 1) {
      cut = make_int4(p.b, p.j, p.tok0, walk.pieces_left(a, share));
      rows = make_int4(p.q0, p.nq, 0, 0);
    }
    if (!out.put(p)) break;
  }
  p.b = -1;
  out.put(p);
  a.ws_desc[2 * walk.cta] = cut;
  a.ws_desc[2 * walk.cta + 1] = rows;
}

// ------------------------------------------------------------------ kernel

template <typename T, int D>
__global__ void __launch_bounds__(kPfThreads, 1)
    pa_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ PfArgs a) {
  using S = PfShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = base + S::kBars;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kBars + PfBars::kAbort);
  long long* scan = reinterpret_cast<long long*>(smem + S::kScan);
  PfStart* start = reinterpret_cast<PfStart*>(smem + S::kScan + 128);
  static_assert(kPfThreads / 32 * sizeof(long long) <= 128 && sizeof(PfStart) <= 128, "prologue scratch");
  if (tid == 0) {
    for (uint32_t s = 0; s < (uint32_t)S::kRing; ++s) {
      mbar_init(bars + PfBars::full(s), 1);
      mbar_init(bars + PfBars::empty(s), S::kTiles);  // an MMA warp each
    }
    for (int y = 0; y < 2; ++y) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(bars + PfBars::s_full(y, x), 1);
        mbar_init(bars + PfBars::p_full(y, x), 4);
      }
      mbar_init(bars + PfBars::pv_done(y), 1);
      mbar_init(bars + PfBars::o_full(y), 1);
      mbar_init(bars + PfBars::pair_ready(y), 4);
      mbar_init(bars + PfBars::pair_read(y), 4);
    }
    for (uint32_t s = 0; s < kPfSlots; ++s) {
      mbar_init(bars + PfBars::piece_full(s), 1);
      mbar_init(bars + PfBars::piece_empty(s), 4 * S::kTiles + 1 + S::kTiles);  // softmax, TMA and MMA warps
    }
    mbar_init(bars + PfBars::kQFull, S::kQInTmem ? 4 : 1);
    mbar_init(bars + PfBars::kQEmpty, S::kTiles);
    mbar_init(bars + PfBars::kDrain, S::kTiles);
    *abort = 0;
    *reinterpret_cast<volatile uint32_t*>(smem + S::kBars + PfBars::kMark) = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if (warp == 0) tmem_alloc(bars + PfBars::kTmem, 512);
  tc_fence_before();
  // a programmatic dependent of the kernel before it on the stream: nothing
  // above touches global memory
  asm volatile("griddepcontrol.wait;" ::: "memory");
  pf_find_start<kPfThreads>(a, (int)blockIdx.x, (int)gridDim.x, scan, start);  // ends in __syncthreads
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kBars + PfBars::kTmem);
  PfIter walk;
  walk.init(a, *start, (int)blockIdx.x);
  __syncthreads();  // the slots lie over the scratch that was just read
  const PfPieces<D> it(base, abort);
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 8) {
    regs_up<kPfRegsSoftmax>();
    if (S::kTiles == 2 || warp < 4) pf_softmax<T, D>(a, it, warp >> 2, base, tmem, abort);
  } else {
    regs_down<kPfRegsRest>();
    if (warp == 8) {
      pf_producer<D>(a, it, &tmq, &tmk, &tmv, base, abort);
    } else if (warp < 9 + S::kTiles) {
      pf_mma<T, D>(a, it, warp - 9, base, tmem, abort);
    } else if (warp == 11) {
      if (lane == 0) pf_schedule<D>(a, walk, it);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) atomicOr(a.status, PA_STATUS_TIMEOUT);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial states of the item that starts in split CTA blockIdx.x and
// runs on into later ones: out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p,
// pieces in order.  Block (cta, 32-row group): lane = row, a warp per 16 dims.
// Bound by latency: the loads of kPfMergeBatch pieces are in flight together
// (one piece after the other, the merge of 8-token steps took 10 us).
constexpr int kPfMergeBatch = 4;

template <typename T, int D>
__global__ void __launch_bounds__(2 * D) pa_prefill_merge_kernel(const PfArgs a) {
  constexpr int kRows = 128 * PfShape<D>::kTiles;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (sequence or -1, kv head, first token, pieces), (first row, rows)
  const int4 d = __ldcg(a.ws_desc + 2 * blockIdx.x), e = __ldcg(a.ws_desc + 2 * blockIdx.x + 1);
  if (d.x < 0) return;
  const int32_t q0 = e.x, nq = e.y;
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  const int y = r >> 7, rt = (r & 127) / a.G, rg = (r & 127) % a.G;
  const int tok = d.z + y * a.tt + rt;
  if (rt >= a.tt || tok >= nq) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + r;
  const float4* acc = reinterpret_cast<const float4*>(a.ws_acc) + (int64_t)(w * 4) * kRows + r;
  const int c0 = blockIdx.x;
  auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)); };
  float M = -INFINITY, l = 0.f;
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < d.w; p0 += kPfMergeBatch) {
    float2 s[kPfMergeBatch];
    float4 v[kPfMergeBatch][4];
#pragma unroll
    for (int p = 0; p < kPfMergeBatch; ++p) {
      const int64_t at = slot(min(p0 + p, d.w - 1));
      s[p] = __ldcg(&ml[at * kRows]);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[p][k] = __ldcg(&acc[(at * (D / 4) + k) * kRows]);
    }
    float to = M;  // the batch may repeat its last piece: its maximum counts once more
#pragma unroll
    for (int p = 0; p < kPfMergeBatch; ++p) to = fmaxf(to, s[p].x);
    const float base = to == -INFINITY ? 0.f : to, f0 = ex2(M - base);
    M = to;
    l *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[k].x *= f0;
      o[k].y *= f0;
      o[k].z *= f0;
      o[k].w *= f0;
    }
#pragma unroll
    for (int p = 0; p < kPfMergeBatch; ++p) {
      if (p0 + p >= d.w) break;
      const float f = ex2(s[p].x - base);
      l += s[p].y * f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k].x += v[p][k].x * f;
        o[k].y += v[p][k].y * f;
        o[k].z += v[p][k].z * f;
        o[k].w += v[p][k].w * f;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t orow = (int64_t)(q0 + tok) * a.H + (int64_t)d.y * a.G + rg;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + w * 16);
#pragma unroll
  for (int k = 0; k < 4; k += 2)
    dst[k / 2] = make_uint4(Cvt<T>::pack(o[k].x * inv, o[k].y * inv), Cvt<T>::pack(o[k].z * inv, o[k].w * inv),
                            Cvt<T>::pack(o[k + 1].x * inv, o[k + 1].y * inv),
                            Cvt<T>::pack(o[k + 1].z * inv, o[k + 1].w * inv));
  if (w == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.6931471805599453f;
}

template <typename T, int D>
const void* prefill_kernel_ptr() {
  return reinterpret_cast<const void*>(&pa_prefill_kernel<T, D>);
}

template <typename T, int D>
cudaError_t launch_prefill(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, const PfArgs& a,
                           int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = PfShape<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, pa_prefill_kernel<T, D>, tmq, tmk, tmv, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(grid, 4 * PfShape<D>::kTiles);
  cfg.blockDim = dim3(2 * D);  // a warp per 16 dims
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, pa_prefill_merge_kernel<T, D>, a);
}

}  // namespace pa

#define PA_INSTANTIATE_PREFILL(T, D)                                                                        \
  template const void* pa::prefill_kernel_ptr<T, D>();                                                     \
  template cudaError_t pa::launch_prefill<T, D>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, \
                                                const pa::PfArgs&, int, cudaStream_t);
