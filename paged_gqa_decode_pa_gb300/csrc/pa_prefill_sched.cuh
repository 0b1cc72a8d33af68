// pa_prefill_sched.cuh -- how pa_prefill deals its work to the persistent
// grid; the same code on host and device.
//
// An item is (sequence, kv head, group of T = tiles * floor(128 / G) tokens).
// It costs the number of keys that its last token sees, plus a charge
// (kPfItemCost), times a weight by how many tiles its rows fill.  Items are laid
// end to end (by sequence, kv head, group), and CTA c takes units [c * share,
// (c + 1) * share) of that line, its ends rounded down to 128-key tiles.  Costs
// are counted in keys, not tiles, so that the cost of a run of items is an
// arithmetic series: the position of any item follows in closed form, nothing
// is stored, and finding a share's first item takes about a microsecond (sums
// of rounded-up tile counts took up to twelve).
#pragma once

#include <stdint.h>

#include "pa_kernels.cuh"
#include "pagedgqa.h"

namespace pa {

// An item's charge besides its keys (fetching Q, draining the pipeline, writing
// the rows), in keys.  256, 320, 448: 43.6, 44.4, 45 us for rows that all
// see 700 to 2500 keys at d = 64, the same within 1% for prompts.
constexpr int kPfItemCost = 256;
// Units per key: where one tile of rows takes all of an item (d <= 128), less,
// since the two softmax warpgroups share its keys.  At d = 128, decode rows
// beside chunks, weights 2, 3, 3.5 and 4 of 4: 208, 151, 151.5, 152 us; d = 64,
// 3 and 4: 44.4 and 45.5 us.
constexpr int kPfUnits = 4, kPfUnitsOneTile = 3;
// The least share of a CTA, in units: below it, cutting an item costs more (a
// second state, the merge) than it saves; single tokens 640, 512, 384 keys:
// 19.7, 18.8, 18.1 us when measured (17.3 now).  (More than twice 128 keys, so
// that no share of an item but its first falls inside one tile.)
constexpr int kPfMinShare = 384 * kPfUnits;

struct PfArgs {
  const int32_t* cu_q;
  const int32_t* table;
  const int32_t* seqlens;
  const void* q;      // (d = 256; the other head dimensions fetch it by TMA)
  int64_t q_stride;
  const void* v;
  void* out;
  float* lse;
  float* ws_acc;   // [2 * grid][d / 4][rows][4] partial O
  float* ws_ml;    // [2 * grid][rows][2] (max, sum)
  int4* ws_desc;   // [grid][2] what the merge joins
  uint32_t* status;
  float qscale;    // |scale| log2(e), above 0
  int32_t negate;  // scale < 0
  int32_t causal;
  int32_t B, H, Hkv, G, bs, maxblk, P, total_q;
  int32_t tt;      // tokens of a 128-row tile
  int32_t T;       // tokens of an item
  int32_t one;     // units per key of an item whose rows fill one tile
};

// One sequence's rows and keys.  A span that is not one has no rows; a length
// that is none has no keys and its rows are NaN (bad).
struct PfSeq {
  int32_t q0, nq, len;
  int32_t whole, n_items;  // items with all T tokens; all items
  int32_t none;            // causal: leading whole items that see no key
  bool bad, bad_span;

  PA_HD void set(const PfArgs& a, int32_t c0, int32_t c1, int32_t n) {
    bad_span = c0 < 0 || c1 < c0 || c1 > a.total_q;
    q0 = c0;
    nq = bad_span ? 0 : c1 - c0;
    bad = n < 0 || (int64_t)n > (int64_t)a.maxblk * a.bs;
    len = bad ? 0 : n;
    whole = (int32_t)((uint32_t)nq / (uint32_t)a.T);
    n_items = whole + (whole * a.T < nq);
    none = len < nq ? (int32_t)((uint32_t)(nq - len) / (uint32_t)a.T) : 0;
  }
  // Keys that item i's last token sees.
  PA_HD int32_t keys(const PfArgs& a, int32_t i) const {
    const int32_t last = nq < (i + 1) * a.T ? nq : (i + 1) * a.T;
    if (!a.causal) return len;
    const int32_t k = len - nq + last;
    return k < 0 ? 0 : (k > len ? len : k);
  }
  // Units per key of item i.
  PA_HD int32_t weight(const PfArgs& a, int32_t i) const { return nq - i * a.T > a.tt && a.T > a.tt ? kPfUnits : a.one; }
  PA_HD int64_t cost(const PfArgs& a, int32_t i) const {
    return (int64_t)weight(a, i) * (keys(a, i) + kPfItemCost);  // keys <= 2^30
  }
};

// Cost of a sequence's first n items of one kv head.
PA_HD int64_t pf_cost_before(const PfArgs& a, const PfSeq& q, int32_t n) {
  const int64_t f = n < q.whole ? n : q.whole;
  int64_t sum = f * kPfItemCost;
  if (a.causal) {
    // item k - 1 < whole sees d + k T keys, none where that is negative
    const int32_t d = q.len - q.nq;
    const int64_t z = q.none < f ? q.none : f;
    sum += (f - z) * d + a.T * ((f * (f + 1) - z * (z + 1)) / 2);
  } else {
    sum += f * q.len;
  }
  sum *= a.T > a.tt ? kPfUnits : a.one;
  return n > f ? sum + q.cost(a, q.whole) : sum;  // the last item, which sees all keys
}

// Where a CTA's share begins.
struct PfStart {
  int64_t at, end;  // units on the line; at >= end: nothing to do
  int32_t b, j, i;  // sequence, kv head, item
  int64_t pos;      // units into the item
};

struct PfPiece {
  int32_t b, j, q0, nq, len, tok0;
  int32_t rows;    // packed rows of the item (above 128: two tiles)
  int32_t keys;    // the item's keys
  int32_t t0, t1;  // key tiles of this piece
  int32_t slot;    // partial state, or -1: the whole item
  bool bad;
};

PA_HD int32_t pf_load(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

PA_HD PfSeq pf_seq(const PfArgs& a, int32_t b) {
  PfSeq s;
  s.set(a, pf_load(a.cu_q + b), pf_load(a.cu_q + b + 1), pf_load(a.seqlens + b));
  return s;
}

PA_HD int64_t pf_seq_cost(const PfArgs& a, const PfSeq& s) {
  return (int64_t)a.Hkv * pf_cost_before(a, s, s.n_items);
}

// a / b for a >= 0, b > 0, mostly below 2^32 (a 64-bit division takes several
// times as long).
PA_HD int64_t pf_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

PA_HD int64_t pf_share(int64_t total, int grid) {
  const int64_t s = pf_div(total + grid - 1, grid);
  return s < kPfMinShare ? kPfMinShare : s;
}

// The item at unit `at`, which lies `rest` units past the start of sequence b.
PA_HD PfStart pf_locate(const PfArgs& a, int64_t at, int64_t end, int32_t b, int64_t rest) {
  PfSeq s = pf_seq(a, b);
  int64_t cost = pf_seq_cost(a, s);
  while (rest >= cost) {
    rest -= cost;
    s = pf_seq(a, ++b);
    cost = pf_seq_cost(a, s);
  }
  const int64_t head = pf_cost_before(a, s, s.n_items);
  const int32_t j = (int32_t)pf_div(rest, head);
  rest -= j * head;
  int32_t lo = 0, hi = s.n_items;  // the last item that begins at or before rest
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (pf_cost_before(a, s, mid) <= rest)
      lo = mid;
    else
      hi = mid;
  }
  return PfStart{at, end, b, j, lo, rest - pf_cost_before(a, s, lo)};
}

// The pieces of a CTA's share in order.  A piece is the part of one item
// inside the share: an item's units are its charge, then its keys, so a share
// that ends inside the charge or the first tile leaves the whole item to the
// next CTA, and what an item's end leaves is never empty.
struct PfIter {
  int64_t at, end, pos;
  int32_t b, j, i, cta;
  PfSeq s;

  PA_HD void init(const PfArgs& a, const PfStart& st, int c) {
    at = st.at;
    end = st.end;
    b = st.b;
    j = st.j;
    i = st.i;
    pos = st.pos;
    cta = c;
    if (at < end) s = pf_seq(a, b);
  }

  // On to the next item (an empty sequence has none).
  PA_HD void step(const PfArgs& a) {
    pos = 0;
    if (++i < s.n_items) return;
    i = 0;
    if (++j < a.Hkv) return;
    j = 0;
    if (at >= end) return;
    do {
      s = pf_seq(a, ++b);  // units are left, so a sequence with rows follows
    } while (s.nq == 0);
  }

  // The pieces of the item that the share has just ended in (it begins in this
  // share).
  PA_HD int32_t pieces_left(const PfArgs& a, int64_t share) const {
    const int64_t rest = s.cost(a, i) - pos;  // units past the share
    return 1 + (int32_t)pf_div(rest + share - 1, share);
  }

  PA_HD bool next(const PfArgs& a, PfPiece& p) {
    while (at < end) {
      const int64_t cost = s.cost(a, i), left = end - at;
      const int64_t stop = left < cost - pos ? pos + left : cost;
      const bool done = stop == cost;
      const int32_t w = s.weight(a, i);
      const int64_t k0 = pf_div(pos, w) - kPfItemCost, k1 = pf_div(stop, w) - kPfItemCost;
      const int32_t t0 = k0 > 0 ? (int32_t)(k0 / 128) : 0;
      const int32_t t1 = k1 > 0 ? (int32_t)((done ? k1 + 127 : k1) / 128) : 0;
      const bool any = done || t1 > 0;
      if (any) {
        p.b = b;
        p.j = j;
        p.q0 = s.q0;
        p.nq = s.nq;
        p.len = s.len;
        p.bad = s.bad;
        p.tok0 = i * a.T;
        p.rows = s.nq - p.tok0 > a.tt && a.T > a.tt ? 256 : 128;
        p.keys = s.keys(a, i);
        p.t0 = t0;
        p.t1 = t1;
        p.slot = t0 > 0 ? 2 * cta : (done ? -1 : 2 * cta + 1);
      }
      at += stop - pos;
      if (done)
        step(a);
      else
        pos = stop;
      if (any) return true;
    }
    return false;
  }
};

// What the merge must join: the item that starts in this CTA's share and runs
// on into the next CTAs' (the number of pieces it has), or x = -1.
struct PfCut {
  int32_t b, j, tok0, pieces;
};

PA_HD PfCut pf_cut(const PfArgs& a, PfIter it) {
  PfCut d = {-1, 0, 0, 0};
  PfPiece p;
  const int64_t share = it.end - it.at;  // a share that an item runs out of is whole
  while (it.next(a, p)) {
    if (p.slot == 2 * it.cta + 1) {
      d = PfCut{p.b, p.j, p.tok0, it.pieces_left(a, share)};
    }
  }
  return d;
}

#ifdef __CUDACC__

// Adds up all sequences' costs (thread t: a run of sequences), then the thread
// whose run holds the CTA's first unit finds the item.  CTA 0 reports bad
// lengths and spans.
template <int NT>
__device__ void pf_find_start(const PfArgs& a, int cta, int grid, long long* scan, PfStart* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const PfSeq s = pf_seq(a, b);
    if (cta == 0 && (s.bad_span || s.bad)) atomicOr(a.status, PA_STATUS_BAD_SEQLEN);
    mine += pf_seq_cost(a, s);
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) inc += scan[w];
    total += scan[w];
  }
  const int64_t share = pf_share(total, grid);
  const int64_t at = (int64_t)cta * share, end = min((int64_t)total, at + share);
  if (at >= end) {
    if (tid == 0) *out = PfStart{0, 0, 0, 0, 0, 0};
  } else if (at >= inc - mine && at < inc) {
    *out = pf_locate(a, at, end, b0, at - (inc - mine));
  }
  __syncthreads();
}

#endif  // __CUDACC__

}  // namespace pa
