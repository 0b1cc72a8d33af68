// pa_step.cu -- the kernels of a serving step around the attention: block
// tables and slot maps from request lengths (pa_build_slots), the cache write
// of many new tokens by slot map (pa_cache_write), and the verification of
// drafted tokens (pa_verify_drafts).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pa_kernels.cuh"
#include "pa_ptx.cuh"
#include "pagedgqa.h"

namespace {

using namespace pa;

constexpr size_t kStatusBytes = 256;  // every workspace begins with the status word

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every kernel here is a programmatic dependent of the kernel before it on the
// stream: it is launched while that one runs, and waits for it before it
// touches memory (after_previous, the first thing it does).  Small steps, whose
// kernels take a few microseconds, otherwise pay a launch each.
template <class Args>
int launch(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------ slot maps

// With need_b = ceil((len_b + new_b) / bs) and h_b blocks held, sequence b
// gives back max(0, h_b - need_b) blocks and takes max(0, need_b - h_b).  The
// three running sums over the sequences (new rows, blocks given back, blocks
// taken) place every row, every push and every pop, so all of them are
// independent once the sums are known.
//
// Bound by latency (the lengths, a scan, a search, a table entry).  Every CTA
// adds up all sequences by itself, so no CTA waits for another, and deals its
// share of the rows, pushes and pops to its threads by binary search in the
// sums: a sequence with a thousand rows costs what a thousand sequences with
// one row cost.  A pop that falls on a block pushed in this call takes it from
// the pusher's table row, not from the stack.  The per-sequence outputs may be
// the inputs, so the last CTA to have read the inputs writes them.
// 4096 sequences, 507,000 rows: 17 us (88 us with one cluster of 8 CTAs); 8
// sequences, one row each: 3.4 us a call in a row of calls, 3.3 of them the
// host's.
constexpr int kSlotThreads = 1024;
constexpr int kSlotThreadsSmall = 256;
constexpr int kSlotRows = 2048;  // rows per CTA before another one joins
constexpr int kSlotMaxCtas = 152;  // one per SM
constexpr size_t kTicketOffset = 32;  // in the status word's 256 bytes; zero between calls

struct SlotArgs {
  const int32_t* seqlens;
  const int32_t* new_lens;
  const int32_t* held;
  int32_t* table;
  int32_t* free_list;
  const int32_t* free_count;
  int32_t* cu_q;
  int64_t* slots;
  int32_t* seqlens_out;
  int32_t* held_out;
  int32_t* free_count_out;
  uint32_t* status;
  uint32_t* ticket;
  int32_t B, maxblk, P, T;
  int32_t bs_log2;
};

struct Sums {
  long long rows, back, take;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return Sums{a.rows + b.rows, a.back + b.back, a.take + b.take};
}

__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, v.rows, d), __shfl_up_sync(0xffffffffu, v.back, d),
              __shfl_up_sync(0xffffffffu, v.take, d)};
}

// The last i in [0, n) with pre[i] <= x, for non-decreasing pre with pre[0] <= x.
__device__ __forceinline__ int owner(const int32_t* pre, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp31(long long x) { return (int32_t)min(x, (long long)INT32_MAX); }

// Shared memory of B sequences: running sums (exclusive, B + 1), lengths
// (negative: not served) and blocks held.
size_t slot_smem(int32_t B) { return sizeof(int32_t) * (3 * ((size_t)B + 1) + 2 * (size_t)B); }

template <int NT>
__global__ void __launch_bounds__(NT) pa_slots_kernel(const SlotArgs a) {
  after_previous();
  extern __shared__ int32_t slot_mem[];
  __shared__ Sums s_warp[NT / 32];
  __shared__ long long s_taken[NT / 32];
  __shared__ int s_last;
  const int B = a.B;
  int32_t* rows = slot_mem;       // [B + 1]
  int32_t* back = rows + B + 1;   // [B + 1]
  int32_t* take = back + B + 1;   // [B + 1]
  int32_t* lens = take + B + 1;   // [B]
  int32_t* held = lens + B;       // [B]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int bs = 1 << a.bs_log2;
  const int64_t cap = (int64_t)a.maxblk << a.bs_log2;
  int32_t count = *const_cast<const volatile int32_t*>(a.free_count);
  for (int b = tid; b < B; b += NT) {
    rows[b] = a.new_lens[b];
    lens[b] = a.seqlens[b];
    held[b] = a.held[b];
  }
  __syncthreads();
  // every input that an output may overwrite has been read
  if (ctas > 1) {
    __threadfence();
    if (tid == 0) s_last = atomicAdd(a.ticket, 1u) == (unsigned)ctas - 1;
  } else if (tid == 0) {
    s_last = 1;
  }
  uint32_t status = 0;
  if (count < 0 || count > a.P) status |= PA_STATUS_BAD_BLOCK;
  count = min(max(count, 0), a.P);
  // a run of sequences per thread
  const int per = (B + NT - 1) / NT, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto sequence = [&](int b, bool& bad, Sums& v) {
    const int32_t len = lens[b], add = rows[b], h = held[b];
    const int64_t end = (int64_t)len + add;
    bad = len < 0 || add < 0 || end > cap || h < 0 || h > a.maxblk || ((int64_t)len + bs - 1) >> a.bs_log2 > h;
    const int32_t need = bad ? h : (int32_t)((end + bs - 1) >> a.bs_log2);
    v = Sums{max(add, 0), max(0, h - need), max(0, need - h)};
  };
  Sums mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    bool bad;
    Sums v;
    sequence(b, bad, v);
    mine = mine + v;
  }
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(inc, d);
    if (lane >= d) inc = inc + o;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sums v = lane < NT / 32 ? s_warp[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(v, d);
      if (lane >= d) v = v + o;
    }
    if (lane < NT / 32) s_warp[lane] = v;
  }
  __syncthreads();
  const Sums all = s_warp[NT / 32 - 1], before = warp ? s_warp[warp - 1] : Sums{0, 0, 0};
  Sums run = {before.rows + inc.rows - mine.rows, before.back + inc.back - mine.back,
              before.take + inc.take - mine.take};
  const bool last = s_last != 0;
  if (count + all.back > a.P) status |= PA_STATUS_BAD_BLOCK;
  const long long top = min((long long)a.P, count + all.back);
  // a sequence is served while the stack lasts and its rows fit the slot map
  long long taken = 0;
  for (int b = b0; b < b1; ++b) {
    bool bad;
    Sums v;
    sequence(b, bad, v);
    const bool fits = v.rows == 0 || run.rows + v.rows <= a.T;
    const bool blocks = v.take == 0 || run.take + v.take <= top;
    const bool served = !bad && fits && blocks;
    if (bad || !fits)
      status |= PA_STATUS_BAD_SEQLEN;
    else if (!blocks)
      status |= PA_STATUS_NO_BLOCKS;
    if (served) taken += v.take;
    if (last) {
      const int32_t need = held[b] - (int32_t)v.back + (int32_t)v.take;
      a.cu_q[b] = (int32_t)min((long long)a.T, run.rows);
      a.seqlens_out[b] = served ? lens[b] + (int32_t)v.rows : lens[b];
      a.held_out[b] = served ? need : min(held[b], need);
    }
    rows[b] = clamp31(run.rows);
    back[b] = clamp31(run.back);
    take[b] = clamp31(run.take);
    if (!served) lens[b] = -1;
    run = run + v;
  }
  if (tid == 0) {
    rows[B] = clamp31(all.rows);
    back[B] = clamp31(all.back);
    take[B] = clamp31(all.take);
  }
  if (cta == 0 && status) atomicOr(a.status, status);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) taken += __shfl_xor_sync(0xffffffffu, taken, d);
  if (lane == 0) s_taken[warp] = taken;
  __syncthreads();
  if (last && tid == 0) {
    taken = 0;
    for (int w = 0; w < NT / 32; ++w) taken += s_taken[w];
    *a.free_count_out = (int32_t)(top - taken);
    a.cu_q[B] = (int32_t)min((long long)a.T, all.rows);
    if (ctas > 1) *a.ticket = 0;  // for the next call
  }
  // the x-th block that goes back
  auto pushed = [&](int32_t x) {
    const int b = owner(back, B, x);
    const int32_t need = held[b] - (back[b + 1] - back[b]);
    return a.table[(int64_t)b * a.maxblk + need + (x - back[b])];
  };
  // the x-th block that is taken, from the top of the stack
  auto popped = [&](int32_t x) {
    const long long at = top - 1 - x;
    return at >= count ? pushed((int32_t)(at - count)) : a.free_list[at];
  };
  const int at0 = cta * NT + tid, step = ctas * NT;
  bool bad_id = false;
  // pushes: given-back blocks go on top of the stack, by sequence and column; one
  // outside the pool is reported here, not when it is taken
  for (long long x = at0; x < top - count; x += step) {
    const int32_t id = pushed((int32_t)x);
    bad_id |= id < 0 || id >= a.P;
    a.free_list[count + x] = id;
  }
  // pops, by sequence and column
  for (long long x = at0; x < min(all.take, top); x += step) {
    const int b = owner(take, B, (int32_t)x);
    if (lens[b] >= 0) a.table[(int64_t)b * a.maxblk + held[b] + ((int32_t)x - take[b])] = popped((int32_t)x);
  }
  // the slot of each new row, and -1 behind the last sequence's
  const long long nrow = min((long long)a.T, all.rows);
  for (long long x = at0; x < a.T; x += step) {
    int64_t slot = -1;
    if (x < nrow) {
      const int b = owner(rows, B, (int32_t)x);
      if (lens[b] >= 0) {
        const int32_t pos = lens[b] + (int32_t)x - rows[b];
        const int32_t col = pos >> a.bs_log2;
        const int32_t id =
            col >= held[b] ? popped(take[b] + (col - held[b])) : a.table[(int64_t)b * a.maxblk + col];
        if (id >= 0 && id < a.P)
          slot = ((int64_t)id << a.bs_log2) + (pos & (bs - 1));
        else
          bad_id = true;
      }
    }
    a.slots[x] = slot;
  }
  if (bad_id) atomicOr(a.status, PA_STATUS_BAD_BLOCK);
}

// ------------------------------------------------------------ cache write

// pool[slot[t]] = new[t] for K and V: a copy, bound by memory.  One warp moves
// one token's K row and V row, 16 bytes a lane, kWriteUnroll loads in flight
// per lane before the first store.  50,000 tokens of 8 heads of 128 dims, 410
// MB read and written: 63 us, 6.5 TB/s, 0.96 of the copy rate.
constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 8;

struct WriteArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int64_t* slots;
  uint16_t* k_cache;
  uint16_t* v_cache;
  uint32_t* status;
  int64_t k_stride, v_stride;  // elements between tokens
  int64_t num_slots;
  int32_t T, units;            // 16-byte units of a row
};

__global__ void __launch_bounds__(kWriteThreads) pa_cache_write_kernel(const WriteArgs a) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int64_t slot = __ldg(a.slots + t);
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) atomicOr(a.status, PA_STATUS_NO_SLOT);
    return;
  }
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_new + t * a.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_new + t * a.v_stride);
  uint4* kd = reinterpret_cast<uint4*>(a.k_cache) + slot * a.units;
  uint4* vd = reinterpret_cast<uint4*>(a.v_cache) + slot * a.units;
  for (int u0 = lane; u0 < 2 * a.units; u0 += 32 * kWriteUnroll) {
    uint4 v[kWriteUnroll];
#pragma unroll
    for (int i = 0; i < kWriteUnroll; ++i) {
      const int u = u0 + 32 * i;
      if (u < a.units)
        v[i] = __ldcs(ks + u);
      else if (u < 2 * a.units)
        v[i] = __ldcs(vs + u - a.units);
    }
#pragma unroll
    for (int i = 0; i < kWriteUnroll; ++i) {
      const int u = u0 + 32 * i;
      if (u < a.units)
        kd[u] = v[i];
      else if (u < 2 * a.units)
        vd[u - a.units] = v[i];
    }
  }
}

// ------------------------------------------------------------ draft verification

// Sequence b has k drafted tokens x_0..x_{k-1}, target rows p_0..p_k and draft
// rows q_0..q_{k-1}.  Token i is accepted while u_i q_i(x_i) < p_i(x_i); with n
// the first that is not, the emitted token is drawn from w = max(p_n - q_n, 0)
// (w = p_k when n = k) by inverse CDF: the first index whose running sum
// exceeds u * sum(w).
//
// The comparison is exact: a product of two fp32 values fits a double.  The
// running sums decide a whole number, so they must not depend on the order of
// the additions: p and q are rounded to multiples of 2^-46 and added as whole
// numbers.  (fp64 adds would take longer than the row takes to read.)  Adding 1
// to a value in [0, 1] leaves it rounded to 2^-23 in the low mantissa bits;
// adding 1.5 to 2^23 times what that cut off leaves the next 23 bits.
//
// Bound by the read of one or two rows per sequence.  A row is dealt out in
// segments of kSegment values, a warp per segment; the last CTA of the
// sequence to finish scans the segment sums, finds the crossing segment and
// reads it once more (from L2).  256 rows of 131,071 fp32 values and 120 draft
// rows (197 MB): 49 us, 4.0 TB/s, bound by the latency of its 4-byte loads (rows
// of an odd length are aligned to one value only); 127 us with 64-bit shifts per
// value.  Bulk copies into shared memory took 64 us (16 to 24 warps cannot keep
// up with the sums), a kernel of its own for the accepted counts 49 us, with
// 1.4 us more for the smallest calls.
constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCtasPerSm = 3;
constexpr int kVerifyWaves = 4;  // rounds of CTAs: a rejected draft's sequence has two rows to read, others one
constexpr int kSegment = 512;
constexpr int kVerifyUnroll = 16;  // all of a lane's loads of a segment are in flight together

// One segment's sum (in steps of 2^-46), and whether it held a value that is no
// probability.
struct __align__(16) SegSum {
  unsigned long long sum;
  uint32_t bad;
};

struct VerifyArgs {
  const int32_t* tokens;
  const int32_t* cu;
  const void* q;  // NULL: a draft's distribution is its token alone
  const void* p;
  const float* u_accept;
  const float* u_sample;
  int32_t* out;
  int32_t* accepted;
  uint32_t* status;
  uint32_t* tickets;  // [B], zero between calls
  SegSum* sums;       // [B][nseg]
  int64_t q_stride, p_stride;
  int32_t B, V, D, nseg;
};

template <typename T>
__device__ __forceinline__ float prob(const T* p, int64_t i);
template <>
__device__ __forceinline__ float prob<float>(const float* p, int64_t i) {
  return __ldg(p + i);
}
template <>
__device__ __forceinline__ float prob<__half>(const __half* p, int64_t i) {
  return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p) + i)));
}
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(const __nv_bfloat16* p, int64_t i) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << 16);
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The sum of values in [0, 1], in parts: `high` steps of 2^-23 and `low` of
// 2^-46.  Two values at a time.
struct Parts {
  uint32_t high;
  int32_t low;

  template <bool kMinus>
  __device__ __forceinline__ void add(uint64_t x) {
    const uint64_t one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
    const uint64_t t = add2(x, one);
    const uint64_t rest = fma2(add2(t, minus), minus, x);  // exact
    const uint64_t u = fma2(rest, pack2(0x1p23f, 0x1p23f), pack2(1.5f, 1.5f));
    const uint32_t h = (uint32_t)t + (uint32_t)(t >> 32) - 2u * 0x3f800000u;
    const uint32_t l = (uint32_t)u + (uint32_t)(u >> 32) - 2u * 0x3fc00000u;
    high = kMinus ? high - h : high + h;
    low = kMinus ? low - (int32_t)l : low + (int32_t)l;
  }
  __device__ __forceinline__ unsigned long long value() const {
    return (unsigned long long)(((long long)high << 23) + low);
  }
};

// One value, rounded the same way.
__device__ __forceinline__ unsigned long long fixed46(float x) {
  Parts s = {0u, 0};
  s.add<false>(pack2(x, 0.f));
  return s.value();
}

// A probability as it is used: NaN, infinity and negative values count as 0
// and are flagged, values above 1 count as 1.
__device__ __forceinline__ float checked(float x, uint32_t& bad) {
  bad |= !(x >= 0.f && x < INFINITY);
  return x >= 0.f ? fminf(x, 1.f) : 0.f;
}

// The weight rows of one sequence.
template <typename T>
struct Weights {
  const T* p;
  const T* q;       // NULL: nothing is taken off
  int64_t zero_at;  // index that weighs nothing (lookup drafts), or -1

  __device__ __forceinline__ unsigned long long operator()(int64_t i, uint32_t& bad) const {
    const unsigned long long w = fixed46(checked(prob(p, i), bad));
    const unsigned long long t = q ? fixed46(checked(prob(q, i), bad)) : 0ull;
    return i == zero_at || w < t ? 0ull : w - t;
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Sum of w over [i0, i1) by one warp, i1 - i0 <= kSegment.
template <typename T, bool kQ>
__device__ __forceinline__ SegSum warp_segment_of(const Weights<T>& w, int64_t i0, int64_t i1) {
  const int lane = threadIdx.x & 31;
  Parts s = {0u, 0};
  uint32_t most = 0;  // of the values' bits: above 1's for what is above 1, negative or no number
#pragma unroll 1
  for (int64_t i = i0 + lane; i < i1; i += 32 * kVerifyUnroll) {
    float pv[kVerifyUnroll], qv[kVerifyUnroll];
#pragma unroll
    for (int j = 0; j < kVerifyUnroll; ++j) {
      const int64_t x = i + 32 * j;
      pv[j] = x < i1 ? prob(w.p, x) : 0.f;
      qv[j] = kQ && x < i1 ? prob(w.q, x) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kVerifyUnroll; j += 2) {
      most = max(max(most, __float_as_uint(pv[j])), __float_as_uint(pv[j + 1]));
      if (kQ) {
        most = max(max(most, __float_as_uint(qv[j])), __float_as_uint(qv[j + 1]));
        const bool a = pv[j] > qv[j], b = pv[j + 1] > qv[j + 1];
        s.add<false>(pack2(a ? pv[j] : 0.f, b ? pv[j + 1] : 0.f));
        s.add<true>(pack2(a ? qv[j] : 0.f, b ? qv[j + 1] : 0.f));
      } else {
        s.add<false>(pack2(pv[j], pv[j + 1]));
      }
    }
  }
  // the usual case: every value in [0, 1], no lane's sum above 2 (so the
  // warp's parts below stay in 32 bits)
  const unsigned long long v = s.value();
  const bool plain = most <= 0x3f800000u && v <= (2ull << 46) && !(w.zero_at >= i0 && w.zero_at < i1);
  if (__all_sync(0xffffffffu, plain)) {
    const unsigned long long hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 24));
    const unsigned long long lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0xffffffu);
    return SegSum{(hi << 24) + lo, 0u};
  }
  SegSum r = {0ull, 0u};
  for (int64_t i = i0 + lane; i < i1; i += 32) r.sum += w(i, r.bad);
  r.sum = warp_sum(r.sum);
  r.bad = __reduce_or_sync(0xffffffffu, r.bad);
  return r;
}

template <typename T>
__device__ __forceinline__ SegSum warp_segment(const Weights<T>& w, int64_t i0, int64_t i1) {
  return w.q ? warp_segment_of<T, true>(w, i0, i1) : warp_segment_of<T, false>(w, i0, i1);
}

// Accepted drafts of sequence b (the block agrees on the answer).
template <typename T>
__device__ int accepted_drafts(const VerifyArgs& a, int b, int c0, int k, int* s_first) {
  if (threadIdx.x == 0) *s_first = k;
  __syncthreads();
  for (int i = threadIdx.x; i < k; i += kVerifyThreads) {
    const int32_t x = __ldg(a.tokens + c0 + i);
    bool ok = false;
    if (x >= 0 && x < a.V) {
      const float p = prob(static_cast<const T*>(a.p), (int64_t)(c0 + b + i) * a.p_stride + x);
      const float q = a.q ? prob(static_cast<const T*>(a.q), (int64_t)(c0 + i) * a.q_stride + x) : 1.f;
      ok = (double)__ldg(a.u_accept + c0 + i) * (double)q < (double)p;
    } else if (blockIdx.x == 0) {
      atomicOr(a.status, PA_STATUS_BAD_TOKEN);
    }
    if (!ok) atomicMin(s_first, i);
  }
  __syncthreads();
  return *s_first;
}

// u * total rounded down, exactly (u in [0, 1)): a whole number exceeds the
// product where it exceeds this.  (The product has up to 72 bits; rounded to a
// double's 53 it may reach a running sum that lies just above it.)
__device__ __forceinline__ unsigned long long floor_product(float u, unsigned long long total) {
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint32_t shift = 150u - max(e, 1u);  // u = m 2^-shift; 24 or more
  const unsigned long long hi = __umul64hi(m, total), lo = m * total;
  return shift < 64u ? hi << (64u - shift) | lo >> shift : (shift < 128u ? hi >> (shift - 64u) : 0ull);
}

// The first index of the row whose running sum exceeds u * total, from the
// segment sums (all threads of the block; the answer in *s_pick).
template <typename T>
__device__ void pick(const VerifyArgs& a, const Weights<T>& w, const SegSum* sums, unsigned long long total,
                     float u, unsigned long long* s_scan, int* s_pick) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  u = u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f;
  const unsigned long long t = floor_product(u, total);  // below total
  __shared__ int s_seg;
  __shared__ unsigned long long s_base;
  if (tid == 0) s_seg = -1;
  __syncthreads();
  // the segment: sums scanned kVerifyThreads at a time
  unsigned long long run = 0;
  for (int g0 = 0; g0 < a.nseg; g0 += kVerifyThreads) {
    const unsigned long long v = g0 + tid < a.nseg ? __ldcg(&sums[g0 + tid].sum) : 0ull;
    unsigned long long inc = warp_scan(v);
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    unsigned long long before = run;
    for (int i = 0; i < warp; ++i) before += s_scan[i];
    for (int i = 0; i < kVerifyWarps; ++i) run += s_scan[i];
    inc += before;
    if (inc > t && inc - v <= t) {
      s_seg = g0 + tid;
      s_base = inc - v;
    }
    __syncthreads();
    if (s_seg >= 0) break;
  }
  const int seg = s_seg;  // always found: total > t
  unsigned long long base = s_base;
  // within the segment: a share of 32 kPer values per warp, a row of 32 at a time
  constexpr int kPer = kSegment / kVerifyThreads;
  const int64_t end = min((int64_t)a.V, (int64_t)(seg + 1) * kSegment);
  const int64_t i0 = (int64_t)seg * kSegment + warp * (32 * kPer) + lane;
  unsigned long long v[kPer], mine = 0;
  uint32_t bad = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    v[k] = i0 + 32 * k < end ? w(i0 + 32 * k, bad) : 0ull;
    mine += v[k];
  }
  mine = warp_sum(mine);
  if (lane == 0) s_scan[warp] = mine;
  __syncthreads();
  for (int i = 0; i < warp; ++i) base += s_scan[i];
  if (base <= t && base + mine > t) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const unsigned long long inc = base + warp_scan(v[k]);
      const unsigned hit = __ballot_sync(0xffffffffu, inc > t);
      if (hit) {
        if (lane == 0) *s_pick = (int)(i0 + 32 * k + __ffs(hit) - 1);
        break;
      }
      base = __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtasPerSm) pa_verify_kernel(const VerifyArgs a) {
  after_previous();
  __shared__ int s_first, s_last, s_pick;
  __shared__ unsigned long long s_scan[kVerifyWarps];
  __shared__ double s_approx[kVerifyWarps];
  __shared__ uint32_t s_bad;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  if (c0 < 0 || c1 < c0 || c1 > a.D) {
    if (blockIdx.x == 0 && tid == 0) {
      atomicOr(a.status, PA_STATUS_BAD_SEQLEN);
      a.accepted[b] = -1;
    }
    return;
  }
  const int k = c1 - c0;
  const int n = accepted_drafts<T>(a, b, c0, k, &s_first);
  Weights<T> w;
  w.p = static_cast<const T*>(a.p) + (int64_t)(c0 + b + n) * a.p_stride;
  w.q = a.q && n < k ? static_cast<const T*>(a.q) + (int64_t)(c0 + n) * a.q_stride : nullptr;
  w.zero_at = !a.q && n < k ? (int64_t)__ldg(a.tokens + c0 + n) : -1;
  SegSum* sums = a.sums + (int64_t)b * a.nseg;
  // this CTA's segments, a warp each
  for (int seg = (int)blockIdx.x * kVerifyWarps + warp; seg < a.nseg; seg += (int)gridDim.x * kVerifyWarps) {
    const SegSum s = warp_segment(w, (int64_t)seg * kSegment, min((int64_t)a.V, (int64_t)(seg + 1) * kSegment));
    if (lane == 0) sums[seg] = s;
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    s_last = atomicAdd(a.tickets + b, 1u) == gridDim.x - 1;
    if (s_last) a.tickets[b] = 0;  // for the next call
    s_bad = 0;
    s_pick = -1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // the sequence's last CTA: total, then the token
  unsigned long long total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long part = 0;
    double approx = 0.0;
    uint32_t bad = 0;
    for (int i = tid; i < a.nseg; i += kVerifyThreads) {
      const unsigned long long v = __ldcg(&sums[i].sum);
      part += v;
      approx += (double)v;
      bad |= __ldcg(&sums[i].bad);
    }
    part = warp_sum(part);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) approx += __shfl_xor_sync(0xffffffffu, approx, d);
    if (lane == 0) {
      s_scan[warp] = part;
      s_approx[warp] = approx;
    }
    if (bad) atomicOr(&s_bad, 1u);
    __syncthreads();
    total = 0;
    approx = 0.0;
    for (int i = 0; i < kVerifyWarps; ++i) {
      total += s_scan[i];
      approx += s_approx[i];
    }
    // weights that sum to more than 2 could overflow the whole numbers
    if (tid == 0 && approx > 0x1p47) s_bad = 1u;
    __syncthreads();
    if (s_bad || total || pass) break;
    // nothing is left of p after q was taken off: draw from p itself
    w.q = nullptr;
    w.zero_at = -1;
    for (int seg = warp; seg < a.nseg; seg += kVerifyWarps) {
      const SegSum s = warp_segment(w, (int64_t)seg * kSegment, min((int64_t)a.V, (int64_t)(seg + 1) * kSegment));
      if (lane == 0) sums[seg] = s;
    }
    __syncthreads();
  }
  if (!s_bad && total) pick(a, w, sums, total, __ldg(a.u_sample + b), s_scan, &s_pick);
  __syncthreads();
  int32_t* out = a.out + c0 + b;
  for (int i = tid; i <= k; i += kVerifyThreads) out[i] = i < n ? __ldg(a.tokens + c0 + i) : (i == n ? s_pick : -1);
  if (tid == 0) {
    a.accepted[b] = n;
    if (s_pick < 0) atomicOr(a.status, PA_STATUS_BAD_PROB);
  }
}

// The large slot kernel's shared memory, once per device.
bool allow_slot_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (done[dev].load()) return true;
  if (cudaFuncSetAttribute(pa_slots_kernel<kSlotThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)slot_smem(PA_MAX_BATCH)) != cudaSuccess)
    return false;
  done[dev].store(true);
  return true;
}

int verify_segments(int32_t vocab) { return (vocab + kSegment - 1) / kSegment; }

// The tickets, zero between calls, have the same place whatever the batch: a
// workspace made for a large batch may serve smaller ones in between, whose sums
// must not lie where the large one's tickets are.
constexpr size_t kVerifySums = kStatusBytes + 4 * (size_t)PA_MAX_BATCH;
static_assert(kVerifySums % alignof(SegSum) == 0, "sums are loaded whole");

size_t verify_bytes(int32_t batch, int32_t vocab) {
  return kVerifySums + sizeof(SegSum) * (size_t)batch * verify_segments(vocab);
}

bool verify_shape_ok(int32_t batch, int32_t vocab) {
  return batch >= 0 && batch <= PA_MAX_BATCH && vocab >= 1 && vocab <= PA_MAX_VOCAB;
}

}  // namespace

extern "C" int pa_build_slots(const pa_shape* shape, const int32_t* cache_seqlens, const int32_t* new_lens,
                              const int32_t* held_blocks, int32_t* block_table, int32_t* free_list,
                              const int32_t* free_count, int32_t total_new, int32_t* cu_seqlens_q, int64_t* slots,
                              int32_t* seqlens_out, int32_t* held_out, int32_t* free_count_out, void* workspace,
                              size_t workspace_bytes, pa_stream_t stream) {
  if (!shape) return PA_ERR_NULL;
  const int32_t bs = shape->block_size;
  if (shape->batch < 0 || shape->batch > PA_MAX_BATCH || total_new < 0 || shape->num_blocks < 1 ||
      shape->max_blocks_per_seq < 1 || (bs != 16 && bs != 32 && bs != 64) ||
      (int64_t)shape->max_blocks_per_seq * bs > INT32_MAX ||
      (int64_t)shape->batch * shape->max_blocks_per_seq > INT32_MAX)
    return PA_ERR_SHAPE;
  if (!free_count || !cu_seqlens_q || !free_count_out || !workspace || (total_new > 0 && !slots)) return PA_ERR_NULL;
  if (shape->batch > 0 && (!cache_seqlens || !new_lens || !held_blocks || !block_table || !free_list || !seqlens_out ||
                           !held_out))
    return PA_ERR_NULL;
  for (const void* p : {(const void*)cache_seqlens, (const void*)new_lens, (const void*)held_blocks,
                        (const void*)block_table, (const void*)free_list, (const void*)free_count,
                        (const void*)cu_seqlens_q, (const void*)slots, (const void*)seqlens_out, (const void*)held_out,
                        (const void*)free_count_out, (const void*)workspace})
    if (!aligned16(p)) return PA_ERR_ALIGN;
  if (workspace_bytes < kStatusBytes) return PA_ERR_WORKSPACE;
  SlotArgs a;
  a.seqlens = cache_seqlens;
  a.new_lens = new_lens;
  a.held = held_blocks;
  a.table = block_table;
  a.free_list = free_list;
  a.free_count = free_count;
  a.cu_q = cu_seqlens_q;
  a.slots = slots;
  a.seqlens_out = seqlens_out;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  a.status = static_cast<uint32_t*>(workspace);
  a.B = shape->batch;
  a.maxblk = shape->max_blocks_per_seq;
  a.P = shape->num_blocks;
  a.T = total_new;
  a.bs_log2 = bs == 16 ? 4 : (bs == 32 ? 5 : 6);
  a.ticket = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kTicketOffset);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // a step of few sequences and rows fits one small CTA
  if (a.B <= kSlotThreadsSmall && a.T <= kSlotRows)
    return launch(pa_slots_kernel<kSlotThreadsSmall>, dim3(1), kSlotThreadsSmall, slot_smem(a.B), st, a);
  // (in every call: what a launch may take without it is 48 KB less the kernel's
  // own variables)
  if (!allow_slot_smem()) return PA_ERR_CUDA;
  const int ctas = std::max(1, std::min(kSlotMaxCtas, (a.T + kSlotRows - 1) / kSlotRows));
  return launch(pa_slots_kernel<kSlotThreads>, dim3(ctas), kSlotThreads, slot_smem(a.B), st, a);
}

extern "C" int pa_cache_write(const pa_shape* shape, const void* k_new, int64_t k_stride, const void* v_new,
                              int64_t v_stride, const int64_t* slots, int32_t total_new, void* k_cache, void* v_cache,
                              void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (!shape) return PA_ERR_NULL;
  const int64_t row = (int64_t)shape->num_kv_heads * shape->head_dim;
  if (total_new < 0 || shape->num_kv_heads < 1 || shape->head_dim < 8 || shape->head_dim % 8 != 0 ||
      row > (1 << 24) || shape->block_size < 1 || shape->num_blocks < 1 ||
      (shape->dtype != PA_F16 && shape->dtype != PA_BF16) || k_stride < row || v_stride < row || k_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return PA_ERR_SHAPE;
  if (total_new == 0) return PA_OK;
  if (!k_new || !v_new || !slots || !k_cache || !v_cache || !workspace) return PA_ERR_NULL;
  for (const void* p : {k_new, v_new, (const void*)slots, (const void*)k_cache, (const void*)v_cache,
                        (const void*)workspace})
    if (!aligned16(p)) return PA_ERR_ALIGN;
  if (workspace_bytes < kStatusBytes) return PA_ERR_WORKSPACE;
  WriteArgs a;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.slots = slots;
  a.k_cache = static_cast<uint16_t*>(k_cache);
  a.v_cache = static_cast<uint16_t*>(v_cache);
  a.status = static_cast<uint32_t*>(workspace);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_slots = (int64_t)shape->num_blocks * shape->block_size;
  a.T = total_new;
  a.units = (int32_t)(row / 8);
  constexpr int kPer = kWriteThreads / 32;
  return launch(pa_cache_write_kernel, dim3((unsigned)((total_new + (int64_t)kPer - 1) / kPer)), kWriteThreads, 0,
                reinterpret_cast<cudaStream_t>(stream), a);
}

extern "C" int pa_workspace_size_verify(int32_t batch, int32_t vocab, size_t* bytes) {
  if (!bytes) return PA_ERR_NULL;
  if (!verify_shape_ok(batch, vocab)) return PA_ERR_SHAPE;
  *bytes = verify_bytes(batch, vocab);
  return PA_OK;
}

extern "C" int pa_verify_drafts(int32_t batch, int32_t vocab, int32_t total_drafts, int32_t prob_dtype,
                                const int32_t* draft_tokens, const int32_t* cu_drafts, const void* draft_probs,
                                int64_t draft_stride, const void* target_probs, int64_t target_stride,
                                const float* u_accept, const float* u_sample, int32_t* tokens, int32_t* accepted,
                                void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (!verify_shape_ok(batch, vocab) || total_drafts < 0 || total_drafts > INT32_MAX - PA_MAX_BATCH ||
      (prob_dtype != PA_F16 && prob_dtype != PA_BF16 && prob_dtype != PA_F32) || target_stride < vocab ||
      (draft_probs && draft_stride < vocab))
    return PA_ERR_SHAPE;
  if (batch == 0) return PA_OK;
  if (!cu_drafts || !target_probs || !u_sample || !tokens || !accepted || !workspace ||
      (total_drafts > 0 && (!draft_tokens || !u_accept)))
    return PA_ERR_NULL;
  for (const void* p : {(const void*)draft_tokens, (const void*)cu_drafts, draft_probs, target_probs,
                        (const void*)u_accept, (const void*)u_sample, (const void*)tokens, (const void*)accepted,
                        (const void*)workspace})
    if (!aligned16(p)) return PA_ERR_ALIGN;
  if (workspace_bytes < verify_bytes(batch, vocab)) return PA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  VerifyArgs a;
  a.tokens = draft_tokens;
  a.cu = cu_drafts;
  a.q = draft_probs;
  a.p = target_probs;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.out = tokens;
  a.accepted = accepted;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.tickets = reinterpret_cast<uint32_t*>(ws + kStatusBytes);
  a.sums = reinterpret_cast<SegSum*>(ws + kVerifySums);
  a.q_stride = draft_stride;
  a.p_stride = target_stride;
  a.B = batch;
  a.V = vocab;
  a.D = total_drafts;
  a.nseg = verify_segments(vocab);
  // several rounds of CTAs where there are many rows, a segment for each warp
  // where there are few
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  const int most = (a.nseg + kVerifyWarps - 1) / kVerifyWarps;
  const dim3 grid(std::max(1, std::min(most, kVerifyWaves * sms * kVerifyCtasPerSm / batch)), batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (prob_dtype == PA_F32) return launch(pa_verify_kernel<float>, grid, kVerifyThreads, 0, st, a);
  if (prob_dtype == PA_F16) return launch(pa_verify_kernel<__half>, grid, kVerifyThreads, 0, st, a);
  return launch(pa_verify_kernel<__nv_bfloat16>, grid, kVerifyThreads, 0, st, a);
}
