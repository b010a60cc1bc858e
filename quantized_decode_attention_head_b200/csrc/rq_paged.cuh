// Device helpers of the paged 16-bit cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rq_device.cuh"
#include "rq_paged.h"

namespace rq {

// Bounded wait for a barrier's phase (false after about a second).  The clock
// is read on every 64th try only: it costs more than a try.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0)
        t0 = t;
      else if (t - t0 > kWaitLimitNs)
        return false;
    }
  }
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// The status word: a wait that gave up is not hidden by an index out of range,
// whichever comes first.
__device__ __forceinline__ void flag_index(int* status) {
  if (status) atomicCAS(status, 0, kDeviceIndex);
}
__device__ __forceinline__ void flag_timeout(int* status) { atomicExch(status, kDeviceTimeout); }

// After a wait that gave up: time (10 ms) for copies still in flight to land
// before the shared memory goes to another CTA.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 10000000ull) {
  }
}

// Loads of what a caller passes.  A kernel is resident while the call before it
// still writes (programmatic launch), and queries may be rotated in place, so
// none of it is read-only for the life of a kernel: not through ld.global.nc,
// which the compiler may also move above griddepcontrol.wait.  once: what one
// launch reads once (new tokens, partial states, whole rows of queries), from
// L2; the decode kernel reads a query's words four warps at a time, through L1
// (from L2: attend 64 ragged sequences 148 us for 142).
template <class V>
__device__ __forceinline__ V ld_in(const V* p) {
  return *p;
}
template <class V>
__device__ __forceinline__ V ld_once(const V* p) {
  return __ldcg(p);
}

// Brings a tensor map into the descriptor cache.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// 16-bit element types of the pages: conversions to and from fp32.
// Weights enter the second product in the type, as powers of two relative to
// the row's running maximum.  bf16 has fp32's exponents; fp16 ends at 2^-24,
// and its weights are held 2^kUp (two terms) or 2^kUpLag (one term, with a
// maximum that lags by up to 2^kLag) larger, which the sums and the stored
// maximum share, so that what a long tail adds to the sum it adds to the
// product too: the largest is 2^14, or in one term 2^6 to 2^14, the smallest
// step 2^-38 or 2^-30 of it.  (A lag of 2^4 and a factor of 2^10 held steps of
// 2^-34, but moves the maximum more often: 8192-token prompt 471 us for 446.)
struct Bf16 {
  static constexpr int kType = 1;  // of tcgen05 instruction descriptors
  static constexpr float kUp = 0.f, kUpLag = 0.f, kLag = 8.f;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_bf16_k16(d, a[0], a[1], a[2], a[3], b0, b1);
  }
};
struct Fp16 {
  static constexpr int kType = 0;
  static constexpr float kUp = 14.f, kUpLag = 6.f, kLag = 8.f;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// A sequence of the batch as the device finds it: its packed tokens are
// [t0, t0 + n), new token i is token end - n + i of the sequence, of which the
// table has room for the first len.  Out of range, and flagged: a length past
// the table (len ends there, positions stay what the length makes them), one
// below zero (counts as zero), and offsets that leave the packed rows (no new
// tokens).  So nothing is read or written outside the caller's tensors, nor
// any token in another's place.
struct Seq {
  int t0, n, len, end;
};
__device__ __forceinline__ Seq load_seq(const PagedBatch& b, int i) {
  Seq s;
  const int len = ld_in(b.kv_lens + i);
  const int64_t cap64 = (int64_t)b.width << b.page_shift;
  const int cap = cap64 > 0x7FFFFFFF ? 0x7FFFFFFF : (int)cap64;
  s.len = len < 0 ? 0 : (len > cap ? cap : len);
  s.end = len < 0 ? 0 : (len > b.top ? b.top : len);
  bool bad = s.len != len;
  if (b.cu) {
    const int lo = ld_in(b.cu + i), hi = ld_in(b.cu + i + 1);
    const bool out = lo < 0 || hi < lo || hi > b.n_tokens;
    bad |= out;
    s.t0 = out ? 0 : lo;
    s.n = out ? 0 : hi - lo;
  } else {
    s.t0 = i;
    s.n = 1;
  }
  if (bad) flag_index(b.status);
  return s;
}

// The sequence that packed token t belongs to; -1 behind the last one.
__device__ __forceinline__ int seq_of(const PagedBatch& b, int t) {
  if (!b.cu) return t < b.n_seqs ? t : -1;
  int lo = 0, hi = b.n_seqs;  // first index with cu[index + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ld_in(b.cu + mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo < b.n_seqs ? lo : -1;
}

// Row (of the layer's first kv head) where page number `page` begins, or -1
// when the number is out of range.
__device__ __forceinline__ int64_t page_row(const PagedBatch& b, int page) {
  if ((unsigned)page >= (unsigned)b.n_pages) {
    flag_index(b.status);
    return -1;
  }
  return b.page_base + (((int64_t)page * b.hkv) << b.page_shift);
}

constexpr int kChunk = 16;      // tokens that the decode kernel copies at once (a stage)
constexpr int kUnitChunks = 4;  // chunks of a unit, by which it divides its work

// One sequence as the decode kernel walks it: the 16-token chunks that any of its
// queries sees are, in order, chunks [0, ns) (first tokens) and [lo_c, ...).
struct Walk {
  int t0, n, len;      // packed tokens, tokens held
  int first;           // place of the first query in the sequence
  int lo, sink;        // tokens [0, sink) and [lo, len) are seen by some query
  int ns, lo_c, chunks, units;
};
// (not inlined: the decode kernel's start is bound by fetching its code)
static __device__ __noinline__ Walk walk_of(const PagedAttnArgs& a, int b) {
  Walk w = {};
  if (b >= a.b.n_seqs) return w;  // no units
  const Seq s = load_seq(a.b, b);
  w.t0 = s.t0;
  w.n = s.n;
  w.len = s.len;
  w.first = s.end - s.n;
  int lo = a.window > 0 ? w.first + 1 - a.window : 0;
  lo = lo < 0 ? 0 : (lo > s.len ? s.len : lo);
  int sink = a.window > 0 ? a.n_sink - a.prefix_len : 0;
  sink = sink < 0 ? 0 : (sink > s.len ? s.len : sink);
  w.lo = lo;
  w.sink = sink;
  w.lo_c = lo / kChunk;
  const int sc = (sink + kChunk - 1) / kChunk;
  w.ns = sc < w.lo_c ? sc : w.lo_c;
  w.chunks = w.ns + (s.len + kChunk - 1) / kChunk - w.lo_c;
  const bool mine = s.n > 0 && (s.n << a.b.g_shift) <= kDecodeRows;
  if (s.n > 0 && !mine && a.few_rows_only) flag_index(a.b.status);  // more new tokens than max_new said
  w.units = mine ? (w.chunks > kUnitChunks ? (w.chunks + kUnitChunks - 1) / kUnitChunks : 1) : 0;  // a stream that sees nothing still writes
  return w;
}

// How the SMs are divided when the prefix (prompt kernel) and what follows it
// (decode kernel) run side by side, from the units that the lengths on the
// device make of the latter.  128 keys take a CTA of either about as long (1.9
// us measured: two units of the decode kernel's two teams, or a step of 256
// rows), so the shares go by them.  The same in every kernel of a call.
struct Shares {
  int splits;  // of the prefix's keys
  int ctas;    // of the decode kernel
};
__device__ __forceinline__ Shares shares_of(const PagedAttnArgs& a, int64_t tail_units) {
  Shares s = {1, a.n_ctas};
  if (a.front_ctas >= a.n_ctas) return s;  // the prefix fills the device for a while: one after the other
  const int x = (int)(a.n_ctas * ((float)tail_units / ((float)tail_units + a.front_units)));
  s.splits = (a.n_ctas - x) / a.front_ctas;
  s.splits = s.splits < 1 ? 1 : (s.splits > a.max_splits ? a.max_splits : s.splits);
  const int left = a.n_ctas - a.front_ctas * s.splits;
  s.ctas = x > left ? x : left;
  if (s.ctas < 1) s.ctas = 1;
  return s;
}

// Four channels of a row's state (v not yet divided by l, maximum m in log2
// units): the result, or the row's partial state for the merge of the parts.
template <class T, int D>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, int token, int head, int c4, float4 v, float m,
                                          float l) {
  const int64_t row = (int64_t)token * a.b.hq + head;
  if (a.rows_o) {
    const int64_t at = (int64_t)a.row_slot * a.b.n_tokens * a.b.hq + row;
    *reinterpret_cast<float4*>(a.rows_o + at * D + 4 * c4) = v;
    if (c4 == 0) *reinterpret_cast<float2*>(a.rows_ml + 2 * at) = make_float2(m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(a.out + row * D + 4 * c4) =
      make_uint2(T::pack(v.x * inv, v.y * inv), T::pack(v.z * inv, v.w * inv));
  if (c4 == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

}  // namespace rq
