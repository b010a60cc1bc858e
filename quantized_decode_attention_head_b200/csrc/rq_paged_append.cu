// Appending new tokens to the paged 16-bit cache: keys and queries rotated by
// position, keys and values written to their pages, in one pass.
//
// Every element is read once and written once; there is no reuse but that of
// a position's cosines and sines by the heads of its token.  Memory bound:
// (2 Hq + 4 Hkv) D 16-bit values a token.  A lane owns one 16-byte vector of
// a head, or the two vectors whose channels are paired, with their cosines and
// sines in registers, and walks over the heads of its token, several loads in
// flight; neighbouring lanes own neighbouring vectors.  A block takes several
// tokens at a time, and a warp of its own finds the places of the next ones
// (sequence, page, positions: a chain of dependent loads) meanwhile; one token
// a block when there are few, where the call is that chain's latency.
// Measured: 251 MB of prompts (three axes, 32/8 heads, D = 128) 48.7 us, 5.2 TB/s;
// one token of each of eight sequences 4.3 us on the device.
#include "rq_paged.cuh"
#include "rq_paged_launch.h"

namespace rq {
namespace {

constexpr int kThreads = 256;  // that move data; one more warp finds the next tokens' places
constexpr int kResident = 3;   // blocks an SM: 4 would spill registers (62 us for 50, 20k tokens of three axes)
constexpr int kMaxTokens = 8;  // of a block at a time

// Where a token goes.
struct Place {
  int64_t row;         // its row of kv head 0 in the pages, -1: not written
  int pos[kMaxAxes];   // its position on each axis
  int state;           // 0: no sequence's, 1: whole, 2: position outside the table of angles
};

// (a, b) turned by (c, s): products and differences each rounded once in fp32
// (no contraction), so that the result does not depend on the compiler.
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// The position of pair j on its axis.
__device__ __forceinline__ int pair_position(const PagedAppendArgs& a, const int* pos, int j) {
  int ax = 0, end = a.sections[0];
#pragma unroll
  for (int k = 1; k < kMaxAxes; ++k)
    if (k < a.n_axes && j >= end) {
      ax = k;
      end += a.sections[k];
    }
  return pos[ax];
}

// Cosines and sines of N pairs from j on: wide loads when one position serves
// them all (an axis may end between two of them).
template <int N>
__device__ __forceinline__ void load_angles(const PagedAppendArgs& a, const int* pos, int j, float (&c)[8], float (&s)[8]) {
  const int half = a.rot / 2, p0 = pair_position(a, pos, j);
  bool one = true;
  if (a.n_axes > 1) {
#pragma unroll
    for (int e = 1; e < N; ++e) one &= pair_position(a, pos, j + e) == p0;
  }
  if (one) {
    const float4* tc = reinterpret_cast<const float4*>(a.cos_sin + (int64_t)p0 * a.rot + j);
    const float4* ts = reinterpret_cast<const float4*>(a.cos_sin + (int64_t)p0 * a.rot + half + j);
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
      const float4 x = ld_in(tc + e), y = ld_in(ts + e);
      c[4 * e] = x.x, c[4 * e + 1] = x.y, c[4 * e + 2] = x.z, c[4 * e + 3] = x.w;
      s[4 * e] = y.x, s[4 * e + 1] = y.y, s[4 * e + 2] = y.z, s[4 * e + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float* t = a.cos_sin + (int64_t)pair_position(a, pos, j + e) * a.rot;
      c[e] = ld_in(t + j + e);
      s[e] = ld_in(t + half + j + e);
    }
  }
}

__device__ __forceinline__ Place place_of(const PagedAppendArgs& a, int64_t t64) {
  Place o = {-1, {0, 0, 0, 0}, 0};
  if (t64 >= a.b.n_tokens) return o;
  const int t = (int)t64;
  const int seq = seq_of(a.b, t);
  if (seq < 0) return o;
  const Seq s = load_seq(a.b, seq);
  if (t < s.t0 || t >= s.t0 + s.n) return o;  // offsets out of order: the token has no sequence
  const int at = s.end - s.n + (t - s.t0);
  o.state = 1;
  if (a.cos_sin) {
#pragma unroll
    for (int k = 0; k < kMaxAxes; ++k)
      if (k < a.n_axes) {
        o.pos[k] = a.positions ? ld_in(a.positions + (int64_t)k * a.b.n_tokens + t) : at;
        if ((unsigned)o.pos[k] >= (unsigned)a.n_positions) o.state = 2;
      }
  }
  if (at >= 0 && at < s.len) {
    o.row = page_row(a.b, ld_in(a.b.table + (int64_t)seq * a.b.width + (at >> a.b.page_shift)));
    if (o.row >= 0) o.row += at & ((1 << a.b.page_shift) - 1);
  }
  if (at < 0 || o.state == 2) flag_index(a.b.status);
  if (o.state == 2) o.row = -1;
  return o;
}

// kPairs: channels j and j + rot/2 are paired (else 2j and 2j + 1).
template <class T, int D, bool kPairs>
__device__ __forceinline__ void move_tokens(const PagedAppendArgs& a, const Place* places, int64_t t0) {
  const int tokens = a.block_tokens;
  const int rot = a.cos_sin ? a.rot : 0, half = rot / 2;
  // a head's items: half/8 pairs of vectors and the rest single vectors, or
  // D/8 single vectors when neighbouring channels are paired
  const int pairs = kPairs ? half / 8 : 0;
  const int per_head = D / 8 - pairs;
  const int lanes = tokens * per_head, groups = kThreads / lanes;  // lanes of a group walk over the same heads
  const int group = threadIdx.x / lanes, x = threadIdx.x - group * lanes;
  const int token = x / per_head, v = x - token * per_head;
  if (group >= groups) return;
  const Place& p = places[token];
  if (p.state == 0) return;
  const int64_t t = t0 + token;
  const bool paired = v < pairs;
  const int first = kPairs && !paired ? v + pairs : v;  // the item's (first) vector of a head
  const bool turns = paired || (!kPairs && 8 * v < rot);
  float c[8], s[8];
  if (turns && p.state == 1) {
    if (paired)
      load_angles<8>(a, p.pos, 8 * v, c, s);
    else
      load_angles<4>(a, p.pos, 4 * v, c, s);
  }
  const int heads_q = a.q ? a.b.hq : 0, heads = heads_q + 2 * a.b.hkv;
  const int64_t row = p.row;
  auto source = [&](int h) {
    if (h < heads_q) return a.q + t * a.q_stride + h * D;
    h -= heads_q;
    return h < a.b.hkv ? a.k_new + t * a.k_stride + h * D : a.v_new + t * a.v_stride + (h - a.b.hkv) * D;
  };
  constexpr int kAhead = 2;  // heads loaded at once (4: fewer blocks an SM, 58 us for 50)
  for (int h0 = group; h0 < heads; h0 += kAhead * groups) {
    uint4 lo[kAhead], hi[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * groups;
      if (h < heads) {
        const uint16_t* src = source(h);
        lo[i] = ld_once(reinterpret_cast<const uint4*>(src) + first);
        if (paired) hi[i] = ld_once(reinterpret_cast<const uint4*>(src + half) + first);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * groups;
      if (h >= heads) break;
      uint16_t* dst;
      bool turn_it = turns;
      if (h < heads_q) {
        dst = a.q_out + (t * a.b.hq + h) * D;
        if (p.state == 2) {  // no such position
          lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
          turn_it = false;
        }
      } else {
        if (row < 0) break;
        const int kh = h - heads_q;
        const bool key = kh < a.b.hkv;
        const int64_t hh = key ? kh : kh - a.b.hkv;
        dst = (key ? a.k_pages : a.v_pages) + (row + (hh << a.b.page_shift)) * D;
        turn_it = turns && key;
      }
      if (turn_it) {
        uint32_t* xp = reinterpret_cast<uint32_t*>(&lo[i]);
        if (paired) {
          uint32_t* yp = reinterpret_cast<uint32_t*>(&hi[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x2 = T::unpack(xp[e]), y2 = T::unpack(yp[e]);
            const float2 r0 = turn(x2.x, y2.x, c[2 * e], s[2 * e]), r1 = turn(x2.y, y2.y, c[2 * e + 1], s[2 * e + 1]);
            xp[e] = T::pack(r0.x, r1.x);
            yp[e] = T::pack(r0.y, r1.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x2 = T::unpack(xp[e]);
            const float2 r = turn(x2.x, x2.y, c[e], s[e]);
            xp[e] = T::pack(r.x, r.y);
          }
        }
      }
      reinterpret_cast<uint4*>(dst)[first] = lo[i];
      if (paired) reinterpret_cast<uint4*>(dst + half)[first] = hi[i];
    }
  }
}

template <class T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads + 32, kResident) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Place places[2][kMaxTokens];
  const int tokens = a.block_tokens, stride = gridDim.x * tokens;
  const int finder = (int)threadIdx.x - kThreads;  // lane of the warp that finds places
  int64_t t0 = (int64_t)blockIdx.x * tokens;
  if (finder >= 0 && finder < tokens) places[0][finder] = place_of(a, t0 + finder);
  for (int turn = 0; t0 < a.b.n_tokens; t0 += stride, turn ^= 1) {
    __syncthreads();
    if (finder < 0)
      move_tokens<T, D, kPairs>(a, places[turn], t0);
    else if (finder < tokens)
      places[turn ^ 1][finder] = place_of(a, t0 + stride + finder);
  }
}

template <class T, int D>
cudaError_t launch(PagedAppendArgs a, cudaStream_t s) {
  // tokens of a block: 8 when that still leaves four blocks an SM
  static_assert(kMaxTokens * D / 8 <= kThreads, "one lane an item at least");
  a.block_tokens = 1;
  while (a.block_tokens < kMaxTokens && a.b.n_tokens / (2 * a.block_tokens) >= 4 * a.sms) a.block_tokens *= 2;
  int64_t blocks = (a.b.n_tokens + (int64_t)a.block_tokens - 1) / a.block_tokens;
  if (a.block_tokens == kMaxTokens && blocks > kResident * a.sms) blocks = kResident * a.sms;  // one wave, several rounds each
  const dim3 grid((unsigned)blocks);
  return a.interleaved ? launch_pdl<paged_append_kernel<T, D, false>>(grid, kThreads + 32, 0, s, a)
                       : launch_pdl<paged_append_kernel<T, D, true>>(grid, kThreads + 32, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128) return dtype == 0 ? launch<Bf16, 128>(a, s) : launch<Fp16, 128>(a, s);
  return dtype == 0 ? launch<Bf16, 64>(a, s) : launch<Fp16, 64>(a, s);
}

}  // namespace rq
