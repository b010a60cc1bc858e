// Appending new tokens to the paged 16-bit cache: keys and queries rotated by
// position, keys and values written to their pages, in one pass.
//
// Every element is read once and written once; there is no reuse but that of
// a position's cosines and sines by the heads of its token, which L1 serves.
// Memory bound: (2 Hq + 4 Hkv) D 16-bit values a token.  A work item is one
// 16-byte vector of a head, or the two vectors whose channels are paired; a
// block takes one token, its items one after another, so that neighbouring
// threads move neighbouring vectors.
#include "rq_paged.cuh"
#include "rq_paged_launch.h"

namespace rq {
namespace {

constexpr int kThreads = 128;

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

template <class T, int D>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x;
  const int seq = seq_of(a.b, t);
  if (seq < 0) return;
  const Seq s = load_seq(a.b, seq);
  if (t < s.t0 || t >= s.t0 + s.n) return;  // offsets out of order: the token has no sequence
  const int place = s.len - s.n + (t - s.t0);
  int64_t row = -1;
  if (place >= 0) {
    row = page_row(a.b, __ldg(a.b.table + (int64_t)seq * a.b.width + (place >> a.b.page_shift)));
    if (row >= 0) row += place & ((1 << a.b.page_shift) - 1);
  } else {
    flag_index(a.b.status);
  }
  // the token's position on each axis; outside the table of angles: bad
  int pos[kMaxAxes];
  bool bad = false;
  if (a.cos_sin) {
#pragma unroll
    for (int k = 0; k < kMaxAxes; ++k) {
      pos[k] = 0;
      if (k < a.n_axes) {
        pos[k] = a.positions ? __ldg(a.positions + (int64_t)k * a.b.n_tokens + t) : place;
        if ((unsigned)pos[k] >= (unsigned)a.n_positions) bad = true;
      }
    }
    if (bad) flag_index(a.b.status);
  }
  const int rot = a.cos_sin ? a.rot : 0;
  const int half = rot / 2;
  // items of a head: half/8 pairs of vectors and the rest single vectors, or
  // D/8 single vectors when the pairs are neighbours
  const int pairs = a.interleaved ? 0 : half / 8;
  const int per_head = D / 8 - pairs;
  const int heads_q = a.q ? a.b.hq : 0;
  const int items = (heads_q + 2 * a.b.hkv) * per_head;
  const int item0 = blockIdx.y * kThreads + threadIdx.x;
  for (int it = item0; it < items; it += gridDim.y * kThreads) {
    const int h = it / per_head, v = it - h * per_head;
    const uint16_t* src;
    uint16_t* dst;
    bool turns = true;
    if (h < heads_q) {
      src = a.q + t * a.q_stride + h * D;
      dst = a.q_out + ((int64_t)t * a.b.hq + h) * D;
    } else {
      if (row < 0 || bad) continue;
      const int kh = h - heads_q;
      const bool key = kh < a.b.hkv;
      const int hh = key ? kh : kh - a.b.hkv;
      src = (key ? a.k_new + t * a.k_stride : a.v_new + t * a.v_stride) + hh * D;
      dst = (key ? a.k_pages : a.v_pages) + (row + ((int64_t)hh << a.b.page_shift)) * D;
      turns = key;
    }
    if (v < pairs) {
      uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + v);
      uint4 y = __ldg(reinterpret_cast<const uint4*>(src + half) + v);
      if (turns) {
        uint32_t* xp = reinterpret_cast<uint32_t*>(&x);
        uint32_t* yp = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * v + 2 * e;
          const float2 lo = T::unpack(xp[e]), hi = T::unpack(yp[e]);
          float2 r0 = make_float2(0.f, 0.f), r1 = r0;
          if (!bad) {
            const float* t0 = a.cos_sin + (int64_t)pair_position(a, pos, j) * rot;
            const float* t1 = a.cos_sin + (int64_t)pair_position(a, pos, j + 1) * rot;
            r0 = turn(lo.x, hi.x, __ldg(t0 + j), __ldg(t0 + half + j));
            r1 = turn(lo.y, hi.y, __ldg(t1 + j + 1), __ldg(t1 + half + j + 1));
          }
          xp[e] = T::pack(r0.x, r1.x);
          yp[e] = T::pack(r0.y, r1.y);
        }
      }
      reinterpret_cast<uint4*>(dst)[v] = x;
      reinterpret_cast<uint4*>(dst + half)[v] = y;
    } else {
      const int vv = a.interleaved ? v : v + pairs;
      uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + vv);
      if (turns && (bad || 8 * vv < rot)) {
        uint32_t* xp = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * vv + e;
          const float2 ab = T::unpack(xp[e]);
          float2 r = make_float2(0.f, 0.f);
          if (!bad) {
            const float* tj = a.cos_sin + (int64_t)pair_position(a, pos, j) * rot;
            r = turn(ab.x, ab.y, __ldg(tj + j), __ldg(tj + half + j));
          }
          xp[e] = T::pack(r.x, r.y);
        }
      }
      reinterpret_cast<uint4*>(dst)[vv] = x;
    }
  }
}

template <class T>
cudaError_t launch(const PagedAppendArgs& a, int head_dim, cudaStream_t s) {
  const dim3 grid(a.b.n_tokens, 1);
  return head_dim == 128 ? launch_pdl<paged_append_kernel<T, 128>>(grid, kThreads, 0, s, a)
                         : launch_pdl<paged_append_kernel<T, 64>>(grid, kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int head_dim, int dtype, cudaStream_t s) {
  return dtype == 0 ? launch<Bf16>(a, head_dim, s) : launch<Fp16>(a, head_dim, s);
}

}  // namespace rq
