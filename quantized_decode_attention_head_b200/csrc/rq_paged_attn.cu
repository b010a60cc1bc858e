// Attention over the paged 16-bit cache: the plain kernel, one warp for each
// query head of a token, one key after another, online softmax in base 2.
#include "rq_paged.cuh"

namespace rq {
namespace {

constexpr int kWarps = 4;

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_attention_kernel(const __grid_constant__ PagedAttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(w / a.b.hq), h = (int)(w % a.b.hq);
  if (t >= a.b.n_tokens) return;
  const int seq = seq_of(a.b, t);
  if (seq < 0) return;
  const Seq s = load_seq(a.b, seq);
  if (t < s.t0 || t >= s.t0 + s.n) return;
  constexpr int E = D / 64;  // pairs of channels a lane holds
  float2 q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = T::unpack(__ldg(reinterpret_cast<const uint32_t*>(a.q + t * a.q_stride + h * D) + 32 * e + lane));
    o[e] = make_float2(0.f, 0.f);
  }
  const int64_t end = (int64_t)a.prefix_len + s.len;             // keys of the sequence
  const int64_t p = end - s.n + (t - s.t0);                      // the query's position
  const int64_t lo = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
  const int ps = 1 << a.b.page_shift;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = lo < a.n_sink ? 0 : (a.n_sink > 0 ? 0 : lo); j <= p; ++j) {
    if (j >= a.n_sink && j < lo) {
      j = lo;
    }
    const int jj = (int)(j < a.prefix_len ? j : j - a.prefix_len);
    const int page = __ldg((j < a.prefix_len ? a.prefix : a.b.table + (int64_t)seq * a.b.width) + (jj >> a.b.page_shift));
    int64_t row = page_row(a.b, page);
    if (row < 0) continue;
    row += ((int64_t)(h >> a.b.g_shift) << a.b.page_shift) + (jj & (ps - 1));
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(a.k_pages + row * D);
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(a.v_pages + row * D);
    float x = 0.f;
    float2 v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 k = T::unpack(__ldg(kr + 32 * e + lane));
      v[e] = T::unpack(__ldg(vr + 32 * e + lane));
      x = fmaf(q[e].x, k.x, fmaf(q[e].y, k.y, x));
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x);
    const float alpha = ex2(m - mn), pr = ex2(x - mn);
    m = mn;
    l = fmaf(l, alpha, pr);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e].x = fmaf(o[e].x, alpha, pr * v[e].x);
      o[e].y = fmaf(o[e].y, alpha, pr * v[e].y);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t r = (int64_t)t * a.b.hq + h;
#pragma unroll
  for (int e = 0; e < E; ++e)
    reinterpret_cast<uint32_t*>(a.out + r * D)[32 * e + lane] = T::pack(o[e].x * inv, o[e].y * inv);
  if (a.lse && lane == 0) a.lse[r] = l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
}

template <class T>
cudaError_t launch(const PagedAttnArgs& a, int head_dim, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.b.n_tokens * a.b.hq + kWarps - 1) / kWarps;
  if (head_dim == 128)
    paged_attention_kernel<T, 128><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
  else
    paged_attention_kernel<T, 64><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int head_dim, int dtype, cudaStream_t s) {
  return dtype == 0 ? launch<Bf16>(a, head_dim, s) : launch<Fp16>(a, head_dim, s);
}

}  // namespace rq
