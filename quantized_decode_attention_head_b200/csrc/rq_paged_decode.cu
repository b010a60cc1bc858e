// Attention of few query rows per sequence over the paged 16-bit cache
// (sm_100a): single tokens and short drafts, n_b * G <= 16 rows a kv head.
//
// Memory bound: every visible key and value row is read once for the G query
// heads (and drafted tokens) that share it, 4 G flops for 4 bytes.  So the
// design is a stream: each warp owns a ring of stages, 16 tokens of keys and
// values each, that its first lane keeps filling with tiled TMA copies (one
// for the keys and one for the values, 128-byte swizzle, so that the ldmatrix
// reads are free of bank conflicts); 192 KB an SM are in flight at head_dim
// 128.
//
// Work is split over the tokens, whatever the lengths: the visible tokens of
// all (sequence, kv head) streams, in units of 64, form one line that the
// teams divide evenly.  A team is four warps, each with every fourth 16 tokens
// of a unit; a CTA holds two teams and fills an SM, so that one team's latency
// (a stream's queries, the merge of its warps) passes under the other's work.
// The line is laid out on the device from the lengths, so a captured launch
// follows them.  A team whose share ends inside a stream publishes a partial
// softmax state (at most two a team: its first and its last stream); the last
// of a stream's teams to arrive merges them in the order of the teams, so
// results do not depend on timing.
//
// Products run on mma.sync m16n8k16 (rows = token, head), fp32 accumulation;
// the weights enter the second product as two 16-bit terms (high and rest:
// 2^-16 relative or better; fp16: or 2^-39 of the row's largest weight), which
// costs tensor issue slots that a stream of memory leaves idle and keeps their
// rounding out of the result.
//
// Measured (32/8 heads, D = 128, bf16): 64 ragged sequences up to 8192 tokens
// 142 us, 5.8 TB/s; one of 131072 tokens 94 us, 5.7 TB/s; 16 with a window of
// 4096 55 us, 4.5 TB/s.  About 5 us pass before the first keys arrive and 2 at
// the end; between them DRAM runs at about 7 TB/s, and the SMs finish their
// equal shares up to 15 % apart.  One team of four warps and 32-token stages:
// 148, 90 and 52 us; one team with 16-token stages: 191, 119 and 64 us.
#include <cuda.h>

#include "rq_paged.cuh"
#include "rq_paged_launch.h"

namespace rq {
namespace {

constexpr int NW = kUnitChunks;  // warps a team, a chunk of a unit each
constexpr int kTeams = 2;     // teams a CTA
constexpr int kThreads = kTeams * NW * 32;
constexpr int kRows = 16;     // query rows of an MMA
static_assert(kRows == kDecodeRows, "one MMA holds a stream's rows");
constexpr int kMergeRows = 4; // rows a team merges at once

template <int D>
struct Cfg {
  static constexpr int P = D / 64;                      // 64-channel panels of a row
  static constexpr int PANEL = kChunk * 128;            // bytes of a panel of a stage
  static constexpr int HALF = P * PANEL;                // keys or values of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int S = 24576 / STAGE;               // stages a warp
  static constexpr int RING = NW * S * STAGE;           // 96 KB a team
  static constexpr int OSTR = D + 4;                    // floats of a row of the merge buffer
  static constexpr int MERGE = NW * kMergeRows * OSTR * 4;
  static constexpr int SMEM = 1024 + kTeams * (RING + MERGE);  // rings aligned to 1024 bytes
};

// Shared state of a team.
template <int S>
struct Team {
  uint64_t full[NW][S];
  uint32_t page_ok[NW][S];
  float ml[NW][kRows][2];
  int64_t n[2 * NW + 1];
  int v[2];
};

// A place on the line of units: unit i of kv head h of sequence b.
struct Cursor {
  Walk w;
  int b, h, i;
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    if (++i < w.units) return;
    i = 0;
    if (++h < a.b.hkv) return;
    h = 0;
    do {
      w = walk_of(a, ++b);
    } while (b < a.b.n_seqs && w.units == 0);
  }
};

__device__ __forceinline__ int chunk_token(const Walk& w, int c) {
  return kChunk * (c < w.ns ? c : w.lo_c + c - w.ns);
}

// All channels of 16 rows from row y on: [panel][row][64 channels].
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2}], [%4];\n" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void team_sync(int team) { asm volatile("bar.sync %0, 128;\n" ::"r"(team + 1) : "memory"); }

// First unit of team c when U units are divided among n CTAs (n <= U).
__device__ __forceinline__ int64_t share_begin(int64_t c, int64_t U, int64_t n) { return c * U / n; }
// The team whose share holds unit u.
__device__ __forceinline__ int share_of(int64_t u, int64_t U, int64_t n) { return (int)(((u + 1) * n + U - 1) / U - 1); }

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Team<C::S> teams[kTeams];
  const int team = threadIdx.x / (NW * 32);
  uint8_t* rings = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = rings + team * C::RING;
  float* merge = reinterpret_cast<float*>(rings + kTeams * C::RING + team * C::MERGE);
  Team<C::S>& tm = teams[team];
  const int tid = threadIdx.x % (NW * 32), lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;

  if (tid < NW * C::S) mbar_init(&tm.full[tid / C::S][tid % C::S], 1);
  mbar_fence_init();
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  // the first kernel of a call, or after another of the same call: nothing
  // that one writes is read here
  if (a.first) griddep_wait();
  griddep_launch_dependents();

  // ---- the line of units: its length, and where this team's share begins
  const Walk w0 = walk_of(a, tid);  // of sequence tid: all there is in batches up to 128
  int64_t scan = w0.units;          // inclusive over the sequences of the block
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, scan, k);
    if (lane >= k) scan += y;
  }
  int64_t more = 0;
  for (int b = tid + NW * 32; b < a.b.n_seqs; b += NW * 32) more += walk_of(a, b).units;
#pragma unroll
  for (int k = 16; k; k >>= 1) more += __shfl_xor_sync(0xffffffffu, more, k);
  if (lane == 31) {
    tm.n[warp] = scan;
    tm.n[NW + warp] = more;
  }
  team_sync(team);
  int64_t block = 0;
  more = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    if (k < warp) scan += tm.n[k];
    block += tm.n[k];
    more += tm.n[NW + k];
  }
  const int64_t U = (block + more) * a.b.hkv;
  const int ctas = a.divide ? min(shares_of(a, block + more).ctas, (int)gridDim.x) : (int)gridDim.x;
  const int64_t most = (int64_t)kTeams * ctas;
  const int64_t N = U < most ? U : most;
  const int cta = blockIdx.x * kTeams + team;
  if (cta >= N) {
    griddep_wait();
    return;
  }
  const int64_t u0 = share_begin(cta, U, N), u1 = share_begin(cta + 1, U, N);
  Cursor cur;
  int64_t base;  // first unit of the current sequence
  {
    const int64_t want = u0 / a.b.hkv;  // in units of one head: sequence b takes units * hkv
    int64_t before = 0;
    int64_t v = w0.units;
    for (int b0 = 0;;) {
      if (want >= before + scan - v && want < before + scan) {
        tm.v[0] = b0 + tid;
        tm.n[2 * NW] = before + scan - v;
      }
      team_sync(team);
      if (want < before + block) break;
      before += block;
      b0 += NW * 32;
      if (b0 >= a.b.n_seqs) {  // the lengths changed under the call
        griddep_wait();
        return;
      }
      scan = v = walk_of(a, b0 + tid).units;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, k);
        if (lane >= k) scan += y;
      }
      if (lane == 31) tm.n[warp] = scan;
      team_sync(team);
      block = 0;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        if (k < warp) scan += tm.n[k];
        block += tm.n[k];
      }
      team_sync(team);
    }
    cur.b = tm.v[0];
    base = tm.n[2 * NW] * a.b.hkv;
    cur.w = walk_of(a, cur.b);
    const int64_t rem = u0 - base;
    cur.h = (int)(rem / cur.w.units);
    cur.i = (int)(rem % cur.w.units);
  }

  // ---- the warp's ring: its producer runs ahead on the same line
  Cursor ahead = cur;
  int64_t left = u1 - u0;  // units the producer has not passed
  int put = 0, put_n = 0;  // next slot to fill, chunks issued and not yet consumed
  auto produce = [&]() {
    // issue chunks until the ring is full or the share ends
    while (left > 0 && put_n < C::S) {
      const int c = ahead.i * NW + warp;
      if (c < ahead.w.chunks) {
        if (lane == 0) {
          // a chunk lies in one page: pages hold a multiple of 16 tokens
          const int t = chunk_token(ahead.w, c);
          const int64_t r = page_row(a.b, ld_in(a.b.table + (int64_t)ahead.b * a.b.width + (t >> a.b.page_shift)));
          uint64_t* bar = &tm.full[warp][put];
          tm.page_ok[warp][put] = r >= 0;
          if (r >= 0) {
            const int at = (int)r + (ahead.h << a.b.page_shift) + (t & ((1 << a.b.page_shift) - 1));
            const uint32_t st = smem_u32(ring + (warp * C::S + put) * C::STAGE);
            mbar_arrive_expect_tx(bar, C::STAGE);
            tma_rows(st, &kmap, at, bar);
            tma_rows(st + C::HALF, &vmap, at, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        put = put + 1 == C::S ? 0 : put + 1;
        ++put_n;
      }
      ahead.next(a);
      --left;
    }
  };
  produce();

  int get = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait gave up (the whole warp's)
  const int G = 1 << a.b.g_shift;
  int64_t u = u0;
  while (u < u1 && cur.b < a.b.n_seqs) {
    // ---- one stream's part of the share: units [cur.i, i_end) of (b, h)
    const Walk w = cur.w;
    const int h = cur.h, i_begin = cur.i;
    const int64_t stream = base + (int64_t)h * w.units;  // its first unit
    const int i_end = (int)(w.units < i_begin + (u1 - u) ? w.units : i_begin + (u1 - u));
    const int R = w.n << a.b.g_shift;

    uint32_t qf[D / 16][4];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int r = gid + 8 * rr;
      const uint16_t* qp = a.q + (w.t0 + (r >> a.b.g_shift)) * a.q_stride + (h * G + (r & (G - 1))) * D + 2 * tig;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][rr] = r < R ? ld_in(reinterpret_cast<const uint32_t*>(qp + 16 * ks)) : 0u;
        qf[ks][2 + rr] = r < R ? ld_in(reinterpret_cast<const uint32_t*>(qp + 16 * ks + 8)) : 0u;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    const int p_first = w.first;  // local positions (the prefix left out)
    const int p_row[2] = {p_first + (gid >> a.b.g_shift), p_first + ((gid + 8) >> a.b.g_shift)};

    for (int i = i_begin; i < i_end; ++i) {
      const int c = i * NW + warp;
      if (c >= w.chunks) break;
      const int t = chunk_token(w, c);
      if (!dead && !__all_sync(0xffffffffu, bar_wait(&tm.full[warp][get], phase))) {
        // nothing more is copied or multiplied; the warp still counts its
        // streams as done, so that the counters return to zero
        dead = true;
        left = 0;
        if (lane == 0) flag_timeout(a.b.status);
      }
      if (dead) break;
      __syncwarp();
      uint8_t* st = ring + (warp * C::S + get) * C::STAGE;
      const uint32_t kb = smem_u32(st), vb = smem_u32(st + C::HALF);
      // tokens that some query sees; the values of the others are made zero,
      // since 0 * NaN would reach the sum
      const int j = t + (lane & 15);
      const bool live = j < w.len && (j >= w.lo || j < w.sink) && tm.page_ok[warp][get];
      const uint32_t lives = __ballot_sync(0xffffffffu, live) & 0xFFFFu;
      if (lives != 0xFFFFu) {
        if (!live) {
          // half of the row's vectors each of its two lanes
#pragma unroll
          for (int e = 0; e < 4 * C::P; ++e) {
            const int x = (lane >> 4) * 4 * C::P + e;
            *reinterpret_cast<uint4*>(st + C::HALF + (x >> 3) * C::PANEL + (lane & 15) * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // before a later copy into this slot
        __syncwarp();
      }
      float s[2][4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
      const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int c16 = (ks & 3) * 2 + (mi & 1), tok = (mi >> 1) * 8 + mr;
        uint32_t kf[4];
        ldsm_x4(kf, kb + (ks >> 2) * C::PANEL + tok * 128 + ((c16 ^ mr) << 4));
        T::mma(s[0], qf[ks], kf[0], kf[1]);
        T::mma(s[1], qf[ks], kf[2], kf[3]);
      }
      const bool whole = lives == 0xFFFFu && t + kChunk - 1 <= p_first &&
                         (a.window == 0 || t > p_first + w.n - 1 - a.window || t + kChunk <= w.sink);
      if (!whole) {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          // keys of the chunk that the row sees: up to itself, and in its window or among the first
          const int w_lo = a.window > 0 ? p_row[rr] + 1 - a.window : 0;
          const uint32_t see = (lives & low_bits(p_row[rr] + 1 - t) & (~low_bits(w_lo - t) | low_bits(w.sink - t))) >> (2 * tig);
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((see >> (8 * nb + e)) & 1u)) s[nb][2 * rr + e] = -INFINITY;
        }
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float mx = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) mx = fmaxf(mx, fmaxf(s[nb][2 * rr], s[nb][2 * rr + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[rr], fmaf(mx, a.scale_log2, -T::kUp));
        const float mu = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: weights become 0
        const float alpha = ex2(m[rr] - mu);
        m[rr] = mn;
        float sum = 0.f;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float pr = ex2(fmaf(s[nb][2 * rr + e], a.scale_log2, -mu));
            s[nb][2 * rr + e] = pr;
            sum += pr;
          }
        l[rr] = fmaf(l[rr], alpha, sum);
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc) {
          o[cc][2 * rr] *= alpha;
          o[cc][2 * rr + 1] *= alpha;
        }
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const float x = s[f >> 1][2 * (f & 1)], y = s[f >> 1][2 * (f & 1) + 1];
        hi[f] = T::pack(x, y);
        const float2 r = T::unpack(hi[f]);
        lo[f] = T::pack(x - r.x, y - r.y);
      }
#pragma unroll
      for (int cp = 0; cp < D / 16; ++cp) {
        const int tok = (mi & 1) * 8 + mr, c16 = (cp & 3) * 2 + (mi >> 1);
        uint32_t vf[4];
        ldsm_x4_trans(vf, vb + (cp >> 2) * C::PANEL + tok * 128 + ((c16 ^ mr) << 4));
        T::mma(o[2 * cp], hi, vf[0], vf[1]);
        T::mma(o[2 * cp + 1], hi, vf[2], vf[3]);
        T::mma(o[2 * cp], lo, vf[0], vf[1]);
        T::mma(o[2 * cp + 1], lo, vf[2], vf[3]);
      }
      __syncwarp();  // every lane has read the slot
      if (++get == C::S) {
        get = 0;
        phase ^= 1;
      }
      --put_n;
      produce();
    }

    // ---- merge the four warps, kMergeRows rows at a time
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
      if (tig == 0) *reinterpret_cast<float2*>(tm.ml[warp][gid + 8 * rr]) = make_float2(m[rr], l[rr]);
    }
    const bool all = i_begin == 0 && i_end == w.units;
    float* part = a.parts + (int64_t)(2 * cta + (u == u0 ? 0 : 1)) * part_floats(D);
    for (int r0 = 0; r0 < R; r0 += kMergeRows) {
      const int mine = gid - (r0 & 7);
      if (mine >= 0 && mine < kMergeRows) {
        float* dst = merge + (warp * kMergeRows + mine) * C::OSTR + 2 * tig;
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc)
          *reinterpret_cast<float2*>(dst + 8 * cc) =
              r0 < 8 ? make_float2(o[cc][0], o[cc][1]) : make_float2(o[cc][2], o[cc][3]);
      }
      team_sync(team);
      for (int it = tid; it < kMergeRows * (D / 4); it += NW * 32) {
        const int rl = it / (D / 4), r = r0 + rl, c4 = it % (D / 4);
        if (r >= R) break;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < NW; ++k) M = fmaxf(M, tm.ml[k][r][0]);
        const float mu = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          const float f = ex2(tm.ml[k][r][0] - mu);
          const float4 x = *reinterpret_cast<const float4*>(merge + (k * kMergeRows + rl) * C::OSTR + 4 * c4);
          L = fmaf(f, tm.ml[k][r][1], L);
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
        }
        if (all) {
          store_row<T, D>(a, w.t0 + (r >> a.b.g_shift), h * G + (r & (G - 1)), c4, v, M, L);
        } else {
          *reinterpret_cast<float4*>(part + r * D + 4 * c4) = v;
          if (c4 == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(M, L);
        }
      }
      team_sync(team);
    }
    if (!all) {
      // the parts of the stream lie with teams first..last; the last to arrive merges them
      const int first = share_of(stream, U, N), last = share_of(stream + w.units - 1, U, N);
      const int parts = last - first + 1;
      if (tid == 0) tm.v[1] = count_acq_rel(a.counters + first) == (uint32_t)(parts - 1);
      team_sync(team);
      if (tm.v[1]) {
        if (tid == 0) a.counters[first] = 0;
        // a team holds the stream in its first slot unless its share begins before it
        const float* p0 = a.parts + (int64_t)(2 * first + (share_begin(first, U, N) < stream ? 1 : 0)) * part_floats(D);
        const float* p1 = a.parts + (int64_t)(2 * (first + 1)) * part_floats(D);
        auto at = [&](int k) { return k == 0 ? p0 : p1 + (int64_t)(2 * (k - 1)) * part_floats(D); };
        for (int r = warp; r < R; r += NW) {
          float M = -INFINITY, L = 0.f;
          for (int k = lane; k < parts; k += 32) M = fmaxf(M, ld_once(at(k) + kRows * D + 2 * r));
#pragma unroll
          for (int k = 16; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
          const float mu = M == -INFINITY ? 0.f : M;
          for (int k = lane; k < parts; k += 32) {
            const float2 x = ld_once(reinterpret_cast<const float2*>(at(k) + kRows * D + 2 * r));
            L = fmaf(ex2(x.x - mu), x.y, L);
          }
#pragma unroll
          for (int k = 16; k; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
          if (lane == 0) *reinterpret_cast<float2*>(tm.ml[0][r]) = make_float2(M, L);
        }
        team_sync(team);
        for (int it = tid; it < R * (D / 4); it += NW * 32) {
          const int r = it / (D / 4), c4 = it % (D / 4);
          const float M = tm.ml[0][r][0], mu = M == -INFINITY ? 0.f : M;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < parts; ++k) {
            const float4 x = ld_once(reinterpret_cast<const float4*>(at(k) + r * D + 4 * c4));
            const float f = ex2(ld_once(at(k) + kRows * D + 2 * r) - mu);
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
          }
          store_row<T, D>(a, w.t0 + (r >> a.b.g_shift), h * G + (r & (G - 1)), c4, v, M, tm.ml[0][r][1]);
        }
        team_sync(team);
      }
    }
    // ---- on to the next stream of the share
    u += i_end - i_begin;
    if (u < u1) {
      const int64_t seq_units = (int64_t)w.units * a.b.hkv;
      const int b = cur.b;
      cur.i = i_end - 1;
      cur.next(a);
      if (cur.b != b) base += seq_units;
    }
  }
  if (dead) let_copies_land();
  if (!a.first) griddep_wait();
}

template <class T, int D>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas, cudaStream_t s) {
  static_assert(Cfg<D>::SMEM + sizeof(Team<Cfg<D>::S>) * kTeams <= 227 * 1024, "shared memory");
  static_assert(NW * Cfg<D>::S <= NW * 32, "one thread initialises each barrier");
  return launch_pdl<paged_decode_kernel<T, D>>(dim3(ctas), kThreads, Cfg<D>::SMEM, s, km, vm, a);
}

}  // namespace

cudaError_t launch_paged_decode(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas,
                                int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128) return dtype == 0 ? launch<Bf16, 128>(km, vm, a, ctas, s) : launch<Fp16, 128>(km, vm, a, ctas, s);
  return dtype == 0 ? launch<Bf16, 64>(km, vm, a, ctas, s) : launch<Fp16, 64>(km, vm, a, ctas, s);
}

}  // namespace rq
