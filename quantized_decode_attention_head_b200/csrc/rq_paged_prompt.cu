// Attention of many query rows over the paged 16-bit cache (sm_100a): prompts
// and pieces of prompts, and all queries of a batch over the prefix they share.
//
// A CTA takes 256 query rows of one kv head (two tiles of 128; a row is a
// token and one of the G heads, so the heads of a group share every key they
// read) and walks over tiles of 128 keys.  Both products run on tcgen05 with
// the accumulators in TMEM:
//   S_t = Q_t K^T     (A and B from shared memory, K-major)
//   O_t += P_t V      (A = P_t from TMEM, B = V from shared memory, MN-major)
// One warp issues TMA copies of the pages (64-channel boxes, 128-byte swizzle),
// one warp issues the MMAs, and a group of four warps per tile does the
// softmax, one thread a row: no shuffles.  The MMA warp alternates between the
// tiles, so one tile's products run while the other's weights are computed.
// P_t overwrites S_t (16-bit pairs, half its columns).  TMEM columns:
// [S_0 | S_1 | O_0 | O_1].  The running maximum moves only when a row's scores
// exceed it by 2^8, so O is rarely rescaled.  Weights are rounded
// once to 16 bits, half a step of the type, where they enter the product.  A
// second term fits the columns that P leaves free and makes the error that of
// the result's own rounding (8192-token prompt: rms 1.08e-4, with one term
// 1.42e-4), but adds half to the tensor work: 602 us for 451, 64 sequences
// behind 32768 tokens 82 for 67.  Sums are fp32 of the unrounded weights.
//
// Bound.  At D = 128 a step (256 rows, 128 keys) is 2048 clocks of tensor work
// and as many of exponentials (16 a clock an SM).  Measured (8192-token prompt,
// 4096-token window, 32/8 heads, in a loop, at the 1 kW power cap): 450 to 460 us,
// 895 TFLOP/s of visible pairs, about 3400 clocks a step.  With the softmax taken
// out the step still takes 2830:
// queries, keys and values read by the MMAs and written by TMA are 256 KB of
// shared-memory traffic, 128 bytes a clock; the rest is TMEM traffic of the
// softmax beside the MMAs.  A block starts in about 5 us (rows, first keys)
// and stores in 2 to 3.
#include <cuda.h>

#include <climits>

#include "rq_paged.cuh"
#include "rq_paged_launch.h"

namespace rq {
namespace {

constexpr int kTileRows = 128;
constexpr int kBlockRows = kPromptRows;
constexpr int kKeys = 128;  // keys a step
constexpr int kThreads = 384;
static_assert(kBlockRows == 2 * kTileRows, "two tiles a CTA");

template <int D>
struct Cfg {
  static constexpr int P = D / 64;                  // 64-channel panels
  static constexpr int PANEL = 128 * 128;           // bytes: 128 rows of 64 channels
  static constexpr int TILE = P * PANEL;
  static constexpr int NS = D == 128 ? 2 : 4;       // stages of keys, and of values
  static constexpr int SMEM = 1024 + 2 * TILE + 2 * NS * TILE;
  static constexpr int COLS = 512;                  // TMEM columns: 2 x 128 (S) + 2 x D (O), up to a power of two
};

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// One lane of the warp (the same at every call).  The MMAs and commits below
// are predicated on it: the flow stays uniform, and with it the compiler keeps
// descriptors and addresses in uniform registers.  (A 128 x 128 x 16 MMA takes
// 64 clocks, and issuing blocks after about four; a commit is seen some 300
// clocks after the last MMA began.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}
// Arrives on bar when every tcgen05 operation that the lane issued before is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
// D += A B (D = A B unless acc).  Descriptors come as (low, high) words: only
// the low one, the address, varies.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc,
                                       uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((int)acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc,
                                       uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 b, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((int)acc), "r"(one)
      : "memory");
}

#define RQ_OUT(i) "=r"(r[i])
#define RQ_IN(i) "r"(r[i])
#define RQ_TIE(i) "+r"(r[i])
#define RQ_32(M)                                                                                                    \
  M(0), M(1), M(2), M(3), M(4), M(5), M(6), M(7), M(8), M(9), M(10), M(11), M(12), M(13), M(14), M(15), M(16),      \
      M(17), M(18), M(19), M(20), M(21), M(22), M(23), M(24), M(25), M(26), M(27), M(28), M(29), M(30), M(31)

// 32 columns of this thread's TMEM lane (the warp's 32 lanes at addr).
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];\n"
      : RQ_32(RQ_OUT)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31};\n" ::RQ_32(RQ_IN),
      "r"(addr)
      : "memory");
}

// Waits for this thread's TMEM loads.  The loaded registers pass through, so
// that no use of them can be moved before the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" : RQ_32(RQ_TIE)::"memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  Low word: address and
// leading stride; high word: stride of 8 rows (1024 bytes), version, swizzle.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t kDescHi = 1024 >> 4 | 1u << 14 | 2u << 29;
// Instruction descriptor: fp32 accumulator, A and B of the pages' type (0
// fp16, 1 bf16), B K-major or MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int type, bool b_mn, int m, int n) {
  return 1u << 4 | (uint32_t)type << 7 | (uint32_t)type << 10 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(m >> 4) << 24;
}

// A page's rows from row y on, 64 channels (panel p).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int p, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(y), "r"(p), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A warp's wait: all lanes go on, or none (the tcgen05 accesses need the whole warp).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity));
}

// Barrier of the MMA warp and the softmax warps.
__device__ __forceinline__ void named_barrier() { asm volatile("bar.sync 1, 288;\n" ::: "memory"); }

// Eight words to a 32-byte boundary.
__device__ __forceinline__ void st_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

struct Shared {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_ready[2][2], o_final[2];  // p_ready: halves of a tile's keys
  uint32_t tmem;
  int seq, block;          // the CTA's sequence and row block in it
  int row_token[kBlockRows];  // packed token, -1: no row
  int row_p[kBlockRows];      // position of the row's query
  int p_min[8], p_max[8];     // of each warp's 32 rows
  int64_t tail[4];         // units of the decode kernel, by the warp that counted them
  int splits;
  int dead;
  int bad;  // a page number out of range in the CTA's walk
};

// The keys a CTA walks over, as tokens of its page list: tiles [0, ns) and
// [lo_t, lo_t + tiles - ns), of which this split takes [t0, t1).
struct Keys {
  int base;  // position of key 0
  int end;   // keys there are
  int lo, hi, sink;  // keys [lo, hi) and [0, sink) are seen by some row
  int ns, lo_t, t0, t1;
  const int* pages;
  // Does some row see a key of the page (of ps keys) that begins at key j?
  // Other pages are not looked up, though a tile may reach over them: they may
  // have been freed.
  __device__ __forceinline__ bool needs(int j, int ps) const {
    return j < sink || (j < hi && j > lo - ps && lo < hi);
  }
};
__device__ __forceinline__ int key_of(const Keys& k, int tile) {
  return kKeys * (tile < k.ns ? tile : k.lo_t + tile - k.ns);
}

// kPrefix: all rows of the batch over the prefix (two kernels: what one of them
// does not need costs the other registers, which its softmax has none to spare of).
template <class T, int D, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_sm = smem_u32(sm), k_sm = q_sm + 2 * C::TILE, v_sm = k_sm + C::NS * C::TILE;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const int h = blockIdx.y, G = 1 << a.b.g_shift;

  // the first kernel of a call, or after another of the same call: nothing
  // that one writes is read here before it ends
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (a.first) griddep_wait();
  griddep_launch_dependents();

  // ---- which rows
  int row0 = 0, rows = 0;
  Seq seq = {};
  if (kPrefix) {
    row0 = blockIdx.x * kBlockRows;
    rows = a.b.n_tokens << a.b.g_shift;
  } else {
    // the last blocks first: they see the most keys
    const int want = gridDim.x - 1 - blockIdx.x;
    if (warp == 0) {
      int before = 0, found = -1, block = 0;
      for (int b0 = 0; b0 < a.b.n_seqs && found < 0; b0 += 32) {
        int x = 0;
        if (b0 + lane < a.b.n_seqs) {
          const Seq s = load_seq(a.b, b0 + lane);
          const int r = s.n << a.b.g_shift;
          if (!(a.few_rows_apart && r <= kDecodeRows)) x = (r + kBlockRows - 1) / kBlockRows;
        }
        const int v = x;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, k);
          if (lane >= k) x += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, want >= before + x - v && want < before + x);
        if (hit) {
          const int src = __ffs(hit) - 1;
          found = b0 + src;
          block = want - before - __shfl_sync(0xffffffffu, x - v, src);
        }
        before += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) {
        sh.seq = found;
        sh.block = block;
      }
    }
    __syncthreads();
    if (sh.seq < 0) {
      griddep_wait();
      return;
    }
    seq = load_seq(a.b, sh.seq);
    row0 = sh.block * kBlockRows;
    rows = seq.n << a.b.g_shift;
  }
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_ready[t][0], 4);
      mbar_init(&sh.p_ready[t][1], 4);
      mbar_init(&sh.o_final[t], 1);
    }
    mbar_fence_init();
    sh.dead = 0;
    sh.bad = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sh.tmem)),
                 "r"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  if (tid < kBlockRows) {
    const int r = row0 + tid;
    int token = -1, p = 0;
    if (r < rows) {
      token = r >> a.b.g_shift;
      if (kPrefix) {
        const int b = seq_of(a.b, token);
        if (b >= 0) {
          const Seq s = load_seq(a.b, b);
          if (token >= s.t0 && token < s.t0 + s.n)
            p = a.prefix_len + s.end - s.n + (token - s.t0);
          else
            token = -1;
        } else {
          token = -1;
        }
      } else {
        p = a.prefix_len + seq.end - seq.n + token;
        token += seq.t0;
      }
    }
    sh.row_token[tid] = token;
    sh.row_p[tid] = p;
    int lo = token >= 0 ? p : INT_MAX - 1, hi = token >= 0 ? p : INT_MIN;
#pragma unroll
    for (int k = 16; k; k >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, k));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, k));
    }
    if (lane == 0) {
      sh.p_min[warp] = lo;
      sh.p_max[warp] = hi;
    }
  }
  if (kPrefix && a.divide && warp >= 8) {
    int64_t units = 0;
    for (int b = tid - 256; b < a.b.n_seqs; b += 128) units += walk_of(a, b).units;
#pragma unroll
    for (int k = 16; k; k >>= 1) units += __shfl_xor_sync(0xffffffffu, units, k);
    if (lane == 0) sh.tail[warp - 8] = units;
    asm volatile("bar.sync 2, 128;\n" ::: "memory");
    if (tid == 256) {
      sh.splits = shares_of(a, sh.tail[0] + sh.tail[1] + sh.tail[2] + sh.tail[3]).splits;
      if (blockIdx.x + blockIdx.y + blockIdx.z == 0) *a.plan = sh.splits;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int splits = kPrefix && a.divide ? sh.splits : (int)gridDim.z;
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  int p_lo[2], p_hi[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    p_lo[t] = min(min(sh.p_min[4 * t], sh.p_min[4 * t + 1]), min(sh.p_min[4 * t + 2], sh.p_min[4 * t + 3]));
    p_hi[t] = max(max(sh.p_max[4 * t], sh.p_max[4 * t + 1]), max(sh.p_max[4 * t + 2], sh.p_max[4 * t + 3]));
  }
  // row tiles with any row; none where the SM is the decode kernel's
  const int tiles_q = kPrefix && (int)blockIdx.z >= splits ? 0 : (p_hi[1] != INT_MIN ? 2 : (p_hi[0] != INT_MIN ? 1 : 0));

  // ---- which keys
  Keys key;
  key.base = kPrefix ? 0 : a.prefix_len;
  key.end = kPrefix ? a.prefix_len : seq.len;
  key.pages = kPrefix ? a.prefix : a.b.table + (int64_t)sh.seq * a.b.width;
  {
    const int first = min(p_lo[0], p_lo[1]), last = max(p_hi[0], p_hi[1]);
    int hi = tiles_q ? last + 1 - key.base : 0;
    hi = hi < 0 ? 0 : (hi > key.end ? key.end : hi);
    int lo = a.window > 0 && tiles_q ? first + 1 - a.window - key.base : 0;
    lo = lo < 0 ? 0 : (lo > hi ? hi : lo);
    int sink = a.window > 0 ? a.n_sink - key.base : 0;
    key.sink = sink < 0 ? 0 : (sink > hi ? hi : sink);
    key.lo = lo;
    key.hi = hi;
    key.lo_t = lo / kKeys;
    const int st = (key.sink + kKeys - 1) / kKeys;
    key.ns = st < key.lo_t ? st : key.lo_t;
    const int n = key.ns + (hi + kKeys - 1) / kKeys - key.lo_t;
    key.t0 = (int)((int64_t)n * blockIdx.z / splits);
    key.t1 = (int)((int64_t)n * (blockIdx.z + 1) / splits);
  }
  const int n_steps = key.t1 - key.t0;

  // registers: launched with 168 a thread (64512); 64 + 2 * 216 a lane of the three groups are 63488
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
  if (n_steps > 0) {
    if (warp == 0) {
      // ------------------------------------------------ producer
      if (lane == 0) {
        const int per = kKeys >> a.b.page_shift, ps = 1 << a.b.page_shift;
        const int head_row = h << a.b.page_shift;
        bool ok = true;
        for (int k = 0; k < n_steps && ok; ++k) {
          const int slot = k % C::NS;
          const uint32_t par = ((k / C::NS) & 1) ^ 1;
          const int j = key_of(key, key.t0 + k);
          int row[8];
          uint32_t bytes = 0;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            row[g] = -1;
            const int jj = j + (g << a.b.page_shift);
            if (g < per && key.needs(jj, ps)) {
              const int64_t r = page_row(a.b, ld_in(key.pages + (jj >> a.b.page_shift)));
              if (r >= 0) {
                row[g] = (int)r + head_row;
                bytes += ps * D * 2;
              }
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2 && ok; ++kv) {
            uint64_t* full = kv ? &sh.v_full[slot] : &sh.k_full[slot];
            ok = bar_wait(kv ? &sh.v_empty[slot] : &sh.k_empty[slot], par);
            if (!ok) break;
            if (bytes)
              mbar_arrive_expect_tx(full, bytes);
            else
              mbar_arrive(full);
            const uint32_t dst = (kv ? v_sm : k_sm) + slot * C::TILE;
#pragma unroll
            for (int g = 0; g < 8; ++g)
              if (row[g] >= 0) {
#pragma unroll
                for (int p = 0; p < C::P; ++p)
                  tma_box(dst + p * C::PANEL + (g << a.b.page_shift) * 128, kv ? &vmap : &kmap, p, row[g], full);
              }
          }
        }
        if (!ok) sh.dead = 1;
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issue
      constexpr uint32_t id_s = instr_desc(T::kType, false, kTileRows, kKeys);
      constexpr uint32_t id_o = instr_desc(T::kType, true, kTileRows, D);
      const uint32_t q_desc = desc_lo(q_sm, 16), k_desc = desc_lo(k_sm, 16), v_desc = desc_lo(v_sm, C::PANEL);
      const uint32_t one = elect_one();
      named_barrier();  // the queries are in shared memory
      const bool any_bad = sh.bad != 0;
      auto scores = [&](int t, int slot) {
        const uint32_t qd = q_desc + t * (C::TILE >> 4), kd = k_desc + slot * (C::TILE >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          constexpr int kPanel16 = C::PANEL >> 4;
          const uint32_t off = (ks >> 2) * kPanel16 + (ks & 3) * 2;
          mma_ss(tmem + t * kKeys, qd + off, kd + off, kDescHi, id_s, ks > 0, one);
        }
        tc_commit(&sh.s_full[t], one);
      };
      bool ok = warp_wait(&sh.k_full[0], 0);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < tiles_q; ++t) scores(t, 0);
        tc_commit(&sh.k_empty[0], one);
      }
      for (int k = 0; k < n_steps && ok; ++k) {
        const int slot = k % C::NS, next = (k + 1) % C::NS;
        for (int t = 0; t < tiles_q && ok; ++t) {
          if (t == 0) {
            ok = warp_wait(&sh.v_full[slot], (k / C::NS) & 1);
            // values that no row sees become zero: 0 * NaN would reach the sums
            const int j = key_of(key, key.t0 + k);
            if (ok && (any_bad || j + kKeys > key.hi || (j < key.lo && j + kKeys > key.sink))) {
              for (int i = lane; i < kKeys; i += 32) {
                const int jj = j + i;
                bool live = jj < key.hi && (jj >= key.lo || jj < key.sink);
                if (live && any_bad) live = page_row(a.b, ld_in(key.pages + (jj >> a.b.page_shift))) >= 0;
                if (!live)
#pragma unroll
                  for (int c = 0; c < C::P * 8; ++c)
                    *reinterpret_cast<uint4*>(sm + (v_sm - q_sm) + slot * C::TILE + (c >> 3) * C::PANEL + i * 128 +
                                              (c & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && warp_wait(&sh.p_ready[t][half], k & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t vd = v_desc + slot * (C::TILE >> 4);
#pragma unroll
            for (int kt = 4 * half; kt < 4 * half + 4; ++kt)
              mma_ts(tmem + 2 * kKeys + t * D, tmem + t * kKeys + kt * 8, vd + kt * (2048 >> 4), kDescHi, id_o,
                     k > 0 || kt > 0, one);
          }
          if (!ok) break;
          if (t == tiles_q - 1) tc_commit(&sh.v_empty[slot], one);
          if (k + 1 < n_steps) {
            if (t == 0) {
              ok = warp_wait(&sh.k_full[next], ((k + 1) / C::NS) & 1);
              if (!ok) break;
              tc_fence_after();
            }
            scores(t, next);
            if (t == tiles_q - 1) tc_commit(&sh.k_empty[next], one);
          } else {
            tc_commit(&sh.o_final[t], one);
          }
        }
      }
      if (!ok && lane == 0) sh.dead = 1;
    }
  }
  if (warp >= 4 && n_steps > 0) {
    // ---- queries to shared memory, in the layout a TMA copy would give them:
    // each warp the 32 rows whose softmax it does, all loads in flight at once
    constexpr int kVec = D / 8, kRowsAt = 32 / kVec, kLoads = 32 / kRowsAt;  // 16-byte vectors of a row, rows a load
    const int r0 = (warp - 4) * 32;
    if (r0 < tiles_q * kTileRows) {
      uint4 x[kLoads];
      const int c = lane % kVec;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kRowsAt + lane / kVec;
        const int token = sh.row_token[r];
        x[i] = make_uint4(0, 0, 0, 0);
        if (token >= 0)
          x[i] = ld_once(reinterpret_cast<const uint4*>(a.q + token * a.q_stride + (h * G + ((row0 + r) & (G - 1))) * D) + c);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kRowsAt + lane / kVec, rr = r & (kTileRows - 1);
        *reinterpret_cast<uint4*>(sm + (r / kTileRows) * C::TILE + (c >> 3) * C::PANEL + rr * 128 +
                                  (((c & 7) ^ (rr & 7)) << 4)) = x[i];
      }
    }
    // ---- page numbers out of range anywhere in the walk: the masked path
    const int per = kKeys >> a.b.page_shift;  // pages a tile
    for (int i = tid - 128; i < n_steps * per; i += 256) {
      const int j = key_of(key, key.t0 + i / per) + ((i % per) << a.b.page_shift);
      if (key.needs(j, 1 << a.b.page_shift) && page_row(a.b, ld_in(key.pages + (j >> a.b.page_shift))) < 0) sh.bad = 1;
    }
    fence_proxy_async_smem();
    named_barrier();
  }
  if (warp >= 4 && (warp - 4) / 4 < tiles_q) {
    const bool any_bad = sh.bad != 0;
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
    // -------------------------------------------------- softmax, one row a thread
    const int t = (warp - 4) / 4;
    const int r = t * kTileRows + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + t * kKeys + lanes, o_at = tmem + 2 * kKeys + t * D + lanes;
    // every row of the tile sees all keys of (all_lo, all_end)
    const int all_end = min(key.end, p_lo[t] + 1 - key.base);
    const int all_lo = a.window > 0 && p_hi[t] != INT_MIN ? p_hi[t] - a.window - key.base : INT_MIN;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int k = 0; k < n_steps; ++k) {
      const int j = key_of(key, key.t0 + k);
      ok = warp_wait(&sh.s_full[t], k & 1);
      if (!ok) break;
      tc_fence_after();
      const bool whole = !any_bad && j + kKeys <= all_end && (j > all_lo || j + kKeys <= key.sink);
      if (__any_sync(0xffffffffu, !whole)) {
        // masked in place, 32 columns at a time: a CTA meets one to three such
        // tiles, and code unrolled over 128 columns cost more to fetch than to run
        // keys the row sees: [w_lo, limit) and [0, sink), the latter below limit too
        const int p = sh.row_p[r] - key.base;
        const int limit = sh.row_token[r] >= 0 ? min(key.end, p + 1) : 0;
        const int w_lo = a.window > 0 ? p + 1 - a.window : 0;
        uint32_t pages = 0xFFu;  // bit g: the page of keys 16 g.. of the tile was loaded
        if (any_bad) {
          pages = 0;
          for (int g = 0; g < 8; ++g) {
            const int jj = j + 16 * g;
            const int first = jj >> a.b.page_shift << a.b.page_shift;
            if (key.needs(first, 1 << a.b.page_shift) && page_row(a.b, ld_in(key.pages + (jj >> a.b.page_shift))) >= 0) pages |= 1u << g;
          }
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          // seen: below the limit, and in the window or among the first tokens
          const int j0 = j + 32 * c;
          uint32_t see = low_bits(limit - j0) & (~low_bits(w_lo - j0) | low_bits(key.sink - j0));
          see &= ((pages >> (2 * c)) & 1u ? 0xFFFFu : 0u) | ((pages >> (2 * c + 1)) & 1u ? 0xFFFF0000u : 0u);
          uint32_t x[32];
          tc_ld32(x, s_at + 32 * c);
          tc_wait_ld(x);
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = (see >> e) & 1u ? x[e] : 0xFF800000u;
          tc_st32(s_at + 32 * c, x);
        }
        tc_wait_st();
      }
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc_ld32(s[c], s_at + 32 * c);
#pragma unroll
      for (int c = 0; c < 4; ++c) tc_wait_ld(s[c]);
      float mx4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx4[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int e = 1; e < 31; e += 2) mx4[c] = max3(mx4[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        mx4[c] = fmaxf(mx4[c], __uint_as_float(s[c][31]));
      }
      float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
      mx = fmaf(mx, a.scale_log2, -T::kUpLag);
      const bool move = mx > m + T::kLag;  // true at the first score of a row (m = -inf)
      if (__any_sync(0xffffffffu, move)) {
        const float mn = move ? mx : m;
        const float alpha = move ? ex2(m - mn) : 1.f;
        m = mn;
        l *= alpha;
        if (k > 0) {
          // the product before this step's scores is complete (s_full follows it)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc_ld32(o, o_at + 32 * c);
            tc_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc_st32(o_at + 32 * c, o);
          }
        }
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mu2 = make_float2(-mu, -mu);
      // weights of 64 keys at a time, so that their product starts while the
      // other half's are computed; the first half's store completes under the
      // first weights of the second
      auto weights = [&](int half, int e, uint32_t(&w)[32]) {
        uint32_t &x = s[2 * half + e / 16][2 * (e % 16)], &y = s[2 * half + e / 16][2 * (e % 16) + 1];
        const float2 d = __ffma2_rn(make_float2(__uint_as_float(x), __uint_as_float(y)), sc2, mu2);
        const float2 p = make_float2(ex2(d.x), ex2(d.y));
        x = __float_as_uint(p.x);
        y = __float_as_uint(p.y);
        w[e] = T::pack(p.x, p.y);
      };
      auto hand_over = [&](int half) {
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[t][half]);
      };
      uint32_t w0[32], w1[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) weights(0, e, w0);
      tc_st32(s_at, w0);
#pragma unroll
      for (int e = 0; e < 8; ++e) weights(1, e, w1);
      hand_over(0);
#pragma unroll
      for (int e = 8; e < 32; ++e) weights(1, e, w1);
      tc_st32(s_at + 32, w1);
      hand_over(1);
      // the row's sum, off the way to the products
      float2 sum[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sum[c] = make_float2(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2)
          sum[c] = __fadd2_rn(sum[c], make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])));
      }
      const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
      l += all.x + all.y;
    }
    if (ok && n_steps > 0) {
      ok = warp_wait(&sh.o_final[t], 0);
      tc_fence_after();
    }
    if (!ok) sh.dead = 1;
    const int token = sh.row_token[r];
    const int64_t row = (int64_t)token * a.b.hq + h * G + ((row0 + r) & (G - 1));
    const int64_t at = (int64_t)(a.row_slot + blockIdx.z) * a.b.n_tokens * a.b.hq + row;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (n_steps > 0) {
        tc_ld32(o, o_at + 32 * c);
        tc_wait_ld(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if (ok && token >= 0) {
        if (a.rows_o) {
#pragma unroll
          for (int e = 0; e < 4; ++e) st_v8(a.rows_o + at * D + 32 * c + 8 * e, o + 8 * e);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = l == 0.f ? 0u : T::pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(a.out + row * D + 32 * c + 8 * e) =
                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
    }
    if (ok && token >= 0) {
      if (a.rows_o)
        *reinterpret_cast<float2*>(a.rows_ml + 2 * at) = make_float2(m, l);
      else if (a.lse)
        a.lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (sh.dead) {
    // a wait gave up: report it
    if (tid == 0) {
      flag_timeout(a.b.status);
      let_copies_land();
    }
    __syncthreads();
  }
  if (!a.first) griddep_wait();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::COLS));
}

// Rows whose state lies in parts: slots [0, shared) of every row (as many of
// them as the plan says, where the SMs were divided), then, from slot `shared`
// on, one of the decode kernel or `own` of the prompt kernel.  One warp a
// row; the parts of a row are read in order, so results do not depend on
// timing.
template <class T, int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ PagedAttnArgs a, int shared, int own) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t n_rows = (int64_t)a.b.n_tokens * a.b.hq;
  griddep_launch_dependents();
  if (row >= n_rows) {
    griddep_wait();
    return;
  }
  const int token = (int)(row / a.b.hq);
  const int b = seq_of(a.b, token);
  const Seq s = b >= 0 ? load_seq(a.b, b) : Seq{};
  griddep_wait();
  if (token < s.t0 || token >= s.t0 + s.n) return;  // no sequence's
  const bool few = a.few_rows_apart && (s.n << a.b.g_shift) <= kDecodeRows;
  if (few && shared == 0) return;  // the decode kernel wrote the result
  const int over = a.divide ? ld_once(a.plan) : shared, skip = shared - over;
  const int slots = over + (few ? 1 : own);
  auto slot = [&](int k) { return (int64_t)(k < over ? k : k + skip) * n_rows + row; };
  float M = -INFINITY;
  for (int k = lane; k < slots; k += 32) M = fmaxf(M, ld_once(a.rows_ml + 2 * slot(k)));
#pragma unroll
  for (int k = 16; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  const float mu = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  constexpr int E = D / 32;
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
  // (a part that saw nothing holds zeros and the maximum -inf: weight 0); eight
  // parts' loads in flight at once
  constexpr int kAtOnce = 8;
  for (int k0 = 0; k0 < slots; k0 += kAtOnce) {
    float2 x[kAtOnce];
    float o[kAtOnce][E];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      x[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.f;
      if (k0 + i < slots) {
        const int64_t at = slot(k0 + i);
        x[i] = ld_once(reinterpret_cast<const float2*>(a.rows_ml + 2 * at));
        if constexpr (E == 4) {
          const float4 y = ld_once(reinterpret_cast<const float4*>(a.rows_o + at * D) + lane);
          o[i][0] = y.x, o[i][1] = y.y, o[i][2] = y.z, o[i][3] = y.w;
        } else {
          const float2 y = ld_once(reinterpret_cast<const float2*>(a.rows_o + at * D) + lane);
          o[i][0] = y.x, o[i][1] = y.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float f = ex2(x[i].x - mu);
      L = fmaf(f, x[i].y, L);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf(f, o[i][e], v[e]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = T::pack(v[2 * e] * inv, v[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
}

template <class T, int D>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int blocks, int splits,
                   cudaStream_t s) {
  static_assert(Cfg<D>::SMEM + sizeof(Shared) + 64 <= 227 * 1024, "shared memory");
  const dim3 grid(blocks, a.b.hkv, splits);
  return a.over_prefix ? launch_pdl<paged_prompt_kernel<T, D, true>>(grid, kThreads, Cfg<D>::SMEM, s, km, vm, a)
                       : launch_pdl<paged_prompt_kernel<T, D, false>>(grid, kThreads, Cfg<D>::SMEM, s, km, vm, a);
}

template <class T, int D>
cudaError_t merge(const PagedAttnArgs& a, int shared, int own, cudaStream_t s) {
  const int64_t rows = (int64_t)a.b.n_tokens * a.b.hq;
  return launch_pdl<paged_merge_kernel<T, D>>(dim3((unsigned)((rows + 3) / 4)), 128, 0, s, a, shared, own);
}

}  // namespace

cudaError_t launch_paged_prompt(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int blocks,
                                int splits, int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128)
    return dtype == 0 ? launch<Bf16, 128>(km, vm, a, blocks, splits, s) : launch<Fp16, 128>(km, vm, a, blocks, splits, s);
  return dtype == 0 ? launch<Bf16, 64>(km, vm, a, blocks, splits, s) : launch<Fp16, 64>(km, vm, a, blocks, splits, s);
}

cudaError_t launch_paged_merge(const PagedAttnArgs& a, int shared, int own, int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128) return dtype == 0 ? merge<Bf16, 128>(a, shared, own, s) : merge<Fp16, 128>(a, shared, own, s);
  return dtype == 0 ? merge<Bf16, 64>(a, shared, own, s) : merge<Fp16, 64>(a, shared, own, s);
}

}  // namespace rq
