// Host side of the paged 16-bit cache: argument checks, workspace layout and
// launches.  See include/rq.h for the contract.
#include <cmath>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "rq.h"
#include "rq_paged.h"

struct rq_paged_cache {
  rq_paged_config cfg;
  int page_shift, g_shift;
  uint16_t *k, *v;
  int sms;
  bool mapped;
  CUtensorMap k16, v16;  // boxes of the decode kernel: all channels of 16 tokens
  CUtensorMap kp, vp;    // boxes of the prompt kernel: 64 channels of a page
};

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return (1 << s) == x ? s : -1;
}

rq_status cuda_status(cudaError_t e) {
  rq::note_cuda_error(e);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}

// Checks what all calls of a batch share and fills the kernels' view of it.
rq_status fill_batch(const rq_paged_cache* c, int layer, const rq_paged_batch* b, rq::PagedBatch& o) {
  if (!c || !b || layer < 0 || layer >= c->cfg.n_layers) return RQ_ERR_INVALID_ARG;
  if (b->n_seqs < 0 || b->n_tokens < 0 || b->max_new < 0 || b->table_width < 1) return RQ_ERR_INVALID_ARG;
  if (b->n_seqs > 0 && (!b->page_table || !b->kv_lens)) return RQ_ERR_INVALID_ARG;
  if (!aligned4(b->page_table) || !aligned4(b->kv_lens) || !aligned4(b->cu_new)) return RQ_ERR_INVALID_ARG;
  if (!b->cu_new && b->n_tokens < b->n_seqs) return RQ_ERR_INVALID_ARG;
  o.table = b->page_table;
  o.kv_lens = b->kv_lens;
  o.cu = b->cu_new;
  o.n_seqs = b->n_seqs;
  o.n_tokens = b->n_tokens;
  o.width = b->table_width;
  o.n_pages = c->cfg.n_pages;
  o.page_shift = c->page_shift;
  o.hq = c->cfg.n_q_heads;
  o.hkv = c->cfg.n_kv_heads;
  o.g_shift = c->g_shift;
  o.top = 0x7FFFFFFF;
  o.page_base = (int64_t)layer * c->cfg.n_pages * c->cfg.n_kv_heads * c->cfg.page_size;
  return RQ_OK;
}

bool good_stride(int64_t stride, int heads, int d) { return stride >= (int64_t)heads * d && stride % 8 == 0; }

// Workspace: status word and plan at its start, then, from the next multiple of 256
// bytes that leaves room for it: counters, the decode kernel's partial states,
// parts of whole rows.  The counters' place does not depend on the batch (they
// are zero between calls, all else is written before it is read), so calls of
// different batches may share a workspace one after another.
constexpr size_t kStatusBytes = 256, kPlanOffset = 64;
constexpr size_t kCounterBytes = (rq::kMaxParts * 4 + 255) / 256 * 256;
size_t parts_bytes(const rq_paged_cache* c) {
  return (size_t)2 * rq::kMaxParts * rq::part_floats(c->cfg.head_dim) * 4;
}

// Rows of partial states that one pass of the prompt kernel may write: its
// splits keep CTAs (256 rows a kv head each) at or below one a SM.
int64_t part_rows(const rq_paged_cache* c, int n_tokens) {
  const int64_t rows = (int64_t)n_tokens * c->cfg.n_q_heads;
  const int64_t most = (int64_t)rq::kMaxCtas * rq::kPromptRows;
  const int64_t split = rows * rq::kMaxSplits < most ? rows * rq::kMaxSplits : most;
  return rows > split ? rows : split;
}

int decode_ctas(const rq_paged_cache* c) { return c->sms < rq::kMaxCtas ? c->sms : rq::kMaxCtas; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The pages as [head_dim / 64][rows][64 channels], read in boxes of `panels`
// panels of `rows` rows of 64 channels (128 bytes, swizzled).
bool encode(EncodeTiled fn, const rq_paged_cache* c, void* base, int box_rows, int panels, CUtensorMap* map) {
  const rq_paged_config& f = c->cfg;
  const cuuint64_t dims[3] = {64, (cuuint64_t)f.n_layers * f.n_pages * f.n_kv_heads * f.page_size,
                              (cuuint64_t)f.head_dim / 64};
  const cuuint64_t strides[2] = {(cuuint64_t)f.head_dim * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)panels};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, f.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims,
            strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The device's size, at the first call.
rq_status find_sms(rq_paged_cache* c) {
  if (c->sms > 0) return RQ_OK;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_status(e);
  c->sms = sms;
  return RQ_OK;
}

// The tensor maps of the pages too, at the first attention call.
rq_status prepare(rq_paged_cache* c) {
  if (c->mapped) return RQ_OK;
  const rq_status st = find_sms(c);
  if (st != RQ_OK) return st;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return cuda_status(e);
  if (!fn || found != cudaDriverEntryPointSuccess) return cuda_status(cudaErrorNotSupported);
  const EncodeTiled enc = reinterpret_cast<EncodeTiled>(fn);
  const int page = c->cfg.page_size, panels = c->cfg.head_dim / 64;
  if (!encode(enc, c, c->k, 16, panels, &c->k16) || !encode(enc, c, c->v, 16, panels, &c->v16) ||
      !encode(enc, c, c->k, page, 1, &c->kp) || !encode(enc, c, c->v, page, 1, &c->vp))
    return cuda_status(cudaErrorInvalidValue);
  c->mapped = true;
  return RQ_OK;
}

// CTAs among which the prompt kernel divides the keys of the same rows: as
// many as fill the device once, while each keeps at least four tiles of 128 keys.
int splits_of(const rq_paged_cache* c, int64_t blocks, int64_t keys, int window, int n_sink, int max_new, int sms) {
  const int64_t ctas = blocks * c->cfg.n_kv_heads;
  if (ctas <= 0) return 1;
  const int64_t reach = (int64_t)window + n_sink + max_new;
  if (window > 0 && reach < keys) keys = reach;
  int64_t s = sms / ctas;
  const int64_t by_work = (keys + 511) / 512;
  if (s > by_work) s = by_work;
  if (s > rq::kMaxSplits) s = rq::kMaxSplits;
  return s < 1 ? 1 : (int)s;
}

rq_status attention(rq_paged_cache* c, int layer, const rq_paged_batch* batch, const int* prefix, int prefix_len,
                    const void* q, int64_t q_stride, void* out, float* lse, float softmax_scale, int window,
                    int n_sink, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  rq::PagedAttnArgs a = {};
  const rq_status st = fill_batch(c, layer, batch, a.b);
  if (st != RQ_OK) return st;
  if (window < 0 || n_sink < 0 || prefix_len < 0 || !(softmax_scale <= 3.0e38f)) return RQ_ERR_INVALID_ARG;
  if (prefix_len > 0 && (!prefix || !aligned4(prefix))) return RQ_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace)) return RQ_ERR_INVALID_ARG;
  if (batch->n_tokens > 0 && (!q || !out || !aligned16(q) || !aligned16(out) || !aligned4(lse) ||
                              !good_stride(q_stride, c->cfg.n_q_heads, c->cfg.head_dim)))
    return RQ_ERR_INVALID_ARG;
  size_t need = 0;
  if (rq_paged_workspace_bytes(c, batch->n_seqs, batch->n_tokens, &need) != RQ_OK) return RQ_ERR_INVALID_ARG;
  if (ws_bytes < need) return RQ_ERR_WORKSPACE;
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return RQ_OK;
  // positions are counted in 32 bits
  const int64_t most = (int64_t)prefix_len + (int64_t)batch->table_width * c->cfg.page_size;
  if (most + batch->n_tokens > 0x7FFFFFFF || (int64_t)batch->n_tokens * 8 > 0x7FFFFFFF) return RQ_ERR_UNSUPPORTED;
  a.b.top = 0x7FFFFFFF - prefix_len - batch->n_tokens;
  if (window > most) window = 0;  // wider than any sequence
  if (n_sink > most) n_sink = (int)most;
  const rq_status pr = prepare(c);
  if (pr != RQ_OK) return pr;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* body = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 2 * kStatusBytes - 1) / kStatusBytes * kStatusBytes);
  a.counters = reinterpret_cast<uint32_t*>(body);
  a.parts = reinterpret_cast<float*>(body + kCounterBytes);
  a.rows_o = a.rows_ml = nullptr;
  a.row_slot = a.over_prefix = 0;
  a.n_ctas = decode_ctas(c);
  a.few_rows_only = (int64_t)batch->max_new << c->g_shift <= rq::kDecodeRows;
  a.b.status = static_cast<int*>(workspace);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt((float)c->cfg.head_dim);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window;
  a.n_sink = n_sink;
  a.prefix = prefix_len > 0 ? prefix : nullptr;
  a.prefix_len = prefix_len;
  const int d = c->cfg.head_dim, type = c->cfg.dtype;
  const int64_t all_rows = (int64_t)batch->n_tokens << c->g_shift;  // of one kv head

  // Which kernels: sequences of at most 16 rows a kv head go to the decode
  // kernel, which splits the tokens evenly whatever the lengths, the others
  // to the prompt kernel; when no sequence can have few rows (one sequence,
  // or all as long as they may be) the decode kernel is not launched.
  const bool decode = a.few_rows_only || (batch->n_seqs > 1 && (int64_t)batch->n_seqs * batch->max_new != batch->n_tokens);
  const bool prompt = !a.few_rows_only;
  a.few_rows_apart = decode;
  int own = 0, shared = 0;
  int64_t blocks = 0;
  if (prompt) {
    const int64_t seqs = decode ? all_rows / (rq::kDecodeRows + 1) : all_rows;  // that can have a block of their own
    blocks = all_rows / rq::kPromptRows + (seqs < batch->n_seqs ? seqs : batch->n_seqs);
    own = splits_of(c, blocks, (int64_t)batch->table_width * c->cfg.page_size, window, n_sink, batch->max_new,
                    decode_ctas(c));
  }
  const int64_t shared_blocks = (all_rows + rq::kPromptRows - 1) / rq::kPromptRows;
  const bool side_by_side = prefix_len > 0 && decode && !prompt;
  int decode_grid = a.n_ctas;
  a.divide = 0;
  if (prefix_len > 0) {
    // no query sees more of the prefix than its window and the first tokens
    const int64_t seen = window > 0 && (int64_t)window + n_sink < prefix_len ? (int64_t)window + n_sink : prefix_len;
    shared = splits_of(c, shared_blocks, seen, 0, 0, 0, a.n_ctas - side_by_side);
    if (side_by_side) {
      // The decode kernel (what follows the prefix) and the prompt kernel (the
      // prefix) run side by side, with grids as large as either share may be;
      // the decode kernel's no larger than its units if all lengths were the
      // tables'.  Where both fit there is nothing to divide (a small call: 14
      // us for 15.5).  Else they divide the SMs by the lengths they find, and
      // blocks left over end at once: 64 sequences behind 32768 tokens take 66
      // us however wide the table; divided by the table's width they took 65
      // with the narrowest table, 231 with one 16 times as wide.
      const int64_t ctas = shared_blocks * c->cfg.n_kv_heads;
      const int64_t units = (int64_t)batch->n_seqs * c->cfg.n_kv_heads * (((int64_t)batch->table_width * c->cfg.page_size + 63) / 64);
      if (units < 2 * decode_grid) decode_grid = (int)(units + 1) / 2;
      a.divide = ctas * shared + decode_grid > a.n_ctas;
      a.front_ctas = ctas < a.n_ctas ? (int)ctas : a.n_ctas;
      a.max_splits = shared;
      a.front_units = (float)(2 * shared_blocks * ((seen + 127) / 128));
      a.plan = reinterpret_cast<int*>(ws + kPlanOffset);
    }
  }
  if (blocks > 0x7FFFFFFF || shared_blocks > 0x7FFFFFFF) return RQ_ERR_UNSUPPORTED;
  const bool merge = shared > 0 || own > 1;
  if (merge) {
    a.rows_o = reinterpret_cast<float*>(body + kCounterBytes + parts_bytes(c));
    a.rows_ml = a.rows_o + 2 * part_rows(c, batch->n_tokens) * d;
  }
  cudaError_t e = cudaSuccess;
  a.first = 1;
  auto run_decode = [&]() {
    rq::PagedAttnArgs f = a;
    f.row_slot = shared;
    if (shared == 0) f.rows_o = f.rows_ml = nullptr;  // straight to out
    e = rq::launch_paged_decode(c->k16, c->v16, f, decode_grid, d, type, stream);
    a.first = 0;
  };
  if (side_by_side) run_decode();  // what it leaves over ends first
  if (e == cudaSuccess && shared > 0) {
    a.over_prefix = 1;
    e = rq::launch_paged_prompt(c->kp, c->vp, a, (int)shared_blocks, shared, d, type, stream);
    a.over_prefix = a.first = 0;
    a.row_slot = shared;
  }
  if (e == cudaSuccess && prompt && blocks > 0) {
    e = rq::launch_paged_prompt(c->kp, c->vp, a, (int)blocks, own, d, type, stream);
    a.first = 0;
  }
  if (e == cudaSuccess && decode && !side_by_side) run_decode();
  if (e == cudaSuccess && merge) e = rq::launch_paged_merge(a, shared, own, d, type, stream);
  return cuda_status(e);
}

}  // namespace

extern "C" {

rq_status rq_paged_cache_init(const rq_paged_config* cfg, void* k_pages, void* v_pages, rq_paged_cache** out) {
  if (!cfg || !k_pages || !v_pages || !out) return RQ_ERR_INVALID_ARG;
  if (cfg->n_layers < 1 || cfg->n_pages < 1 || cfg->n_q_heads < 1 || cfg->n_kv_heads < 1) return RQ_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return RQ_ERR_INVALID_ARG;
  if (cfg->head_dim != 64 && cfg->head_dim != 128) return RQ_ERR_UNSUPPORTED;
  if (cfg->page_size != 16 && cfg->page_size != 32 && cfg->page_size != 64 && cfg->page_size != 128)
    return RQ_ERR_UNSUPPORTED;
  if (cfg->dtype != 0 && cfg->dtype != 1) return RQ_ERR_UNSUPPORTED;
  if (cfg->n_q_heads % cfg->n_kv_heads != 0) return RQ_ERR_UNSUPPORTED;
  const int g = cfg->n_q_heads / cfg->n_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return RQ_ERR_UNSUPPORTED;
  const double rows = (double)cfg->n_layers * cfg->n_pages * cfg->n_kv_heads * cfg->page_size;
  if (rows >= 2147483648.0 || cfg->n_kv_heads > 8192) return RQ_ERR_UNSUPPORTED;
  rq_paged_cache* c = new (std::nothrow) rq_paged_cache();
  if (!c) return RQ_ERR_INVALID_ARG;
  c->cfg = *cfg;
  c->page_shift = log2_of(cfg->page_size);
  c->g_shift = log2_of(g);
  c->k = static_cast<uint16_t*>(k_pages);
  c->v = static_cast<uint16_t*>(v_pages);
  *out = c;
  return RQ_OK;
}

void rq_paged_cache_destroy(rq_paged_cache* cache) { delete cache; }

rq_status rq_paged_append(rq_paged_cache* c, int layer, const rq_paged_batch* batch, const rq_rotation* rot,
                          const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, const void* q,
                          int64_t q_stride, void* q_out, int* dev_status, cudaStream_t stream) {
  rq::PagedAppendArgs a = {};
  const rq_status st = fill_batch(c, layer, batch, a.b);
  if (st != RQ_OK) return st;
  if (!aligned4(dev_status) || (q && !rot)) return RQ_ERR_INVALID_ARG;
  const int d = c->cfg.head_dim;
  if (batch->n_tokens > 0) {
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return RQ_ERR_INVALID_ARG;
    if (!good_stride(k_stride, c->cfg.n_kv_heads, d) || !good_stride(v_stride, c->cfg.n_kv_heads, d))
      return RQ_ERR_INVALID_ARG;
    if (q && (!q_out || !aligned16(q) || !aligned16(q_out) || !good_stride(q_stride, c->cfg.n_q_heads, d)))
      return RQ_ERR_INVALID_ARG;
  }
  if (rot) {
    if (!rot->cos_sin || !aligned16(rot->cos_sin) || rot->n_positions < 1) return RQ_ERR_INVALID_ARG;
    if (rot->rot_dim < 16 || rot->rot_dim > d || rot->rot_dim % 16 != 0) return RQ_ERR_UNSUPPORTED;
    if (rot->n_axes < 1 || rot->n_axes > rq::kMaxAxes) return RQ_ERR_UNSUPPORTED;
    if (!aligned4(rot->positions) || (!rot->positions && rot->n_axes != 1)) return RQ_ERR_INVALID_ARG;
    int64_t sum = 0;
    for (int k = 0; k < rot->n_axes; ++k) {
      if (rot->sections[k] < 0) return RQ_ERR_INVALID_ARG;
      sum += rot->sections[k];
      a.sections[k] = rot->sections[k];
    }
    if (sum != rot->rot_dim / 2) return RQ_ERR_INVALID_ARG;
    a.cos_sin = rot->cos_sin;
    a.positions = rot->positions;
    a.n_positions = rot->n_positions;
    a.rot = rot->rot_dim;
    a.interleaved = rot->interleaved ? 1 : 0;
    a.n_axes = rot->n_axes;
  }
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return RQ_OK;
  const rq_status sized = find_sms(c);
  if (sized != RQ_OK) return sized;
  a.sms = c->sms;
  a.b.status = dev_status;
  a.k_pages = c->k;
  a.v_pages = c->v;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  return cuda_status(rq::launch_paged_append(a, d, c->cfg.dtype, stream));
}

rq_status rq_paged_workspace_bytes(const rq_paged_cache* c, int n_seqs, int n_tokens, size_t* bytes) {
  if (!c || !bytes || n_seqs < 0 || n_tokens < 0) return RQ_ERR_INVALID_ARG;
  // the shared prefix and what follows it are one pass each
  *bytes = 2 * kStatusBytes + kCounterBytes + parts_bytes(c) +
           (size_t)(2 * part_rows(c, n_tokens)) * (c->cfg.head_dim + 2) * 4;
  return RQ_OK;
}

rq_status rq_paged_attention(rq_paged_cache* c, int layer, const rq_paged_batch* batch, const void* q,
                             int64_t q_stride, void* out, float* lse, float softmax_scale, int window, int n_sink,
                             void* workspace, size_t ws_bytes, cudaStream_t stream) {
  return attention(c, layer, batch, nullptr, 0, q, q_stride, out, lse, softmax_scale, window, n_sink, workspace,
                   ws_bytes, stream);
}

rq_status rq_paged_shared_attention(rq_paged_cache* c, int layer, const rq_paged_batch* batch,
                                    const int* prefix_pages, int prefix_len, const void* q, int64_t q_stride,
                                    void* out, float* lse, float softmax_scale, int window, int n_sink,
                                    void* workspace, size_t ws_bytes, cudaStream_t stream) {
  return attention(c, layer, batch, prefix_pages, prefix_len, q, q_stride, out, lse, softmax_scale, window, n_sink,
                   workspace, ws_bytes, stream);
}

}  // extern "C"
