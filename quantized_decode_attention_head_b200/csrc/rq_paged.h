// Internal declarations of the paged 16-bit cache (append with rotation,
// attention over pages).  Not part of the public C ABI (include/rq.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace rq {

void note_cuda_error(cudaError_t e);  // rq_last_cuda_error (rq_host.cpp)

constexpr int kDeviceIndex = 8;  // == RQ_ERR_DEVICE_INDEX
constexpr int kMaxAxes = 4;

// What every paged kernel needs of a cache's layer and a batch.
struct PagedBatch {
  const int* table;    // [n_seqs][width]
  const int* kv_lens;  // [n_seqs]
  const int* cu;       // [n_seqs + 1] or null
  int n_seqs, n_tokens, width;
  int n_pages, page_shift;  // page_size = 1 << page_shift
  int hq, hkv, g_shift;     // G = 1 << g_shift
  int64_t page_base;        // rows before the layer's first page
  int top;                  // lengths are counted up to here: every position stays below 2^31
  int* status;              // nullable in appends
};

struct PagedAppendArgs {
  PagedBatch b;
  uint16_t* k_pages;
  uint16_t* v_pages;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const uint16_t* q;
  uint16_t* q_out;
  int64_t k_stride, v_stride, q_stride;
  const float* cos_sin;  // null: no rotation
  const int* positions;
  int n_positions, rot, interleaved, n_axes;
  int sections[kMaxAxes];
  int sms;
  int block_tokens;  // tokens of a block (set by the launch)
};

struct PagedAttnArgs {
  PagedBatch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;             // nullable
  float scale_log2;       // softmax scale * log2(e)
  int window;             // 0: none
  int n_sink;
  const int* prefix;      // pages of the shared prefix, or null
  int prefix_len;
  int first;              // first kernel of the call (see rq_paged_launch.h)
  int over_prefix;        // prompt kernel: all rows of the batch over the prefix
  int few_rows_apart;     // sequences of at most kDecodeRows rows are the decode kernel's
  int few_rows_only;      // the call said that no sequence has more than 16 rows a kv head
  int n_ctas;             // SMs that may run the decode kernel's CTAs, of two teams each
  // The decode kernel runs beside the prompt kernel over the prefix (divide):
  int divide;             // both take their shares of n_ctas SMs from the lengths (shares_of)
  int front_ctas;         // CTAs of the prefix, not split
  int max_splits;         // most splits of it: what its grid holds
  float front_units;      // its units
  int* plan;              // the splits that shares_of found, for the merge
  float* parts;           // its partial states: two slots of part_floats(D) a team
  uint32_t* counters;     // one a team: parts of the stream that begins to be split there
  float* rows_o;          // null: results go to out; else partial states of whole rows,
  float* rows_ml;         //   [row_slot][n_tokens][hq][D] and [..][2] (maximum in log2 units, sum)
  int row_slot;
};

constexpr int kMaxCtas = 160;             // of the decode kernel
constexpr int kMaxParts = 2 * kMaxCtas;  // teams among which it divides its work
constexpr int kPromptRows = 256;  // rows of a CTA of the prompt kernel
constexpr int kMaxSplits = 128;   // CTAs among which it splits the keys of the same rows
constexpr int kDecodeRows = 16;  // rows of a kv head that the decode kernel takes
// o[16][D], then (m, l) of each row
__host__ __device__ constexpr int part_floats(int D) { return kDecodeRows * D + 2 * kDecodeRows; }

cudaError_t launch_paged_append(const PagedAppendArgs& a, int head_dim, int dtype, cudaStream_t s);
cudaError_t launch_paged_decode(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas,
                                int head_dim, int dtype, cudaStream_t s);
cudaError_t launch_paged_prompt(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int blocks,
                                int splits, int head_dim, int dtype, cudaStream_t s);
// Merges slots [0, shared) and the rows' own (one of the decode kernel or `own` of the prompt kernel).
cudaError_t launch_paged_merge(const PagedAttnArgs& a, int shared, int own, int head_dim, int dtype, cudaStream_t s);

}  // namespace rq
