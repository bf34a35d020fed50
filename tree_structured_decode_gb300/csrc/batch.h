// Parameter blocks and launchers of the operators whose lengths live on the
// GPU: page tables, append by slot, shared-prefix attention, sampling.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ta {

// Element types of the C ABI (tree_attn_dtype).
enum { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

constexpr int kPage = 16;           // tokens per page
constexpr unsigned kMaxPages = 1u << 27;  // a slot number (page * 16 + place) stays below 2^31
constexpr int kMaxRequests = 16384; // three scans of a batch stay in shared memory

// Bits of the status word (TREE_ATTN_BATCH_* of the C ABI).
enum { kBatchNoPages = 1, kBatchTableFull = 2, kBatchBadInput = 4, kBatchBadSlot = 8,
       kBatchTimeout = 16 };

struct ExtendParams {
  int32_t* lens;
  const int32_t* n_new;
  int32_t* table;
  long long table_stride;
  int32_t* free_pages;
  int32_t* n_free;
  int32_t *slots, *positions, *cu_new, *status;
  int n_req, width, free_cap, max_new, position_base;
};
cudaError_t launch_extend_tables(const ExtendParams& p, cudaStream_t s);

struct AppendSlotsParams {
  const uint16_t *k_new, *v_new;
  long long k_stride, v_stride;  // elements from one token to the next
  const int32_t* slots;
  uint16_t *k_pages, *v_pages;
  int32_t* status;
  long long n_slots;             // num_pages * 16
  int n_tokens, hkv, d;
};
cudaError_t launch_append_slots(const AppendSlotsParams& p, cudaStream_t s);

struct PrefixParams {
  const uint16_t* q;
  long long q_stride;            // elements from one token to the next
  const uint16_t *k_pages, *v_pages;
  const int32_t* table;
  long long table_stride;
  const int32_t* lens;
  const int32_t* cu;             // tokens before each request; null: one each
  const int32_t* prefix_pages;
  uint16_t* out;                 // [tokens][hq][d], q's type
  float* lse;                    // [tokens][hq] natural log, or null
  int32_t* status;
  int width, prefix_len, n_tokens, n_req, hq, hkv, gqa, d, num_pages, dtype, num_sms;
  float scale_log2;              // softmax scale * log2(e)
};
// Workspace of a run; 0 where there is nothing to do.
size_t prefix_workspace(const PrefixParams& p);
cudaError_t launch_prefix_attention(const PrefixParams& p, void* workspace, cudaStream_t s);

constexpr int kMaxVocab = 262144;
struct SampleParams {
  const void* logits;            // [rows][vocab], rows `stride` elements apart
  long long stride;
  int dtype, rows, vocab, draws;
  const float* u;                // [rows][draws]
  // per row, or one value for all where the pointer is null
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  int32_t* tokens;               // [rows][draws]
  float* logprobs;               // [rows][draws] or null
  int num_sms;
  int slice, held;               // logits of a CTA, whether in shared memory (set by the launch)
};
cudaError_t launch_sample(const SampleParams& p, cudaStream_t s);

}  // namespace ta
