// Parameter blocks and launchers of the operators that take prompts in and
// verify trees of drafted tokens: attention of several new tokens a request, the
// drafts that stand, their keys and values moved together, scores of tokens.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "batch.h"

namespace ta {

constexpr int kMaxNodes = 128;  // of a request's tree (TREE_ATTN_NODES_MAX of the C ABI)
constexpr int kMaxTop = 64;     // alternatives of a row (TREE_ATTN_TOP_MAX)

struct ChunkParams {
  const uint16_t* q;
  long long q_stride;            // elements from one token to the next
  const uint16_t *k_pages, *v_pages;
  const int32_t* table;
  long long table_stride;
  const int32_t* lens;
  const int32_t* cu;             // tokens before each request; null: one each
  const int32_t* parents;        // [tokens] node above, within the request; null: a chain
  uint16_t* out;                 // [tokens][hq][d], q's type
  float* lse;                    // [tokens][hq] natural log, or null
  int32_t* status;
  int width, n_tokens, n_req, hq, hkv, gqa, d, num_pages, dtype, num_sms;
  float scale_log2;              // softmax scale * log2(e)
};
// Workspace of a run; 0 where there is nothing to do.
size_t chunk_workspace(const ChunkParams& p);
cudaError_t launch_chunk_attention(const ChunkParams& p, void* workspace, cudaStream_t s);

struct AcceptParams {
  const int32_t *drafted, *parents, *cu, *sampled;
  int32_t *path, *kept, *next, *back, *status;
  int n_req, n_tokens;
};
cudaError_t launch_accept_drafts(const AcceptParams& p, cudaStream_t s);

struct KeepParams {
  const int32_t *path, *cu, *lens, *table;
  long long table_stride;
  uint16_t *k_pages, *v_pages;
  long long layer_stride;        // elements from one layer's pool to the next
  int32_t* status;
  int width, n_req, n_tokens, num_pages, layers, hkv, d;
};
cudaError_t launch_keep_drafts(const KeepParams& p, cudaStream_t s);

struct ScoreParams {
  const void* logits;            // [rows][vocab], rows `stride` elements apart
  long long stride;
  int dtype, rows, vocab, n_given, top;
  const int32_t* given;          // [rows][n_given]
  const float* temperature;      // per row, or null
  float temperature_all;
  float *given_logprobs, *entropy;  // [rows][n_given], [rows] or null
  int32_t* top_tokens;           // [rows][top]
  float* top_logprobs;
  int num_sms;
};
cudaError_t launch_token_logprobs(const ScoreParams& p, cudaStream_t s);

}  // namespace ta
