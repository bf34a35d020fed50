// C ABI of the operators that take prompts in and verify trees of drafted
// tokens: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/tree_attn.h"
#include "api_checks.h"
#include "drafts.h"

static_assert(ta::kMaxNodes == TREE_ATTN_NODES_MAX && ta::kMaxTop == TREE_ATTN_TOP_MAX, "limits");

namespace {

using ta::api::device_sms;
using ta::api::fail;
using ta::api::guarded;
using ta::api::launched;
using ta::api::off;

tree_attn_status too_many_requests() {
  return fail(TA_ERR_UNSUPPORTED, "more than " + std::to_string(TREE_ATTN_MAX_REQUESTS) + " requests");
}

// (the kernels step through what they count in 32 bits)
bool uncountable(int32_t n) { return n > INT32_MAX / 2; }

// The sizes that decide the workspace of a chunk run.
tree_attn_status chunk_sizes(int32_t n_requests, int32_t n_tokens, int32_t n_q_heads,
                             int32_t n_kv_heads, int32_t head_dim, ta::ChunkParams* p) {
  if (n_requests < 0 || n_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0)
    return fail(TA_ERR_INVALID_ARG, "a count is out of range");
  if (head_dim != 64 && head_dim != 128) return fail(TA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 128)
    return fail(TA_ERR_UNSUPPORTED, "n_q_heads must be a multiple of n_kv_heads, at most 128 times it");
  if (n_requests > TREE_ATTN_MAX_REQUESTS) return too_many_requests();
  if ((int64_t)n_tokens * n_q_heads > INT32_MAX / 2)
    return fail(TA_ERR_UNSUPPORTED, "2^30 query rows or more");
  p->n_req = n_requests;
  p->n_tokens = n_tokens;
  p->hq = n_q_heads;
  p->hkv = n_kv_heads;
  p->gqa = n_q_heads / n_kv_heads;
  p->d = head_dim;
  p->num_sms = device_sms();
  return TA_OK;
}

}  // namespace

extern "C" {

tree_attn_status tree_attn_chunk_run(const void* q, int64_t q_stride, const void* k_pages,
                                     const void* v_pages, int32_t num_pages,
                                     const int32_t* block_table, int64_t table_stride,
                                     int32_t table_width, const int32_t* lens,
                                     const int32_t* cu_new, const int32_t* parents,
                                     int32_t n_requests, int32_t n_tokens, int32_t n_q_heads,
                                     int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                     float softmax_scale, void* out, float* lse, int32_t* status,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> tree_attn_status {
    ta::ChunkParams p{};
    const tree_attn_status st =
        chunk_sizes(n_requests, n_tokens, n_q_heads, n_kv_heads, head_dim, &p);
    if (st != TA_OK) return st;
    if (dtype != TA_BF16 && dtype != TA_FP16)
      return fail(TA_ERR_UNSUPPORTED, "queries and pages must be bf16 or fp16");
    if (table_width < 0 || (n_requests > 1 && table_stride < table_width))
      return fail(TA_ERR_INVALID_ARG, "table_width is negative or table_stride below it");
    // (the keys of a request's last step and its pages, a step more at most, are counted in 32 bits)
    if ((int64_t)table_width * ta::kPage > INT32_MAX - 256 || (uint32_t)num_pages > ta::kMaxPages)
      return fail(TA_ERR_UNSUPPORTED, "rows of 2^31 - 256 tokens or more, or num_pages out of range");
    if (!cu_new && n_tokens != n_requests)
      return fail(TA_ERR_INVALID_ARG, "without cu_new there is one query a request: n_tokens must be n_requests");
    // an SM's share of the steps is counted in 32 bits
    const int64_t blocks = ((int64_t)n_tokens * p.gqa / 128 + n_requests + 1) * n_kv_heads;
    const int64_t steps = table_width / 8 + 1;
    if (blocks > INT64_MAX / steps || blocks * steps / p.num_sms > INT32_MAX / 4)
      return fail(TA_ERR_UNSUPPORTED, "too many query rows for tables this wide");
    if (n_tokens == 0) return TA_OK;
    if (!q || !out || !k_pages || !v_pages || num_pages == 0 ||
        (n_requests > 0 && (!lens || (table_width > 0 && !block_table))))
      return fail(TA_ERR_INVALID_ARG, "q, out, the pools, lens and block_table must be non-NULL");
    if (n_tokens > 1 && q_stride < (int64_t)n_q_heads * head_dim)
      return fail(TA_ERR_INVALID_ARG, "q_stride must be at least n_q_heads * head_dim");
    if (off(q, 16) || off(k_pages, 16) || off(v_pages, 16) || off(out, 32) || q_stride % 8)
      return fail(TA_ERR_ALIGNMENT,
                  "q and the pools must be 16-byte aligned, out 32-byte, q_stride a multiple of 8 elements");
    if (off(block_table, 4) || off(lens, 4) || off(cu_new, 4) || off(parents, 4) || off(lse, 4) ||
        off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 and fp32 buffers must be 4-byte aligned");
    const size_t need = ta::chunk_workspace(p);
    if (workspace_bytes < need)
      return fail(TA_ERR_BUFFER_TOO_SMALL, "the workspace needs " + std::to_string(need) + " bytes");
    if (need > 0 && (!workspace || off(workspace, 256)))
      return fail(workspace ? TA_ERR_ALIGNMENT : TA_ERR_INVALID_ARG,
                  "the workspace must be non-NULL and 256-byte aligned");
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.k_pages = static_cast<const uint16_t*>(k_pages);
    p.v_pages = static_cast<const uint16_t*>(v_pages);
    p.num_pages = num_pages;
    p.table = block_table;
    p.table_stride = table_stride;
    p.width = table_width;
    p.lens = lens;
    p.cu = cu_new;
    p.parents = parents;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.status = status;
    p.dtype = dtype;
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)head_dim)) * 1.4426950408889634f;
    return launched(ta::launch_chunk_attention(p, workspace, static_cast<cudaStream_t>(stream)),
                    "chunk attention launch");
  });
}

tree_attn_status tree_attn_chunk_workspace(int32_t n_requests, int32_t n_tokens, int32_t n_q_heads,
                                           int32_t n_kv_heads, int32_t head_dim, size_t* bytes) {
  return guarded([&]() -> tree_attn_status {
    if (!bytes) return fail(TA_ERR_INVALID_ARG, "bytes is NULL");
    ta::ChunkParams p{};
    const tree_attn_status st =
        chunk_sizes(n_requests, n_tokens, n_q_heads, n_kv_heads, head_dim, &p);
    if (st != TA_OK) return st;
    *bytes = ta::chunk_workspace(p);
    return TA_OK;
  });
}

tree_attn_status tree_attn_accept_drafts(const int32_t* drafted, const int32_t* parents,
                                         const int32_t* cu_new, const int32_t* sampled,
                                         int32_t n_requests, int32_t n_tokens, int32_t* path,
                                         int32_t* n_kept, int32_t* next_tokens, int32_t* n_back,
                                         int32_t* status, void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_requests < 0 || n_tokens < 0) return fail(TA_ERR_INVALID_ARG, "a count is negative");
    if (n_requests > TREE_ATTN_MAX_REQUESTS) return too_many_requests();
    if (uncountable(n_tokens)) return fail(TA_ERR_UNSUPPORTED, "2^30 nodes or more");
    if (!cu_new && n_tokens != n_requests)
      return fail(TA_ERR_INVALID_ARG, "without cu_new there is one node a request: n_tokens must be n_requests");
    if ((n_requests > 0 && (!n_kept || !next_tokens)) ||
        (n_tokens > 0 && (!drafted || !parents || !sampled || !path)))
      return fail(TA_ERR_INVALID_ARG, "drafted, parents, sampled, path, n_kept and next_tokens must be non-NULL");
    if (off(drafted, 4) || off(parents, 4) || off(cu_new, 4) || off(sampled, 4) || off(path, 4) ||
        off(n_kept, 4) || off(next_tokens, 4) || off(n_back, 4) || off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 buffers must be 4-byte aligned");
    ta::AcceptParams p{};
    p.drafted = drafted;
    p.parents = parents;
    p.cu = cu_new;
    p.sampled = sampled;
    p.path = path;
    p.kept = n_kept;
    p.next = next_tokens;
    p.back = n_back;
    p.status = status;
    p.n_req = n_requests;
    p.n_tokens = n_tokens;
    return launched(ta::launch_accept_drafts(p, static_cast<cudaStream_t>(stream)), "accept launch");
  });
}

tree_attn_status tree_attn_keep_drafts(const int32_t* path, const int32_t* cu_new,
                                       const int32_t* lens, const int32_t* block_table,
                                       int64_t table_stride, int32_t table_width,
                                       int32_t n_requests, int32_t n_tokens, void* k_pages,
                                       void* v_pages, int64_t layer_stride, int32_t n_layers,
                                       int32_t num_pages, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t* status, void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_requests < 0 || n_tokens < 0 || table_width < 0 || n_layers < 0 || num_pages < 0 || n_kv_heads <= 0)
      return fail(TA_ERR_INVALID_ARG, "a count is out of range");
    if (head_dim != 64 && head_dim != 128) return fail(TA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (n_kv_heads > 4096 || (uint32_t)num_pages > ta::kMaxPages || n_layers > 65535)
      return fail(TA_ERR_UNSUPPORTED, "more than 4096 kv heads, 65535 layers or 2^27 pages");
    if (n_requests > TREE_ATTN_MAX_REQUESTS) return too_many_requests();
    if (uncountable(n_tokens)) return fail(TA_ERR_UNSUPPORTED, "2^30 nodes or more");
    if ((int64_t)table_width * ta::kPage > INT32_MAX)
      return fail(TA_ERR_UNSUPPORTED, "rows of 2^31 tokens or more");
    if (!cu_new && n_tokens != n_requests)
      return fail(TA_ERR_INVALID_ARG, "without cu_new there is one node a request: n_tokens must be n_requests");
    if (n_requests > 1 && table_stride < table_width)
      return fail(TA_ERR_INVALID_ARG, "table_stride is below table_width");
    if (n_requests == 0 || n_tokens == 0 || n_layers == 0) return TA_OK;
    if (!path || !lens || (table_width > 0 && !block_table) || (num_pages > 0 && (!k_pages || !v_pages)))
      return fail(TA_ERR_INVALID_ARG, "path, lens, block_table and the pools must be non-NULL");
    const int64_t pool = (int64_t)num_pages * n_kv_heads * ta::kPage * head_dim;
    if (layer_stride == 0) layer_stride = pool;
    if (n_layers > 1 && layer_stride < pool)
      return fail(TA_ERR_INVALID_ARG, "layer_stride is below a pool's size");
    if (off(k_pages, 16) || off(v_pages, 16) || layer_stride % 8)
      return fail(TA_ERR_ALIGNMENT, "the pools must be 16-byte aligned, layer_stride a multiple of 8 elements");
    if (off(path, 4) || off(cu_new, 4) || off(lens, 4) || off(block_table, 4) || off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 buffers must be 4-byte aligned");
    ta::KeepParams p{};
    p.path = path;
    p.cu = cu_new;
    p.lens = lens;
    p.table = block_table;
    p.table_stride = table_stride;
    p.k_pages = static_cast<uint16_t*>(k_pages);
    p.v_pages = static_cast<uint16_t*>(v_pages);
    p.layer_stride = layer_stride;
    p.status = status;
    p.width = table_width;
    p.n_req = n_requests;
    p.n_tokens = n_tokens;
    p.num_pages = num_pages;
    p.layers = n_layers;
    p.hkv = n_kv_heads;
    p.d = head_dim;
    return launched(ta::launch_keep_drafts(p, static_cast<cudaStream_t>(stream)), "move launch");
  });
}

tree_attn_status tree_attn_token_logprobs(const void* logits, int64_t stride, int32_t dtype,
                                          int32_t n_rows, int32_t vocab, const int32_t* given,
                                          int32_t n_given, const float* temperature,
                                          float temperature_all, int32_t top,
                                          float* given_logprobs, float* entropy,
                                          int32_t* top_tokens, float* top_logprobs, void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_rows < 0 || n_given < 0 || top < 0 || vocab <= 0)
      return fail(TA_ERR_INVALID_ARG, "n_rows, n_given, top or vocab out of range");
    if (dtype != TA_BF16 && dtype != TA_FP16 && dtype != TA_FP32)
      return fail(TA_ERR_UNSUPPORTED, "logits must be bf16, fp16 or fp32");
    if (vocab > TREE_ATTN_MAX_VOCAB)
      return fail(TA_ERR_UNSUPPORTED, "vocab is above " + std::to_string(TREE_ATTN_MAX_VOCAB));
    if (top > TREE_ATTN_TOP_MAX)
      return fail(TA_ERR_UNSUPPORTED, "top is above " + std::to_string(TREE_ATTN_TOP_MAX));
    if (n_rows > INT32_MAX / 8) return fail(TA_ERR_UNSUPPORTED, "2^28 rows or more");
    if (uncountable(n_given)) return fail(TA_ERR_UNSUPPORTED, "2^30 given tokens a row or more");
    if (n_rows == 0) return TA_OK;
    if (!logits || (n_given > 0 && (!given || !given_logprobs)) || (top > 0 && (!top_tokens || !top_logprobs)))
      return fail(TA_ERR_INVALID_ARG, "logits, and what is asked for, must be non-NULL");
    if (n_rows > 1 && stride < vocab) return fail(TA_ERR_INVALID_ARG, "stride is below vocab");
    if (off(logits, dtype == TA_FP32 ? 4 : 2) || off(given, 4) || off(temperature, 4) ||
        off(given_logprobs, 4) || off(entropy, 4) || off(top_tokens, 4) || off(top_logprobs, 4))
      return fail(TA_ERR_ALIGNMENT, "a buffer is not aligned to its elements");
    if (n_given == 0 && top == 0 && !entropy) return TA_OK;
    ta::ScoreParams p{};
    p.logits = logits;
    p.stride = stride;
    p.dtype = dtype;
    p.rows = n_rows;
    p.vocab = vocab;
    p.given = given;
    p.n_given = n_given;
    p.temperature = temperature;
    p.temperature_all = temperature_all;
    p.top = top;
    p.given_logprobs = given_logprobs;
    p.entropy = entropy;
    p.top_tokens = top_tokens;
    p.top_logprobs = top_logprobs;
    p.num_sms = device_sms();
    return launched(ta::launch_token_logprobs(p, static_cast<cudaStream_t>(stream)), "scores launch");
  });
}

}  // extern "C"
