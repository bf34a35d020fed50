// C ABI of the operators whose lengths live on the GPU: argument checks and
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/tree_attn.h"
#include "batch.h"
#include "plan_state.h"

// The limits that the kernels rest on, and the codes, are those of the ABI.
static_assert(ta::kMaxRequests == TREE_ATTN_MAX_REQUESTS && ta::kMaxVocab == TREE_ATTN_MAX_VOCAB, "limits");
static_assert((int)ta::kBf16 == TA_BF16 && (int)ta::kFp16 == TA_FP16 && (int)ta::kFp32 == TA_FP32, "types");
static_assert((int)ta::kBatchNoPages == TREE_ATTN_BATCH_NO_PAGES &&
                  (int)ta::kBatchTableFull == TREE_ATTN_BATCH_TABLE_FULL &&
                  (int)ta::kBatchBadInput == TREE_ATTN_BATCH_BAD_INPUT &&
                  (int)ta::kBatchBadSlot == TREE_ATTN_BATCH_BAD_SLOT &&
                  (int)ta::kBatchTimeout == TREE_ATTN_BATCH_TIMEOUT,
              "status bits");

namespace {

tree_attn_status fail(tree_attn_status s, const std::string& msg) {
  ta::set_last_error(msg);
  return s;
}
tree_attn_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TA_OK;
  return fail(TA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Nothing is thrown across the ABI.
template <class F>
tree_attn_status guarded(F&& f) {
  try {
    ta::set_last_error("");
    return f();
  } catch (...) {
    return TA_ERR_OOM;
  }
}

// SMs of the current device (152 where there is none).
int device_sms() {
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
    return 152;
  return sms;
}

// The sizes that decide the workspace of a prefix run.
tree_attn_status prefix_sizes(int32_t n_requests, int32_t n_tokens, int32_t prefix_len,
                              int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                              ta::PrefixParams* p) {
  if (n_requests < 0 || n_tokens < 0 || prefix_len < 0 || n_q_heads <= 0 || n_kv_heads <= 0)
    return fail(TA_ERR_INVALID_ARG, "a count or length is out of range");
  if (head_dim != 64 && head_dim != 128) return fail(TA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 128)
    return fail(TA_ERR_UNSUPPORTED, "n_q_heads must be a multiple of n_kv_heads, at most 128 times it");
  if (n_requests > TREE_ATTN_MAX_REQUESTS)
    return fail(TA_ERR_UNSUPPORTED, "more than " + std::to_string(TREE_ATTN_MAX_REQUESTS) + " requests");
  if ((int64_t)n_tokens * n_q_heads > INT32_MAX / 2)
    return fail(TA_ERR_UNSUPPORTED, "2^30 query rows or more");
  p->n_req = n_requests;
  p->n_tokens = n_tokens;
  p->prefix_len = prefix_len;
  p->hq = n_q_heads;
  p->hkv = n_kv_heads;
  p->gqa = n_q_heads / n_kv_heads;
  p->d = head_dim;
  p->num_sms = device_sms();
  return TA_OK;
}

}  // namespace

extern "C" {

tree_attn_status tree_attn_extend_tables(int32_t* lens, const int32_t* n_new, int32_t n_requests,
                                         int32_t* block_table, int64_t table_stride,
                                         int32_t table_width, int32_t* free_pages,
                                         int32_t free_capacity, int32_t* n_free, int32_t max_new,
                                         int32_t position_base, int32_t* slots,
                                         int32_t* positions, int32_t* cu_new, int32_t* status,
                                         void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_requests < 0 || table_width < 0 || free_capacity < 0 || max_new < 0 || position_base < 0)
      return fail(TA_ERR_INVALID_ARG, "a count, size or the position base is negative");
    if (!n_free || (n_requests > 0 && (!lens || !n_new)) ||
        (n_requests > 0 && table_width > 0 && !block_table) || (free_capacity > 0 && !free_pages) ||
        (max_new > 0 && (!slots || !positions)))
      return fail(TA_ERR_INVALID_ARG, "a buffer of the tables is NULL");
    if (table_stride < table_width)
      return fail(TA_ERR_INVALID_ARG, "table_stride is below table_width");
    if (n_requests > TREE_ATTN_MAX_REQUESTS)
      return fail(TA_ERR_UNSUPPORTED, "more than " + std::to_string(TREE_ATTN_MAX_REQUESTS) + " requests");
    if ((int64_t)table_width * ta::kPage + position_base > INT32_MAX)
      return fail(TA_ERR_UNSUPPORTED, "table_width * 16 + position_base passes 2^31");
    if (off(lens, 4) || off(n_new, 4) || off(block_table, 4) || off(free_pages, 4) ||
        off(n_free, 4) || off(slots, 4) || off(positions, 4) || off(cu_new, 4) || off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 buffers must be 4-byte aligned");
    ta::ExtendParams p{};
    p.lens = lens;
    p.n_new = n_new;
    p.table = block_table;
    p.table_stride = table_stride;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.slots = slots;
    p.positions = positions;
    p.cu_new = cu_new;
    p.status = status;
    p.n_req = n_requests;
    p.width = table_width;
    p.free_cap = free_capacity;
    p.max_new = max_new;
    p.position_base = position_base;
    return launched(ta::launch_extend_tables(p, static_cast<cudaStream_t>(stream)),
                    "table extension launch");
  });
}

tree_attn_status tree_attn_append_slots(const void* k_new, const void* v_new, int64_t k_stride,
                                        int64_t v_stride, const int32_t* slots, int32_t n_tokens,
                                        int32_t n_kv_heads, int32_t head_dim, void* k_pages,
                                        void* v_pages, int32_t num_pages, int32_t* status,
                                        void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_tokens < 0 || n_kv_heads <= 0 || num_pages < 0)
      return fail(TA_ERR_INVALID_ARG, "n_tokens, n_kv_heads or num_pages out of range");
    if (head_dim != 64 && head_dim != 128)
      return fail(TA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (n_kv_heads > 4096 || (uint32_t)num_pages > ta::kMaxPages)
      return fail(TA_ERR_UNSUPPORTED, "more than 4096 kv heads or 2^27 pages");
    if (n_tokens == 0) return TA_OK;
    if (!k_new || !v_new || !slots || (num_pages > 0 && (!k_pages || !v_pages)))
      return fail(TA_ERR_INVALID_ARG, "k_new, v_new, slots, k_pages and v_pages must be non-NULL");
    const int64_t row = (int64_t)n_kv_heads * head_dim;
    if (n_tokens > 1 && (k_stride < row || v_stride < row))
      return fail(TA_ERR_INVALID_ARG, "k_stride and v_stride must be at least n_kv_heads * head_dim");
    if (off(k_new, 16) || off(v_new, 16) || off(k_pages, 16) || off(v_pages, 16) || k_stride % 8 ||
        v_stride % 8)
      return fail(TA_ERR_ALIGNMENT,
                  "k_new, v_new, k_pages and v_pages must be 16-byte aligned, strides multiples of 8 elements");
    if (off(slots, 4) || off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 buffers must be 4-byte aligned");
    ta::AppendSlotsParams p{};
    p.k_new = static_cast<const uint16_t*>(k_new);
    p.v_new = static_cast<const uint16_t*>(v_new);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.k_pages = static_cast<uint16_t*>(k_pages);
    p.v_pages = static_cast<uint16_t*>(v_pages);
    p.status = status;
    p.n_slots = (long long)num_pages * ta::kPage;
    p.n_tokens = n_tokens;
    p.hkv = n_kv_heads;
    p.d = head_dim;
    return launched(ta::launch_append_slots(p, static_cast<cudaStream_t>(stream)), "append launch");
  });
}

tree_attn_status tree_attn_prefix_run(const void* q, int64_t q_stride, const void* k_pages,
                                      const void* v_pages, int32_t num_pages,
                                      const int32_t* block_table, int64_t table_stride,
                                      int32_t table_width, const int32_t* lens,
                                      const int32_t* cu_new, int32_t n_requests, int32_t n_tokens,
                                      const int32_t* prefix_pages, int32_t prefix_len,
                                      int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t dtype, float softmax_scale, void* out, float* lse,
                                      int32_t* status, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return guarded([&]() -> tree_attn_status {
    ta::PrefixParams p{};
    const tree_attn_status st =
        prefix_sizes(n_requests, n_tokens, prefix_len, n_q_heads, n_kv_heads, head_dim, &p);
    if (st != TA_OK) return st;
    if (dtype != TA_BF16 && dtype != TA_FP16)
      return fail(TA_ERR_UNSUPPORTED, "queries and pages must be bf16 or fp16");
    if (table_width < 0 || (n_requests > 1 && table_stride < table_width))
      return fail(TA_ERR_INVALID_ARG, "table_width is negative or table_stride below it");
    if ((int64_t)table_width * ta::kPage > INT32_MAX || (uint32_t)num_pages > ta::kMaxPages)
      return fail(TA_ERR_UNSUPPORTED, "rows of 2^31 tokens or more, or num_pages out of range");
    // a warp's, or CTA's, share of the work is counted in 32 bits
    const int64_t kv_tiles = ((int64_t)n_tokens * p.gqa / 8 + n_requests + 1) * n_kv_heads;
    const int64_t most = std::max<int64_t>(table_width, prefix_len / ta::kPage + 1);
    if (kv_tiles > INT64_MAX / most || kv_tiles * most / p.num_sms > INT32_MAX / 8)
      return fail(TA_ERR_UNSUPPORTED, "too many query rows for tables this wide or a prefix this long");
    if (!cu_new && n_tokens != n_requests)
      return fail(TA_ERR_INVALID_ARG, "without cu_new there is one query a request: n_tokens must be n_requests");
    if (n_tokens == 0) return TA_OK;
    if (!q || !out || !k_pages || !v_pages || num_pages == 0 ||
        (n_requests > 0 && (!lens || (table_width > 0 && !block_table))) ||
        (prefix_len > 0 && !prefix_pages))
      return fail(TA_ERR_INVALID_ARG, "q, out, the pools, lens, block_table and prefix_pages must be non-NULL");
    if (n_tokens > 1 && q_stride < (int64_t)n_q_heads * head_dim)
      return fail(TA_ERR_INVALID_ARG, "q_stride must be at least n_q_heads * head_dim");
    if (off(q, 16) || off(k_pages, 16) || off(v_pages, 16) || off(out, 16) || q_stride % 8)
      return fail(TA_ERR_ALIGNMENT,
                  "q, out and the pools must be 16-byte aligned, q_stride a multiple of 8 elements");
    if (off(block_table, 4) || off(lens, 4) || off(cu_new, 4) || off(prefix_pages, 4) ||
        off(lse, 4) || off(status, 4))
      return fail(TA_ERR_ALIGNMENT, "int32 and fp32 buffers must be 4-byte aligned");
    const size_t need = ta::prefix_workspace(p);
    if (workspace_bytes < need)
      return fail(TA_ERR_BUFFER_TOO_SMALL, "the workspace needs " + std::to_string(need) + " bytes");
    if (!workspace || off(workspace, 256))
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
    p.prefix_pages = prefix_pages;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.status = status;
    p.dtype = dtype;
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)head_dim)) * 1.4426950408889634f;
    return launched(ta::launch_prefix_attention(p, workspace, static_cast<cudaStream_t>(stream)),
                    "prefix attention launch");
  });
}

tree_attn_status tree_attn_prefix_workspace(int32_t n_requests, int32_t n_tokens,
                                            int32_t prefix_len, int32_t n_q_heads,
                                            int32_t n_kv_heads, int32_t head_dim, size_t* bytes) {
  return guarded([&]() -> tree_attn_status {
    if (!bytes) return fail(TA_ERR_INVALID_ARG, "bytes is NULL");
    ta::PrefixParams p{};
    const tree_attn_status st =
        prefix_sizes(n_requests, n_tokens, prefix_len, n_q_heads, n_kv_heads, head_dim, &p);
    if (st != TA_OK) return st;
    *bytes = ta::prefix_workspace(p);
    return TA_OK;
  });
}

tree_attn_status tree_attn_sample(const void* logits, int64_t stride, int32_t dtype,
                                  int32_t n_rows, int32_t vocab, const float* u, int32_t draws,
                                  const float* temperature, float temperature_all,
                                  const int32_t* top_k, int32_t top_k_all, const float* top_p,
                                  float top_p_all, const float* min_p, float min_p_all,
                                  int32_t* tokens, float* logprobs, void* stream) {
  return guarded([&]() -> tree_attn_status {
    if (n_rows < 0 || draws < 0 || vocab <= 0)
      return fail(TA_ERR_INVALID_ARG, "n_rows, draws or vocab out of range");
    if (dtype != TA_BF16 && dtype != TA_FP16 && dtype != TA_FP32)
      return fail(TA_ERR_UNSUPPORTED, "logits must be bf16, fp16 or fp32");
    if (vocab > TREE_ATTN_MAX_VOCAB)
      return fail(TA_ERR_UNSUPPORTED, "vocab is above " + std::to_string(TREE_ATTN_MAX_VOCAB));
    if (n_rows > INT32_MAX / 8) return fail(TA_ERR_UNSUPPORTED, "2^28 rows or more");
    if (n_rows == 0 || draws == 0) return TA_OK;
    if (!logits || !u || !tokens)
      return fail(TA_ERR_INVALID_ARG, "logits, u and tokens must be non-NULL");
    if (n_rows > 1 && stride < vocab) return fail(TA_ERR_INVALID_ARG, "stride is below vocab");
    if (off(logits, dtype == TA_FP32 ? 4 : 2) || off(u, 4) || off(temperature, 4) ||
        off(top_k, 4) || off(top_p, 4) || off(min_p, 4) || off(tokens, 4) || off(logprobs, 4))
      return fail(TA_ERR_ALIGNMENT, "a buffer is not aligned to its elements");
    ta::SampleParams p{};
    p.logits = logits;
    p.stride = stride;
    p.dtype = dtype;
    p.rows = n_rows;
    p.vocab = vocab;
    p.draws = draws;
    p.u = u;
    p.temperature = temperature;
    p.temperature_all = temperature_all;
    p.top_k = top_k;
    p.top_k_all = top_k_all;
    p.top_p = top_p;
    p.top_p_all = top_p_all;
    p.min_p = min_p;
    p.min_p_all = min_p_all;
    p.tokens = tokens;
    p.logprobs = logprobs;
    p.num_sms = device_sms();
    return launched(ta::launch_sample(p, static_cast<cudaStream_t>(stream)), "sampling launch");
  });
}

}  // extern "C"
