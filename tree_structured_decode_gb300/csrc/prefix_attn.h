// Structures shared by the kernels of the shared-prefix attention.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "batch.h"

namespace ta {

// What the kernels know of a request, checked: its first token and row count
// lie in the batch, its pages in the table.
struct Request {
  long long p0;  // steps in the line before it
  int len, n, tok0, np;  // tokens held, queries, the first one, steps of a segment
};

// One line of segments (a tile of query rows of one kv head against one
// request's keys), cut into equal runs of steps: the requests' own tokens, or
// the prefix as a request of its own whose rows are all tokens'.
struct Line {
  Request* req;       // null: `one`
  long long* sizes;   // [0] steps in the line, [1] a run; null: `total`, `run`
  float* piece_o;     // [2 * runs][tile_rows][d]
  float2* piece_ml;   // [2 * runs][tile_rows]: {m, l}
  float* row_o;       // [tokens * hq][d]: segments in one run
  float2* row_ml;
  const int32_t* table;
  long long table_stride;
  long long total, run;
  Request one;
  int n_req, width, causal, tile_rows;

  __device__ __forceinline__ Request request(int b) const { return req ? req[b] : one; }
  __device__ __forceinline__ long long steps() const { return sizes ? sizes[0] : total; }
  __device__ __forceinline__ long long length() const { return sizes ? sizes[1] : run; }
};

struct Args {
  PrefixParams p;
  Line line[2];  // own tokens, prefix
};


// Most query rows of a tile of the tensor-core prefix kernel: two of 128.
constexpr int kTileRows = 256;
constexpr int kTileTokens = 128;  // keys of a step
// The prefix's pieces by tcgen05 (a.line[1] cut in steps of kTileTokens keys).
cudaError_t launch_prefix_tiles(const Args& a, const CUtensorMap& mk_half, const CUtensorMap& mv,
                                cudaStream_t s);

}  // namespace ta
