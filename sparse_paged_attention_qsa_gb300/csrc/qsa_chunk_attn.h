// qsa_chunk_attn.h -- what the entry points of the chunk attention
// (include/qsa_chunk.h) hand to its kernels.
#pragma once

#include "qsa_cache_host.h"

#include <cstdint>

namespace qsa {

struct ChunkParams {
  CacheView c;
  const int32_t* prefix_table;  // nullable: no prefix
  int32_t prefix_cap;           // entries that its columns can hold
  const int32_t* prefix_len;
  const unsigned char* q;
  int64_t q_row, q_head;        // bytes
  unsigned char* out;
  int64_t out_row, out_head;    // bytes
  const int32_t* starts;        // [num_reqs + 1]
  const int32_t* ctx;
  int32_t tokens, heads, group;
  float scale_log2;             // scale * log2(e)
  int32_t window;               // 0: none; at most INT32_MAX - 16
  int32_t sink;
  float* lse;                   // nullable
  uint32_t* err;
};

}  // namespace qsa
