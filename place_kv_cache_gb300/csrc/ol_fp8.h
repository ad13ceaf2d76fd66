// ol_fp8.h -- parameter blocks and launchers of the operators of an E4M3 cache:
// the quantising append and reading back (ol_fp8.cu), attention (ol_fast_fp8.cu), and
// the norms of queries and keys with their rotation (ol_norm_rope.cu). Not part of the public ABI.
#pragma once

#include "ol_draft.h"

namespace ol {

constexpr float kFp8Top = 448.f;         // the largest E4M3 value
constexpr float kFp8LeastScale = 0x1p-80f;

struct Fp8Cache {
  uint8_t* codes;
  float* scales;
  const int32_t* block_table;  // NULL: contiguous
  int batch, kv_heads, capacity, head_dim;
  int num_pages, page_size, max_pages;
  int block_log2;
};

struct Fp8AppendParams {
  Fp8Cache cache;
  int dtype, new_len;
  int blocks;                // blocks that a row's tokens may lie in
  RopeView in[2];            // k, v
  const int32_t* positions;  // [batch]
  const int32_t* counts;     // [batch], or NULL: new_len
  int vec;                   // 1: every vector starts on a 16-byte boundary
};
cudaError_t launch_fp8_append(const Fp8AppendParams& p, cudaStream_t s);

struct Fp8ReadParams {
  Fp8Cache cache;
  int dtype, tokens;
  RopeView out[2];           // k, v; data NULL: not wanted
  const int32_t* starts;     // [batch]
  const int32_t* counts;     // [batch], or NULL: tokens
  int vec;
};
cudaError_t launch_fp8_read(const Fp8ReadParams& p, cudaStream_t s);

// Attention: the work split, outputs, partial results and merge are those of a
// chain of drafted tokens (TreeParams with no mask; its cache describes sizes and
// the block table only). dtype is that of q.
struct Fp8AttnParams {
  TreeParams t;
  Fp8Cache cache;
};
void plan_fp8_attention(Fp8AttnParams& p, int sms);
cudaError_t launch_fp8_attention(const Fp8AttnParams& p, cudaStream_t s);

struct NormRopeParams {
  const uint64_t* turns;     // NULL: no rotation (rot_dim 0)
  int rot_dim, style;
  float magnitude;
  const void* weight[2];     // q's, k's, or NULL
  float eps, weight_offset;
  int dtype, head_dim, batch, tokens;
  int q_heads, kv_heads;
  RopeView in[2], out[2];    // q, k
  const int32_t* positions;  // [batch] first positions, or NULL
  const int32_t* angles;     // [batch, tokens], or NULL
  int vec;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s);

}  // namespace ol
