// ol_draft.h -- parameter blocks, shared arithmetic and launchers of the
// operators around drafted tokens: rotary positions and the rotating append
// (ol_rope.cu), attention of a tree over a cache (ol_tree.cu, ol_fast_tree.cu)
// and the accepted path's move (ol_tree.cu). Not part of the public ABI.
#pragma once

#include "ol_internal.h"

#if defined(__CUDACC__)
#define OL_HD __host__ __device__
#else
#define OL_HD
#endif

namespace ol {

// Where a token of a contiguous or paged cache lives.
struct CacheRef {
  void* base;                  // cache or pool
  const int32_t* block_table;  // NULL: contiguous [2, batch, kv_heads, capacity, D]
  int batch, kv_heads, capacity;
  int num_pages, page_size, max_pages;
};

// ------------------------------------------------------------ rotary positions

struct RopeView {  // strides in elements
  char* data;
  int64_t sb, sh, st;
};

struct RopeParams {
  const uint64_t* turns;
  int rot_dim, style;
  float magnitude;
  int dtype, head_dim, batch, tokens;
  int q_heads, kv_heads;        // kv_heads 0: rotation of q alone
  RopeView q, q_out, k, v;
  CacheRef cache;               // destination of k and v
  const int32_t* positions;     // [batch] first positions, or NULL
  const int32_t* counts;        // [batch], or NULL
  const int32_t* angles;        // [batch, tokens], or NULL: positions[b] + t
  int vec;                      // 1: every vector and its rotated part is 16-byte aligned
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t s);

// ------------------------------------------------------------- tree attention

constexpr int kTreeMaxNodes = 512;
constexpr int kTreeMaxCtas = 192;  // CTAs of the tensor-core kernel, one per SM
constexpr int kTreeGenTileLog2 = 5;   // tokens of its tile: 32
constexpr int kTreeFastTileLog2 = 7;  // 128

// What there is to merge: of the unit that begins in a share and reaches past its
// end, or of a unit (TreeParams::by_unit).
struct alignas(16) TreeSplit {
  int first, last;  // shares of the unit's segments; last -1: nothing to merge
  int count;  // nodes of its row
  int rows;   // live (head, node) rows
  long long out;  // row of q and out of its row 0
  int row0;       // (head, node) row 0 of the unit
  int pad;
};

struct TreeParams {
  CacheRef cache;
  int dtype, batch, q_heads, kv_heads, group, head_dim;
  int nodes, words;             // mask words per node
  const void* q;                // [batch, q_heads, nodes, D]
  const int32_t* lens;
  const int32_t* counts;        // [batch], or NULL: nodes
  const uint64_t* mask;         // NULL: a chain
  const int32_t* node_pos;      // NULL: prefix + i
  float scale_log2;             // softmax scale * log2(e)
  int window;                   // < 0: unbounded
  void* out;
  int out_dtype;
  int32_t* status;
  struct TreeSplit* splits;     // [nctas] or [units], written by the attention's CTAs for the merge
  float* partials;
  // work split
  int rows_per_unit;            // (head, node) rows r = head * nodes + node of a unit
  int units_per_head;           // ceil(group * nodes / rows_per_unit)
  int tile_log2;                // tokens per tile
  int nctas;                    // the tiles of all units in contiguous equal shares
  int extra;                    // tiles that a unit's begin and end cost besides
  int by_unit;                  // 1: few units, each cut into many segments; the merge goes by units
};
// Few units of many segments are merged by units, 8 rows a CTA, while those CTAs
// are one wave; else by shares. Measured (bf16, 8 kv heads, 4000 tokens; by units /
// by shares): 2 rows of 64 (head, node) rows 16.3 / 17.2 us, 2 of 256 34.7 / 28.4
// us, 4 of 64 24.4 / 22.3 us, 4 of 256 54.5 / 36.2 us.
inline bool tree_few_units(const TreeParams& p) {
  const int all = p.group * p.nodes, rows = all < p.rows_per_unit ? all : p.rows_per_unit;
  return (long long)p.batch * p.kv_heads * p.units_per_head * ((rows + 7) / 8) <= p.nctas;
}

// A row's tokens as the work split sees them: drafted tokens are
// [prefix, len), tokens [start, len) form ntiles tiles (start is a multiple of
// the tile at or below the lowest token that any node may see).
struct TreeRow {
  int len, count, prefix, start, ntiles;
};
OL_HD inline TreeRow tree_row(int len, int count, int window, int tile_log2) {
  TreeRow r;
  r.len = len;
  r.count = count;
  r.prefix = len - count;
  const int lo = window < 0 || r.prefix <= window ? 0 : r.prefix - window;
  r.start = lo >> tile_log2 << tile_log2;
  r.ntiles = count > 0 ? ((len - r.start - 1) >> tile_log2) + 1 : 0;  // (len may be 2^31 - 1)
  return r;
}

// One partial slot: m[rows] (log2 domain), l[rows], o[ceil(D / 4)][rows] float4.
OL_HD inline size_t tree_slot_floats(int rows, int head_dim) { return (size_t)rows * (2 + (head_dim + 3) / 4 * 4); }
constexpr size_t kTreeSplitBytes = 4 * kTreeMaxCtas * sizeof(TreeSplit);
// (head, node) rows of a unit of the CUDA-core and of the tensor-core kernel
inline int tree_gen_rows(int group, int nodes) { return group * nodes <= 32 ? 32 : 64; }
inline int tree_fast_rows(int group, int nodes) { return group * nodes <= 128 ? 128 : 256; }
// Notes and partial slots lie behind the ticket counters of decode steps and of
// chunked steps of up to `nodes` tokens of this batch, which stay as they are. (A
// decode step's own partial slots lie over those of chunked steps.)
inline size_t tree_splits_offset(int batch, int kv_heads, int nodes) {
  return partials_offset(batch, kv_heads, nodes);
}
inline size_t tree_workspace_bytes(int batch, int q_heads, int kv_heads, int head_dim, int nodes) {
  const size_t fast = 2ull * kTreeMaxCtas * tree_slot_floats(tree_fast_rows(q_heads / kv_heads, nodes), head_dim);
  const int rows = tree_gen_rows(q_heads / kv_heads, nodes);
  const size_t gen = 2ull * (128 / rows) * kTreeMaxCtas * tree_slot_floats(rows, head_dim);
  return tree_splits_offset(batch, kv_heads, nodes) + kTreeSplitBytes + sizeof(float) * (fast > gen ? fast : gen);
}

bool fast_tree_supported(const TreeParams& p);
// Fill the work split of a kernel.
void plan_fast_tree(TreeParams& p, int sms);
void plan_generic_tree(TreeParams& p, int sms);
// Tiles are counted in 32 bits on the device, whatever lengths it finds there.
inline bool tree_counts_fit(const TreeParams& p) {
  const unsigned __int128 tiles = (unsigned __int128)((p.cache.capacity >> p.tile_log2) + 1 + p.extra) * p.batch * p.kv_heads *
                                  p.units_per_head;
  return tiles < (1u << 31);
}
cudaError_t launch_fast_tree(const TreeParams& p, cudaStream_t s);
cudaError_t launch_generic_tree(const TreeParams& p, cudaStream_t s);
cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t s);

// --------------------------------------------------------------- accepted path

struct KeepParams {
  CacheRef cache;
  int dtype, head_dim, nodes;
  const int32_t* starts;  // [batch]
  const int32_t* kept;    // [batch, nodes]
  const int32_t* counts;  // [batch], of kept
  const int32_t* drafted; // [batch], or NULL: nodes
  int32_t* status;        // or NULL
};
cudaError_t launch_tree_keep(const KeepParams& p, cudaStream_t s);

}  // namespace ol

#undef OL_HD
