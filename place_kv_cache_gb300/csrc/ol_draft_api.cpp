// ol_draft_api.cpp -- the C ABI of the operators around drafted tokens (see
// include/ol.h): rotary positions, the rotating append, attention of a tree
// over a cache, the accepted path's move. Host-side validation and dispatch;
// as in ol_api.cpp every check runs before any launch.
#include <algorithm>
#include <cmath>
#include <vector>

#include "ol_draft.h"
#include "ol_host.h"

namespace ol {
namespace {

// Host memory exhausted (the page checks keep a table) ends a call with a
// status, never with an exception through the C boundary.
template <typename F>
ol_status guarded_call(F&& f) {
  try {
    return f();
  } catch (...) {
    return OL_ERR_CUDA;
  }
}

ol_status view_dense(int layout, const void* desc, CacheView& v) {
  if (layout == OL_LAYOUT_CONTIGUOUS) return view_contiguous(static_cast<const ol_kv_cache*>(desc), v);
  if (layout == OL_LAYOUT_PAGED) return view_paged(static_cast<const ol_paged_kv*>(desc), v);
  return OL_ERR_UNSUPPORTED;
}

CacheRef cache_ref(int layout, const void* desc, const CacheView& v) {
  CacheRef r = {};
  r.batch = v.batch;
  r.kv_heads = v.kv_heads;
  r.capacity = v.capacity;
  if (layout == OL_LAYOUT_PAGED) {
    const ol_paged_kv* c = static_cast<const ol_paged_kv*>(desc);
    r.base = c->data;
    r.block_table = c->block_table;
    r.num_pages = c->num_pages;
    r.page_size = c->page_size;
    r.max_pages = c->max_pages;
  } else {
    r.base = static_cast<const ol_kv_cache*>(desc)->data;
  }
  return r;
}

ol_status table_overlap(int layout, const void* desc, const CacheView& v) {
  if (layout != OL_LAYOUT_PAGED) return OL_OK;
  const ol_paged_kv* c = static_cast<const ol_paged_kv*>(desc);
  return no_overlap(v, c->block_table, sizeof(int32_t) * (size_t)c->batch * c->max_pages);
}

// Whether one of a row's entries [first, end) is outside the pool: bit 31 of
// x | (pages - 1 - x) is set for such an x. A function of its own, without an early
// end, is vectorised: rows have up to thousands of pages (32768 entries 4 us, 25
// one at a time).
__attribute__((noinline)) bool pages_outside(const int32_t* row, int first, int end, int num_pages) {
  const uint32_t top = (uint32_t)num_pages - 1;
  uint32_t bits = 0;
  for (int i = first; i < end; ++i) bits |= (uint32_t)row[i] | (top - (uint32_t)row[i]);
  return bits >> 31;
}

// Pages that tokens [first[b], first[b] + n_b) of the rows are written to: in
// the pool, and none of them twice. The stamps live per thread, so a call
// costs the pages that it writes, not the pool's size.
ol_status check_written_pages(const ol_paged_kv* c, const int32_t* first, const int32_t* counts, int n) {
  static thread_local std::vector<uint64_t> stamps;  // the last call that wrote each page
  static thread_local uint64_t call = 0;
  if (stamps.size() < (size_t)c->num_pages) stamps.resize(c->num_pages, 0);
  ++call;
  const int S = c->page_size;
  for (int b = 0; b < c->batch; ++b) {
    const int cnt = counts ? counts[b] : n;
    if (cnt <= 0) continue;
    for (int pg = first[b] / S; pg <= (first[b] + cnt - 1) / S; ++pg) {
      const int page = c->block_table_host[(size_t)b * c->max_pages + pg];
      if (page < 0 || page >= c->num_pages || stamps[page] == call) return OL_ERR_PAGE;
      stamps[page] = call;
    }
  }
  return OL_OK;
}

// ------------------------------------------------------------- views of vectors

struct Dims {
  int64_t batch, heads, tokens, head_dim;
  bool empty() const { return batch == 0 || heads == 0 || tokens == 0; }
};

constexpr int64_t kMaxStride = 1ll << 40;

// Bytes from a view's first element to its last one's end (0: no element).
unsigned __int128 rows_bytes(const ol_rows& r, const Dims& d, size_t es) {
  if (d.empty()) return 0;
  const unsigned __int128 last = (unsigned __int128)(d.batch - 1) * r.stride_batch +
                                 (unsigned __int128)(d.heads - 1) * r.stride_head +
                                 (unsigned __int128)(d.tokens - 1) * r.stride_token + d.head_dim;
  return last * es;
}

// A view's pointer, strides and extent; `out` also wants vectors that do not
// overlap one another: every stride reaches past what the smaller ones span.
ol_status check_rows(const ol_rows* r, const Dims& d, size_t es, bool out, Range& range) {
  range = {0, 0};
  if (!r) return OL_ERR_NULL;
  if (!r->data) return d.empty() ? OL_OK : OL_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(r->data) % es != 0) return OL_ERR_ALIGN;
  for (int64_t s : {r->stride_batch, r->stride_head, r->stride_token})
    if (s < 0 || s > kMaxStride) return OL_ERR_SHAPE;
  const unsigned __int128 bytes = rows_bytes(*r, d, es);
  if (bytes >> 62) return OL_ERR_SHAPE;
  range = range_of(r->data, (size_t)bytes);
  if (out && !d.empty()) {
    std::pair<int64_t, int64_t> dim[3] = {
        {r->stride_batch, d.batch}, {r->stride_head, d.heads}, {r->stride_token, d.tokens}};
    std::sort(dim, dim + 3);
    unsigned __int128 span = d.head_dim;
    for (const auto& x : dim) {
      if (x.second == 1) continue;
      if ((unsigned __int128)x.first < span) return OL_ERR_SHAPE;
      span += (unsigned __int128)(x.second - 1) * x.first;
    }
  }
  return OL_OK;
}

bool same_view(const ol_rows& a, const ol_rows& b) {
  return a.data == b.data && a.stride_batch == b.stride_batch && a.stride_head == b.stride_head &&
         a.stride_token == b.stride_token;
}

// Whether a vector of `a`, a view that may be written (check_rows), and one of `b`
// may share an element. Views of other strides than a's may; else two vectors are
// delta + sum n_i s_i elements apart, n_i being differences of their indices, and
// as each stride reaches past what the smaller ones span, only the two n_i
// around zero can bring that below head_dim.
bool may_share(const ol_rows& a, const Dims& da, const ol_rows& b, const Dims& db, size_t es) {
  struct Dim {
    int64_t stride, lo, hi;  // lo <= n <= hi
  } dim[3];
  const int64_t sa[3] = {a.stride_batch, a.stride_head, a.stride_token}, sb[3] = {b.stride_batch, b.stride_head, b.stride_token};
  const int64_t na[3] = {da.batch, da.heads, da.tokens}, nb[3] = {db.batch, db.heads, db.tokens};
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (na[i] == 1 && nb[i] == 1) continue;
    if (na[i] > 1 && nb[i] > 1 && sa[i] != sb[i]) return true;
    if (na[i] < nb[i]) return true;  // (a's strides say nothing about so many)
    dim[n++] = {sa[i], 1 - na[i], nb[i] - 1};
  }
  const int64_t bytes = static_cast<char*>(b.data) - static_cast<char*>(a.data);
  if (bytes % (int64_t)es != 0) return true;
  std::sort(dim, dim + n, [](const Dim& x, const Dim& y) { return x.stride > y.stride; });
  int64_t apart[8] = {bytes / (int64_t)es};
  int count = 1;
  for (int i = 0; i < n; ++i) {
    int64_t next[8];
    int m = 0;
    for (int c = 0; c < count && m < 8; ++c) {
      int64_t k = -apart[c] / dim[i].stride;
      if (k * dim[i].stride > -apart[c]) --k;  // floor
      for (int64_t x : {k, k + 1})
        if (x >= dim[i].lo && x <= dim[i].hi) next[m++] = apart[c] + x * dim[i].stride;
    }
    std::copy(next, next + m, apart);
    count = m;
  }
  for (int c = 0; c < count; ++c)
    if (apart[c] < da.head_dim && -apart[c] < da.head_dim) return true;
  return false;
}

// Every vector of the view starts on a 16-byte boundary.
bool rows_aligned(const ol_rows& r, const Dims& d, size_t es) {
  const int64_t ve = 16 / es;
  return aligned16(r.data) && (d.batch == 1 || r.stride_batch % ve == 0) &&
         (d.heads == 1 || r.stride_head % ve == 0) && (d.tokens == 1 || r.stride_token % ve == 0);
}

RopeView rope_view(const ol_rows* r) {
  return {static_cast<char*>(r->data), r->stride_batch, r->stride_head, r->stride_token};
}

constexpr int kRopeMaxDim = 1024;

ol_status check_rope(const ol_rope* rope, int dtype, int64_t batch, int64_t tokens, int head_dim) {
  if (!rope || !rope->turns) return OL_ERR_NULL;
  if (!valid_dtype(dtype)) return OL_ERR_DTYPE;
  if (batch < 0 || tokens < 0 || head_dim <= 0) return OL_ERR_SHAPE;
  if (rope->rot_dim < 2 || rope->rot_dim % 2 != 0 || rope->rot_dim > head_dim) return OL_ERR_SHAPE;
  if (rope->style != OL_ROPE_HALF && rope->style != OL_ROPE_INTERLEAVED) return OL_ERR_SHAPE;
  if (!(rope->magnitude > 0.f) || !std::isfinite(rope->magnitude)) return OL_ERR_SHAPE;
  if (head_dim > kRopeMaxDim || batch * tokens >= (1ll << 31)) return OL_ERR_UNSUPPORTED;
  if (!aligned16(rope->turns)) return OL_ERR_ALIGN;
  return OL_OK;
}

// The rotation works on whole 16-byte pieces: those of a pair's two elements
// (half style), or pieces of adjacent pairs.
bool rope_pieces(const ol_rope& r, int head_dim, size_t es) {
  const int ve = (int)(16 / es);
  return head_dim % ve == 0 && (r.style == OL_ROPE_HALF ? r.rot_dim / 2 : r.rot_dim) % ve == 0;
}

RopeParams rope_params(const ol_rope& r, int dtype, int batch, int tokens, int head_dim) {
  RopeParams p = {};
  p.turns = r.turns;
  p.rot_dim = r.rot_dim;
  p.style = r.style;
  p.magnitude = r.magnitude;
  p.dtype = dtype;
  p.head_dim = head_dim;
  p.batch = batch;
  p.tokens = tokens;
  return p;
}

ol_status rope_rows(const ol_rope* rope, int32_t dtype, int32_t batch, int32_t heads, int32_t tokens,
                    int32_t head_dim, const ol_rows* in, const ol_rows* out, const int32_t* positions_dev,
                    int32_t per_token, cudaStream_t s) {
  ol_status st = check_rope(rope, dtype, batch, tokens, head_dim);
  if (st != OL_OK) return st;
  if (heads < 0) return OL_ERR_SHAPE;
  if (!positions_dev) return OL_ERR_NULL;
  if (!aligned16(positions_dev)) return OL_ERR_ALIGN;
  const size_t es = elt_bytes(dtype);
  const Dims d = {batch, heads, tokens, head_dim};
  Range ri, ro;
  if ((st = check_rows(in, d, es, false, ri)) != OL_OK) return st;
  if ((st = check_rows(out, d, es, true, ro)) != OL_OK) return st;
  if (!same_view(*in, *out) && overlaps(ri, ro)) return OL_ERR_ALIAS;
  if (overlaps(ro, range_of(positions_dev, sizeof(int32_t) * (size_t)batch * (per_token ? tokens : 1))) ||
      overlaps(ro, range_of(rope->turns, sizeof(uint64_t) * (size_t)(rope->rot_dim / 2))))
    return OL_ERR_ALIAS;
  ol_stats stats = {};  // no cache takes part: the call alone is counted
  stats.calls = 1;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (d.empty()) return OL_OK;
  RopeParams p = rope_params(*rope, dtype, batch, tokens, head_dim);
  p.q_heads = heads;
  p.q = rope_view(in);
  p.q_out = rope_view(out);
  (per_token ? p.angles : p.positions) = positions_dev;
  p.vec = rope_pieces(*rope, head_dim, es) && rows_aligned(*in, d, es) && rows_aligned(*out, d, es);
  return launch_rope(p, s) == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

ol_status rope_append(int32_t layout, const void* cache_desc, void* updated, const ol_rope* rope, int32_t new_len,
                      const ol_rows* k, const ol_rows* v, int32_t q_heads, const ol_rows* q, const ol_rows* q_out,
                      const int32_t* positions_host, const int32_t* positions_dev, const int32_t* counts_host,
                      const int32_t* counts_dev, const int32_t* angles_dev, cudaStream_t s) {
  CacheView c;
  ol_status st = view_dense(layout, cache_desc, c);
  if (st != OL_OK) return st;
  if ((st = writable(c, updated)) != OL_OK) return st;
  if ((st = check_rope(rope, c.dtype, c.batch, new_len, c.head_dim)) != OL_OK) return st;
  if (!positions_host || !positions_dev || !counts_host != !counts_dev || !q != !q_out) return OL_ERR_NULL;
  if (q ? q_heads <= 0 : q_heads != 0) return OL_ERR_SHAPE;
  if (!aligned16(positions_dev) || !aligned16(counts_dev) || !aligned16(angles_dev)) return OL_ERR_ALIGN;
  const size_t es = elt_bytes(c.dtype);
  const Dims dk = {c.batch, c.kv_heads, new_len, c.head_dim}, dq = {c.batch, q_heads, new_len, c.head_dim};
  Range rk, rv, rq = {0, 0}, ro = {0, 0};
  if ((st = check_rows(k, dk, es, false, rk)) != OL_OK) return st;
  if ((st = check_rows(v, dk, es, false, rv)) != OL_OK) return st;
  if (q) {
    if ((st = check_rows(q, dq, es, false, rq)) != OL_OK) return st;
    if ((st = check_rows(q_out, dq, es, true, ro)) != OL_OK) return st;
    if (!same_view(*q, *q_out)) {
      if (overlaps(ro, rq) || overlaps(ro, rk) || overlaps(ro, rv)) return OL_ERR_ALIAS;
    } else if (!dq.empty()) {
      if (overlaps(ro, rk) && may_share(*q_out, dq, *k, dk, es)) return OL_ERR_ALIAS;
      if (overlaps(ro, rv) && may_share(*q_out, dq, *v, dk, es)) return OL_ERR_ALIAS;
    }
  }
  int64_t appended = 0;
  for (int b = 0; b < c.batch; ++b) {
    const int n = counts_host ? counts_host[b] : new_len;
    if (n < 0 || n > new_len) return OL_ERR_SHAPE;
    if (positions_host[b] < 0 || (long long)positions_host[b] + n > c.capacity) return OL_ERR_CAPACITY;
    appended += n;
  }
  const Range small[] = {range_of(positions_dev, sizeof(int32_t) * (size_t)c.batch),
                         range_of(counts_dev, counts_dev ? sizeof(int32_t) * (size_t)c.batch : 0),
                         range_of(angles_dev, angles_dev ? sizeof(int32_t) * (size_t)c.batch * new_len : 0),
                         range_of(rope->turns, sizeof(uint64_t) * (size_t)(rope->rot_dim / 2)), rk, rv, rq, ro};
  for (const Range& r : small)
    if (!r.empty() && (st = no_overlap(c, reinterpret_cast<void*>(r.lo), r.hi - r.lo)) != OL_OK) return st;
  for (int i = 0; i < 4; ++i)
    if (overlaps(small[i], ro)) return OL_ERR_ALIAS;
  if ((st = table_overlap(layout, cache_desc, c)) != OL_OK) return st;
  if (layout == OL_LAYOUT_PAGED) {
    const ol_paged_kv* pk = static_cast<const ol_paged_kv*>(cache_desc);
    if (overlaps(ro, range_of(pk->block_table, sizeof(int32_t) * (size_t)pk->batch * pk->max_pages)))
      return OL_ERR_ALIAS;
    if ((st = check_written_pages(pk, positions_host, counts_host, new_len)) != OL_OK) return st;
  }
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  ol_stats stats = {};
  stats.calls = 1;
  stats.storage_append_copied_bytes = 2ll * appended * c.kv_heads * token_payload(c);
  stats.storage_reuse_count = appended > 0 ? 2 : 0;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (dk.empty()) return OL_OK;
  RopeParams p = rope_params(*rope, c.dtype, c.batch, new_len, c.head_dim);
  p.kv_heads = c.kv_heads;
  p.k = rope_view(k);
  p.v = rope_view(v);
  p.cache = cache_ref(layout, cache_desc, c);
  p.positions = positions_dev;
  p.counts = counts_dev;
  p.angles = angles_dev;
  p.vec = rope_pieces(*rope, c.head_dim, es) && rows_aligned(*k, dk, es) && rows_aligned(*v, dk, es);
  if (q) {
    p.q_heads = q_heads;
    p.q = rope_view(q);
    p.q_out = rope_view(q_out);
    p.vec = p.vec && rows_aligned(*q, dq, es) && rows_aligned(*q_out, dq, es);
  }
  return launch_rope(p, s) == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

ol_status tree_attention(int32_t layout, const void* cache_desc, const void* q, int32_t q_heads, int32_t nodes,
                         const int32_t* lens_host, const int32_t* lens_dev, const int32_t* counts_host,
                         const int32_t* counts_dev, const uint64_t* mask_dev, const int32_t* node_positions_dev,
                         float scale, int32_t window, void* out, int32_t out_dtype, void* workspace, size_t ws_bytes,
                         cudaStream_t s) {
  CacheView c;
  ol_status st = view_dense(layout, cache_desc, c);
  if (st != OL_OK) return st;
  if (!q || !lens_host || !lens_dev || !out || !workspace || !counts_host != !counts_dev) return OL_ERR_NULL;
  if (window >= 0 && mask_dev && !node_positions_dev) return OL_ERR_NULL;
  if (q_heads <= 0 || q_heads % c.kv_heads != 0 || nodes < 1) return OL_ERR_SHAPE;
  if (c.head_dim > 256 || nodes > kTreeMaxNodes) return OL_ERR_UNSUPPORTED;
  if (!valid_dtype(out_dtype)) return OL_ERR_DTYPE;
  if (!aligned16(q) || !aligned16(lens_dev) || !aligned16(counts_dev) || !aligned16(mask_dev) ||
      !aligned16(node_positions_dev) || !aligned16(out) || !aligned16(workspace))
    return OL_ERR_ALIGN;
  for (int b = 0; b < c.batch; ++b) {
    if (lens_host[b] < 0 || lens_host[b] > c.capacity) return OL_ERR_CAPACITY;
    const int n = counts_host ? counts_host[b] : nodes;
    if (n < 0 || n > nodes) return OL_ERR_SHAPE;
    if (n > lens_host[b]) return OL_ERR_CAPACITY;
  }
  const int words = (nodes + 63) / 64;
  const size_t vectors = (size_t)c.batch * q_heads * nodes;
  const size_t need = tree_workspace_bytes(c.batch, q_heads, c.kv_heads, c.head_dim, nodes);
  if (ws_bytes < need) return OL_ERR_WORKSPACE;
  const Range ro = range_of(out, vectors * c.head_dim * elt_bytes(out_dtype)), rw = range_of(workspace, need);
  const size_t tree = (size_t)c.batch * nodes;
  const Range in[] = {range_of(q, vectors * c.head_dim * elt_bytes(c.dtype)),
                      range_of(lens_dev, sizeof(int32_t) * (size_t)c.batch),
                      range_of(counts_dev, counts_dev ? sizeof(int32_t) * (size_t)c.batch : 0),
                      range_of(mask_dev, mask_dev ? sizeof(uint64_t) * tree * words : 0),
                      range_of(node_positions_dev, node_positions_dev ? sizeof(int32_t) * tree : 0)};
  for (const Range& r : in) {
    if (!r.empty() && (st = no_overlap(c, reinterpret_cast<void*>(r.lo), r.hi - r.lo)) != OL_OK) return st;
    if (overlaps(r, ro) || overlaps(r, rw)) return OL_ERR_ALIAS;
  }
  if ((st = no_overlap(c, out, ro.hi - ro.lo)) != OL_OK) return st;
  if ((st = no_overlap(c, workspace, need)) != OL_OK) return st;
  if (overlaps(ro, rw)) return OL_ERR_ALIAS;
  if ((st = table_overlap(layout, cache_desc, c)) != OL_OK) return st;
  ol_stats stats = {};
  stats.calls = 1;
  const ol_paged_kv* pk = layout == OL_LAYOUT_PAGED ? static_cast<const ol_paged_kv*>(cache_desc) : nullptr;
  if (pk) {
    const Range rt = range_of(pk->block_table, sizeof(int32_t) * (size_t)pk->batch * pk->max_pages);
    if (overlaps(rt, ro) || overlaps(rt, rw)) return OL_ERR_ALIAS;
  }
  for (int b = 0; b < c.batch; ++b) {
    // tokens that some node may see
    const int n = counts_host ? counts_host[b] : nodes;
    if (n == 0) continue;
    const int prefix = lens_host[b] - n;
    const int lo = window < 0 || prefix <= window ? 0 : prefix - window;
    if (pk && pages_outside(pk->block_table_host + (size_t)b * pk->max_pages, lo / pk->page_size,
                            (lens_host[b] - 1) / pk->page_size + 1, pk->num_pages))
      return OL_ERR_PAGE;
    stats.attended_tokens += (int64_t)n * (lens_host[b] - lo) * c.kv_heads;
    stats.kv_payload_bytes_read += 2ll * (lens_host[b] - lo) * c.kv_heads * token_payload(c);
  }
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  TreeParams p = {};
  p.cache = cache_ref(layout, cache_desc, c);
  p.dtype = c.dtype;
  p.batch = c.batch;
  p.q_heads = q_heads;
  p.kv_heads = c.kv_heads;
  p.group = q_heads / c.kv_heads;
  p.head_dim = c.head_dim;
  p.nodes = nodes;
  p.words = words;
  p.q = q;
  p.lens = lens_dev;
  p.counts = counts_dev;
  p.mask = mask_dev;
  p.node_pos = node_positions_dev;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)c.head_dim)) * 1.4426950408889634f;
  p.window = window < 0 ? -1 : window;
  p.out = out;
  p.out_dtype = out_dtype;
  p.status = static_cast<int32_t*>(workspace);
  char* const splits = static_cast<char*>(workspace) + tree_splits_offset(c.batch, c.kv_heads, nodes);
  p.splits = reinterpret_cast<TreeSplit*>(splits);
  p.partials = reinterpret_cast<float*>(splits + kTreeSplitBytes);
  const bool fast = fast_tree_supported(p);
  if (fast)
    plan_fast_tree(p, sm_count_cached());
  else
    plan_generic_tree(p, sm_count_cached());
  if (!tree_counts_fit(p)) return OL_ERR_UNSUPPORTED;
  stats.workspace_bytes = (int64_t)need;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (c.batch == 0) return OL_OK;
  cudaError_t e = fast ? launch_fast_tree(p, s) : launch_generic_tree(p, s);
  if (e == cudaSuccess) e = launch_tree_merge(p, s);
  return e == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

ol_status tree_keep(int32_t layout, const void* cache_desc, void* updated, int32_t nodes, const int32_t* starts_host,
                    const int32_t* starts_dev, const int32_t* counts_host, const int32_t* counts_dev,
                    const int32_t* kept_dev, const int32_t* kept_counts_dev, void* workspace, cudaStream_t s) {
  CacheView c;
  ol_status st = view_dense(layout, cache_desc, c);
  if (st != OL_OK) return st;
  if ((st = writable(c, updated)) != OL_OK) return st;
  if (!starts_host || !starts_dev || !kept_dev || !kept_counts_dev || !counts_host != !counts_dev) return OL_ERR_NULL;
  if (nodes < 1) return OL_ERR_SHAPE;
  if (!aligned16(starts_dev) || !aligned16(counts_dev) || !aligned16(kept_dev) || !aligned16(kept_counts_dev) ||
      !aligned16(workspace))
    return OL_ERR_ALIGN;
  for (int b = 0; b < c.batch; ++b) {
    const int n = counts_host ? counts_host[b] : nodes;
    if (n < 0 || n > nodes) return OL_ERR_SHAPE;
    if (starts_host[b] < 0 || (long long)starts_host[b] + n > c.capacity) return OL_ERR_CAPACITY;
  }
  if ((st = no_overlap(c, starts_dev, sizeof(int32_t) * (size_t)c.batch)) != OL_OK ||
      (counts_dev && (st = no_overlap(c, counts_dev, sizeof(int32_t) * (size_t)c.batch)) != OL_OK) ||
      (st = no_overlap(c, kept_dev, sizeof(int32_t) * (size_t)c.batch * nodes)) != OL_OK ||
      (st = no_overlap(c, kept_counts_dev, sizeof(int32_t) * (size_t)c.batch)) != OL_OK ||
      (st = no_overlap(c, workspace, kStatusBytes)) != OL_OK ||
      (st = table_overlap(layout, cache_desc, c)) != OL_OK)
    return st;
  const Range status = range_of(workspace, workspace ? sizeof(int32_t) : 0);
  for (const Range& r : {range_of(starts_dev, sizeof(int32_t) * (size_t)c.batch),
                         range_of(counts_dev, counts_dev ? sizeof(int32_t) * (size_t)c.batch : 0),
                         range_of(kept_dev, sizeof(int32_t) * (size_t)c.batch * nodes),
                         range_of(kept_counts_dev, sizeof(int32_t) * (size_t)c.batch)})
    if (overlaps(r, status)) return OL_ERR_ALIAS;
  if (layout == OL_LAYOUT_PAGED) {
    const ol_paged_kv* pk = static_cast<const ol_paged_kv*>(cache_desc);
    if (overlaps(status, range_of(pk->block_table, sizeof(int32_t) * (size_t)pk->batch * pk->max_pages)))
      return OL_ERR_ALIAS;
  }
  if (layout == OL_LAYOUT_PAGED &&
      (st = check_written_pages(static_cast<const ol_paged_kv*>(cache_desc), starts_host, counts_host, nodes)) != OL_OK)
    return st;
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  ol_stats stats = {};  // what moves is known on the device only: the call alone is counted
  stats.calls = 1;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (c.batch == 0) return OL_OK;
  KeepParams p = {};
  p.cache = cache_ref(layout, cache_desc, c);
  p.dtype = c.dtype;
  p.head_dim = c.head_dim;
  p.nodes = nodes;
  p.starts = starts_dev;
  p.kept = kept_dev;
  p.counts = kept_counts_dev;
  p.drafted = counts_dev;
  p.status = static_cast<int32_t*>(workspace);
  return launch_tree_keep(p, s) == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

}  // namespace
}  // namespace ol

using namespace ol;

extern "C" {

ol_status ol_rope_turns(int32_t scaling, int32_t rot_dim, double base, double factor, double original_len,
                        double low, double high, uint64_t* turns_host) {
  if (!turns_host) return OL_ERR_NULL;
  if (rot_dim < 2 || rot_dim % 2 != 0) return OL_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return OL_ERR_SHAPE;
  if (scaling < OL_ROPE_UNSCALED || scaling > OL_ROPE_BY_PARTS) return OL_ERR_SHAPE;
  if (!(factor >= 1.0) || !std::isfinite(factor)) return OL_ERR_SHAPE;
  if (scaling == OL_ROPE_NTK && rot_dim < 4) return OL_ERR_SHAPE;
  if (scaling == OL_ROPE_BY_PARTS && (!(original_len > 0.0) || !std::isfinite(original_len) || !(low >= 0.0) ||
                                      !(low < high) || !std::isfinite(high)))
    return OL_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925286766559;
  const double b = scaling == OL_ROPE_NTK ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
  if (!std::isfinite(b)) return OL_ERR_SHAPE;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == OL_ROPE_LINEAR) f /= factor;
    if (scaling == OL_ROPE_BY_PARTS) {
      const double r = original_len * f / two_pi;
      const double k = std::min(1.0, std::max(0.0, (r - low) / (high - low)));
      f = (1.0 - k) * f / factor + k * f;
    }
    // f <= 1 radian per position: less than a turn, so the 2^-64 turns fit (a
    // double carries 53 of the 64 bits: 2^-53 of a turn's share per position)
    turns_host[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64));
  }
  return OL_OK;
}

ol_status ol_rope_rows(const ol_rope* rope, int32_t dtype, int32_t batch, int32_t heads, int32_t tokens,
                       int32_t head_dim, const ol_rows* in, const ol_rows* out, const int32_t* positions_dev,
                       int32_t per_token, ol_stream stream) {
  return guarded_call([&] {
    return rope_rows(rope, dtype, batch, heads, tokens, head_dim, in, out, positions_dev, per_token,
                     static_cast<cudaStream_t>(stream));
  });
}

ol_status ol_rope_append(int32_t layout, const void* cache_desc, void* updated, const ol_rope* rope, int32_t new_len,
                         const ol_rows* k, const ol_rows* v, int32_t q_heads, const ol_rows* q, const ol_rows* q_out,
                         const int32_t* positions_host, const int32_t* positions_dev, const int32_t* counts_host,
                         const int32_t* counts_dev, const int32_t* angles_dev, ol_stream stream) {
  return guarded_call([&] {
    return rope_append(layout, cache_desc, updated, rope, new_len, k, v, q_heads, q, q_out, positions_host,
                       positions_dev, counts_host, counts_dev, angles_dev, static_cast<cudaStream_t>(stream));
  });
}

size_t ol_workspace_size_tree(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t nodes) {
  if (batch < 0 || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 || nodes < 1) return 0;
  return tree_workspace_bytes(batch, q_heads, kv_heads, head_dim, nodes);
}

ol_status ol_tree_attention(int32_t layout, const void* cache_desc, const void* q, int32_t q_heads, int32_t nodes,
                            const int32_t* lens_host, const int32_t* lens_dev, const int32_t* counts_host,
                            const int32_t* counts_dev, const uint64_t* mask_dev, const int32_t* node_positions_dev,
                            float scale, int32_t window, void* out, int32_t out_dtype, void* workspace,
                            size_t ws_bytes, ol_stream stream) {
  return guarded_call([&] {
    return tree_attention(layout, cache_desc, q, q_heads, nodes, lens_host, lens_dev, counts_host, counts_dev,
                          mask_dev, node_positions_dev, scale, window, out, out_dtype, workspace, ws_bytes,
                          static_cast<cudaStream_t>(stream));
  });
}

ol_status ol_tree_keep(int32_t layout, const void* cache_desc, void* updated, int32_t nodes,
                       const int32_t* starts_host, const int32_t* starts_dev, const int32_t* kept_dev,
                       const int32_t* kept_counts_dev, void* workspace, ol_stream stream) {
  return guarded_call([&] {
    return tree_keep(layout, cache_desc, updated, nodes, starts_host, starts_dev, nullptr, nullptr, kept_dev,
                     kept_counts_dev, workspace, static_cast<cudaStream_t>(stream));
  });
}

ol_status ol_tree_keep_counted(int32_t layout, const void* cache_desc, void* updated, int32_t nodes,
                               const int32_t* starts_host, const int32_t* starts_dev, const int32_t* counts_host,
                               const int32_t* counts_dev, const int32_t* kept_dev, const int32_t* kept_counts_dev,
                               void* workspace, ol_stream stream) {
  return guarded_call([&] {
    return tree_keep(layout, cache_desc, updated, nodes, starts_host, starts_dev, counts_host, counts_dev, kept_dev,
                     kept_counts_dev, workspace, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
