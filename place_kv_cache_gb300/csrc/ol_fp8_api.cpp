// ol_fp8_api.cpp -- the C ABI of the E4M3 cache (see include/ol.h): the
// quantising append, reading back, attention. Host-side validation and dispatch;
// as in ol_api.cpp every check runs before any launch.
#include <cmath>

#include "ol_fp8.h"
#include "ol_host.h"

namespace ol {
namespace {

constexpr int kMaxDim = 256;

size_t blocks_of(int tokens, int block) { return ((size_t)tokens + block - 1) / block; }

ol_status view_fp8(const ol_fp8_kv* c, CacheView& v) {
  if (!c || !c->codes || !c->scales || !c->block_table != !c->block_table_host) return OL_ERR_NULL;
  const bool paged = c->block_table != nullptr;
  if (c->batch < 0 || c->kv_heads <= 0 || c->capacity < 0 || c->head_dim <= 0) return OL_ERR_SHAPE;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return OL_ERR_SHAPE;
  if (paged ? c->num_pages <= 0 || c->page_size <= 0 || c->max_pages < 0 || c->capacity != 0 ||
                  c->page_size % c->block != 0
            : c->num_pages != 0 || c->page_size != 0 || c->max_pages != 0)
    return OL_ERR_SHAPE;
  if ((long long)c->max_pages * c->page_size > (1ll << 30)) return OL_ERR_SHAPE;
  if (c->head_dim % 16 != 0 || c->head_dim > kMaxDim) return OL_ERR_UNSUPPORTED;
  if (!aligned16(c->codes) || !aligned16(c->scales) || !aligned16(c->block_table)) return OL_ERR_ALIGN;
  v = {};
  v.batch = c->batch;
  v.kv_heads = c->kv_heads;
  v.head_dim = c->head_dim;
  v.capacity = paged ? c->max_pages * c->page_size : c->capacity;
  v.access = c->access & ~OL_HISTORY_STABLE;
  v.history_stable = (c->access & OL_HISTORY_STABLE) != 0;
  v.owner = c->owner;
  v.alias_ptr = c->codes;
  const size_t heads = 2ull * (paged ? c->num_pages : c->batch) * c->kv_heads;
  const int tokens = paged ? c->page_size : c->capacity;
  v.ranges[0] = range_of(c->codes, heads * tokens * c->head_dim);
  v.ranges[1] = range_of(c->scales, heads * blocks_of(tokens, c->block) * sizeof(float));
  v.nranges = 2;
  if (overlaps(v.ranges[0], v.ranges[1])) return OL_ERR_ALIAS;
  return OL_OK;
}

Range table_range(const ol_fp8_kv* c) {
  return range_of(c->block_table, c->block_table ? sizeof(int32_t) * (size_t)c->batch * c->max_pages : 0);
}

// The pool as a plain paged cache, for the checks of written pages.
ol_paged_kv paged_shape_of(const ol_fp8_kv* c) {
  ol_paged_kv k = {};
  k.block_table_host = c->block_table_host;
  k.num_pages = c->num_pages;
  k.page_size = c->page_size;
  k.batch = c->batch;
  k.max_pages = c->max_pages;
  return k;
}

Fp8Cache fp8_ref(const ol_fp8_kv* c, const CacheView& v) {
  Fp8Cache r = {};
  r.codes = c->codes;
  r.scales = c->scales;
  r.block_table = c->block_table;
  r.batch = c->batch;
  r.kv_heads = c->kv_heads;
  r.capacity = v.capacity;
  r.head_dim = c->head_dim;
  r.num_pages = c->num_pages;
  r.page_size = c->page_size;
  r.max_pages = c->max_pages;
  r.block_log2 = c->block == 16 ? 4 : c->block == 32 ? 5 : c->block == 64 ? 6 : 7;
  return r;
}

RopeView view_of(const ol_rows* r) {
  return {static_cast<char*>(r->data), r->stride_batch, r->stride_head, r->stride_token};
}

// Places [first[b], first[b] + n) of every row; sums the tokens and the blocks they lie in.
ol_status check_places(const CacheView& v, int block, const int32_t* first, const int32_t* counts, int most,
                       int64_t& tokens, int64_t& blocks) {
  tokens = blocks = 0;
  for (int b = 0; b < v.batch; ++b) {
    const int n = counts ? counts[b] : most;
    if (n < 0 || n > most) return OL_ERR_SHAPE;
    if (first[b] < 0 || (long long)first[b] + n > v.capacity) return OL_ERR_CAPACITY;
    tokens += n;
    if (n > 0) blocks += (first[b] + n - 1) / block - first[b] / block + 1;
  }
  return OL_OK;
}

ol_status fp8_append(const ol_fp8_kv* kv, void* updated, int32_t dtype, int32_t new_len, const ol_rows* k,
                     const ol_rows* v, const int32_t* positions_host, const int32_t* positions_dev,
                     const int32_t* counts_host, const int32_t* counts_dev, cudaStream_t s) {
  CacheView c;
  ol_status st = view_fp8(kv, c);
  if (st != OL_OK) return st;
  if ((st = writable(c, updated)) != OL_OK) return st;
  if (!valid_dtype(dtype)) return OL_ERR_DTYPE;
  if (new_len < 0) return OL_ERR_SHAPE;
  if (!positions_host || !positions_dev || !counts_host != !counts_dev) return OL_ERR_NULL;
  if (!aligned16(positions_dev) || !aligned16(counts_dev)) return OL_ERR_ALIGN;
  const size_t es = elt_bytes(dtype);
  const Dims d = {c.batch, c.kv_heads, new_len, c.head_dim};
  Range rk, rv;
  if ((st = check_rows(k, d, es, false, rk)) != OL_OK) return st;
  if ((st = check_rows(v, d, es, false, rv)) != OL_OK) return st;
  int64_t tokens, touched;
  if ((st = check_places(c, kv->block, positions_host, counts_host, new_len, tokens, touched)) != OL_OK) return st;
  const size_t rows = sizeof(int32_t) * (size_t)c.batch;
  for (const Range& r : {rk, rv, range_of(positions_dev, rows), range_of(counts_dev, counts_dev ? rows : 0),
                         table_range(kv)})
    if (!r.empty() && (st = no_overlap(c, reinterpret_cast<void*>(r.lo), r.hi - r.lo)) != OL_OK) return st;
  if (kv->block_table) {
    const ol_paged_kv shape = paged_shape_of(kv);
    if ((st = check_written_pages(&shape, positions_host, counts_host, new_len)) != OL_OK) return st;
  }
  // blocks of a row's tokens, wherever they begin
  const int64_t blocks = new_len > 0 ? ((int64_t)new_len + kv->block - 2) / kv->block + 1 : 0;
  if (blocks * c.batch * c.kv_heads >= (1ll << 31)) return OL_ERR_UNSUPPORTED;
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  ol_stats stats = {};
  stats.calls = 1;
  stats.storage_append_copied_bytes = 2ll * c.kv_heads * (tokens * c.head_dim + touched * (int64_t)sizeof(float));
  stats.storage_reuse_count = tokens > 0 ? 2 : 0;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (d.empty()) return OL_OK;
  Fp8AppendParams p = {};
  p.cache = fp8_ref(kv, c);
  p.dtype = dtype;
  p.new_len = new_len;
  p.blocks = (int)blocks;
  p.in[0] = view_of(k);
  p.in[1] = view_of(v);
  p.positions = positions_dev;
  p.counts = counts_dev;
  p.vec = rows_aligned(*k, d, es) && rows_aligned(*v, d, es);
  return launch_fp8_append(p, s) == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

ol_status fp8_read(const ol_fp8_kv* kv, int32_t dtype, int32_t tokens, const ol_rows* k_out, const ol_rows* v_out,
                   const int32_t* starts_host, const int32_t* starts_dev, const int32_t* counts_host,
                   const int32_t* counts_dev, cudaStream_t s) {
  CacheView c;
  ol_status st = view_fp8(kv, c);
  if (st != OL_OK) return st;
  if (!valid_dtype(dtype)) return OL_ERR_DTYPE;
  if (tokens < 0) return OL_ERR_SHAPE;
  if ((!k_out && !v_out) || !starts_host || !starts_dev || !counts_host != !counts_dev) return OL_ERR_NULL;
  if (!aligned16(starts_dev) || !aligned16(counts_dev)) return OL_ERR_ALIGN;
  const size_t es = elt_bytes(dtype);
  const Dims d = {c.batch, c.kv_heads, tokens, c.head_dim};
  const ol_rows* const out[2] = {k_out, v_out};
  const size_t rows = sizeof(int32_t) * (size_t)c.batch;
  const Range in[] = {range_of(starts_dev, rows), range_of(counts_dev, counts_dev ? rows : 0), table_range(kv)};
  Range ro[2] = {{0, 0}, {0, 0}};
  for (int i = 0; i < 2; ++i) {
    if (!out[i]) continue;
    if ((st = check_rows(out[i], d, es, true, ro[i])) != OL_OK) return st;
    if (!ro[i].empty() && (st = no_overlap(c, reinterpret_cast<void*>(ro[i].lo), ro[i].hi - ro[i].lo)) != OL_OK) return st;
    for (const Range& r : in)
      if (overlaps(r, ro[i])) return OL_ERR_ALIAS;
  }
  if (overlaps(ro[0], ro[1]) && may_share(*k_out, d, *v_out, d, es)) return OL_ERR_ALIAS;
  int64_t read, touched;
  if ((st = check_places(c, kv->block, starts_host, counts_host, tokens, read, touched)) != OL_OK) return st;
  if (kv->block_table)
    for (int b = 0; b < c.batch; ++b) {
      const int n = counts_host ? counts_host[b] : tokens;
      if (n > 0 && pages_outside(kv->block_table_host + (size_t)b * kv->max_pages, starts_host[b] / kv->page_size,
                                 (starts_host[b] + n - 1) / kv->page_size + 1, kv->num_pages))
        return OL_ERR_PAGE;
    }
  if ((int64_t)c.batch * c.kv_heads * tokens >= (1ll << 31)) return OL_ERR_UNSUPPORTED;
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  const int planes = (k_out != nullptr) + (v_out != nullptr);
  ol_stats stats = {};
  stats.calls = 1;
  stats.dequantized_bytes = 4 * planes * read * c.kv_heads * c.head_dim;
  stats.kv_payload_bytes_read = planes * c.kv_heads * (read * c.head_dim + touched * (int64_t)sizeof(float));
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (d.empty()) return OL_OK;
  Fp8ReadParams p = {};
  p.cache = fp8_ref(kv, c);
  p.dtype = dtype;
  p.tokens = tokens;
  p.vec = 1;
  for (int i = 0; i < 2; ++i)
    if (out[i]) {
      p.out[i] = view_of(out[i]);
      p.vec = p.vec && rows_aligned(*out[i], d, es);
    }
  p.starts = starts_dev;
  p.counts = counts_dev;
  return launch_fp8_read(p, s) == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

ol_status fp8_attention(const ol_fp8_kv* kv, int32_t dtype, const void* q, int32_t q_heads, int32_t new_len,
                        const int32_t* lens_host, const int32_t* lens_dev, const int32_t* counts_host,
                        const int32_t* counts_dev, float scale, int32_t window, void* out, int32_t out_dtype,
                        void* workspace, size_t ws_bytes, cudaStream_t s) {
  CacheView c;
  ol_status st = view_fp8(kv, c);
  if (st != OL_OK) return st;
  if (!q || !lens_host || !lens_dev || !out || !workspace || !counts_host != !counts_dev) return OL_ERR_NULL;
  if (q_heads <= 0 || q_heads % c.kv_heads != 0 || new_len < 1) return OL_ERR_SHAPE;
  if (new_len > kTreeMaxNodes) return OL_ERR_UNSUPPORTED;
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return OL_ERR_DTYPE;
  if (!aligned16(q) || !aligned16(lens_dev) || !aligned16(counts_dev) || !aligned16(out) || !aligned16(workspace))
    return OL_ERR_ALIGN;
  for (int b = 0; b < c.batch; ++b) {
    if (lens_host[b] < 0 || lens_host[b] > c.capacity) return OL_ERR_CAPACITY;
    const int n = counts_host ? counts_host[b] : new_len;
    if (n < 0 || n > new_len) return OL_ERR_SHAPE;
    if (n > lens_host[b]) return OL_ERR_CAPACITY;
  }
  const size_t vectors = (size_t)c.batch * q_heads * new_len;
  const size_t need = tree_workspace_bytes(c.batch, q_heads, c.kv_heads, c.head_dim, new_len);
  if (ws_bytes < need) return OL_ERR_WORKSPACE;
  const Range ro = range_of(out, vectors * c.head_dim * elt_bytes(out_dtype)), rw = range_of(workspace, need);
  const size_t rows = sizeof(int32_t) * (size_t)c.batch;
  for (const Range& r : {range_of(q, vectors * c.head_dim * elt_bytes(dtype)), range_of(lens_dev, rows),
                         range_of(counts_dev, counts_dev ? rows : 0), table_range(kv)}) {
    if (!r.empty() && (st = no_overlap(c, reinterpret_cast<void*>(r.lo), r.hi - r.lo)) != OL_OK) return st;
    if (overlaps(r, ro) || overlaps(r, rw)) return OL_ERR_ALIAS;
  }
  if ((st = no_overlap(c, out, ro.hi - ro.lo)) != OL_OK) return st;
  if ((st = no_overlap(c, workspace, need)) != OL_OK) return st;
  if (overlaps(ro, rw)) return OL_ERR_ALIAS;
  ol_stats stats = {};
  stats.calls = 1;
  for (int b = 0; b < c.batch; ++b) {
    const int n = counts_host ? counts_host[b] : new_len;
    if (n == 0) continue;
    const int prefix = lens_host[b] - n;
    const int lo = window < 0 || prefix <= window ? 0 : prefix - window;  // tokens [lo, len) that some query sees
    if (kv->block_table && pages_outside(kv->block_table_host + (size_t)b * kv->max_pages, lo / kv->page_size,
                                         (lens_host[b] - 1) / kv->page_size + 1, kv->num_pages))
      return OL_ERR_PAGE;
    const int64_t seen = lens_host[b] - lo, blocks = (lens_host[b] - 1) / kv->block - lo / kv->block + 1;
    stats.attended_tokens += n * seen * c.kv_heads;
    stats.dequantized_bytes += 8 * seen * c.kv_heads * c.head_dim;
    stats.kv_payload_bytes_read += 2 * c.kv_heads * (seen * c.head_dim + blocks * (int64_t)sizeof(float));
  }
  if ((st = check_owner(c.ranges, c.nranges, c.owner)) != OL_OK) return st;
  Fp8AttnParams p = {};
  p.cache = fp8_ref(kv, c);
  TreeParams& t = p.t;
  t.cache.block_table = kv->block_table;
  t.cache.batch = c.batch;
  t.cache.kv_heads = c.kv_heads;
  t.cache.capacity = c.capacity;
  t.cache.num_pages = kv->num_pages;
  t.cache.page_size = kv->page_size;
  t.cache.max_pages = kv->max_pages;
  t.dtype = dtype;
  t.batch = c.batch;
  t.q_heads = q_heads;
  t.kv_heads = c.kv_heads;
  t.group = q_heads / c.kv_heads;
  t.head_dim = c.head_dim;
  t.nodes = new_len;
  t.q = q;
  t.lens = lens_dev;
  t.counts = counts_dev;
  t.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)c.head_dim)) * 1.4426950408889634f;
  t.window = window < 0 ? -1 : window;
  t.out = out;
  t.out_dtype = out_dtype;
  t.status = static_cast<int32_t*>(workspace);
  char* const splits = static_cast<char*>(workspace) + tree_splits_offset(c.batch, c.kv_heads, new_len);
  t.splits = reinterpret_cast<TreeSplit*>(splits);
  t.partials = reinterpret_cast<float*>(splits + kTreeSplitBytes);
  t.ticket = static_cast<uint32_t*>(workspace) + kTreeTicketWord;
  plan_fp8_attention(p, sm_count_cached());
  if (!tree_counts_fit(t)) return OL_ERR_UNSUPPORTED;
  stats.workspace_bytes = (int64_t)need;
  record(stats);
  if (fault_injected()) return OL_ERR_INJECTED;
  if (c.batch == 0 || c.capacity == 0) return OL_OK;  // (there are no tokens)
  cudaError_t e = launch_fp8_attention(p, s);
  if (e == cudaSuccess) e = launch_tree_merge(t, s);
  return e == cudaSuccess ? OL_OK : OL_ERR_CUDA;
}

}  // namespace
}  // namespace ol

using namespace ol;

extern "C" {

ol_status ol_fp8kv_append(const ol_fp8_kv* kv, void* updated, int32_t dtype, int32_t new_len, const ol_rows* k,
                          const ol_rows* v, const int32_t* positions_host, const int32_t* positions_dev,
                          const int32_t* counts_host, const int32_t* counts_dev, ol_stream stream) {
  return guarded_call([&] {
    return fp8_append(kv, updated, dtype, new_len, k, v, positions_host, positions_dev, counts_host, counts_dev,
                      static_cast<cudaStream_t>(stream));
  });
}

ol_status ol_fp8kv_read(const ol_fp8_kv* kv, int32_t dtype, int32_t tokens, const ol_rows* k_out, const ol_rows* v_out,
                        const int32_t* starts_host, const int32_t* starts_dev, const int32_t* counts_host,
                        const int32_t* counts_dev, ol_stream stream) {
  return guarded_call([&] {
    return fp8_read(kv, dtype, tokens, k_out, v_out, starts_host, starts_dev, counts_host, counts_dev,
                    static_cast<cudaStream_t>(stream));
  });
}

size_t ol_workspace_size_fp8kv(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t new_len) {
  return ol_workspace_size_tree(batch, q_heads, kv_heads, head_dim, new_len);
}

ol_status ol_fp8kv_attention(const ol_fp8_kv* kv, int32_t dtype, const void* q, int32_t q_heads, int32_t new_len,
                             const int32_t* lens_host, const int32_t* lens_dev, const int32_t* counts_host,
                             const int32_t* counts_dev, float scale, int32_t window, void* out, int32_t out_dtype,
                             void* workspace, size_t ws_bytes, ol_stream stream) {
  return guarded_call([&] {
    return fp8_attention(kv, dtype, q, q_heads, new_len, lens_host, lens_dev, counts_host, counts_dev, scale, window,
                         out, out_dtype, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
