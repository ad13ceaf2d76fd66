// ol_host.h -- host-side validation shared by the translation units of the C
// ABI (ol_api.cpp, ol_draft_api.cpp): descriptor views, overlap, ownership and
// page checks, the statistics record. Not part of the public ABI.
#pragma once

#include "ol_internal.h"
#include "ol_launch.h"

namespace ol {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  bool empty() const { return hi <= lo; }
};
Range range_of(const void* p, size_t bytes);
bool overlaps(Range a, Range b);
bool aligned16(const void* p);

struct CacheView {
  int layout;
  int dtype;
  int batch, kv_heads, head_dim, capacity;
  int access;
  bool history_stable;
  uint64_t owner;
  void* alias_ptr;  // pointer that `updated` must equal
  Range ranges[3];  // cache storage (INT4: three planes)
  int nranges;
};
ol_status view_contiguous(const ol_kv_cache* c, CacheView& v);
ol_status view_paged(const ol_paged_kv* c, CacheView& v);

// OL_ERR_ALIAS where the buffer overlaps a cache storage range.
ol_status no_overlap(const CacheView& v, const void* p, size_t bytes);
ol_status writable(const CacheView& v, const void* updated);
ol_status check_owner(const Range* ranges, int nranges, uint64_t owner);
// Every page a row reads or writes is inside the pool (see ol_api.cpp).
ol_status check_pages(const ol_paged_kv* c, const int32_t* lens_or_pos, int new_len, bool append, int window);

bool fault_injected();
size_t elt_bytes(int dtype);
bool valid_dtype(int d);
int sm_count_cached();

// Adds the record of a validated call to this thread's statistics.
void record(const ol_stats& s);
// Stored payload bytes of one token of one kv head in one plane (K or V).
int64_t token_payload(const CacheView& v);

// ------------------------------------------- views of vectors, written pages (ol_draft_api.cpp)

struct Dims {
  int64_t batch, heads, tokens, head_dim;
  bool empty() const { return batch == 0 || heads == 0 || tokens == 0; }
};
// A view's pointer, strides and extent; `out` also wants vectors that do not overlap one another.
ol_status check_rows(const ol_rows* r, const Dims& d, size_t es, bool out, Range& range);
bool same_view(const ol_rows& a, const ol_rows& b);
// Whether a vector of `a`, a view that may be written, and one of `b` may share an element.
bool may_share(const ol_rows& a, const Dims& da, const ol_rows& b, const Dims& db, size_t es);
// Every vector of the view starts on a 16-byte boundary.
bool rows_aligned(const ol_rows& r, const Dims& d, size_t es);
// Whether one of a row's block-table entries [first, end) is outside the pool.
bool pages_outside(const int32_t* row, int first, int end, int num_pages);
// Pages that tokens [first[b], first[b] + n_b) of the rows are written to: in the pool, and none of them twice.
ol_status check_written_pages(const ol_paged_kv* c, const int32_t* first, const int32_t* counts, int n);

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

}  // namespace ol
