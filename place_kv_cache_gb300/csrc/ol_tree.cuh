// ol_tree.cuh -- device helpers of the tree kernels: the walk over a CTA's
// share of the work, visibility, addresses of cache rows, outputs and slots.
#pragma once

#include <atomic>

#include "ol_common.cuh"
#include "ol_draft.h"

namespace ol {

// Row index (in head_dim elements) of token t in a cache plane; -1 where the
// block table names no page of the pool.
__device__ __forceinline__ long long cache_row(const CacheRef& c, int plane, int b, int g, int t) {
  if (!c.block_table) return (((long long)plane * c.batch + b) * c.kv_heads + g) * c.capacity + t;
  const int page = c.block_table[(size_t)b * c.max_pages + t / c.page_size];
  if (page < 0 || page >= c.num_pages) return -1;
  return (((long long)plane * c.num_pages + page) * c.kv_heads + g) * c.page_size + t % c.page_size;
}

// Row of q and out of the (head, node) row r of kv head g.
__device__ __forceinline__ size_t tree_out_row(const TreeParams& p, int b, int g, int r) {
  return ((size_t)b * p.q_heads + (size_t)g * p.group) * p.nodes + r;
}

__device__ __forceinline__ float* tree_slot(const TreeParams& p, int slot) {
  return p.partials + slot * tree_slot_floats(p.rows_per_unit, p.head_dim);
}

// Position of a node: no lower than its row's prefix length.
__device__ __forceinline__ int tree_position(const TreeParams& p, const TreeRow& row, int b, int node) {
  if (!p.node_pos) return row.prefix + min(node, row.count);  // (of nodes past the count: whatever fits an int)
  return max(row.prefix, p.node_pos[(size_t)b * p.nodes + node]);
}

// Lowest prefix token that a node sees (with a window).
__device__ __forceinline__ int tree_low(const TreeParams& p, const TreeRow& row, int b, int node) {
  const int at = tree_position(p, row, b, node);
  return at <= p.window ? 0 : at - p.window;
}

// Whether a node sees drafted token j (j < count).
__device__ __forceinline__ bool tree_sees_drafted(const TreeParams& p, const TreeRow& row, int b, int node, int j) {
  if (p.mask) {
    const uint64_t w = p.mask[((size_t)b * p.nodes + node) * p.words + j / 64];
    if (!(w >> (j % 64) & 1)) return false;
  } else if (j > node) {
    return false;
  }
  return p.window < 0 ||
         (long long)tree_position(p, row, b, node) - tree_position(p, row, b, j) <= p.window;
}

// Bits [a, b) of a 32-bit word (a and b may lie outside it).
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0;
  return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// Visibility of tokens [t, t + 32) for a node, as bits, but for the window among
// drafted tokens. v: the drafted ones' mask bits (mask_bits; ignored for a chain).
__device__ __forceinline__ uint32_t visible_bits(bool chain, uint32_t v, int prefix, int count, int node, int low, int t) {
  const int j0 = t - prefix;  // drafted index of bit 0
  const uint32_t tree = chain ? bit_range(-32, node + 1 - j0) : v;
  return bit_range(low - t, prefix - t) | (tree & bit_range(-j0, count - j0));
}
// Bits [j0, j0 + 32) of a node's mask words m, which have bits [j0, j0 + 32) or more (j0 > -32).
__device__ __forceinline__ uint32_t mask_bits(const uint64_t* m, int words, int j0) {
  if (j0 < 0) return (uint32_t)m[0] << -j0;
  const int w = j0 / 64, s = j0 % 64;
  uint64_t v = m[w] >> s;
  if (s > 32 && w + 1 < words) v |= m[w + 1] << (64 - s);
  return (uint32_t)v;
}
// The same for tokens [t, t + 64) of a node with mask words m (NULL: a chain).
__device__ __forceinline__ uint64_t bit_range64(int a, int b) {
  a = max(a, 0);
  b = min(b, 64);
  return a >= b ? 0 : ~0ull >> (64 - b) & ~0ull << a;
}
static __device__ __noinline__ uint64_t visible64(const uint64_t* m, int words, int prefix, int count, int node, int low,
                                                  int t) {
  const uint64_t bits = bit_range64(low - t, prefix - t);
  const int j0 = t - prefix;
  if (j0 <= -64 || j0 >= count) return bits;
  uint64_t tree;
  if (!m) {
    tree = bit_range64(0, node + 1 - j0);
  } else if (j0 < 0) {
    tree = m[0] << -j0;
  } else {
    const int w = j0 / 64, s = j0 % 64;
    const uint64_t a = m[w], b = s && w + 1 < words ? m[w + 1] : 0;
    tree = a >> s | (s ? b << (64 - s) : 0);
  }
  return bits | (tree & bit_range64(-j0, count - j0));
}

__device__ __forceinline__ TreeRow read_tree_row(const TreeParams& p, int b) {
  int n = p.lens[b], c = p.counts ? p.counts[b] : p.nodes;
  if (n < 0 || n > p.cache.capacity) {
    set_status(p.status, OL_DEVICE_GUARD);
    n = n < 0 ? 0 : p.cache.capacity;
  }
  if (c < 0 || c > p.nodes || c > n) {
    set_status(p.status, OL_DEVICE_GUARD);
    c = c < 0 ? 0 : min(min(c, p.nodes), n);
  }
  return tree_row(n, c, p.window, p.tile_log2);
}

// The tiles of all units, in the order (row, kv head, row group of the unit,
// tile), each unit's behind `extra` tiles that stand for what a unit costs
// besides, are cut into n = min(CTAs, T) contiguous shares, none of them empty, of
// T / n tiles, the first T % n of one more. A walk gives the CTA its share's
// segments, one unit's tiles [tile0, tile1) each. A segment that is not its whole
// unit puts its state into a slot. A share has at most two of them: the end or the
// middle of a unit (slot 2 c), and a unit's begin (slot 2 c + 1).
// Equal shares keep ragged batches balanced to one tile per SM.
// The constructor is for whole warps; next() may be called by single threads.
struct TreeWalk {
  int b, g, qg;
  TreeRow row;
  int tile0, tile1;
  int slot;
  int at, end;           // next tile of the share; its end
  int share, total;      // its first tile; all tiles
  int each, more;        // tiles of a share; shares of one more
  int v1;                // tiles of the unit, extra ones included, up to `at`
  int first_nt;          // tiles of row `lane` of the first 32 rows

  __device__ __forceinline__ static int tiles(const TreeParams& p, const TreeRow& r) {
    return r.ntiles > 0 ? r.ntiles + p.extra : 0;
  }

  __device__ __forceinline__ explicit TreeWalk(const TreeParams& p) {
    const int lane = threadIdx.x & 31, c = blockIdx.x;
    total = 0;
    for (int base = 0; base < p.batch; base += 32) {
      int nt = base + lane < p.batch ? tiles(p, read_tree_row(p, base + lane)) : 0;
      if (base == 0) first_nt = nt;
      total += __reduce_add_sync(0xffffffffu, nt);
    }
    total *= p.kv_heads * p.units_per_head;
    const int shares = min(total, (int)gridDim.x);
    at = end = share = each = more = tile0 = tile1 = slot = 0;
    if (c < shares) {
      each = total / shares;
      more = total - each * shares;
      at = share = c * each + min(c, more);
      end = share + each + (c < more);
    }
    v1 = at < end ? locate(p, at) : 0;
  }

  // Finds the unit of tile x (x < total); returns the tile's index in it.
  __device__ __forceinline__ int locate(const TreeParams& p, int x) {
    const int lane = threadIdx.x & 31;
    const int per_row = p.kv_heads * p.units_per_head;
    b = g = qg = 0;
    row = TreeRow{0, 0, 0, 0, 1};
    for (int base = 0; base < p.batch; base += 32) {
      const int nt = base == 0 ? first_nt : base + lane < p.batch ? tiles(p, read_tree_row(p, base + lane)) : 0;
      int incl = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31) * per_row;
      if (x < all) {
        const int src = __ffs(__ballot_sync(0xffffffffu, x < incl * per_row)) - 1;
        x -= __shfl_sync(0xffffffffu, incl - nt, src) * per_row;
        const int mine = __shfl_sync(0xffffffffu, nt, src);
        b = base + src;
        row = read_tree_row(p, b);
        const int unit = x / mine;
        g = unit / p.units_per_head;
        qg = unit - g * p.units_per_head;
        return x - unit * mine;
      }
      x -= all;
    }
    return 0;
  }

  // Moves to the share's next segment.
  __device__ __forceinline__ bool next(const TreeParams& p) {
    while (at < end) {
      if (v1 == tiles(p, row)) {  // the unit is done: the next one
        v1 = 0;
        if (++qg == p.units_per_head) {
          qg = 0;
          if (++g == p.kv_heads) {
            g = 0;
            do {
              if (++b >= p.batch) return false;
              row = read_tree_row(p, b);
            } while (row.ntiles == 0);
          }
        }
      }
      tile0 = max(v1 - p.extra, 0);
      const int step = min(tiles(p, row) - v1, end - at);
      v1 += step;
      at += step;
      tile1 = max(v1 - p.extra, 0);
      if (tile1 > tile0) {
        slot = 2 * blockIdx.x + (tile0 == 0);
        return true;
      }
    }
    return false;
  }

  __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == row.ntiles; }

  // The share's notes for the merge, by one thread, on a walk of its own.
  __device__ __forceinline__ void write_splits(const TreeParams& p) {
    TreeSplit s = {};
    s.last = -1;
    while (next(p)) {
      if (tile0 > 0) continue;  // the unit began in an earlier share
      s.first = blockIdx.x;
      s.last = -1;
      if (tile1 < row.ntiles) {
        const int back = end + (row.ntiles - tile1) - 1;  // the unit's last tile
        const int big = more * (each + 1);                // tiles of the shares of one more
        s.last = back < big ? back / (each + 1) : more + (back - big) / each;
        s.count = row.count;
        s.row0 = qg * p.rows_per_unit;
        s.rows = min(p.rows_per_unit, p.group * p.nodes - s.row0);
        s.out = (long long)tree_out_row(p, b, g, s.row0);
      }
      if (p.by_unit) p.splits[(b * p.kv_heads + g) * p.units_per_head + qg] = s;
    }
    // (only the share's last unit can reach past its end)
    if (!p.by_unit) p.splits[blockIdx.x] = s;
  }
};

// Sets a kernel's attributes (f) before its first launch on each device.
template <typename F>
inline cudaError_t once_per_device(std::atomic<uint64_t>& done, F f) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = f();
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A launch that may begin while the kernel ahead of it in the stream drains;
// the kernels wait for it (griddepcontrol.wait) before they touch memory.
template <typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ol
