// ol_fast_tree.cu -- attention of drafted trees over a cache on the 5th
// generation tensor cores: bf16, head_dim 64 or 128, contiguous cache or paged
// pool with pages of a multiple of 16 tokens.
//
// A unit is up to 256 (head, node) rows r = head * nodes + node of one row's kv
// head: the vectors of q they read are consecutive, and every K/V byte is read
// once per unit. Its tokens form tiles of 128; equal contiguous shares of all
// units' tiles go to one CTA per SM (TreeWalk in ol_tree.cuh).
//
// Two softmax streams of 128 threads (one row each) work on halves of tiles, 64
// tokens a step, each with two S buffers: the tensor core has the next step's
// scores ready while a step's weights are formed. With more than 128 rows
// (NQ = 2) a stream has a query tile of its own and takes both halves of every
// tile; with up to 128 (NQ = 1) both have the same queries and a stream takes its
// half of every tile, and they are joined at the segment's end.
//   S = Q K^T      128 x 64 x D, both operands in shared memory, S in TMEM
//   P = 2^(S - m)  registers, back to TMEM over S: its bf16 part and its remainder's
//   O += P V       128 x D x 64 for each of the two, P from TMEM, V from shared memory,
//                  O in TMEM
// m is a reference near the row's maximum: it is set from a segment's first
// scores and again only when a step's weights sum to more than 2^10 (fp32 and
// bf16 carry such weights as exactly as smaller ones), so the maximum is looked
// for, and O rescaled, rarely. Sums and O are fp32. P's product takes bf16: P is the
// sum of its leading 8 bits and of the remainder's, 16 together, as the weights of the
// decode and chunked steps are (one part alone: 3.5e-3 off in fp32 outputs near 1,
// as much again as the output's own rounding in bf16 ones).
//
// Warps: 0 producer (TMA; a lane per box of a tile: pages of 16 tokens are
// boxes of 16 rows), 1 and 2 MMA issue for a stream each, 3 V's tiles and the
// note for the merge, 4-7 and 8-11 the streams. In tiles that hold drafted tokens,
// tokens behind some node's window or the row's end, warp 3 first zeroes the rows outside
// the row's tokens and the non-finite elements of tokens that are hidden from some node:
// a product with P = 0 must not see them.
// Where there was such an element, the non-finite values of the tokens that a row
// sees are added to its outputs at the end (rare, unhurried).
//
// Bounds: 4 * D bytes per token and kv head against 4 * D * rows flops (of which
// P V's are done twice). Up to 128 rows the memory (16 nodes over 64 rows of 8000
// tokens, group 4: 307 us, 6.8 TB/s; 8192 tokens in pages of 16: 352 us, 6.1 TB/s).
// With two query tiles the products: a tile of 128 tokens takes 32 of S, 49 cycles
// each (the 6 KB that they read from shared memory; the tensor core's own time is
// 32), and 32 of P V, 65 cycles each (the tensor core's), 3650 in all. Beside them
// the shared memory moves 192 KB for S (a stream's queries are read for each 64
// tokens), 128 KB of V and 64 KB in, 3070 cycles at 128 bytes a cycle. 4200 to 4900
// cycles are measured (64 nodes over 64 rows of 4000: 286 us, 935 TFLOP/s; the
// tensor pipe is busy 70 % of a launch of 27 tiles an SM), the rest are waits between a
// step's scores, weights and sums. Under seconds of it the power limit takes the clock
// to 1.7 GHz (315 us). With one product of P V it was 241 us: the price of the 16 bits.
// (Figures of trials at other places of this file are from then: 64 nodes over 32 rows
// 137 us, now 163; 256 over 8 rows 126, now 145.)
#include "ol_tree.cuh"

namespace ol {
namespace {

constexpr int kTile = 1 << kTreeFastTileLog2;
constexpr int kStep = kTile / 2;  // tokens of a step
constexpr int kThreads = 384;
constexpr float kGrown = 1024.f;  // a step's sum of weights that makes a row look for its maximum

template <int D, int NQ>
struct Lay {
  static constexpr int kHalves = D / 64;                // 64-element (128-byte) column blocks
  static constexpr int kTileBytes = kTile * D * 2;      // K, V or Q tile
  // K and V have rings of their own: whoever waits for a slot sees each of its
  // phases. K's slots are free earlier (after S) than V's.
  static constexpr int kK = D == 128 ? (NQ == 1 ? 3 : 2) : 6;
  static constexpr int kV = D == 128 ? 3 : 6;
  static constexpr int kSlots = kK + kV;                // K's, then V's
  static constexpr int kQ = 0;
  static constexpr int kRing = NQ * kTileBytes;
  static constexpr int kStats = kRing + kSlots * kTileBytes;  // float2 [2][128]: streams' (m, l)
  static constexpr int kBars = kStats + 2 * 128 * 8;
  // full, empty [kSlots], landed [kV]; qfull, qempty, sfull[2][2], pready[2][2], pvdone[2][2], drain[2], join
  static constexpr int kNumBars = 2 * kSlots + kV + 17;
  static constexpr int kMisc = kBars + kNumBars * 8;    // TMEM address, abort flag, whether V had non-finite elements
  static constexpr int kTotal = kMisc + 12;
  static_assert(kTotal <= 232448, "shared memory of one CTA");
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  // start, leading and stride offsets in 16 bytes; version 1; 128-byte swizzle
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lbo_bytes >> 4) << 16 | (uint64_t)(sbo_bytes >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// f32 accumulator, bf16 operands; M = 128
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn_major) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define OL_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define OL_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : OL_R8(x, 0), OL_R8(x, 8), OL_R8(x, 16), OL_R8(x, 24)
      : "r"(addr));
}
// Waits for the loads; x are registers that a load fills (so that no use of them moves ahead of the wait).
#define OL_U8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : OL_U8(x, 0), OL_U8(x, 8), OL_U8(x, 16), OL_U8(x, 24)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      OL_W8(x, 0), OL_W8(x, 8), OL_W8(x, 16), OL_W8(x, 24)
      : "memory");
}

// The same value in every lane of a converged warp, known as such to the compiler.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ uint64_t pack_b32x2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  return pack_b32x2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void unpack_b32x2(uint64_t x, uint32_t& a, uint32_t& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The leading 8 bits of two numbers, as bf16.
__device__ __forceinline__ uint32_t cut_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// ----------------------------------------------------------------------- roles

template <int D, int NQ>
struct Bars {
  using L = Lay<D, NQ>;
  uint32_t at;
  __device__ uint32_t full(int s) const { return at + 8 * s; }
  __device__ uint32_t empty(int s) const { return at + 8 * (L::kSlots + s); }
  // V's copies are there; its slot is full once warp 3 has set it to rights
  __device__ uint32_t landed(int s) const { return at + 8 * (2 * L::kSlots + s - L::kK); }
  __device__ uint32_t qfull() const { return at + 8 * (2 * L::kSlots + L::kV); }
  __device__ uint32_t qempty() const { return qfull() + 8; }
  __device__ uint32_t sfull(int j, int b) const { return qfull() + 16 + 16 * j + 8 * b; }  // S buffer b of stream j
  __device__ uint32_t pready(int j, int b) const { return qfull() + 48 + 16 * j + 8 * b; }  // P in its place
  __device__ uint32_t pvdone(int j, int b) const { return qfull() + 80 + 16 * j + 8 * b; }  // and taken
  __device__ uint32_t drain(int j) const { return qfull() + 112 + 8 * j; }
  __device__ uint32_t join() const { return qfull() + 128; }
};

// A wait that ends: after about two seconds, or once another warp has given up,
// it returns false; the CTA then winds down with a device status.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort = 1;
      set_status(status, OL_DEVICE_GUARD);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The same for a whole warp: one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, status));
}

// The warp's arrival, after all its lanes' work.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// Four lanes times four pieces of four words: piece x of lane q becomes piece q of lane x's row.
__device__ __forceinline__ void quad_transpose(uint32_t* z, int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit *= 2) {
    const bool up = lane & bit;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x & bit) continue;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t& lo = z[4 * x + y];
        uint32_t& hi = z[4 * (x | bit) + y];
        const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        (up ? lo : hi) = other;
      }
    }
  }
}

// Walks the slots [first, first + count) of a ring, tile after tile.
struct Cursor {
  int slot, first, end;
  uint32_t phase = 0;
  __device__ __forceinline__ Cursor(int f, int count) : slot(f), first(f), end(f + count) {}
  __device__ __forceinline__ void next() {
    if (++slot == end) {
      slot = first;
      phase ^= 1;
    }
  }
};

// Lowest token of the row that any node may see.
__device__ __forceinline__ int row_low(const TreeParams& p, const TreeRow& r) {
  return p.window < 0 || r.prefix <= p.window ? 0 : r.prefix - p.window;
}
// End of the prefix tokens that a window hides from some node: tokens from
// row_low to this one are seen by some nodes only (or by none). Whole warps.
__device__ __forceinline__ int row_hidden_end(const TreeParams& p, const TreeRow& r, int b) {
  if (p.window < 0) return 0;
  int end = 0;
  for (int n = threadIdx.x % 32; n < r.count; n += 32) end = max(end, tree_low(p, r, b, n));
  return min(__reduce_max_sync(0xffffffffu, end), r.prefix);
}
// The tile holds tokens that are not the prefix of all rows: drafted ones, the
// end of the row, or tokens below the window.
__device__ __forceinline__ bool edge_tile(const TreeRow& r, int low, int t0) {
  return t0 + kTile > r.prefix || t0 < low;
}
// Streams with work on a unit.
template <int NQ>
__device__ __forceinline__ int unit_streams(const TreeParams& p, const TreeWalk& w) {
  return NQ == 2 && p.group * p.nodes - w.qg * p.rows_per_unit <= 128 ? 1 : 2;
}

struct Maps {
  CUtensorMap q, kv;
};

// Whether one of eight bf16 elements is infinite or NaN: its exponent of ones carries into the sign's place.
__device__ __forceinline__ bool nonfinite_in(uint4 x) {
  auto full = [](uint32_t e) { return (e & 0x7f807f80u) + 0x00800080u; };
  return ((full(x.x) | full(x.y) | full(x.z) | full(x.w)) & 0x80008000u) != 0;
}

// Drafted tokens [j0, j0 + 32) among `bits` that lie within the window of a node.
__device__ __noinline__ uint32_t in_window(const TreeParams& p, const TreeRow row, int b, int node, int j0, uint32_t bits) {
  const int at = tree_position(p, row, b, node);
  for (uint32_t left = bits; left; left &= left - 1) {
    const int c = __ffs(left) - 1;
    if ((long long)at - tree_position(p, row, b, j0 + c) > p.window) bits &= ~(1u << c);
  }
  return bits;
}

// Adds the non-finite elements, in dimensions [d0, d1), of the V of the segment's
// tokens that are hidden from some node, [low_all, hidden_end) and the drafted
// ones, and that this node sees, to what this thread has written for it: to the
// slot's row `place`, or to row `out` of the output.
__device__ __noinline__ void add_nonfinite(const TreeParams& p, TreeRow row, int b, int g, int tile0, int tile1, int node,
                                           int low_all, int hidden_end, int d0, int d1, float* slot, int place, size_t out) {
  const int a = max(row.start + tile0 * kTile, low_all), e = min(row.start + tile1 * kTile, row.len);
  const int low = p.window < 0 ? 0 : tree_low(p, row, b, node);
  for (int t = a; t < e; ++t) {
    if (t < row.prefix && t >= hidden_end) t = row.prefix;  // what all nodes see is in the products
    if (t >= e) break;
    if (t < row.prefix ? t < low : !tree_sees_drafted(p, row, b, node, t - row.prefix)) continue;
    const long long at = cache_row(p.cache, 1, b, g, t);
    if (at < 0) continue;
    const uint16_t* const v = reinterpret_cast<const uint16_t*>(p.cache.base) + at * p.head_dim;
    for (int d8 = d0; d8 < d1; d8 += 8) {
      const uint4 x8 = *reinterpret_cast<const uint4*>(v + d8);
      if (!nonfinite_in(x8)) continue;
      for (int d = d8; d < d8 + 8; ++d) {
        if ((v[d] & 0x7f80u) != 0x7f80u) continue;
        const float x = bf16_bits_to_float(v[d]);
        if (slot) {
          slot[2 * p.rows_per_unit + ((size_t)(d / 4) * p.rows_per_unit + place) * 4 + d % 4] += x;
        } else if (p.out_dtype == OL_F32) {
          reinterpret_cast<float*>(p.out)[out * p.head_dim + d] += x;
        } else {
          uint16_t& y = reinterpret_cast<uint16_t*>(p.out)[out * p.head_dim + d];
          y = float_to_bf16_bits(bf16_bits_to_float(y) + x);
        }
      }
    }
  }
}

template <int D, int NQ, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) fast_tree_kernel(const __grid_constant__ Maps maps,
                                                                const __grid_constant__ TreeParams p, const int box,
                                                                const int qbox, const int keep_l2) {
  using L = Lay<D, NQ>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sa = smem_u32(smem);
  if (sa % 1024 != 0) {  // the swizzled tiles need it; the launch has no other shared memory
    if (threadIdx.x == 0) set_status(p.status, OL_DEVICE_GUARD);
    return;
  }
  const Bars<D, NQ> bar{sa + L::kBars};
  volatile uint32_t* const abort = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  volatile uint32_t* const bad = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 8);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.kv);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar.full(s), 1);
      mbar_init(bar.empty(s), 2);
    }
    mbar_init(bar.qfull(), 1);
    mbar_init(bar.qempty(), 2);
    for (int j = 0; j < 2; ++j) {
      mbar_init(bar.sfull(j, 0), 1);
      mbar_init(bar.sfull(j, 1), 1);
      mbar_init(bar.pready(j, 0), 4);
      mbar_init(bar.pready(j, 1), 4);
      mbar_init(bar.pvdone(j, 0), 1);
      mbar_init(bar.pvdone(j, 1), 1);
      mbar_init(bar.drain(j), 1);
    }
    for (int s = L::kK; s < L::kSlots; ++s) mbar_init(bar.landed(s), 1);
    mbar_init(bar.join(), 8);
    fence_mbar_init();
    *abort = 0;
    *bad = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sa + L::kMisc) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  pdl_wait();
  pdl_launch_dependents();

  TreeWalk w(p);

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    const uint64_t policy = keep_l2 ? policy_evict_normal() : policy_evict_first();
    const uint64_t keep = policy_evict_normal();
    // One tile ahead: its boxes and this lane's page are known (the table's entry
    // on its way) before the ring has room for it. Lane = box.
    struct Tile {
      int t0, first, last;  // token; boxes
      int y;                // cache row of this lane's box in plane K
      int q;                // row of q of a segment's first tile, else -1
    } cur = {}, nxt = {};
    const int v_rows = (PAGED ? p.cache.num_pages * p.cache.page_size : p.batch * p.cache.capacity) * p.kv_heads;
    int tile;
    auto fetch = [&](Tile& t) {
      t.q = -1;
      if (tile == w.tile1) {
        if (!w.next(p)) return false;
        tile = w.tile0;
        t.q = (int)tree_out_row(p, w.b, w.g, w.qg * p.rows_per_unit);
      }
      t.t0 = w.row.start + tile++ * kTile;
      t.first = max(row_low(p, w.row) - t.t0, 0) / box;
      t.last = (min(w.row.len - t.t0, kTile) + box - 1) / box;
      const int at = t.t0 + lane * box;
      if (!PAGED) {
        t.y = (w.b * p.kv_heads + w.g) * p.cache.capacity + at;
      } else if (lane >= t.first && lane < t.last) {
        int page = p.cache.block_table[(size_t)w.b * p.cache.max_pages + at / p.cache.page_size];
        if (page < 0 || page >= p.cache.num_pages) {
          set_status(p.status, OL_DEVICE_GUARD);
          page = 0;
        }
        t.y = (page * p.kv_heads + w.g) * p.cache.page_size + at % p.cache.page_size;
      }
      return true;
    };
    Cursor k(0, L::kK), v(L::kK, L::kV);
    uint32_t seg = 0;
    bool ok = true;
    auto load = [&](Cursor& c, int y) {
      if (!warp_wait(bar.empty(c.slot), c.phase ^ 1, abort, p.status)) return false;
      const uint32_t there = c.first == 0 ? bar.full(c.slot) : bar.landed(c.slot);
      if (lane == 0) mbar_arrive_expect_tx(there, (uint32_t)(cur.last - cur.first) * box * D * 2);
      __syncwarp();
      if (lane >= cur.first && lane < cur.last)
        tma_load_3d(sa + L::kRing + c.slot * L::kTileBytes + lane * box * (D * 2), &maps.kv, 0, y, 0, there, policy);
      c.next();
      return true;
    };
    tile = w.tile1;  // none yet
    bool more = fetch(nxt);
    while (ok && more) {
      cur = nxt;
      more = fetch(nxt);
      ok = load(k, cur.y);
      if (ok && cur.q >= 0) {
        ok = warp_wait(bar.qempty(), (seg & 1) ^ 1, abort, p.status);  // the last segment's queries are read
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(bar.qfull(), (uint32_t)NQ * qbox * D * 2);
          for (int j = 0; j < NQ; ++j)
            for (int c = 0; c < L::kHalves; ++c)
              tma_load_3d(sa + L::kQ + j * L::kTileBytes + c * (kTile * 128), &maps.q, 0, cur.q + j * 128, c,
                          bar.qfull(), keep);
        }
        if (ok) ++seg;
      }
      ok = ok && load(v, cur.y + v_rows);
    }
    if (!ok) {  // copies in flight end before the CTA does
      if (seg) mbar_wait_bounded(bar.qfull(), (seg - 1) & 1);
      for (Cursor* c : {&k, &v})  // a slot's last load: of this lap before the cursor, else of the one before
        for (int i = c->first; i < c->end; ++i)
          mbar_wait_bounded(c->first == 0 ? bar.full(i) : bar.landed(i), i < c->slot ? c->phase : c->phase ^ 1);
    }
  } else if (warp < 3) {
    // --------------------------------------------------------------- MMA issue
    // A warp per stream. The whole warp walks and waits, so that what the
    // products are given stays in uniform registers; one elected lane issues
    // them. (One warp for both streams, at some 1500 cycles a step of waits and
    // addresses, left the tensor core idle half of the time; lane 0 alone in the
    // loop, 160 cycles a product for its operands.)
    constexpr uint32_t kDescS = mma_desc(kStep, false), kDescO = mma_desc(D, true);
    const int j = uniform(warp) - 1;
    const uint32_t tm = uniform(tmem), base = uniform(sa);
    const uint32_t ts = tm + j * 128, to = tm + 256 + j * D;
    const uint64_t q = smem_desc(base + L::kQ + (NQ == 2 ? j : 0) * L::kTileBytes, 16, 1024);
    // A tile is [box][column block][rows of the box][128 bytes]. A step's 64 tokens
    // are 8 groups of 8 rows, evenly spaced: half a tile, or (boxes of 16 rows) the
    // first or the last 8 rows of each box.
    const uint32_t boxes = uniform(box), block = boxes * 128;
    const uint32_t group = boxes == 16 ? block * L::kHalves : 1024;
    const uint32_t step = boxes == 16 ? 1024 : boxes == 64 ? block * L::kHalves : kStep * 128;
    Cursor k(0, L::kK), v(L::kK, L::kV);
    uint32_t seg = 0;         // segments
    uint32_t pphase = 0;      // of the P buffers, a bit each
    bool ok = true;
    // S into buffer b from the given half of K
    auto scores = [&](int half, int b) {
      if (elect_one()) {
        const uint64_t kd = smem_desc(base + L::kRing + k.slot * L::kTileBytes + half * step, 16, group);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          constexpr uint32_t kBlock = kTile * 128 / 16, kK = 2;  // q's column block, 16 elements; in 16 bytes
          mma_ss(ts + b * kStep, q + (x / 4 * kBlock + x % 4 * kK), kd + (x / 4 * (block / 16) + x % 4 * kK), kDescS,
                 x > 0);
        }
        mma_commit(bar.sfull(j, b));
      }
    };
    auto k_wait = [&] { return warp_wait(bar.full(k.slot), k.phase, abort, p.status); };
    auto k_read = [&](bool last) {  // this stream's reads of K (of Q) are issued
      if (elect_one()) {
        mma_commit(bar.empty(k.slot));
        if (last) mma_commit(bar.qempty());
      }
      k.next();
    };
    // O += P V with P of buffer b and the given half of V
    auto sums = [&](int half, int b, bool first, bool wait_v, bool last_of_v) {
      if (!warp_wait(bar.pready(j, b), pphase >> b & 1, abort, p.status)) return false;
      pphase ^= 1u << b;
      if (wait_v && !warp_wait(bar.full(v.slot), v.phase, abort, p.status)) return false;
      tmem_fence_after();
      if (elect_one()) {
        const uint64_t vd = smem_desc(base + L::kRing + v.slot * L::kTileBytes + half * step, block, group);
#pragma unroll
        for (int x = 0; x < kStep / 16; ++x) {
          const uint64_t v16 = vd + x * (2 * group / 16);  // 16 tokens: times P, times its remainder
          if (x == 0)
            mma_ts(to, ts + b * kStep, v16, kDescO, !first);
          else
            mma_ts(to, ts + b * kStep + x * 8, v16, kDescO, true);
          mma_ts(to, ts + b * kStep + kStep / 2 + x * 8, v16, kDescO, true);
        }
        mma_commit(bar.pvdone(j, b));
        if (last_of_v) mma_commit(bar.empty(v.slot));
      }
      if (last_of_v) v.next();
      return true;
    };
    while (ok && w.next(p)) {
      const int tiles = uniform(w.tile1 - w.tile0);
      ok = warp_wait(bar.qfull(), seg & 1, abort, p.status);
      ++seg;
      if (NQ == 2 && j >= unit_streams<NQ>(p, w)) {
        // nothing to do but to release what the other stream uses
        for (int i = 0; ok && i < tiles; ++i) {
          ok = k_wait();
          if (ok) warp_arrive(bar.empty(k.slot));
          ok = ok && warp_wait(bar.full(v.slot), v.phase, abort, p.status);
          if (ok) warp_arrive(bar.empty(v.slot));
          k.next();
          v.next();
        }
        if (ok) warp_arrive(bar.qempty());
      } else if (NQ == 2) {
        ok = ok && k_wait();
        if (ok) {
          scores(0, 0);
          scores(1, 1);
          k_read(tiles == 1);
        }
        for (int i = 0; ok && i < tiles; ++i) {
          const bool more = i + 1 < tiles;
          ok = sums(0, 0, i == 0, true, false);
          if (ok && more && (ok = k_wait())) scores(0, 0);
          ok = ok && sums(1, 1, false, false, true);
          if (ok && more) {
            scores(1, 1);
            k_read(i + 2 == tiles);
          }
        }
      } else {
        for (int i = 0; ok && i < 2 && i < tiles; ++i)
          if ((ok = k_wait())) {
            scores(j, i);
            k_read(i + 1 == tiles);
          }
        for (int i = 0; ok && i < tiles; ++i) {
          ok = sums(j, i & 1, i == 0, true, true);
          if (ok && i + 2 < tiles && (ok = k_wait())) {
            scores(j, i & 1);
            k_read(i + 3 == tiles);
          }
        }
      }
    }
    if (!ok) {  // products in flight end before TMEM is freed
      if (elect_one()) mma_commit(bar.drain(j));
      mbar_wait_bounded(bar.drain(j), 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------- V to rights, the merge's note
    // Rows of a V tile outside the row's tokens become zeros, tokens hidden from some
    // node lose their non-finite elements, before the tile counts as full. A tile or two
    // ahead of the products, so that its time is hidden; in the streams it was not
    // (256 nodes over 8 rows 138 us, here 126).
    if (lane == 0) {
      TreeWalk notes(w);
      notes.write_splits(p);
    }
    __syncwarp();
    const int box_log2 = 31 - __clz(box);
    Cursor v(L::kK, L::kV);
    bool ok = true;
    while (ok && w.next(p)) {
      const int low = row_low(p, w.row), hidden_end = row_hidden_end(p, w.row, w.b);
      for (int i = w.tile0; i < w.tile1; ++i) {
        if (!(ok = warp_wait(bar.landed(v.slot), v.phase, abort, p.status))) break;
        const int t0 = w.row.start + i * kTile;
        if (edge_tile(w.row, max(low, hidden_end), t0)) {
          uint4* const tile = reinterpret_cast<uint4*>(smem + L::kRing + v.slot * L::kTileBytes);
          // rows of the tile
          const int r_low = low - t0, r_hidden = hidden_end - t0, r_tree = w.row.prefix - t0, r_end = w.row.len - t0;
          constexpr int kAhead = 8, kPieces = kTile * D / 8;  // pieces of 16 bytes: of a lane at a time, all
          bool found = false;
#pragma unroll 1
          for (int x0 = lane; x0 < kPieces; x0 += 32 * kAhead) {
            uint4 x[kAhead];
            bool zero[kAhead], hit = false;
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
              const int line = (x0 + 32 * c) / 8;  // of 128 bytes, among [box][column block][row]
              const int r = (line >> box_log2) / L::kHalves << box_log2 | (line & (box - 1));
              zero[c] = r < r_low || r >= r_end;
              x[c] = make_uint4(0, 0, 0, 0);
              if (!zero[c] && (r >= r_tree || r < r_hidden)) x[c] = tile[x0 + 32 * c];
            }
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
              if (zero[c]) tile[x0 + 32 * c] = x[c];
              hit |= nonfinite_in(x[c]);
            }
            if (hit) {
              found = true;
#pragma unroll
              for (int c = 0; c < kAhead; ++c) {
                uint32_t* const e = reinterpret_cast<uint32_t*>(&x[c]);
                bool one = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((e[k] & 0x7f80u) == 0x7f80u) e[k] &= 0xffff0000u, one = true;
                  if ((e[k] & 0x7f800000u) == 0x7f800000u) e[k] &= 0xffffu, one = true;
                }
                if (one) tile[x0 + 32 * c] = x[c];
              }
            }
          }
          if (found) *bad = 1;
          fence_proxy_async_smem();
        }
        warp_arrive(bar.full(v.slot));
        v.next();
      }
    }
  } else {
    // ----------------------------------------------------------------- streams
    const int j = (warp - 4) / 4, row = tid % 128;  // TMEM lane
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + j * 128 + lanes, to = tmem + 256 + j * D + lanes;
    const int R = p.group * p.nodes;
    float2* const stats = reinterpret_cast<float2*>(smem + L::kStats);
    uint32_t phases = 0;           // of the S buffers, a bit each
    // Whether the products with the last P of buffer b are done: a buffer's next
    // S, and so its next P, comes only after them.
    auto taken = [&](int b) { return warp_wait(bar.pvdone(j, b), phases >> b & 1 ^ 1, abort, p.status); };
    bool ok = true;
    uint32_t joins = 0;
    auto join = [&] {  // both streams
      warp_arrive(bar.join());
      return warp_wait(bar.join(), joins++ & 1, abort, p.status);
    };
    while (ok && w.next(p)) {
      const int r = w.qg * p.rows_per_unit + (NQ == 2 ? j * 128 : 0) + row;  // (head, node)
      const int tiles = w.tile1 - w.tile0;
      if (j >= unit_streams<NQ>(p, w)) continue;
      const bool live = r < R, live_warp = r - lane < R;
      const int node = r % p.nodes;
      const int low = p.window < 0 ? 0 : tree_low(p, w.row, w.b, node);
      const int low_all = row_low(p, w.row);
      const uint64_t* const words = p.mask ? p.mask + ((size_t)w.b * p.nodes + node) * p.words : nullptr;
      if (words)  // on their way to L1 before the tiles that need them
        for (int x = 0; x < p.words; x += 4) asm volatile("prefetch.global.L1 [%0];" ::"l"(words + x));
      auto visible = [&](int t) {  // tokens [t, t + 64)
        uint64_t bits = visible64(words, p.words, w.row.prefix, w.row.count, node, low, t);
        const int j0 = t - w.row.prefix;
        if (p.window >= 0 && j0 > -64) {
          const uint64_t tree = bits & bit_range64(-j0, 64);
          uint32_t lo = (uint32_t)tree, hi = (uint32_t)(tree >> 32);
          bits ^= tree;
          if (lo) lo = in_window(p, w.row, w.b, node, j0, lo);
          if (hi) hi = in_window(p, w.row, w.b, node, j0 + 32, hi);
          bits |= (uint64_t)hi << 32 | lo;
        }
        return bits;
      };
      float m = -INFINITY, l = 0.f;  // reference (raw scores) and sum
      const int steps = NQ * tiles;
      uint32_t s[kStep];  // S of the step, on its way while the last step ends
      auto fetch = [&](int i) {
        phases ^= 1u << (i & 1);
        tmem_fence_after();
        if (live_warp) {
          tmem_ld32(ts + (i & 1) * kStep, s);
          tmem_ld32(ts + (i & 1) * kStep + 32, s + 32);
        }
      };
      if (!(ok = warp_wait(bar.sfull(j, 0), phases & 1, abort, p.status))) break;
      fetch(0);
      for (int i = 0; i < steps; ++i) {
        const int tile = NQ == 2 ? i / 2 : i, half = NQ == 2 ? i % 2 : j;
        const int t0 = w.row.start + (w.tile0 + tile) * kTile;
        const bool edge = edge_tile(w.row, low_all, t0);
        if (live_warp) {
          // Weights against the reference as it is, unless there is none yet; their
          // sum shows whether the maximum has outgrown it, and only then is it looked
          // for, with S read again: the weights' remainders take its registers.
          bool look = __any_sync(0xffffffffu, live && m == -INFINITY);
          float sum_step;
          uint32_t pk[kStep / 2];
          for (;;) {
            tmem_wait_ld(s);
            tmem_wait_ld(s + 32);
            if (edge || (p.window >= 0 && __any_sync(0xffffffffu, low > t0))) {
              uint32_t seen[2] = {0, 0};
              if (live && box == 16) {  // 8 tokens of each of 8 boxes
                const uint64_t a = visible(t0), b = visible(t0 + 64);
                seen[0] = __byte_perm((uint32_t)a, (uint32_t)(a >> 32), half ? 0x7531 : 0x6420);
                seen[1] = __byte_perm((uint32_t)b, (uint32_t)(b >> 32), half ? 0x7531 : 0x6420);
              } else if (live) {
                const uint64_t a = visible(t0 + kStep * half);
                seen[0] = (uint32_t)a;
                seen[1] = (uint32_t)(a >> 32);
              }
#pragma unroll
              for (int x = 0; x < kStep; ++x)
                if (!(seen[x / 32] >> (x % 32) & 1)) s[x] = 0xff800000u;  // -inf
            }
            if (look) {
              float mx = -INFINITY;
#pragma unroll
              for (int x = 0; x < kStep; ++x) mx = fmaxf(mx, __uint_as_float(s[x]));
              const bool grow = live && mx > m;  // false for NaN, and -inf both
              if (__any_sync(0xffffffffu, grow)) {
                const float m2 = grow ? mx : m;
                const float f = grow ? exp2f((m - m2) * p.scale_log2) : 1.f;  // 0 where m is -inf
                m = m2;
                l *= f;
                if (i > 0) {
                  ok = taken(i + 1 & 1);
                  tmem_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D; c += 32) {
                    tmem_ld32(to + c, pk);
                    tmem_wait_ld(pk);
#pragma unroll
                    for (int x = 0; x < 32; ++x) pk[x] = __float_as_uint(__uint_as_float(pk[x]) * f);
                    tmem_st32(to + c, pk);
                  }
                }
              }
            }
            const float base = m == -INFINITY ? 0.f : -m * p.scale_log2;
            const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2), base2 = pack_f32x2(base, base);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int x = 0; x < kStep / 2; ++x) {
              uint32_t a, b;
              unpack_b32x2(fma_f32x2(pack_b32x2(s[2 * x], s[2 * x + 1]), scale2, base2), a, b);
              const float ea = fast_exp2(__uint_as_float(a)), eb = fast_exp2(__uint_as_float(b));
              sum[x & 1] = add_f32x2(sum[x & 1], pack_f32x2(ea, eb));
              // Cut, not rounded, and the remainder 2^-23 of the weight larger: neither part is
              // negative or (of weights above 2^-103) zero, so that an infinity in V stays one.
              // (The cut by bytes, and pairs of remainders, cost more: 64 nodes over 32 rows
              // 168 and 182 us, 163 so.)
              pk[x] = cut_bf16x2(ea, eb);
              s[x] = pack_bf16x2(fmaf(ea, 1.f + 0x1p-23f, -__uint_as_float(pk[x] << 16)),
                                 fmaf(eb, 1.f + 0x1p-23f, -__uint_as_float(pk[x] & 0xffff0000u)));
            }
            uint32_t a, b;
            unpack_b32x2(add_f32x2(sum[0], sum[1]), a, b);
            sum_step = __uint_as_float(a) + __uint_as_float(b);
            if (look || !__any_sync(0xffffffffu, live && !(sum_step <= kGrown))) break;
            look = true;  // (also for NaN)
            tmem_ld32(ts + (i & 1) * kStep, s);
            tmem_ld32(ts + (i & 1) * kStep + 32, s + 32);
          }
          tmem_st32(ts + (i & 1) * kStep, pk);
          tmem_st32(ts + (i & 1) * kStep + kStep / 2, s);
          l += sum_step;
        }
        // the next scores, if they are there, come in while P settles
        const bool next = i + 1 < steps;
        const uint32_t next_full = bar.sfull(j, i + 1 & 1);
        bool early = false;
        if (next && (early = __all_sync(0xffffffffu, mbar_test(next_full, phases >> (i + 1 & 1) & 1)))) fetch(i + 1);
        if (live_warp) tmem_wait_st();
        if (!ok) break;
        tmem_fence_before();
        warp_arrive(bar.pready(j, i & 1));
        if (next && !early) {
          if (!(ok = warp_wait(next_full, phases >> (i + 1 & 1) & 1, abort, p.status))) break;
          fetch(i + 1);
        }
      }
      if (!ok) break;
      if (!(ok = taken(steps + 1 & 1))) break;
      tmem_fence_after();

      // the segment's state: m in log2 units
      float ml = m == -INFINITY ? -INFINITY : m * p.scale_log2;
      float f0 = 1.f, f1 = 0.f;  // factors of O (of both streams' O)
      if (NQ == 1) {
        tmem_fence_before();
        stats[j * 128 + row] = make_float2(ml, l);
        if (!(ok = join())) break;
        tmem_fence_after();
        const float2 a = stats[row], b = stats[128 + row];
        ml = fmaxf(a.x, b.x);
        const float top = ml == -INFINITY ? 0.f : ml;
        f0 = exp2f(a.x - top);
        f1 = exp2f(b.x - top);
        l = a.y * f0 + b.y * f1;
      }
      const bool whole = w.whole();
      float* const slot = whole ? nullptr : tree_slot(p, w.slot);
      const int place = (NQ == 2 ? j * 128 : 0) + row;  // in the unit
      const bool mine = live && (!whole || node < w.row.count);
      if (slot && live && (NQ == 2 || j == 0)) {
        slot[place] = ml;
        slot[p.rows_per_unit + place] = l;
      }
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      if (live_warp) {
        // NQ == 1: each stream writes half of the dimensions
        constexpr int kCols = NQ == 2 ? D : D / 2;
        const int c0 = NQ == 2 ? 0 : j * kCols;
        const uint32_t t = tmem + 256 + lanes;
        const size_t at = tree_out_row(p, w.b, w.g, r) * D;
#pragma unroll 1
        for (int c = c0; c < c0 + kCols; c += 32) {
          uint32_t o[32];
          if (NQ == 2) {
            tmem_ld32(to + c, o);
            tmem_wait_ld(o);
          } else {
            uint32_t b[32];
            tmem_ld32(t + c, o);
            tmem_ld32(t + D + c, b);
            tmem_wait_ld(o);
            tmem_wait_ld(b);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              o[x] = __float_as_uint(__uint_as_float(o[x]) * f0 + __uint_as_float(b[x]) * f1);
          }
          if (slot) {
            float4* const y = reinterpret_cast<float4*>(slot + 2 * p.rows_per_unit) + (size_t)(c / 4) * p.rows_per_unit + place;
            if (mine)
#pragma unroll
              for (int x = 0; x < 8; ++x) reinterpret_cast<uint4*>(y)[x * p.rows_per_unit] =
                  make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          } else if (p.out_dtype == OL_F32) {
            uint4* const y = reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.out) + at + c);
            if (mine)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                y[x] = make_uint4(__float_as_uint(__uint_as_float(o[4 * x]) * inv),
                                  __float_as_uint(__uint_as_float(o[4 * x + 1]) * inv),
                                  __float_as_uint(__uint_as_float(o[4 * x + 2]) * inv),
                                  __float_as_uint(__uint_as_float(o[4 * x + 3]) * inv));
          } else {
            // Four lanes exchange their rows' four pieces of 16 bytes, so that
            // together they write 64 bytes of one row after another.
            uint32_t z[16];
#pragma unroll
            for (int x = 0; x < 16; ++x)
              z[x] = pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
            quad_transpose(z, lane);
            const unsigned who = __ballot_sync(0xffffffffu, mine);
            const size_t first = tree_out_row(p, w.b, w.g, r - lane % 4) * D + c + lane % 4 * 8;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (who >> (lane / 4 * 4 + x) & 1)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + first + (size_t)x * D) =
                    make_uint4(z[4 * x], z[4 * x + 1], z[4 * x + 2], z[4 * x + 3]);
          }
        }
        __syncwarp();  // add_nonfinite reads what other lanes wrote
        const bool any_bad = __any_sync(0xffffffffu, *bad != 0);  // (of this or an earlier segment)
        const int hidden_end = any_bad ? row_hidden_end(p, w.row, w.b) : 0;
        if (any_bad && mine)
          add_nonfinite(p, w.row, w.b, w.g, w.tile0, w.tile1, node, low_all, hidden_end, c0, c0 + kCols, slot, place,
                        tree_out_row(p, w.b, w.g, r));
      }
      if (NQ == 1) {  // both streams have read both O before either's next product
        tmem_fence_before();
        ok = join();
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ------------------------------------------------------------------------ host

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A bf16 buffer as rows of D elements, seen as [column block][row][64 elements];
// boxes of `box` rows and all (or one) of the column blocks, 128-byte swizzle.
bool encode_rows(CUtensorMap* map, const void* base, int D, uint64_t rows, int box, bool all_blocks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, rows, (cuuint64_t)D / 64};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
  cuuint32_t boxes[3] = {64, (cuuint32_t)box, all_blocks ? (cuuint32_t)D / 64 : 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t kv_rows(const TreeParams& p) {
  return p.cache.block_table ? 2ull * p.cache.num_pages * p.kv_heads * p.cache.page_size
                             : 2ull * p.batch * p.kv_heads * p.cache.capacity;
}

template <int D, int NQ, bool PAGED>
cudaError_t launch_cfg(const Maps& maps, const TreeParams& p, int box, int qbox, cudaStream_t s) {
  auto kern = fast_tree_kernel<D, NQ, PAGED>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, NQ>::kTotal);
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(kern, dim3(p.nctas), dim3(kThreads), Lay<D, NQ>::kTotal, s, maps, p, box, qbox,
                    p.units_per_head > 1 ? 1 : 0);
}

template <int D>
cudaError_t launch_dim(const Maps& maps, const TreeParams& p, int box, int qbox, cudaStream_t s) {
  const bool two = p.rows_per_unit == 256;
  if (p.cache.block_table)
    return two ? launch_cfg<D, 2, true>(maps, p, box, qbox, s) : launch_cfg<D, 1, true>(maps, p, box, qbox, s);
  return two ? launch_cfg<D, 2, false>(maps, p, box, qbox, s) : launch_cfg<D, 1, false>(maps, p, box, qbox, s);
}

}  // namespace

bool fast_tree_supported(const TreeParams& p) {
  if (p.dtype != OL_BF16 || (p.head_dim != 64 && p.head_dim != 128)) return false;
  if (p.cache.block_table && p.cache.page_size % 16 != 0) return false;
  // TMA row coordinates are 32-bit
  return kv_rows(p) < (1ull << 31) && (uint64_t)p.batch * p.q_heads * p.nodes + 256 < (1ull << 31);
}

void plan_fast_tree(TreeParams& p, int sms) {
  p.rows_per_unit = tree_fast_rows(p.group, p.nodes);
  p.units_per_head = (p.group * p.nodes + p.rows_per_unit - 1) / p.rows_per_unit;
  p.tile_log2 = kTreeFastTileLog2;
  p.nctas = sms < kTreeMaxCtas ? sms : kTreeMaxCtas;
  // Measured (0 / 2 / 3 / 4 tiles): 64 nodes over 32 ragged rows (two query tiles) 182 / 161 / 162 / 162 us, 16 nodes
  // over 64 ragged rows (one) 383 / 378 / 378 / 381 us.
  p.extra = p.rows_per_unit == 256 ? 3 : 2;
  p.by_unit = tree_few_units(p);
}

cudaError_t launch_fast_tree(const TreeParams& p, cudaStream_t s) {
  const int R = p.group * p.nodes;
  // rows of a box: a tile of the contiguous cache, else 128, 64 or 16, what divides a page
  int box = kTile;
  if (p.cache.block_table && p.cache.page_size % box != 0) box = p.cache.page_size % 64 == 0 ? 64 : 16;
  const int qbox = R < 128 ? (R + 7) / 8 * 8 : 128;
  Maps maps;
  if (!encode_rows(&maps.q, p.q, p.head_dim, (uint64_t)p.batch * p.q_heads * p.nodes, qbox, false) ||
      !encode_rows(&maps.kv, p.cache.base, p.head_dim, kv_rows(p), box, true))
    return cudaErrorInvalidValue;
  return p.head_dim == 128 ? launch_dim<128>(maps, p, box, qbox, s) : launch_dim<64>(maps, p, box, qbox, s);
}

}  // namespace ol
