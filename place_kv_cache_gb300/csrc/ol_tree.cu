// ol_tree.cu -- attention of drafted trees over a cache on CUDA cores (every
// dtype and head size that the tensor-core kernel of ol_fast_tree.cu does not
// take), the merge of both kernels' partial results, and the move of an
// accepted path.
//
// A unit is 32 or 64 (head, node) rows of one row's kv head; its tokens form tiles
// of 32. All units' tiles in order are cut into equal shares, one per CTA
// (TreeWalk). A CTA runs the online softmax over its segment of a unit with the
// scores S = Q K^T and the sums O += P V in registers: 4 rows x 2 tokens of S,
// 4 rows x D / 16 dimensions of O per thread, operands from shared memory four
// dimensions at a time. K and V lie there as they are in the cache; the next tile
// is copied in meanwhile. Bound for many rows by fp32 FMAs and the shared-memory
// loads that feed them (4 * D flops per row and token against 2 * D elements a
// token; fp32 trees of 16 over 64 rows of 4000 tokens 1800 us, 37 TFLOP/s), by
// latency for few (5 nodes, 6 rows, a window of 1000: 22 us). The loops over
// dimensions and tokens hold no branch: one in the sums, past the head's end,
// kept their loads from running ahead (2170 us and 26 us).
#include <type_traits>

#include "ol_tree.cuh"

namespace ol {
namespace {

constexpr int TB = 1 << kTreeGenTileLog2;
constexpr int kGenStages = 2;

__host__ __device__ inline int padded(int D) { return (D + 3) / 4 * 4; }
// bytes of a K or V row in shared memory: 16 more, so that 8 rows cover the banks
template <typename T>
__host__ __device__ inline int row_bytes(int D) { return (padded(D) * (int)sizeof(T) + 15) / 16 * 16 + 16; }
template <typename T, int RB>
inline size_t gen_smem(int D) {
  return sizeof(float) * (size_t)TB * (RB + 4) + (size_t)(RB + kGenStages * 2 * TB) * row_bytes<T>(D);
}

__device__ __forceinline__ float4 load4(const float* x) { return *reinterpret_cast<const float4*>(x); }
__device__ __forceinline__ float4 load4(const uint16_t* x) {
  const uint2 w = *reinterpret_cast<const uint2*>(x);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// CTAs of RB rows per SM that 128 registers a thread allow (up to 128 dimensions; beyond, half as many)
constexpr int gen_per_sm(int NC, int RB) { return (NC <= 2 ? 128 : 64) / RB; }

// NC: chunks of 64 dimensions (16 threads x 4); RB: rows of a unit, 4 threads each
template <typename T, int NC, int RB>
__global__ void __launch_bounds__(4 * RB, gen_per_sm(NC, RB)) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr int kThreads = 4 * RB, kPer = kThreads / TB;  // threads that copy a row
  constexpr int kPStride = RB + 4;                        // P is kept [token][row]
  extern __shared__ __align__(16) uint8_t smem[];
  const int D = p.head_dim, Dp = padded(D), rb = row_bytes<T>(D);
  float* const sp = reinterpret_cast<float*>(smem);
  uint8_t* const sq = reinterpret_cast<uint8_t*>(sp + TB * kPStride);
  uint8_t* const ring = sq + RB * rb;
  const int tid = threadIdx.x, rg = tid / 16, cg = tid % 16;  // rows 4 rg .. 4 rg + 3
  const int R = p.group * p.nodes;
  const bool vec = D * sizeof(T) % 16 == 0;
  pdl_wait();
  pdl_launch_dependents();
  TreeWalk w(p);
  if (tid == kThreads - 1) {
    TreeWalk notes = w;
    notes.write_splits(p);
  }
  while (w.next(p)) {
    const int r0 = w.qg * RB;
    const int low_all = p.window < 0 || w.row.prefix <= p.window ? 0 : w.row.prefix - p.window;
    // a row of D elements (or zeros) to shared memory, by `lanes` threads
    auto copy_row = [&](uint8_t* to, const T* from, bool there, int lane, int lanes) {
      if (vec) {
        for (int c = lane * 16; c < D * (int)sizeof(T); c += lanes * 16)
          copy16(smem_u32(to + c), reinterpret_cast<const uint8_t*>(from) + c, there);
      } else {
        for (int d = lane; d < Dp; d += lanes) reinterpret_cast<T*>(to)[d] = there && d < D ? from[d] : T(0);
      }
    };
    // tile `tile` into stage `tile` % 2
    auto copy = [&](int tile) {
      const int j = tid / kPer, t0 = w.row.start + tile * TB;
      uint8_t* const to = ring + (tile % kGenStages * 2 * TB + j) * rb;
      const bool there = j >= low_all - t0 && j < w.row.len - t0;  // (t0 + TB may pass 2^31)
#pragma unroll
      for (int plane = 0; plane < 2; ++plane) {
        const long long row = there ? cache_row(p.cache, plane, w.b, w.g, t0 + j) : -1;
        if (there && row < 0) set_status(p.status, OL_DEVICE_GUARD);
        copy_row(to + plane * TB * rb, reinterpret_cast<const T*>(p.cache.base) + (row < 0 ? 0 : row * D), row >= 0,
                 tid % kPer, kPer);
      }
      copies_commit();
    };
    __syncthreads();  // the last segment's tiles are read
    {
      const int r = tid / 4;
      const T* const q = reinterpret_cast<const T*>(p.q) + tree_out_row(p, w.b, w.g, r0) * D;
      copy_row(sq + r * rb, r0 + r < R ? q + (size_t)r * D : q, r0 + r < R, tid % 4, 4);
    }
    copy(w.tile0);
    int node[4];
    int at[4], low[4];  // with a window: the rows' positions, their lowest prefix token
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      node[r] = (r0 + 4 * rg + r) % p.nodes;
      at[r] = p.window < 0 ? 0 : tree_position(p, w.row, w.b, node[r]);
      low[r] = p.window < 0 || at[r] <= p.window ? 0 : at[r] - p.window;
    }
    float m[4], l[4];
    float4 o[4][NC];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int tile = w.tile0; tile < w.tile1; ++tile) {
      const int t0 = w.row.start + tile * TB;
      if (tile + 1 < w.tile1) {
        copy(tile + 1);
        copies_wait<1>();
      } else {
        copies_wait<0>();
      }
      __syncthreads();
      const uint8_t* const sk = ring + tile % kGenStages * 2 * TB * rb;
      const uint8_t* const sv = sk + TB * rb;
      float s[4][2];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r][0] = s[r][1] = 0.f;
      const T* const k_lo = reinterpret_cast<const T*>(sk + cg * rb);
      const T* const k_hi = reinterpret_cast<const T*>(sk + (cg + 16) * rb);
#pragma unroll 4
      for (int d = 0; d < Dp; d += 4) {
        const float4 k0 = load4(k_lo + d), k1 = load4(k_hi + d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 a = load4(reinterpret_cast<const T*>(sq + (4 * rg + r) * rb) + d);
          s[r][0] = fmaf(a.w, k0.w, fmaf(a.z, k0.z, fmaf(a.y, k0.y, fmaf(a.x, k0.x, s[r][0]))));
          s[r][1] = fmaf(a.w, k1.w, fmaf(a.z, k1.z, fmaf(a.y, k1.y, fmaf(a.x, k1.x, s[r][1]))));
        }
      }
      const int j0 = t0 - w.row.prefix;  // index among the drafted of the tile's first token
      const bool drafted = j0 > -TB;
      bool some = drafted;  // some row of the warp may not see some token of the tile
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r][0] *= p.scale_log2, s[r][1] *= p.scale_log2;
      if (drafted) {
        int pos[2] = {0, 0};  // of this thread's tokens
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = j0 + cg + 16 * u;
          if (p.window >= 0 && j >= 0 && j < w.row.count) pos[u] = tree_position(p, w.row, w.b, j);
        }
        uint32_t bits[4] = {};  // all rows' on their way together
        if (p.mask && j0 < w.row.count)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            bits[r] = mask_bits(p.mask + ((size_t)w.b * p.nodes + node[r]) * p.words, p.words, j0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t seen = visible_bits(!p.mask, bits[r], w.row.prefix, w.row.count, node[r], low[r], t0);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (!(seen >> (cg + 16 * u) & 1) || (p.window >= 0 && j0 + cg + 16 * u >= 0 &&
                                                 (long long)at[r] - pos[u] > p.window))
              s[r][u] = -INFINITY;
        }
      } else if (p.window >= 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (t0 + cg + 16 * u < low[r]) s[r][u] = -INFINITY, some = true;
        some = __any_sync(0xffffffffu, some);
      }
      float pr[4][2];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float top = fmaxf(s[r][0], s[r][1]);
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float mn = fmaxf(m[r], top);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float keep = m[r] == mn ? 1.f : exp2f(m[r] - base);
        m[r] = mn;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          pr[r][u] = exp2f(s[r][u] - base);
          sum += pr[r][u];
        }
        l[r] = l[r] * keep + sum;  // of this thread's tokens
        if (keep != 1.f)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            o[r][c].x *= keep;
            o[r][c].y *= keep;
            o[r][c].z *= keep;
            o[r][c].w *= keep;
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<float4*>(sp + (cg + 16 * u) * kPStride + 4 * rg) =
            make_float4(pr[0][u], pr[1][u], pr[2][u], pr[3][u]);
      __syncwarp();  // P of the warp's eight rows: its own
      int dims[NC];  // (past the head: some other dimension, for sums that no one reads)
#pragma unroll
      for (int c = 0; c < NC; ++c) dims[c] = c * 64 + cg * 4 < Dp ? c * 64 + cg * 4 : 0;
      auto add = [&](auto hidden) {  // whether there may be tokens hidden from some row: their V may hold infinities or NaN
#pragma unroll 4
        for (int j = 0; j < TB; ++j) {
          const float4 p4 = *reinterpret_cast<const float4*>(sp + j * kPStride + 4 * rg);
          const float pj[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = load4(reinterpret_cast<const T*>(sv + j * rb) + dims[c]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (decltype(hidden)::value && pj[r] == 0.f) continue;
              o[r][c].x += pj[r] * v.x;
              o[r][c].y += pj[r] * v.y;
              o[r][c].z += pj[r] * v.z;
              o[r][c].w += pj[r] * v.w;
            }
          }
        }
      };
      if (some)
        add(std::true_type());
      else
        add(std::false_type());
      __syncthreads();  // the stage is read
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    // the rows that this segment holds alone are done; others go to its slot
    float* const slot = w.whole() ? nullptr : tree_slot(p, w.slot);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * rg + r;
      if (r0 + row >= R) continue;
      if (slot) {
        if (cg == 0) {
          slot[row] = m[r];
          slot[RB + row] = l[r];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d4 = c * 16 + cg;
          if (d4 * 4 < Dp) reinterpret_cast<float4*>(slot + 2 * RB)[d4 * RB + row] = o[r][c];
        }
      } else if (node[r] < w.row.count) {
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        const size_t at = tree_out_row(p, w.b, w.g, r0 + row) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = c * 64 + cg * 4;
          const float v[4] = {o[r][c].x, o[r][c].y, o[r][c].z, o[r][c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d + j < D) store_out(p.out, p.out_dtype, at + d + j, v[j] * inv);
        }
      }
    }
  }
}

template <typename T, int NC, int RB>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [] {
    const cudaError_t e = cudaFuncSetAttribute(tree_kernel<T, NC, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)gen_smem<T, RB>(64 * NC));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(tree_kernel<T, NC, RB>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(tree_kernel<T, NC, RB>, dim3(p.nctas), dim3(4 * RB), gen_smem<T, RB>(p.head_dim), s, p);
}

template <typename T>
cudaError_t launch_rows(const TreeParams& p, cudaStream_t s) {
  const int nc = (p.head_dim + 63) / 64;
  if (p.rows_per_unit == 32)
    return nc == 1   ? launch_tree<T, 1, 32>(p, s)
           : nc == 2 ? launch_tree<T, 2, 32>(p, s)
           : nc == 3 ? launch_tree<T, 3, 32>(p, s)
                     : launch_tree<T, 4, 32>(p, s);
  return nc == 1   ? launch_tree<T, 1, 64>(p, s)
         : nc == 2 ? launch_tree<T, 2, 64>(p, s)
         : nc == 3 ? launch_tree<T, 3, 64>(p, s)
                   : launch_tree<T, 4, 64>(p, s);
}

// ------------------------------------------------------------------- the merge

// CTA x merges the unit that begins in share x and reaches past it, if there is
// one, or unit x (TreeSplit): rows [ROWS y, ROWS (y + 1)).
//   M = max m_s, L = sum l_s 2^(m_s - M), y = sum o_s 2^(m_s - M) / L
// A thread has a row, KG groups of four dimensions (the slots' layout keeps the
// rows of a group together) and one of G shares of the segments. Its first loads
// of o are on their way before the weights are known; more segments than those are
// taken in chunks with a running maximum. Bound by latency for few units: 8 rows a
// CTA, for more CTAs, 20 loads a thread. Else by reading the partials from L2, for
// which many resident warps do more than many loads each: 16 rows a CTA, 8 loads,
// four CTAs an SM (64 nodes over 32 rows 137 us in all; 32 rows, 16 loads 141).
template <int ROWS, int THREADS, int D4>  // D4: groups of four dimensions, 32 or 64
__global__ void __launch_bounds__(THREADS, ROWS > 8 ? 4 : 1) tree_merge_kernel(const TreeParams p) {
  constexpr int kLanes = THREADS / ROWS;  // threads of a row
  constexpr int G = kLanes > D4 ? kLanes / D4 : 1, KG = kLanes > D4 ? 1 : D4 / kLanes;
  constexpr int C = (ROWS > 8 ? 8 : D4 == 32 ? 20 : 16) / KG, kChunk = C * G;  // segments of a thread and of the CTA at a time
  static_assert(C >= 2 && kChunk * ROWS <= THREADS, "a thread loads one state");
  __shared__ float2 state[kChunk][ROWS];  // m, l
  __shared__ float4 other[G > 1 ? (G - 1) * ROWS * D4 : 1];
  __shared__ float other_l[G > 1 ? (G - 1) * ROWS : 1];
  pdl_wait();
  pdl_launch_dependents();
  if (p.by_unit && read_tree_row(p, blockIdx.x / (p.kv_heads * p.units_per_head)).ntiles == 0) return;  // no note
  const TreeSplit u = p.splits[blockIdx.x];
  if (u.last < 0 || (int)blockIdx.y * ROWS >= u.rows) return;
  const int RU = p.rows_per_unit, D = p.head_dim;
  const int lr = threadIdx.x % ROWS, lane = threadIdx.x / ROWS, d0 = lane % D4, grp = lane / D4;
  const int place = blockIdx.y * ROWS + lr;  // row of the unit
  const bool mine = place < u.rows && (u.row0 + place) % p.nodes < u.count;
  const int segs = u.last - u.first + 1;
  auto slot_of = [&](int i) { return tree_slot(p, 2 * (u.first + i) + (i == 0)); };
  float M = -INFINITY, L = 0.f;
  float4 acc[KG];
#pragma unroll
  for (int k = 0; k < KG; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < segs; i0 += kChunk) {
    float4 v[C][KG];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = i0 + grp + c * G;
      const float4* const o = reinterpret_cast<const float4*>(slot_of(i < segs ? i : 0) + 2 * RU) + place;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const int d4 = d0 + k * kLanes;
        v[c][k] = mine && i < segs && d4 * 4 < D ? o[(size_t)d4 * RU] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    if (threadIdx.x < kChunk * ROWS) {
      const int i = i0 + threadIdx.x / ROWS;
      const bool there = i < segs && place < u.rows;
      const float* const s = slot_of(there ? i : 0);
      state[threadIdx.x / ROWS][lr] = there ? make_float2(s[place], s[RU + place]) : make_float2(-INFINITY, 0.f);
    }
    __syncthreads();
    float top = M;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) top = fmaxf(top, state[i][lr].x);
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(M - base);
    M = top;
    L *= keep;
#pragma unroll
    for (int k = 0; k < KG; ++k) acc[k] = make_float4(acc[k].x * keep, acc[k].y * keep, acc[k].z * keep, acc[k].w * keep);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float2 st = state[grp + c * G][lr];
      const float f = exp2f(st.x - base);
      L += st.y * f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        acc[k].x += v[c][k].x * f;
        acc[k].y += v[c][k].y * f;
        acc[k].z += v[c][k].z * f;
        acc[k].w += v[c][k].w * f;
      }
    }
    __syncthreads();
  }
  if (G > 1) {
    if (grp > 0) {
      other[((grp - 1) * D4 + d0) * ROWS + lr] = acc[0];
      if (d0 == 0) other_l[(grp - 1) * ROWS + lr] = L;
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int x = 0; x < G - 1; ++x) {
      const float4 o = other[(x * D4 + d0) * ROWS + lr];
      acc[0].x += o.x;
      acc[0].y += o.y;
      acc[0].z += o.z;
      acc[0].w += o.w;
      L += other_l[x * ROWS + lr];
    }
  }
  if (!mine) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t out = (size_t)(u.out + place) * D;
#pragma unroll
  for (int k = 0; k < KG; ++k) {
    const int d = (d0 + k * kLanes) * 4;
    if (d >= D) break;
    const float v[4] = {acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv};
    if (D % 4 != 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (d + j < D) store_out(p.out, p.out_dtype, out + d + j, v[j]);
    } else if (p.out_dtype == OL_F32) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + out + d) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + out + d) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
}

template <int ROWS, int THREADS>
cudaError_t launch_merge(const TreeParams& p, int rows, cudaStream_t s) {
  const dim3 grid(p.by_unit ? p.batch * p.kv_heads * p.units_per_head : p.nctas, (rows + ROWS - 1) / ROWS), block(THREADS);
  return p.head_dim <= 128 ? launch_pdl(tree_merge_kernel<ROWS, THREADS, 32>, grid, block, 0, s, p)
                           : launch_pdl(tree_merge_kernel<ROWS, THREADS, 64>, grid, block, 0, s, p);
}

// --------------------------------------------------------------- accepted path

// One CTA per (row, kv head, plane) moves the kept tokens' vectors. kept ascends
// strictly, so kept[j] >= j and vector j's source is behind every place written
// before it: a pass reads its vectors, waits for the CTA, then writes them. The
// places of the first 512 tokens are looked up once, with the check of the list.
// Thread (x, y) has piece x of every step-th token: no division in the loops.
// Bound by a chain of latencies (count, list, table, vectors) for small trees, of
// which small CTAs start more at once: 16 nodes over 64 paged rows 3.2 us, 4.8 with
// CTAs of 256 threads; 64 fp32 nodes over 128 rows (67 MB) 16 us with either: the
// chain's latencies, 1.7 times over (2048 CTAs, 8 an SM by registers); with the
// cache's tokens in L2 9 us.
constexpr int kKeepThreads = 128;
constexpr int kKeepUnroll = 4;
constexpr int kKeepRows = 512;

template <typename P>  // the piece that a thread moves
__global__ void __launch_bounds__(kKeepThreads) tree_keep_kernel(const __grid_constant__ KeepParams p, int pieces) {
  __shared__ long long from[kKeepRows], to[kKeepRows];
  const CacheRef& c = p.cache;
  const int b = blockIdx.x / c.kv_heads, g = blockIdx.x - b * c.kv_heads, plane = blockIdx.y;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int start = p.starts[b], n = p.counts[b], drafted = p.drafted ? p.drafted[b] : p.nodes;
  const int32_t* const kept = p.kept + (size_t)b * p.nodes;
  auto place = [&](int t) { return cache_row(c, plane, b, g, start + t); };
  bool bad = n < 0 || n > drafted || drafted > p.nodes || start < 0 || (long long)start + drafted > c.capacity;
  if (!bad)
    for (int j = tid; j < n; j += blockDim.x * blockDim.y) {
      const int k = kept[j], last = j > 0 ? kept[j - 1] : -1;
      if (k <= last || k >= drafted) {
        bad = true;
        break;
      }
      const long long src = place(k), dst = place(j);
      bad |= src < 0 || dst < 0;
      if (j < kKeepRows) {
        from[j] = src;
        to[j] = dst;
      }
    }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(p.status, OL_DEVICE_GUARD);
    return;
  }
  P* const base = reinterpret_cast<P*>(c.base);
  const int step = blockDim.y * kKeepUnroll;
  for (int c0 = 0; c0 < pieces; c0 += blockDim.x) {
    const int x = c0 + threadIdx.x;
    for (int j0 = threadIdx.y; j0 - (int)threadIdx.y < n; j0 += step) {
      P v[kKeepUnroll];
#pragma unroll
      for (int u = 0; u < kKeepUnroll; ++u) {
        const int j = j0 + u * blockDim.y;
        if (j < n && x < pieces) v[u] = base[(j < kKeepRows ? from[j] : place(kept[j])) * pieces + x];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kKeepUnroll; ++u) {
        const int j = j0 + u * blockDim.y;
        if (j < n && x < pieces) base[(j < kKeepRows ? to[j] : place(j)) * pieces + x] = v[u];
      }
    }
  }
}

template <typename P>
cudaError_t launch_keep(const KeepParams& p, cudaStream_t s) {
  const int pieces = (int)((size_t)p.head_dim * (p.dtype == OL_F32 ? 4 : 2) / sizeof(P));
  const int x = pieces < kKeepThreads ? pieces : kKeepThreads;
  return launch_pdl(tree_keep_kernel<P>, dim3(p.cache.batch * p.cache.kv_heads, 2), dim3(x, kKeepThreads / x), 0, s, p,
                    pieces);
}

}  // namespace

void plan_generic_tree(TreeParams& p, int sms) {
  // one unit where 64 rows hold all of a kv head's: its K/V are read once
  p.rows_per_unit = tree_gen_rows(p.group, p.nodes);
  p.units_per_head = (p.group * p.nodes + p.rows_per_unit - 1) / p.rows_per_unit;
  p.tile_log2 = kTreeGenTileLog2;
  // as many CTAs as are resident
  const bool f32 = p.dtype == OL_F32, few = p.rows_per_unit == 32;
  const size_t smem = f32 ? (few ? gen_smem<float, 32>(p.head_dim) : gen_smem<float, 64>(p.head_dim))
                          : (few ? gen_smem<uint16_t, 32>(p.head_dim) : gen_smem<uint16_t, 64>(p.head_dim));
  const int fit = (int)(228 * 1024 / (smem + 1024)), regs = gen_per_sm((p.head_dim + 63) / 64, p.rows_per_unit);
  p.nctas = (fit < regs ? fit : regs) * (sms < kTreeMaxCtas ? sms : kTreeMaxCtas);
  p.extra = 2;
  p.by_unit = tree_few_units(p);
}

cudaError_t launch_generic_tree(const TreeParams& p, cudaStream_t s) {
  return p.dtype == OL_F32 ? launch_rows<float>(p, s) : launch_rows<uint16_t>(p, s);
}

cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t s) {
  const int rows = p.group * p.nodes < p.rows_per_unit ? p.group * p.nodes : p.rows_per_unit;
  return p.by_unit ? launch_merge<8, 512>(p, rows, s) : launch_merge<16, 256>(p, rows, s);
}

cudaError_t launch_tree_keep(const KeepParams& p, cudaStream_t s) {
  const size_t bytes = (size_t)p.head_dim * (p.dtype == OL_F32 ? 4 : 2);
  return bytes % 16 == 0 ? launch_keep<uint4>(p, s) : launch_keep<uint16_t>(p, s);
}

}  // namespace ol
