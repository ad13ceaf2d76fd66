// ol_rope.cu -- rotary positions: q, K (and any view of vectors) rotated on
// their way to the output or to the cache, V copied along, in one launch.
//
// Pair i of a vector at position p turns by p * f_i. The table holds
// f_i / (2 pi) in units of 2^-64 turn, so p * turns[i] in wrapping 64-bit
// integers is the angle modulo a turn without loss: what is off is the table's
// entry times p. ol_rope_turns computes it in doubles, off by a few 2^-56 turn: at
// position a million a few 2^-36 turn, where p * f_i in fp32 is off by 2^-24 * p
// radians. The
// signed product over 2^63 is the angle in half turns, in [-1, 1): sincospif's
// argument. Rotation in fp32, one rounding to the row's type.
//
// Bounds: 2 * D * elt bytes per vector against 3 * rot_dim flops: memory, or
// the launch itself for a decode step. One CTA takes one token of one row and
// all of its q, k and v vectors, so the token's sines and cosines are computed
// once (rot_dim / 2 threads, through shared memory) and serve every head. Its
// first vectors are on their way before the positions are known. Measured:
// 4 x 4096 fp32 tokens of 40 heads of 128 97 us, 6.9 TB/s; in bf16 58 us, 5.8 TB/s
// (interleaved 76 us, 4.4 TB/s). Where 16-byte pieces do not fit the rotation (half
// style: half of the rotated part; interleaved: all of it), the head or the views, an
// access moves one element: 4 x 2048 bf16 tokens of 40 heads of 80, 40 rotated, half
// style 62 us, 1.7 TB/s (interleaved, whole pieces: 30 us, 3.5 TB/s); of 96, 24
// rotated 99 us, 1.3 TB/s.
#include "ol_common.cuh"
#include "ol_draft.h"

namespace ol {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxHalf = 512;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t x) { return bf16_bits_to_float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t from_float<uint16_t>(float x) { return float_to_bf16_bits(x); }

// VE consecutive elements, moved as one access (16 bytes, or one element).
template <typename T, int VE>
struct alignas(sizeof(T) * VE) Piece {
  T e[VE];
};

// The work item i of a vector covers pieces a and b: in the half style the
// two halves of VE pairs, in the interleaved one VE / 2 pairs in one piece
// (or, element by element, the two elements of a pair). Items past the rotated
// part are single pieces that are copied.
template <int VE, bool HALF>
struct Items {
  static constexpr bool kTwo = HALF || VE == 1;  // a rotated item has two pieces
  static constexpr int kUnroll = kTwo ? 2 : 4;   // items in flight per thread
  int rotated, total;                            // items
  __device__ Items(int rot_dim, int head_dim)
      : rotated(kTwo ? rot_dim / 2 / VE : rot_dim / VE), total(rotated + (head_dim - rot_dim) / VE) {}
  __device__ int first(int i, int rot_dim) const {
    if (i >= rotated) return rot_dim + (i - rotated) * VE;
    return HALF || VE > 1 ? i * VE : 2 * i;
  }
  __device__ int second(int i, int rot_dim) const { return HALF ? rot_dim / 2 + i * VE : 2 * i + 1; }
};

template <typename T, int VE, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  using P = Piece<T, VE>;
  constexpr bool kTwo = Items<VE, HALF>::kTwo;
  constexpr int NP = kTwo ? VE : VE / 2;  // pairs of an item
  constexpr int kUnroll = Items<VE, HALF>::kUnroll;
  __shared__ float2 turn[kRopeMaxHalf];   // (cos, sin) * magnitude of this token
  const int b = blockIdx.x / p.tokens, t = blockIdx.x - b * p.tokens;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthreads = blockDim.x * blockDim.y;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const Items<VE, HALF> items(p.rot_dim, p.head_dim);
  const T* const q_row = reinterpret_cast<const T*>(p.q.data) + b * p.q.sb + t * p.q.st;
  const T* const k_row = reinterpret_cast<const T*>(p.k.data) + b * p.k.sb + t * p.k.st;
  const T* const v_row = reinterpret_cast<const T*>(p.v.data) + b * p.v.sb + t * p.v.st;
  P a[kUnroll], c[kUnroll];
  // pieces of item i of heads h0, h0 + blockDim.y, ...
  auto load = [&](int i, int h0) {
    const int ea = items.first(i, p.rot_dim), eb = items.second(i, p.rot_dim);
    const bool two = kTwo && i < items.rotated;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * blockDim.y;
      if (h >= heads) continue;
      const int g = h - p.q_heads;
      const T* const from = g < 0              ? q_row + h * p.q.sh
                            : g < p.kv_heads ? k_row + g * p.k.sh
                                             : v_row + (g - p.kv_heads) * p.v.sh;
      a[u] = *reinterpret_cast<const P*>(from + ea);
      if (two) c[u] = *reinterpret_cast<const P*>(from + eb);
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  if (p.counts && t >= p.counts[b]) return;
  load(threadIdx.x, threadIdx.y);  // (every thread has an item: blockDim.x is at most their number)
  const int start = p.positions ? p.positions[b] : 0;
  const long long at = p.angles ? p.angles[(size_t)b * p.tokens + t] : (long long)start + t;
  // where this token's K and V go: element offset of (plane 0, head 0), and the strides
  size_t slot = 0, head_stride = 0, plane_stride = 0;
  if (p.kv_heads) {
    const CacheRef& r = p.cache;
    const long long pos = (long long)start + t;
    if (start < 0 || pos >= r.capacity) return;  // device guard
    if (r.block_table) {
      const int n = (int)pos / r.page_size;
      const int page = r.block_table[(size_t)b * r.max_pages + n];
      if (page < 0 || page >= r.num_pages) return;  // device guard
      head_stride = (size_t)r.page_size * p.head_dim;
      slot = (size_t)page * r.kv_heads * head_stride + (size_t)((int)pos - n * r.page_size) * p.head_dim;
      plane_stride = (size_t)r.num_pages * r.kv_heads * head_stride;
    } else {
      head_stride = (size_t)r.capacity * p.head_dim;
      slot = (size_t)b * r.kv_heads * head_stride + (size_t)pos * p.head_dim;
      plane_stride = (size_t)r.batch * r.kv_heads * head_stride;
    }
  }
  for (int i = tid; i < p.rot_dim / 2; i += nthreads) {
    const long long phase = (long long)((unsigned long long)at * p.turns[i]);
    float s, co;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &co);
    turn[i] = make_float2(co * p.magnitude, s * p.magnitude);
  }
  __syncthreads();
  T* const q_out = reinterpret_cast<T*>(p.q_out.data) + b * p.q_out.sb + t * p.q_out.st;
  T* const cache = reinterpret_cast<T*>(p.cache.base) + slot;
  bool loaded = true;  // the first pieces
  for (int i = threadIdx.x; i < items.total; i += blockDim.x) {
    const bool rotated = i < items.rotated, two = kTwo && rotated;
    const int ea = items.first(i, p.rot_dim), eb = items.second(i, p.rot_dim);
    float2 cs[NP];
    if (rotated)
#pragma unroll
      for (int j = 0; j < NP; ++j) cs[j] = turn[i * NP + j];
    for (int h0 = threadIdx.y; h0 < heads; h0 += blockDim.y * kUnroll) {
      if (!loaded) load(i, h0);
      loaded = false;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * blockDim.y, g = h - p.q_heads;
        if (h >= heads) continue;
        if (rotated && g < p.kv_heads) {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            T& ex = kTwo ? a[u].e[j] : a[u].e[2 * j];
            T& ey = kTwo ? c[u].e[j] : a[u].e[(2 * j + 1) % VE];
            const float x = to_float<T>(ex), y = to_float<T>(ey);
            ex = from_float<T>(x * cs[j].x - y * cs[j].y);
            ey = from_float<T>(x * cs[j].y + y * cs[j].x);
          }
        }
        T* const to = g < 0              ? q_out + h * p.q_out.sh
                      : g < p.kv_heads ? cache + g * head_stride
                                       : cache + plane_stride + (g - p.kv_heads) * head_stride;
        *reinterpret_cast<P*>(to + ea) = a[u];
        if (two) *reinterpret_cast<P*>(to + eb) = c[u];
      }
    }
  }
}

template <typename T, int VE, bool HALF>
cudaError_t launch_style(const RopeParams& p, cudaStream_t s) {
  using I = Items<VE, HALF>;
  const int items = (I::kTwo ? p.rot_dim / 2 : p.rot_dim) / VE + (p.head_dim - p.rot_dim) / VE;
  const int heads = p.q_heads + 2 * p.kv_heads;
  cudaLaunchConfig_t cfg = {};
  // 16-bit vectors of many tokens: CTAs of 64 threads, whose loads and stores
  // interleave finer (4 x 4096 tokens of 32 + 2 * 8 heads of 128: half style
  // 69 us against 90 of 256 threads, interleaved 91 against 110). fp32 has twice
  // the bytes a thread: 118 us of 256 threads against 122 of 64, 122 against
  // 130. A few tokens are one wave either way: all of a token's vectors in one
  // round of loads (a decode step's append 3.4 us).
  const bool many = (long long)p.batch * p.tokens > 2048;
  const int most = sizeof(T) == 2 && many ? 64 : kRopeThreads;
  const int x = items < most ? items : most;
  const int fit = most / x, want = (heads + I::kUnroll - 1) / I::kUnroll;
  const int y = fit < want ? fit : want;
  cfg.gridDim = dim3(p.batch * p.tokens, 1, 1);
  cfg.blockDim = dim3(x, y, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<T, VE, HALF>, p);
}

template <typename T>
cudaError_t launch_type(const RopeParams& p, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T);
  if (p.style == OL_ROPE_HALF) return p.vec ? launch_style<T, VE, true>(p, s) : launch_style<T, 1, true>(p, s);
  return p.vec ? launch_style<T, VE, false>(p, s) : launch_style<T, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
  return p.dtype == OL_F32 ? launch_type<float>(p, s) : launch_type<uint16_t>(p, s);
}

}  // namespace ol
