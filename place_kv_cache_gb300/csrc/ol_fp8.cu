// ol_fp8.cu -- the E4M3 cache: the append that quantises, reading back, and
// attention on CUDA cores (fp32 queries, caches of more vectors than the tensor-core kernel of
// ol_fast_fp8.cu counts).
#include <type_traits>

#include "ol_fp8.cuh"
#include "ol_tree.cuh"

namespace ol {
namespace {

__device__ __forceinline__ uint32_t abs_max(uint32_t top, float x) { return max(top, __float_as_uint(x) & 0x7fffffffu); }
template <typename T>
__device__ __forceinline__ float value_of(T x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<uint16_t>(uint16_t x) { return bf16_bits_to_float(x); }
template <typename T>
__device__ __forceinline__ T rounded_to(float x);
template <>
__device__ __forceinline__ float rounded_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t rounded_to<uint16_t>(float x) { return float_to_bf16_bits(x); }

// N consecutive elements, moved as one access.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T e[N];
};

// The codes of N = 8, 4 or 1 elements.
template <int N>
using Codes = std::conditional_t<N == 8, uint2, std::conditional_t<N == 4, uint32_t, uint8_t>>;

// N codes times s, rounded to T.
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> values_of(Codes<N> z, float s) {
  Pack<T, N> w;
  auto two = [&](uint32_t codes, int j) {  // elements j, j + 1
    const float2 v = from_e4m3x2(codes);
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint32_t*>(&w.e[j]) = pack_bf16x2(v.x * s, v.y * s);
    } else {
      w.e[j] = v.x * s;
      w.e[j + 1] = v.y * s;
    }
  };
  if constexpr (N == 8) {
    two(z.x, 0);
    two(z.x >> 16, 2);
    two(z.y, 4);
    two(z.y >> 16, 6);
  } else if constexpr (N == 4) {
    two(z, 0);
    two(z >> 16, 2);
  } else {
    w.e[0] = rounded_to<T>(from_e4m3x2(z).x * s);
  }
  return w;
}

// ---------------------------------------------------------------------- append

// The scale that a block takes for a largest new element `most` (its bits, of the
// absolute value: NaN compares above infinity above numbers), given the scale `old`
// of the tokens that it holds already (begun) -- and what the earlier codes are
// multiplied by (1: they stay).
__device__ __forceinline__ float block_scale(uint32_t most, bool begun, float old, float& shrink) {
  shrink = 1.f;
  const float a = __uint_as_float(most);
  const bool finite = most < 0x7f800000u;
  if (begun && old != 0.f) {
    // (a scale that is no number above 0, which no append has written, would never reach a)
    if (!finite || !(old > 0.f) || !(old < INFINITY)) return __uint_as_float(0x7fc00000u);
    float limit = kFp8Top * old;
    while (a > limit) {  // few rounds: a token's largest element against its block's
      limit *= 2.f;
      old *= 2.f;
      shrink *= 0.5f;
    }
    return old;
  }
  if (!finite) return __uint_as_float(0x7fc00000u);
  return most == 0 ? 0.f : fmaxf(__fdiv_rn(a, kFp8Top), kFp8LeastScale);
}

// One CTA per block of tokens, head and plane that the call may reach. Its new
// elements stay in registers between the search for the largest and their
// quantising: KEEP pieces of VE elements a thread, every blockDim.x-th.
// The quotient x / s is x times the rounded inverse, set right by its remainder:
// q = x r, q + (x - q s) r is x / s rounded to nearest where r is 1 / s rounded to
// nearest (Markstein, Computation of elementary functions on the IBM RISC System/6000,
// 1990); the remainder is exact for all quotients that do not round to a code of 0.
template <typename T, int VE, int KEEP>
__global__ void __launch_bounds__(VE == 8 ? 512 : 1024, VE == 8 ? 2 : 1)
    fp8_append_kernel(const __grid_constant__ Fp8AppendParams p) {
  using P = Pack<T, VE>;
  __shared__ uint32_t tops[32];
  const Fp8Cache& c = p.cache;
  const int plane = blockIdx.y, tid = threadIdx.x;
  const int unit = blockIdx.x / c.kv_heads, g = blockIdx.x - unit * c.kv_heads;
  const int b = unit / p.blocks, nth = unit - b * p.blocks;
  const int pieces = c.head_dim / VE;
  // piece tid of the block's, and the way to every next one of this thread
  const int t_first = tid / pieces, x_first = tid - t_first * pieces;
  const int t_step = blockDim.x / pieces, x_step = blockDim.x - t_step * pieces;
  pdl_wait();
  pdl_launch_dependents();
  const int start = p.positions[b], n = p.counts ? p.counts[b] : p.new_len;
  if (start < 0 || start >= c.capacity || n <= 0 || n > p.new_len) return;  // (device guard)
  const int end = min(c.capacity - start, n) + start;
  const int first = ((start >> c.block_log2) + nth) << c.block_log2;  // the block's first token
  if (first >= end) return;
  const int lo = max(start, first), tokens = min(end, first + (1 << c.block_log2)) - lo;
  const RopeView& in = p.in[plane];
  const T* const from = reinterpret_cast<const T*>(in.data) + b * in.sb + g * in.sh + (long long)(lo - start) * in.st;
  P x[KEEP];
  int t = t_first, d = x_first;
  auto next = [&] {
    t += t_step;
    d += x_step;
    if (d >= pieces) d -= pieces, ++t;
  };
#pragma unroll
  for (int u = 0; u < KEEP; ++u, next())
    if (t < tokens) x[u] = *reinterpret_cast<const P*>(from + t * in.st + d * VE);
  long long row, at;
  if (!fp8_place(c, plane, b, g, first, row, at)) return;  // (device guard)
  const bool begun = lo > first;
  const float old = begun ? c.scales[at] : 0.f;
  uint32_t most = 0;
  t = t_first, d = x_first;
#pragma unroll
  for (int u = 0; u < KEEP; ++u, next())
    if (t < tokens) {
      if constexpr (VE == 8) {  // the absolute values' bits, two at a time
        const uint32_t* const w = reinterpret_cast<const uint32_t*>(&x[u]);
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                       __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu)));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) most = abs_max(most, value_of<T>(x[u].e[j]));
      }
    }
  if constexpr (VE == 8) most = max(most << 16, most & 0xffff0000u);
  most = __reduce_max_sync(0xffffffffu, most);
  if (blockDim.x > 32) {
    if (tid % 32 == 0) tops[tid / 32] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, tid % 32 < (int)blockDim.x / 32 ? tops[tid % 32] : 0);
  }
  float shrink;
  const float scale = block_scale(most, begun, old, shrink);
  uint8_t* const codes = c.codes + row * c.head_dim;
  if (shrink != 1.f) {
    const int words = (lo - first) * c.head_dim / 4;
    for (int i = tid; i < words; i += blockDim.x) {
      uint32_t* const w = reinterpret_cast<uint32_t*>(codes) + i;
      const float2 a = from_e4m3x2(*w), z = from_e4m3x2(*w >> 16);
      *w = e4m3x2(a.x * shrink, a.y * shrink) | e4m3x2(z.x * shrink, z.y * shrink) << 16;
    }
  }
  const bool coded = scale > 0.f;  // false for 0 and NaN
  const float inverse = coded ? __frcp_rn(scale) : 0.f;
  const uint64_t inverse2 = pack2(inverse, inverse), minus2 = pack2(-scale, -scale);
  auto coded_pair = [&](float v0, float v1) {
    const uint64_t v = pack2(v0, v1), q = mul2(v, inverse2);
    const float2 r = unpack2(fma2(fma2(q, minus2, v), inverse2, q));
    return coded ? e4m3x2(r.x, r.y) : 0u;
  };
  uint8_t* const to = codes + (long long)(lo - first) * c.head_dim;
  t = t_first, d = x_first;
#pragma unroll
  for (int u = 0; u < KEEP; ++u, next()) {
    if (t >= tokens) continue;
    auto two = [&](int j) { return coded_pair(value_of<T>(x[u].e[j]), value_of<T>(x[u].e[VE > 1 ? j + 1 : j])); };
    Codes<VE> y;
    if constexpr (VE == 8)
      y = make_uint2(two(0) | two(2) << 16, two(4) | two(6) << 16);
    else if constexpr (VE == 4)
      y = two(0) | two(2) << 16;
    else
      y = (uint8_t)two(0);
    *reinterpret_cast<Codes<VE>*>(to + t * c.head_dim + d * VE) = y;
  }
  if (tid == 0) c.scales[at] = scale;  // (every thread has read the old one)
}

template <typename T, int VE, int KEEP>
cudaError_t launch_append_cfg(const Fp8AppendParams& p, cudaStream_t s) {
  const int block = 1 << p.cache.block_log2, tokens = p.new_len < block ? p.new_len : block;
  const int pieces = tokens * (p.cache.head_dim / VE);
  const int threads = ((pieces + KEEP - 1) / KEEP + 31) / 32 * 32;
  return launch_pdl(fp8_append_kernel<T, VE, KEEP>, dim3((unsigned)p.cache.batch * p.blocks * p.cache.kv_heads, 2),
                    dim3(threads), 0, s, p);
}

// ------------------------------------------------------------------------ read

constexpr int kReadThreads = 256, kReadUnroll = 8, kReadMost = 128;

// A CTA reads a run of one row's tokens of a head, K and V: places and scales are
// looked up once a token, then a thread has VE consecutive elements (16 bytes of
// output) of up to 8 tokens, all on their way together.
template <typename T, int VE>
__global__ void __launch_bounds__(kReadThreads, 4) fp8_read_kernel(const __grid_constant__ Fp8ReadParams p, int runs, int run_tokens) {
  __shared__ long long rows[2][kReadMost];  // of the token's codes; -1: it is not read
  __shared__ float scales[2][kReadMost];
  const Fp8Cache& c = p.cache;
  const int unit = blockIdx.x / c.kv_heads, g = blockIdx.x - unit * c.kv_heads;
  const int b = unit / runs, first = (unit - b * runs) * run_tokens, tid = threadIdx.x;
  const int pieces = c.head_dim / VE, y = tid / pieces, x = tid - y * pieces, step = kReadThreads / pieces;
  pdl_wait();
  pdl_launch_dependents();
  const int start = p.starts[b], n = min(p.counts ? p.counts[b] : p.tokens, p.tokens);
  if (start < 0 || first >= n) return;  // (device guard)
  for (int i = tid; i < 2 * run_tokens; i += kReadThreads) {
    const int plane = i >= run_tokens, t = i - plane * run_tokens;
    long long row = -1, at;
    if (p.out[plane].data && first + t < n && (long long)start + first + t < c.capacity &&
        fp8_place(c, plane, b, g, start + first + t, row, at))
      scales[plane][t] = c.scales[at];
    else
      row = -1;
    rows[plane][t] = row;
  }
  __syncthreads();
  if (y >= step) return;
#pragma unroll
  for (int plane = 0; plane < 2; ++plane) {
    const RopeView& out = p.out[plane];
    if (!out.data) continue;
    T* const to = reinterpret_cast<T*>(out.data) + b * out.sb + g * out.sh + (long long)first * out.st + x * VE;
    Codes<VE> z[kReadUnroll];
    long long row[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int t = y + u * step;
      row[u] = t < run_tokens ? rows[plane][t] : -1;
      if (row[u] >= 0) z[u] = *reinterpret_cast<const Codes<VE>*>(c.codes + row[u] * c.head_dim + x * VE);
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int t = y + u * step;
      if (row[u] < 0) continue;
      *reinterpret_cast<Pack<T, VE>*>(to + t * out.st) = values_of<T, VE>(z[u], scales[plane][t]);
    }
  }
}

template <typename T, int VE>
cudaError_t launch_read_cfg(const Fp8ReadParams& p, cudaStream_t s) {
  const int step = kReadThreads / (p.cache.head_dim / VE), run = step * kReadUnroll;  // tokens a pass, and a CTA
  const int tokens = run < kReadMost ? run : kReadMost;
  const int runs = (p.tokens + tokens - 1) / tokens;
  return launch_pdl(fp8_read_kernel<T, VE>, dim3((unsigned)p.cache.batch * runs * p.cache.kv_heads), dim3(kReadThreads), 0, s,
                    p, runs, tokens);
}

// ------------------------------------------------------- attention, CUDA cores

// A unit is 32 or 64 (head, query) rows r = head * count + query of one row's kv head,
// its tokens form tiles of 32; all units' tiles in equal shares, one per CTA (TreeWalk). Scores and sums
// in registers: 4 rows x 2 tokens of S, 4 rows x D / 16 dimensions of O a thread. A
// tile's codes come into registers while the tile before is worked on, and lie in
// shared memory as fp32 values, their scales multiplied in.
constexpr int TB = 1 << kTreeGenTileLog2;
__host__ __device__ inline int padded_floats(int D) { return D + 4; }  // of a row: 8 rows cover the banks
template <int RB>
inline size_t gen_smem(int D) {
  return sizeof(float) * ((size_t)TB * (RB + 4) + (size_t)(RB + 2 * TB) * padded_floats(D));
}
template <typename T, int NC, int RB>
__global__ void __launch_bounds__(4 * RB) fp8_attention_kernel(const __grid_constant__ Fp8AttnParams fp) {
  constexpr int kThreads = 4 * RB, kPStride = RB + 4;
  constexpr int kPieces = 2 * TB * NC * 4 / kThreads;  // 16 codes each, of a thread
  extern __shared__ __align__(16) uint8_t smem[];
  const TreeParams& p = fp.t;
  const Fp8Cache& fc = fp.cache;
  const int D = p.head_dim, Dp = padded_floats(D), per_row = D / 16;
  float* const sp = reinterpret_cast<float*>(smem);
  float* const sq = sp + TB * kPStride;
  float* const sk = sq + RB * Dp;
  float* const sv = sk + TB * Dp;
  const int tid = threadIdx.x, rg = tid / 16, cg = tid % 16;
  pdl_wait();
  pdl_launch_dependents();
  TreeWalk w(p);
  if (tid == kThreads - 1) {
    TreeWalk notes = w;
    notes.write_splits(p);
  }
  while (w.next(p)) {
    const int r0 = w.qg * RB, R = p.group * w.row.count;
    const size_t base_row = tree_out_row(p, w.b, w.g, 0);  // of q and out
    const int low_all = p.window < 0 || w.row.prefix <= p.window ? 0 : w.row.prefix - p.window;
    uint4 code[kPieces];
    float scale[kPieces];
    auto fetch = [&](int tile) {
      const int t0 = w.row.start + tile * TB;
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int i = tid + u * kThreads;
        code[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0.f;
        if (i >= 2 * TB * per_row) continue;
        const int vec = i / per_row, plane = vec / TB, j = vec % TB;
        if (j < low_all - t0 || j >= w.row.len - t0) continue;
        long long row, at;
        if (!fp8_place(fc, plane, w.b, w.g, t0 + j, row, at)) {
          set_status(p.status, OL_DEVICE_GUARD);
          continue;
        }
        code[u] = *reinterpret_cast<const uint4*>(fc.codes + row * D + (i - vec * per_row) * 16);
        scale[u] = fc.scales[at];
      }
    };
    auto put = [&] {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int i = tid + u * kThreads;
        if (i >= 2 * TB * per_row) continue;
        const int vec = i / per_row;
        float* const to = (vec < TB ? sk : sv) + (vec % TB) * Dp + (i - vec * per_row) * 16;
        const uint32_t z[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 a = from_e4m3x2(z[x]), e = from_e4m3x2(z[x] >> 16);
          const float sc = scale[u];
          *reinterpret_cast<float4*>(to + 4 * x) = make_float4(a.x * sc, a.y * sc, e.x * sc, e.y * sc);
        }
      }
    };
    __syncthreads();  // the last segment's queries and tiles are read
    {
      const int r = tid / 4;  // four threads a row
      const T* const q = reinterpret_cast<const T*>(p.q) +
                         (base_row + (r0 + r < R ? tree_live_row(p, w.row.count, r0 + r) : 0)) * D;
      for (int d = tid % 4 * 4; d < D; d += 16)
#pragma unroll
        for (int e = 0; e < 4; ++e) sq[r * Dp + d + e] = r0 + r < R ? value_of<T>(q[d + e]) : 0.f;
    }
    fetch(w.tile0);
    int at[4], low[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      at[r] = w.row.prefix + (r0 + 4 * rg + r) % w.row.count;
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
      __syncthreads();  // the last tile is read
      put();
      __syncthreads();
      if (tile + 1 < w.tile1) fetch(tile + 1);
      float s[4][2];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(sk + cg * Dp + d);
        const float4 k1 = *reinterpret_cast<const float4*>(sk + (cg + 16) * Dp + d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 a = *reinterpret_cast<const float4*>(sq + (4 * rg + r) * Dp + d);
          s[r][0] = fmaf(a.w, k0.w, fmaf(a.z, k0.z, fmaf(a.y, k0.y, fmaf(a.x, k0.x, s[r][0]))));
          s[r][1] = fmaf(a.w, k1.w, fmaf(a.z, k1.z, fmaf(a.y, k1.y, fmaf(a.x, k1.x, s[r][1]))));
        }
      }
      bool some = false;  // some row of the warp may not see some token of the tile
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = cg + 16 * u;
          s[r][u] *= p.scale_log2;
          if (j > at[r] - t0 || j < low[r] - t0) s[r][u] = -INFINITY, some = true;
        }
      some = __any_sync(0xffffffffu, some);
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
      for (int c = 0; c < NC; ++c) dims[c] = c * 64 + cg * 4 < D ? c * 64 + cg * 4 : 0;
      auto add = [&](auto hidden) {  // whether there may be tokens hidden from some row: their V may be NaN
#pragma unroll 4
        for (int j = 0; j < TB; ++j) {
          const float4 p4 = *reinterpret_cast<const float4*>(sp + j * kPStride + 4 * rg);
          const float pj[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(sv + j * Dp + dims[c]);
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
          if (d4 * 4 < D) reinterpret_cast<float4*>(slot + 2 * RB)[d4 * RB + row] = o[r][c];
        }
      } else {
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        const size_t out = (base_row + tree_live_row(p, w.row.count, r0 + row)) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = c * 64 + cg * 4;
          const float v[4] = {o[r][c].x, o[r][c].y, o[r][c].z, o[r][c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d < D) store_out(p.out, p.out_dtype, out + d + j, v[j] * inv);
        }
      }
    }
  }
}

template <typename T, int NC, int RB>
cudaError_t launch_attention(const Fp8AttnParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [] {
    const cudaError_t e = cudaFuncSetAttribute(fp8_attention_kernel<T, NC, RB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)gen_smem<RB>(64 * NC));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fp8_attention_kernel<T, NC, RB>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(fp8_attention_kernel<T, NC, RB>, dim3(p.t.nctas), dim3(4 * RB), gen_smem<RB>(p.t.head_dim), s, p);
}

template <typename T, int RB>
cudaError_t launch_attention_dim(const Fp8AttnParams& p, cudaStream_t s) {
  const int nc = (p.t.head_dim + 63) / 64;
  return nc == 1   ? launch_attention<T, 1, RB>(p, s)
         : nc == 2 ? launch_attention<T, 2, RB>(p, s)
         : nc == 3 ? launch_attention<T, 3, RB>(p, s)
                   : launch_attention<T, 4, RB>(p, s);
}

template <typename T>
cudaError_t launch_attention_type(const Fp8AttnParams& p, cudaStream_t s) {
  return p.t.rows_per_unit == 32 ? launch_attention_dim<T, 32>(p, s) : launch_attention_dim<T, 64>(p, s);
}

}  // namespace

cudaError_t launch_fp8_append(const Fp8AppendParams& p, cudaStream_t s) {
  if (p.dtype == OL_F32) return p.vec ? launch_append_cfg<float, 4, 8>(p, s) : launch_append_cfg<float, 1, 32>(p, s);
  return p.vec ? launch_append_cfg<uint16_t, 8, 8>(p, s) : launch_append_cfg<uint16_t, 1, 32>(p, s);
}

cudaError_t launch_fp8_read(const Fp8ReadParams& p, cudaStream_t s) {
  if (p.dtype == OL_F32) return p.vec ? launch_read_cfg<float, 4>(p, s) : launch_read_cfg<float, 1>(p, s);
  return p.vec ? launch_read_cfg<uint16_t, 8>(p, s) : launch_read_cfg<uint16_t, 1>(p, s);
}

void plan_generic_fp8(Fp8AttnParams& fp, int sms) {
  TreeParams& p = fp.t;
  p.rows_per_unit = tree_gen_rows(p.group, p.nodes);
  p.units_per_head = (p.group * p.nodes + p.rows_per_unit - 1) / p.rows_per_unit;
  p.tile_log2 = kTreeGenTileLog2;
  const size_t smem = p.rows_per_unit == 32 ? gen_smem<32>(p.head_dim) : gen_smem<64>(p.head_dim);
  const int fit = (int)(228 * 1024 / (smem + 1024)), most = 128 / p.rows_per_unit;  // (the workspace's slots)
  p.nctas = (fit < most ? fit : most) * (sms < kTreeMaxCtas ? sms : kTreeMaxCtas);
  p.extra = 2;
  p.compact = 1;
  p.by_unit = tree_few_units(p);
}

cudaError_t launch_generic_fp8(const Fp8AttnParams& p, cudaStream_t s) {
  return p.t.dtype == OL_F32 ? launch_attention_type<float>(p, s) : launch_attention_type<uint16_t>(p, s);
}

}  // namespace ol
