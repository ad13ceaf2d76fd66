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

// A unit is up to eight (head, query) rows r = head * count + query of one row's kv head;
// all units' tiles of 32 tokens in equal shares, one per CTA (TreeWalk), so that short rows
// and few long ones fill the card alike. RB = 1, 2, 4 or 8 rows are what the call's units
// need. A group of LG = 8, 16 or 32 lanes has a token's head, eight dimensions a lane, and
// U = 16 / RB tokens in a row at a time, all of one page and one block:
//   s = sum q code, over the lanes by halves: a step sends half of the 16 sums away and
//       keeps the other, so that in the end a lane has one (or two, or half a) sum
//   p = 2^(s s_k scale log2(e) - m), m the group's running maximum of the row
//   o += (p s_v) code, the weights by shared memory; l += p
// q and o stay in registers (q of eight rows in shared memory), two fp32 products at a time.
// The groups' states are joined at a segment's end. The next codes of K are on their way
// while V's are worked on, and the other way round.
constexpr int TB = 1 << kTreeGenTileLog2;
constexpr int kFewRows = 16;
constexpr int kRowsThreads = 128, kRowsWarps = kRowsThreads / 32, kRowsCtas = 3;
template <int RB, int LG, bool MANY>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtas) fp8_attention_kernel(const __grid_constant__ Fp8AttnParams fp) {
  constexpr int NS = RB == 8 ? 32 : 16, U = NS / RB, GW = 32 / LG;          // sums and tokens of a group; groups of a warp
  constexpr int OWN = LG < NS ? NS / LG : 1, DUP = LG > NS ? LG / NS : 1;  // sums of a lane; lanes of a sum
  constexpr int RU = MANY ? RB * kRowsWarps : 8;                             // rows of a unit
  constexpr bool kHold = RB < 8;                                             // q in registers
  __shared__ float4 qs[kHold ? 1 : (MANY ? kRowsWarps : 1) * RB * 2 * LG];
  __shared__ ulonglong2 weights[kRowsWarps][GW][NS / 2];  // (w, w) of (token, row)
  __shared__ uint64_t keeps[kRowsWarps][GW][RB];          // (keep, keep) of a row
  __shared__ float2 states[kRowsWarps][RB];               // m, l
  __shared__ float4 sums[MANY ? 1 : kRowsWarps][MANY ? 1 : RB][2 * LG];
  const TreeParams& p = fp.t;
  const Fp8Cache& fc = fp.cache;
  const int D = p.head_dim, tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gl = lane % LG, gi = lane / LG;
  const bool there = gl * 8 < D;  // the lane's dimensions
  const int own = gl / DUP * OWN, own_r = own / U, own_u = own % U;  // its sums' row and first token
  const long long plane = (fc.block_table ? (long long)fc.num_pages * fc.page_size : (long long)fc.batch * fc.capacity) *
                          fc.kv_heads;  // vectors, and blocks, of K
  const long long plane_blocks =
      fc.block_table ? (long long)fc.num_pages * fc.kv_heads * (fc.page_size >> fc.block_log2)
                     : (long long)fc.batch * fc.kv_heads * ((fc.capacity + (1 << fc.block_log2) - 1) >> fc.block_log2);
  auto load_q = [&](long long row, int x, float4& a, float4& b) {  // elements 8 x .. 8 x + 7 of a row of q
    const long long at = row * D + 8 * x;
    if (p.dtype == OL_F32) {
      const float4* const q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at);
      a = q[0];
      b = q[1];
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + at);
      a = make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                      __uint_as_float(q.y & 0xffff0000u));
      b = make_float4(__uint_as_float(q.z << 16), __uint_as_float(q.z & 0xffff0000u), __uint_as_float(q.w << 16),
                      __uint_as_float(q.w & 0xffff0000u));
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  TreeWalk w(p);
  if (tid == kRowsThreads - 1) {
    TreeWalk notes = w;
    notes.write_splits(p);
  }
  while (w.next(p)) {
    const int r0 = w.qg * RU + (MANY ? warp * RB : 0), R = p.group * w.row.count;
    if (MANY && r0 >= R) continue;
    const long long base_row = tree_out_row(p, w.b, w.g, 0);  // of q and out
    const int t0 = w.row.start + w.tile0 * TB;
    const int n = min(w.row.len - t0, (w.tile1 - w.tile0) * TB);  // tokens of the segment
    const int low = (p.window < 0 || w.row.prefix <= p.window ? 0 : w.row.prefix - p.window) - t0;  // those before are hidden from all
    // token rel, rel + 1, .. of the segment: U at a time, a group each
    int rel = (MANY ? gi : warp * GW + gi) * U;
    constexpr int kStep = (MANY ? 1 : kRowsWarps) * GW * U;
    int page = 0;
    auto look = [&](int at) {  // the page of token `at`
      if (fc.block_table && at < n && at + U > low) page = fc.block_table[(size_t)w.b * fc.max_pages + (t0 + at) / fc.page_size];
    };
    const uint2 none = make_uint2(0, 0);
    uint2 k[U], v[U];
    float k_scale, v_scale;
    long long vec = 0, block = 0;  // of the group's first token, of its block
    bool known = false;            // the group has tokens that are seen, in a page of the pool
    auto load_k = [&](int at) {
      known = at < n && at + U > low;
      if (known) {
        if (!fc.block_table) {
          const long long head = (long long)w.b * fc.kv_heads + w.g;
          vec = head * fc.capacity + t0 + at;
          block = head * ((fc.capacity + (1 << fc.block_log2) - 1) >> fc.block_log2) + ((t0 + at) >> fc.block_log2);
        } else if (page >= 0 && page < fc.num_pages) {
          const long long head = (long long)page * fc.kv_heads + w.g;
          const int in = (t0 + at) % fc.page_size;
          vec = head * fc.page_size + in;
          block = head * (fc.page_size >> fc.block_log2) + (in >> fc.block_log2);
        } else {
          set_status(p.status, OL_DEVICE_GUARD);
          known = false;
        }
      }
      k_scale = known ? fc.scales[block] * p.scale_log2 : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        k[u] = known && there && at + u >= low && at + u < n
                   ? *reinterpret_cast<const uint2*>(fc.codes + (vec + u) * D + gl * 8) : none;
    };
    auto load_v = [&](int at) {
      v_scale = known ? fc.scales[block + plane_blocks] : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = known && there && at + u >= low && at + u < n
                   ? *reinterpret_cast<const uint2*>(fc.codes + (plane + vec + u) * D + gl * 8) : none;
    };
    look(rel);
    uint64_t q[kHold ? RB : 1][4];
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kHold) {
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        float4 a = zero, b = zero;
        if (there && r0 + r < R) load_q(base_row + tree_live_row(p, w.row.count, r0 + r), gl, a, b);
        q[kHold ? r : 0][0] = pack2(a.x, a.y);
        q[kHold ? r : 0][1] = pack2(a.z, a.w);
        q[kHold ? r : 0][2] = pack2(b.x, b.y);
        q[kHold ? r : 0][3] = pack2(b.z, b.w);
      }
    }
    load_k(rel);
    load_v(rel);
    float4* const mine = qs + (MANY ? warp * RB * 2 * LG : 0);  // of the unit, or of the warp
    auto sync = [] {
      if (MANY)
        __syncwarp();
      else
        __syncthreads();
    };
    sync();  // the last segment's queries and sums are read
    if (!kHold) {
      for (int i = MANY ? lane : tid; i < RB * LG; i += MANY ? 32 : kRowsThreads) {
        const int r = i / LG, x = i % LG;
        float4 a = zero, b = zero;
        if (x * 8 < D && r0 + r < R) load_q(base_row + tree_live_row(p, w.row.count, r0 + r), x, a, b);
        mine[(2 * r) * LG + x] = a;
        mine[(2 * r + 1) * LG + x] = b;
      }
      sync();
    }
    // of the lane's row: its last visible token, its first, from t0
    const int last = r0 + own_r < R ? w.row.prefix + (r0 + own_r) % w.row.count - t0 : -1;
    const int begin = p.window < 0 || last + t0 <= p.window ? -t0 : last - p.window;
    float m = -INFINITY, l = 0.f;
    uint64_t o[RB][4];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][e] = 0;
    for (int at = 0; at < n; at += kStep, rel += kStep) {  // (whole warps)
      look(rel + kStep);
      float s[NS];
      {
        uint64_t c[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = from_e4m3x2((e < 2 ? k[u].x : k[u].y) >> (e % 2 * 16));
            c[u][e] = pack2(x.x, x.y);
          }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          uint64_t q0 = q[kHold ? r : 0][0], q1 = q[kHold ? r : 0][1], q2 = q[kHold ? r : 0][2], q3 = q[kHold ? r : 0][3];
          if (!kHold) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&mine[kHold ? 0 : 2 * r * LG + gl]);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&mine[kHold ? 0 : (2 * r + 1) * LG + gl]);
            q0 = a.x, q1 = a.y, q2 = b.x, q3 = b.y;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float2 x = unpack2(fma2(c[u][3], q3, fma2(c[u][2], q2, fma2(c[u][1], q1, mul2(c[u][0], q0)))));
            s[r * U + u] = x.x + x.y;
          }
        }
      }
      const float ks = k_scale, vs = v_scale;
      load_k(rel + kStep);
#pragma unroll
      for (int step = 0; step < (LG == 8 ? 3 : LG == 16 ? 4 : 5); ++step) {
        const int h = NS / 2 >> step, x = LG / 2 >> step;
        if (h == 0) {
          s[0] += __shfl_xor_sync(0xffffffffu, s[0], x);
          continue;
        }
        const bool up = gl & x;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const float give = up ? s[i] : s[i + h], stay = up ? s[i + h] : s[i];
          s[i] = stay + __shfl_xor_sync(0xffffffffu, give, x);
        }
      }
      bool sees[OWN];
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const int t = rel + own_u + i;
        sees[i] = t <= last && t >= begin && t < n;
        s[i] = sees[i] ? s[i] * ks : -INFINITY;
        most = fmaxf(most, s[i]);
      }
#pragma unroll
      for (int x = DUP; x < U / OWN * DUP; x *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
      const float top = fmaxf(m, most), base = top == -INFINITY ? 0.f : top;
      const float keep = m == top ? 1.f : exp2f(m - base);
      m = top;
      l *= keep;
      __syncwarp();  // the last weights are read
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const float e = exp2f(s[i] - base), x = sees[i] ? e * vs : 0.f;  // (a scale of NaN is not seen)
        l += e;
        if (gl % DUP == 0) reinterpret_cast<uint64_t*>(weights[warp][gi])[(own_u + i) * RB + own_r] = pack2(x, x);
      }
      const bool grown = __any_sync(0xffffffffu, keep != 1.f);
      if (grown && gl % DUP == 0 && own_u == 0) keeps[warp][gi][own_r] = pack2(keep, keep);
      __syncwarp();
      if (grown)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const uint64_t f = keeps[warp][gi][r];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][e] = mul2(o[r][e], f);
        }
      uint64_t c[4];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int u = i / RB, r = i % RB;
        if (r == 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = from_e4m3x2((e < 2 ? v[u].x : v[u].y) >> (e % 2 * 16));
            c[e] = pack2(x.x, x.y);
          }
        const ulonglong2 two = weights[warp][gi][i / 2];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][e] = fma2(c[e], i % 2 ? two.y : two.x, o[r][e]);
      }
      load_v(rel + kStep);
    }
    // l of a row, then the warp's groups, then (in shared memory) the warps
#pragma unroll
    for (int x = DUP; x < U / OWN * DUP; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (GW > 1) {
      float top = m;
#pragma unroll
      for (int x = LG; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float f = exp2f(m - (top == -INFINITY ? 0.f : top));
      m = top;
      l *= f;
#pragma unroll
      for (int x = LG; x < 32; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
      __syncwarp();
      if (own_u == 0) keeps[warp][gi][own_r] = pack2(f, f);
    }
    if (gi == 0 && gl % DUP == 0 && own_u == 0) states[warp][own_r] = make_float2(m, l);
    __syncwarp();
    // the rows that this segment holds alone are done; others go to its slot
    float* const slot = w.whole() ? nullptr : tree_slot(p, w.slot);
    auto store = [&](int r, int d4, float top, float total, float4 y) {
      if (r0 + r >= R || 4 * d4 >= D) return;
      if (slot) {
        const int place = MANY ? warp * RB + r : r;
        if (d4 == 0) {
          slot[place] = top;
          slot[RU + place] = total;
        }
        reinterpret_cast<float4*>(slot + 2 * RU)[d4 * RU + place] = y;
        return;
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const size_t out = (size_t)(base_row + tree_live_row(p, w.row.count, r0 + r)) * D + 4 * d4;
      if (p.out_dtype == OL_F32)
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + out) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      else
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + out) =
            make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
    };
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float x[8];
      const uint64_t f = keeps[warp][gi][r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2(GW > 1 ? mul2(o[r][e], f) : o[r][e]);
        x[2 * e] = y.x;
        x[2 * e + 1] = y.y;
      }
#pragma unroll
      for (int i = LG; i < 32; i *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], i);
      const float4 y = make_float4(x[0], x[1], x[2], x[3]), z = make_float4(x[4], x[5], x[6], x[7]);
      if (gi != 0) continue;
      if (MANY) {
        const float2 state = states[warp][r];
        store(r, 2 * gl, state.x, state.y, y);
        store(r, 2 * gl + 1, state.x, state.y, z);
      } else {
        sums[MANY ? 0 : warp][MANY ? 0 : r][2 * gl] = y;
        sums[MANY ? 0 : warp][MANY ? 0 : r][2 * gl + 1] = z;
      }
    }
    if (MANY) continue;
    __syncthreads();
    for (int i = tid; i < RB * 2 * LG; i += kRowsThreads) {
      const int r = i / (2 * LG), d4 = i % (2 * LG);
      float top = -INFINITY, total = 0.f;
#pragma unroll
      for (int x = 0; x < kRowsWarps; ++x) top = fmaxf(top, states[x][r].x);
      float4 y = zero;
#pragma unroll
      for (int x = 0; x < kRowsWarps; ++x) {
        const float f = exp2f(states[x][r].x - (top == -INFINITY ? 0.f : top));
        const float4 z = sums[MANY ? 0 : x][MANY ? 0 : r][d4];
        total = fmaf(states[x][r].y, f, total);
        y = make_float4(fmaf(z.x, f, y.x), fmaf(z.y, f, y.y), fmaf(z.z, f, y.z), fmaf(z.w, f, y.w));
      }
      store(r, d4, top, total, y);
    }
  }
}

template <int RB, int LG, bool MANY>
cudaError_t launch_attention(const Fp8AttnParams& p, cudaStream_t s) {
  return launch_pdl(fp8_attention_kernel<RB, LG, MANY>, dim3(p.t.nctas), dim3(kRowsThreads), 0, s, p);
}

template <int RB, bool MANY>
cudaError_t launch_attention_dim(const Fp8AttnParams& p, cudaStream_t s) {
  return p.t.head_dim <= 64    ? launch_attention<RB, 8, MANY>(p, s)
         : p.t.head_dim <= 128 ? launch_attention<RB, 16, MANY>(p, s)
                               : launch_attention<RB, 32, MANY>(p, s);
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
  const int rows = p.group * p.nodes;
  p.rows_per_unit = rows > kFewRows ? 32 : 8;
  p.units_per_head = (rows + p.rows_per_unit - 1) / p.rows_per_unit;
  p.tile_log2 = kTreeGenTileLog2;
  const int ctas = kRowsCtas * sms;  // (as many notes as the workspace has at most)
  p.nctas = ctas < kTreeMaxShares ? ctas : kTreeMaxShares;
  p.extra = 2;
  p.compact = 1;
  p.by_unit = tree_few_units(p);
}

cudaError_t launch_generic_fp8(const Fp8AttnParams& p, cudaStream_t s) {
  const int rows = p.t.group * p.t.nodes;
  return rows == 1          ? launch_attention_dim<1, false>(p, s)
         : rows == 2        ? launch_attention_dim<2, false>(p, s)
         : rows <= 4        ? launch_attention_dim<4, false>(p, s)
         : rows <= kFewRows ? launch_attention_dim<8, false>(p, s)
                            : launch_attention_dim<8, true>(p, s);
}

}  // namespace ol
