// ol_norm_rope.cu -- root-mean-square norms of queries and keys for each head and
// their rotation, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * (w + offset), then the pairs of y's leading
//   rot_dim elements turn by their position's angle (ol_rope.cu has the table's
//   arithmetic).
//
// One CTA takes one token of one row and all of its q and k vectors, so that the
// token's sines and cosines are computed once. A group of LANES lanes has a vector:
// it is read once, its squares are summed by shuffles in fp32, and it is written
// once. Bounds: 2 * D * elt bytes a vector: memory, or the launch for a decode step.
#include "ol_common.cuh"
#include "ol_fp8.h"

namespace ol {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxHalf = 512;

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return bf16_bits_to_float(x); }
template <typename T>
__device__ __forceinline__ T rounded_to(float x);
template <>
__device__ __forceinline__ float rounded_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t rounded_to<uint16_t>(float x) { return float_to_bf16_bits(x); }

template <typename T, int VE>
struct alignas(sizeof(T) * VE) Piece {
  T e[VE];
};

// Item i of a vector: in the rotated part two pieces, of VE pairs' two elements (half
// style), or one piece of VE / 2 pairs (interleaved; the two elements of a pair where
// VE is 1); past it single pieces.
template <int VE, bool HALF>
struct Items {
  static constexpr bool kTwo = HALF || VE == 1;
  int rotated, total;
  __host__ __device__ Items(int rot, int dim)
      : rotated(kTwo ? rot / 2 / VE : rot / VE), total(rotated + (dim - rot) / VE) {}
  __device__ int first(int i, int rot) const {
    if (i >= rotated) return rot + (i - rotated) * VE;
    return HALF || VE > 1 ? i * VE : 2 * i;
  }
  __device__ int second(int i, int rot) const { return HALF ? rot / 2 + i * VE : 2 * i + 1; }
};

// NI items of a vector a lane.
template <typename T, int VE, bool HALF, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int lanes) {
  using P = Piece<T, VE>;
  using I = Items<VE, HALF>;
  constexpr int NP = I::kTwo ? VE : VE / 2;    // pairs of an item
  constexpr int U = NI == 1 ? 2 : 1;           // vectors of a group in flight
  __shared__ float2 turn[kMaxHalf];
  const int b = blockIdx.x / p.tokens, t = blockIdx.x - b * p.tokens;
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = blockDim.x / lanes;
  const int heads = p.q_heads + p.kv_heads;
  const I items(p.rot_dim, p.head_dim);
  const T* const q = reinterpret_cast<const T*>(p.in[0].data) + b * p.in[0].sb + t * p.in[0].st;
  const T* const k = reinterpret_cast<const T*>(p.in[1].data) + b * p.in[1].sb + t * p.in[1].st;
  P x[U][NI], z[U][NI];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * groups;
      if (h >= heads) continue;
      const T* const from = h < p.q_heads ? q + h * p.in[0].sh : k + (h - p.q_heads) * p.in[1].sh;
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int i = lane + n * lanes;
        if (i >= items.total) continue;
        x[u][n] = *reinterpret_cast<const P*>(from + items.first(i, p.rot_dim));
        if (I::kTwo && i < items.rotated) z[u][n] = *reinterpret_cast<const P*>(from + items.second(i, p.rot_dim));
      }
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  load(group);
  if (p.turns) {
    const long long at = p.angles ? p.angles[(size_t)b * p.tokens + t] : (long long)p.positions[b] + t;
    for (int i = threadIdx.x; i < p.rot_dim / 2; i += blockDim.x) {
      const long long phase = (long long)((unsigned long long)at * p.turns[i]);
      float s, c;
      sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
      turn[i] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    __syncthreads();
  }
  T* const q_out = reinterpret_cast<T*>(p.out[0].data) + b * p.out[0].sb + t * p.out[0].st;
  T* const k_out = reinterpret_cast<T*>(p.out[1].data) + b * p.out[1].sb + t * p.out[1].st;
  const float per = 1.f / p.head_dim;
  for (int h0 = group; h0 - group < heads; h0 += groups * U) {  // (whole warps: the shuffles)
    if (h0 != group) load(h0);
    float sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u] = 0.f;
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int i = lane + n * lanes;
        if (i >= items.total || h0 + u * groups >= heads) continue;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float v = value_of(x[u][n].e[j]);
          sum[u] = fmaf(v, v, sum[u]);
        }
        if (I::kTwo && i < items.rotated)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float v = value_of(z[u][n].e[j]);
            sum[u] = fmaf(v, v, sum[u]);
          }
      }
    }
    for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * groups;
      if (h >= heads) continue;
      const bool is_q = h < p.q_heads;
      const float r = 1.f / sqrtf(fmaf(sum[u], per, p.eps));
      const T* const weight = reinterpret_cast<const T*>(p.weight[is_q ? 0 : 1]);
      T* const to = is_q ? q_out + h * p.out[0].sh : k_out + (h - p.q_heads) * p.out[1].sh;
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int i = lane + n * lanes;
        if (i >= items.total) continue;
        const int ea = items.first(i, p.rot_dim), eb = items.second(i, p.rot_dim);
        const bool rotated = i < items.rotated, two = I::kTwo && rotated;
        P wa, wb;
        if (weight) {
          wa = *reinterpret_cast<const P*>(weight + ea);
          if (two) wb = *reinterpret_cast<const P*>(weight + eb);
        }
        auto normed = [&](T e, T w) { return value_of(e) * r * (weight ? value_of(w) + p.weight_offset : 1.f); };
        float ya[VE], yb[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          ya[j] = normed(x[u][n].e[j], wa.e[j]);
          if (two) yb[j] = normed(z[u][n].e[j], wb.e[j]);
        }
        if (rotated)
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float2 cs = turn[i * NP + j];
            float& a = I::kTwo ? ya[j] : ya[2 * j];
            float& c = I::kTwo ? yb[j] : ya[(2 * j + 1) % VE];
            const float a0 = a, c0 = c;
            a = a0 * cs.x - c0 * cs.y;
            c = a0 * cs.y + c0 * cs.x;
          }
        P y;
#pragma unroll
        for (int j = 0; j < VE; ++j) y.e[j] = rounded_to<T>(ya[j]);
        *reinterpret_cast<P*>(to + ea) = y;
        if (two) {
#pragma unroll
          for (int j = 0; j < VE; ++j) y.e[j] = rounded_to<T>(yb[j]);
          *reinterpret_cast<P*>(to + eb) = y;
        }
      }
    }
  }
}

template <typename T, int VE, bool HALF, int NI>
cudaError_t launch_items(const NormRopeParams& p, int lanes, cudaStream_t s) {
  constexpr int U = NI == 1 ? 2 : 1;
  const int heads = p.q_heads + p.kv_heads;
  const int want = ((heads + U - 1) / U * lanes + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch * p.tokens);
  cfg.blockDim = dim3(want < kNormThreads ? want : kNormThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, VE, HALF, NI>, p, lanes);
}

template <typename T, int VE, bool HALF>
cudaError_t launch_style(const NormRopeParams& p, cudaStream_t s) {
  const int items = Items<VE, HALF>(p.rot_dim, p.head_dim).total;
  int lanes = 1;
  while (lanes < 32 && lanes < items) lanes *= 2;
  if (items <= 32) return launch_items<T, VE, HALF, 1>(p, lanes, s);
  if (items <= 128) return launch_items<T, VE, HALF, 4>(p, lanes, s);
  return launch_items<T, VE, HALF, VE == 1 ? 32 : 8>(p, lanes, s);  // head_dim is 1024 at most
}

template <typename T>
cudaError_t launch_type(const NormRopeParams& p, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T);
  if (p.style == OL_ROPE_HALF) return p.vec ? launch_style<T, VE, true>(p, s) : launch_style<T, 1, true>(p, s);
  return p.vec ? launch_style<T, VE, false>(p, s) : launch_style<T, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
  return p.dtype == OL_F32 ? launch_type<float>(p, s) : launch_type<uint16_t>(p, s);
}

}  // namespace ol
