// Rotate-half rotary positions with several axes: pair i (elements i and
// i + R/2 of a head, R the rotated width) turns by the table row of its own
// axis' position,
//   y_i = x_i c - x_{i+R/2} s,   y_{i+R/2} = x_{i+R/2} c + x_i s,
//   (c, s) = table[positions[axis(i)][t]][i]
// ("[Feature] Sage Attention Support Varlen & write kv cache BF16/FP16",
// Description item 1, with the position a vector).  As in the cache write,
// each product and sum is rounded to float32 separately and the result once
// to the type.  With `inverse` the angle is negated: the inverse rotation,
// which is also the transposed one that a gradient needs.
//
// HBM-bound: every element is read and written once.  A token's table values
// are shared by all its heads, so a warp takes one token, keeps the values of
// its pairs in registers and walks the heads: with 8 pairs a lane (16 bytes
// of each half) 64 pairs take 8 lanes, and 4 heads go side by side.  When the
// tokens alone do not fill the GPU the heads are split over blockIdx.y.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace qpkv {
namespace {

constexpr int kWarps = 4;

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
  E v[V];
};

template <typename E>
__device__ __forceinline__ float to_f32(E x) {
  if constexpr (std::is_same<E, float>::value) return x;
  if constexpr (std::is_same<E, __half>::value) return __half2float(x);
  if constexpr (std::is_same<E, __nv_bfloat16>::value) return __bfloat162float(x);
}
template <typename E>
__device__ __forceinline__ E from_f32(float x) {
  if constexpr (std::is_same<E, float>::value) return x;
  if constexpr (std::is_same<E, __half>::value) return __float2half_rn(x);
  if constexpr (std::is_same<E, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
}

struct RopeArgs {
  int T, Hq, Hkv, D, half, num_axes, max_pos, inverse, heads_per_block;
  long long axis_stride;
  const int32_t* pos;
  const float *cos_t, *sin_t;
  const void *q, *k;
  void *q_out, *k_out;
  long long qs_t, qs_h, ks_t, ks_h, qo_t, qo_h, ko_t, ko_h;   // elements
  int* err;
  uint8_t axis[128];
};

template <typename E, int V>
__global__ void __launch_bounds__(kWarps * 32) rope_axes_kernel(const __grid_constant__ RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  int pos[4] = {0, 0, 0, 0};
  bool bad = false;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (x < a.num_axes) {
      pos[x] = __ldg(a.pos + x * a.axis_stride + t);
      bad |= pos[x] < 0 || pos[x] >= a.max_pos;
    }
  }
  if (bad) {   // -1 on the first axis: a padding row; anything else is reported
    if (lane == 0 && blockIdx.y == 0 && pos[0] != -1) report_error(a.err, kDevErrBadLength);
    return;
  }
  const int slots = a.half / V;
  const int side = slots >= 32 ? 1 : 32 / slots;   // heads next to one another in the warp
  const int h0 = blockIdx.y * a.heads_per_block;
  const int h1 = min(a.Hq + a.Hkv, h0 + a.heads_per_block);
  const int hl = lane / slots;                     // this lane's head among them
  if (slots < 32 && hl >= side) return;
  for (int s = slots >= 32 ? lane : lane % slots; s < slots; s += slots >= 32 ? 32 : slots) {
    float c[V], d[V];
    const int i0 = s * V;
    bool same = true;
#pragma unroll
    for (int e = 1; e < V; ++e) same &= a.axis[i0 + e] == a.axis[i0];
    if (same) {
      const int x = a.axis[i0];
      const size_t row = static_cast<size_t>(x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3]) * a.half + i0;
      if constexpr (V >= 4) {   // half is a multiple of V: 16-byte rows
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const float4 cc = __ldg(reinterpret_cast<const float4*>(a.cos_t + row + e));
          const float4 ss = __ldg(reinterpret_cast<const float4*>(a.sin_t + row + e));
          c[e] = cc.x, c[e + 1] = cc.y, c[e + 2] = cc.z, c[e + 3] = cc.w;
          d[e] = ss.x, d[e + 1] = ss.y, d[e + 2] = ss.z, d[e + 3] = ss.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          c[e] = __ldg(a.cos_t + row + e);
          d[e] = __ldg(a.sin_t + row + e);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int x = a.axis[i0 + e];
        const size_t row = static_cast<size_t>(x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3]) * a.half + i0 + e;
        c[e] = __ldg(a.cos_t + row);
        d[e] = __ldg(a.sin_t + row);
      }
    }
    if (a.inverse) {
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = -d[e];
    }
    using VE = Vec<E, V>;
#pragma unroll 1   // more warps rather than more loads a warp: 57 us against 66 (unroll 4) for 16384 tokens
    for (int h = h0 + hl; h < h1; h += side) {
      const bool isq = h < a.Hq;
      const int hh = isq ? h : h - a.Hq;
      const E* src = static_cast<const E*>(isq ? a.q : a.k) + (isq ? t * a.qs_t + hh * a.qs_h : t * a.ks_t + hh * a.ks_h);
      E* dst = static_cast<E*>(isq ? a.q_out : a.k_out) + (isq ? t * a.qo_t + hh * a.qo_h : t * a.ko_t + hh * a.ko_h);
      const VE x1 = *reinterpret_cast<const VE*>(src + i0);
      const VE x2 = *reinterpret_cast<const VE*>(src + a.half + i0);
      VE y1, y2;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = to_f32(x1.v[e]), w = to_f32(x2.v[e]);
        y1.v[e] = from_f32<E>(__fsub_rn(__fmul_rn(u, c[e]), __fmul_rn(w, d[e])));
        y2.v[e] = from_f32<E>(__fadd_rn(__fmul_rn(w, c[e]), __fmul_rn(u, d[e])));
      }
      *reinterpret_cast<VE*>(dst + i0) = y1;
      *reinterpret_cast<VE*>(dst + a.half + i0) = y2;
    }
  }
  // the elements behind the rotated width go over as they are
  const int rest = a.D - 2 * a.half;
  if (rest > 0) {
    for (int h = h0; h < h1; ++h) {
      const bool isq = h < a.Hq;
      const int hh = isq ? h : h - a.Hq;
      const E* src = static_cast<const E*>(isq ? a.q : a.k) + (isq ? t * a.qs_t + hh * a.qs_h : t * a.ks_t + hh * a.ks_h);
      E* dst = static_cast<E*>(isq ? a.q_out : a.k_out) + (isq ? t * a.qo_t + hh * a.qo_h : t * a.ko_t + hh * a.ko_h);
      if (src == dst) continue;
      const int lanes = slots >= 32 ? 32 : side * slots;
      for (int e = 2 * a.half + lane; e < a.D; e += lanes) dst[e] = src[e];
    }
  }
}

template <typename E, int V>
cudaError_t go(const RopeArgs& a, int head_blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + kWarps - 1) / kWarps), static_cast<unsigned>(head_blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_axes_kernel<E, V>, a);
}

template <typename E>
cudaError_t pick(const RopeArgs& a, int vec, int head_blocks, cudaStream_t stream) {
  if constexpr (sizeof(E) == 2) {
    if (vec >= 8) return go<E, 8>(a, head_blocks, stream);
  }
  if (vec >= 4) return go<E, 4>(a, head_blocks, stream);
  if (vec >= 2) return go<E, 2>(a, head_blocks, stream);
  return go<E, 1>(a, head_blocks, stream);
}

}  // namespace

cudaError_t launch_rope_axes(const qpkv_rope_axes_params& p, cudaStream_t stream) {
  RopeArgs a;
  a.T = p.num_tokens;
  a.Hq = p.num_heads_q;
  a.Hkv = p.k != nullptr ? p.num_heads_kv : 0;
  a.D = p.head_dim;
  a.half = p.rot_dim / 2;
  a.num_axes = p.num_axes;
  a.max_pos = p.rope_max_pos;
  a.inverse = p.inverse;
  a.axis_stride = p.axis_stride;
  a.pos = p.positions;
  a.cos_t = p.rope_cos;
  a.sin_t = p.rope_sin;
  a.q = p.q;
  a.k = p.k;
  a.q_out = p.q_out;
  a.k_out = p.k_out;
  a.qs_t = p.q_stride_t, a.qs_h = p.q_stride_h, a.ks_t = p.k_stride_t, a.ks_h = p.k_stride_h;
  a.qo_t = p.q_out_stride_t, a.qo_h = p.q_out_stride_h;
  a.ko_t = p.k_out_stride_t, a.ko_h = p.k_out_stride_h;
  a.err = p.error_word;
  for (int i = 0; i < 128; ++i) a.axis[i] = i < a.half ? p.pair_axis[i] : 0;
  // the widest vector (at most 16 bytes) that every row start allows
  const int es = p.dtype == QPKV_DTYPE_F32 ? 4 : 2;
  int vec = 16 / es;
  auto fits = [&](int v) {
    if (a.half % v) return false;
    const long long st[8] = {a.qs_t, a.qs_h, a.qo_t, a.qo_h, a.ks_t, a.ks_h, a.ko_t, a.ko_h};
    const void* pt[4] = {a.q, a.q_out, a.k, a.k_out};
    for (int i = 0; i < (a.Hkv ? 8 : 4); ++i)
      if (st[i] % v) return false;
    for (int i = 0; i < (a.Hkv ? 4 : 2); ++i)
      if (reinterpret_cast<uintptr_t>(pt[i]) % (static_cast<uintptr_t>(v) * es)) return false;
    return true;
  };
  while (vec > 1 && !fits(vec)) vec /= 2;
  if (vec >= 4 && (reinterpret_cast<uintptr_t>(a.cos_t) % 16 || reinterpret_cast<uintptr_t>(a.sin_t) % 16))
    vec = 2;
  // about 8 warps for each scheduler before the heads of a token share a warp
  const int heads = a.Hq + a.Hkv;
  const int slots = a.half / vec, side = slots >= 32 ? 1 : 32 / slots;
  const long long want = 152ll * 32;
  int blocks = static_cast<int>((want + a.T - 1) / a.T);
  const int most = (heads + side - 1) / side;
  blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
  blocks = blocks > 65535 ? 65535 : blocks;   // gridDim.y
  a.heads_per_block = ((heads + blocks - 1) / blocks + side - 1) / side * side;
  blocks = (heads + a.heads_per_block - 1) / a.heads_per_block;
  switch (p.dtype) {
    case QPKV_DTYPE_BF16: return pick<__nv_bfloat16>(a, vec, blocks, stream);
    case QPKV_DTYPE_F16: return pick<__half>(a, vec, blocks, stream);
    default: return pick<float>(a, vec, blocks, stream);
  }
}

}  // namespace qpkv
