// Append to a paged cache in 8 bits with one scale per (page, kv head)
// ("KvQuantSparseFlashAttention" README, 参数说明 rows key / block_table:
// PA_BSND pages; the scale takes the place of the per-token ones).
//
// A piece is what one call adds to one page of one sequence: tokens at
// positions [p0, p0 + n), o0 = p0 % ps tokens of the page being there
// already.  Per kv head, K and V each:
//   amax = max |x| over the piece,   s_new = amax / QMAX          (o0 = 0)
//                                    s = max(s_old, amax / QMAX)  (o0 > 0)
//   code = RNE(x / s), and when s > s_old the o0 codes that are there become
//   RNE((code * s_old) / s).
// QMAX = 448 (E4M3) or 127 (INT8); divisions are IEEE float32, products are
// rounded to float32, s = 0 gives zero codes.
//
// HBM-bound: 2 bytes in and 1 out per element and tensor.  Pieces are found
// without a plan: sequence b owns work items [floor(cu[b-1] / ps) + 2 b, ...),
// since n tokens touch at most floor(n / ps) + 2 pages, so a block finds its
// sequence by a binary search and items past a sequence's last piece return.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace qpkv {
namespace {

constexpr int kVecs = 8;   // 16-byte vectors of a piece that a thread holds

struct WriteArgs {
  int B, T, H, ps, num_pages, bt_stride;
  const int32_t *cu, *start, *bt;
  const void *k, *v;
  long long ks_t, ks_h, vs_t, vs_h;    // elements
  uint8_t *k_pool, *v_pool;
  long long page_stride, tok_stride, head_stride;   // bytes
  float *k_scale, *v_scale;            // [P, H]
  int* err;
  int tg;                              // threads of one (piece, head)
};

template <typename E>
__device__ __forceinline__ float2 pair_f32(uint32_t w) {
  if constexpr (std::is_same<E, __half>::value) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}

template <bool kInt8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (kInt8) {
    const int x = max(-127, min(127, __float2int_rn(a))), y = max(-127, min(127, __float2int_rn(b)));
    const int z = max(-127, min(127, __float2int_rn(c))), w = max(-127, min(127, __float2int_rn(d)));
    return (x & 0xFF) | (y & 0xFF) << 8 | (z & 0xFF) << 16 | static_cast<uint32_t>(w & 0xFF) << 24;
  } else {
    return static_cast<uint32_t>(f32x2_to_e4m3x2(b, a)) | static_cast<uint32_t>(f32x2_to_e4m3x2(d, c)) << 16;
  }
}

template <bool kInt8>
__device__ __forceinline__ float4 decode4(uint32_t w) {
  if constexpr (kInt8) {
    return make_float4(static_cast<float>(static_cast<int8_t>(w)), static_cast<float>(static_cast<int8_t>(w >> 8)),
                       static_cast<float>(static_cast<int8_t>(w >> 16)), static_cast<float>(static_cast<int8_t>(w >> 24)));
  } else {
    const float2 a = e4m3x2_to_f32x2(static_cast<uint16_t>(w)), b = e4m3x2_to_f32x2(static_cast<uint16_t>(w >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

template <typename E, int D, bool kInt8>
__global__ void __launch_bounds__(1024) write_page8_kernel(const WriteArgs a) {
  constexpr int VR = D / 8;             // 16-byte vectors of a row
  constexpr float kMax = kInt8 ? 127.f : 448.f;
  __shared__ float s_max[32];
  griddep_wait();
  griddep_launch_dependents();
  // the sequence of this work item: the last b with floor(cu[b-1] / ps) + 2 b <= item
  const int item = blockIdx.x, ps = a.ps;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu + mid - 1) / ps + 2 * mid <= item) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  const int t0 = seq_begin(a.cu, b), t1 = __ldg(a.cu + b);
  const int start = a.start != nullptr ? __ldg(a.start + b) : 0;
  const int nth = item - (t0 / ps + 2 * b);             // which page of the sequence's new tokens
  if (t0 < 0 || t1 < t0 || t1 > a.T || start < 0 || nth < 0) {
    if (threadIdx.x == 0 && (t1 < t0 || t1 > a.T || start < 0)) report_error(a.err, kDevErrBadLength);
    return;
  }
  const long long page_no = static_cast<long long>(start / ps) + nth;
  const long long p0 = nth == 0 ? start : page_no * ps;
  const long long p_end = static_cast<long long>(start) + (t1 - t0);
  if (p0 >= p_end) return;
  const int o0 = static_cast<int>(p0 - page_no * ps);
  const int n = static_cast<int>(min(static_cast<long long>(ps - o0), p_end - p0));
  if (page_no >= a.bt_stride) {
    if (threadIdx.x == 0) report_error(a.err, kDevErrBadLength);
    return;
  }
  const int page = __ldg(a.bt + static_cast<size_t>(b) * a.bt_stride + page_no);
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0) report_error(a.err, kDevErrBadPage);
    return;
  }
  const int groups = blockDim.x / a.tg;                 // heads side by side in this block
  const int grp = threadIdx.x / a.tg, th = threadIdx.x - grp * a.tg;
  const int h = blockIdx.y * groups + grp;
  const bool live = h < a.H;
  const bool is_v = blockIdx.z != 0;
  const long long st = is_v ? a.vs_t : a.ks_t;
  const E* src = static_cast<const E*>(is_v ? a.v : a.k) + (t0 + (p0 - start)) * st +
                 static_cast<long long>(h) * (is_v ? a.vs_h : a.ks_h);
  uint8_t* dst = (is_v ? a.v_pool : a.k_pool) + page * a.page_stride + static_cast<long long>(h) * a.head_stride;
  float* scale_at = (is_v ? a.v_scale : a.k_scale) + static_cast<size_t>(page) * a.H + h;
  const int vecs = live ? n * VR : 0;

  uint4 x[kVecs];
  float amax = 0.f;
  auto top = [&](const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair_f32<E>(w[i]);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  };
  auto load = [&](int i) { return __ldg(reinterpret_cast<const uint4*>(src + (i / VR) * st + (i % VR) * 8)); };
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = th + j * a.tg;
    x[j] = i < vecs ? load(i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) top(x[j]);
  for (int i = th + kVecs * a.tg; i < vecs; i += a.tg) top(load(i));   // pages beyond the registers
  amax = warp_max(amax);
  if (a.tg > 32) {   // the same for all threads of the block
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = grp * (a.tg >> 5); w < (grp + 1) * (a.tg >> 5); ++w) amax = fmaxf(amax, s_max[w]);
  }
  if (!live) return;
  float s = __fdiv_rn(amax, kMax);
  if (o0 > 0) {
    const float was = *scale_at;
    if (s > was) {
      // the tokens that are there, in units of the new scale
      for (int i = th; i < o0 * (D / 4); i += a.tg) {
        uint32_t* at = reinterpret_cast<uint32_t*>(dst + (i / (D / 4)) * a.tok_stride + (i % (D / 4)) * 4);
        const float4 v = decode4<kInt8>(*at);
        *at = encode4<kInt8>(__fdiv_rn(__fmul_rn(v.x, was), s), __fdiv_rn(__fmul_rn(v.y, was), s),
                             __fdiv_rn(__fmul_rn(v.z, was), s), __fdiv_rn(__fmul_rn(v.w, was), s));
      }
    } else {
      s = was;
    }
    // every thread of the group has read the old scale before it is replaced
    if (a.tg > 32) {
      named_barrier(1 + grp, a.tg);
    } else {
      __syncwarp();
    }
  }
  if (th == 0) *scale_at = s;
  auto put = [&](int i, const uint4& r) {
    uint2 code = make_uint2(0, 0);
    if (s > 0.f) {
      const float2 f0 = pair_f32<E>(r.x), f1 = pair_f32<E>(r.y), f2 = pair_f32<E>(r.z), f3 = pair_f32<E>(r.w);
      code.x = encode4<kInt8>(__fdiv_rn(f0.x, s), __fdiv_rn(f0.y, s), __fdiv_rn(f1.x, s), __fdiv_rn(f1.y, s));
      code.y = encode4<kInt8>(__fdiv_rn(f2.x, s), __fdiv_rn(f2.y, s), __fdiv_rn(f3.x, s), __fdiv_rn(f3.y, s));
    }
    *reinterpret_cast<uint2*>(dst + (o0 + i / VR) * a.tok_stride + (i % VR) * 8) = code;
  };
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = th + j * a.tg;
    if (i < vecs) put(i, x[j]);
  }
  for (int i = th + kVecs * a.tg; i < vecs; i += a.tg) put(i, load(i));
}

template <typename E, int D, bool kInt8>
cudaError_t go(const WriteArgs& a, cudaStream_t stream) {
  const int threads = a.tg < 128 ? 128 : a.tg;
  const int groups = threads / a.tg;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T / a.ps + 2 * a.B), static_cast<unsigned>((a.H + groups - 1) / groups), 2);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, write_page8_kernel<E, D, kInt8>, a);
}

template <typename E>
cudaError_t pick(const WriteArgs& a, int D, bool int8, cudaStream_t s) {
  if (D == 64) return int8 ? go<E, 64, true>(a, s) : go<E, 64, false>(a, s);
  return int8 ? go<E, 128, true>(a, s) : go<E, 128, false>(a, s);
}

}  // namespace

cudaError_t launch_write_page8(const qpkv_write_page8_params& p, cudaStream_t stream) {
  WriteArgs a;
  a.B = p.num_seqs;
  a.T = p.num_tokens;
  a.H = p.num_heads_kv;
  a.ps = p.page_size;
  a.num_pages = p.num_pages;
  a.bt_stride = p.bt_stride;
  a.cu = p.cu_seqlens_q;
  a.start = p.start_pos;
  a.bt = p.block_table;
  a.k = p.k;
  a.v = p.v;
  a.ks_t = p.k_stride_t, a.ks_h = p.k_stride_h, a.vs_t = p.v_stride_t, a.vs_h = p.v_stride_h;
  a.k_pool = static_cast<uint8_t*>(p.k_pool);
  a.v_pool = static_cast<uint8_t*>(p.v_pool);
  a.page_stride = static_cast<long long>(p.page_size) * p.num_heads_kv * p.head_dim;
  const bool hnd = p.kv_layout == QPKV_KV_LAYOUT_HND;
  a.tok_stride = hnd ? p.head_dim : static_cast<long long>(p.num_heads_kv) * p.head_dim;
  a.head_stride = hnd ? static_cast<long long>(p.page_size) * p.head_dim : p.head_dim;
  a.k_scale = p.k_scale;
  a.v_scale = p.v_scale;
  a.err = p.error_word;
  // threads of a (piece, head): the power of two that holds a full page in
  // kVecs vectors a thread, between a warp and a block of 1024
  int tg = 32;
  while (tg < 1024 && tg * kVecs < p.page_size * p.head_dim / 8) tg *= 2;
  a.tg = tg;
  const bool int8 = p.format == QPKV_FORMAT_INT8;
  return p.dtype == QPKV_DTYPE_F16 ? pick<__half>(a, p.head_dim, int8, stream)
                                   : pick<__nv_bfloat16>(a, p.head_dim, int8, stream);
}

}  // namespace qpkv
