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
// HBM-bound: 2 bytes in and 1 out per element and tensor, if the quantiser is
// kept short: the IEEE division is what fixes the codes, but x (1 / s) times
// 1 - 2^-21 and 1 + 2^-21 lies on both sides of it, so where both give one code
// that is the division's (rounding is monotonic).  A thread's words of four
// codes where they differ (~2 %, many of them exact ties) are noted and done by
// division afterwards.  Neighbouring blocks take neighbouring heads of a page,
// so that rows are read whole.  Pieces are found
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
  int hblocks, rounds;                 // blocks of a piece's heads, heads one after another in each
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

// Codes of four values under a scale s with lo / hi = (1 -+ 2^-21) / s; *same:
// they are those of the IEEE quotients.
template <bool kInt8>
__device__ __forceinline__ uint32_t encode4_fast(float2 a, float2 b, float lo, float hi, bool* same) {
  const uint64_t x0 = f32x2_pack(a.x, a.y), x1 = f32x2_pack(b.x, b.y);
  const uint64_t lo2 = f32x2_pack(lo, lo), hi2 = f32x2_pack(hi, hi);
  if constexpr (kInt8) {
    // + 1.5 * 2^23 rounds to the nearest integer (ties to even) into the low bits
    const uint64_t magic = f32x2_pack(12582912.f, 12582912.f);
    const uint64_t l0 = f32x2_fma(x0, lo2, magic), l1 = f32x2_fma(x1, lo2, magic);
    const uint64_t h0 = f32x2_fma(x0, hi2, magic), h1 = f32x2_fma(x1, hi2, magic);
    *same = l0 == h0 && l1 == h1;
    const uint32_t c0 = __byte_perm(static_cast<uint32_t>(l0), static_cast<uint32_t>(l0 >> 32), 0x0040);
    const uint32_t c1 = __byte_perm(static_cast<uint32_t>(l1), static_cast<uint32_t>(l1 >> 32), 0x0040);
    return __byte_perm(c0, c1, 0x5410);
  } else {
    const uint64_t zero = f32x2_pack(-0.f, -0.f);   // x + -0 is x, signs of zero too
    const float2 l0 = f32x2_unpack(f32x2_fma(x0, lo2, zero)), l1 = f32x2_unpack(f32x2_fma(x1, lo2, zero));
    const float2 h0 = f32x2_unpack(f32x2_fma(x0, hi2, zero)), h1 = f32x2_unpack(f32x2_fma(x1, hi2, zero));
    const uint32_t l = encode4<false>(l0.x, l0.y, l1.x, l1.y);
    *same = l == encode4<false>(h0.x, h0.y, h1.x, h1.y);
    return l;
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

template <typename E, int D, bool kInt8, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) write_page8_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int VR = D / 8;             // 16-byte vectors of a row
  constexpr float kMax = kInt8 ? 127.f : 448.f;
  __shared__ float s_max[2][32];        // by round: one barrier a round is enough
  griddep_wait();
  griddep_launch_dependents();
  // blocks of a page's heads lie side by side, K before V
  const int hblocks = a.hblocks, which = blockIdx.x / hblocks, hblock = blockIdx.x - which * hblocks;
  const bool is_v = which & 1;
  // the sequence of this work item: the last b with floor(cu[b-1] / ps) + 2 b <= item
  const int item = which >> 1, ps = a.ps;
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
    // a start of -1 is a refused request: its tokens have no place, and that has been reported
    if (threadIdx.x == 0 && (t1 < t0 || t1 > a.T || start < -1)) report_error(a.err, kDevErrBadLength);
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
  const int h0 = hblock * groups * a.rounds + grp;
  const long long st = is_v ? a.vs_t : a.ks_t, sh = is_v ? a.vs_h : a.ks_h;
  const E* src0 = static_cast<const E*>(is_v ? a.v : a.k) + (t0 + (p0 - start)) * st;
  uint8_t* pool = (is_v ? a.v_pool : a.k_pool) + page * a.page_stride + o0 * a.tok_stride;
  float* scales = (is_v ? a.v_scale : a.k_scale) + static_cast<size_t>(page) * a.H;
  // tg is a multiple of VR: a thread's vectors lie rows_per rows apart in one column
  const int row0 = th / VR, rows_per = a.tg / VR;
  src0 += row0 * st + (th % VR) * 8;
  pool += row0 * a.tok_stride + (th % VR) * 8;
  const long long src_step = rows_per * st, dst_step = rows_per * a.tok_stride;
  auto load = [&](int h, int j) {
    return __ldg(reinterpret_cast<const uint4*>(src0 + h * sh + j * src_step));
  };
  auto fill = [&](int h, uint4 (&x)[kVecs]) {
    const E* p = src0 + h * sh;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      x[j] = make_uint4(0, 0, 0, 0);
      if (h < a.H && row0 + j * rows_per < n) x[j] = __ldg(reinterpret_cast<const uint4*>(p));
      p += src_step;
    }
  };
  uint4 x[kVecs], next[kVecs];
  fill(h0, x);
#pragma unroll 1
  for (int round = 0; round < a.rounds; ++round) {
    const int h = h0 + round * groups;
    const bool live = h < a.H;
    if (round + 1 < a.rounds) fill(h + groups, next);
    const int rows = live ? n : 0;
    // magnitudes of 16-bit floats are ordered like their bits
    uint32_t top = 0;
    auto take = [&](const uint4& r) {
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu),
                                   __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu)));
    };
#pragma unroll
    for (int j = 0; j < kVecs; ++j) take(x[j]);
    for (int j = kVecs; row0 + j * rows_per < rows; ++j) take(load(h, j));   // pages beyond the registers
    const float2 two = pair_f32<E>(top);
    float amax = warp_max(fmaxf(two.x, two.y));
    if (a.tg > 32) {   // the same for all threads of the block
      float* mx = s_max[round & 1];
      if ((threadIdx.x & 31) == 0) mx[threadIdx.x >> 5] = amax;
      __syncthreads();
      for (int w = grp * (a.tg >> 5); w < (grp + 1) * (a.tg >> 5); ++w) amax = fmaxf(amax, mx[w]);
    }
    if (live) {
      uint8_t* dst = pool + h * a.head_stride;
      float s = __fdiv_rn(amax, kMax);
      if (o0 > 0) {
        const float was = scales[h];
        if (s > was) {
          // the tokens that are there, in units of the new scale
          uint8_t* first = dst - (o0 + row0) * a.tok_stride - (th % VR) * 8;
          for (int i = th; i < o0 * (D / 4); i += a.tg) {
            uint32_t* at = reinterpret_cast<uint32_t*>(first + (i / (D / 4)) * a.tok_stride + (i % (D / 4)) * 4);
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
      if (th == 0) scales[h] = s;
      auto at = [&](int j) { return reinterpret_cast<uint2*>(dst + j * dst_step); };
      auto divide = [&](uint32_t r0, uint32_t r1) {
        const float2 f0 = pair_f32<E>(r0), f1 = pair_f32<E>(r1);
        return encode4<kInt8>(__fdiv_rn(f0.x, s), __fdiv_rn(f0.y, s), __fdiv_rn(f1.x, s), __fdiv_rn(f1.y, s));
      };
      const float inv = 1.f / s, lo_inv = inv * (1.f - 0x1p-21f), hi_inv = inv * (1.f + 0x1p-21f);
      const bool fast = s > 0x1p-100f && s < 0x1p100f;    // neither 1 / s nor x / s leaves float32's range
      uint32_t again = 0;                                 // words of codes to be done by division
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        if (row0 + j * rows_per < rows) {
          bool same0, same1;
          uint2 code;
          code.x = encode4_fast<kInt8>(pair_f32<E>(x[j].x), pair_f32<E>(x[j].y), lo_inv, hi_inv, &same0);
          code.y = encode4_fast<kInt8>(pair_f32<E>(x[j].z), pair_f32<E>(x[j].w), lo_inv, hi_inv, &same1);
          *at(j) = s > 0.f ? code : make_uint2(0, 0);
          if (!(same0 && fast)) again |= 1u << 2 * j;
          if (!(same1 && fast)) again |= 2u << 2 * j;
        }
      }
      if (!(s > 0.f)) again = 0;
      while (again) {
        const int k = __ffs(again) - 1, j = k >> 1;
        again &= again - 1;
        // its two words of values, from L1 or L2
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(src0 + h * sh + j * src_step) + (k & 1));
        reinterpret_cast<uint32_t*>(at(j))[k & 1] = divide(r.x, r.y);
      }
      for (int j = kVecs; row0 + j * rows_per < rows; ++j) {
        const uint4 r = load(h, j);
        *at(j) = s > 0.f ? make_uint2(divide(r.x, r.y), divide(r.z, r.w)) : make_uint2(0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) x[j] = next[j];
  }
}

template <typename E, int D, bool kInt8>
cudaError_t go(const WriteArgs& a, cudaStream_t stream) {
  const int threads = a.tg < 128 ? 128 : a.tg;
  const int groups = threads / a.tg;
  WriteArgs w = a;
  // up to eight heads one after another, the next one's loads ahead of the work
  // on this one's, while that leaves every SM eight blocks (8 prompts of 32
  // heads: 177 us with one, 112 with two, 97 with eight; 93 now, with the redo by words)
  const long long pieces = (a.T / a.ps + 2ll * a.B) * 2;
  w.rounds = 8;
  while (w.rounds > 1 && (a.H < groups * w.rounds || pieces * (a.H / (groups * w.rounds)) < 152 * 8)) w.rounds /= 2;
  w.hblocks = (a.H + groups * w.rounds - 1) / (groups * w.rounds);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pieces * w.hblocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (threads == 128) return cudaLaunchKernelEx(&cfg, write_page8_kernel<E, D, kInt8, 128>, w);
  return cudaLaunchKernelEx(&cfg, write_page8_kernel<E, D, kInt8, 512>, w);
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
  // kVecs vectors a thread, between a warp and a block of 512
  int tg = 32;
  while (tg < 512 && tg * kVecs < p.page_size * p.head_dim / 8) tg *= 2;
  a.tg = tg;
  const bool int8 = p.format == QPKV_FORMAT_INT8;
  return p.dtype == QPKV_DTYPE_F16 ? pick<__half>(a, p.head_dim, int8, stream)
                                   : pick<__nv_bfloat16>(a, p.head_dim, int8, stream);
}

}  // namespace qpkv
