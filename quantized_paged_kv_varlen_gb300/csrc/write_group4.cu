// Append to the paged cache in 4 bits, with the rotation of k and q on the way
// ("[Feature] Sage Attention Support Varlen & write kv cache BF16/FP16",
// Description item 1: RoPE fused into the cache write), and read it back.
//
//   y = rotated x (pairs i, i + R/2; products and sums rounded one by one), / mul
//   s = E4M3(min(448, amax / 6)) of 16 channels,  code = E2M1(y / s)
// and per page and channel the bounds floor(min / u), ceil(max / u) of the keys
// as they read back.
//
// Divisions are IEEE float32 by definition.  y / s is done as q = y r, q' = q + (y -
// q s) r with r near 1 / s (Markstein's correction; y - q s is exact in one fma):
// q' gives the code of the rounded quotient.  s has 4 significant bits and the
// codes' midpoints m at most 3, so m s is a float32, at which q' is exactly m; any
// other y is off by a step of its own or more, which takes y / s further from m
// than 1.07 half steps of float32, and q' is good to half a step and 2^-22 of one.
// amax / 6 the same, with the midpoints of E4M3 (5 bits).
//
// HBM-bound: 2 bytes in and 9/16 out per element.  A thread takes 16 channels of
// a token: one scale, 8 bytes of codes.  What one call adds to a page of a
// sequence is a piece; a block takes a piece's K or V for some heads, 16 tokens
// (32 with D = 64) at a time, so that bounds are made where the codes are.  A
// page's table rows come from L1 after its first head.  Pieces are found without
// a plan, as in the page-scaled write: sequence b owns work items [floor(cu[b-1] /
// ps) + 2 b, ...).  Blocks behind those of the pieces rotate q, with the table
// values of a token in registers while they walk the heads.
#include <type_traits>

#include "common.cuh"
#include "group4.cuh"
#include "internal.h"

namespace qpkv {
namespace {

constexpr int kThreads = 128;

struct WriteArgs {
  int B, T, Hq, H, ps, num_pages, bt_stride, half, max_pos;
  const int32_t *cu, *start, *bt;
  const void *k, *v, *q;
  void* q_out;
  long long ks_t, ks_h, vs_t, vs_h, qs_t, qs_h, qo_t, qo_h;   // elements
  const float *cos_t, *sin_t, *k_mul, *v_mul;
  uint8_t *k_pool, *v_pool;
  int8_t* bounds;
  float* bscale;
  int* err;
  int k_wide, v_wide;        // rows of 16 channels lie on 32 bytes
  int hblocks, heads;        // blocks of a piece's heads, heads of each
  int kv_blocks;             // the first blocks; the others rotate q
  int q_splits, q_heads;     // blocks of a token tile's heads, heads of each
};

template <typename E>
__device__ __forceinline__ float2 pair_f32(uint32_t w) {
  if constexpr (std::is_same<E, __half>::value) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <typename E>
__device__ __forceinline__ uint32_t f32_pair(float lo, float hi) {
  if constexpr (std::is_same<E, __half>::value) {
    return f32x2_to_f16x2(hi, lo);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// max(|a|, |b|, |c|) of values of which none or any is NaN: then NaN.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

// 32 bytes by one access where they lie on 32, else by two.
__device__ __forceinline__ void load32(const void* p, bool wide, uint4& a, uint4& b) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = __ldg(static_cast<const uint4*>(p));
    b = __ldg(static_cast<const uint4*>(p) + 1);
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// 16 channels -> codes and scale.
__device__ __forceinline__ uint2 encode16(const float (&x)[16], uint32_t* scale) {
  const float top = absmax3(absmax3(absmax3(x[0], x[1], x[2]), absmax3(x[3], x[4], x[5]), absmax3(x[6], x[7], x[8])),
                            absmax3(x[9], x[10], x[11]), absmax3(absmax3(x[12], x[13], x[14]), x[15], 0.f));
  if (!(top < INFINITY)) {
    *scale = 0x7Fu;
    return make_uint2(0, 0);
  }
  constexpr float sixth = 1.f / 6.f;
  const float t0 = top * sixth;
  const uint32_t code = f32x2_to_e4m3x2(0.f, fmaf(fmaf(-t0, 6.f, top), sixth, t0)) & 0xFFu;
  *scale = code;
  const float s = e4m3_to_f32(static_cast<uint8_t>(code));
  if (s == 0.f) return make_uint2(0, 0);
  float r;      // good to 2^-23: the correction makes up for it
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  float y[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = x[i] * r;
    y[i >> 3][i & 7] = fmaf(fmaf(-q, s, x[i]), r, q);
  }
  return make_uint2(f32x8_to_e2m1(y[0]), f32x8_to_e2m1(y[1]));
}

__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename E, int D>
__device__ __forceinline__ void rotate_q(const WriteArgs& a, int block) {
  constexpr int TPR = D / 16, R = kThreads / TPR;
  const int tile = block / a.q_splits, split = block - tile * a.q_splits;
  const int tok0 = tile * R, c = threadIdx.x % TPR, tok = tok0 + threadIdx.x / TPR;
  int b = warp_last_at_most(a.B, tok0, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1)); });
  if (tok >= a.T) return;
  while (b < a.B && __ldg(a.cu + b) <= tok) ++b;
  if (b >= a.B) return;                                  // behind the last sequence
  const int t0 = seq_begin(a.cu, b), t1 = __ldg(a.cu + b);
  const int start = a.start != nullptr ? __ldg(a.start + b) : 0;
  if (t0 < 0 || t0 > tok || t1 > a.T || start < 0) return;    // reported with the pieces
  if (start + static_cast<long long>(t1 - t0) > a.max_pos) return;
  const size_t pos = static_cast<size_t>(start) + (tok - t0);
  const bool turns = 8 * c < a.half;
  float cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos_t + pos * a.half + 8 * c + i));
      const float4 y = __ldg(reinterpret_cast<const float4*>(a.sin_t + pos * a.half + 8 * c + i));
      cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
      sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
    }
  }
  const int h0 = split * a.q_heads, h1 = min(a.Hq, h0 + a.q_heads);
  const E* src = static_cast<const E*>(a.q) + tok * a.qs_t;
  E* dst = static_cast<E*>(a.q_out) + tok * a.qo_t;
  if (turns) {
    constexpr int kAhead = 4;     // heads whose loads are in flight together
    for (int h = h0; h < h1; h += kAhead) {
      uint4 u[kAhead], w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (h + j < h1) {
          const E* p = src + (h + j) * a.qs_h + 8 * c;
          u[j] = *reinterpret_cast<const uint4*>(p);
          w[j] = *reinterpret_cast<const uint4*>(p + a.half);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (h + j < h1) {
          const uint32_t uu[4] = {u[j].x, u[j].y, u[j].z, u[j].w}, ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
          uint32_t x[4], y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 p = pair_f32<E>(uu[i]), r = pair_f32<E>(ww[i]);
            x[i] = f32_pair<E>(__fsub_rn(__fmul_rn(p.x, cs[2 * i]), __fmul_rn(r.x, sn[2 * i])),
                               __fsub_rn(__fmul_rn(p.y, cs[2 * i + 1]), __fmul_rn(r.y, sn[2 * i + 1])));
            y[i] = f32_pair<E>(__fadd_rn(__fmul_rn(r.x, cs[2 * i]), __fmul_rn(p.x, sn[2 * i])),
                               __fadd_rn(__fmul_rn(r.y, cs[2 * i + 1]), __fmul_rn(p.y, sn[2 * i + 1])));
          }
          E* o = dst + (h + j) * a.qo_h + 8 * c;
          *reinterpret_cast<uint4*>(o) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(o + a.half) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  }
  // elements behind the rotated ones
  for (int x = a.half / 4 + c; x < D / 8; x += TPR)
    for (int h = h0; h < h1; ++h)
      *reinterpret_cast<uint4*>(dst + h * a.qo_h + 8 * x) = *reinterpret_cast<const uint4*>(src + h * a.qs_h + 8 * x);
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 6) write_group4_kernel(const __grid_constant__ WriteArgs a) {
  using L = Group4<D>;
  constexpr int TPR = D / 16;                 // threads of a token
  constexpr int R = kThreads / TPR;           // tokens of a round
  __shared__ uint32_t s_mn[4][D / 2], s_mx[4][D / 2];
  __shared__ uint32_t s_top[4];
  griddep_wait();
  griddep_launch_dependents();
  const int block_no = blockIdx.x;
  if (block_no >= a.kv_blocks) {
    rotate_q<E, D>(a, block_no - a.kv_blocks);
    return;
  }
  // blocks of a page's heads lie side by side, K before V
  const int which = block_no / a.hblocks, hblock = block_no - which * a.hblocks;
  const bool is_v = which & 1;
  const int item = which >> 1, ps = a.ps, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = warp_last_at_most(a.B, item, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1) / ps) + 2ll * m; });
  const int t0 = seq_begin(a.cu, b), t1 = __ldg(a.cu + b);
  const int start = a.start != nullptr ? __ldg(a.start + b) : 0;
  const int nth = item - (t0 / ps + 2 * b);             // which page of the sequence's new tokens
  if (t0 < 0 || t1 < t0 || t1 > a.T || start < 0 || nth < 0) {
    if (tid == 0 && (t1 < t0 || t1 > a.T || start < -1)) report_error(a.err, kDevErrBadLength);
    return;
  }
  const long long p_end = static_cast<long long>(start) + (t1 - t0);
  if (a.half > 0 && p_end > a.max_pos) {
    if (tid == 0 && t1 > t0) report_error(a.err, kDevErrBadLength);
    return;
  }
  const long long page_no = static_cast<long long>(start / ps) + nth;
  const long long p0 = nth == 0 ? start : page_no * ps;
  if (p0 >= p_end) return;
  const int o0 = static_cast<int>(p0 - page_no * ps);
  const int end = static_cast<int>(min(static_cast<long long>(ps), p_end - page_no * ps));   // tokens of the page
  if (page_no >= a.bt_stride) {
    if (tid == 0) report_error(a.err, kDevErrBadLength);
    return;
  }
  const int page = __ldg(a.bt + static_cast<size_t>(b) * a.bt_stride + page_no);
  if (page < 0 || page >= a.num_pages) {
    if (tid == 0) report_error(a.err, kDevErrBadPage);
    return;
  }
  const int g = tid % TPR, row = tid / TPR;
  const bool bounds = !is_v && a.bounds != nullptr, turns = !is_v && 16 * g < 2 * a.half;
  const long long st = is_v ? a.vs_t : a.ks_t, sh = is_v ? a.vs_h : a.ks_h;
  // of the token at slot 0 of the page (which may lie before the first new one)
  const E* src0 = static_cast<const E*>(is_v ? a.v : a.k) + 16 * g;
  const long long tok0 = t0 + (page_no * ps - start);
  const bool first_half = 16 * g < a.half;
  const int partner = (lane & ~(TPR - 1)) | (turns ? (first_half ? g + a.half / 16 : g - a.half / 16) : g);
  const int i0 = first_half ? 16 * g : 16 * g - a.half;      // of its pairs
  const int from = bounds ? 0 : o0 / R * R;
  const float* muls = is_v ? a.v_mul : a.k_mul;
  const int h0 = hblock * a.heads, h1 = min(a.H, h0 + a.heads);
  // a round's inputs, loaded while the one before is worked on: new tokens' values,
  // kept tokens' codes and scales
  const bool wide = is_v ? a.v_wide : a.k_wide;
  struct In {
    uint4 x0, x1;
    uint2 codes;
    uint32_t scale;
  };
  const size_t head_bytes = static_cast<size_t>(ps / 16) * L::kBlock;
  uint8_t* pool = (is_v ? a.v_pool : a.k_pool) + (static_cast<size_t>(page) * a.H + h0) * head_bytes;
  // slot r + row lies in block r / 16 (and one on, for the upper half of 32)
  const int codes_off = (row >> 4) * L::kBlock + (row & 15) * L::kRow + 8 * g;
  const int scale_off = (row >> 4) * L::kBlock + L::kScaleAt + (row & 15) * L::kScales + g;
  const E* src_row = src0 + (tok0 + from + row) * st;      // of the round that is loaded next
  auto load = [&](const E* src, const uint8_t* base, int r) {
    In in = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint2(0, 0), 0};
    const int slot = r + row;
    if (slot >= o0 && slot < end) {
      load32(src, wide, in.x0, in.x1);
    } else if (bounds && slot < o0) {
      const uint8_t* block = base + (r >> 4) * L::kBlock;
      in.codes = *reinterpret_cast<const uint2*>(block + codes_off);
      in.scale = block[scale_off];
    }
    return in;
  };
  const E* src_h = src_row + h0 * sh;
  In in = load(src_h, pool, from);
  for (int h = h0; h < h1; ++h, pool += head_bytes) {
    const float mul = muls != nullptr ? __ldg(muls + h) : 1.f;
    uint32_t mn[8], mx[8], nan = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mn[i] = 0x7C007C00u, mx[i] = 0xFC00FC00u;
    const E* src = src_h;
    src_h += sh;
    for (int r = from; r < end; r += R) {
      const int slot = r + row;
      const bool fresh = slot >= o0 && slot < end, kept = bounds && slot < o0;
      const In now = in;
      src += R * st;
      if (r + R < end) in = load(src, pool, r + R);
      else if (h + 1 < h1) in = load(src_h, pool + head_bytes, from);
      uint2 codes = now.codes;
      uint32_t scale = now.scale;
      const uint32_t w[8] = {now.x0.x, now.x0.y, now.x0.z, now.x0.w, now.x1.x, now.x1.y, now.x1.z, now.x1.w};
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = pair_f32<E>(w[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
      if (!is_v && a.half > 0) {    // the same in all threads
        const size_t at = static_cast<size_t>(page_no * ps + (fresh ? slot : o0)) * a.half + i0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
          if (turns) {
            c = __ldg(reinterpret_cast<const float4*>(a.cos_t + at + 2 * i));
            s = __ldg(reinterpret_cast<const float4*>(a.sin_t + at + 2 * i));
          }
          const float2 u = pair_f32<E>(__shfl_sync(0xffffffffu, w[i], partner));
          const float2 v = pair_f32<E>(__shfl_sync(0xffffffffu, w[i + 1], partner));
          if (turns) {
            // a - b is a + (-b)
            const float sg = first_half ? -1.f : 1.f;
            x[2 * i] = __fadd_rn(__fmul_rn(x[2 * i], c.x), sg * __fmul_rn(u.x, s.x));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], c.y), sg * __fmul_rn(u.y, s.y));
            x[2 * i + 2] = __fadd_rn(__fmul_rn(x[2 * i + 2], c.z), sg * __fmul_rn(v.x, s.z));
            x[2 * i + 3] = __fadd_rn(__fmul_rn(x[2 * i + 3], c.w), sg * __fmul_rn(v.y, s.w));
          }
        }
      }
      if (muls != nullptr) {
        if (mul > 0x1p-100f && mul < 0x1p100f) {
          // x / mul, rounded: two of Markstein's corrections, as mul has 24 significant bits.
          // (Where they underflow the group is zero beside its scale's smallest step.)
          const float r = __frcp_rn(mul);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float q0 = x[i] * r, q1 = fmaf(fmaf(-q0, mul, x[i]), r, q0);
            x[i] = fmaf(fmaf(-q1, mul, x[i]), r, q1);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], mul);
        }
      }
      if (fresh) {
        codes = encode16(x, &scale);
        uint8_t* block = pool + (r >> 4) * L::kBlock;
        *reinterpret_cast<uint2*>(block + codes_off) = codes;
        block[scale_off] = static_cast<uint8_t>(scale);
      }
      if (bounds && (fresh || kept)) {
        if (e4m3_is_nan(scale)) {
          nan = 1;
        } else {
          const uint32_t s2 = e4m3_to_f16x2_both(scale);
          uint32_t f[2][4];
          e2m1x8_to_f16(codes.x, f[0]);
          e2m1x8_to_f16(codes.y, f[1]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t y = f16x2_mul(f[i >> 2][i & 3], s2);
            mn[i] = hmin2(mn[i], y);
            mx[i] = hmax2(mx[i], y);
          }
        }
      }
    }
    if (bounds) {
      nan = __any_sync(0xffffffffu, nan);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) {
          mn[i] = hmin2(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
          mx[i] = hmax2(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
        }
        if (lane < TPR) s_mn[warp][8 * g + i] = mn[i], s_mx[warp][8 * g + i] = mx[i];
      }
      if (lane == 0) s_top[warp] = nan;
      __syncthreads();
      nan = s_top[0] | s_top[1] | s_top[2] | s_top[3];
      // two channels a thread; all warps do the same, so that no sums cross them
      uint32_t top = 0;
      int lo[2][D / 64], hi[2][D / 64];
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const int i = lane + 32 * k;
        const uint32_t l2 = hmin2(hmin2(s_mn[0][i], s_mn[1][i]), hmin2(s_mn[2][i], s_mn[3][i]));
        const uint32_t h2 = hmax2(hmax2(s_mx[0][i], s_mx[1][i]), hmax2(s_mx[2][i], s_mx[3][i]));
        const float2 l = pair_f32<__half>(l2), u = pair_f32<__half>(h2);
        lo[0][k] = static_cast<int>(l.x * 1024.f), lo[1][k] = static_cast<int>(l.y * 1024.f);
        hi[0][k] = static_cast<int>(u.x * 1024.f), hi[1][k] = static_cast<int>(u.y * 1024.f);
#pragma unroll
        for (int x = 0; x < 2; ++x) top = max(top, static_cast<uint32_t>(max(abs(lo[x][k]), abs(hi[x][k]))));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      int e = 0;
      while (top > 127u << e) ++e;      // top < 2^22
      if (warp == 0) {
        const size_t at = static_cast<size_t>(page) * a.H + h;
        uint16_t* out = reinterpret_cast<uint16_t*>(a.bounds + at * 2 * D);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const int l0 = lo[0][k] >> e, l1 = lo[1][k] >> e, u0 = -(-hi[0][k] >> e), u1 = -(-hi[1][k] >> e);
          out[lane + 32 * k] = nan ? 0 : static_cast<uint16_t>((l0 & 0xFF) | (l1 & 0xFF) << 8);
          out[D / 2 + lane + 32 * k] = nan ? 0 : static_cast<uint16_t>((u0 & 0xFF) | (u1 & 0xFF) << 8);
        }
        if (lane == 0) a.bscale[at] = nan ? INFINITY : __uint_as_float(static_cast<uint32_t>(127 - 10 + e) << 23);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- read back

struct ReadArgs {
  int B, T, H, ps, num_pages, bt_stride;
  const int32_t *cu, *start, *bt;
  const uint8_t *k_pool, *v_pool;
  const float *k_mul, *v_mul;
  void *k_out, *v_out;
  int* err;
  int hblocks, heads;
};

// A thread takes 16 channels of a token, a block 16 tokens (32 with D = 64) of
// K or V for some heads: 256-byte rows out.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) read_group4_kernel(const __grid_constant__ ReadArgs a) {
  using L = Group4<D>;
  constexpr int TPR = D / 16, R = kThreads / TPR;
  griddep_wait();
  griddep_launch_dependents();
  const int which = blockIdx.x / a.hblocks, hblock = blockIdx.x - which * a.hblocks;
  const bool is_v = which & 1;
  if ((is_v ? a.v_out : a.k_out) == nullptr) return;
  const int tok0 = (which >> 1) * R, g = threadIdx.x % TPR, tok = tok0 + threadIdx.x / TPR;
  int b = warp_last_at_most(a.B, tok0, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1)); });
  if (tok >= a.T) return;
  while (b < a.B && __ldg(a.cu + b) <= tok) ++b;
  if (b >= a.B) return;
  const int t0 = seq_begin(a.cu, b), t1 = __ldg(a.cu + b);
  const int start = a.start != nullptr ? __ldg(a.start + b) : 0;
  if (t0 < 0 || t0 > tok || t1 > a.T || start < 0) {
    if (start != -1 && g == 0) report_error(a.err, kDevErrBadLength);
    return;
  }
  const long long pos = static_cast<long long>(start) + (tok - t0), page_no = pos / a.ps;
  if (page_no >= a.bt_stride) {
    if (g == 0) report_error(a.err, kDevErrBadLength);
    return;
  }
  const int page = __ldg(a.bt + static_cast<size_t>(b) * a.bt_stride + page_no);
  if (page < 0 || page >= a.num_pages) {
    if (g == 0) report_error(a.err, kDevErrBadPage);
    return;
  }
  const int slot = static_cast<int>(pos - page_no * a.ps), blocks = a.ps / 16;
  const int h0 = hblock * a.heads, h1 = min(a.H, h0 + a.heads);
  const uint8_t* block = (is_v ? a.v_pool : a.k_pool) +
                         ((static_cast<size_t>(page) * a.H + h0) * blocks + (slot >> 4)) * L::kBlock;
  const size_t step = static_cast<size_t>(blocks) * L::kBlock;
  E* out = static_cast<E*>(is_v ? a.v_out : a.k_out) + (static_cast<size_t>(tok) * a.H + h0) * D + 16 * g;
  const float* muls = is_v ? a.v_mul : a.k_mul;
  const bool wide = reinterpret_cast<uintptr_t>(is_v ? a.v_out : a.k_out) % 32 == 0;
#pragma unroll 4
  for (int h = h0; h < h1; ++h, block += step, out += D) {
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(block + (slot & 15) * L::kRow + 8 * g));
    const uint32_t scale = __ldg(block + L::kScaleAt + (slot & 15) * L::kScales + g);
    const float mul = muls != nullptr ? __ldg(muls + h) : 1.f;
    const float s = e4m3_to_f32(static_cast<uint8_t>(scale));
    uint32_t f[2][4], o[8];
    e2m1x8_to_f16(codes.x, f[0]);
    e2m1x8_to_f16(codes.y, f[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = pair_f32<__half>(f[i >> 2][i & 3]);
      o[i] = f32_pair<E>(v.x * s * mul, v.y * s * mul);     // code times scale is exact
    }
    store32(out, wide, o);
  }
}

template <typename K, typename A>
cudaError_t launch(K kernel, long long grid, const A& args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace

cudaError_t launch_write_group4(const qpkv_write_group4_params& p, cudaStream_t stream) {
  WriteArgs a;
  a.B = p.num_seqs, a.T = p.num_tokens, a.Hq = p.q != nullptr ? p.num_heads_q : 0, a.H = p.num_heads_kv;
  a.ps = p.page_size, a.num_pages = p.num_pages, a.bt_stride = p.bt_stride;
  a.half = p.rope_cos != nullptr ? p.rot_dim / 2 : 0;
  a.max_pos = p.rope_max_pos;
  a.cu = p.cu_seqlens_q, a.start = p.start_pos, a.bt = p.block_table;
  a.k = p.k, a.v = p.v, a.q = p.q, a.q_out = p.q_out;
  a.ks_t = p.k_stride_t, a.ks_h = p.k_stride_h, a.vs_t = p.v_stride_t, a.vs_h = p.v_stride_h;
  a.qs_t = p.q_stride_t, a.qs_h = p.q_stride_h, a.qo_t = p.q_out_stride_t, a.qo_h = p.q_out_stride_h;
  a.cos_t = p.rope_cos, a.sin_t = p.rope_sin, a.k_mul = p.k_mul, a.v_mul = p.v_mul;
  a.k_pool = static_cast<uint8_t*>(p.k_pool), a.v_pool = static_cast<uint8_t*>(p.v_pool);
  a.bounds = static_cast<int8_t*>(p.k_bounds), a.bscale = p.bound_scale;
  a.err = p.error_word;
  auto wide = [](const void* x, long long t, long long h) {
    return reinterpret_cast<uintptr_t>(x) % 32 == 0 && t % 16 == 0 && h % 16 == 0;
  };
  a.k_wide = wide(p.k, a.ks_t, a.ks_h), a.v_wide = wide(p.v, a.vs_t, a.vs_h);
  // two heads one after another in a block while every SM keeps eight blocks (8
  // prompts, 18,803 tokens of 8 heads: K and V alone 49 us with one head, 46 with
  // two, 52 with four, whose blocks make two waves); eight of q (all: 79 us)
  const long long pieces = (a.T / a.ps + 2ll * a.B) * 2;
  a.heads = 2;
  while (a.heads > 1 && (a.H < a.heads || pieces * (a.H / a.heads) < 152 * 8)) a.heads /= 2;
  a.hblocks = (a.H + a.heads - 1) / a.heads;
  a.kv_blocks = static_cast<int>(pieces * a.hblocks);
  const int R = kThreads / (p.head_dim / 16), tiles = (a.T + R - 1) / R;
  a.q_heads = 8;
  while (a.q_heads > 1 && (a.Hq < a.q_heads || static_cast<long long>(tiles) * (a.Hq / a.q_heads) < 152 * 4)) a.q_heads /= 2;
  a.q_splits = a.Hq > 0 ? (a.Hq + a.q_heads - 1) / a.q_heads : 0;
  const long long grid = a.kv_blocks + static_cast<long long>(tiles) * a.q_splits;
  const bool f16 = p.dtype == QPKV_DTYPE_F16;
  if (p.head_dim == 64)
    return f16 ? launch(write_group4_kernel<__half, 64>, grid, a, stream) : launch(write_group4_kernel<__nv_bfloat16, 64>, grid, a, stream);
  return f16 ? launch(write_group4_kernel<__half, 128>, grid, a, stream) : launch(write_group4_kernel<__nv_bfloat16, 128>, grid, a, stream);
}

cudaError_t launch_read_group4(const qpkv_read_group4_params& p, cudaStream_t stream) {
  ReadArgs a;
  a.B = p.num_seqs, a.T = p.num_tokens, a.H = p.num_heads_kv, a.ps = p.page_size;
  a.num_pages = p.num_pages, a.bt_stride = p.bt_stride;
  a.cu = p.cu_seqlens_q, a.start = p.start_pos, a.bt = p.block_table;
  a.k_pool = static_cast<const uint8_t*>(p.k_pool), a.v_pool = static_cast<const uint8_t*>(p.v_pool);
  a.k_mul = p.k_mul, a.v_mul = p.v_mul, a.k_out = p.k_out, a.v_out = p.v_out;
  a.err = p.error_word;
  const int R = kThreads / (p.head_dim / 16);
  const long long tiles = 2ll * ((a.T + R - 1) / R);
  a.heads = 8;
  while (a.heads > 1 && (a.H < a.heads || tiles * (a.H / a.heads) < 152 * 8)) a.heads /= 2;
  a.hblocks = (a.H + a.heads - 1) / a.heads;
  const long long grid = tiles * a.hblocks;
  const bool f16 = p.dtype == QPKV_DTYPE_F16;
  if (p.head_dim == 64)
    return f16 ? launch(read_group4_kernel<__half, 64>, grid, a, stream) : launch(read_group4_kernel<__nv_bfloat16, 64>, grid, a, stream);
  return f16 ? launch(read_group4_kernel<__half, 128>, grid, a, stream) : launch(read_group4_kernel<__nv_bfloat16, 128>, grid, a, stream);
}

}  // namespace qpkv
