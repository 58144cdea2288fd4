// What the kernels over the page-scaled 8-bit cache share: their arguments,
// the keys that a query row sees, and small arithmetic.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace qpkv {

// P = 2^(y - m): log2 of the row's largest P when m is set, and the largest
// it may become before m moves.
constexpr float kSetP = 7.0f, kMaxP = 15.0f;
// Value scales below this, zero among them, count as this: values that small
// are zero beside anything a model computes, and the keys of such a page move
// no row's m away from those that count.  P <= 2^kMaxP over it, summed over
// fewer than 2^31 keys, stays in float32.
constexpr float kMinScale = 8.271806e-25f;   // 2^-80
// A cap multiplies the error of tanh_of: up to this one to 2e-5 of a logit at
// most, above it scores would drown in it (0.1 of a logit at a cap of 1e6).
constexpr float kNearCap = 64.f;

struct Page8Args {
  int B, T, Hq, Hkv, G, ps, num_pages, bt_stride, causal, window, hnd;
  int split_rows;          // sequences with more query rows per kv head go in tiles of 128
  float scale_log2;        // softmax scale * log2(e)
  float scale_cap;         // softmax scale / cap
  float cap_log2;          // cap * log2(e), 0: no cap
  int far_cap;             // a cap above kNearCap
  const int32_t *cu, *lens, *bt, *prefix;
  const float *slopes, *ks, *vs;
  const void* q;
  const uint8_t *k, *v;
  void* o;
  float* lse;
  int* err;
};

inline Page8Args page8_args(const qpkv_attend_page8_params& p) {
  Page8Args a;
  a.B = p.num_seqs, a.T = p.num_tokens, a.Hq = p.num_heads_q, a.Hkv = p.num_heads_kv;
  a.G = p.num_heads_q / p.num_heads_kv;
  a.ps = p.page_size, a.num_pages = p.num_pages, a.bt_stride = p.bt_stride;
  a.causal = p.causal ? 1 : 0;
  a.window = p.window;
  const float scale = p.sm_scale;
  a.scale_log2 = scale * kLog2e;
  a.scale_cap = p.logit_cap > 0.f ? scale / p.logit_cap : 0.f;
  a.cap_log2 = p.logit_cap > 0.f ? p.logit_cap * kLog2e : 0.f;
  a.far_cap = p.logit_cap > kNearCap;
  a.hnd = p.kv_layout == QPKV_KV_LAYOUT_HND;
  a.cu = p.cu_seqlens_q, a.lens = p.seqlens_kv, a.bt = p.block_table, a.prefix = p.prefix_lens;
  a.slopes = p.alibi_slopes, a.ks = p.k_scale, a.vs = p.v_scale;
  a.q = p.q;
  a.k = static_cast<const uint8_t*>(p.k_pool), a.v = static_cast<const uint8_t*>(p.v_pool);
  a.o = p.o, a.lse = p.lse, a.err = p.error_word;
  return a;
}

// A pool for TMA: rows of D codes, boxes of `rows` tokens of one head.  NHD:
// coordinates (0, head, page * ps + token); HND: (0, 0, (page * Hkv + head) * ps
// + token).  Rows are 64 or 128 bytes wide and swizzled by as much.
inline bool pool_map(const Page8Args& a, int D, const void* pool, uint32_t rows, CUtensorMap* map) {
  const uint64_t d = static_cast<uint64_t>(D), heads = a.hnd ? 1 : a.Hkv;
  const uint64_t dims[3] = {d, heads, static_cast<uint64_t>(a.num_pages) * a.ps * (a.hnd ? a.Hkv : 1)};
  const uint64_t strides[2] = {d, heads * d};
  const uint32_t box[3] = {static_cast<uint32_t>(D), 1u, rows};
  return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box,
                           D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) == CUDA_SUCCESS;
}

// Query rows [t0, t0 + n) of a sequence and its cached tokens.
struct Rows {
  int t0, n, len, prefix;
};

// Lengths that do not fit the arrays are reported (err may be null) and give
// a sequence without rows, or without keys.
__device__ __forceinline__ Rows rows_of(const Page8Args& a, int b, int* err) {
  Rows r;
  r.t0 = seq_begin(a.cu, b);
  r.n = __ldg(a.cu + b) - r.t0;
  r.len = __ldg(a.lens + b);
  r.prefix = a.prefix != nullptr ? __ldg(a.prefix + b) : 0;
  if (r.n < 0 || r.t0 < 0 || r.t0 + static_cast<long long>(r.n) > a.T) {
    report_error(err, kDevErrBadLength);
    r.n = 0;
  }
  if (r.len < 0 || r.len > static_cast<long long>(a.bt_stride) * a.ps) {
    report_error(err, kDevErrBadLength);
    r.len = 0;
  }
  return r;
}

// Row i sees keys [row_lo, row_hi); both grow with i.  Its position is
// len - n + i (negative for the rows of a prompt longer than its cache).
__device__ __forceinline__ int row_hi(const Page8Args& a, const Rows& r, int i) {
  if (!a.causal) return r.len;
  return min(r.len, max(r.len - r.n + i + 1, r.prefix));
}
__device__ __forceinline__ int row_lo(const Page8Args& a, const Rows& r, int i) {
  if (a.window <= 0) return 0;
  return static_cast<int>(max(0ll, static_cast<long long>(r.len) - r.n + i + 1 - a.window));
}

// Where the pieces of a query token's results lie, for the join kernel: one
// load instead of a search through the lengths.
struct alignas(16) TokenInfo {
  long long u0;     // first unit of its row tiles (of kv head 0)
  long long run;    // units of a worker
  int ng;           // units of a task that have results (-1: no sequence has the token)
  int stride;       // units of a task
  int nt, r0;       // tasks per kv head, first row in the task (or tasks)
  int kind;         // 0: the split form, 1: the tiled form
  int pad[3];
};

// The tiled form (attend_page8_tile.cu): 128 / G whole queries per tile, two
// tiles per item, one worker per CTA.
struct TileArgs {
  Page8Args p;
  int tq;
  float* part_o;      // [2 * CTAs][256][D]
  float2* part_ml;    // [2 * CTAs][256] (m, l)
  TokenInfo* info;    // [T]
};
cudaError_t launch_attend_tiles(const TileArgs& a, int head_dim, bool int8, bool f16, int sms, cudaStream_t stream);

// Four 8-bit codes as two pairs of f16 (exact).
template <bool kInt8>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    // 1024 + (code + 128) as f16 by its bits, minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 c = __floats2half2_rn(1152.f, 1152.f);
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), c), y = __hsub2(*reinterpret_cast<__half2*>(&b), c);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  } else {
    lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xFFFFu));
    hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
  }
}

// 2^x by the hardware approximation (relative error ~2^-22; -inf -> 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (1 + e^(2x)): absolute error below 3e-7 (the hardware's
// tanh is good to 2^-11 only, which a cap of 50 turns into 0.02 of a logit).
__device__ __forceinline__ float tanh_of(float x) {
  float r;
  const float d = 1.f + fast_exp2(x * (2.f * kLog2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return fmaf(-2.f, r, 1.f);
}
// tanh(x) for caps above kNearCap, good to 2^-19 of itself: below 1/2 Taylor's series
// up to x^11 (off by its next term, 9e-7 of x), from there on the form above
// (3e-7, which is 7e-7 of tanh(1/2)).
__device__ __forceinline__ float tanh_far(float x) {
  const float t = x * x;
  float p = fmaf(-1382.f / 155925.f, t, 62.f / 2835.f);
  p = fmaf(p, t, -17.f / 315.f);
  p = fmaf(p, t, 2.f / 15.f);
  p = fmaf(p, t, -1.f / 3.f);
  return fabsf(x) < 0.5f ? fmaf(x * t, p, x) : tanh_of(x);
}

// The power of two that takes a row of bf16 values with the given largest
// magnitude to [2^14, 2^15), and its inverse: f16 then holds the row's values
// (8 significant bits) exactly down to 2^-31 of the largest.
__device__ __forceinline__ float q_to_f16_scale(float amax, float* inv) {
  int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  e = e < -100 ? -100 : e > 127 ? 127 : e;
  *inv = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
  return __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
}

template <typename E>
__device__ __forceinline__ uint32_t pack_out(float hi, float lo) {
  if constexpr (std::is_same<E, __half>::value) {
    return f32x2_to_f16x2(hi, lo);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace qpkv
