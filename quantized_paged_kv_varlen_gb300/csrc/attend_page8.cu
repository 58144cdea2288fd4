// Attention over a paged cache in 8 bits with one scale per (page, kv head):
// the split form for few query rows (single tokens, drafted tokens).
//
//   x(r, j) = sm_scale * q_r . k8_j * ks[page(j)]       (k8, v8: the codes)
//   x = cap * tanh(x / cap)        with a cap
//   x = x + slope_h * (j - at_r)   with a bias, at_r the position of row r
//   o_r = sum_j softmax_j(x(r, .)) * v8_j * vs[page(j)],  j in [lo_r, hi_r)
//
// Every row's visible keys are one interval: hi_r = at_r + 1 (causal) raised
// to the prefix length and cut at L, lo_r = at_r + 1 - window.
//
// Each cached byte is needed once per 16 query rows and then thrown away, so
// the kernel is bound by HBM and built to keep loads in flight: warps work
// alone (no block barrier after the start), each streaming groups of 16
// tokens of one kv head through a ring of its own of cp.async stages.  Every
// thread copies exactly the bytes it will use, in the order the matrix
// instruction wants them, so no operand crosses threads:
//   S = Q K^T    m16n8k16: row = query row, n = token; a thread holds 32 of a
//                token's dims (16-byte chunks t and t + 4), taken as the k
//                index in any order that Q follows
//   O += P V     k = token, n = dim: thread (g, t) holds chunk g of tokens
//                2t, 2t + 1, 2t + 8, 2t + 9, whose scores it also holds
// (g = lane / 4, t = lane % 4).  E4M3 and INT8 codes are exact in f16; a bf16
// query row enters as f16 times a power of two that puts its largest element
// in [2^14, 2^15), exact for everything within 2^-31 of it.  P is f16 (2^-12
// relative); statistics and O are float32.
//
// The value scale joins the running maximum: with y = x log2(e) + log2(vs)
// P = 2^(y - m) multiplies raw codes, and the denominator takes P / vs.  m is
// 7 below the maximum when it is set and moves only when some y exceeds it by
// more than 15: P <= 2^15 stays in f16's range, and keys down to 2^-21 of the
// largest keep all 11 bits (a value of 448 may meet one of 2^-9).
//
// Work is split without a plan, so that lengths may change on the device (and
// in a captured graph): all (sequence, kv head, 16-row tile, 16-token group)
// units in a row are cut into equal runs, one per warp.  A run that covers a
// whole (sequence, head, tile) writes the output; pieces go to the workspace
// (at most two per warp: the one it begins with and the one it ends with) and
// the join kernel adds them up in the order of the runs.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

constexpr int kWarps = 4;               // per block
constexpr int kBlocksPerSm = 3;
constexpr int kStages = 4;
constexpr int kGroup = 16;              // tokens of a unit
constexpr int kMinRun = 4;              // units of a run at least (64 tokens)
constexpr uint32_t kBadPageMark = 0x7FFFDEADu;   // in the place of a scale: skip the group

struct SplitArgs {
  Page8Args p;
  int workers;
  int ws_rows;             // rows a piece holds in the workspace (at most 16)
  float* part_o;           // [2 * workers][ws_rows][D]
  float2* part_ml;         // [2 * workers][ws_rows] (m, l)
  long long* sched;        // [B + 1] units before each sequence, [B + 1]: run length
};

// Units of sequence b: groups [g0, g0 + ng) for each of nt row tiles and Hkv heads.
struct Span {
  int t0, n, len, g0, ng, nt;
};

__device__ __forceinline__ Span span_of(const Page8Args& a, int b, int* err) {
  Span s = {0, 0, 0, 0, 0, 0};
  Rows r = rows_of(a, b, err);
  s.t0 = r.t0;
  s.n = r.n;
  s.len = r.len;
  if (r.n <= 0) return s;
  const int hi = row_hi(a, r, r.n - 1), lo = row_lo(a, r, 0);
  if (hi > lo) {
    s.g0 = lo / kGroup;
    s.ng = (hi + kGroup - 1) / kGroup - s.g0;
    s.nt = (r.n * a.G + 15) / 16;
  }
  return s;
}

template <bool kInt8>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    // 1024 + (code + 128) as f16 by its bits, minus 1152: exact
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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

__device__ __forceinline__ void cp_async_8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int D>
struct Ring {
  static constexpr int kK = D / 64;                  // 16-byte chunks of a token a thread copies
  static constexpr int kVB = D / 8;                  // bytes of a V token a thread copies
  static constexpr int kStage = 2 * kGroup * D;      // K and V of a group
  static constexpr int kWarpBytes = kStages * kStage;
};

template <typename E, int D, bool kInt8, bool kCap, bool kBias>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm) attend_split_kernel(const __grid_constant__ SplitArgs sa) {
  constexpr int KS = D / 16;      // k steps of Q K^T
  constexpr int NT = D / 8;       // 8-dim tiles of O: thread g's dim i of its chunk
  constexpr int KC = Ring<D>::kK;
  constexpr int VB = Ring<D>::kVB;
  constexpr int VW = VB / 4;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long s_prefix[kWarps * 32 + 1];
  __shared__ float2 s_scale[kWarps][kStages];
  const Page8Args& a = sa.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();

  // ---- units before each block of `per` sequences
  const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
  {
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Span s = span_of(a, b, blockIdx.x == 0 ? a.err : nullptr);
      mine += static_cast<long long>(s.ng) * s.nt * a.Hkv;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __shared__ long long w_sum[kWarps];
    if (lane == 31) w_sum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += w_sum[w];
    s_prefix[tid + 1] = inc;
    if (tid == 0) s_prefix[0] = 0;
    __syncthreads();
  }
  const long long total = s_prefix[kWarps * 32];
  long long run = (total + sa.workers - 1) / sa.workers;
  run = run < kMinRun ? kMinRun : run;
  if (blockIdx.x == 0) {   // what the join kernel needs to know of the split
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long at = s_prefix[tid];
    for (int b = b0; b < b1; ++b) {
      sa.sched[b] = at;
      const Span s = span_of(a, b, nullptr);
      at += static_cast<long long>(s.ng) * s.nt * a.Hkv;
    }
    if (tid == 0) {
      sa.sched[a.B] = total;
      sa.sched[a.B + 1] = run;
    }
  }
  const int worker = blockIdx.x * kWarps + warp;
  long long u = worker * run;
  const long long u_end = u + run < total ? u + run : total;
  const long long u_begin = u;
  if (u >= u_end) return;

  uint8_t* ring = smem + warp * Ring<D>::kWarpBytes;
  // the sequence of unit u
  int blk = 0;
  {
    int lo = 0, hi = kWarps * 32 - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (u < s_prefix[mid + 1]) hi = mid; else lo = mid + 1;
    }
    blk = lo;
  }
  int b = blk * per;
  long long before = s_prefix[blk];
  Span sp = span_of(a, b, nullptr);

  while (u < u_end) {
    long long in_b = static_cast<long long>(sp.ng) * sp.nt * a.Hkv;
    while (u >= before + in_b) {   // a run may cross into later sequences
      before += in_b;
      ++b;
      sp = span_of(a, b, nullptr);
      in_b = static_cast<long long>(sp.ng) * sp.nt * a.Hkv;
    }
    const long long local = u - before;
    const int task = static_cast<int>(local / sp.ng);
    const int first = static_cast<int>(local - static_cast<long long>(task) * sp.ng);
    const int h = task / sp.nt, rt = task - h * sp.nt;
    const int count = static_cast<int>(min(static_cast<long long>(sp.ng - first), u_end - u));
    const bool whole_task = count == sp.ng;
    const size_t piece = 2 * static_cast<size_t>(worker) + (u == u_begin ? 0 : 1);
    const int gbeg = sp.g0 + first;

    // ---- the ring: page ids of 32 groups at a time, one per lane
    const long long head_off = static_cast<long long>(h) * a.head_stride;
    const int32_t* bt = a.bt + static_cast<size_t>(b) * a.bt_stride;
    const int gpp = a.ps / kGroup;
    int ids = -1, in_page = 0;
    auto lookup = [&](int i0) {   // groups gbeg + i0 + lane
      const int i = i0 + lane;
      ids = -1;
      if (i < count) {
        const int gi = gbeg + i, pg = gi / gpp;
        in_page = gi - pg * gpp;
        ids = __ldg(bt + pg);
        if (ids < 0 || ids >= a.num_pages) {
          report_error(a.err, kDevErrBadPage);
          ids = -1;
        }
      }
    };
    auto issue = [&](int i) {
      if (i < count) {
        if ((i & 31) == 0) lookup(i);
        const int page = __shfl_sync(0xffffffffu, ids, i & 31);
        const int off = __shfl_sync(0xffffffffu, in_page, i & 31);
        const int st = i % kStages;
        uint8_t* dst = ring + st * Ring<D>::kStage;
        if (page >= 0) {
          const long long base = page * a.page_stride + static_cast<long long>(off) * kGroup * a.tok_stride + head_off;
          const uint8_t* kp = a.k + base + g * a.tok_stride + 16 * t;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            cp_async_16(dst + (2 * c) * 512 + lane * 16, kp + 64 * c);
            cp_async_16(dst + (2 * c + 1) * 512 + lane * 16, kp + 8 * a.tok_stride + 64 * c);
          }
          const uint8_t* vp = a.v + base + 2 * t * a.tok_stride + VB * g;
          uint8_t* vd = dst + kGroup * D;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint8_t* src = vp + ((c & 1) + (c >> 1) * 8) * a.tok_stride;
            if constexpr (VB == 16) cp_async_16(vd + c * 512 + lane * 16, src);
            else cp_async_8(vd + c * 256 + lane * 8, src);
          }
          if (lane < 2)
            cp_async_4(reinterpret_cast<float*>(&s_scale[warp][st]) + lane,
                       (lane == 0 ? a.ks : a.vs) + static_cast<size_t>(page) * a.Hkv + h);
        } else if (lane == 0) {
          s_scale[warp][st].x = __uint_as_float(kBadPageMark);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- Q: rows rt * 16 + g and + 8; row r is query r / G, head h * G + r % G
    Rows rows;
    rows.t0 = sp.t0, rows.n = sp.n, rows.len = sp.len;
    rows.prefix = a.prefix != nullptr ? __ldg(a.prefix + b) : 0;
    uint32_t qf[KS][4];
    float sc[2], slope[2];
    int hi[2], lo[2], at[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rt * 16 + g + 8 * x;
      const bool live = r < sp.n * a.G;
      const int rr = live ? r : sp.n * a.G - 1;       // dead rows: zeros with the last row's limits
      const int i = rr / a.G, head = h * a.G + (rr - i * a.G);
      at[x] = sp.len - sp.n + i;
      hi[x] = row_hi(a, rows, i);
      lo[x] = row_lo(a, rows, i);
      slope[x] = kBias ? __ldg(a.slopes + head) * kLog2e : 0.f;
      const E* src = static_cast<const E*>(a.q) + (static_cast<size_t>(sp.t0 + i) * a.Hq + head) * D;
      uint2 raw[KS];
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int dim = (k < 4 ? 16 * t : 16 * (t + 4)) + 4 * (k & 3);
        raw[k] = live ? __ldg(reinterpret_cast<const uint2*>(src + dim)) : make_uint2(0, 0);
      }
      float inv = 1.f;
      if constexpr (std::is_same<E, __half>::value) {
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[k][x] = raw[k].x, qf[k][2 + x] = raw[k].y;
      } else {
        float f[KS][4];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          f[k][0] = __uint_as_float(raw[k].x << 16), f[k][1] = __uint_as_float(raw[k].x & 0xFFFF0000u);
          f[k][2] = __uint_as_float(raw[k].y << 16), f[k][3] = __uint_as_float(raw[k].y & 0xFFFF0000u);
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(f[k][e]));
        }
        const float mul = q_to_f16_scale(quad_max(amax), &inv);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[k][x] = f32x2_to_f16x2(f[k][1] * mul, f[k][0] * mul);
          qf[k][2 + x] = f32x2_to_f16x2(f[k][3] * mul, f[k][2] * mul);
        }
      }
      sc[x] = inv * (kCap ? a.scale_cap : a.scale_log2);
    }
    // keys that every row of the tile sees
    int all_lo = max(lo[0], lo[1]), all_hi = min(hi[0], hi[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
    }

    float O[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      issue(i + kStages - 1);
      cp_async_wait_group<kStages - 1>();
      __syncwarp();                                  // the scales come from lanes 0 and 1
      const int st = i % kStages;
      const uint8_t* src = ring + st * Ring<D>::kStage;
      const float2 kv = s_scale[warp][st];
      const bool skip = __float_as_uint(kv.x) == kBadPageMark;
      if (!skip) {
        float s[2][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(src + (2 * c) * 512 + lane * 16);
          const uint4 x1 = *reinterpret_cast<const uint4*>(src + (2 * c + 1) * 512 + lane * 16);
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1, d0, d1;
            widen<kInt8>(w0[k], b0, b1);
            widen<kInt8>(w1[k], d0, d1);
            mma16816(s[0], qf[4 * c + k], b0, b1);
            mma16816(s[1], qf[4 * c + k], d0, d1);
          }
        }
        // ---- scores in log2 units, with log2 of the value scale
        const int j0 = (gbeg + i) * kGroup;
        const bool whole = j0 >= all_lo && j0 + kGroup <= all_hi;
        const float vs = fmaxf(kv.y, kMinScale);
        const float lv = kv.y == 0.f ? 0.f : log2f(vs), rvs = kv.y == 0.f ? 1.f : 1.f / vs;
        float y[2][4];   // [row][token 2t, 2t+1, 2t+8, 2t+9]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f = sc[x] * kv.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = s[e >> 1][2 * x + (e & 1)] * f;
            if constexpr (kCap) v = a.cap_log2 * tanh_of(v);
            const int j = j0 + 2 * t + (e & 1) + 8 * (e >> 1);
            if constexpr (kBias) v = fmaf(slope[x], static_cast<float>(j - at[x]), v);
            v += lv;
            if (!whole && (j < lo[x] || j >= hi[x])) v = -INFINITY;
            y[x][e] = v;
          }
        }
        bool up = false;
        float top[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(fmaxf(y[x][0], y[x][1]), fmaxf(y[x][2], y[x][3]));
          up |= top[x] > m[x] + kMaxP;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float now = fmaxf(m[x], quad_max(top[x]) - kSetP);
            const float f = m[x] > -INFINITY ? fast_exp2(m[x] - now) : 0.f;
            m[x] = now;
            l[x] *= f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              O[n][2 * x] *= f;
              O[n][2 * x + 1] *= f;
            }
          }
        }
        uint32_t pf[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mm = m[x] > -INFINITY ? m[x] : 0.f;
          const float p0 = fast_exp2(y[x][0] - mm), p1 = fast_exp2(y[x][1] - mm);
          const float p2 = fast_exp2(y[x][2] - mm), p3 = fast_exp2(y[x][3] - mm);
          l[x] = fmaf((p0 + p1) + (p2 + p3), rvs, l[x]);
          pf[x] = f32x2_to_f16x2(p1, p0);
          pf[2 + x] = f32x2_to_f16x2(p3, p2);
        }
        // ---- O += P V
        const uint8_t* vsrc = src + kGroup * D;
        uint32_t vw[4][VW];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (VB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(vsrc + c * 512 + lane * 16);
            vw[c][0] = x.x, vw[c][1] = x.y, vw[c][VW - 2] = x.z, vw[c][VW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vsrc + c * 256 + lane * 8);
            vw[c][0] = x.x, vw[c][1] = x.y;
          }
        }
        if (!kInt8 && !whole) {   // P = 0 does not cancel a NaN code of a token no row sees
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = j0 + 2 * t + (c & 1) + 8 * (c >> 1);
            if (j >= sp.len) {
#pragma unroll
              for (int k = 0; k < VW; ++k) vw[c][k] = 0;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          uint32_t b0[4], b1[4];
          widen<kInt8>(__byte_perm(vw[0][k], vw[1][k], 0x5140), b0[0], b0[1]);
          widen<kInt8>(__byte_perm(vw[0][k], vw[1][k], 0x7362), b0[2], b0[3]);
          widen<kInt8>(__byte_perm(vw[2][k], vw[3][k], 0x5140), b1[0], b1[1]);
          widen<kInt8>(__byte_perm(vw[2][k], vw[3][k], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma16816(O[4 * k + e], pf, b0[e], b1[e]);
        }
      }
      __syncwarp();   // the stage may be filled again
    }
    cp_async_wait_all();

    // ---- the run's part of this task: dims [VB * 2t, VB * 2t + 2 VB) of rows g, g + 8
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rt * 16 + g + 8 * x;
      const float lsum = quad_sum(l[x]);
      if (r >= sp.n * a.G) continue;
      if (whole_task) {
        const int i = r / a.G, head = h * a.G + (r - i * a.G);
        const size_t row = static_cast<size_t>(sp.t0 + i) * a.Hq + head;
        const float so = lsum > 0.f ? 1.f / lsum : 0.f;
        E* out = static_cast<E*>(a.o) + row * D + 2 * VB * t;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[NT / 2];
#pragma unroll
          for (int n = 0; n < NT / 2; ++n)
            w[n] = pack_out<E>(O[2 * n + 1][2 * x + half] * so, O[2 * n][2 * x + half] * so);
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
            reinterpret_cast<uint4*>(out + VB * half)[n] = make_uint4(w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]);
        }
        if (t == 0 && a.lse != nullptr)
          a.lse[row] = lsum > 0.f ? (m[x] + log2f(lsum)) * kLn2 : -INFINITY;
      } else {
        const int pr = g + 8 * x;
        float* out = sa.part_o + (piece * sa.ws_rows + pr) * D + 2 * VB * t;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int n = 0; n < NT / 4; ++n)
            reinterpret_cast<float4*>(out + VB * half)[n] =
                make_float4(O[4 * n][2 * x + half], O[4 * n + 1][2 * x + half], O[4 * n + 2][2 * x + half],
                            O[4 * n + 3][2 * x + half]);
        if (t == 0) sa.part_ml[piece * sa.ws_rows + pr] = make_float2(m[x], lsum);
      }
    }
    __syncwarp();
    u += count;
  }
}

// One warp per (token, head): adds up the pieces of its task in the order of
// the runs, and gives rows that see no key their zeros.
template <typename E, int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ SplitArgs sa) {
  constexpr int EPL = D / 32;
  const Page8Args& a = sa.p;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x) >> 5;
  const int tok = static_cast<int>(w / a.Hq), head = static_cast<int>(w - static_cast<long long>(tok) * a.Hq);
  if (tok >= a.T) return;
  const int b = seq_of_token(a.cu, a.B, tok);
  const Span sp = span_of(a, b, nullptr);
  if (sp.n <= 0 || tok < sp.t0 || tok >= sp.t0 + sp.n) return;   // a row behind the last sequence
  const size_t row = static_cast<size_t>(tok) * a.Hq + head;
  float acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  float M = -INFINITY, l = 0.f;
  if (sp.ng > 0) {
    const int h = head / a.G, r = (tok - sp.t0) * a.G + (head - h * a.G);
    const long long u0 = sa.sched[b] + (static_cast<long long>(h) * sp.nt + r / 16) * sp.ng, u1 = u0 + sp.ng;
    const long long run = sa.sched[a.B + 1];
    const int w0 = static_cast<int>(u0 / run), w1 = static_cast<int>((u1 - 1) / run);
    if (w0 == w1) return;   // written whole by its run
    const int pr = r & 15;
    auto piece = [&](int k) {
      return (2 * static_cast<size_t>(k) + (k == w0 && u0 != k * run ? 1 : 0)) * sa.ws_rows + pr;
    };
    for (int k = w0 + lane; k <= w1; k += 32) M = fmaxf(M, sa.part_ml[piece(k)].x);
    M = warp_max(M);
    if (M > -INFINITY) {
#pragma unroll 4
      for (int k = w0; k <= w1; ++k) {
        const size_t at = piece(k);
        const float2 ml = sa.part_ml[at];
        const float f = fast_exp2(ml.x - M);   // a piece that saw nothing: m = -inf, f = 0
        l = fmaf(ml.y, f, l);
        const float* src = sa.part_o + at * D + lane * EPL;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] = fmaf(src[e], f, acc[e]);
      }
    }
  }
  const float so = l > 0.f ? 1.f / l : 0.f;
  E* out = static_cast<E*>(a.o) + row * D + lane * EPL;
#pragma unroll
  for (int e = 0; e < EPL; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_out<E>(acc[e + 1] * so, acc[e] * so);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l > 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename K>
cudaError_t launch(K kernel, unsigned grid, unsigned threads, size_t smem, const SplitArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename E, int D, bool kInt8, bool kCap, bool kBias>
cudaError_t go(const SplitArgs& a, unsigned blocks, cudaStream_t s) {
  constexpr size_t smem = kWarps * Ring<D>::kWarpBytes;
  auto kernel = attend_split_kernel<E, D, kInt8, kCap, kBias>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if ((e = launch(kernel, blocks, kWarps * 32, smem, a, s)) != cudaSuccess) return e;
  const long long warps = static_cast<long long>(a.p.T) * a.p.Hq;
  return launch(attend_join_kernel<E, D>, static_cast<unsigned>((warps + 3) / 4), 128, 0, a, s);
}

template <typename E, int D, bool kInt8>
cudaError_t pick2(const SplitArgs& a, unsigned blocks, cudaStream_t s) {
  const bool cap = a.p.cap_log2 > 0.f, bias = a.p.slopes != nullptr;
  if (cap) return bias ? go<E, D, kInt8, true, true>(a, blocks, s) : go<E, D, kInt8, true, false>(a, blocks, s);
  return bias ? go<E, D, kInt8, false, true>(a, blocks, s) : go<E, D, kInt8, false, false>(a, blocks, s);
}

template <typename E>
cudaError_t pick(const SplitArgs& a, int D, bool int8, unsigned blocks, cudaStream_t s) {
  if (D == 64) return int8 ? pick2<E, 64, true>(a, blocks, s) : pick2<E, 64, false>(a, blocks, s);
  return int8 ? pick2<E, 128, true>(a, blocks, s) : pick2<E, 128, false>(a, blocks, s);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of a piece and the three arrays' sizes.
void sizes(int B, int T, int Hq, int Hkv, int D, int workers, int* rows, size_t* o, size_t* ml, size_t* sched) {
  const long long most = static_cast<long long>(T) * (Hq / Hkv);
  *rows = most < 16 ? static_cast<int>(most) : 16;
  *o = up256(static_cast<size_t>(2) * workers * *rows * D * sizeof(float));
  *ml = up256(static_cast<size_t>(2) * workers * *rows * sizeof(float2));
  *sched = up256((static_cast<size_t>(B) + 2) * sizeof(long long));
}

}  // namespace

size_t attend_page8_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  int rows;
  size_t o, ml, sched;
  sizes(B, T, Hq, Hkv, D, kAttendMaxSms * kBlocksPerSm * kWarps, &rows, &o, &ml, &sched);
  return o + ml + sched;
}

cudaError_t launch_attend_page8(const qpkv_attend_page8_params& p, cudaStream_t stream) {
  SplitArgs a;
  a.p = page8_args(p);
  int sms = sm_count();
  if (sms > kAttendMaxSms) sms = kAttendMaxSms;
  const unsigned blocks = static_cast<unsigned>(sms) * kBlocksPerSm;
  a.workers = static_cast<int>(blocks) * kWarps;
  size_t o, ml, sched;
  sizes(p.num_seqs, p.num_tokens, p.num_heads_q, p.num_heads_kv, p.head_dim, a.workers, &a.ws_rows, &o, &ml, &sched);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + o);
  a.sched = reinterpret_cast<long long*>(ws + o + ml);
  const bool int8 = p.format == QPKV_FORMAT_INT8;
  return p.dtype == QPKV_DTYPE_F16 ? pick<__half>(a, p.head_dim, int8, blocks, stream)
                                   : pick<__nv_bfloat16>(a, p.head_dim, int8, blocks, stream);
}

}  // namespace qpkv
