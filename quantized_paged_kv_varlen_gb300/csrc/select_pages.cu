// The pages that each query token attends to, by a cheap score of every page
// ("KvQuantSparseFlashAttention" README, 参数说明 row sparse_indices: block-wise
// index lists per query token and kv head, which come from outside there).
//
//   c = RNE(q * 127 / a), a = max |q| over the G heads of a kv head
//   score(page) = scale(page) * max_g sum_d max(c_gd min_d, c_gd max_d)
//               = scale(page) * max_g (c_g^+ . max + c_g^- . min)
// a bound on what any key between the page's bounds can score.  Sums are whole
// numbers of at most 127 * 127 * 128 < 2^21, so f16 products summed in float32
// by the tensor core are exact and so is the order of the scores.
//
// The bounds are read once, 2 D bytes a (page, head): HBM- or L2-bound.  A
// cluster of 1 to 8 blocks takes one (token, kv head): few rows over long caches
// still fill the GPU.  Scores:
// warps take 16 pages at a time as the rows of m16n8k16, heads as its 8 columns
// (padded with copies); a thread's bytes of a page are 16-byte chunks whose
// channels are the k index in an order that the queries follow.  Scores become
// integers of the same order in shared memory; the n-th largest is found eight bits
// at a time by histograms that the cluster adds up through distributed shared
// memory, ties go to the lower page by counting.
#include <cooperative_groups.h>
#include <type_traits>

#include "common.cuh"
#include "group4.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxKeys = 48 * 1024;      // scores of a block in shared memory

struct SelectArgs {
  int B, T, Hq, H, G, ps, num_pages, bt_stride, n, first, last, window;
  const int32_t *cu, *lens, *bt;
  const void* q;
  const int8_t* bounds;
  const float* bscale;
  int32_t* out;
  int* err;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An unsigned integer that orders like the float; finite and infinite scores are above 0.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// A page's key, of its sum and scale: one that is not finite (of a NaN in the page,
// or bounds never made) counts as +inf, as a NaN's bits would be those of kSure.
__device__ __forceinline__ uint32_t key_of(float sum, float scale) {
  return key_of(fabsf(scale) < INFINITY ? sum * scale : INFINITY);
}

template <typename E>
__device__ __forceinline__ float to_f32(uint32_t half_word) {
  if constexpr (std::is_same<E, __half>::value) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(half_word)));
  } else {
    return __uint_as_float(half_word << 16);
  }
}

// c of an element: RNE(q * 127 / a), with 1 / a rounded.  q has 11 significant
// bits at most, so q * 127 is exact; the corrected quotient (as in write_group4.cu)
// meets a tie exactly where there is one, and elsewhere the distance to the next
// is a thousand times its error.
struct Unit {
  float a, r;       // the largest magnitude times k, and one over it
  float k;          // 127 times the power of two that keeps both in range
  bool scored;
};
__device__ __forceinline__ Unit unit_of(float amax) {
  Unit u;
  u.scored = amax > 0.f && amax < INFINITY;
  const float p = amax > 0x1p60f ? 0x1p-64f : amax < 0x1p-60f ? 0x1p64f : 1.f;
  u.a = amax * p;
  u.r = u.scored ? __frcp_rn(u.a) : 0.f;
  u.k = 127.f * p;
  return u;
}
template <typename E>
__device__ __forceinline__ float code_of(uint32_t half_word, const Unit& u) {
  const float x = to_f32<E>(half_word) * u.k, y = x * u.r;
  return rintf(fmaf(fmaf(-y, u.a, x), u.r, y));
}

// A piece of q as f16 codes: the positive ones beside the maxima, the negative
// ones beside the minima.
template <typename E>
__device__ __forceinline__ uint2 codes_of(uint2 w, const Unit& u, bool is_max) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (u.scored) {
    x[0] = code_of<E>(w.x & 0xFFFFu, u), x[1] = code_of<E>(w.x >> 16, u);
    x[2] = code_of<E>(w.y & 0xFFFFu, u), x[3] = code_of<E>(w.y >> 16, u);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = is_max ? fmaxf(x[e], 0.f) : fminf(x[e], 0.f);
  return make_uint2(f32x2_to_f16x2(x[1], x[0]), f32x2_to_f16x2(x[3], x[2]));
}

// What lies between the sure keys (kSure) and those of no candidate (0).
constexpr uint32_t kSure = 0xFFFFFFFFu;
struct Spread {
  uint32_t lo, hi;      // the smallest and largest
  int sure, others;     // how many
  __device__ __forceinline__ void take(uint32_t key) {
    if (key == kSure) {
      ++sure;
    } else if (key != 0) {
      lo = min(lo, key);
      hi = max(hi, key);
      ++others;
    }
  }
  __device__ __forceinline__ void warp_all() {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    sure = __reduce_add_sync(0xffffffffu, sure);
    others = __reduce_add_sync(0xffffffffu, others);
  }
};

// The digit that the `need`-th largest of 256 bins falls into: bins are counted
// from the last down by a warp, 8 a lane.  Returns the digit; *need becomes its
// place among the keys of that bin, *whole whether it is the bin's last.
__device__ __forceinline__ uint32_t find_digit(const uint32_t* bins, int* need, bool* whole) {
  const int lane = threadIdx.x & 31;
  int bin[8], mine = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) mine += bin[k] = static_cast<int>(bins[255 - 8 * lane - k]);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const int who = __ffs(__ballot_sync(0xffffffffu, upto >= *need)) - 1;
  int before = upto - mine, digit = 0, in_bin = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (before + bin[k] >= *need) {
      digit = 255 - 8 * lane - k;
      in_bin = bin[k];
      break;
    }
    before += bin[k];
  }
  *need -= __shfl_sync(0xffffffffu, before, who);
  *whole = *need == __shfl_sync(0xffffffffu, in_bin, who);
  return __shfl_sync(0xffffffffu, digit, who);
}

// The search for the n-th largest key, by digits of eight bits of what keys have
// above the smallest (scores lie close to one another: their own leading bits
// would put them all into a few bins).
struct Search {
  uint32_t base, prefix;
  int bits;             // of the keys' differences that are still open
  int need;             // keys to take among those with the prefix
  uint32_t above;       // in the end: take the keys above this one, and `need` equal to it
  // false: nothing to search
  __device__ __forceinline__ bool begin(const Spread& x, int n) {
    need = 0;
    if (x.sure + x.others <= n) {
      above = 0;
      return false;
    }
    need = n - x.sure;
    if (need <= 0) {
      need = 0;
      above = kSure - 1;
      return false;
    }
    base = x.lo;
    prefix = 0;
    bits = 32 - __clz(x.hi - x.lo);
    above = base;
    return bits > 0;
  }
  __device__ __forceinline__ int width() const { return min(8, bits); }
  // the digit of a key in question, -1: none
  __device__ __forceinline__ int digit(uint32_t key) const {
    if (key == 0 || key == kSure) return -1;
    const uint32_t d = key - base;
    if (bits < 32 && d >> bits != prefix) return -1;
    return static_cast<int>(d >> (bits - width()) & 255u & ((1u << width()) - 1));
  }
  // false: found
  __device__ __forceinline__ bool next(const uint32_t* bins) {
    bool whole;
    const uint32_t d = find_digit(bins, &need, &whole);
    const int w = width();
    prefix = prefix << w | d;
    bits -= w;
    if (whole) {                      // all of the bin: the keys from its first on
      above = base + (prefix << bits) - 1;      // base > 0
      need = 0;
      return false;
    }
    above = base + prefix;            // final once no bits are left
    return bits > 0;
  }
};

template <typename E, int D, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 && D == 128 ? 4 : 1) select_pages_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int KC = D / 32;          // 16-byte chunks of a page's 2 D bounds per thread
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[4][256], s_sum[256];
  __shared__ int s_gt[kWarps], s_eq[kWarps];
  __shared__ int2 s_total;
  __shared__ float s_amax[kWarps];
  __shared__ Spread s_spread[kWarps];
  __shared__ uint2 s_q[NB][4 * KC][32];   // fragments of the queries, the same in all warps
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x / C, tok = row / a.H, h = row - tok * a.H;
  const int b = warp_last_at_most(a.B, tok, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1)); });
  // equal prefix sums: the last of them is the one with the rows
  const int t0 = seq_begin(a.cu, b), n_q = __ldg(a.cu + b) - t0;
  if (tok < t0 || tok >= t0 + n_q) return;                // behind the last sequence
  int len = __ldg(a.lens + b);
  if (t0 < 0 || t0 + static_cast<long long>(n_q) > a.T || len < 0 || len > static_cast<long long>(a.bt_stride) * a.ps) {
    if (tid == 0) report_error(a.err, kDevErrBadLength);
    len = 0;
  }
  int32_t* out = a.out + static_cast<size_t>(row) * a.n;
  const long long at = static_cast<long long>(len) - n_q + (tok - t0);
  if (len == 0 || at < 0) {
    if (rank == 0)
      for (int i = tid; i < a.n; i += kThreads) out[i] = -1;
    return;
  }
  const int p_hi = static_cast<int>(at / a.ps);
  const int p_lo = a.window > 0 ? static_cast<int>(max(0ll, at + 1 - a.window) / a.ps) : 0;
  const int share = (p_hi - p_lo + C) / C;                // candidates of a block
  const int p0 = min(p_lo + rank * share, p_hi + 1), count = min(share, p_hi + 1 - p0);
  const int32_t* bt = a.bt + static_cast<size_t>(b) * a.bt_stride + p0;

  for (int i = tid; i < 4 * 256; i += kThreads) (&s_hist[0][0])[i] = 0;
  // ---- the queries: their largest magnitude, then c
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (static_cast<size_t>(tok) * a.Hq + h * a.G) * D;
  float amax;
  {
    uint32_t top = 0;     // magnitudes are ordered like their bits
    for (int i = tid; i < a.G * D / 8; i += kThreads) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + i);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    const uint32_t one = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if (lane == 0) s_amax[warp] = __uint_as_float(one);
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all = max(all, __float_as_uint(s_amax[w]));
    amax = to_f32<E>(all);
  }
  const Unit unit = unit_of(amax);

  // ---- scores
  for (int c0 = 0; c0 < a.G; c0 += 8 * NB) {
    // columns: heads c0 .. c0 + 8 NB, those behind the last are copies of others
    if (c0 > 0) __syncthreads();
    for (int i = tid; i < NB * 4 * KC * 32; i += kThreads) {
      const int l = i % 32, c = i / 128 % KC, w4 = i / 32 % 4, nb = i / (128 * KC);
      const uint16_t* qh = q + static_cast<size_t>((c0 + 8 * nb + (l >> 2)) % a.G) * D;
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(qh + (16 * ((l & 3) + 4 * c)) % D + 4 * w4));
      s_q[nb][4 * c + w4][l] = codes_of<E>(w, unit, c >= KC / 2);
    }
    __syncthreads();
    for (int i0 = warp * 32; i0 < count; i0 += kWarps * 32) {
      // 32 pages, a lane looks up one
      int page = -1;
      float scale = 0.f;
      if (i0 + lane < count) {
        page = __ldg(bt + i0 + lane);
        if (page < 0 || page >= a.num_pages) {
          report_error(a.err, kDevErrBadPage);
          page = -1;
        } else {
          scale = __ldg(a.bscale + static_cast<size_t>(page) * a.H + h);
        }
      }
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        uint4 x[2][KC];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pg = __shfl_sync(0xffffffffu, page, 16 * s + 8 * e + g);
          const uint4* src = reinterpret_cast<const uint4*>(a.bounds + (static_cast<size_t>(pg < 0 ? 0 : pg) * a.H + h) * 2 * D) + t;
#pragma unroll
          for (int c = 0; c < KC; ++c) x[e][c] = pg < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + 4 * c);
        }
        float d[NB][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint32_t w0[4] = {x[0][c].x, x[0][c].y, x[0][c].z, x[0][c].w};
          const uint32_t w1[4] = {x[1][c].x, x[1][c].y, x[1][c].z, x[1][c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[4];
            widen<true>(w0[k], f[0], f[2]);
            widen<true>(w1[k], f[1], f[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const uint2 w = s_q[nb][4 * c + k][lane];
              mma16816(d[nb], f, w.x, w.y);
            }
          }
        }
        float m0 = fmaxf(d[0][0], d[0][1]), m1 = fmaxf(d[0][2], d[0][3]);
#pragma unroll
        for (int nb = 1; nb < NB; ++nb) {
          m0 = fmaxf(m0, fmaxf(d[nb][0], d[nb][1]));
          m1 = fmaxf(m1, fmaxf(d[nb][2], d[nb][3]));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        // lane 4 g (+ 1) has pages g (+ 8)
        const int mine = 16 * s + (t == 0 ? g : g + 8);
        const float sc = __shfl_sync(0xffffffffu, scale, mine);
        const int pg = __shfl_sync(0xffffffffu, page, mine), i = i0 + mine;
        if (t < 2 && i < count) {
          const int p = p0 + i;
          uint32_t key = 0;
          if (pg >= 0) {
            key = p - p_lo < a.first || p_hi - p < a.last ? kSure
                  : key_of(t == 0 ? m0 : m1, sc);
          }
          s_key[i] = c0 == 0 ? key : max(key, s_key[i]);
        }
      }
    }
    __syncwarp();    // a warp's keys are its own until all columns are through
  }
  __syncthreads();

  // ---- the n-th largest key
  Search find;
  {
    Spread x = {0xFFFFFFFFu, 0u, 0, 0};
    for (int i = tid; i < count; i += kThreads) x.take(s_key[i]);
    x.warp_all();
    if (lane == 0) s_spread[warp] = x;
    if (C > 1) cluster.sync(); else __syncthreads();
    x = {0xFFFFFFFFu, 0u, 0, 0};
    for (int w = lane; w < kWarps * C; w += 32) {
      const Spread y = *cluster.map_shared_rank(&s_spread[w % kWarps], w / kWarps);
      x.lo = min(x.lo, y.lo), x.hi = max(x.hi, y.hi);
      x.sure += y.sure, x.others += y.others;
    }
    x.warp_all();
    bool more = find.begin(x, a.n);
#pragma unroll 1
    for (int pass = 0; more; ++pass) {
      for (int i = tid; i < count; i += kThreads) {
        const int d = find.digit(s_key[i]);
        if (d >= 0) atomicAdd(&s_hist[pass][d], 1u);
      }
      const uint32_t* sums = s_hist[pass];
      if (C > 1) {
        cluster.sync();
        for (int i = tid; i < 256; i += kThreads) {
          uint32_t sum = 0;
          for (int r = 0; r < C; ++r) sum += *cluster.map_shared_rank(&s_hist[pass][i], r);
          s_sum[i] = sum;
        }
        sums = s_sum;
      }
      __syncthreads();
      more = find.next(sums);         // every warp for itself, all the same
      if (C > 1) __syncthreads();     // s_sum is read before it is written again
    }
  }

  // ---- write them in their order
  // A thread takes keys tid * per ...: an odd number apart, so that banks differ.
  const int per = ((count + kThreads - 1) / kThreads) | 1;
  const int i0 = min(count, tid * per), i1 = min(count, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = s_key[i];
    gt += key > find.above;
    eq += key == find.above;
  }
  int gt_at = gt, eq_at = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, gt_at, o), v = __shfl_up_sync(0xffffffffu, eq_at, o);
    if (lane >= o) gt_at += u, eq_at += v;
  }
  if (lane == 31) s_gt[warp] = gt_at, s_eq[warp] = eq_at;
  gt_at -= gt, eq_at -= eq;
  __syncthreads();
  int2 all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) gt_at += s_gt[w], eq_at += s_eq[w];
    all.x += s_gt[w], all.y += s_eq[w];
  }
  if (C > 1) {
    if (tid == 0) s_total = all;
    cluster.sync();
    all = make_int2(0, 0);
    for (int r = 0; r < C; ++r) {
      const int2 x = *cluster.map_shared_rank(&s_total, r);
      if (r < rank) gt_at += x.x, eq_at += x.y;
      all.x += x.x, all.y += x.y;
    }
    cluster.sync();     // nobody leaves while its totals are read
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = s_key[i];
    const bool is_eq = key == find.above;
    if (key > find.above || (is_eq && eq_at < find.need)) out[gt_at + min(eq_at, find.need)] = p0 + i;
    gt_at += key > find.above;
    eq_at += is_eq;
  }
  if (rank == 0)
    for (int i = all.x + min(all.y, find.need) + tid; i < a.n; i += kThreads) out[i] = -1;
}

// Prompts: a block takes neighbouring tokens of a sequence for one kv head, each
// of its four warps up to 16 columns of queries (`kTok` tokens), scores all their
// pages and chooses for each.  32 pages at a time the block widens their bounds
// to f16 once, into fragments in shared memory that all warps read, while the
// next 32 are on their way.  (4 pieces of 250 tokens over 10,000, 28 heads: 43 us;
// a block a token 72; a warp for itself, each widening its pages, 49.)
constexpr int kRowWarps = 4;
constexpr int kRowKeys = 44 * 1024;      // scores of a block beside its fragments

struct RowsArgs {
  SelectArgs s;
  int stride;       // keys of a token
  int tiles;
};

template <typename E, int D, int kGp>
__global__ void __launch_bounds__(kRowWarps * 32, 4) select_rows_kernel(const __grid_constant__ RowsArgs ra) {
  constexpr int KC = D / 32;
  constexpr int kTok = kGp >= 4 ? 16 / kGp : 4;
  constexpr int kBlockTok = kTok * kRowWarps;
  constexpr int NB = kGp >= 4 ? 2 : 1;
  constexpr int kJobs = 2 * KC / kRowWarps;       // (16 pages, chunk) pairs that a warp widens of 32 pages
  const SelectArgs& a = ra.s;
  extern __shared__ __align__(16) uint32_t s_mem[];
  __shared__ uint4 s_frag[2][2][4 * KC][32];
  __shared__ uint32_t s_hist[kRowWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t* keys = s_mem + static_cast<size_t>(warp) * kTok * ra.stride;
  uint32_t* hist = s_hist[warp];
  griddep_wait();
  griddep_launch_dependents();
  // ---- the tile: sequence b owns tiles [floor(cu[b-1] / kBlockTok) + b, ...)
  const int h = blockIdx.x % a.H, tile = blockIdx.x / a.H;
  const int b = warp_last_at_most(a.B, tile, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1) / kBlockTok) + m; });
  const int t0 = seq_begin(a.cu, b), n_q = __ldg(a.cu + b) - t0;
  const int first = (tile - (t0 / kBlockTok + b)) * kBlockTok;
  if (n_q <= 0 || t0 < 0 || first < 0 || first >= n_q) return;
  int len = __ldg(a.lens + b);
  if (t0 + static_cast<long long>(n_q) > a.T || len < 0 || len > static_cast<long long>(a.bt_stride) * a.ps) {
    if (threadIdx.x == 0) report_error(a.err, kDevErrBadLength);
    len = 0;
  }
  // (rows behind the arrays' are none)
  const int block_live = min(min(kBlockTok, n_q - first), a.T - t0 - first);
  if (block_live <= 0) return;
  const int i0 = first + warp * kTok, live = min(kTok, block_live - warp * kTok);    // live <= 0: this warp only helps
  const long long at0 = static_cast<long long>(len) - n_q + i0;
  // candidates of the block: from its first token's first to its last token's last
  const long long at_first = at0 - warp * kTok, at_last = at_first + block_live - 1;
  const int p_lo = a.window > 0 ? static_cast<int>(max(0ll, at_first + 1 - a.window) / a.ps) : 0;
  const int count = len > 0 && at_last >= 0 ? static_cast<int>(at_last / a.ps) - p_lo + 1 : 0;
  // ---- the queries: each token's largest magnitude, then c
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + static_cast<size_t>(t0 + (live > 0 ? i0 : first)) * a.Hq * D;
  float amax[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    uint32_t top = 0;
    const uint4* src = reinterpret_cast<const uint4*>(q + (static_cast<size_t>(k < live ? k : 0) * a.Hq + h * a.G) * D);
    for (int i = lane; i < a.G * D / 8; i += 32) {
      const uint4 v = __ldg(src + i);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    amax[k] = to_f32<E>(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)));
  }
  uint2 qf[NB][4 * KC];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    // column 8 nb + g: heads of a token side by side, copies behind the last
    const int col = 8 * nb + g, k = min(col / kGp, kTok - 1) < live ? min(col / kGp, kTok - 1) : 0;
    float top = amax[0];
#pragma unroll
    for (int x = 1; x < kTok; ++x) top = k == x ? amax[x] : top;
    const Unit unit = unit_of(top);
    const uint16_t* qh = q + (static_cast<size_t>(k) * a.Hq + h * a.G + (col % kGp) % a.G) * D;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
#pragma unroll
      for (int w4 = 0; w4 < 4; ++w4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(qh + (16 * (t + 4 * c)) % D + 4 * w4));
        qf[nb][4 * c + w4] = codes_of<E>(w, unit, c >= KC / 2);
      }
    }
  }
  const int32_t* bt = a.bt + static_cast<size_t>(b) * a.bt_stride + p_lo;
  // ---- scores.  A lane looks up one of 32 pages, two steps ahead of their bounds' use.
  auto look = [&](int j0) {
    int page = -1;
    if (j0 + lane < count) {
      page = __ldg(bt + j0 + lane);
      if (page < 0 || page >= a.num_pages) {
        report_error(a.err, kDevErrBadPage);
        page = -1;
      }
    }
    return page;
  };
  auto scale_of = [&](int page) { return page < 0 ? 0.f : __ldg(a.bscale + static_cast<size_t>(page) * a.H + h); };
  uint4 raw[kJobs][2];
  // job j of a warp: pages 16 s + g and 16 s + 8 + g, chunk t + 4 c
  auto fetch = [&](int page) {
#pragma unroll
    for (int j = 0; j < kJobs; ++j) {
      const int job = warp * kJobs + j, s = job / KC, c = job % KC;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int pg = __shfl_sync(0xffffffffu, page, 16 * s + 8 * e + g);
        raw[j][e] = pg < 0 ? make_uint4(0, 0, 0, 0)
                           : __ldg(reinterpret_cast<const uint4*>(a.bounds + (static_cast<size_t>(pg) * a.H + h) * 2 * D) + t + 4 * c);
      }
    }
  };
  // this lane's tokens, from `mine` on, and their candidates
  constexpr int kMine = kGp == 1 ? 2 : 1;
  const int mine = kMine * t;
  int lo[kMine], hi[kMine];
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const long long at = at0 + mine + x;
    lo[x] = a.window > 0 ? static_cast<int>(max(0ll, at + 1 - a.window) / a.ps) : 0;
    hi[x] = at >= 0 ? static_cast<int>(at / a.ps) : -1;
  }
  int page = look(0), page_next = look(32);
  float scale = scale_of(page);
  fetch(page);
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += 32) {
    auto& frag = s_frag[j0 >> 5 & 1];
#pragma unroll
    for (int j = 0; j < kJobs; ++j) {
      const int job = warp * kJobs + j, s = job / KC, c = job % KC;
      const uint32_t w0[4] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w};
      const uint32_t w1[4] = {raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 f;
        widen<true>(w0[k], f.x, f.z);
        widen<true>(w1[k], f.y, f.w);
        frag[s][4 * c + k][lane] = f;
      }
    }
    fetch(page_next);
    const float scale_next = scale_of(page_next);
    const int page_after = look(j0 + 64);
    // one barrier a step: the fragments that are written next were read before it
    __syncthreads();
    if (live > 0) {
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        float d[NB][4] = {};
#pragma unroll
        for (int k = 0; k < 4 * KC; ++k) {
          const uint4 x = frag[s][k][lane];
          const uint32_t f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(d[nb], f, qf[nb][k].x, qf[nb][k].y);
        }
        // lane (g, t) has pages g, g + 8 of columns 2t, 2t + 1 of each eight: the largest of a token's
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float sc = __shfl_sync(0xffffffffu, scale, 16 * s + 8 * e + g);
          const int pg = __shfl_sync(0xffffffffu, page, 16 * s + 8 * e + g), j = j0 + 16 * s + 8 * e + g;
          auto put = [&](int x, float v) {
            const int p = p_lo + j;
            uint32_t key = 0;
            if (pg >= 0 && p >= lo[x] && p <= hi[x])
              key = p - lo[x] < a.first || hi[x] - p < a.last ? kSure : key_of(v, sc);
            if (mine + x < live && j < count) keys[(mine + x) * ra.stride + j] = key;
          };
          if constexpr (kGp == 1) {
            if (t < 2) {
              put(0, d[0][2 * e]);
              put(1, d[0][2 * e + 1]);
            }
          } else if constexpr (kGp == 2) {
            put(0, fmaxf(d[0][2 * e], d[0][2 * e + 1]));
          } else {
            float m[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              m[nb] = fmaxf(d[nb][2 * e], d[nb][2 * e + 1]);
              m[nb] = fmaxf(m[nb], __shfl_xor_sync(0xffffffffu, m[nb], 1));
              if constexpr (kGp >= 8) m[nb] = fmaxf(m[nb], __shfl_xor_sync(0xffffffffu, m[nb], 2));
            }
            if constexpr (kGp == 16) {
              if (t == 0) put(0, fmaxf(m[0], m[1]));
            } else if constexpr (kGp == 8) {
              if (t < 2) put(0, t == 0 ? m[0] : m[1]);
            } else {
              const float m1 = __shfl_xor_sync(0xffffffffu, m[0], 3), m2 = __shfl_xor_sync(0xffffffffu, m[1], 2);
              put(0, t == 0 ? m[0] : t == 1 ? m1 : t == 2 ? m2 : m[1]);
            }
          }
        }
      }
    }
    page = page_next;
    scale = scale_next;
    page_next = page_after;
  }
  __syncwarp();
  // ---- each token's choice
#pragma unroll 1
  for (int k = 0; k < live; ++k) {
    const uint32_t* key_of_token = keys + k * ra.stride;
    Spread x = {0xFFFFFFFFu, 0u, 0, 0};
    for (int i = lane; i < count; i += 32) x.take(key_of_token[i]);
    x.warp_all();
    Search find;
    bool more = find.begin(x, a.n);
#pragma unroll 1
    while (more) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hist[32 * i + lane] = 0;
      __syncwarp();
      for (int i = lane; i < count; i += 32) {
        const int d = find.digit(key_of_token[i]);
        if (d >= 0) atomicAdd(&hist[d], 1u);
      }
      __syncwarp();
      more = find.next(hist);
      __syncwarp();
    }
    int32_t* out = a.out + (static_cast<size_t>(t0 + i0 + k) * a.H + h) * a.n;
    int done = 0, left = find.need;
    for (int i = 0; i < count; i += 32) {
      const uint32_t key = i + lane < count ? key_of_token[i + lane] : 0;
      const uint32_t eq = __ballot_sync(0xffffffffu, key == find.above && key != 0);
      const bool take = key > find.above || (eq >> lane & 1 && __popc(eq & ((1u << lane) - 1)) < left);
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (take) out[done + __popc(taken & ((1u << lane) - 1))] = p_lo + i + lane;
      left -= min(left, __popc(eq));
      done += __popc(taken);
    }
    for (int i = done + lane; i < a.n; i += 32) out[i] = -1;
    __syncwarp();
  }
}

template <typename E, int D, int kGp>
cudaError_t go_rows(RowsArgs r, cudaStream_t stream) {
  constexpr int kTok = kGp >= 4 ? 16 / kGp : 4;
  auto kernel = select_rows_kernel<E, D, kGp>;
  r.tiles = r.s.T / (kTok * kRowWarps) + r.s.B;
  const size_t smem = static_cast<size_t>(kRowWarps) * kTok * r.stride * 4;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(r.tiles) * r.s.H);
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, r);
}

template <typename E, int D>
cudaError_t pick_rows(const RowsArgs& r, int gp, cudaStream_t s) {
  switch (gp) {
    case 1: return go_rows<E, D, 1>(r, s);
    case 2: return go_rows<E, D, 2>(r, s);
    case 4: return go_rows<E, D, 4>(r, s);
    case 8: return go_rows<E, D, 8>(r, s);
    default: return go_rows<E, D, 16>(r, s);
  }
}

template <typename E, int D, int NB>
cudaError_t go(const SelectArgs& a, int C, cudaStream_t stream) {
  auto kernel = select_pages_kernel<E, D, NB>;
  const size_t smem = static_cast<size_t>((a.bt_stride + C - 1) / C) * 4;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T) * a.H * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename E, int D>
cudaError_t pick(const SelectArgs& a, int C, cudaStream_t s) {
  return a.G <= 8 ? go<E, D, 1>(a, C, s) : go<E, D, 2>(a, C, s);
}

}  // namespace

cudaError_t launch_select_pages(const qpkv_select_pages_params& p, cudaStream_t stream) {
  SelectArgs a;
  a.B = p.num_seqs, a.T = p.num_tokens, a.Hq = p.num_heads_q, a.H = p.num_heads_kv, a.G = p.num_heads_q / p.num_heads_kv;
  a.ps = p.page_size, a.num_pages = p.num_pages, a.bt_stride = p.bt_stride;
  a.n = p.num_selected, a.first = p.first, a.last = p.last, a.window = p.window;
  a.cu = p.cu_seqlens_q, a.lens = p.seqlens_kv, a.bt = p.block_table;
  a.q = p.q, a.bounds = static_cast<const int8_t*>(p.k_bounds), a.bscale = p.bound_scale;
  a.out = p.selected, a.err = p.error_word;
  // blocks of a row: as many as leave an SM two, of 64 pages at least
  const long long rows = static_cast<long long>(a.T) * a.H;
  int C = 1;
  while (C < 8 && ((rows * C * 2 <= 2 * 152 && a.bt_stride / (2 * C) >= 64) || (a.bt_stride + C - 1) / C > kMaxKeys)) C *= 2;
  const bool f16 = p.dtype == QPKV_DTYPE_F16;
  // several queries a sequence, enough of them, and a warp's keys in shared memory, by
  // the width of the table.  4 pieces, 28 heads over 4: 43 us, a block a token 72; behind
  // wider tables, which leave an SM fewer blocks, 62 (1,408 pages) and 102 (2,800), from
  // 5,633 on a block a token.  Drafts of 64 requests come here too, and not always for
  // their good: of 2, 5 and 8, 64 heads over 8: 56, 60 and 64, a block a token 30, 58 and 87
  int gp = 1;
  while (gp < a.G) gp *= 2;
  const int tok = gp >= 4 ? 16 / gp : 4;
  if (gp <= 16 && p.max_seqlen_q != 1 && a.T >= 2 * a.B && rows >= 2 * 152 * tok && static_cast<long long>(a.bt_stride) * tok * kRowWarps <= kRowKeys) {
    RowsArgs r;
    r.s = a;
    r.stride = a.bt_stride;
    if (p.head_dim == 64) return f16 ? pick_rows<__half, 64>(r, gp, stream) : pick_rows<__nv_bfloat16, 64>(r, gp, stream);
    return f16 ? pick_rows<__half, 128>(r, gp, stream) : pick_rows<__nv_bfloat16, 128>(r, gp, stream);
  }
  if (p.head_dim == 64) return f16 ? pick<__half, 64>(a, C, stream) : pick<__nv_bfloat16, 64>(a, C, stream);
  return f16 ? pick<__half, 128>(a, C, stream) : pick<__nv_bfloat16, 128>(a, C, stream);
}

}  // namespace qpkv
