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
// Each cached byte is needed once per tile of query rows and then thrown away,
// so the kernel is bound by HBM and built to keep loads in flight: warps work
// alone (no block barrier after the start), each streaming groups of 16
// tokens of one kv head through a ring of its own that TMA fills: two lanes
// issue the K and the V box (16 rows, swizzled) in one instruction.  Measured
// on the decode batch of 64 requests (537 MB), loads alone: 16-byte cp.async
// 138 us (4 TB/s whatever the depth), TMA boxes from every warp 82 us (6.7
// TB/s).  Tokens (and dims)
// are the 16 rows of m16n8k16 and query rows its 8 columns, so the converted
// codes serve NB tiles of 8 query rows and 8 rows (most decode) waste nothing:
//   S^T = K Q^T      a thread holds 16-byte chunks t and t + 4 of tokens g and
//                    g + 8, whose dims are the k index in an order Q follows
//   O^T += V^T P^T   thread (g, t) holds chunk g of tokens 2t, 2t + 1, 2t + 8,
//                    2t + 9; P^T is the transposed S^T (movmatrix)
// (g = lane / 4, t = lane % 4).  E4M3 and INT8 codes are exact in f16; a bf16
// query row enters as f16 times a power of two that puts its largest element
// in [2^14, 2^15), exact for everything within 2^-31 of it.  P is f16 (2^-11
// relative); statistics and O are float32.
//
// The value scale joins the running maximum: with y = x log2(e) + log2(vs)
// P = 2^(y - m) multiplies raw codes, and the denominator takes P / vs.  m is
// 7 below the maximum when it is set and moves only when some y exceeds it by
// more than 15: P <= 2^15 stays in f16's range, and keys down to 2^-21 of the
// largest keep all 11 bits (a value of 448 may meet one of 2^-9).
//
// Work is split without a plan, so that lengths may change on the device (and
// in a captured graph): all (sequence, kv head, row tile, 16-token group)
// units in a row are cut into equal runs, one per warp.  A run that covers a
// whole (sequence, head, tile) writes the output; pieces go to the workspace
// (at most two per warp: the one it begins with and the one it ends with) and
// the join kernel adds them up in the order of the runs.
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

constexpr int kWarps = 4;               // per block
constexpr int kGroup = 16;              // tokens of a unit
constexpr int kMinRun = 4;              // units of a run at least (64 tokens)
constexpr uint32_t kBadPageMark = 0x7FFFDEADu;   // in the place of a key scale: skip the group

struct SplitArgs {
  Page8Args p;
  int workers;             // warps / side
  int side;                // kv heads that neighbouring warps take over the same tokens
  int tile;                // query rows of a tile (8 NB), and of a piece in the workspace
  float* part_o;           // [2 * workers][tile][D]
  float2* part_ml;         // [2 * workers][tile] (m, l)
  TokenInfo* info;         // [T]
};

// Units of sequence b: groups [g0, g0 + ng) for each of nt row tiles and Hkv heads.
struct Span {
  int t0, n, len, g0, ng, nt;
};

__device__ __forceinline__ Span span_of(const Page8Args& a, int tile, int b, int* err) {
  Span s = {0, 0, 0, 0, 0, 0};
  Rows r = rows_of(a, b, err);
  s.t0 = r.t0;
  s.n = r.n;
  s.len = r.len;
  if (r.n <= 0 || r.n * a.G > a.split_rows) return s;   // none, or in tiles of 128
  const int hi = row_hi(a, r, r.n - 1), lo = row_lo(a, r, 0);
  if (hi > lo) {
    s.g0 = lo / kGroup;
    s.ng = (hi + kGroup - 1) / kGroup - s.g0;
    s.nt = (r.n * a.G + tile - 1) / tile;
  }
  return s;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
// Over the eight lanes with the same lane % 4.
__device__ __forceinline__ float col_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float col_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// Transposes an 8 x 8 matrix of 16-bit elements: lane (g, t) gives elements
// (g, 2t), (g, 2t + 1) and gets (2t, g), (2t + 1, g).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Blocks per SM and ring stages: more query rows take registers from warps,
// and the ring gets what shared memory the warps leave.
template <int D, int NB>
struct Shape {
  static constexpr int kBlocks = NB == 1 ? 4 : NB == 2 ? 3 : 2;
  static constexpr int kStages = NB == 1 ? 2 : 4;
  static constexpr int kStage = 2 * kGroup * D;      // K and V of a group
  // Three tiles keep the query fragments, each lane's own, in shared memory: 32
  // requests of 2,500 tokens with 20 rows took 61.5 us with these 48 registers
  // too (255 in all), 58.5 without.  (12 warps an SM, 168 registers, then spill:
  // 94 us; the next group's scores beside this group's softmax: 61.4.)
  static constexpr bool kQShared = NB == 3;
  static constexpr int kQBytes = kQShared ? NB * (D / 16) * 32 * 8 : 0;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kBytes = kWarps * (kWarpBytes + kQBytes) + 1024;
};

struct RowInfo {
  int lo, hi;         // keys the row sees
  float sc;           // logit multiplier
  float slope, at;    // bias: slope * (j - at), log2 units; at and j from the end of the
                      // cache, as float32 holds no odd position beyond 2^24
};

template <typename E, int D, bool kInt8, bool kCap, bool kBias, int NB>
__global__ void __launch_bounds__(kWarps * 32, (Shape<D, NB>::kBlocks))
    attend_split_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ SplitArgs sa) {
  using Sh = Shape<D, NB>;
  constexpr int kStages = Sh::kStages;
  constexpr int KS = D / 16;      // k steps of K Q^T
  constexpr int NT = D / 16;      // 16-dim tiles of O: rows g, g + 8 are dims 2i, 2i + 1 of chunk g
  constexpr int KC = D / 64;      // 16-byte chunks of a token a thread copies
  constexpr int VB = D / 8;       // bytes of a V token a thread copies
  constexpr int VW = VB / 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ long long s_prefix[kWarps * 32 + 1];
  __shared__ long long w_sum[kWarps];
  __shared__ RowInfo s_rows[kWarps][8 * NB];
  const Page8Args& a = sa.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&s_full[warp][s], 1);
    fence_mbar_init();
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  // No early launch of the dependents: join blocks that wait on an SM kept
  // blocks of this kernel's next launch off it (107 us a call against 95).
  griddep_wait();

  // ---- units before each block of `per` sequences
  const int hgroups = a.Hkv / sa.side;
  const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
  {
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Span s = span_of(a, 8 * NB, b, blockIdx.x == 0 ? a.err : nullptr);
      mine += static_cast<long long>(s.ng) * s.nt * hgroups;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
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
  for (int tok = blockIdx.x + gridDim.x * tid; tok < a.T; tok += gridDim.x * kWarps * 32) {
    const int b = seq_of_token(a.cu, a.B, tok);
    const Span s = span_of(a, 8 * NB, b, nullptr);
    if (s.n * a.G > a.split_rows) continue;   // the tiled form's
    TokenInfo x;
    x.u0 = s_prefix[b / per];
    for (int c = b / per * per; c < b; ++c) {
      const Span y = span_of(a, 8 * NB, c, nullptr);
      x.u0 += static_cast<long long>(y.ng) * y.nt * hgroups;
    }
    x.run = run;
    x.ng = s.n > 0 && tok >= s.t0 && tok < s.t0 + s.n ? s.ng : -1;
    x.stride = s.ng;
    x.nt = s.nt;
    x.r0 = (tok - s.t0) * a.G;
    x.kind = 0;
    sa.info[tok] = x;
  }
  const int me = blockIdx.x * kWarps + warp;
  const int worker = me / sa.side;
  long long u = worker * run;
  const long long u_end = u + run < total ? u + run : total;
  const long long u_begin = u;
  if (u >= u_end) return;

  uint8_t* ring = smem + warp * Sh::kWarpBytes;
  uint64_t* full = s_full[warp];
  uint2* sq = reinterpret_cast<uint2*>(smem + kWarps * Sh::kWarpBytes + warp * Sh::kQBytes) + lane;
  RowInfo* ri = s_rows[warp];
  int in_st = 0, out_st = 0;     // ring stages of the next copy and the next use
  uint32_t out_phase = 0;        // phase of the stage in use
  // a thread's pieces of a stage, as TMA's swizzle places them
  const uint32_t ka = D == 128 ? g * 128 + ((t ^ g) << 4) : g * 64 + ((t ^ (g >> 1)) << 4);
  const uint32_t va = D == 128 ? 2 * t * 128 + (((g ^ (2 * t)) & 7) << 4) : 2 * t * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
  const uint32_t vb = D == 128 ? (2 * t + 1) * 128 + (((g ^ (2 * t + 1)) & 7) << 4) : va + 64;
  // the sequence of unit u
  int b;
  long long before;
  {
    int lo = 0, hi = kWarps * 32 - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (u < s_prefix[mid + 1]) hi = mid; else lo = mid + 1;
    }
    b = lo * per;
    before = s_prefix[lo];
  }
  Span sp = span_of(a, 8 * NB, b, nullptr);

  while (u < u_end) {
    long long in_b = static_cast<long long>(sp.ng) * sp.nt * hgroups;
    while (u >= before + in_b) {   // a run may cross into later sequences
      before += in_b;
      ++b;
      sp = span_of(a, 8 * NB, b, nullptr);
      in_b = static_cast<long long>(sp.ng) * sp.nt * hgroups;
    }
    const long long local = u - before;
    const int task = static_cast<int>(local / sp.ng);
    const int first = static_cast<int>(local - static_cast<long long>(task) * sp.ng);
    const int hg = task / sp.nt, rt = task - hg * sp.nt, h = hg * sa.side + me % sa.side;
    const int count = static_cast<int>(min(static_cast<long long>(sp.ng - first), u_end - u));
    const bool whole_task = count == sp.ng;
    const size_t piece = 2 * static_cast<size_t>(me) + (u == u_begin ? 0 : 1);
    // from the newest group back: with a distance bias the scores then fall, and
    // the running maximum is set once instead of moving with every group
    const int glast = sp.g0 + first + count - 1;
    const int live_rows = min(8 * NB, sp.n * a.G - rt * 8 * NB);

    // ---- the ring.  Lane l looks up group 32 k + l of the run: its row in the
    // pools and its two scales, 32 groups at a time.
    const int32_t* bt = a.bt + static_cast<size_t>(b) * a.bt_stride;
    const int gpp = a.ps / kGroup;
    const int hc = a.hnd ? 0 : h;
    int at = -1;                       // first row of the group, -1: a bad page
    float next_ks = 0.f, next_vs = 0.f;
    auto lookup = [&](int i0) {
      const int i = i0 + lane;
      at = -1;
      if (i < count) {
        const int gi = glast - i, pg = gi / gpp;
        const int page = __ldg(bt + pg);
        if (page >= 0 && page < a.num_pages) {
          at = (a.hnd ? page * a.Hkv + h : page) * a.ps + (gi - pg * gpp) * kGroup;
          const size_t sx = static_cast<size_t>(page) * a.Hkv + h;
          next_ks = __ldg(a.ks + sx);
          next_vs = __ldg(a.vs + sx);
        } else {
          report_error(a.err, kDevErrBadPage);
        }
      }
    };
    auto issue = [&](int i) {
      if (i < count) {
        if ((i & 31) == 0) lookup(i);
        const int row = __shfl_sync(0xffffffffu, at, i & 31);
        if (row >= 0) {
          if (lane == 0) mbar_arrive_expect_tx(&full[in_st], Sh::kStage);
          __syncwarp();
          if (lane < 2)
            tma_load_3d(ring + in_st * Sh::kStage + lane * (kGroup * D), lane == 0 ? &k_map : &v_map, &full[in_st], 0, hc, row);
          __syncwarp();
        } else if (lane == 0) {
          mbar_arrive(&full[in_st]);   // nothing comes; the stage is skipped
        }
        in_st = in_st + 1 == kStages ? 0 : in_st + 1;
      }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- Q: column g of tile nb is row rt * 8 NB + 8 nb + g, query r / G, head h * G + r % G
    uint32_t qf[Sh::kQShared ? 1 : NB][KS][2];
    int all_lo = 0, all_hi = INT_MAX;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int nq = Sh::kQShared ? 0 : nb;
      const int r = 8 * nb + g;
      const bool live = r < live_rows;
      const int rr = rt * 8 * NB + (live ? r : live_rows - 1);   // dead rows: zeros with the last row's limits
      const int i = rr / a.G, head = h * a.G + (rr - i * a.G);
      Rows rows;
      rows.t0 = sp.t0, rows.n = sp.n, rows.len = sp.len;
      rows.prefix = a.prefix != nullptr ? __ldg(a.prefix + b) : 0;
      const E* src = static_cast<const E*>(a.q) + (static_cast<size_t>(sp.t0 + i) * a.Hq + head) * D;
      uint2 raw[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int dim = (k < 4 ? 16 * t : 16 * (t + 4)) + 4 * (k & 3);
        raw[k] = live ? __ldg(reinterpret_cast<const uint2*>(src + dim)) : make_uint2(0, 0);
      }
      float inv = 1.f;
      if constexpr (std::is_same<E, __half>::value) {
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[nq][k][0] = raw[k].x, qf[nq][k][1] = raw[k].y;
      } else {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[k].x << 16)), fabsf(__uint_as_float(raw[k].x & 0xFFFF0000u))));
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[k].y << 16)), fabsf(__uint_as_float(raw[k].y & 0xFFFF0000u))));
        }
        const float mul = q_to_f16_scale(quad_max(amax), &inv);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[nq][k][0] = f32x2_to_f16x2(__uint_as_float(raw[k].x & 0xFFFF0000u) * mul, __uint_as_float(raw[k].x << 16) * mul);
          qf[nq][k][1] = f32x2_to_f16x2(__uint_as_float(raw[k].y & 0xFFFF0000u) * mul, __uint_as_float(raw[k].y << 16) * mul);
        }
      }
      if constexpr (Sh::kQShared) {
#pragma unroll
        for (int k = 0; k < KS; ++k) sq[(nb * KS + k) * 32] = make_uint2(qf[0][k][0], qf[0][k][1]);
      }
      const int hi = row_hi(a, rows, i), lo = row_lo(a, rows, i);
      all_lo = max(all_lo, lo);
      all_hi = min(all_hi, hi);
      if (t == 0) {
        RowInfo x;
        x.lo = lo;
        x.hi = hi;
        x.sc = inv * (kCap ? a.scale_cap : a.scale_log2);
        x.slope = kBias ? __ldg(a.slopes + head) * kLog2e : 0.f;
        x.at = static_cast<float>(i - sp.n);
        ri[r] = x;
      }
    }
    // keys that every row of the tile sees
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
    }
    __syncwarp();
    float sc[NB][2];    // columns 2t, 2t + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) sc[nb][0] = ri[8 * nb + 2 * t].sc, sc[nb][1] = ri[8 * nb + 2 * t + 1].sc;

    float O[NB][NT][4];
    float m[NB][2], l[NB][2];   // m is 0 until the row has seen a key
    uint32_t seen = 0;          // bit 2 nb + x: it has
    bool fresh = true;          // some row has not (the same in all lanes)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < NT; ++i) O[nb][i][0] = O[nb][i][1] = O[nb][i][2] = O[nb][i][3] = 0.f;
      m[nb][0] = m[nb][1] = 0.f;
      l[nb][0] = l[nb][1] = 0.f;
    }

    float blk_ks = 0.f, blk_lv = 0.f, blk_rvs = 1.f;   // of the 32 groups at hand, one per lane
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      if ((i & 31) == 0) {     // before the copies of the next 32 groups are issued
        const float vs = fmaxf(next_vs, kMinScale);
        blk_ks = at >= 0 ? next_ks : __uint_as_float(kBadPageMark);
        blk_lv = log2f(vs);
        blk_rvs = 1.f / vs;
      }
      issue(i + kStages - 1);
      const float ks = __shfl_sync(0xffffffffu, blk_ks, i & 31);
      const float lv = __shfl_sync(0xffffffffu, blk_lv, i & 31);
      const float rvs = __shfl_sync(0xffffffffu, blk_rvs, i & 31);
      if (!mbar_wait(&full[out_st], out_phase)) {
        if (lane == 0) report_error(a.err, kDevErrTimeout);
        // the copies still on their way land (or are given up) before the warp ends
        for (int k = 1; k < kStages && i + k < count; ++k) {
          out_phase ^= out_st + 1 == kStages;
          out_st = out_st + 1 == kStages ? 0 : out_st + 1;
          mbar_wait(&full[out_st], out_phase);
        }
        return;
      }
      __syncwarp();
      const uint8_t* src = ring + out_st * Sh::kStage;
      out_phase ^= out_st + 1 == kStages;
      out_st = out_st + 1 == kStages ? 0 : out_st + 1;
      if (__float_as_uint(ks) != kBadPageMark) {
        uint4 kx[2 * KC];       // chunks t, t + 4 of tokens g, g + 8
#pragma unroll
        for (int c = 0; c < 2 * KC; ++c)
          kx[c] = *reinterpret_cast<const uint4*>(src + (ka ^ ((c >> 1) * 64)) + (c & 1) * 8 * D);
        float s[NB][4] = {};     // token g: columns 2t, 2t + 1; token g + 8: the same
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint32_t w0[4] = {kx[2 * c].x, kx[2 * c].y, kx[2 * c].z, kx[2 * c].w};
          const uint32_t w1[4] = {kx[2 * c + 1].x, kx[2 * c + 1].y, kx[2 * c + 1].z, kx[2 * c + 1].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[4];
            widen<kInt8>(w0[k], f[0], f[2]);
            widen<kInt8>(w1[k], f[1], f[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if constexpr (Sh::kQShared) {
                const uint2 q = sq[(nb * KS + 4 * c + k) * 32];
                mma16816(s[nb], f, q.x, q.y);
              } else {
                mma16816(s[nb], f, qf[nb][4 * c + k][0], qf[nb][4 * c + k][1]);
              }
            }
          }
        }
        const uint8_t* vsrc = src + kGroup * D;
        uint32_t vw[4][VW];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint8_t* vp = vsrc + (c & 1 ? vb : va) + (c >> 1) * 8 * D;
          if constexpr (VB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(vp);
            vw[c][0] = x.x, vw[c][1] = x.y, vw[c][VW - 2] = x.z, vw[c][VW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vp);
            vw[c][0] = x.x, vw[c][1] = x.y;
          }
        }
        // ---- y - m in log2 units, y with log2 of the value scale
        const int j0 = (glast - i) * kGroup;
        float z[NB][4];
        bool up = fresh;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = sc[nb][x] * ks, off = lv - m[nb][x];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = z[nb][2 * e + x];
              v = s[nb][2 * e + x];
              float o = off;
              if constexpr (kBias) {
                const RowInfo& q = ri[8 * nb + 2 * t + x];
                o = fmaf(q.slope, static_cast<float>(j0 + g + 8 * e - sp.len) - q.at, o);
              }
              if constexpr (kCap) v = fmaf(a.cap_log2, a.far_cap ? tanh_far(v * f) : tanh_of(v * f), o);
              else v = fmaf(v, f, o);
            }
          }
        }
        if (j0 < all_lo || j0 + kGroup > all_hi) {   // some row does not see some key
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const RowInfo& q = ri[8 * nb + 2 * t + (e & 1)];
              const int j = j0 + g + 8 * (e >> 1);
              if (j < q.lo || j >= q.hi) z[nb][e] = -INFINITY;
            }
          }
          if (!kInt8) {   // P = 0 does not cancel a NaN code of a token behind the last
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (j0 + 2 * t + (c & 1) + 8 * (c >> 1) >= sp.len) {
#pragma unroll
                for (int k = 0; k < VW; ++k) vw[c][k] = 0;
              }
            }
          }
        }
        // a row's first key, or one that exceeds the range of P
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          up |= fmaxf(fmaxf(z[nb][0], z[nb][1]), fmaxf(z[nb][2], z[nb][3])) > kMaxP;
        if (__any_sync(0xffffffffu, up)) {
          uint32_t now = 0;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const bool was = seen >> (2 * nb + x) & 1;
              // the row's maximum so far lies between m + kSetP and m + kMaxP: m only grows
              const float top = col_max(fmaxf(z[nb][x], z[nb][2 + x])) - kSetP;
              const float d = was ? fmaxf(top, 0.f) : top;      // the move of m
              if (d > -INFINITY) {
                now |= 1u << (2 * nb + x);
                m[nb][x] += d;
                z[nb][x] -= d;
                z[nb][2 + x] -= d;
                const float f = was ? fast_exp2(-d) : 0.f;
                l[nb][x] *= f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  O[nb][n][x] *= f;
                  O[nb][n][2 + x] *= f;
                }
              }
            }
          }
          seen |= now;
          fresh = __any_sync(0xffffffffu, seen != (1u << 2 * NB) - 1);
        }
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = fast_exp2(z[nb][e]);
          l[nb][0] = fmaf(p[0] + p[2], rvs, l[nb][0]);
          l[nb][1] = fmaf(p[1] + p[3], rvs, l[nb][1]);
          pf[nb][0] = transpose8(f32x2_to_f16x2(p[1], p[0]));
          pf[nb][1] = transpose8(f32x2_to_f16x2(p[3], p[2]));
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          uint32_t f[4], d[4];
          widen<kInt8>(__byte_perm(vw[0][k], vw[1][k], 0x5140), f[0], f[1]);
          widen<kInt8>(__byte_perm(vw[2][k], vw[3][k], 0x5140), f[2], f[3]);
          widen<kInt8>(__byte_perm(vw[0][k], vw[1][k], 0x7362), d[0], d[1]);
          widen<kInt8>(__byte_perm(vw[2][k], vw[3][k], 0x7362), d[2], d[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(O[nb][2 * k], f, pf[nb][0], pf[nb][1]);
            mma16816(O[nb][2 * k + 1], d, pf[nb][0], pf[nb][1]);
          }
        }
      }
      __syncwarp();   // the stage may be filled again
    }
    // ---- the run's part of this task: dims [VB g, VB g + VB) of columns 2t, 2t + 1.
    // l = 0: no key seen; NaN (of a NaN score, which moves no m) goes into o and lse.
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * nb + 2 * t + x;
        const float lsum = col_sum(l[nb][x]);
        if (r >= live_rows) continue;
        if (whole_task) {
          const int rr = rt * 8 * NB + r, i = rr / a.G, head = h * a.G + (rr - i * a.G);
          const size_t row = static_cast<size_t>(sp.t0 + i) * a.Hq + head;
          const float so = lsum == 0.f ? 0.f : 1.f / lsum;
          uint32_t w[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) w[n] = pack_out<E>(O[nb][n][2 + x] * so, O[nb][n][x] * so);
          uint4* out = reinterpret_cast<uint4*>(static_cast<E*>(a.o) + row * D + VB * g);
#pragma unroll
          for (int n = 0; n < NT / 4; ++n) out[n] = make_uint4(w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]);
          if (g == 0 && a.lse != nullptr)
            a.lse[row] = lsum == 0.f ? -INFINITY : (m[nb][x] + log2f(lsum)) * kLn2;
        } else {
          float4* out = reinterpret_cast<float4*>(sa.part_o + (piece * (8 * NB) + r) * D + VB * g);
#pragma unroll
          for (int n = 0; n < NT / 2; ++n)
            out[n] = make_float4(O[nb][2 * n][x], O[nb][2 * n][2 + x], O[nb][2 * n + 1][x], O[nb][2 * n + 1][2 + x]);
          if (g == 0) sa.part_ml[piece * (8 * NB) + r] = make_float2(lsum == 0.f ? -INFINITY : m[nb][x], lsum);
        }
      }
    }
    __syncwarp();
    u += count;
  }
}

// Adds up the pieces of a (token, head) in the order of the runs, and gives
// rows that see no key their zeros.  kPer warps share a row: a long context is
// cut into hundreds of pieces when there are few rows (2 requests of 115k
// tokens: one warp per row took 41 us).  With kPer = 1, for many rows, a warp
// takes 32 heads of a token, of which few have pieces.
struct JoinArgs {
  int T, Hq, G;
  const TokenInfo* info;
  struct {
    const float* o;
    const float2* ml;
    int tile, side;
  } set[2];          // by TokenInfo::kind
  void* o;
  float* lse;
};

template <typename E, int D, int kPer>
__global__ void __launch_bounds__(kPer > 8 ? 32 * kPer : 256) attend_join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int EPL = D / 32;
  constexpr int kAll = kPer > 8 ? kPer : 8;   // warps of the block
  __shared__ float s_o[kAll][D];
  __shared__ float s_l[kAll];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kPer;
  const long long w = blockIdx.x * static_cast<long long>(kAll / kPer) + warp / kPer;
  const int heads = kPer == 1 ? 32 : 1;
  const int per_tok = (a.Hq + heads - 1) / heads;
  const int tok = static_cast<int>(w / per_tok), head0 = static_cast<int>(w - static_cast<long long>(tok) * per_tok) * heads;
  TokenInfo x;
  x.ng = -1;
  if (tok < a.T) x = a.info[tok];
  // the runs of this lane's head (all lanes the same with heads = 1)
  int w0 = 0, w1 = 0, cut = 0;
  const int my = head0 + (heads > 1 ? lane : 0);
  if (x.ng > 0 && my < a.Hq) {
    const int tile = a.set[x.kind].tile, side = a.set[x.kind].side;
    const int h = my / a.G, r = x.r0 + (my - h * a.G);
    const long long u0 = x.u0 + (static_cast<long long>(h / side) * x.nt + r / tile) * x.stride;
    w0 = static_cast<int>(u0 / x.run);
    w1 = static_cast<int>((u0 + x.ng - 1) / x.run);
    cut = u0 != w0 * x.run;
  }
  // x.ng < 0: a row behind the last sequence; w0 = w1: written whole by its run
  uint32_t todo = __ballot_sync(0xffffffffu, my < a.Hq && (x.ng == 0 || (x.ng > 0 && w0 != w1)));
  if (heads == 1) todo &= 1u;
  while (kPer > 1 || todo != 0) {
    const int from = kPer > 1 ? 0 : __ffs(todo) - 1;
    const bool write = todo != 0;
    const int head = head0 + (heads > 1 ? from : 0);
    const int k0 = __shfl_sync(0xffffffffu, w0, from), k1 = __shfl_sync(0xffffffffu, w1, from);
    const int k_cut = __shfl_sync(0xffffffffu, cut, from);
    todo &= todo - 1;
    float acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
    float M = -INFINITY, l = 0.f;
    if (write && x.ng > 0) {
      const auto& set = a.set[x.kind];
      const int h = head / a.G, r = x.r0 + (head - h * a.G), pr = r % set.tile;
      auto piece = [&](int k) {
        return (2 * (static_cast<size_t>(k) * set.side + h % set.side) + (k == k0 ? k_cut : 0)) * set.tile + pr;
      };
      for (int k = k0 + lane; k <= k1; k += 32) M = fmaxf(M, set.ml[piece(k)].x);
      M = warp_max(M);
      if (M > -INFINITY) {
#pragma unroll 4
        for (int k = k0 + part; k <= k1; k += kPer) {
          const size_t at = piece(k);
          const float2 ml = set.ml[at];
          const float f = fast_exp2(ml.x - M);   // a piece that saw nothing: m = -inf, f = 0
          l = fmaf(ml.y, f, l);
          const float* src = set.o + at * D + lane * EPL;
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[e] = fmaf(src[e], f, acc[e]);
        }
      }
    }
    if constexpr (kPer > 1) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_o[warp][lane * EPL + e] = acc[e];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (part != 0) return;
#pragma unroll
      for (int k = 1; k < kPer; ++k) {
        l += s_l[warp + k];
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] += s_o[warp + k][lane * EPL + e];
      }
    }
    if (write) {
      const size_t row = static_cast<size_t>(tok) * a.Hq + head;
      const float so = l == 0.f ? 0.f : 1.f / l;
      E* out = static_cast<E*>(a.o) + row * D + lane * EPL;
#pragma unroll
      for (int e = 0; e < EPL; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack_out<E>(acc[e + 1] * so, acc[e] * so);
      if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    }
    if (kPer > 1) return;
  }
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename E, int D, bool kInt8, bool kCap, bool kBias, int NB>
cudaError_t go(SplitArgs& a, int sms, cudaStream_t s) {
  using Sh = Shape<D, NB>;
  constexpr size_t smem = Sh::kBytes;
  auto kernel = attend_split_kernel<E, D, kInt8, kCap, kBias, NB>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(sms * Sh::kBlocks);
  a.workers = static_cast<int>(blocks) * kWarps / a.side;   // side divides kWarps * 2, blocks is even
  CUtensorMap km, vm;
  if (!pool_map(a.p, D, a.p.k, kGroup, &km) || !pool_map(a.p, D, a.p.v, kGroup, &vm)) return cudaErrorInvalidValue;
  return launch(kernel, blocks, kWarps * 32, smem, s, km, vm, a);
}

template <typename E, int D, bool kInt8, bool kCap, bool kBias>
cudaError_t pick3(SplitArgs& a, int sms, cudaStream_t s) {
  switch (a.tile / 8) {
    case 1: return go<E, D, kInt8, kCap, kBias, 1>(a, sms, s);
    case 2: return go<E, D, kInt8, kCap, kBias, 2>(a, sms, s);
    default: return go<E, D, kInt8, kCap, kBias, 3>(a, sms, s);
  }
}

template <typename E, int D, bool kInt8>
cudaError_t pick2(SplitArgs& a, int sms, cudaStream_t s) {
  const bool cap = a.p.cap_log2 > 0.f, bias = a.p.slopes != nullptr;
  if (cap) return bias ? pick3<E, D, kInt8, true, true>(a, sms, s) : pick3<E, D, kInt8, true, false>(a, sms, s);
  return bias ? pick3<E, D, kInt8, false, true>(a, sms, s) : pick3<E, D, kInt8, false, false>(a, sms, s);
}

template <typename E>
cudaError_t pick(SplitArgs& a, int D, bool int8, int sms, cudaStream_t s) {
  if (D == 64) return int8 ? pick2<E, 64, true>(a, sms, s) : pick2<E, 64, false>(a, sms, s);
  return int8 ? pick2<E, 128, true>(a, sms, s) : pick2<E, 128, false>(a, sms, s);
}

template <typename E, int D>
cudaError_t join(const JoinArgs& a, int sms, cudaStream_t s) {
  // warps per row: as many as leave each scheduler eight at most
  const long long rows = static_cast<long long>(a.T) * a.Hq;
  if (rows <= sms) return launch(attend_join_kernel<E, D, 16>, static_cast<unsigned>(rows), 512, 0, s, a);
  if (rows <= sms * 4ll) return launch(attend_join_kernel<E, D, 8>, static_cast<unsigned>(rows), 256, 0, s, a);
  if (rows <= sms * 64ll) return launch(attend_join_kernel<E, D, 2>, static_cast<unsigned>((rows + 3) / 4), 256, 0, s, a);
  const long long warps = static_cast<long long>(a.T) * ((a.Hq + 31) / 32);
  return launch(attend_join_kernel<E, D, 1>, static_cast<unsigned>((warps + 7) / 8), 256, 0, s, a);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Which forms a call needs, by sizes the host knows: the split form takes up
// to kSplitRows query rows of a (sequence, kv head); with a bound on a
// sequence's queries above that the tiled form takes the larger ones, and all
// of them when there is one sequence.
constexpr int kSplitRows = 24;
struct Plan {
  bool split, tiled;
  int tile, split_rows;
};
Plan plan_for(int B, int T, int max_q, int G) {
  Plan p;
  const long long rows = static_cast<long long>(max_q > 0 && max_q < T ? max_q : T) * G;
  p.tiled = rows > kSplitRows && G <= 128;
  p.split = !p.tiled || B > 1;
  p.tile = 8 * (rows <= 8 ? 1 : rows <= 16 ? 2 : 3);
  p.split_rows = !p.tiled ? INT_MAX : p.split ? kSplitRows : -1;
  return p;
}

// The workspace's arrays: the tokens' places, pieces of O and (m, l) of the
// split form, the same of the tiled one.
struct Sizes {
  size_t info, o, ml, to, tml;
  size_t total() const { return info + o + ml + to + tml; }
};
Sizes sizes(const Plan& p, int T, int D, int sms) {
  Sizes s = {};
  s.info = up256(static_cast<size_t>(T) * sizeof(TokenInfo));
  if (p.split) {
    const int blocks = p.tile == 8 ? Shape<128, 1>::kBlocks : p.tile == 16 ? Shape<128, 2>::kBlocks : Shape<128, 3>::kBlocks;
    const size_t rows = static_cast<size_t>(2) * sms * blocks * kWarps * p.tile;
    s.o = up256(rows * D * sizeof(float));
    s.ml = up256(rows * sizeof(float2));
  }
  if (p.tiled) {
    const size_t rows = static_cast<size_t>(2) * sms * 256;
    s.to = up256(rows * D * sizeof(float));
    s.tml = up256(rows * sizeof(float2));
  }
  return s;
}

}  // namespace

size_t attend_page8_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  // whatever max_seqlen_q will be
  size_t most = 0;
  const int G = Hq / Hkv;
  for (int q = 1; ; q = q * 2 < T ? q * 2 : T) {
    const size_t n = sizes(plan_for(B, T, q, G), T, D, kAttendMaxSms).total();
    most = n > most ? n : most;
    if (q >= T || static_cast<long long>(q) * G > 2 * kSplitRows) break;
  }
  const size_t n = sizes(plan_for(B, T, T, G), T, D, kAttendMaxSms).total();
  return n > most ? n : most;
}

cudaError_t launch_attend_page8(const qpkv_attend_page8_params& p, cudaStream_t stream) {
  SplitArgs a;
  a.p = page8_args(p);
  int sms = sm_count();
  if (sms > kAttendMaxSms) sms = kAttendMaxSms;
  const Plan plan = plan_for(p.num_seqs, p.num_tokens, p.max_seqlen_q, a.p.G);
  a.p.split_rows = plan.split_rows;
  a.side = a.p.Hkv % 8 == 0 ? 8 : a.p.Hkv % 4 == 0 ? 4 : a.p.Hkv % 2 == 0 ? 2 : 1;
  a.tile = plan.tile;
  const Sizes sz = sizes(plan, p.num_tokens, p.head_dim, sms);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.info = reinterpret_cast<TokenInfo*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + sz.info);
  a.part_ml = reinterpret_cast<float2*>(ws + sz.info + sz.o);
  TileArgs t;
  t.p = a.p;
  t.tq = a.p.G <= 128 ? 128 / a.p.G : 1;
  t.info = a.info;
  t.part_o = reinterpret_cast<float*>(ws + sz.info + sz.o + sz.ml);
  t.part_ml = reinterpret_cast<float2*>(ws + sz.info + sz.o + sz.ml + sz.to);
  const bool int8 = p.format == QPKV_FORMAT_INT8, f16 = p.dtype == QPKV_DTYPE_F16;
  cudaError_t e = cudaSuccess;
  if (plan.split) {
    const int even = sms - (sms & 1);   // an even number of blocks
    e = f16 ? pick<__half>(a, p.head_dim, int8, even, stream) : pick<__nv_bfloat16>(a, p.head_dim, int8, even, stream);
  }
  if (e == cudaSuccess && plan.tiled) e = launch_attend_tiles(t, p.head_dim, int8, f16, sms, stream);
  if (e != cudaSuccess) return e;
  JoinArgs j;
  j.T = p.num_tokens, j.Hq = p.num_heads_q, j.G = a.p.G;
  j.info = a.info;
  j.set[0] = {a.part_o, a.part_ml, a.tile, a.side};
  j.set[1] = {t.part_o, t.part_ml, 256, 1};
  j.o = p.o, j.lse = p.lse;
  if (f16) return p.head_dim == 64 ? join<__half, 64>(j, sms, stream) : join<__half, 128>(j, sms, stream);
  return p.head_dim == 64 ? join<__nv_bfloat16, 64>(j, sms, stream) : join<__nv_bfloat16, 128>(j, sms, stream);
}

}  // namespace qpkv
