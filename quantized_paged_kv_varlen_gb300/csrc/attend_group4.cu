// Attention over the paged cache in 4 bits (group4.cuh has the layout): the
// split form for few query rows, and for rows that attend to selected pages.
//
//   x(r, j) = sm_scale * k_mul * q_r . K_j     K, V: codes times scales
//   x = cap * tanh(x / cap)        with a cap
//   x = x + slope_h * (j - at_r)   with a bias, at_r the position of row r
//   o_r = v_mul * sum_j softmax_j(x(r, .)) V_j,  j in [lo_r, hi_r)
//
// Every row's visible keys are one interval (page8.cuh), or with selected pages
// the part of it that lies in them.
//
// The work is cut as in attend_page8.cu: units of 16 tokens in equal runs, one
// per warp, warps on their own, pieces joined afterwards.  A unit is two untiled
// bulk copies (K and V, 9 D bytes each, codes and scales together), issued by
// two lanes into a ring of the warp's own.  With selected pages every (token,
// kv head, row tile) is a task of as many units as the list has room for; units
// that list nothing are passed over.
//
// Tokens are the rows of m16n8k16, query rows its 8 columns.  A code times its
// scale is exact in f16, so fragments are one conversion and one packed product
// per two values:
//   S^T = K Q^T      a thread holds a quarter of tokens p(g) and p(g) + 8, whose
//                    dims are the k index in an order Q follows
//   O^T += V^T P^T   thread (g, t) holds chunk g of the four tokens p(2t), p(2t +
//                    1) and those + 8; codes of two tokens are interleaved nibble
//                    by nibble, so that one conversion gives a dim of both
// (g = lane / 4, t = lane % 4, p(2t + e) = 2t + (e xor t % 2): neighbouring rows of
// 64 bytes alternate for both reads, so that banks differ.)
//
// A NaN scale of V must reach only the rows that see its token, and P = 0 does
// not cancel it: where some row of a tile does not see some key of a unit, such
// scales count as zero and the rows that see the token get their NaN afterwards.
#include <cooperative_groups.h>
#include <climits>
#include <type_traits>

#include "attend_split.cuh"
#include "common.cuh"
#include "group4.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kNone = -(1 << 30);       // in the place of a group's first key: it has none

struct SplitArgs {
  Page8Args p;
  int workers;             // warps / side
  int side;                // kv heads that neighbouring warps take over the same tokens
  int tile;                // query rows of a tile (8 NB), and of a piece in the workspace
  float* part_o;           // [2 * workers][tile][D]
  float2* part_ml;         // [2 * workers][tile] (m, l)
  TokenInfo* info;         // [T]
  // the kernel of whole tasks
  const int32_t* sel;      // [T, Hkv, n_sel] or null: all keys
  int n_sel;
  int nt, cluster;         // row tiles of a (sequence or token, kv head), blocks of a task
  long long tasks;         // 0: the split form
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

// Blocks per SM and ring stages: more query rows take registers from warps,
// and the ring gets what shared memory the warps leave.
template <int D, int NB>
struct Shape {
  static constexpr int kBlocks = NB == 1 ? 4 : NB == 2 ? 3 : 2;
  static constexpr int kPair = 2;       // groups of a step
  static constexpr int kStages = 2;
  static constexpr int kBlock = Group4<D>::kBlock;
  static constexpr int kStage = 2 * kPair * kBlock;  // K and V of its groups
  // two tiles and three keep the query fragments, each lane's own, in shared memory
  static constexpr bool kQShared = NB >= 2;
  static constexpr int kQBytes = kQShared ? NB * (D / 16) * 32 * 8 : 0;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kBytes = kWarps * (kWarpBytes + kQBytes) + 1024;
};

// A warp's ring of copies.
struct Ring {
  uint8_t* ring;
  uint64_t* full;
  int in_st, out_st;      // stages of the next copy and the next use
  uint32_t out_phase;     // phase of the stage in use
};

// Groups [first, first + count) of a row tile of a (sequence, kv head), or of a
// (token, kv head) with its list.
struct Task {
  Span sp;
  int b, h, rt, first, count;
  int live_rows;
  bool listed;
  int token_i;            // listed: the query,
  const int32_t* list;    // its pages,
  int lo, hi;             // the keys that it sees
};

template <int D, int NB>
struct Sums {
  float O[NB][D / 16][4];
  float m[NB][2], l[NB][2];   // m is 0 until the row has seen a key; l of this lane's tokens
};

// The warp's part of a task, from its first copies to its last product; false
// after a wait that ran out.
template <typename E, int D, bool kCap, bool kBias, int NB>
__device__ __forceinline__ bool attend_groups(const SplitArgs& sa, const Task& tk, Ring& rg, RowInfo* ri, uint2* sq, Sums<D, NB>& sums) {
  using Sh = Shape<D, NB>;
  using L = Group4<D>;
  constexpr int kStages = Sh::kStages, kPair = Sh::kPair;
  constexpr int KS = D / 16;      // k steps of K Q^T
  constexpr int NT = D / 16;      // 16-dim tiles of O: rows g, g + 8 are dims 2i, 2i + 1 of chunk g
  constexpr int KW = D / 32;      // words of a K token a thread takes
  constexpr int VB = D / 8;       // dims of a V token a thread takes
  constexpr int VW = VB / 8;      // words of them
  const Page8Args& a = sa.p;
  const Span& sp = tk.sp;
  const int b = tk.b, h = tk.h, rt = tk.rt, count = tk.count, live_rows = tk.live_rows, token_i = tk.token_i;
  const bool listed = tk.listed;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, gpp = a.ps / kGroup;
  // from the newest group back: with a distance bias the scores then fall, and
  // the running maximum is set once instead of moving with every group
  const int glast = (listed ? 0 : sp.g0) + tk.first + count - 1;
  // a thread's pieces of a block
  const int pg = 2 * (g >> 1) + ((g ^ (g >> 1)) & 1);                 // p(g)
  const int p0 = 2 * t + (t & 1), p1 = 2 * t + 1 - (t & 1);           // p(2t), p(2t + 1)
  const int ka = pg * L::kRow + t * (KW * 4);
  const int ksa = L::kScaleAt + pg * L::kScales + t * (D / 64);
  const int vsa = L::kScaleAt + (D == 128 ? g : g >> 1);
  auto& O = sums.O;
  auto& m = sums.m;
  auto& l = sums.l;

  // ---- the ring.  Lane l looks up group 32 k + l of the run: its block in the
  // pools and its first key, 32 groups at a time.
  const int32_t* bt = a.bt + static_cast<size_t>(b) * a.bt_stride;
  int at = -1, next_j0 = 0;         // block of the group (-1: no keys), its first key
  auto lookup = [&](int i0) {
    const int i = i0 + lane;
    at = -1;
    if (i < count) {
      const int gi = glast - i, slot = gi / gpp, in = gi - slot * gpp;
      int no = slot;                 // the page's place in the table row
      if (listed) {
        no = __ldg(tk.list + slot);
        if (no < 0 || no >= a.bt_stride || static_cast<long long>(no) * a.ps >= sp.len) {
          if (no != -1) report_error(a.err, kDevErrBadIndex);
          return;
        }
      }
      next_j0 = no * a.ps + in * kGroup;
      if (listed && (next_j0 >= tk.hi || next_j0 + kGroup <= tk.lo)) return;
      const int page = __ldg(bt + no);
      if (page >= 0 && page < a.num_pages) {
        at = (page * a.Hkv + h) * gpp + in;
      } else {
        report_error(a.err, kDevErrBadPage);
      }
    }
  };
  // copies of step i, a lane for K or V of a group
  auto issue = [&](int i) {
    const int base = i * kPair;
    if (base < count) {
      if ((base & 31) == 0) lookup(base);
      __syncwarp();
      const int block = __shfl_sync(0xffffffffu, at, (base + (lane >> 1)) & 31);
      const bool mine = lane < 2 * kPair && block >= 0;
      const int copies = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) mbar_arrive_expect_tx(&rg.full[rg.in_st], copies * Sh::kBlock);
      __syncwarp();
      if (mine)
        bulk_load(rg.ring + rg.in_st * Sh::kStage + lane * Sh::kBlock,
                  (lane & 1 ? a.v : a.k) + static_cast<size_t>(block) * Sh::kBlock, Sh::kBlock, &rg.full[rg.in_st]);
      __syncwarp();
      rg.in_st = rg.in_st + 1 == kStages ? 0 : rg.in_st + 1;
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  const float kmul = a.ks != nullptr ? __ldg(a.ks + h) : 1.f;

  // ---- Q: column g of tile nb is row rt * 8 NB + 8 nb + g, query r / G, head h * G + r % G
  uint32_t qf[Sh::kQShared ? 1 : NB][KS][2];
  int all_lo = 0, all_hi = INT_MAX;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int nq = Sh::kQShared ? 0 : nb;
    const int r = 8 * nb + g;
    const bool live = r < live_rows;
    const int rr = rt * 8 * NB + (live ? r : live_rows - 1);   // dead rows: zeros with the last row's limits
    const int i = listed ? token_i : rr / a.G, head = h * a.G + (listed ? rr : rr - i * a.G);
    Rows rows;
    rows.t0 = sp.t0, rows.n = sp.n, rows.len = sp.len;
    rows.prefix = a.prefix != nullptr ? __ldg(a.prefix + b) : 0;
    const E* src = static_cast<const E*>(a.q) + (static_cast<size_t>(sp.t0 + i) * a.Hq + head) * D;
    uint2 raw[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int dim = D / 4 * t + 4 * k;
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
      x.sc = inv * (kCap ? a.scale_cap : a.scale_log2) * kmul;
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

  uint32_t seen = 0;          // bit 2 nb + x: it has
  bool fresh = true;          // some row has not (the same in all lanes)
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int i = 0; i < NT; ++i) O[nb][i][0] = O[nb][i][1] = O[nb][i][2] = O[nb][i][3] = 0.f;
    m[nb][0] = m[nb][1] = 0.f;
    l[nb][0] = l[nb][1] = 0.f;
  }

  int blk_j0 = kNone;         // of the 32 groups at hand, one per lane
  const int steps = (count + kPair - 1) / kPair;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const int base = i * kPair;
    if ((base & 31) == 0) blk_j0 = at >= 0 ? next_j0 : kNone;     // before the copies of the next 32 groups are issued
    issue(i + kStages - 1);
    int j0[kPair];
    bool some = false, part = false;     // some group has keys; some row does not see some key
#pragma unroll
    for (int p = 0; p < kPair; ++p) {
      j0[p] = __shfl_sync(0xffffffffu, blk_j0, (base + p) & 31);
      some |= j0[p] >= 0;
      part |= j0[p] < all_lo || j0[p] + kGroup > all_hi;
    }
    if (!mbar_wait(&rg.full[rg.out_st], rg.out_phase)) {
      if (lane == 0) report_error(a.err, kDevErrTimeout);
      // the copies still on their way land (or are given up) before the warp ends
      for (int k = 1; k < kStages && i + k < steps; ++k) {
        rg.out_phase ^= rg.out_st + 1 == kStages;
        rg.out_st = rg.out_st + 1 == kStages ? 0 : rg.out_st + 1;
        mbar_wait(&rg.full[rg.out_st], rg.out_phase);
      }
      return false;
    }
    __syncwarp();
    const uint8_t* src = rg.ring + rg.out_st * Sh::kStage;
    rg.out_phase ^= rg.out_st + 1 == kStages;
    rg.out_st = rg.out_st + 1 == kStages ? 0 : rg.out_st + 1;
    if (some) {
      // ---- scores: token p(g): columns 2t, 2t + 1; token p(g) + 8: the same.  A group
      // without keys is computed from whatever lies there and masked like other keys.
      float z[kPair][NB][4];
      float s[kPair][NB][4] = {};
      {
        uint32_t w[kPair][2][KW], sc2[kPair][2][D / 64];
#pragma unroll
        for (int p = 0; p < kPair; ++p) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* kp = src + 2 * p * Sh::kBlock + ka + e * 8 * L::kRow;
            const uint8_t* ksp = src + 2 * p * Sh::kBlock + ksa + e * 8 * L::kScales;
            if constexpr (KW == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(kp);
              w[p][e][0] = x.x, w[p][e][1] = x.y, w[p][e][KW - 2] = x.z, w[p][e][KW - 1] = x.w;
              const uint32_t both = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ksp));
              sc2[p][e][0] = __byte_perm(both, 0, 0x1010), sc2[p][e][D / 64 - 1] = __byte_perm(both, 0, 0x3232);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kp);
              w[p][e][0] = x.x, w[p][e][1] = x.y;
              sc2[p][e][0] = e4m3_to_f16x2_both(*ksp);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          uint2 q[2][NB];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if constexpr (Sh::kQShared) q[x][nb] = sq[(nb * KS + 2 * k + x) * 32];
              else q[x][nb] = make_uint2(qf[nb][2 * k + x][0], qf[nb][2 * k + x][1]);
            }
          }
#pragma unroll
          for (int p = 0; p < kPair; ++p) {
            uint32_t f0[4], f1[4];
            e2m1x8_to_f16(w[p][0][k], f0);
            e2m1x8_to_f16(w[p][1][k], f1);
#pragma unroll
            for (int e = 0; e < 4; ++e) f0[e] = f16x2_mul(f0[e], sc2[p][0][k >> 1]), f1[e] = f16x2_mul(f1[e], sc2[p][1][k >> 1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t f[4] = {f0[2 * x], f1[2 * x], f0[2 * x + 1], f1[2 * x + 1]};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816(s[p][nb], f, q[x][nb].x, q[x][nb].y);
            }
          }
        }
      }
      // y - m in log2 units.  A capped score is good to 2^-19 of itself at any cap, which
      // shows where a row sees few keys; where none comes near the cap its series is enough.
      auto score = [&](auto series) {
#pragma unroll
        for (int p = 0; p < kPair; ++p) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v = s[p][nb][2 * e + x];
                float o = -m[nb][x];
                if constexpr (kBias) {
                  const RowInfo& q = ri[8 * nb + 2 * t + x];
                  o = fmaf(q.slope, static_cast<float>(j0[p] + pg + 8 * e - sp.len) - q.at, o);
                }
                if constexpr (kCap) {
                  const float c = v * sc[nb][x];
                  z[p][nb][2 * e + x] = fmaf(a.cap_log2, decltype(series)::value ? tanh_series(c) : tanh_far(c), o);
                } else {
                  z[p][nb][2 * e + x] = fmaf(v, sc[nb][x], o);
                }
              }
            }
          }
        }
      };
      bool near = true;
      if constexpr (kCap) {
        bool small = true;
#pragma unroll
        for (int p = 0; p < kPair; ++p) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) small &= fabsf(s[p][nb][e] * sc[nb][e & 1]) < 0.5f;
          }
        }
        near = __all_sync(0xffffffffu, small);
      }
      if (near) score(std::true_type()); else score(std::false_type());
      if (part) {
#pragma unroll
        for (int p = 0; p < kPair; ++p) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const RowInfo& q = ri[8 * nb + 2 * t + (e & 1)];
              const int j = j0[p] + pg + 8 * (e >> 1);
              if (j < q.lo || j >= q.hi) z[p][nb][e] = -INFINITY;
            }
          }
        }
      }
      // a row's first key, or one that exceeds the range of P
      bool up = fresh;
#pragma unroll
      for (int p = 0; p < kPair; ++p) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) up |= fmaxf(fmax3(z[p][nb][0], z[p][nb][1], z[p][nb][2]), z[p][nb][3]) > kMaxP;
      }
      if (__any_sync(0xffffffffu, up)) {
        uint32_t now = 0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool was = seen >> (2 * nb + x) & 1;
            // the row's maximum so far lies between m + kSetP and m + kMaxP: m only grows
            float most = fmaxf(z[0][nb][x], z[0][nb][2 + x]);
#pragma unroll
            for (int p = 1; p < kPair; ++p) most = fmax3(most, z[p][nb][x], z[p][nb][2 + x]);
            const float top = col_max(most) - kSetP;
            const float d = was ? fmaxf(top, 0.f) : top;      // the move of m
            if (d > -INFINITY) {
              now |= 1u << (2 * nb + x);
              m[nb][x] += d;
#pragma unroll
              for (int p = 0; p < kPair; ++p) z[p][nb][x] -= d, z[p][nb][2 + x] -= d;
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
      // ---- O^T += V^T P^T
#pragma unroll
      for (int p = 0; p < kPair; ++p) {
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fast_exp2(z[p][nb][e]);
          l[nb][0] += v[0] + v[2];
          l[nb][1] += v[1] + v[3];
          pf[nb][0] = transpose8(f32x2_to_f16x2(v[1], v[0]));
          pf[nb][1] = transpose8(f32x2_to_f16x2(v[3], v[2]));
        }
        const uint8_t* vsrc = src + (2 * p + 1) * Sh::kBlock;
        uint32_t vw[4][VW], vsc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = (c & 1 ? p1 : p0) + (c >> 1) * 8;
          const uint8_t* vp = vsrc + r * L::kRow + VW * 4 * g;
          if constexpr (VW == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(vp);
            vw[c][0] = x.x, vw[c][VW - 1] = x.y;
          } else {
            vw[c][0] = *reinterpret_cast<const uint32_t*>(vp);
          }
          vsc[c] = vsrc[vsa + r * L::kScales];
        }
        uint32_t nan = 0;      // tokens whose V scale of this chunk is NaN and counts as zero
        if (part) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // tokens behind the last may hold anything
            if (j0[p] < 0 || j0[p] + (c & 1 ? p1 : p0) + 8 * (c >> 1) >= sp.len) {
              vsc[c] = 0;
#pragma unroll
              for (int k = 0; k < VW; ++k) vw[c][k] = 0;
            }
            if (e4m3_is_nan(vsc[c])) nan |= 1u << ((c & 1 ? p1 : p0) + 8 * (c >> 1)), vsc[c] = 0;
          }
          nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
          nan |= __shfl_xor_sync(0xffffffffu, nan, 2);
        }
        const uint32_t v01 = e4m3x2_to_f16x2(static_cast<uint16_t>(vsc[0] | vsc[1] << 8));
        const uint32_t v23 = e4m3x2_to_f16x2(static_cast<uint16_t>(vsc[2] | vsc[3] << 8));
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          // byte i: dims 8 k + 2 i (even) and 8 k + 2 i + 1 (odd) of two tokens
          uint32_t even[2][4], odd[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t u0 = vw[2 * e][k], u1 = vw[2 * e + 1][k], low = 0x0F0F0F0Fu, f = e ? v23 : v01;
            e2m1x8_to_f16((u0 & low) | (u1 << 4 & ~low), even[e]);
            e2m1x8_to_f16((u0 >> 4 & low) | (u1 & ~low), odd[e]);
#pragma unroll
            for (int i = 0; i < 4; ++i) even[e][i] = f16x2_mul(even[e][i], f), odd[e][i] = f16x2_mul(odd[e][i], f);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f[4] = {even[0][i], odd[0][i], even[1][i], odd[1][i]};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(O[nb][4 * k + i], f, pf[nb][0], pf[nb][1]);
          }
        }
        if (__builtin_expect(nan != 0, 0)) {     // differs between chunks; no shuffle in here
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const RowInfo& q = ri[8 * nb + 2 * t + x];
              for (uint32_t bits = nan; bits != 0; bits &= bits - 1) {
                const int j = j0[p] + __ffs(bits) - 1;
                if (j < q.lo || j >= q.hi) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n) O[nb][n][x] = O[nb][n][2 + x] = __uint_as_float(0x7FC00000u);
              }
            }
          }
        }
      }
    }
    __syncwarp();   // the stage may be filled again
  }
  return true;
}

template <typename E, int D, bool kCap, bool kBias, int NB>
__global__ void __launch_bounds__(kWarps * 32, (Shape<D, NB>::kBlocks))
    attend_split4_kernel(const __grid_constant__ SplitArgs sa) {
  using Sh = Shape<D, NB>;
  constexpr int kStages = Sh::kStages;
  constexpr int NT = D / 16;      // tiles of O
  constexpr int VB = D / 8;       // dims of a chunk
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
  }
  // No early launch of the dependents: join blocks that wait on an SM keep
  // blocks of this kernel's next launch off it.
  griddep_wait();

  const int hgroups = a.Hkv / sa.side;
  const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
  long long total;
  {
    // ---- units before each block of `per` sequences
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
    total = s_prefix[kWarps * 32];
  }
  long long run = (total + sa.workers - 1) / sa.workers;
  run = run < kMinRun ? kMinRun : run;
  for (int tok = blockIdx.x + gridDim.x * tid; tok < a.T; tok += gridDim.x * kWarps * 32) {
    const int b = seq_of_token(a.cu, a.B, tok);
    TokenInfo x;
    x.run = run;
    x.kind = 0;
    const Span s = span_of(a, 8 * NB, b, nullptr);
    if (s.n * a.G > a.split_rows) continue;   // the tiled form's
    x.u0 = s_prefix[b / per];
    for (int c = b / per * per; c < b; ++c) {
      const Span y = span_of(a, 8 * NB, c, nullptr);
      x.u0 += static_cast<long long>(y.ng) * y.nt * hgroups;
    }
    x.ng = s.n > 0 && tok >= s.t0 && tok < s.t0 + s.n ? s.ng : -1;
    x.stride = s.ng;
    x.nt = s.nt;
    x.r0 = (tok - s.t0) * a.G;
    sa.info[tok] = x;
  }
  const int me = blockIdx.x * kWarps + warp;
  const int worker = me / sa.side;
  long long u = worker * run;
  const long long u_end = u + run < total ? u + run : total;
  const long long u_begin = u;
  if (u >= u_end) return;

  Ring ring = {smem + warp * Sh::kWarpBytes, s_full[warp], 0, 0, 0};
  uint2* sq = reinterpret_cast<uint2*>(smem + kWarps * Sh::kWarpBytes + warp * Sh::kQBytes) + lane;
  RowInfo* ri = s_rows[warp];
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
    const int ng = sp.ng, task = static_cast<int>(local / ng);
    const int first = static_cast<int>(local - static_cast<long long>(task) * ng);
    const int hg = task / sp.nt, rt = task - hg * sp.nt, h = hg * sa.side + me % sa.side;
    const int count = static_cast<int>(min(static_cast<long long>(ng - first), u_end - u));
    const bool whole_task = count == ng;
    const size_t piece = 2 * static_cast<size_t>(me) + (u == u_begin ? 0 : 1);
    const int live_rows = min(8 * NB, sp.n * a.G - rt * 8 * NB);
    const Task part = {sp, b, h, rt, first, count, live_rows, false, 0, nullptr, 0, 0};
    Sums<D, NB> sums;
    if (!attend_groups<E, D, kCap, kBias, NB>(sa, part, ring, ri, sq, sums)) return;
    auto& O = sums.O;
    auto& m = sums.m;
    auto& l = sums.l;
    const float vmul = a.vs != nullptr ? __ldg(a.vs + h) : 1.f;

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
          const float so = lsum == 0.f ? 0.f : vmul / lsum;
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
            out[n] = make_float4(O[nb][2 * n][x] * vmul, O[nb][2 * n][2 + x] * vmul, O[nb][2 * n + 1][x] * vmul, O[nb][2 * n + 1][2 + x] * vmul);
          if (g == 0) sa.part_ml[piece * (8 * NB) + r] = make_float2(lsum == 0.f ? -INFINITY : m[nb][x], lsum);
        }
      }
    }
    __syncwarp();
    u += count;
  }
}

// Calls with few keys to a row (lists, short caches): a cluster of 1 to 8 blocks
// takes a whole task, its warps equal shares of the groups, and joins their sums
// through distributed shared memory: one launch, no workspace.
template <typename E, int D, bool kCap, bool kBias, int NB>
__global__ void __launch_bounds__(kWarps * 32, (Shape<D, NB>::kBlocks)) attend_whole4_kernel(const __grid_constant__ SplitArgs sa) {
  using Sh = Shape<D, NB>;
  constexpr int NT = D / 16, VB = D / 8, kRows = 8 * NB;
  constexpr int kParts = 8 * kWarps;      // at most
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t s_full[kWarps][Sh::kStages];
  __shared__ RowInfo s_rows[kWarps][kRows];
  __shared__ float2 s_ml[kWarps][kRows];
  __shared__ float s_w[kRows][kParts];    // weights of the parts
  float* s_o = reinterpret_cast<float*>(smem);     // [kWarps][kRows][D], where the rings were
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const Page8Args& a = sa.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < Sh::kStages; ++s) mbar_init(&s_full[warp][s], 1);
    fence_mbar_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  // ---- the task: (token or sequence, kv head, row tile)
  const bool listed = sa.sel != nullptr;
  long long x = blockIdx.x / C;
  Task k;
  k.rt = static_cast<int>(x % sa.nt);
  x /= sa.nt;
  k.h = static_cast<int>(x % a.Hkv);
  const int who = static_cast<int>(x / a.Hkv);
  k.listed = listed;
  k.token_i = 0;
  k.list = nullptr;
  int ng;
  if (listed) {
    k.b = warp_last_at_most(a.B, who, [&](int m) { return static_cast<long long>(__ldg(a.cu + m - 1)); });
    const Rows r = rows_of(a, k.b, blockIdx.x / C % (a.Hkv * sa.nt) == 0 && tid == 0 ? a.err : nullptr);
    k.token_i = who - r.t0;
    if (k.token_i < 0 || k.token_i >= r.n) return;      // behind the last sequence: its rows stay as they are
    k.sp = {r.t0, r.n, r.len, 0, 0, sa.nt};
    k.list = sa.sel + (static_cast<size_t>(who) * a.Hkv + k.h) * sa.n_sel;
    k.lo = row_lo(a, r, k.token_i);
    k.hi = row_hi(a, r, k.token_i);
    ng = sa.n_sel * (a.ps / kGroup);
  } else {
    k.b = who;
    const Rows r = rows_of(a, k.b, blockIdx.x / C % (a.Hkv * sa.nt) == 0 && tid == 0 ? a.err : nullptr);
    if (k.rt * kRows >= r.n * a.G) return;
    const int hi = row_hi(a, r, r.n - 1), lo = row_lo(a, r, 0);
    ng = hi > lo ? (hi + kGroup - 1) / kGroup - lo / kGroup : 0;
    k.sp = {r.t0, r.n, r.len, lo / kGroup, ng, sa.nt};
    k.lo = k.hi = 0;
  }
  // (the next row tile only where a sequence has more queries than the call's bound says)
  Ring ring = {smem + warp * Sh::kWarpBytes, s_full[warp], 0, 0, 0};
  const int rows = listed ? a.G : k.sp.n * a.G;
  for (; k.rt * kRows < rows; k.rt += sa.nt) {
    k.live_rows = min(kRows, rows - k.rt * kRows);
    // ---- this warp's share
    const int parts = C * kWarps, me = rank * kWarps + warp;
    const int share = (ng + parts * Sh::kPair - 1) / (parts * Sh::kPair) * Sh::kPair;
    k.first = min(ng, me * share);
    k.count = min(share, ng - k.first);
    Sums<D, NB> sums;
    uint2* sq = reinterpret_cast<uint2*>(smem + kWarps * Sh::kWarpBytes + warp * Sh::kQBytes) + lane;
    bool any = k.count > 0;
    // (a wait that ran out has been reported, and the outputs are undefined)
    if (any) any = attend_groups<E, D, kCap, kBias, NB>(sa, k, ring, s_rows[warp], sq, sums);
    __syncthreads();     // the rings are through
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * nb + 2 * t + c;
        const float lsum = any ? col_sum(sums.l[nb][c]) : 0.f;
        float4* out = reinterpret_cast<float4*>(s_o + (warp * kRows + r) * D + VB * g);
        if (any) {
#pragma unroll
          for (int n = 0; n < NT / 2; ++n)
            out[n] = make_float4(sums.O[nb][2 * n][c], sums.O[nb][2 * n][2 + c], sums.O[nb][2 * n + 1][c], sums.O[nb][2 * n + 1][2 + c]);
        }
        if (g == 0) s_ml[warp][r] = make_float2(lsum == 0.f ? -INFINITY : sums.m[nb][c], any ? lsum : -1.f);
      }
    }
    if (C > 1) cluster.sync(); else __syncthreads();
    // ---- weights: a lane to a part.  -inf: a part that stored no sums.  Those of every
    // other one are added, however small its weight: O may hold a NaN of V.
    const float vmul = a.vs != nullptr ? __ldg(a.vs + k.h) : 1.f;
    auto place = [&](int r) {      // row r of o and lse
      const int rr = k.rt * kRows + r, i = listed ? k.token_i : rr / a.G, head = k.h * a.G + (listed ? rr : rr - i * a.G);
      return static_cast<size_t>(k.sp.t0 + i) * a.Hq + head;
    };
    for (int r = warp; r < k.live_rows; r += kWarps) {
      float2 ml = make_float2(-INFINITY, -1.f);
      if (lane < parts) ml = *cluster.map_shared_rank(&s_ml[lane % kWarps][r], lane / kWarps);
      const float M = warp_max(ml.x);
      const bool none = ml.y <= 0.f;      // it saw nothing (NaN: it did)
      const float f = none ? 0.f : fast_exp2(ml.x - M);
      const float sum = warp_sum(none ? 0.f : ml.y * f);
      if (lane < parts) s_w[r][lane] = ml.y < 0.f ? -INFINITY : none ? 0.f : f * (vmul / sum);
      if (rank == 0 && lane == 0 && a.lse != nullptr) a.lse[place(r)] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
    __syncthreads();
    for (int i = rank * kWarps * 32 + tid; i < k.live_rows * (D / 4); i += C * kWarps * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < parts; ++p) {
        const float w = s_w[r][p];
        if (w == -INFINITY) continue;
        const float4 v = *cluster.map_shared_rank(reinterpret_cast<float4*>(s_o + ((p % kWarps) * kRows + r) * D + d), p / kWarps);
        o.x = fmaf(v.x, w, o.x), o.y = fmaf(v.y, w, o.y), o.z = fmaf(v.z, w, o.z), o.w = fmaf(v.w, w, o.w);
      }
      *reinterpret_cast<uint2*>(static_cast<E*>(a.o) + place(r) * D + d) = make_uint2(pack_out<E>(o.y, o.x), pack_out<E>(o.w, o.z));
    }
    // the next row tile's copies land where this thread has stored sums
    if (rows - k.rt * kRows > sa.nt * kRows) fence_proxy_async_smem();
    if (C > 1) cluster.sync(); else __syncthreads();     // nobody leaves while its sums are read
  }
}

constexpr size_t max_of(size_t x, size_t y) { return x > y ? x : y; }

template <typename E, int D, bool kCap, bool kBias, int NB>
cudaError_t go(SplitArgs& a, int sms, cudaStream_t s) {
  using Sh = Shape<D, NB>;
  constexpr size_t smem = Sh::kBytes;
  auto kernel = attend_split4_kernel<E, D, kCap, kBias, NB>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (a.tasks > 0) {
    constexpr size_t whole = max_of(smem, static_cast<size_t>(kWarps) * 8 * NB * D * 4 + 1024);
    auto kernel = attend_whole4_kernel<E, D, kCap, kBias, NB>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(whole));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tasks * a.cluster));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = whole;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }
  const unsigned blocks = static_cast<unsigned>(sms * Sh::kBlocks);
  a.workers = static_cast<int>(blocks) * kWarps / a.side;   // side divides kWarps * 2, blocks is even
  return launch(kernel, blocks, kWarps * 32, smem, s, a);
}

template <typename E, int D, bool kCap, bool kBias>
cudaError_t pick3(SplitArgs& a, int sms, cudaStream_t s) {
  switch (a.tile / 8) {
    case 1: return go<E, D, kCap, kBias, 1>(a, sms, s);
    case 2: return go<E, D, kCap, kBias, 2>(a, sms, s);
    default: return go<E, D, kCap, kBias, 3>(a, sms, s);
  }
}

template <typename E, int D>
cudaError_t pick2(SplitArgs& a, int sms, cudaStream_t s) {
  const bool cap = a.p.cap_log2 > 0.f, bias = a.p.slopes != nullptr;
  if (cap) return bias ? pick3<E, D, true, true>(a, sms, s) : pick3<E, D, true, false>(a, sms, s);
  return bias ? pick3<E, D, false, true>(a, sms, s) : pick3<E, D, false, false>(a, sms, s);
}

template <typename E>
cudaError_t pick(SplitArgs& a, int D, int sms, cudaStream_t s) {
  return D == 64 ? pick2<E, 64>(a, sms, s) : pick2<E, 128>(a, sms, s);
}

constexpr int kBlocks[3] = {Shape<128, 1>::kBlocks, Shape<128, 2>::kBlocks, Shape<128, 3>::kBlocks};

// Calls whose rows have few keys by what the host knows: lists, and caches whose
// table rows are short, with few query rows.
struct Whole {
  long long tasks;     // 0: not such a call
  int nt, tile, cluster;
};
Whole whole_plan(const qpkv_attend_group4_params& p, int sms) {
  Whole w = {};
  const int G = p.num_heads_q / p.num_heads_kv;
  const bool listed = p.selected != nullptr;
  const long long keys = listed ? static_cast<long long>(p.num_selected) * p.page_size
                                : static_cast<long long>(p.bt_stride) * p.page_size;
  const int max_q = p.max_seqlen_q > 0 && p.max_seqlen_q < p.num_tokens ? p.max_seqlen_q : p.num_tokens;
  const long long rows = listed ? G : static_cast<long long>(max_q) * G;
  if (!listed && rows > kSplitRows) return w;
  w.tile = 8 * (rows <= 8 ? 1 : rows <= 16 ? 2 : 3);
  w.nt = static_cast<int>((rows + w.tile - 1) / w.tile);
  w.tasks = static_cast<long long>(listed ? p.num_tokens : p.num_seqs) * p.num_heads_kv * w.nt;
  // blocks of a task while the SMs have room for them and a warp two steps
  w.cluster = 1;
  while (w.cluster < 8 && w.tasks * w.cluster * 2 <= 3ll * sms && keys / 16 >= 2 * w.cluster * kWarps * 2) w.cluster *= 2;
  // all keys: a warp's share is 16 groups at most (32 requests of 2,500 tokens with
  // three drafts, 64 groups a warp: 49 us, in the split form 47; with five 49 and 58)
  if (!listed && (keys > 16ll * 16 * w.cluster * kWarps || w.tasks > INT_MAX)) w.tasks = 0;
  return w;
}

}  // namespace

size_t attend_group4_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  // whatever max_seqlen_q will be
  const int G = Hq / Hkv;
  size_t most = 0;
  for (int q = 1; ; q = q * 2 < T ? q * 2 : T) {
    const size_t n = sizes(plan_for(B, T, q, G), T, D, kAttendMaxSms, kBlocks).total();
    most = n > most ? n : most;
    if (q >= T || static_cast<long long>(q) * G > 2 * kSplitRows) break;
  }
  const size_t n = sizes(plan_for(B, T, T, G), T, D, kAttendMaxSms, kBlocks).total();
  return n > most ? n : most;
}

static int attend_sms() {
  const int sms = sm_count();
  return sms > kAttendMaxSms ? kAttendMaxSms : sms;
}

bool attend_group4_needs_workspace(const qpkv_attend_group4_params& p) { return whole_plan(p, attend_sms()).tasks == 0; }

cudaError_t launch_attend_group4(const qpkv_attend_group4_params& p, cudaStream_t stream) {
  SplitArgs a;
  Page8Args& x = a.p;
  x.B = p.num_seqs, x.T = p.num_tokens, x.Hq = p.num_heads_q, x.Hkv = p.num_heads_kv;
  x.G = p.num_heads_q / p.num_heads_kv;
  x.ps = p.page_size, x.num_pages = p.num_pages, x.bt_stride = p.bt_stride;
  x.causal = p.causal ? 1 : 0;
  x.window = p.window;
  x.scale_log2 = p.sm_scale * kLog2e;
  x.scale_cap = p.logit_cap > 0.f ? p.sm_scale / p.logit_cap : 0.f;
  x.cap_log2 = p.logit_cap > 0.f ? p.logit_cap * kLog2e : 0.f;
  x.far_cap = p.logit_cap > kNearCap;
  x.hnd = 1;
  x.cu = p.cu_seqlens_q, x.lens = p.seqlens_kv, x.bt = p.block_table, x.prefix = p.prefix_lens;
  x.slopes = p.alibi_slopes, x.ks = p.k_mul, x.vs = p.v_mul;
  x.q = p.q;
  x.k = static_cast<const uint8_t*>(p.k_pool), x.v = static_cast<const uint8_t*>(p.v_pool);
  x.o = p.o, x.lse = p.lse, x.err = p.error_word;
  a.sel = p.selected, a.n_sel = p.num_selected;
  const int sms = attend_sms();
  const bool f16 = p.dtype == QPKV_DTYPE_F16;
  const Whole whole = whole_plan(p, sms);
  a.tasks = whole.tasks, a.nt = whole.nt, a.cluster = whole.cluster;
  if (whole.tasks > 0) {
    a.tile = whole.tile;
    return f16 ? pick<__half>(a, p.head_dim, sms, stream) : pick<__nv_bfloat16>(a, p.head_dim, sms, stream);
  }
  const Plan plan = plan_for(p.num_seqs, p.num_tokens, p.max_seqlen_q, x.G);
  x.split_rows = plan.split_rows;
  a.side = x.Hkv % 8 == 0 ? 8 : x.Hkv % 4 == 0 ? 4 : x.Hkv % 2 == 0 ? 2 : 1;
  a.tile = plan.tile;
  const Sizes sz = sizes(plan, p.num_tokens, p.head_dim, sms, kBlocks);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.info = reinterpret_cast<TokenInfo*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + sz.info);
  a.part_ml = reinterpret_cast<float2*>(ws + sz.info + sz.o);
  TileArgs t;
  t.p = x;
  t.tq = x.G <= 128 ? 128 / x.G : 1;
  t.info = a.info;
  t.part_o = reinterpret_cast<float*>(ws + sz.info + sz.o + sz.ml);
  t.part_ml = reinterpret_cast<float2*>(ws + sz.info + sz.o + sz.ml + sz.to);
  cudaError_t e = cudaSuccess;
  if (plan.split) {
    const int even = sms - (sms & 1);   // an even number of blocks
    e = f16 ? pick<__half>(a, p.head_dim, even, stream) : pick<__nv_bfloat16>(a, p.head_dim, even, stream);
  }
  if (e == cudaSuccess && plan.tiled) e = launch_attend_tiles4(t, p.head_dim, f16, sms, stream);
  if (e != cudaSuccess) return e;
  JoinArgs j;
  j.T = p.num_tokens, j.Hq = p.num_heads_q, j.G = x.G;
  j.info = a.info;
  j.set[0] = {a.part_o, a.part_ml, a.tile, a.side};
  j.set[1] = {t.part_o, t.part_ml, 256, 1};
  j.o = p.o, j.lse = p.lse;
  if (f16) return p.head_dim == 64 ? join<__half, 64>(j, sms, stream) : join<__half, 128>(j, sms, stream);
  return p.head_dim == 64 ? join<__nv_bfloat16, 64>(j, sms, stream) : join<__nv_bfloat16, 128>(j, sms, stream);
}

}  // namespace qpkv
