// Attention over the page-scaled 8-bit cache (attend_page8.cu has the
// formulas): the tiled form for many query rows, on the 5th-generation tensor
// cores.
//
// Rows of a (sequence, kv head) are its queries times the G query heads that
// share the kv head.  A tile is 128 rows of TQ = 128 / G whole queries; an
// item is a pair of tiles A and B, run side by side over one stream of 64-key
// tiles: while one tile's softmax computes its exponentials the tensor core
// works on the other, and each K/V tile is fetched and widened once for both.  One persistent CTA per SM, 15 warps:
//   warps 0-3   widen K and V codes to f16 (exact), from the raw ring into the
//               operand layouts; the item's queries as f16 (bf16 rows times a
//               power of two)
//   warps 4-7   softmax and epilogue of tile A, one thread per row
//   warps 8-11  the same for tile B
//   warps 12, 14  one thread each issues the tcgen05.mma of tile A and tile B:
//               per key tile g QK(g+1) PV(g) (one thread for both tiles took
//               3,600 cycles a step to issue 24 of them)
//   warp 13     walks the work: writes for every step what the others need (the
//               item, the scales) into a ring of eight, and issues the copies of
//               its keys, a TMA box for 16 of them, into the raw ring (loads into
//               registers by warps 0-3 took them 1,100 cycles a step to issue)
// (With the walk in every role the registers spilled, into an L1 that shared
// memory leaves 20 KB: 3.3 ms for a prompt of 8192, 32 heads.)
// TMEM: two S of 64 columns for each tile, O_A, O_B of 128; a step's f16 P
// overwrites the first half of its S.  S(g+1) is ready when the softmax of g
// ends: with 128-key tiles only one S a tile fits beside O, and the chain
// QK - softmax - PV took 5,600 cycles for 128 keys (0.76 ms for the prompt of
// 8192).  The MMAs run in issue order, so QK_X(g+2) overwrites an S only after
// PV_X(g) has read its P.
//
// The softmax reads S once, a row's 64 columns in registers: P = 2^(y - m)
// with the m at hand (see kSetP, kMaxP), and only when some y exceeds the range
// are m, O and the sums rescaled.  Key tiles go from the newest back, so that
// with a distance bias the first tile has the maximum.
//
// Work is split without a plan, as in the other form: all (item, kv head, key
// tile) units in a row are cut into equal runs, one per CTA; a run's first and
// last piece may be partial and go to the workspace for the join kernel.  Each
// (item, kv head) counts kOverhead units more than its key tiles, for its
// queries' load and its results' store (a causal prompt begins with many items
// of one key tile).  9: the prompt of 8192 took 534 us when this was measured (516
// now), against 680 (4), 631 (5), 575 (6), 544 (7), 541 (12); over thirteen
// batches of prompts and pieces 7 to 12 were within 1 %.
//
// The prompt of 8192 with options, us: plain 516, window of 1024 204, bias 627,
// cap of 50 864 (an exponential and a reciprocal a score more), both 1027, a cap
// above kNearCap 1183.
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

constexpr int kT = 128;                       // query rows of a tile
constexpr int kN = 64;                        // keys of a tile
constexpr int kGroups = kN / 16;
constexpr int kWarps = 15, kThreads = kWarps * 32;
constexpr int kSoftA = 4, kSoftB = 8, kMma = 12, kWalk = 13;   // tile B's MMAs: the warp behind kWalk
constexpr int kLoad = 128;                    // threads of the load warps
constexpr int kHalf = kT * 128;               // 16 KB: 128 rows of 64 f16 (Q)
constexpr int kHalfKv = kN * 128;             // 8 KB: 64 keys of 64 f16
constexpr int kRing = 3;                      // K and V tiles as f16
constexpr int kRaw = 3;                       // K and V tiles as codes
constexpr uint32_t kColS = 0, kColO = 256;    // S: [tile][2] of 64 columns
constexpr uint32_t kBadPageMark = 0x7FFFDEADu;   // in the place of a key scale: skip the group
// Ring of steps.  Step g is written once raw slot g - kRaw is free: those keys
// were widened, into the place of step g - kRaw - kRing, whose PVs (tile B's, or
// its passing) were through, and with them all reading of step g - kSteps.
constexpr int kSteps = 8;
static_assert(kSteps >= kRaw + kRing, "a step may be written only once nobody reads the one before it");
constexpr int kOverhead = 9;

// One step of the CTA: a key tile of one (item, kv head).
enum : int { kFirst = 1, kLast = 2, kHasB = 4, kWholeTask = 8, kEnd = 16, kAllKeys = 32 };
struct Step {
  float4 sc[kGroups]; // per 16 keys: ks, log2 vs, 1 / vs
  int at[kGroups];    // per 16 keys: first pool row, -1: no keys
  int flags;          // and the segment's number % 4 << 8
  int j0;             // first key
  int seg;            // segments (runs of steps of one (item, kv head)) before this one
  int t0, n, len, prefix;   // the sequence (Rows)
  int h, i0;          // kv head, first query of the item
  int piece;          // of the workspace, when the segment is not the whole task
};

template <int D>
struct Smem {
  static constexpr int kOp = D / 64 * kHalf;      // a tile of Q
  static constexpr int kOpKv = D / 64 * kHalfKv;  // a tile of K or V
  static constexpr int kRawTile = kN * D;         // codes of K or V
  static constexpr int kQ = 0, kK = 2 * kOp, kV = kK + kRing * kOpKv;
  static constexpr int kCodes = kV + kRing * kOpKv;
  static constexpr int kBytes = kCodes + 2 * kRaw * kRawTile + 1024;
};

struct Shared {
  uint64_t q_raw, q_full, q_free;             // the queries' copy, their f16, their last use
  uint64_t kv_full[kRing], kv_empty[kRing];
  // per tile A / B and S buffer: a softmax warp may be a step ahead of another,
  // whose arrival for its step must not be taken by that one's; and two PVs of a
  // tile may be in flight, with one barrier whose parity tells them apart for
  // nobody: a wait for the second could return behind the one before the first,
  // a wait for the first could miss its phase
  uint64_t s_full[2][2], p_ready[2][2], o_done[2][2];
  uint64_t mma_done[2];
  uint64_t step_full[kSteps];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  Step step[kSteps];
  // [segment % 4][tile][row] logit multiplier: QK runs a step ahead of a softmax,
  // so with segments of one step the queries' load is up to two ahead
  float qsc[4][2][kT];
  int s_step[2][2];                           // per tile and S buffer: its step, -1: the end
  long long seq_prefix[kThreads + 1];         // items before each thread's sequences
  long long unit_prefix[kThreads + 1];        // units before each thread's items
  long long w_sum[kWarps];
  uint32_t tmem_base;
  int abort;
};

// The polls behind a wait that is not over at once, out of line: fifteen roles'
// worth of them inline did not fit the instruction cache.
__device__ __noinline__ bool await_slow(uint64_t* bar, uint32_t parity, Shared* sh, int* err) {
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sh->abort)) return false;
    if (clock64() - t0 > kWaitTimeoutCycles) {
      sh->abort = 1;
      report_error(err, kDevErrTimeout);
      return false;
    }
  }
}

// All lanes wait, and go on converged.  (One lane polling and a shuffle of the
// outcome is slower: a shuffle takes ~230 cycles beside the other warps' polls.)
__device__ __forceinline__ bool warp_await(uint64_t* bar, uint32_t parity, Shared& sh, int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = await_slow(bar, parity, &sh, err);
  __syncwarp();
  return ok;
}

// MMAs and commits issued by one elected lane of a converged warp.  The warp
// computes the operands, which so stay in uniform registers; in code of a
// single lane each MMA first moved them there.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// Items of a sequence: pairs of tiles, none for one that the split form takes.
__device__ __forceinline__ int items_of(const TileArgs& a, const Rows& r) {
  if (r.n <= 0 || r.n * a.p.G <= a.p.split_rows) return 0;
  return (r.n + 2 * a.tq - 1) / (2 * a.tq);
}

// Keys [lo, ...) that some row of item p sees, and how many key tiles they
// touch (from lo / kN on).
__device__ __forceinline__ int key_tiles(const TileArgs& a, const Rows& r, int p, int* lo) {
  const int i0 = p * 2 * a.tq, i1 = min(r.n, i0 + 2 * a.tq) - 1;
  const int hi = row_hi(a.p, r, i1);
  *lo = row_lo(a.p, r, i0);
  return hi > *lo ? (hi - 1) / kN - *lo / kN + 1 : 0;
}
__device__ __forceinline__ int units_of(int key_tiles) { return key_tiles > 0 ? key_tiles + kOverhead : 0; }

// A position in the list of items.
struct Item {
  int b, p, np;
  Rows r;
  __device__ __forceinline__ void seq(const TileArgs& a, int nb, int* err = nullptr) {
    b = nb;
    p = 0;
    r = rows_of(a.p, b, err);
    np = items_of(a, r);
  }
  // the idx-th item of the sequences from first on
  __device__ __forceinline__ void find(const TileArgs& a, int first, long long idx) {
    seq(a, first);
    while (idx >= np) {
      idx -= np;
      seq(a, b + 1);
    }
    p = static_cast<int>(idx);
  }
  __device__ __forceinline__ void next(const TileArgs& a) {
    if (++p < np) return;
    do {
      seq(a, b + 1);
    } while (np == 0);
  }
};

__device__ __forceinline__ int chunk_of(const long long* prefix, long long x) {
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (x < prefix[mid + 1]) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Exclusive prefix sums of one value per thread into out[0 .. kThreads].
__device__ __forceinline__ void cta_prefix(long long v, long long* out, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) sh.w_sum[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += sh.w_sum[w];
  out[threadIdx.x + 1] = v;
  if (threadIdx.x == 0) out[0] = 0;
  __syncthreads();
}

// How the work lies in threads' chunks.
struct Layout {
  int per_seq;          // sequences per thread
  long long per_item;   // items per thread
  long long run;        // units of a CTA
};

// This CTA's units as segments: key tiles of one (item, kv head).
struct Walk {
  long long u, u_begin, u_end;
  long long item_u0;     // first unit of the item
  Item it;
  int lo, nk;            // the item's first key, and its key tiles
  int h, first, count;   // kv head; steps [first, first + count) of nk, newest key tile first
  int skip;              // units of the segment
  int has_b, seg;
  int j;                 // step in the segment
  __device__ __forceinline__ void open(const TileArgs& a) {
    // from u on, the next (item, kv head) with a key tile in this run
    while (u < u_end) {
      while (u >= item_u0 + static_cast<long long>(units_of(nk)) * a.p.Hkv) {
        item_u0 += static_cast<long long>(units_of(nk)) * a.p.Hkv;
        it.next(a);
        nk = key_tiles(a, it.r, it.p, &lo);
      }
      const int per = units_of(nk);
      const long long local = u - item_u0;
      h = static_cast<int>(local / per);
      first = static_cast<int>(local - static_cast<long long>(h) * per);
      skip = static_cast<int>(min(static_cast<long long>(per - first), u_end - u));
      count = min(skip, nk - first);
      has_b = it.p * 2 * a.tq + a.tq < it.r.n;
      if (count > 0) return;
      u += skip;    // the run begins in the overhead of a task
    }
  }
  __device__ __forceinline__ void start(const TileArgs& a, const Layout& lay, const Shared& sh) {
    const long long total = sh.unit_prefix[kThreads];
    u = u_begin = blockIdx.x * lay.run;
    u_end = min(total, u + lay.run);
    seg = j = 0;
    if (u >= u_end) return;
    const int c = chunk_of(sh.unit_prefix, u);
    const long long idx = c * lay.per_item;
    const int s = chunk_of(sh.seq_prefix, idx);
    it.find(a, s * lay.per_seq, idx - sh.seq_prefix[s]);
    item_u0 = sh.unit_prefix[c];
    nk = key_tiles(a, it.r, it.p, &lo);
    open(a);
  }
  __device__ __forceinline__ bool valid() const { return u < u_end; }
  __device__ __forceinline__ int key_tile() const { return lo / kN + nk - 1 - first - j; }
  // n steps on, at most to the segment's end
  __device__ __forceinline__ void advance(const TileArgs& a, int n) {
    j += n;
    if (j < count) return;
    j = 0;
    u += skip;
    ++seg;
    open(a);
  }
};

// Scores without a cap, with one up to kNearCap, with one above: forms of their
// own, as the far caps' code beside the near ones' cost those 7 % (a prompt of
// 8192: 925 us against 860).
enum : int { kNone = 0, kNear = 1, kFar = 2 };

template <typename E, int D, bool kInt8, int kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) attend_tile_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const __grid_constant__ TileArgs ta) {
  using L = Smem<D>;
  const Page8Args& a = ta.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&sh.q_raw, 1);
    mbar_init(&sh.q_full, kLoad / 32);
    mbar_init(&sh.q_free, 2);             // both tiles' MMAs
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.kv_full[i], kLoad / 32);
      mbar_init(&sh.kv_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i][0], 2);       // QK's commit, and s_step's store
      mbar_init(&sh.s_full[i][1], 2);
      mbar_init(&sh.p_ready[i][0], 128);
      mbar_init(&sh.p_ready[i][1], 128);
      mbar_init(&sh.o_done[i][0], 1);
      mbar_init(&sh.o_done[i][1], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kLoad / 32);
    }
    for (int i = 0; i < kSteps; ++i) mbar_init(&sh.step_full[i], 1);
    mbar_init(&sh.mma_done[0], 1);
    mbar_init(&sh.mma_done[1], 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  griddep_wait();
  if (warp == kMma) tmem_alloc(&sh.tmem_base, 512);

  // ---- the split: items per sequence, key tiles per item
  Layout lay;
  lay.per_seq = (a.B + kThreads - 1) / kThreads;
  {
    const int b0 = min(a.B, tid * lay.per_seq), b1 = min(a.B, b0 + lay.per_seq);
    long long n = 0;
    for (int b = b0; b < b1; ++b) n += items_of(ta, rows_of(a, b, blockIdx.x == 0 ? a.err : nullptr));
    cta_prefix(n, sh.seq_prefix, sh);
    const long long items = sh.seq_prefix[kThreads];
    lay.per_item = (items + kThreads - 1) / kThreads;
    lay.per_item = lay.per_item < 1 ? 1 : lay.per_item;
    const long long x0 = min(items, tid * lay.per_item), x1 = min(items, x0 + lay.per_item);
    long long units = 0;
    if (x0 < x1) {
      const int s = chunk_of(sh.seq_prefix, x0);
      Item it;
      it.find(ta, s * lay.per_seq, x0 - sh.seq_prefix[s]);
      for (long long x = x0; x < x1; ++x) {
        int lo;
        units += static_cast<long long>(units_of(key_tiles(ta, it.r, it.p, &lo))) * a.Hkv;
        if (x + 1 < x1) it.next(ta);
      }
    }
    cta_prefix(units, sh.unit_prefix, sh);
    lay.run = (sh.unit_prefix[kThreads] + gridDim.x - 1) / gridDim.x;
    lay.run = lay.run < 1 ? 1 : lay.run;
  }
  // ---- the tokens' places, for the join kernel
  for (int tok = blockIdx.x + gridDim.x * tid; tok < a.T; tok += gridDim.x * kThreads) {
    const int b = seq_of_token(a.cu, a.B, tok);
    Item it;
    it.seq(ta, b);
    if (it.r.n * a.G <= a.split_rows) continue;    // the split form's
    TokenInfo x;
    x.ng = -1;
    x.stride = 0;
    x.nt = 1;
    x.kind = 1;
    x.u0 = 0;
    x.run = lay.run;
    x.r0 = 0;
    if (it.r.n > 0 && tok >= it.r.t0 && tok < it.r.t0 + it.r.n) {
      const int i = tok - it.r.t0, p = i / (2 * ta.tq), iq = i - p * 2 * ta.tq;
      int lo;
      x.ng = key_tiles(ta, it.r, p, &lo);
      x.stride = units_of(x.ng);
      x.r0 = iq / ta.tq * kT + iq % ta.tq * a.G;
      const int sc = b / lay.per_seq;
      long long idx = sh.seq_prefix[sc];
      for (int c = sc * lay.per_seq; c < b; ++c) idx += items_of(ta, rows_of(a, c, nullptr));
      idx += p;
      const long long ic = idx / lay.per_item, from = ic * lay.per_item;
      x.u0 = sh.unit_prefix[ic];
      if (from < idx) {
        const int s = chunk_of(sh.seq_prefix, from);
        it.find(ta, s * lay.per_seq, from - sh.seq_prefix[s]);
        for (long long q = from; q < idx; ++q) {
          x.u0 += static_cast<long long>(units_of(key_tiles(ta, it.r, it.p, &lo))) * a.Hkv;
          it.next(ta);
        }
      }
    }
    ta.info[tok] = x;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem_base;

  if (warp < kSoftA) {
    // --------------------------------------------------------------- widen
    constexpr int kVecs = kN * D / 16 / kLoad;       // 16-byte vectors of a tile per thread
    constexpr int kRowVecs = D / 16;                 // vectors of a row
    constexpr int kRowsPer = kLoad / kRowVecs;       // rows of one round, a multiple of 8:
                                                     // the swizzles are the same in every round
    const int row0 = tid / kRowVecs, c = tid % kRowVecs;
    int copies = 0;                                  // query loads that thread 0 has issued
    const uint32_t in0 = D == 128 ? row0 * 128 + (((c ^ row0) & 7) << 4) : row0 * 64 + (((c ^ (row0 >> 1)) & 3) << 4);
    // A vector's 16 codes are two 16-byte chunks of f16; the lanes of the second
    // 64-column half store theirs in the other order, so that the eight lanes of
    // a row cover all banks.
    const int swap = c >> 2 & 1, c0 = 2 * (c & 3);
    const uint32_t off0 = (c >> 2) * kHalfKv + row0 * 128 + ((((c0 + swap) ^ row0) & 7) << 4);
    const uint32_t off1 = (c >> 2) * kHalfKv + row0 * 128 + ((((c0 + 1 - swap) ^ row0) & 7) << 4);
    // keys without codes (`all` false: behind the last, before the window, in a bad
    // page) become zero
    auto store = [&](uint8_t* dst, const uint8_t* src, const Step& s, bool all) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int r = row0 + k * kRowsPer;
        const uint4 v = *reinterpret_cast<const uint4*>(src + in0 + k * kRowsPer * D);
        uint4 w = swap ? make_uint4(v.z, v.w, v.x, v.y) : v;
        if (!all && (s.j0 + r >= s.len || s.at[r >> 4] < 0)) w = make_uint4(0, 0, 0, 0);
        uint32_t o[8];
        widen<kInt8>(w.x, o[0], o[1]);
        widen<kInt8>(w.y, o[2], o[3]);
        widen<kInt8>(w.z, o[4], o[5]);
        widen<kInt8>(w.w, o[6], o[7]);
        *reinterpret_cast<uint4*>(dst + off0 + k * kRowsPer * 128) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + off1 + k * kRowsPer * 128) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    };
    // the pair's queries: TMA boxes of (64 dims, G heads, TQ queries), whose rows
    // are a tile's rows, then (bf16) turned into f16 in place, a thread to a row.
    // Rows behind the sequence's last are whatever the boxes bring (or were left
    // with): nothing of them is written.
    auto load_q = [&](const Step& s) -> bool {
      const int tiles = s.flags & kHasB ? 2 : 1, seg = s.seg;
      if (tid == 0) {
        mbar_arrive_expect_tx(&sh.q_raw, tiles * D * ta.tq * a.G * 2);
        for (int k = 0; k < tiles * (D / 64); ++k) {
          const int tile = k / (D / 64), half = k % (D / 64);
          tma_load_3d(smem + L::kQ + tile * L::kOp + half * kHalf, &q_map, &sh.q_raw, 64 * half, s.h * a.G,
                      s.t0 + s.i0 + tile * ta.tq);
        }
        ++copies;
      }
      __syncwarp();
      if (!warp_await(&sh.q_raw, seg & 1, sh, a.err)) return false;
      if constexpr (!std::is_same<E, __half>::value) {
        for (int tile = 0; tile < tiles; ++tile) {
          uint8_t* row = smem + L::kQ + tile * L::kOp + tid * 128;
          float amax = 0.f;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + (k >> 3) * kHalf + (((k ^ tid) & 7) << 4));
            const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              amax = fmax3(amax, fabsf(__uint_as_float(wv[q] << 16)), fabsf(__uint_as_float(wv[q] & 0xFFFF0000u)));
          }
          float inv;
          const float mul = q_to_f16_scale(amax, &inv);
          sh.qsc[seg & 3][tile][tid] = inv * (kCap ? a.scale_cap : a.scale_log2);
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            uint4* at = reinterpret_cast<uint4*>(row + (k >> 3) * kHalf + (((k ^ tid) & 7) << 4));
            const uint4 v = *at;
            uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              wv[q] = f32x2_to_f16x2(__uint_as_float(wv[q] & 0xFFFF0000u) * mul, __uint_as_float(wv[q] << 16) * mul);
            *at = make_uint4(wv[0], wv[1], wv[2], wv[3]);
          }
        }
      }
      return true;
    };

    for (int g = 0;; ++g) {
      if (!warp_await(&sh.step_full[g % kSteps], (g / kSteps) & 1, sh, a.err)) break;
      const Step& s = sh.step[g % kSteps];
      if (s.flags & kEnd) break;
      const uint32_t ph = (g / kRing) & 1;
      if (s.flags & kFirst) {
        if (!warp_await(&sh.q_free, (s.seg & 1) ^ 1, sh, a.err)) break;
        if (!load_q(s)) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
      }
      const bool all = s.flags & kAllKeys;
      const uint8_t* raw = smem + L::kCodes + (g % kRaw) * 2 * L::kRawTile;
      if (!warp_await(&sh.raw_full[g % kRaw], (g / kRaw) & 1, sh, a.err)) break;
      if (!warp_await(&sh.kv_empty[g % kRing], ph ^ 1, sh, a.err)) break;
      store(smem + L::kK + (g % kRing) * L::kOpKv, raw, s, all);
      store(smem + L::kV + (g % kRing) * L::kOpKv, raw + L::kRawTile, s, all);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.kv_full[g % kRing]);
        mbar_arrive(&sh.raw_empty[g % kRaw]);
      }
    }
    // a query load still on its way (after a wait that ran out) lands before the CTA ends
    if (tid == 0 && copies > 0) mbar_wait(&sh.q_raw, (copies - 1) & 1);
  } else if (warp == kWalk) {
    // ---------------------------------------------------------------- walk
    // Eight steps at a time, a lane for each 16 keys: the next eight are looked
    // up before the ones in hand are written as the ring's places come free.
    // (One step at a time took 2,600 cycles a step for its dependent loads, more
    // than anything else in the kernel.)
    constexpr int kBatch = 32 / kGroups;
    const int gpp = a.ps / 16, mine = lane / kGroups, grp = lane % kGroups;
    Walk w;
    w.start(ta, lay, sh);
    struct Batch {
      int n;            // steps, 0: the end
      int flags, j0;    // of the segment; first key of its first step
      int seg, t0, rows, len, prefix, h, i0, piece;
      int at;           // this lane's 16 keys
      float ks, vs;
    };
    auto fetch = [&]() {
      Batch x;
      x.n = 0;
      x.flags = kEnd;
      x.j0 = x.seg = x.t0 = x.rows = x.len = x.prefix = x.h = x.i0 = x.piece = 0;
      x.at = -1;
      x.ks = x.vs = 0.f;
      if (!w.valid()) return x;
      x.n = min(kBatch, w.count - w.j);
      x.flags = (w.has_b ? kHasB : 0) | (w.count == w.nk ? kWholeTask : 0) | (w.j == 0 ? kFirst : 0) |
                (w.j + x.n == w.count ? kLast : 0);
      x.j0 = w.key_tile() * kN;
      x.seg = w.seg;
      x.t0 = w.it.r.t0, x.rows = w.it.r.n, x.len = w.it.r.len, x.prefix = w.it.r.prefix;
      x.h = w.h;
      x.i0 = w.it.p * 2 * ta.tq;
      x.piece = 2 * blockIdx.x + (w.u == w.u_begin ? 0 : 1);
      const int gi = (x.j0 >> 4) - mine * kGroups + grp;
      // 16 keys that lie wholly before the window of every row are no keys: their
      // page may have been given back
      if (mine < x.n && gi * 16 < x.len && gi >= w.lo / 16) {
        const int pg = gi / gpp;
        const int page = __ldg(a.bt + static_cast<size_t>(w.it.b) * a.bt_stride + pg);
        if (page >= 0 && page < a.num_pages) {
          x.at = (a.hnd ? page * a.Hkv + x.h : page) * a.ps + (gi - pg * gpp) * 16;
          const size_t sx = static_cast<size_t>(page) * a.Hkv + x.h;
          x.ks = __ldg(a.ks + sx);
          x.vs = __ldg(a.vs + sx);
        } else {
          report_error(a.err, kDevErrBadPage);
        }
      }
      w.advance(ta, x.n);
      return x;
    };
    Batch x = fetch();
    bool ok = true;
    int issued = 0;
    for (int g = 0; ok;) {
      const Batch next = x.n > 0 ? fetch() : x;
      const float sv = fmaxf(x.vs, kMinScale);
      const float4 sc = make_float4(x.at >= 0 ? x.ks : __uint_as_float(kBadPageMark), log2f(sv), 1.f / sv, 0.f);
      const int n = x.n > 0 ? x.n : 1;     // the end is a step too
      for (int i = 0; i < n; ++i, ++g) {
        ok = warp_await(&sh.raw_empty[g % kRaw], ((g / kRaw) & 1) ^ 1, sh, a.err);
        if (!ok) break;
        const bool here = mine == i && x.at >= 0;
        const int keys = __popc(__ballot_sync(0xffffffffu, here && x.j0 - i * kN + grp * 16 + 16 <= x.len));
        if (!(x.flags & kEnd)) {
          // the codes: lane (i, grp) copies 16 keys of K and of V
          const int boxes = __popc(__ballot_sync(0xffffffffu, here));
          uint8_t* raw = smem + L::kCodes + (g % kRaw) * 2 * L::kRawTile + grp * 16 * D;
          if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[g % kRaw], boxes * 2 * 16 * D);
          __syncwarp();
          if (here) {
            tma_load_3d(raw, &k_map, &sh.raw_full[g % kRaw], 0, a.hnd ? 0 : x.h, x.at);
            tma_load_3d(raw + L::kRawTile, &v_map, &sh.raw_full[g % kRaw], 0, a.hnd ? 0 : x.h, x.at);
          }
          issued = g + 1;
          __syncwarp();
        }
        Step& s = sh.step[g % kSteps];
        if (mine == i) {
          s.at[grp] = x.at;
          s.sc[grp] = sc;
        }
        if (lane == 0) {
          s.flags = (x.flags & ((i == 0 ? ~0 : ~kFirst) & (i == n - 1 ? ~0 : ~kLast))) | (keys == kGroups ? kAllKeys : 0) |
                    (x.seg & 3) << 8;
          s.j0 = x.j0 - i * kN, s.seg = x.seg, s.t0 = x.t0, s.n = x.rows, s.len = x.len;
          s.prefix = x.prefix, s.h = x.h, s.i0 = x.i0, s.piece = x.piece;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.step_full[g % kSteps]);
      }
      if (x.n == 0) break;
      x = next;
    }
    // copies still on their way (after a wait that ran out) land before the CTA ends
    if (lane == 0)
      for (int k = issued > kRaw ? issued - kRaw : 0; k < issued; ++k) mbar_wait(&sh.raw_full[k % kRaw], (k / kRaw) & 1);
  } else if (warp >= kMma) {
    // ----------------------------------------------------------------- MMA
    {
      const int x = __shfl_sync(0xffffffffu, warp == kMma ? 0 : 1, 0);   // tile A or B, the same in all lanes
      const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc_qk = make_idesc(kFmtF16, kFmtF16, 0, 0, kT, kN);
      const uint32_t idesc_pv = make_idesc(kFmtF16, kFmtF16, 0, 1, kT, D);
      const uint64_t qdesc = make_smem_desc(smem_u32(smem + L::kQ + x * L::kOp), 16, 1024, kSwizzle128B);
      const uint64_t kdesc = make_smem_desc(smem_u32(smem + L::kK), 16, 1024, kSwizzle128B);
      // MN-major V: 64-column atoms 8 KB apart, 16 key rows (2 KB) per K = 16 step
      const uint64_t vdesc = make_smem_desc(smem_u32(smem + L::kV), kHalfKv, 1024, kSwizzle128B);
      const uint32_t scol = tmem_u + kColS + 128u * x, ocol = tmem_u + kColO + 128u * x;
      int cnt_s = 0, cnt_p = 0;                      // QKs and PVs issued
      // A step's number, its place in the K/V ring and that place's parity, counted
      // along: a division by three per use is a chain of its own in this warp.
      struct At {
        int g, place, parity, flags;
        __device__ __forceinline__ void next() {
          ++g;
          if (++place == kRing) place = 0, parity ^= 1;
        }
      };
      auto qk = [&](const At& s) -> bool {
        if ((s.flags & kFirst) && !warp_await(&sh.q_full, (s.flags >> 8) & 1, sh, a.err)) return false;
        if (!warp_await(&sh.kv_full[s.place], s.parity, sh, a.err)) return false;
        tc_fence_after_sync();
        const uint64_t db = kdesc + static_cast<uint64_t>((s.place * L::kOpKv) >> 4);
        const uint32_t cs = scol + 64u * (cnt_s & 1);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(cs, qdesc + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), db + (((kk >> 2) * kHalfKv + (kk & 3) * 32) >> 4),
                     idesc_qk, kk > 0);
        if (lane == 0) {   // a commit publishes MMAs, not stores: an arrival of its own does
          sh.s_step[x][cnt_s & 1] = s.g;
          mbar_arrive(&sh.s_full[x][cnt_s & 1]);
        }
        __syncwarp();
        commit(&sh.s_full[x][cnt_s & 1]);
        if (s.flags & kLast) {
          commit(&sh.q_free);
          if (!(s.flags & kHasB)) commit(&sh.q_free);   // tile B's arrival too
        }
        ++cnt_s;
        return true;
      };
      auto pv = [&](const At& s) -> bool {
        if (!warp_await(&sh.p_ready[x][cnt_p & 1], (cnt_p >> 1) & 1, sh, a.err)) return false;
        tc_fence_after_sync();
        const uint64_t db = vdesc + static_cast<uint64_t>((s.place * L::kOpKv) >> 4);
        const uint32_t cs = scol + 64u * (cnt_p & 1);
#pragma unroll
        for (int kk = 0; kk < kN / 16; ++kk)
          mma_ts(ocol, cs + 8 * kk, db + static_cast<uint64_t>((kk * 16 * 128) >> 4), idesc_pv,
                            (!(s.flags & kFirst) || kk > 0) ? 1u : 0u);
        commit(&sh.kv_empty[s.place]);
        commit(&sh.o_done[x][cnt_p & 1]);
        ++cnt_p;
        return true;
      };
      // from s on, the next step that this tile takes part in
      bool ok = true;
      auto find = [&](At s) {
        while (true) {
          ok = warp_await(&sh.step_full[s.g % kSteps], (s.g / kSteps) & 1, sh, a.err);
          if (!ok) break;
          s.flags = sh.step[s.g % kSteps].flags;
          if ((s.flags & kEnd) || x == 0 || (s.flags & kHasB)) break;
          // not tile B's: its place is free for this tile, once it is this step's
          // (so every phase of every place is waited for, and none mistaken)
          ok = warp_await(&sh.kv_full[s.place], s.parity, sh, a.err);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&sh.kv_empty[s.place]);
          __syncwarp();
          s.next();
        }
        return s;
      };
      // QK(g+1) PV(g); the first QK of a segment comes behind the last PV of the
      // one before, as its queries take a while
      At cur = find(At{0, 0, 0, 0});
      if (ok && !(cur.flags & kEnd)) ok = qk(cur);
      while (ok && !(cur.flags & kEnd)) {
        At s = cur;
        s.next();
        if (cur.flags & kLast) ok = pv(cur);
        if (ok) s = find(s);
        if (ok && !(s.flags & kEnd)) ok = qk(s);
        if (ok && !(cur.flags & kLast)) ok = pv(cur);
        cur = s;
      }
      if (lane == 0) {
        sh.s_step[x][cnt_s & 1] = -1;
        mbar_arrive(&sh.s_full[x][cnt_s & 1]);
        mbar_arrive(&sh.s_full[x][cnt_s & 1]);   // in the place of a QK
      }
      __syncwarp();
      // every MMA issued here completes before TMEM is released
      commit(&sh.mma_done[x]);
      const long long t0 = clock64();
      while (!mbar_try_wait(&sh.mma_done[x], 0)) {
        if (clock64() - t0 > kWaitTimeoutCycles) {
          report_error(a.err, kDevErrTimeout);
          break;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and epilogue
    const int x = warp < kSoftB ? 0 : 1;          // tile A or B
    const int r = (warp & 3) * 32 + lane;         // tile row = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t srow2 = tmem + lane_base + kColS + 128u * x;
    const uint32_t orow = tmem + lane_base + kColO + 128u * x;
    int cnt = 0;                                  // steps of this tile
    float m = 0.f, l = 0.f, sc = 0.f, slope = 0.f;
    bool seen = false;
    int hi = 0, lo = 0, at = 0;
    bool live = false;
    size_t row = 0;                               // its row of o or of the workspace
    while (true) {
      if (!warp_await(&sh.s_full[x][cnt & 1], (cnt >> 1) & 1, sh, a.err)) break;
      tc_fence_after_sync();
      const int g = sh.s_step[x][cnt & 1];
      if (g < 0) break;
      const Step& st = sh.step[g % kSteps];       // until the last PV of this step: none of it is read behind p_ready
      const int flags = st.flags;
      const uint32_t srow = srow2 + 64u * (cnt & 1);
      if (__builtin_expect(flags & kFirst, 0)) {
        const int q = r / a.G, i = st.i0 + x * ta.tq + q;
        Rows rows;
        rows.t0 = st.t0, rows.n = st.n, rows.len = st.len, rows.prefix = st.prefix;
        live = q < ta.tq && i < st.n;
        hi = live ? row_hi(a, rows, i) : 0;
        lo = live ? row_lo(a, rows, i) : 0;
        at = st.len - st.n + i;
        row = flags & kWholeTask ? static_cast<size_t>(st.t0 + i) * a.Hq + st.h * a.G + r - q * a.G
                                 : static_cast<size_t>(st.piece) * (2 * kT) + x * kT + r;
        if constexpr (kBias) slope = live ? __ldg(a.slopes + st.h * a.G + r - q * a.G) * kLog2e : 0.f;
        sc = std::is_same<E, __half>::value ? (kCap ? a.scale_cap : a.scale_log2) : sh.qsc[st.seg & 3][x][r];
        m = l = 0.f;
        seen = !live;         // dead rows never wait for a key
      }
      const float4* gs = st.sc;
      const int j0 = st.j0;
      const bool whole = __all_sync(0xffffffffu, !live || (lo <= j0 && j0 + kN <= hi));

      // z = y - m, -inf for keys the row does not see; m is 0 until it has seen one
      uint32_t v[2][32];
      tmem_ld32(srow, v[0]);
      tmem_ld32(srow + 32, v[1]);
      float rvs[kGroups], top = -INFINITY;
      tmem_ld_wait();
      if constexpr (kCap == kFar) {
        // 16 columns at a time through TMEM: unrolled, all 64 do not fit the instruction
        // cache (a prompt of 8192 with a cap of 1000: 1.53 ms against 1.18)
#pragma unroll 1
        for (int q = 0; q < kGroups; ++q) {
          uint32_t w[16];
          tmem_ld16(srow + 16 * q, w);
          const float4 s4 = gs[q];
          const bool bad = __float_as_uint(s4.x) == kBadPageMark;
          const float f = bad ? 0.f : sc * s4.x, off = bad ? -INFINITY : s4.y - m;
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float o = kBias ? fmaf(slope, static_cast<float>(j0 + 16 * q + i - at), off) : off;
            w[i] = __float_as_uint(fmaf(a.cap_log2, tanh_far(__uint_as_float(w[i]) * f), o));
          }
          tmem_st16(srow + 16 * q, w);
        }
        tmem_st_wait();
        tmem_ld32(srow, v[0]);
        tmem_ld32(srow + 32, v[1]);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) rvs[q] = gs[q].z;
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          uint32_t(&w)[32] = v[q >> 1];
          const float4 s4 = gs[q];
          rvs[q] = s4.z;
          const bool bad = __float_as_uint(s4.x) == kBadPageMark;
          const float f = bad ? 0.f : sc * s4.x, off = bad ? -INFINITY : s4.y - m;
          const int w0 = 16 * (q & 1);
          if constexpr (!kCap && !kBias) {
            const uint64_t f2 = f32x2_pack(f, f), o2 = f32x2_pack(off, off);
#pragma unroll
            for (int i = w0; i < w0 + 16; i += 2) {
              const float2 z = f32x2_unpack(
                  f32x2_fma(f32x2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), f2, o2));
              w[i] = __float_as_uint(z.x);
              w[i + 1] = __float_as_uint(z.y);
            }
          } else {
#pragma unroll
            for (int i = w0; i < w0 + 16; ++i) {
              float o = off;
              if constexpr (kBias) o = fmaf(slope, static_cast<float>(j0 + 32 * (q >> 1) + i - at), o);
              const float s = __uint_as_float(w[i]);
              w[i] = __float_as_uint(kCap ? fmaf(a.cap_log2, tanh_of(s * f), o) : fmaf(s, f, o));
            }
          }
        }
      }
      if (__builtin_expect(!whole, 0)) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (j0 + i < lo || j0 + i >= hi) v[i >> 5][i & 31] = 0xFF800000u;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          t4[(i >> 1) & 3] = fmax3(t4[(i >> 1) & 3], __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
        top = fmax3(top, fmax3(t4[0], t4[1], t4[2]), t4[3]);
      }
      if (!live) top = -INFINITY;   // what lies in a dead row moves nobody's m
      if (__builtin_expect(__any_sync(0xffffffffu, top > (seen ? kMaxP : -INFINITY)), 0)) {
        // m is set, or moves with everything so far: O once its last PV has landed
        float d = 0.f;
        if (seen) d = fmaxf(top - kSetP, 0.f);
        else if (top > -INFINITY) d = top - kSetP;
        const float f = seen ? fast_exp2(-d) : 1.f;
        m += d;
        l *= f;
        if (__any_sync(0xffffffffu, f != 1.f)) {   // never in a segment's first step
          // (of this barrier, PV(g-3) is behind the QK(g) that s_full saw, and PV(g+1)
          // in front of this warp's P(g): its current phase is PV(g-1)'s or just over)
          if (!warp_await(&sh.o_done[x][(cnt - 1) & 1], ((cnt - 1) >> 1) & 1, sh, a.err)) break;
          tc_fence_after_sync();
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            tmem_ld16(orow + 16 * k, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(orow + 16 * k, o);
          }
        }
        seen |= top > -INFINITY;
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i >> 5][i & 31] = __float_as_uint(__uint_as_float(v[i >> 5][i & 31]) - d);
      }
      // P over the first half of S, which has been read
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint64_t ls2 = f32x2_pack(0.f, 0.f);
#pragma unroll
          for (int i = 8 * q; i < 8 * q + 8; ++i) {
            const float p0 = fast_exp2(__uint_as_float(v[c][2 * i])), p1 = fast_exp2(__uint_as_float(v[c][2 * i + 1]));
            ls2 = f32x2_add(ls2, f32x2_pack(p0, p1));
            pk[i] = f32x2_to_f16x2(p1, p0);
          }
          const float2 ls = f32x2_unpack(ls2);
          l = fmaf(ls.x + ls.y, rvs[2 * c + q], l);
        }
        tmem_st16(srow + 16 * c, pk);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&sh.p_ready[x][cnt & 1]);
      ++cnt;
      if (__builtin_expect(flags & kLast, 0)) {
        // ---- the segment's rows, once its last PV has landed (and with it the one before)
        if (!warp_await(&sh.o_done[x][(cnt - 1) & 1], ((cnt - 1) >> 1) & 1, sh, a.err)) break;
        tc_fence_after_sync();
        // l = 0: no key seen; NaN (of a NaN score, which moves no m) goes into o and lse
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (flags & kWholeTask) {
          const float so = l == 0.f ? 0.f : 1.f / l;
          E* out = static_cast<E*>(a.o) + row * D;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(orow + 32 * c, v);
            tmem_ld_wait();
            if (live) {
              uint4* o4 = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t pk[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  pk[k] = pack_out<E>(__uint_as_float(v[8 * i + 2 * k + 1]) * so, __uint_as_float(v[8 * i + 2 * k]) * so);
                o4[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              }
            }
          }
          if (live && a.lse != nullptr) a.lse[row] = lse2 * kLn2;
        } else {
          float* out = ta.part_o + row * D;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(orow + 32 * c, v);
            tmem_ld_wait();
            if (live) {
              uint4* o4 = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
              for (int i = 0; i < 8; ++i) o4[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          }
          if (live) ta.part_ml[row] = make_float2(l == 0.f ? -INFINITY : m, l);
        }
        tc_fence_before_sync();
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <typename E, int D, bool kInt8, int kCap, bool kBias>
cudaError_t go(const TileArgs& a, int sms, cudaStream_t stream) {
  auto kernel = attend_tile_kernel<E, D, kInt8, kCap, kBias>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap q_map, k_map, v_map;
  if (!pool_map(a.p, D, a.p.k, 16, &k_map) || !pool_map(a.p, D, a.p.v, 16, &v_map)) return cudaErrorInvalidValue;
  const uint64_t dims[3] = {D, static_cast<uint64_t>(a.p.Hq), static_cast<uint64_t>(a.p.T)};
  const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(a.p.Hq) * D * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(a.p.G), static_cast<uint32_t>(a.tq)};
  if (encode_tensor_map(&q_map, std::is_same<E, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        3, const_cast<void*>(a.p.q), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, q_map, k_map, v_map, a);
}

template <typename E, int D, bool kInt8>
cudaError_t pick2(const TileArgs& a, int sms, cudaStream_t s) {
  const bool cap = a.p.cap_log2 > 0.f, bias = a.p.slopes != nullptr;
  if (a.p.far_cap) return bias ? go<E, D, kInt8, kFar, true>(a, sms, s) : go<E, D, kInt8, kFar, false>(a, sms, s);
  if (cap) return bias ? go<E, D, kInt8, kNear, true>(a, sms, s) : go<E, D, kInt8, kNear, false>(a, sms, s);
  return bias ? go<E, D, kInt8, kNone, true>(a, sms, s) : go<E, D, kInt8, kNone, false>(a, sms, s);
}

template <typename E>
cudaError_t pick(const TileArgs& a, int D, bool int8, int sms, cudaStream_t s) {
  if (D == 64) return int8 ? pick2<E, 64, true>(a, sms, s) : pick2<E, 64, false>(a, sms, s);
  return int8 ? pick2<E, 128, true>(a, sms, s) : pick2<E, 128, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_attend_tiles(const TileArgs& a, int head_dim, bool int8, bool f16, int sms, cudaStream_t stream) {
  return f16 ? pick<__half>(a, head_dim, int8, sms, stream) : pick<__nv_bfloat16>(a, head_dim, int8, sms, stream);
}

}  // namespace qpkv
