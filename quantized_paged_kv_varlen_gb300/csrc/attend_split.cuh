// What the split forms of the attention kernels share (attend_page8.cu, attend_group4.cu):
// fragments, the pieces of a row and the kernel that joins them, the plan of a call.
#pragma once
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "page8.cuh"

namespace qpkv {
namespace {

constexpr int kWarps = 4;               // per block
constexpr int kGroup = 16;              // tokens of a unit
constexpr int kMinRun = 4;              // units of a run at least (64 tokens)

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

struct RowInfo {
  int lo, hi;         // keys the row sees
  float sc;           // logit multiplier
  float slope, at;    // bias: slope * (j - at), log2 units; at and j from the end of the
                      // cache, as float32 holds no odd position beyond 2^24
};

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

inline int sm_count() {
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

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Which forms a call needs, by sizes the host knows: the split form takes up
// to kSplitRows query rows of a (sequence, kv head); with a bound on a
// sequence's queries above that the tiled form takes the larger ones, and all
// of them when there is one sequence.
constexpr int kSplitRows = 24;
struct Plan {
  bool split, tiled;
  int tile, split_rows;
};
inline Plan plan_for(int B, int T, int max_q, int G) {
  Plan p;
  const long long rows = static_cast<long long>(max_q > 0 && max_q < T ? max_q : T) * G;
  p.tiled = rows > kSplitRows && G <= 128;
  p.split = !p.tiled || B > 1;
  p.tile = 8 * (rows <= 8 ? 1 : rows <= 16 ? 2 : 3);
  p.split_rows = !p.tiled ? INT_MAX : p.split ? kSplitRows : -1;
  return p;
}

// The workspace's arrays: the tokens' places, pieces of O and (m, l) of the
// split form (`blocks`: its blocks per SM for tiles of 8, 16, 24 rows), the same
// of the tiled one.
struct Sizes {
  size_t info, o, ml, to, tml;
  size_t total() const { return info + o + ml + to + tml; }
};
inline Sizes sizes(const Plan& p, int T, int D, int sms, const int (&blocks)[3]) {
  Sizes s = {};
  s.info = up256(static_cast<size_t>(T) * sizeof(TokenInfo));
  if (p.split) {
    const size_t rows = static_cast<size_t>(2) * sms * blocks[p.tile / 8 - 1] * kWarps * p.tile;
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
}  // namespace qpkv
