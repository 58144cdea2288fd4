// Page and slot assignment for one serving step, from request lengths that
// live on the device (README 参数说明 rows block_table and
// actual_seq_lengths_query / _kv give the arrays it fills).
//
// Request b holds H_b = ceil(L_b / ps) pages and grows by n_b tokens, so it
// takes N_b = ceil((L_b + n_b) / ps) - H_b pages.  With X_b the exclusive
// prefix sum of N, its i-th new page is free_pages[count - 1 - (X_b + i)]
// (the free list is a stack), and its token k goes to position p = L_b + k,
// slot page(p / ps) * ps + p % ps.
//
// A few kilobytes in, at most a few megabytes out: latency-bound, so the
// whole call is one launch.  Every CTA of one thread-block cluster scans all
// requests (three int32 per request stay in its shared memory), the cluster
// meets, and the CTAs share the table rows and the tokens out among them.
// The meeting is what lets the lengths, the count and the table be updated in
// place: nothing is written before every CTA has read them.  One CTA alone is
// used for up to 8192 words of output, where eight would each repeat a scan
// that costs more than the stores they save.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace qpkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kClusterCtas = 8;

__device__ __forceinline__ long long warp_scan_ll(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Inclusive sums of two values per thread over the CTA.
__device__ __forceinline__ void cta_scan2(long long& x, long long& y, long long (&wx)[32],
                                          long long (&wy)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan_ll(x, lane);
  y = warp_scan_ll(y, lane);
  if (lane == 31) {
    wx[warp] = x;
    wy[warp] = y;
  }
  __syncthreads();
  if (warp == 0) {
    wx[lane] = warp_scan_ll(wx[lane], lane);
    wy[lane] = warp_scan_ll(wy[lane], lane);
  }
  __syncthreads();
  if (warp > 0) {
    x += wx[warp - 1];
    y += wy[warp - 1];
  }
}

__global__ void __launch_bounds__(kThreads, 1) assign_pages_kernel(const qpkv_assign_params p) {
  extern __shared__ int32_t sm[];
  __shared__ long long wx[32], wy[32];
  __shared__ int taken;
  const int B = p.num_seqs, ps = p.page_size, W = p.bt_stride;
  int32_t* s_end = sm;            // tokens up to and with request b (at most num_tokens)
  int32_t* s_old = sm + B;        // L_b, -1 for one that cannot be read
  int32_t* s_first = sm + 2 * B;  // X_b, -1 for a refused request
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x;

  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) taken = 0;
  int count = *p.free_count;
  int err = 0;
  if (count < 0 || count > p.num_free) {
    err |= kDevErrBadLength;
    count = 0;
  }
  const long long room = static_cast<long long>(W) * ps;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long tokens = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = p.new_lens[b], len = p.seqlens[b];
    if (n < 0 || len < 0) continue;
    tokens += n;
    if (static_cast<long long>(len) + n <= room)
      pages += (static_cast<long long>(len) + n + ps - 1) / ps - (static_cast<long long>(len) + ps - 1) / ps;
  }
  long long tok_in = tokens, pg_in = pages;
  cta_scan2(tok_in, pg_in, wx, wy);
  long long tok = tok_in - tokens, pg = pg_in - pages;
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = p.new_lens[b], len = p.seqlens[b];
    bool ok = n >= 0 && len >= 0;
    long long need = 0;
    if (ok) {
      tok += n;
      ok = static_cast<long long>(len) + n <= room;
      if (ok)
        need = (static_cast<long long>(len) + n + ps - 1) / ps -
               (static_cast<long long>(len) + ps - 1) / ps;
    }
    if (!ok || tok > p.num_tokens) {
      err |= kDevErrBadLength;
      ok = false;
    }
    const long long first = pg;
    pg += need;
    if (ok && pg > count) {
      if (need > 0) err |= kDevErrNoPages;
      ok = need == 0;   // a request that needs no page is served all the same
    }
    s_end[b] = static_cast<int32_t>(tok < p.num_tokens ? tok : p.num_tokens);
    s_old[b] = len >= 0 && len <= room ? len : -1;
    s_first[b] = ok ? static_cast<int32_t>(need > 0 ? first : 0) : -1;
    if (ok) mine += static_cast<int>(need);
  }
  if (mine > 0) atomicAdd(&taken, mine);   // integers: any order gives the same sum
  if (rank == 0 && err) report_error(p.error_word, err);
  // every CTA has read the lengths and the count; its own arrays are complete
  cluster.sync();

  if (rank == 0 && tid == 0) *p.free_count_out = count - taken;
  const int step = kThreads * ctas, me = rank * kThreads + tid;
  for (int b = me; b < B; b += step) {
    const int n = s_end[b] - (b > 0 ? s_end[b - 1] : 0);
    p.cu_seqlens[b] = s_end[b];
    if (s_first[b] >= 0) {
      p.seqlens_out[b] = s_old[b] + n;
    } else if (p.seqlens_out != p.seqlens) {
      p.seqlens_out[b] = p.seqlens[b];
    }
    if (p.start_pos != nullptr) p.start_pos[b] = s_first[b] >= 0 ? s_old[b] : -1;   // may be seqlens itself
  }
  // free page i of the demand
  auto fresh = [&](int i) -> int {
    const int page = __ldg(p.free_pages + (count - 1 - i));
    if (page >= 0 && page < p.num_pages) return page;
    report_error(p.error_word, kDevErrBadPage);
    return -1;
  };
  // table rows: one warp each
  const bool in_place = p.block_table_out == p.block_table;
  const int lane = tid & 31;
  for (int b = me >> 5; b < B; b += step >> 5) {
    const int old = s_old[b], first = s_first[b];
    if (old < 0) {   // a length that fits no row: the row stays as it is
      if (!in_place)
        for (int j = lane; j < W; j += 32)
          p.block_table_out[static_cast<size_t>(b) * W + j] = p.block_table[static_cast<size_t>(b) * W + j];
      continue;
    }
    const int n = first >= 0 ? s_end[b] - (b > 0 ? s_end[b - 1] : 0) : 0;
    const int held = (old - 1 + ps) / ps;   // old <= room: no overflow below 2^31 - ps
    const int all = static_cast<int>((static_cast<long long>(old) + n + ps - 1) / ps);
    for (int j = lane; j < W; j += 32) {
      const size_t at = static_cast<size_t>(b) * W + j;
      if (j < held) {
        if (!in_place) p.block_table_out[at] = p.block_table[at];
      } else {
        p.block_table_out[at] = j < all ? fresh(first + j - held) : -1;
      }
    }
  }
  // tokens
  for (int t = me; t < p.num_tokens; t += step) {
    int slot = -1, pos = -1;
    if (t < s_end[B - 1]) {
      int lo = 0, hi = B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t < s_end[mid]) hi = mid; else lo = mid + 1;
      }
      const int first = s_first[lo];
      if (first >= 0) {
        const int old = s_old[lo];
        pos = old + t - (lo > 0 ? s_end[lo - 1] : 0);
        const int j = pos / ps, held = (old - 1 + ps) / ps;
        int page;
        if (j < held) {   // never written by this call, in place or not
          page = p.block_table[static_cast<size_t>(lo) * W + j];
          if (page < 0 || page >= p.num_pages) {
            report_error(p.error_word, kDevErrBadPage);
            page = -1;
          }
        } else {
          page = fresh(first + j - held);
        }
        if (page >= 0) slot = page * ps + (pos - j * ps);
      }
    }
    p.slot_mapping[t] = slot;
    p.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_assign_pages(const qpkv_assign_params& p, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.num_seqs) * 3 * sizeof(int32_t);
  cudaError_t e = cudaFuncSetAttribute(assign_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kAssignMaxSeqs * 3 * static_cast<int>(sizeof(int32_t)));
  if (e != cudaSuccess) return e;
  const long long words = 2ll * p.num_tokens + static_cast<long long>(p.num_seqs) * p.bt_stride;
  cudaLaunchConfig_t cfg = {};
  const unsigned ctas = words <= 8192 ? 1u : static_cast<unsigned>(kClusterCtas);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, assign_pages_kernel, p);
}

}  // namespace qpkv
