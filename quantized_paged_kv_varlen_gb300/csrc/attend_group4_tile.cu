// The tiled form (attend_tile.cuh) over the 4-bit cache.
#include "attend_tile.cuh"

namespace qpkv {
namespace {

template <typename E>
cudaError_t pick(const TileArgs& a, int D, int sms, cudaStream_t s) {
  return D == 64 ? pick_tiles<E, 64, kE2m1>(a, sms, s) : pick_tiles<E, 128, kE2m1>(a, sms, s);
}

}  // namespace

cudaError_t launch_attend_tiles4(const TileArgs& a, int head_dim, bool f16, int sms, cudaStream_t stream) {
  return f16 ? pick<__half>(a, head_dim, sms, stream) : pick<__nv_bfloat16>(a, head_dim, sms, stream);
}

}  // namespace qpkv
