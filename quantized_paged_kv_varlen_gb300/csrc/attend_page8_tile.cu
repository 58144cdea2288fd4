// The tiled form (attend_tile.cuh) over the page-scaled 8-bit cache.
#include "attend_tile.cuh"

namespace qpkv {
namespace {

template <typename E>
cudaError_t pick(const TileArgs& a, int D, bool int8, int sms, cudaStream_t s) {
  if (D == 64) return int8 ? pick_tiles<E, 64, kInt8>(a, sms, s) : pick_tiles<E, 64, kE4m3>(a, sms, s);
  return int8 ? pick_tiles<E, 128, kInt8>(a, sms, s) : pick_tiles<E, 128, kE4m3>(a, sms, s);
}

}  // namespace

cudaError_t launch_attend_tiles(const TileArgs& a, int head_dim, bool int8, bool f16, int sms, cudaStream_t stream) {
  return f16 ? pick<__half>(a, head_dim, int8, sms, stream) : pick<__nv_bfloat16>(a, head_dim, int8, sms, stream);
}

}  // namespace qpkv
