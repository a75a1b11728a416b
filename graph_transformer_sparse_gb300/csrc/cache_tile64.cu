// cache_tile64.cu -- the cache attention's tensor-core kernel for heads of 64,
// and of fewer features (a multiple of 16) padded to that.
#include "cache_tile.cuh"

namespace gt {
gtattn_status cache_tile_64(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s) {
    return launch_tile_d<64>(a, dtype, rows, s);
}
gtattn_status cache_tile_to_64(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    return launch_tile_padded<64>(a, dtype, s);
}
}  // namespace gt
