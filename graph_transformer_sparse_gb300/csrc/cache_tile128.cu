// cache_tile128.cu -- the cache attention's tensor-core kernel for heads of 128,
// and of fewer features (a multiple of 16) padded to that.
#include "cache_tile.cuh"

namespace gt {
gtattn_status cache_tile_128(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s) {
    return launch_tile_d<128>(a, dtype, rows, s);
}
gtattn_status cache_tile_to_128(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    return launch_tile_padded<128>(a, dtype, s);
}
}  // namespace gt
