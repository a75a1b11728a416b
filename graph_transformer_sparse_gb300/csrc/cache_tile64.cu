// cache_tile64.cu -- the cache attention's tensor-core kernel for heads of 64.
#include "cache_tile.cuh"

namespace gt {
gtattn_status cache_tile_64(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s) {
    return launch_tile_d<64>(a, dtype, rows, s);
}
}  // namespace gt
