// cache_tile32.cu -- the cache attention's tensor-core kernel for heads of 32.
#include "cache_tile.cuh"

namespace gt {
gtattn_status cache_tile_32(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s) {
    return launch_tile_d<32>(a, dtype, rows, s);
}
}  // namespace gt
