// cache_attn.cuh -- what the cache attention's entry point (cache_attn.cu) and
// its tensor-core kernel (cache_tile.cuh) share.
#pragma once

#include "cache.cuh"

namespace gt {

struct CacheAttn {
    CacheView c;
    CacheRows r;
    const void* Q;
    void* out;
    const int* sel;   // [T, Hkv, n_sel] page numbers within the request, or null
    int H, G, n_sel;
    float qscale;     // scale * log2(e)
    int q_vec, o_vec; // Q and out are 16-byte aligned
};

// The tensor-core kernel for heads of D features; `rows`: (token, head) rows
// that a request (selection: a token) brings per K/V head, on average.
gtattn_status cache_tile_32(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s);
gtattn_status cache_tile_64(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s);
gtattn_status cache_tile_128(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s);
// The same for narrower heads, a multiple of 16 features, padded in shared memory.
gtattn_status cache_tile_to_64(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s);
gtattn_status cache_tile_to_128(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s);

// The same for many rows, on tcgen05 (cache_tc.cu): whether it takes the
// call, and the call.
constexpr int kCacheTcMinRows = 64;
bool cache_tc_takes(const CacheAttn& a, gtattn_dtype dtype, int64_t rows);
gtattn_status cache_tc(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s);

}  // namespace gt
