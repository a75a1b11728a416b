// cache.cuh -- internal definitions of the 8-bit K/V cache operators
// (cache.cu: slots and append; cache_select.cu: page selection;
// cache_attn.cu: attention over the cache).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace gt {

constexpr int kCacheMaxD = 256;
constexpr int kCacheMaxHeads = 1024;
// scale exponents: an all-zero page gets 2^-64; fp32's largest value needs 2^120
constexpr int kScaleMinExp = -64, kScaleMaxExp = 120;

// Device view of a gtattn_cache.
struct CacheView {
    uint8_t* k8;
    uint8_t* v8;
    float* kscale;
    float* vscale;
    __nv_bfloat16* kmean;
    int pages, page, lp;   // page = 1 << lp
    int Hkv, D;
};

// The requests' side of a call: new token rows [tok_off[s], tok_off[s+1]) of
// request s are its last ones, at positions length[s] - n .. length[s] - 1.
struct CacheRows {
    const int* table;     // [S, max_pages] page ids
    const int* length;    // [S]
    const int* tok_off;   // [S + 1]
    int S, T, max_pages;
};

// Host checks shared by the entry points; `need` is a mask of what the call
// reads of the cache: 1 k8/v8 and their scales, 2 kmean.
gtattn_status check_cache(const gtattn_cache* c, int need, CacheView* v);
gtattn_status check_cache_rows(const int32_t* table, const int32_t* length, const int32_t* tok_off, int64_t S,
                               int64_t T, int64_t max_pages, int page, CacheRows* r);

// The error word of the tensor-core cache attention on the current device
// (gtattn_device_errors).
cudaError_t cache_tc_errors(int* code, int reset);

// Request of token row t (t < tok_off[S]): the largest s with tok_off[s] <= t.
// Looked for at s = t first: with a token for each request it is there, and
// the search's dependent loads are saved.
__device__ __forceinline__ bool request_guess(const int* __restrict__ tok_off, int S, int t, int* s) {
    *s = min(t, S - 1);
    const int a = __ldg(tok_off + *s), b = __ldg(tok_off + *s + 1);
    return a <= t && t < b;
}
__device__ __forceinline__ int request_of(const int* __restrict__ tok_off, int S, int t) {
    int lo;
    if (request_guess(tok_off, S, t, &lo)) return lo;
    lo = 0;
    int hi = S;   // tok_off[lo] <= t < tok_off[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(tok_off + m) <= t) lo = m;
        else hi = m;
    }
    return lo;
}
// The same by a whole warp, 32 places a look.
__device__ __forceinline__ int request_of_warp(const int* __restrict__ tok_off, int S, int t, int lane) {
    int lo;
    if (request_guess(tok_off, S, t, &lo)) return lo;
    lo = 0;
    int n = S;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && __ldg(tok_off + lo + lane * step) <= t;
        const int i = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += i * step;
        n = min(step, n - i * step);
    }
    return lo;
}

// Position of row t of request s in its request; -1 when the request holds
// fewer tokens than it has rows, capped at the table's last position.
__device__ __forceinline__ int position_of(const CacheRows& r, int page, int s, int t) {
    const long long p = static_cast<long long>(__ldg(r.length + s)) - (__ldg(r.tok_off + s + 1) - t);
    const long long last = static_cast<long long>(r.max_pages) * page - 1;
    return static_cast<int>(p < -1 ? -1 : p > last ? last : p);
}

__device__ __forceinline__ float e4m3_f32(uint8_t x) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}
// Nearest e4m3 value, ties to even, saturating; NaN and infinities give NaN.
__device__ __forceinline__ uint8_t f32_e4m3(float x) {
    if (!(fabsf(x) < INFINITY)) return 0x7f;
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// Programmatic launch: a kernel launched by launch_after may start while the
// one before it in the stream still runs, and calls after_previous() before it
// touches memory; let_next_start() lets the next one do the same.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Eight features by 16-byte loads (16-byte aligned).
template <typename T> struct Eight;
template <> struct Eight<float> {
    float x[8];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <> struct Eight<__nv_bfloat16> {
    float x[8];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        x[0] = bf16lo(a.x); x[1] = bf16hi(a.x); x[2] = bf16lo(a.y); x[3] = bf16hi(a.y);
        x[4] = bf16lo(a.z); x[5] = bf16hi(a.z); x[6] = bf16lo(a.w); x[7] = bf16hi(a.w);
    }
};

}  // namespace gt
