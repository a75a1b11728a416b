// cache_select.cu -- for each new token and K/V head, the pages of the cache
// that score highest against the token's queries.
#include "cache.cuh"

#include <algorithm>

namespace gt {
namespace {

constexpr int kSelThreads = 128;

// score(p, g) = sum over the heads h of group g of q_h . kmean[p, g], in 64
// bits; the token's own page is taken without a score, the n_sel - 1 others
// by falling score (equal ones, and NaN as the lowest: by rising page).
// Simplest form: a block per (token, K/V head), n_sel - 1 searches.
template <typename T>
__global__ void __launch_bounds__(kSelThreads)
k_select(CacheView c, CacheRows r, const T* __restrict__ Q, int* __restrict__ sel, int H, int n_sel,
         double* __restrict__ scratch, int n_items) {
    __shared__ double qs[kCacheMaxD];
    __shared__ double best_s[kSelThreads / 32];
    __shared__ int best_i[kSelThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int end = r.tok_off[r.S];
    const int G = H / c.Hkv;
    double* score = scratch + (int64_t)blockIdx.x * r.max_pages;
    for (int64_t it = blockIdx.x; it < n_items; it += gridDim.x) {
        const int t = (int)(it / c.Hkv), g = (int)(it % c.Hkv);
        if (t >= end) return;
        const int s = request_of(r.tok_off, r.S, t);
        const int pos = position_of(r, c.page, s, t);
        int* out = sel + it * n_sel;
        const int own = pos < 0 ? -1 : pos >> c.lp;
        __syncthreads();
        for (int d = tid; d < c.D; d += kSelThreads) {
            double v = 0;
            for (int h = 0; h < G; ++h) v += load_elem(Q, ((int64_t)t * H + g * G + h) * c.D + d);
            qs[d] = v;
        }
        __syncthreads();
        for (int p = warp; p < own; p += kSelThreads / 32) {
            const int pid = r.table[(int64_t)s * r.max_pages + p];
            double v = 0;
            if ((unsigned)pid < (unsigned)c.pages) {
                const __nv_bfloat16* m = c.kmean + ((int64_t)pid * c.Hkv + g) * c.D;
                for (int d = lane; d < c.D; d += 32) v += qs[d] * (double)__bfloat162float(m[d]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) score[p] = v == v ? v : -INFINITY;
        }
        __syncthreads();
        const int k = min(own, n_sel - 1);   // earlier pages taken (own < 0: none)
        for (int j = 0; j < k; ++j) {
            double b = -INFINITY;
            int bi = 0x7fffffff;
            for (int p = tid; p < own; p += kSelThreads) {
                const double v = score[p];
                if (v == v && (v > b || bi == 0x7fffffff)) { b = v; bi = p; }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double v = __shfl_xor_sync(0xffffffffu, b, o);
                const int vi = __shfl_xor_sync(0xffffffffu, bi, o);
                if (vi != 0x7fffffff && (bi == 0x7fffffff || v > b || (v == b && vi < bi))) { b = v; bi = vi; }
            }
            if (lane == 0) { best_s[warp] = b; best_i[warp] = bi; }
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kSelThreads / 32; ++w)
                    if (best_i[w] != 0x7fffffff &&
                        (bi == 0x7fffffff || best_s[w] > b || (best_s[w] == b && best_i[w] < bi))) {
                        b = best_s[w];
                        bi = best_i[w];
                    }
                if (bi != 0x7fffffff) score[bi] = NAN;   // taken
            }
            __syncthreads();
        }
        // emit in rising order
        if (tid == 0) {
            int w = 0;
            for (int p = 0; p < own && w < k; ++p)
                if (score[p] != score[p]) out[w++] = p;
            if (own >= 0 && w < n_sel) out[w++] = own;
            for (; w < n_sel; ++w) out[w] = -1;
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" gtattn_status gtattn_cache_select(const gtattn_cache* cache, const void* Q, const int32_t* table,
                                             const int32_t* length, const int32_t* tok_off, int32_t* sel, int64_t S,
                                             int64_t T, int64_t max_pages, int H, int n_sel, gtattn_dtype dtype,
                                             cudaStream_t stream) {
    CacheView c;
    CacheRows r;
    GT_TRY(check_cache(cache, 2, &c));
    GT_TRY(check_cache_rows(table, length, tok_off, S, T, max_pages, c.page, &r));
    if (dtype != GTATTN_F32 && dtype != GTATTN_BF16 && dtype != GTATTN_BF16_OUT_F32) return GTATTN_ERR_INVALID_ARG;
    if (H < 1 || H > kCacheMaxHeads || H % c.Hkv || n_sel < 1 || n_sel > (1 << 20)) return GTATTN_ERR_INVALID_ARG;
    if (T > 0 && (!Q || !sel)) return GTATTN_ERR_INVALID_ARG;
    const uintptr_t esz = dtype == GTATTN_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(Q) & (esz - 1)) || (reinterpret_cast<uintptr_t>(sel) & 3u))
        return GTATTN_ERR_INVALID_ARG;
    if (T * c.Hkv >= (1ll << 31)) return GTATTN_ERR_UNSUPPORTED;
    if (T == 0 || S == 0) return GTATTN_OK;
    const int items = (int)(T * c.Hkv);
    const int blocks = std::min(items, num_sms() * 8);
    void* scratch = nullptr;
    GT_TRY(pool_alloc(&scratch, sizeof(double) * (size_t)blocks * std::max<int64_t>(max_pages, 1), stream));
    {
        ProfScope ps(GTATTN_KCAT_CACHE, 1, stream);
        if (dtype == GTATTN_F32)
            k_select<float><<<blocks, kSelThreads, 0, stream>>>(c, r, static_cast<const float*>(Q), sel, H, n_sel,
                                                                 static_cast<double*>(scratch), items);
        else
            k_select<__nv_bfloat16><<<blocks, kSelThreads, 0, stream>>>(c, r, static_cast<const __nv_bfloat16*>(Q),
                                                                         sel, H, n_sel,
                                                                         static_cast<double*>(scratch), items);
    }
    const cudaError_t e = cudaGetLastError();
    pool_free(scratch, stream);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}
