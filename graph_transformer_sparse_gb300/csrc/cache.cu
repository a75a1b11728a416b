// cache.cu -- the 8-bit K/V cache: argument checks, slots for new tokens,
// and the append that quantises keys and values into the pages.
#include "cache.cuh"

#include <algorithm>

namespace gt {

gtattn_status check_cache(const gtattn_cache* c, int need, CacheView* v) {
    if (!c) return GTATTN_ERR_INVALID_ARG;
    if (c->page != 16 && c->page != 32 && c->page != 64) return GTATTN_ERR_INVALID_ARG;
    if (c->pages < 0 || (int64_t)c->pages * c->page >= (1ll << 31)) return GTATTN_ERR_INVALID_ARG;
    if (c->Hkv < 1 || c->Hkv > kCacheMaxHeads || c->D < 1 || c->D > kCacheMaxD) return GTATTN_ERR_INVALID_ARG;
    if (c->pages > 0) {
        if ((need & 1) && (!c->k8 || !c->v8 || !c->kscale || !c->vscale)) return GTATTN_ERR_INVALID_ARG;
        if ((need & 2) && !c->kmean) return GTATTN_ERR_INVALID_ARG;
    }
    auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if ((bits(c->k8) | bits(c->v8) | bits(c->kmean)) & 15u) return GTATTN_ERR_INVALID_ARG;
    if ((bits(c->kscale) | bits(c->vscale)) & 3u) return GTATTN_ERR_INVALID_ARG;
    v->k8 = static_cast<uint8_t*>(c->k8);
    v->v8 = static_cast<uint8_t*>(c->v8);
    v->kscale = c->kscale;
    v->vscale = c->vscale;
    v->kmean = static_cast<__nv_bfloat16*>(c->kmean);
    v->pages = c->pages;
    v->page = c->page;
    v->lp = c->page == 16 ? 4 : c->page == 32 ? 5 : 6;
    v->Hkv = c->Hkv;
    v->D = c->D;
    return GTATTN_OK;
}

gtattn_status check_cache_rows(const int32_t* table, const int32_t* length, const int32_t* tok_off, int64_t S,
                               int64_t T, int64_t max_pages, int page, CacheRows* r) {
    constexpr int64_t kLim = (1ll << 31) - 1;
    if (S < 0 || T < 0 || max_pages < 0 || S >= kLim || T >= kLim || max_pages >= kLim) return GTATTN_ERR_INVALID_ARG;
    if (max_pages * page >= (1ll << 31)) return GTATTN_ERR_INVALID_ARG;
    if (S > 0 && (!length || !tok_off || (max_pages > 0 && !table))) return GTATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(length) |
         reinterpret_cast<uintptr_t>(tok_off)) & 3u)
        return GTATTN_ERR_INVALID_ARG;
    r->table = table;
    r->length = length;
    r->tok_off = tok_off;
    r->S = (int)S;
    r->T = (int)T;
    r->max_pages = (int)max_pages;
    return GTATTN_OK;
}

namespace {

// ---------------------------------------------------------------------------
// slots
// ---------------------------------------------------------------------------
struct SlotsArgs {
    const int* len;
    const int* add;
    int* table;
    const int* free_pages;
    int* new_len;
    int* tok_off;
    int* slots;
    int* counts;
    int S, max_pages, n_free, T, page;
};

// One request's sizes: tokens held and added, pages held and needed, and
// whether its sizes are out of range (it then adds nothing).
__device__ __forceinline__ void slots_need(const SlotsArgs& a, int s, int& len, int& add, int& have, int& need,
                                           int& bad) {
    len = a.len[s];
    add = a.add[s];
    bad = len < 0 || add < 0 || (long long)len + add > (long long)a.max_pages * a.page;
    if (bad) add = 0;
    const unsigned up = a.page - 1;
    have = (static_cast<unsigned>(max(len, 0)) + up) / a.page;
    need = bad ? 0 : static_cast<int>((static_cast<unsigned>(len + add) + up) / a.page) - have;
}

// Simplest form: one thread walks the requests in order.
__global__ void k_slots_serial(SlotsArgs a) {
    if (threadIdx.x || blockIdx.x) return;
    long long tok = 0, pages = 0;
    int taken = 0, refused = 0;
    for (int s = 0; s < a.S; ++s) {
        int len, add, have, need, bad;
        slots_need(a, s, len, add, have, need, bad);
        const bool ok = !bad && (add == 0 || tok + add <= a.T) && (need == 0 || pages + need <= a.n_free);
        a.tok_off[s] = (int)min(tok, (long long)a.T);
        a.new_len[s] = ok ? len + add : len;
        refused += !ok;
        if (ok) {
            if (need) taken = (int)(pages + need);
            for (int p = 0; p < need; ++p) a.table[(int64_t)s * a.max_pages + have + p] = a.free_pages[pages + p];
        }
        for (int i = 0; i < add && tok + i < a.T; ++i) {
            const int pos = len + i;
            a.slots[tok + i] = ok ? a.table[(int64_t)s * a.max_pages + pos / a.page] * a.page + pos % a.page : -1;
        }
        tok += add;
        pages += need;
    }
    const int end = (int)min(tok, (long long)a.T);
    a.tok_off[a.S] = end;
    for (int t = end; t < a.T; ++t) a.slots[t] = -1;
    a.counts[0] = taken;
    a.counts[1] = end;
    a.counts[2] = refused;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// The smallest power of two 2^e with amax <= 448 * 2^e, e clamped.
__device__ __forceinline__ float power_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);   // 448 = 1.75 * 2^8
    e = min(max(e, kScaleMinExp), kScaleMaxExp);   // (zero and subnormals: the least)
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

constexpr int kAppendThreads = 128;

// A block per (token, K/V head, K or V): blocks whose token does not begin a
// run of consecutive slots in a page leave; the others take the whole run.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
k_append(CacheView c, const T* __restrict__ K, const T* __restrict__ V, const int* __restrict__ slots, int T_rows) {
    __shared__ float red[kAppendThreads / 32];
    __shared__ int s_n;
    const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    const bool is_v = blockIdx.z != 0;
    const int total = c.pages * c.page;
    const int slot = slots[t];
    if (slot < 0 || slot >= total) return;
    const int f = slot & (c.page - 1), pid = slot >> c.lp;
    if (f > 0 && t > 0 && slots[t - 1] == slot - 1) return;
    if (tid == 0) {
        int n = 1;
        while (f + n < c.page && t + n < T_rows && slots[t + n] == slot + n) ++n;
        s_n = n;
    }
    __syncthreads();
    const int n = s_n, D = c.D, HD = c.Hkv * D;
    const T* x = (is_v ? V : K) + (int64_t)t * HD + g * D;
    float amax = 0.f;
    for (int i = tid; i < n * D; i += kAppendThreads) {
        const float v = fabsf(load_elem(x, (int64_t)(i / D) * HD + i % D));
        if (v < INFINITY) amax = fmaxf(amax, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const int64_t ph = (int64_t)pid * c.Hkv + g;
    float* sp = (is_v ? c.vscale : c.kscale) + ph;
    uint8_t* tile = (is_v ? c.v8 : c.k8) + ph * c.page * D;
    const float old = f > 0 ? *sp : 0.f;
    const float now = fmaxf(old, power_scale(amax));
    if (f > 0 && now != old) {
        const float ratio = old / now;
        for (int i = tid; i < f * D; i += kAppendThreads) tile[i] = f32_e4m3(e4m3_f32(tile[i]) * ratio);
    }
    for (int i = tid; i < n * D; i += kAppendThreads)
        tile[f * D + i] = f32_e4m3(load_elem(x, (int64_t)(i / D) * HD + i % D) / now);
    __syncthreads();   // (also: everyone has read *sp)
    if (tid == 0) *sp = now;
    if (!is_v && c.kmean) {
        for (int d = tid; d < D; d += kAppendThreads) {
            float sum = 0.f;   // exact: at most 64 multiples of 2^-9 up to 448
            for (int i = 0; i < f + n; ++i) sum += e4m3_f32(tile[i * D + d]);
            c.kmean[ph * D + d] = __float2bfloat16_rn(sum * now / static_cast<float>(f + n));
        }
    }
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" gtattn_status gtattn_cache_slots(const int32_t* length, const int32_t* add, int32_t* table,
                                            const int32_t* free_pages, int32_t* new_length, int32_t* tok_off,
                                            int32_t* slots, int32_t* counts, int64_t S, int64_t max_pages,
                                            int64_t n_free, int64_t T, int page, cudaStream_t stream) {
    constexpr int64_t kLim = (1ll << 31) - 1;
    if (S < 0 || max_pages < 0 || n_free < 0 || T < 0 || S >= kLim || max_pages >= kLim || n_free >= kLim || T >= kLim)
        return GTATTN_ERR_INVALID_ARG;
    if (page != 16 && page != 32 && page != 64) return GTATTN_ERR_INVALID_ARG;
    if (max_pages * page >= (1ll << 31)) return GTATTN_ERR_INVALID_ARG;
    if (!tok_off || !counts || (T > 0 && !slots) || (n_free > 0 && !free_pages)) return GTATTN_ERR_INVALID_ARG;
    if (S > 0 && (!length || !add || !new_length || (max_pages > 0 && !table))) return GTATTN_ERR_INVALID_ARG;
    uintptr_t al = 0;
    for (const void* p : {(const void*)length, (const void*)add, (const void*)table, (const void*)free_pages,
                          (const void*)new_length, (const void*)tok_off, (const void*)slots, (const void*)counts})
        al |= reinterpret_cast<uintptr_t>(p);
    if (al & 3u) return GTATTN_ERR_INVALID_ARG;
    const SlotsArgs a{length, add, table, free_pages, new_length, tok_off, slots, counts,
                      (int)S, (int)max_pages, (int)n_free, (int)T, page};
    ProfScope ps(GTATTN_KCAT_CACHE, 1, stream);
    k_slots_serial<<<1, 32, 0, stream>>>(a);
    GT_CUDA(cudaGetLastError());
    return GTATTN_OK;
}

extern "C" gtattn_status gtattn_cache_append(const gtattn_cache* cache, const void* K, const void* V,
                                             const int32_t* slots, int64_t T, gtattn_dtype dtype,
                                             cudaStream_t stream) {
    CacheView c;
    GT_TRY(check_cache(cache, 1, &c));
    if (T < 0 || T >= (1ll << 31) - 1) return GTATTN_ERR_INVALID_ARG;
    if (dtype != GTATTN_F32 && dtype != GTATTN_BF16 && dtype != GTATTN_BF16_OUT_F32) return GTATTN_ERR_INVALID_ARG;
    if (T > 0 && (!K || !V || !slots)) return GTATTN_ERR_INVALID_ARG;
    const uintptr_t esz = dtype == GTATTN_F32 ? 4 : 2;
    if (((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & (esz - 1)) ||
        (reinterpret_cast<uintptr_t>(slots) & 3u))
        return GTATTN_ERR_INVALID_ARG;
    if (T == 0 || c.pages == 0) return GTATTN_OK;
    ProfScope ps(GTATTN_KCAT_CACHE, 1, stream);
    const dim3 grid((unsigned)T, c.Hkv, 2);
    if (dtype == GTATTN_F32)
        k_append<float><<<grid, kAppendThreads, 0, stream>>>(c, static_cast<const float*>(K),
                                                              static_cast<const float*>(V), slots, (int)T);
    else
        k_append<__nv_bfloat16><<<grid, kAppendThreads, 0, stream>>>(c, static_cast<const __nv_bfloat16*>(K),
                                                                      static_cast<const __nv_bfloat16*>(V), slots,
                                                                      (int)T);
    GT_CUDA(cudaGetLastError());
    return GTATTN_OK;
}
