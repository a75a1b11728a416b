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

// A block owns kSlotThreads consecutive requests: it adds up the sizes of all
// requests before them, scans its own, and its threads then take the
// requests' tokens one by one (a binary search in shared memory names the
// token's request), so that one long prompt is spread as evenly as many short
// ones; gridDim.y blocks share a group's tokens.  Bound by latency: two
// dependent loads, two scans and the stores.
constexpr int kSlotThreads = 256;

// exclusive scan over the block; *total receives the sum
__device__ __forceinline__ long long slot_scan(long long v, long long* total) {
    __shared__ long long sums[kSlotThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSlotThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSlotThreads) k_slots(SlotsArgs a, int lp) {
    __shared__ long long s_tok[kSlotThreads + 1];                  // first token of each own request
    __shared__ int s_len[kSlotThreads], s_have[kSlotThreads], s_page[kSlotThreads];   // s_page: first new page; -1: refused
    let_next_start();
    after_previous();
    const int tid = threadIdx.x, s0 = blockIdx.x * kSlotThreads, s = s0 + tid;
    const bool lead = blockIdx.y == 0, final_block = blockIdx.x == gridDim.x - 1;
    int len = 0, add = 0, have = 0, need = 0, bad = 0;
    // everything before this block's requests
    long long tok = 0, pages = 0, refused = 0;
    for (int i = tid; i < s0; i += kSlotThreads) {
        slots_need(a, i, len, add, have, need, bad);
        tok += add;
        pages += need;
        refused += bad;
    }
    len = add = have = need = bad = 0;
    if (s < a.S) slots_need(a, s, len, add, have, need, bad);
    long long tok0 = 0, pages0 = 0, own_tok, own_pages;
    if (s0 > 0) {
        slot_scan(tok, &tok0);
        slot_scan(pages, &pages0);
    }
    const long long t_at = tok0 + slot_scan(add, &own_tok), p_at = pages0 + slot_scan(need, &own_pages);
    const bool ok = !bad && (add == 0 || t_at + add <= a.T) && (need == 0 || p_at + need <= a.n_free);
    s_tok[tid] = t_at;
    s_len[tid] = len;
    s_have[tid] = have;
    s_page[tid] = ok ? static_cast<int>(p_at) : -1;
    if (lead && s < a.S) {
        a.tok_off[s] = static_cast<int>(min(t_at, (long long)a.T));
        a.new_len[s] = ok ? len + add : len;
    }
    __syncthreads();
    const long long end = min(tok0 + own_tok, (long long)a.T);
    const int mask = a.page - 1;
    for (long long t = tok0 + blockIdx.y * kSlotThreads + tid; t < end; t += static_cast<long long>(gridDim.y) * kSlotThreads) {
        int lo = 0;      // the last own request that begins at or before t
#pragma unroll
        for (int step = kSlotThreads / 2; step > 0; step >>= 1)
            if (s_tok[lo + step] <= t) lo += step;
        int slot = -1;
        if (s_page[lo] >= 0) {
            const int pos = s_len[lo] + static_cast<int>(t - s_tok[lo]), p = pos >> lp;
            int* row = a.table + static_cast<int64_t>(s0 + lo) * a.max_pages;
            int id;
            if (p >= s_have[lo]) {     // a new page: its first token is a new one, and writes it down
                id = a.free_pages[s_page[lo] + p - s_have[lo]];
                if ((pos & mask) == 0) row[p] = id;
            } else {
                id = row[p];
            }
            slot = static_cast<int>(static_cast<unsigned>(id) * a.page + (pos & mask));
        }
        a.slots[t] = slot;
    }
    if (!final_block) return;
    for (long long t = end + blockIdx.y * kSlotThreads + tid; t < a.T; t += static_cast<long long>(gridDim.y) * kSlotThreads)
        a.slots[t] = -1;
    if (!lead) return;
    long long taken = pages0 + own_pages, no = 0;
    if (tok0 + own_tok <= a.T && pages0 + own_pages <= a.n_free) {     // all fit: only bad sizes are refused
        slot_scan(refused + bad, &no);
    } else {                                                           // walk them all again
        long long carry_t = 0, carry_p = 0;
        long long best = 0;
        refused = 0;
        for (int i0 = 0; i0 < a.S; i0 += kSlotThreads) {
            len = add = have = need = bad = 0;
            if (i0 + tid < a.S) slots_need(a, i0 + tid, len, add, have, need, bad);
            long long all_t, all_p;
            const long long ta = carry_t + slot_scan(add, &all_t), pa = carry_p + slot_scan(need, &all_p);
            const bool fine = !bad && (add == 0 || ta + add <= a.T) && (need == 0 || pa + need <= a.n_free);
            if (i0 + tid < a.S) refused += !fine;
            if (fine && need) best = pa + need;      // (rises with the request)
            carry_t += all_t;
            carry_p += all_p;
        }
        slot_scan(refused, &no);
        // the largest of the threads' last pages
        __shared__ long long s_best[kSlotThreads];
        s_best[tid] = best;
        __syncthreads();
        taken = 0;
        for (int i = 0; i < kSlotThreads; ++i) taken = max(taken, s_best[i]);
    }
    if (tid == 0) {
        const int all = static_cast<int>(min(tok0 + own_tok, (long long)a.T));
        a.tok_off[a.S] = all;
        a.counts[0] = static_cast<int>(taken);
        a.counts[1] = all;
        a.counts[2] = static_cast<int>(no);
    }
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
constexpr int kAppendSpan = 16;

// A block per (token, K/V head, K or V): blocks whose token does not begin a
// run of consecutive slots in a page leave; the others take the whole run.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
k_append(CacheView c, const T* __restrict__ K, const T* __restrict__ V, const int* __restrict__ slots, int T_rows) {
    __shared__ float red[kAppendThreads / 32];
    __shared__ int s_n;
    let_next_start();
    after_previous();
    const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    const bool is_v = blockIdx.z != 0;
    const int total = c.pages * c.page;
    const int slot = slots[t];
    if (slot < 0 || slot >= total) return;
    const int f = slot & (c.page - 1), pid = slot >> c.lp;
    if (f > 0 && t > 0 && slots[t - 1] == slot - 1) return;
    if (tid == 0) {
        int n = 1;
        while (f + n < c.page && T_rows - t > n && slots[t + n] == slot + n) ++n;
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


// The same for D a power of two from 8 on, rows 16-byte aligned: WPR warps per
// run (and head, and K or V), a lane 8 features at a time, always the same 8
// columns, so the column sums of the mean stay in its registers (they are
// exact in fp32, in any order).  Prompts take a warp per run, which looks at
// `span` consecutive tokens for runs that begin there: with a block per run
// its barriers and set-up were most of the 350 instructions a thread spent on
// 16 elements (14 k fp32 tokens of 8 x 64: 26.4 us, now 21.4).  Batches too small
// to fill the SMs with warps take a block per run, four warps on the page's
// rows (128 single tokens of 8 x 128: 7.0 us, with a warp 10.6: the earlier
// keys that the mean reads come one after another).
// Bound by memory: the new rows are read once from DRAM (the second pass over
// them hits L1), a page's earlier keys are read for its mean.
__device__ __forceinline__ uint2 eight_e4m3(const float (&x)[8], bool finite) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if (!finite) {               // (a NaN converts to NaN by itself, an infinity would to 448)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f32_e4m3(x[2 * i]) | (f32_e4m3(x[2 * i + 1]) << 8);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
__device__ __forceinline__ void eight_f32(uint2 c, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3)));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The largest |x| of eight as bits (what is not finite is at or above 0x7f800000).
__device__ __forceinline__ uint32_t eight_top(const float (&x)[8]) {
    uint32_t t = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(x[k]) & 0x7fffffffu);
    return t;
}
// The same of the finite ones.
__device__ __forceinline__ uint32_t eight_finite_top(const float (&x)[8]) {
    uint32_t t = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = __float_as_uint(x[k]) & 0x7fffffffu;
        if (u < 0x7f800000u) t = max(t, u);
    }
    return t;
}

template <typename T, int WPR>
__global__ void __launch_bounds__(kAppendThreads, 12)
k_append8(CacheView c, const T* __restrict__ K, const T* __restrict__ V, const int* __restrict__ slots, int T_rows,
          int span, int l8) {       // l8 = log2(D / 8)
    let_next_start();
    after_previous();
    const unsigned full = 0xffffffffu;
    constexpr int WARPS = kAppendThreads / 32;
    static_assert(WPR == 1 || WPR == WARPS, "a warp or the block per run");
    __shared__ uint32_t red[WARPS];
    __shared__ float cols[WPR > 1 ? WARPS : 1][WPR > 1 ? kCacheMaxD : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // K and V of each K/V head in turn; the heads of a token side by side in the grid (they share DRAM pages)
    const unsigned heads = WPR > 1 ? 2 * c.Hkv : (2 * c.Hkv + WARPS - 1) / WARPS;
    const int head = WPR > 1 ? blockIdx.x % heads : (blockIdx.x % heads) * WARPS + warp;
    if (head >= 2 * c.Hkv) return;
    auto run_max = [&](uint32_t v) {     // over the run's warps
        v = __reduce_max_sync(full, v);
        if constexpr (WPR > 1) {
            __syncthreads();
            if (lane == 0) red[warp] = v;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v = max(v, red[w]);
        }
        return v;
    };
    const int g = head >> 1;
    const bool is_v = head & 1;
    const int D = c.D, HD = c.Hkv * D, W = 1 << l8;
    const unsigned total = static_cast<unsigned>(c.pages) * c.page;
    const int first = static_cast<int>(min(static_cast<long long>(blockIdx.x / heads) * span, 0x7fffffffll));
    const int cc = lane & (W - 1), rows = (32 * WPR) >> l8;                       // this lane's columns, the row step
    const int rr = (WPR > 1 ? warp * 32 + lane : lane) >> l8;                     // and its first row
    const bool mean = !is_v && c.kmean;
    // lane i looks at token first + i
    bool begins = false;
    if (lane < span && T_rows - first > lane) {
        const int slot = slots[first + lane];
        begins = static_cast<unsigned>(slot) < total &&
                 ((slot & (c.page - 1)) == 0 || first + lane == 0 || slots[first + lane - 1] != slot - 1);
    }
    unsigned todo = __ballot_sync(full, begins);
    while (todo) {
        const int t = first + __ffs(todo) - 1;
        todo &= todo - 1;
        const int slot = slots[t];
        const int f = slot & (c.page - 1), pid = slot >> c.lp;
        // run length: tokens t + i in slot + i, as far as the page goes
        int n;
        {
            const int i0 = lane, i1 = lane + 32;
            const bool b0 = !(f + i0 < c.page && T_rows - t > i0 && slots[t + i0] == slot + i0);
            const bool b1 = !(f + i1 < c.page && T_rows - t > i1 && slots[t + i1] == slot + i1);
            const unsigned m0 = __ballot_sync(full, b0), m1 = __ballot_sync(full, b1);
            n = m0 ? __ffs(m0) - 1 : m1 ? 32 + __ffs(m1) - 1 : 64;
        }
        const T* x = (is_v ? V : K) + static_cast<int64_t>(t) * HD + g * D + cc * 8;
        const int64_t ph = static_cast<int64_t>(pid) * c.Hkv + g;
        float* sp = (is_v ? c.vscale : c.kscale) + ph;
        uint8_t* tile = (is_v ? c.v8 : c.k8) + (ph << c.lp) * D + cc * 8;
        const float old = f > 0 ? *sp : 0.f;
        uint32_t top = 0;
#pragma unroll(WPR > 1 ? 2 : 8)
        for (int i = rr; i < n; i += rows) {
            Eight<T> e;
            e.load(x + static_cast<int64_t>(i) * HD);
            top = max(top, eight_top(e.x));
        }
        top = run_max(top);
        const bool finite = top < 0x7f800000u;
        if (!finite) {                                      // once more, of the finite ones
            top = 0;
            for (int i = rr; i < n; i += rows) {
                Eight<T> e;
                e.load(x + static_cast<int64_t>(i) * HD);
                top = max(top, eight_finite_top(e.x));
            }
            top = run_max(top);
        }
        const float now = fmaxf(old, power_scale(__uint_as_float(top)));
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const bool grown = f > 0 && now != old;
        if (grown || mean) {
            const float ratio = grown ? old / now : 1.f;
#pragma unroll(WPR > 1 ? 4 : 8)
            for (int i = rr; i < f; i += rows) {
                uint2* p = reinterpret_cast<uint2*>(tile + i * D);
                uint2 code = *p;
                float y[8];
                eight_f32(code, y);
                if (grown) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= ratio;
                    code = eight_e4m3(y, true);
                    *p = code;
                    eight_f32(code, y);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += y[k];
            }
        }
        const float inv = 1.f / now;                        // (a power of two: exact)
#pragma unroll(WPR > 1 ? 2 : 4)
        for (int i = rr; i < n; i += rows) {
            Eight<T> e;
            e.load(x + static_cast<int64_t>(i) * HD);
#pragma unroll
            for (int k = 0; k < 8; ++k) e.x[k] *= inv;
            const uint2 code = eight_e4m3(e.x, finite);
            *reinterpret_cast<uint2*>(tile + (f + i) * D) = code;
            if (mean) {
                float y[8];
                eight_f32(code, y);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += y[k];
            }
        }
        if (lane == 0 && (WPR == 1 || warp == 0)) *sp = now;      // (a block's warps have read `old`: run_max)
        if (mean) {      // (exact sums: the order of the additions does not matter)
            const float count = static_cast<float>(f + n);
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                for (int o = W; o < 32; o <<= 1) sum[k] += __shfl_xor_sync(full, sum[k], o);
                if (WPR > 1 && lane < W) cols[warp][cc * 8 + k] = sum[k];
            }
            if constexpr (WPR > 1) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = (cols[0][cc * 8 + k] + cols[1][cc * 8 + k]) + (cols[2][cc * 8 + k] + cols[3][cc * 8 + k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = sum[k] * now / count;
            if (lane < W && (WPR == 1 || warp == 0))
                *reinterpret_cast<uint4*>(c.kmean + ph * D + cc * 8) =
                    make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
        __syncwarp();
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
    // every block reads the lengths before its own requests again: they must not change meanwhile
    if (S > 0 && new_length < length + S && length < new_length + S) return GTATTN_ERR_INVALID_ARG;
    const SlotsArgs a{length, add, table, free_pages, new_length, tok_off, slots, counts,
                      (int)S, (int)max_pages, (int)n_free, (int)T, page};
    ProfScope ps(GTATTN_KCAT_CACHE, 1, stream);
    const int groups = std::max<int>(1, (int)((S + kSlotThreads - 1) / kSlotThreads));
    // blocks of a group: about 1024 tokens each, all groups within a wave or two
    const int share = (int)std::min<int64_t>(std::max<int64_t>(1, T / groups / 1024), std::max(1, 4 * num_sms() / groups));
    GT_CUDA(launch_after(k_slots, dim3(groups, share), kSlotThreads, 0, stream, a, page == 16 ? 4 : page == 32 ? 5 : 6));
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
    const bool eights = c.D >= 8 && (c.D & (c.D - 1)) == 0 &&
                        ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15u) == 0;
    if (eights) {
        int l8 = 0;
        while ((8 << l8) < c.D) ++l8;
        const int64_t warps = T * c.Hkv * 2;
        const int span = (int)std::min<int64_t>(kAppendSpan, std::max<int64_t>(1, warps / (32 * num_sms())));
        constexpr int WARPS = kAppendThreads / 32;
        const bool block = span == 1;
        const auto go = [&](auto* one, auto* all, auto* Kp, auto* Vp) {
            const int64_t heads = block ? 2 * c.Hkv : (2 * c.Hkv + WARPS - 1) / WARPS;
            const dim3 grid((unsigned)((T + span - 1) / span * heads));     // (below 2^31: so many rows fill no GPU)
            return launch_after(block ? all : one, grid, kAppendThreads, 0, stream, c, Kp, Vp, slots, (int)T, span, l8);
        };
        using B = __nv_bfloat16;
        GT_CUDA(dtype == GTATTN_F32
                    ? go(k_append8<float, 1>, k_append8<float, WARPS>, static_cast<const float*>(K), static_cast<const float*>(V))
                    : go(k_append8<B, 1>, k_append8<B, WARPS>, static_cast<const B*>(K), static_cast<const B*>(V)));
        return GTATTN_OK;
    }
    const dim3 grid((unsigned)T, c.Hkv, 2);
    GT_CUDA(dtype == GTATTN_F32
                ? launch_after(k_append<float>, grid, kAppendThreads, 0, stream, c, static_cast<const float*>(K),
                               static_cast<const float*>(V), slots, (int)T)
                : launch_after(k_append<__nv_bfloat16>, grid, kAppendThreads, 0, stream, c,
                               static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V), slots, (int)T));
    return GTATTN_OK;
}
