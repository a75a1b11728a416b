// cache_select.cu -- for each new token and K/V head, the pages of the cache
// that score highest against the token's queries.
//
// score(p, g) = sum over the heads h of group g of q_h . kmean[p, g]: the
// group's queries are added first, so a page costs one dot product of D.  Two
// steps: k_scores forms every score in fp32 -- it reads the page means, which
// is what bounds the call -- and k_pick, a block per (token, head), finds the
// k-th largest and lists the pages.
//
// The choice has to be that of 64 bits.  An fp32 score is off by at most
// E = gamma * |q|_1 * max|kmean| (standard bound of a sum of products), so a
// page above (k-th + 2E) is in and one below (k-th - 2E) is out whatever the
// rounding; if what lies between is more than is still wanted, those pages,
// and only those, are scored again in 64 bits.  With scores that spread like
// their terms that is a page in some thousand rows; rows whose bound is not
// finite (fp32 overflows, a mean holds a NaN) take all their pages there.
#include "cache.cuh"

#include <algorithm>

namespace gt {
namespace {

struct SelArgs {
    CacheView c;
    CacheRows r;
    const void* Q;
    int* sel;
    float2* score;     // [items, max_pages]: fp32 score and the largest |mean| of the page
    float* qnorm;      // [items]: sum of |q| over the group
    int H, G, n_sel;
    int t0;            // first token of this pass
    int chunks;        // blocks per item of k_scores
    int q_vec;         // Q's rows are 16-byte aligned (and D a multiple of 8)
};

constexpr int kScoreWarps = 4;
constexpr int kScorePages = 128;     // pages of a block: 32 a warp, 8 at a time

// Row of pass item i, its K/V head, request, position; false behind the last row.
struct SelItem {
    int t, g, s, pos, own;
};
__device__ __forceinline__ bool sel_item(const SelArgs& a, int64_t item, SelItem* it) {
    it->t = a.t0 + static_cast<int>(item / a.c.Hkv);
    it->g = static_cast<int>(item % a.c.Hkv);
    if (it->t >= __ldg(a.r.tok_off + a.r.S)) return false;
    it->s = request_of(a.r.tok_off, a.r.S, it->t);
    it->pos = position_of(a.r, a.c.page, it->s, it->t);
    it->own = it->pos < 0 ? -1 : it->pos >> a.c.lp;
    return true;
}

// Four lanes hold a page's mean: lane cq takes the 16-byte pieces cq, cq + 4,
// ... of it (NCH of them), eight pages a warp at a time; the lane's part of
// the group's query stays in registers.
template <typename T, int NCH>
__global__ void __launch_bounds__(kScoreWarps * 32) k_scores(SelArgs a) {
    const int64_t item = blockIdx.x / a.chunks;
    const int p0 = static_cast<int>(blockIdx.x % a.chunks) * kScorePages;
    SelItem it;
    if (!sel_item(a, item, &it)) return;
    // (a row that takes every page needs no score)
    if (it.own <= a.n_sel - 1 || (p0 >= it.own && p0 > 0)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cq = lane & 3;
    const CacheView& c = a.c;
    const int D = c.D;
    const bool vec = (D & 7) == 0;       // (means are 16-byte aligned, so are rows of 8 features)
    float q[NCH][8], norm = 0.f;
    const T* Q = static_cast<const T*>(a.Q) + (static_cast<int64_t>(it.t) * a.H + it.g * a.G) * D;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int d = (cq + 4 * i) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) q[i][k] = 0.f;
        if (a.q_vec) {
            if (d < D) {
#pragma unroll 4
                for (int h = 0; h < a.G; ++h) {
                    Eight<T> e;
                    e.load(Q + h * D + d);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        q[i][k] += e.x[k];
                        norm += fabsf(e.x[k]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (d + k < D)
                    for (int h = 0; h < a.G; ++h) {
                        const float v = load_elem(Q, h * D + d + k);
                        q[i][k] += v;
                        norm += fabsf(v);
                    }
        }
    }
    if (p0 == 0 && warp == 0) {
        norm += __shfl_xor_sync(0xffffffffu, norm, 1);
        norm += __shfl_xor_sync(0xffffffffu, norm, 2);
        if (lane == 0) a.qnorm[item] = norm;
    }
    const int* row = a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages;
    const int pw = p0 + warp * 32;
    const int end = min(it.own, pw + 32);
    const int id = pw + lane < end ? __ldg(row + pw + lane) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int p = pw + u * 8 + (lane >> 2);
        const int pid = __shfl_sync(0xffffffffu, id, u * 8 + (lane >> 2));
        const bool ok = p < end && static_cast<unsigned>(pid) < static_cast<unsigned>(c.pages);
        const __nv_bfloat16* m = c.kmean + (static_cast<int64_t>(ok ? pid : 0) * c.Hkv + it.g) * D;
        uint4 w[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int d = (cq + 4 * i) * 8;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (ok && d < D) {
                if (vec) {
                    w[i] = __ldg(reinterpret_cast<const uint4*>(m + d));
                } else {
                    uint32_t* x = reinterpret_cast<uint32_t*>(&w[i]);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (d + k < D)
                            x[k >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(m[d + k])) << (16 * (k & 1));
                }
            }
        }
        float s = 0.f;
        uint32_t big = 0;         // the largest |mean|, as bits, two at a time
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s = fmaf(q[i][2 * k], bf16lo(x[k]), s);
                s = fmaf(q[i][2 * k + 1], bf16hi(x[k]), s);
                big = __vmaxu2(big, x[k] & 0x7fff7fffu);
            }
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        big = max(big & 0xffffu, big >> 16);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        if (cq == 0 && p < end)
            a.score[item * a.r.max_pages + p] = make_float2(s, __uint_as_float(big << 16));
    }
}

constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickKeys = 8192;      // keys held in shared memory; rows of more pages read them again

__device__ __forceinline__ uint32_t key_of(float x) {        // rises with x; -0 as 0
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ unsigned long long key_of(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// sum over the block; two barriers
__device__ __forceinline__ int block_sum(int v, int* sums) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
    __syncthreads();
    int x = 0;
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w) x += sums[w];
    return x;
}

// The k-th largest of key(0 .. n-1), bit by bit from the top: the largest
// value that at least k keys reach.
template <typename U, typename F> __device__ __forceinline__ U kth_largest(int n, int k, F key, int* sums) {
    U v = 0;
    for (U bit = U(1) << (8 * sizeof(U) - 1); bit; bit >>= 1) {
        const U x = v | bit;
        int cnt = 0;
        for (int i = threadIdx.x; i < n; i += kPickThreads) cnt += key(i) >= x;
        if (block_sum(cnt, sums) >= k) v = x;
    }
    return v;
}

// The group's queries added up in 64 bits (a block; a barrier has to follow).
template <typename T> __device__ void query_sums(const SelArgs& a, const SelItem& it, double* qs) {
    for (int d = threadIdx.x; d < a.c.D; d += kPickThreads) {
        double v = 0;
        for (int h = 0; h < a.G; ++h)
            v += load_elem(static_cast<const T*>(a.Q), (static_cast<int64_t>(it.t) * a.H + it.g * a.G + h) * a.c.D + d);
        qs[d] = v;
    }
}
// Page p's score in 64 bits, NaN as -inf (a warp).
__device__ __forceinline__ double exact_score(const SelArgs& a, const SelItem& it, const double* qs, int p, int lane) {
    const int pid = __ldg(a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages + p);
    double v = 0;
    if (static_cast<unsigned>(pid) < static_cast<unsigned>(a.c.pages)) {
        const __nv_bfloat16* m = a.c.kmean + (static_cast<int64_t>(pid) * a.c.Hkv + it.g) * a.c.D;
        for (int d = lane; d < a.c.D; d += 32) v = fma(qs[d], static_cast<double>(__bfloat162float(m[d])), v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v != v ? -INFINITY : v;
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) k_pick(SelArgs a, int64_t items) {
    __shared__ uint32_t keys[kPickKeys];
    __shared__ double qs[kCacheMaxD];
    __shared__ int sums[kPickWarps];
    __shared__ uint32_t s_big[kPickWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t item = blockIdx.x;
    SelItem it;
    if (item >= items || !sel_item(a, item, &it)) return;
    const CacheView& c = a.c;
    const int own = it.own, k = a.n_sel - 1;
    int* out = a.sel + (static_cast<int64_t>(it.t) * c.Hkv + it.g) * a.n_sel;
    if (own <= k) {                      // every page up to its own
        for (int i = tid; i < a.n_sel; i += kPickThreads) out[i] = i <= own ? i : -1;
        return;
    }
    // (own > k >= 0: k of the earlier pages, then its own)
    if (tid == 0) out[k] = own;
    if (k == 0) return;
    float2* score = a.score + item * a.r.max_pages;
    const bool held = own <= kPickKeys;
    uint32_t bits = 0;                   // of the largest |mean| (a NaN is above all)
    for (int i = tid; i < own; i += kPickThreads) {
        const float2 x = score[i];
        if (held) keys[i] = key_of(x.x);
        bits = max(bits, __float_as_uint(x.y));
    }
    bits = __reduce_max_sync(0xffffffffu, bits);
    if (lane == 0) s_big[warp] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w) bits = max(bits, s_big[w]);
    const float big = __uint_as_float(bits);
    // roundings of one score: G - 1 in the group's sum, D / 4 + 2 in the dot product, one each product
    const float gamma = (a.G + c.D / 4 + 8) * 6.0e-8f * 1.01f;
    const float norm = a.qnorm[item];
    const float bound = 2.f * (gamma * norm * big) + 1e-36f;     // 2E; the last: products below fp32's range
    auto key = [&](int i) { return held ? keys[i] : key_of(score[i].x); };
    float lo = 0.f, hi = 0.f;
    bool all = !(bound < 1e37f) || !(norm < 1e37f) || !(big < 1e37f) || !(norm * big < 1e37f);
    bool redo = all;
    int mid = 0, want = 0;               // pages between, and how many of them are in
    if (!all) {
        const float kth = key_value(kth_largest<uint32_t>(own, k, key, sums));
        const float pad = bound + fabsf(kth) * 3e-7f;            // (and the rounding of these two)
        lo = kth - pad;
        hi = kth + pad;
        int in = 0;
        for (int i = tid; i < own; i += kPickThreads) {
            const float x = key_value(key(i));
            in += x > hi;
            mid += x >= lo && x <= hi;
        }
        in = block_sum(in, sums);
        mid = block_sum(mid, sums);
        want = k - in;
        redo = mid != want;
    }
    // few pages between (the usual case): each scored by a warp in 64 bits and
    // ranked among them; its fp32 score then says in or out
    const int few = all ? 0 : mid;
    if (redo && few > 0 && few <= kPickThreads) {
        __shared__ int z_at[kPickThreads];
        __shared__ double z_score[kPickThreads];
        __shared__ int z_n;
        if (tid == 0) z_n = 0;
        query_sums<T>(a, it, qs);
        __syncthreads();
        for (int i = tid; i < own; i += kPickThreads) {
            const float x = key_value(key(i));
            if (x >= lo && x <= hi) z_at[atomicAdd(&z_n, 1)] = i;
        }
        __syncthreads();
        for (int z = warp; z < few; z += kPickWarps) {
            const double v = exact_score(a, it, qs, z_at[z], lane);
            if (lane == 0) z_score[z] = v;
        }
        __syncthreads();
        if (tid < few) {
            const double v = z_score[tid];
            const int i = z_at[tid];
            int rank = 0;
            for (int z = 0; z < few; ++z) rank += z_score[z] > v || (z_score[z] == v && z_at[z] < i);
            const float x = rank < want ? INFINITY : -INFINITY;
            if (held) keys[i] = key_of(x);
            else score[i].x = x;
        }
        __syncthreads();
        redo = false;
    }
    unsigned long long edge = 0;       // redo: the k-th largest, and how many of that value are in
    int ties = 0;
    double* fine = reinterpret_cast<double*>(score);     // redo: a page's score in 64 bits, +inf: in, NaN: out
    if (redo) {
        query_sums<T>(a, it, qs);
        __syncthreads();
        for (int i = warp; i < own; i += kPickWarps) {
            const float x = score[i].x;
            __syncwarp();
            double v;
            if (!all && x > hi) {
                v = INFINITY;
            } else if (!all && !(x >= lo)) {
                v = NAN;
            } else {
                v = exact_score(a, it, qs, i, lane);
            }
            if (lane == 0) fine[i] = v;
        }
        __syncthreads();
        // (pages that are in by their fp32 scores rank before the others: +inf)
        auto fkey = [&](int i) { const double v = fine[i]; return v != v ? 0ull : key_of(v); };
        edge = kth_largest<unsigned long long>(own, k, fkey, sums);
        int above = 0;
        for (int i = tid; i < own; i += kPickThreads) above += fkey(i) > edge;
        ties = k - block_sum(above, sums);
    }
    // list them in rising order: 256 pages at a time
    int at = 0, tied = 0;
    for (int i0 = 0; i0 < own && at < k; i0 += kPickThreads) {
        const int i = i0 + tid;
        bool in = false, tie = false;
        if (i < own) {
            if (redo) {
                const double v = fine[i];
                const unsigned long long f = v != v ? 0ull : key_of(v);
                in = f > edge;
                tie = f == edge;
            } else {
                in = key_value(key(i)) >= lo;
            }
        }
        if (redo) {                      // the first `ties` of the equal ones
            const unsigned m = __ballot_sync(0xffffffffu, tie);
            __syncthreads();
            if (lane == 0) sums[warp] = __popc(m);
            __syncthreads();
            int before = tied, total = 0;
#pragma unroll
            for (int w = 0; w < kPickWarps; ++w) {
                if (w < warp) before += sums[w];
                total += sums[w];
            }
            before += __popc(m & ((1u << lane) - 1));
            in |= tie && before < ties;
            tied += total;
        }
        const unsigned m = __ballot_sync(0xffffffffu, in);
        __syncthreads();
        if (lane == 0) sums[warp] = __popc(m);
        __syncthreads();
        int before = at, total = 0;
#pragma unroll
        for (int w = 0; w < kPickWarps; ++w) {
            if (w < warp) before += sums[w];
            total += sums[w];
        }
        before += __popc(m & ((1u << lane) - 1));
        if (in && before < k) out[before] = i;
        at += total;
    }
}

template <typename T> void launch_scores(const SelArgs& a, int64_t blocks, cudaStream_t s) {
    const unsigned n = static_cast<unsigned>(blocks);
    if (a.c.D <= 32) k_scores<T, 1><<<n, kScoreWarps * 32, 0, s>>>(a);
    else if (a.c.D <= 64) k_scores<T, 2><<<n, kScoreWarps * 32, 0, s>>>(a);
    else if (a.c.D <= 128) k_scores<T, 4><<<n, kScoreWarps * 32, 0, s>>>(a);
    else k_scores<T, 8><<<n, kScoreWarps * 32, 0, s>>>(a);
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" gtattn_status gtattn_cache_select(const gtattn_cache* cache, const void* Q, const int32_t* table,
                                             const int32_t* length, const int32_t* tok_off, int32_t* sel, int64_t S,
                                             int64_t T, int64_t max_pages, int H, int n_sel, gtattn_dtype dtype,
                                             cudaStream_t stream) {
    SelArgs a{};
    GT_TRY(check_cache(cache, 2, &a.c));
    GT_TRY(check_cache_rows(table, length, tok_off, S, T, max_pages, a.c.page, &a.r));
    if (dtype != GTATTN_F32 && dtype != GTATTN_BF16 && dtype != GTATTN_BF16_OUT_F32) return GTATTN_ERR_INVALID_ARG;
    if (H < 1 || H > kCacheMaxHeads || H % a.c.Hkv || n_sel < 1 || n_sel > (1 << 20)) return GTATTN_ERR_INVALID_ARG;
    if (T > 0 && (!Q || !sel)) return GTATTN_ERR_INVALID_ARG;
    const uintptr_t esz = dtype == GTATTN_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(Q) & (esz - 1)) || (reinterpret_cast<uintptr_t>(sel) & 3u))
        return GTATTN_ERR_INVALID_ARG;
    if (T * a.c.Hkv >= (1ll << 31)) return GTATTN_ERR_UNSUPPORTED;
    if (T == 0 || S == 0) return GTATTN_OK;
    a.Q = Q;
    a.sel = sel;
    a.H = H;
    a.G = H / a.c.Hkv;
    a.q_vec = (a.c.D & 7) == 0 && (reinterpret_cast<uintptr_t>(Q) & 15u) == 0;
    a.n_sel = n_sel;
    // rows of at most n_sel pages take them all: nothing to score then
    const bool score = max_pages > n_sel && n_sel > 1;
    a.chunks = score ? (int)((max_pages + kScorePages - 1) / kScorePages) : 1;
    // scores of as many tokens at a time as 256 MB hold (all, but for prompts over long requests)
    const int64_t row = score ? (int64_t)a.c.Hkv * max_pages * sizeof(float2) : 1;
    const int64_t tokens = std::max<int64_t>(1, std::min<int64_t>(T, score ? (256ll << 20) / row : T));
    void* ws = nullptr;
    if (score) {
        GT_TRY(pool_alloc(&ws, (size_t)(tokens * row) + sizeof(float) * (size_t)tokens * a.c.Hkv, stream));
        a.score = static_cast<float2*>(ws);
        a.qnorm = reinterpret_cast<float*>(static_cast<char*>(ws) + tokens * row);
    }
    cudaError_t e = cudaSuccess;
    for (int64_t t0 = 0; t0 < T && e == cudaSuccess; t0 += tokens) {
        a.t0 = (int)t0;
        const int64_t items = std::min(tokens, T - t0) * a.c.Hkv;
        ProfScope ps(GTATTN_KCAT_CACHE, score ? 2 : 1, stream);
        if (dtype == GTATTN_F32) {
            if (score) launch_scores<float>(a, items * a.chunks, stream);
            k_pick<float><<<(unsigned)items, kPickThreads, 0, stream>>>(a, items);
        } else {
            if (score) launch_scores<__nv_bfloat16>(a, items * a.chunks, stream);
            k_pick<__nv_bfloat16><<<(unsigned)items, kPickThreads, 0, stream>>>(a, items);
        }
        e = cudaGetLastError();
    }
    pool_free(ws, stream);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}
