// cache_select.cu -- for each new token and K/V head, the pages of the cache
// that score highest against the token's queries.
//
// score(p, g) = sum over the heads h of group g of q_h . kmean[p, g]: the
// group's queries are added first, so a page costs one dot product of D.  Two
// steps: k_scores forms every score in fp32 -- it reads the page means, which
// is what bounds the call -- and k_pick, a block per (token, head), finds the
// k-th largest and lists the pages; k_select does both where its items alone
// fill the GPU.  64 requests of 9-32 thousand tokens, 8 K/V heads of 128: 16.6
// us in one launch (11 of them reading 43 MB of means), 31 in two.
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
    const int end = __ldg(a.r.tok_off + a.r.S);
    it->s = request_of_warp(a.r.tok_off, a.r.S, it->t, threadIdx.x & 31);
    if (it->t >= end) return false;
    it->pos = position_of(a.r, a.c.page, it->s, it->t);
    it->own = it->pos < 0 ? -1 : it->pos >> a.c.lp;
    return true;
}

// Four lanes hold a page's mean: lane cq takes the 16-byte pieces cq, cq + 4,
// ... of it (NCH of them), eight pages a warp at a time; the lane's part of
// the group's query stays in registers.
template <typename T, int NCH> struct Query {
    float q[NCH][8];
    float norm;      // sum of |q| over the group (all four lanes)
    __device__ __forceinline__ void load(const SelArgs& a, const SelItem& it, int cq) {
        const int D = a.c.D;
        const T* Q = static_cast<const T*>(a.Q) + (static_cast<int64_t>(it.t) * a.H + it.g * a.G) * D;
        norm = 0.f;
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
        norm += __shfl_xor_sync(0xffffffffu, norm, 1);
        norm += __shfl_xor_sync(0xffffffffu, norm, 2);
    }
};
// Roundings that a term of the dot product goes through: the FMAs of its
// chain, two sums of chains, two of lanes.
constexpr int dot_depth(int D) { return 2 * ((D + 31) / 32) + 4; }

// One lane's pieces of a page's mean.
template <int NCH> struct Mean {
    uint4 w[NCH];
    __device__ __forceinline__ void load(const SelArgs& a, const SelItem& it, int pid, bool ok, int cq) {
        const int D = a.c.D;
        ok = ok && static_cast<unsigned>(pid) < static_cast<unsigned>(a.c.pages);
        const __nv_bfloat16* m = a.c.kmean + (static_cast<int64_t>(ok ? pid : 0) * a.c.Hkv + it.g) * D;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int d = (cq + 4 * i) * 8;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (ok && d < D) {
                if ((D & 7) == 0) {      // (means are 16-byte aligned, so are rows of 8 features)
                    w[i] = __ldg(reinterpret_cast<const uint4*>(m + d));
                } else {
                    uint32_t* x = reinterpret_cast<uint32_t*>(&w[i]);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (d + k < D) x[k >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(m[d + k])) << (16 * (k & 1));
                }
            }
        }
    }
    // the score, and the bits of the largest |mean| (all four lanes)
    template <typename T> __device__ __forceinline__ void score(const Query<T, NCH>& q, float& s, uint32_t& big) const {
        float part[4] = {0.f, 0.f, 0.f, 0.f};      // (short chains: dot_depth)
        big = 0;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                part[k] = fmaf(q.q[i][2 * k], bf16lo(x[k]), part[k]);
                part[k] = fmaf(q.q[i][2 * k + 1], bf16hi(x[k]), part[k]);
                big = __vmaxu2(big, x[k] & 0x7fff7fffu);
            }
        }
        s = (part[0] + part[1]) + (part[2] + part[3]);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        big = max(big & 0xffffu, big >> 16);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2)) << 16;
    }
};

template <typename T, int NCH>
__global__ void __launch_bounds__(kScoreWarps * 32) k_scores(SelArgs a) {
    let_next_start();
    after_previous();
    const int64_t item = blockIdx.x / a.chunks;
    const int p0 = static_cast<int>(blockIdx.x % a.chunks) * kScorePages;
    SelItem it;
    if (!sel_item(a, item, &it)) return;
    // (a row that takes every page needs no score)
    if (it.own <= a.n_sel - 1 || (p0 >= it.own && p0 > 0)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cq = lane & 3;
    const int pw = p0 + warp * 32, end = min(it.own, pw + 32);
    const int id = pw + lane < end ? __ldg(a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages + pw + lane) : -1;
    Query<T, NCH> q;
    q.load(a, it, cq);
    if (p0 == 0 && threadIdx.x == 0) a.qnorm[item] = q.norm;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int p = pw + u * 8 + (lane >> 2);
        Mean<NCH> m;
        m.load(a, it, __shfl_sync(0xffffffffu, id, u * 8 + (lane >> 2)), p < end, cq);
        float s;
        uint32_t big;
        m.score(q, s, big);
        if (cq == 0 && p < end) a.score[item * a.r.max_pages + p] = make_float2(s, __uint_as_float(big));
    }
}

constexpr int kPickThreads = 256;    // of k_pick
constexpr int kFusedThreads = 128;   // of k_select
constexpr int kPickKeys = 8192;      // keys held in shared memory; k_pick reads those of rows of more pages again
constexpr int kPickClose = 128;      // close pages ranked in shared memory
constexpr int kPickBins = 256;       // of the scores' histogram

__device__ __forceinline__ uint32_t key_of(float x) {        // rises with x; -0 as 0
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ unsigned long long key_of(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// Sums over the block, one barrier each: the partial sums alternate between
// two places, so that the next call's do not meet this one's readers.
template <int THREADS> struct BlockSum {
    int (*at)[THREADS / 32];     // [2] in shared memory
    int turn;
    __device__ __forceinline__ int operator()(int v) {
        v = __reduce_add_sync(0xffffffffu, v);
        if ((threadIdx.x & 31) == 0) at[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        int x = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) x += at[turn][w];
        turn ^= 1;
        return x;
    }
    // sum over the warps before this one and over all, of one value a warp
    __device__ __forceinline__ int before(int v, int* all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) at[turn][warp] = v;
        __syncthreads();
        int x = 0, sum = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) x += at[turn][w];
            sum += at[turn][w];
        }
        turn ^= 1;
        *all = sum;
        return x;
    }
};

// The k-th largest of key(0 .. n-1), bit by bit from the top: the largest
// value that at least k keys reach.  `top`: no key differs above this bit
// from `common`, whose bits from it down are 0.  Where exactly k keys reach a
// value the least of them is it (half the bits on average).
template <int THREADS, typename U, typename F>
__device__ __forceinline__ U kth_largest(int n, int k, U common, U top, F key, BlockSum<THREADS>& sum, U* least) {
    U v = common;
    for (U bit = top; bit; bit >>= 1) {
        const U x = v | bit;
        int cnt = 0;
        for (int i = threadIdx.x; i < n; i += THREADS) cnt += key(i) >= x;
        cnt = sum(cnt);
        if (cnt >= k) v = x;
        if (cnt == k) {
            U m = ~U(0);
            for (int i = threadIdx.x; i < n; i += THREADS) {
                const U y = key(i);
                if (y >= x) m = min(m, y);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = min(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((threadIdx.x & 31) == 0) least[threadIdx.x >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) m = min(m, least[w]);
            return m;
        }
    }
    return v;
}

// The group's queries added up in 64 bits (a block; a barrier has to follow).
template <typename T, int THREADS> __device__ void query_sums(const SelArgs& a, const SelItem& it, double* qs) {
    for (int d = threadIdx.x; d < a.c.D; d += THREADS) {
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

// The same without the sums at hand: the few pages that are scored again need
// no barrier then (what it reads has just been read: it is in L1 or L2).
template <typename T>
__device__ __forceinline__ double exact_score_alone(const SelArgs& a, const SelItem& it, int p, int lane) {
    const int pid = __ldg(a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages + p);
    const T* Q = static_cast<const T*>(a.Q) + (static_cast<int64_t>(it.t) * a.H + it.g * a.G) * a.c.D;
    double v = 0;
    if (static_cast<unsigned>(pid) < static_cast<unsigned>(a.c.pages)) {
        const __nv_bfloat16* m = a.c.kmean + (static_cast<int64_t>(pid) * a.c.Hkv + it.g) * a.c.D;
        for (int d = lane; d < a.c.D; d += 32) {
            double q = 0;
#pragma unroll 4
            for (int h = 0; h < a.G; ++h) q += load_elem(Q, h * a.c.D + d);
            v = fma(q, static_cast<double>(__bfloat162float(m[d])), v);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v != v ? -INFINITY : v;
}

// Lists the k best of the row's `own` earlier pages (own > k > 0), by a block.
// held: the fp32 scores' keys stand in keys[0 .. own), to be seen after a
// barrier, else in score[].x.  bits: those of this thread's largest |mean|.
// score: [max_pages] in global memory; with `held` only used, and written,
// when many pages are close.
template <typename T, int THREADS>
__device__ __forceinline__ void pick_pages(const SelArgs& a, const SelItem& it, bool held, uint32_t* keys, float2* score,
                                           uint32_t bits, float norm, int* out) {
    constexpr int WARPS = THREADS / 32;
    __shared__ double qs[kCacheMaxD];
    __shared__ int s_sums[2][WARPS];
    __shared__ uint32_t s_red[3][WARPS];
    __shared__ unsigned long long s_least[WARPS];
    __shared__ int z_at[kPickClose];
    __shared__ double z_score[kPickClose];
    __shared__ int z_n, z_members;
    __shared__ int s_bin[kPickBins];
    __shared__ uint32_t z_key[kPickClose], s_kth;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int own = it.own, k = a.n_sel - 1;
    BlockSum<THREADS> sum{s_sums, 0};
    auto key = [&](int i) { return held ? keys[i] : key_of(score[i].x); };
    __syncthreads();
    uint32_t highest = 0, lowest = 0xffffffffu;       // the largest and the least key
    for (int i = tid; i < own; i += THREADS) {
        const uint32_t x = key(i);
        highest = max(highest, x);
        lowest = min(lowest, x);
    }
    for (int i = tid; i < kPickBins; i += THREADS) s_bin[i] = 0;
    bits = __reduce_max_sync(0xffffffffu, bits);
    highest = __reduce_max_sync(0xffffffffu, highest);
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    if (lane == 0) {
        s_red[0][warp] = bits;
        s_red[1][warp] = highest;
        s_red[2][warp] = lowest;
    }
    if (tid == 0) z_n = z_members = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        bits = max(bits, s_red[0][w]);
        highest = max(highest, s_red[1][w]);
        lowest = min(lowest, s_red[2][w]);
    }
    const float big = __uint_as_float(bits);         // (a NaN's bits are above all)
    // roundings of one score: G - 1 in the group's sum, and the dot product's (2^-24 each, and their products)
    const float gamma = (a.G + dot_depth(a.c.D)) * 6.0e-8f * 1.01f;
    const float bound = 2.f * (gamma * norm * big) + 1e-36f;     // 2E; the last: products below fp32's range
    float lo = 0.f, hi = 0.f;
    const bool all = !(bound < 1e37f) || !(norm < 1e37f) || !(big < 1e37f) || !(norm * big < 1e37f);
    bool redo = all;
    int mid = 0, want = 0;               // pages between, and how many of them are in
    if (!all) {
        // the k-th largest: by a histogram over the scores' range and the members of its bin, or, where
        // too many share that, bit by bit
        const float least = key_value(lowest), width = key_value(highest) - least;
        const float to_bin = width > 0.f ? (kPickBins - 1) / width : 0.f;
        auto bin_of = [&](float x) { return min(kPickBins - 1, static_cast<int>((x - least) * to_bin)); };
        for (int i = tid; i < own; i += THREADS) atomicAdd(&s_bin[bin_of(key_value(key(i)))], 1);
        __syncthreads();
        int here = -1, above = 0;        // the bin that the k-th is in, the keys in higher ones
        {
            constexpr int PER = kPickBins / 32;
            int cnt[PER], mine = 0;      // lane 0 has the highest bins
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += cnt[i] = s_bin[kPickBins - 1 - (lane * PER + i)];
            int x = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const int at = __ffs(__ballot_sync(0xffffffffu, x >= k)) - 1;       // (the last lane has all: own > k)
            int run = x - mine;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (here < 0 && run + cnt[i] >= k) {
                    here = kPickBins - 1 - (lane * PER + i);
                    above = run;
                }
                run += cnt[i];
            }
            here = __shfl_sync(0xffffffffu, here, at);
            above = __shfl_sync(0xffffffffu, above, at);
        }
        uint32_t kth_key;
        if (s_bin[here] <= kPickClose) {
            const int members = s_bin[here];
            for (int i = tid; i < own; i += THREADS) {
                const uint32_t x = key(i);
                if (bin_of(key_value(x)) == here) z_key[atomicAdd(&z_members, 1)] = x;
            }
            __syncthreads();
            for (int y = tid; y < members; y += THREADS) {
                const uint32_t x = z_key[y];
                int more = 0, same = 0;
                for (int z = 0; z < members; ++z) {
                    more += z_key[z] > x;
                    same += z_key[z] == x;
                }
                if (above + more < k && k <= above + more + same) s_kth = x;      // (equal keys write the same)
            }
            __syncthreads();
            kth_key = s_kth;
        } else {
            const uint32_t low = key_of(least), differ = low ^ highest;       // (keys between two share their common top)
            const uint32_t top = differ ? 1u << (31 - __clz(differ)) : 0u;
            const uint32_t common = top ? low & ~(2 * top - 1) : low;
            kth_key = kth_largest<THREADS, uint32_t>(own, k, common, top, key, sum, s_red[0]);
        }
        const float kth = key_value(kth_key);
        const float pad = bound + fabsf(kth) * 3e-7f;            // (and the rounding of these two)
        lo = kth - pad;
        hi = kth + pad;
        int in = 0;
        for (int i = tid; i < own; i += THREADS) {
            const float x = key_value(key(i));
            in += x > hi;
            if (x >= lo && x <= hi) {
                ++mid;
                const int z = atomicAdd(&z_n, 1);
                if (z < kPickClose) z_at[z] = i;
            }
        }
        want = k - sum(in);
        mid = z_n;
        redo = mid != want;
    }
    // few pages between (the usual case): each scored by a warp in 64 bits and
    // ranked among them; its fp32 score then says in or out
    if (redo && !all && mid <= kPickClose) {
        for (int z = warp; z < mid; z += WARPS) {
            const double v = exact_score_alone<T>(a, it, z_at[z], lane);
            if (lane == 0) z_score[z] = v;
        }
        __syncthreads();
        for (int y = tid; y < mid; y += THREADS) {
            const double v = z_score[y];
            const int i = z_at[y];
            int rank = 0;
            for (int z = 0; z < mid; ++z) rank += z_score[z] > v || (z_score[z] == v && z_at[z] < i);
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
        query_sums<T, THREADS>(a, it, qs);
        __syncthreads();
        for (int i = warp; i < own; i += WARPS) {
            const float x = key_value(key(i));
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
        edge = kth_largest<THREADS, unsigned long long>(own, k, 0ull, 1ull << 63, fkey, sum, s_least);
        int above = 0;
        for (int i = tid; i < own; i += THREADS) above += fkey(i) > edge;
        ties = k - sum(above);
    }
    // list them in rising order, THREADS pages at a time
    int at = 0, tied = 0;
    for (int i0 = 0; i0 < own && at < k; i0 += THREADS) {
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
        int total;
        if (redo) {                      // the first `ties` of the equal ones
            const unsigned m = __ballot_sync(0xffffffffu, tie);
            const int before = tied + sum.before(__popc(m), &total) + __popc(m & ((1u << lane) - 1));
            in |= tie && before < ties;
            tied += total;
        }
        const unsigned m = __ballot_sync(0xffffffffu, in);
        const int before = at + sum.before(__popc(m), &total) + __popc(m & ((1u << lane) - 1));
        if (in && before < k) out[before] = i;
        at += total;
    }
}

// Rows that need no choice: every page up to their own, or their own alone.
template <int THREADS> __device__ __forceinline__ bool pick_plain(const SelArgs& a, const SelItem& it, int* out) {
    const int own = it.own, k = a.n_sel - 1;
    if (own <= k) {
        for (int i = threadIdx.x; i < a.n_sel; i += THREADS) out[i] = i <= own ? i : -1;
        return true;
    }
    // (own > k >= 0: k of the earlier pages, then its own)
    if (threadIdx.x == 0) out[k] = own;
    return k == 0;
}

// The second step: a block per item, on the scores that k_scores left.
template <typename T>
__global__ void __launch_bounds__(kPickThreads) k_pick(SelArgs a, int64_t items) {
    __shared__ uint32_t keys[kPickKeys];
    let_next_start();
    after_previous();
    const int64_t item = blockIdx.x;
    SelItem it;
    if (item >= items || !sel_item(a, item, &it)) return;
    int* out = a.sel + (static_cast<int64_t>(it.t) * a.c.Hkv + it.g) * a.n_sel;
    if (pick_plain<kPickThreads>(a, it, out)) return;
    float2* score = a.score + item * a.r.max_pages;
    const bool held = it.own <= kPickKeys;
    uint32_t bits = 0;                   // of the largest |mean|
    for (int i = threadIdx.x; i < it.own; i += kPickThreads) {
        const float2 x = score[i];
        if (held) keys[i] = key_of(x.x);
        bits = max(bits, __float_as_uint(x.y));
    }
    pick_pages<T, kPickThreads>(a, it, held, keys, score, bits, a.qnorm[item], out);
}

// Both steps in one, a block per item: the scores go to shared memory.  For
// many items or few pages; otherwise too few blocks would read the means.
template <typename T, int NCH>
__global__ void __launch_bounds__(kFusedThreads, NCH <= 4 ? 5 : 3) k_select(SelArgs a, int64_t items) {
    extern __shared__ uint32_t dyn_keys[];
    let_next_start();
    after_previous();
    const int64_t item = blockIdx.x;
    SelItem it;
    if (item >= items || !sel_item(a, item, &it)) return;
    int* out = a.sel + (static_cast<int64_t>(it.t) * a.c.Hkv + it.g) * a.n_sel;
    if (pick_plain<kFusedThreads>(a, it, out)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cq = lane & 3;
    const int* row = a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages;
    Query<T, NCH> q;
    uint32_t bits = 0;
    constexpr int STEP = kFusedThreads / 4, U = NCH <= 2 ? 4 : NCH == 4 ? 2 : 1;    // pages a block at once, times U
    int p = warp * 8 + (lane >> 2);
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = p + u * STEP < it.own ? __ldg(row + p + u * STEP) : -1;
    q.load(a, it, cq);
    for (int p0 = 0; p0 < it.own; p0 += U * STEP, p += U * STEP) {       // (the same steps for every lane: shuffles)
        Mean<NCH> m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u].load(a, it, id[u], p + u * STEP < it.own, cq);
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = p + (U + u) * STEP < it.own ? __ldg(row + p + (U + u) * STEP) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s;
            uint32_t big;
            m[u].score(q, s, big);
            bits = max(bits, big);
            if (cq == 0 && p + u * STEP < it.own) dyn_keys[p + u * STEP] = key_of(s);
        }
    }
    pick_pages<T, kFusedThreads>(a, it, true, dyn_keys, a.score + item * a.r.max_pages, bits, q.norm, out);
}

template <typename T> cudaError_t launch_scores(const SelArgs& a, int64_t blocks, cudaStream_t s) {
    const auto kernel = a.c.D <= 32 ? k_scores<T, 1> : a.c.D <= 64 ? k_scores<T, 2> : a.c.D <= 128 ? k_scores<T, 4> : k_scores<T, 8>;
    return launch_after(kernel, dim3(static_cast<unsigned>(blocks)), kScoreWarps * 32, 0, s, a);
}
template <typename T> cudaError_t launch_select(const SelArgs& a, int64_t items, bool score, bool fused, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(items));
    if (fused) {
        const auto kernel = a.c.D <= 32 ? k_select<T, 1> : a.c.D <= 64 ? k_select<T, 2> : a.c.D <= 128 ? k_select<T, 4> : k_select<T, 8>;
        const int smem = std::min(a.r.max_pages, kPickKeys) * static_cast<int>(sizeof(uint32_t));
        return launch_after(kernel, grid, kFusedThreads, smem, s, a, items);
    }
    if (score) {
        const cudaError_t e = launch_scores<T>(a, items * a.chunks, s);
        if (e != cudaSuccess) return e;
    }
    return launch_after(k_pick<T>, grid, kPickThreads, 0, s, a, items);
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
    // One launch where the items alone give every SM a block or two, or a
    // block's pages are few; the two steps otherwise (one request's 8 heads
    // over thousands of pages).
    cudaError_t e = cudaSuccess;
    for (int64_t t0 = 0; t0 < T && e == cudaSuccess; t0 += tokens) {
        a.t0 = (int)t0;
        const int64_t items = std::min(tokens, T - t0) * a.c.Hkv;
        const bool fused = max_pages <= kPickKeys && (items >= 2 * num_sms() || max_pages <= 512);
        ProfScope ps(GTATTN_KCAT_CACHE, score && !fused ? 2 : 1, stream);
        e = dtype == GTATTN_F32 ? launch_select<float>(a, items, score, fused, stream)
                                : launch_select<__nv_bfloat16>(a, items, score, fused, stream);
    }
    pool_free(ws, stream);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}
