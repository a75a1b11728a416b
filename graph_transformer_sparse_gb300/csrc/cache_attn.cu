// cache_attn.cu -- attention of new tokens over the 8-bit cache: all pages up
// to the token's position, or the pages selected for it.
#include <algorithm>

#include "cache_attn.cuh"

namespace gt {
namespace {

constexpr int kGenWarps = 4;
constexpr int kGenVpl = kCacheMaxD / 32;

// Any head width: a block per (token, query head) and share of its pages, its
// warps over those, lanes over the features; one pass with the running maximum
// and sum.  Few items over many pages are cut into shares whose sums
// k_cache_generic_join adds up in order (one request of 262150 tokens, 16
// heads: with a block per head 85 ms).
struct GenericShare {
    float* acc;      // [items][shares][D]
    float2* ml;      // [items][shares]
    int shares;
};

template <typename TI, typename TO>
__global__ void __launch_bounds__(kGenWarps * 32) k_cache_attn_generic(CacheAttn a, int64_t n_items, GenericShare sh) {
    __shared__ float sm_acc[kGenWarps][kCacheMaxD];
    __shared__ float sm_m[kGenWarps], sm_l[kGenWarps];
    let_next_start();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CacheView& c = a.c;
    const int end = a.r.tok_off[a.r.S];
    const int D = c.D;
    for (int64_t w = blockIdx.x; w < n_items * sh.shares; w += gridDim.x) {
        const int64_t it = w / sh.shares;
        const int share = static_cast<int>(w % sh.shares);
        const int t = (int)(it / a.H), h = (int)(it % a.H), g = h / a.G;
        if (t >= end) return;
        const int s = request_of(a.r.tok_off, a.r.S, t);
        const int pos = position_of(a.r, c.page, s, t);
        float q[kGenVpl], acc[kGenVpl];
#pragma unroll
        for (int k = 0; k < kGenVpl; ++k) {
            const int d = lane + 32 * k;
            q[k] = d < D ? load_elem(static_cast<const TI*>(a.Q), it * D + d) : 0.f;
            acc[k] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        const int n_pages = pos < 0 ? 0 : a.sel ? a.n_sel : (pos >> c.lp) + 1;
        for (int i = share * kGenWarps + warp; i < n_pages; i += kGenWarps * sh.shares) {
            const int p = a.sel ? a.sel[((int64_t)t * c.Hkv + g) * a.n_sel + i] : i;
            if (p < 0 || p > (pos >> c.lp)) continue;
            const int pid = a.r.table[(int64_t)s * a.r.max_pages + p];
            if ((unsigned)pid >= (unsigned)c.pages) continue;
            const int64_t ph = (int64_t)pid * c.Hkv + g;
            const float ks = c.kscale[ph] * a.qscale, vs = c.vscale[ph];
            const uint8_t* kt = c.k8 + ph * c.page * D;
            const uint8_t* vt = c.v8 + ph * c.page * D;
            const int n = min(c.page, pos - p * c.page + 1);
            for (int j = 0; j < n; ++j) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < kGenVpl; ++k) {
                    const int d = lane + 32 * k;
                    if (d < D) x += q[k] * e4m3_f32(kt[j * D + d]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                x *= ks;
                const float mn = fmaxf(m, x);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float w2 = ex2(x - mu), cr = ex2(m - mu);
                l = l * cr + w2;
                m = mn;
#pragma unroll
                for (int k = 0; k < kGenVpl; ++k) {
                    const int d = lane + 32 * k;
                    if (d < D) acc[k] = acc[k] * cr + w2 * (vs * e4m3_f32(vt[j * D + d]));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kGenVpl; ++k) sm_acc[warp][lane + 32 * k] = acc[k];
        if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
        __syncthreads();
        float mm = -INFINITY;
#pragma unroll
        for (int x = 0; x < kGenWarps; ++x) mm = fmaxf(mm, sm_m[x]);
        const float top = mm;
        if (mm == -INFINITY) mm = 0.f;
        float total = 0.f;
#pragma unroll
        for (int x = 0; x < kGenWarps; ++x) total += sm_l[x] * ex2(sm_m[x] - mm);
        for (int d = threadIdx.x; d < D; d += kGenWarps * 32) {
            float o = 0.f;
#pragma unroll
            for (int x = 0; x < kGenWarps; ++x) o += sm_acc[x][d] * ex2(sm_m[x] - mm);
            if (sh.shares > 1) sh.acc[w * D + d] = o;
            else store_elem(static_cast<TO*>(a.out), it * D + d, total == 0.f ? 0.f : o / total);
        }
        if (sh.shares > 1 && threadIdx.x == 0) sh.ml[w] = make_float2(top, total);
        __syncthreads();
    }
}

template <typename TO> __global__ void __launch_bounds__(kCacheMaxD) k_cache_generic_join(CacheAttn a, int64_t n_items, GenericShare sh) {
    let_next_start();
    after_previous();
    const int end = a.r.tok_off[a.r.S], D = a.c.D, d = threadIdx.x;
    for (int64_t it = blockIdx.x; it < n_items; it += gridDim.x) {
        if (it / a.H >= end) return;
        float top = -INFINITY;
        for (int i = 0; i < sh.shares; ++i) top = fmaxf(top, sh.ml[it * sh.shares + i].x);
        if (top == -INFINITY) top = 0.f;
        float o = 0.f, total = 0.f;
#pragma unroll 4
        for (int i = 0; i < sh.shares; ++i) {
            const float2 ml = sh.ml[it * sh.shares + i];
            const float f = ex2(ml.x - top);
            total = fmaf(f, ml.y, total);
            if (d < D) o = fmaf(f, sh.acc[(it * sh.shares + i) * D + d], o);
        }
        if (d < D) store_elem(static_cast<TO*>(a.out), it * D + d, total == 0.f ? 0.f : o / total);
    }
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" gtattn_status gtattn_fwd_cache(const gtattn_cache* cache, const void* Q, const int32_t* table,
                                          const int32_t* length, const int32_t* tok_off, const int32_t* sel, void* out,
                                          int64_t S, int64_t T, int64_t max_pages, int H, int n_sel, float scale,
                                          gtattn_dtype dtype, cudaStream_t stream) {
    CacheAttn a{};
    GT_TRY(check_cache(cache, 1, &a.c));
    GT_TRY(check_cache_rows(table, length, tok_off, S, T, max_pages, a.c.page, &a.r));
    if (dtype != GTATTN_F32 && dtype != GTATTN_BF16 && dtype != GTATTN_BF16_OUT_F32) return GTATTN_ERR_INVALID_ARG;
    if (H < 1 || H > kCacheMaxHeads || H % a.c.Hkv) return GTATTN_ERR_INVALID_ARG;
    if (sel ? (n_sel < 1 || n_sel > (1 << 20)) : n_sel != 0) return GTATTN_ERR_INVALID_ARG;
    if (T > 0 && (!Q || !out)) return GTATTN_ERR_INVALID_ARG;
    const uintptr_t esz = dtype == GTATTN_F32 ? 4 : 2, osz = dtype == GTATTN_BF16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(Q) & (esz - 1)) || (reinterpret_cast<uintptr_t>(out) & (osz - 1)) ||
        (reinterpret_cast<uintptr_t>(sel) & 3u))
        return GTATTN_ERR_INVALID_ARG;
    if (T * H >= (1ll << 31)) return GTATTN_ERR_UNSUPPORTED;
    if (T == 0 || S == 0) return GTATTN_OK;
    a.Q = Q;
    a.out = out;
    a.sel = sel;
    a.H = H;
    a.G = H / a.c.Hkv;
    a.n_sel = n_sel;
    a.qscale = scale * kLog2e;
    a.q_vec = (reinterpret_cast<uintptr_t>(Q) & 15u) == 0;
    a.o_vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    const int64_t rows = sel ? a.G : (T * a.G + S - 1) / S;
    if (a.c.pages > 0 && cache_tc_takes(a, dtype, rows)) return cache_tc(a, dtype, stream);
    if (a.c.pages > 0) switch (a.c.D) {
        case 32: return cache_tile_32(a, dtype, rows, stream);
        case 64: return cache_tile_64(a, dtype, rows, stream);
        case 128: return cache_tile_128(a, dtype, rows, stream);
        default:
            if (a.c.D % 16 == 0 && a.c.D < 64) return cache_tile_to_64(a, dtype, stream);
            if (a.c.D % 16 == 0 && a.c.D < 128) return cache_tile_to_128(a, dtype, stream);
            break;
    }
    const int64_t items = T * H;
    // shares: about eight blocks an SM, eight pages a block and share at least
    const int64_t most = (sel ? n_sel : max_pages) / (2 * kGenWarps);
    const int64_t want = std::min<int64_t>(most, 8 * num_sms() / items);
    GenericShare sh{nullptr, nullptr, (int)std::max<int64_t>(1, want)};
    void* ws = nullptr;
    if (sh.shares > 1) {
        const size_t n_acc = sizeof(float) * (size_t)items * sh.shares * a.c.D;
        GT_TRY(pool_alloc(&ws, n_acc + 8 + sizeof(float2) * (size_t)items * sh.shares, stream));
        sh.acc = static_cast<float*>(ws);
        sh.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + (n_acc + 7) / 8 * 8);
    }
    const int blocks = (int)std::min<int64_t>(items * sh.shares, num_sms() * 16);
    cudaError_t e;
    {
        ProfScope ps(GTATTN_KCAT_CACHE, sh.shares > 1 ? 2 : 1, stream);
        using B = __nv_bfloat16;
        const auto kernel = dtype == GTATTN_F32 ? k_cache_attn_generic<float, float>
                            : dtype == GTATTN_BF16 ? k_cache_attn_generic<B, B> : k_cache_attn_generic<B, float>;
        e = launch_after(kernel, dim3(blocks), kGenWarps * 32, 0, stream, a, items, sh);
        if (e == cudaSuccess && sh.shares > 1)
            e = launch_after(dtype == GTATTN_BF16 ? k_cache_generic_join<B> : k_cache_generic_join<float>,
                             dim3((unsigned)std::min<int64_t>(items, num_sms() * 8)), kCacheMaxD, 0, stream, a, items, sh);
    }
    pool_free(ws, stream);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}
