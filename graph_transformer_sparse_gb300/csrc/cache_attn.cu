// cache_attn.cu -- attention of new tokens over the 8-bit cache: all pages up
// to the token's position, or the pages selected for it.
#include "cache.cuh"

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

namespace gt {
namespace {

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

constexpr int kGenWarps = 4;
constexpr int kGenVpl = kCacheMaxD / 32;

// Any head width: a block per (token, query head), its warps over the pages,
// lanes over the features; one pass with the running maximum and sum.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kGenWarps * 32) k_cache_attn_generic(CacheAttn a, int64_t n_items) {
    __shared__ float sm_acc[kGenWarps][kCacheMaxD];
    __shared__ float sm_m[kGenWarps], sm_l[kGenWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CacheView& c = a.c;
    const int end = a.r.tok_off[a.r.S];
    const int D = c.D;
    for (int64_t it = blockIdx.x; it < n_items; it += gridDim.x) {
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
        for (int i = warp; i < n_pages; i += kGenWarps) {
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
                const float w = ex2(x - mu), cr = ex2(m - mu);
                l = l * cr + w;
                m = mn;
#pragma unroll
                for (int k = 0; k < kGenVpl; ++k) {
                    const int d = lane + 32 * k;
                    if (d < D) acc[k] = acc[k] * cr + w * (vs * e4m3_f32(vt[j * D + d]));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kGenVpl; ++k) sm_acc[warp][lane + 32 * k] = acc[k];
        if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
        __syncthreads();
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kGenWarps; ++w) mm = fmaxf(mm, sm_m[w]);
        if (mm == -INFINITY) mm = 0.f;
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kGenWarps; ++w) total += sm_l[w] * ex2(sm_m[w] - mm);
        for (int d = threadIdx.x; d < D; d += kGenWarps * 32) {
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kGenWarps; ++w) o += sm_acc[w][d] * ex2(sm_m[w] - mm);
            store_elem(static_cast<TO*>(a.out), it * D + d, total == 0.f ? 0.f : o / total);
        }
        __syncthreads();
    }
}


// N consecutive elements as fp32, by 16-byte loads where `vec` says they are aligned.
template <typename T, int N> __device__ __forceinline__ void load_part(const T* p, bool vec, float* x) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < N * static_cast<int>(sizeof(T)) / 16; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 4) {
                    x[4 * i + k] = __uint_as_float(w[k]);
                } else {
                    x[8 * i + 2 * k] = bf16lo(w[k]);
                    x[8 * i + 2 * k + 1] = bf16hi(w[k]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = load_elem(p, i);
    }
}

// out[at .. at + 3] = acc / sum (zeros for sum 0)
template <typename TO>
__device__ __forceinline__ void store_out(TO* out, int64_t at, float4 acc, float sum, bool vec) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    if (vec) {
        if constexpr (sizeof(TO) == 4)
            *reinterpret_cast<float4*>(out + at) = acc;
        else
            *reinterpret_cast<uint2*>(out + at) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    } else {
        store_elem(out, at, acc.x);
        store_elem(out, at + 1, acc.y);
        store_elem(out, at + 2, acc.z);
        store_elem(out, at + 3, acc.w);
    }
}

// A step's values hold a NaN at a key that some row does not see: a weight of
// 0 would carry it there.  The rows that see it get their NaN here, and the
// code becomes 0.  (V's tile in shared memory; the warp's own.)
template <int D, int MT>
__device__ void hide_nan(uint8_t* vt, const int (&rpos)[MT][2], int key0, int r, int cq, float (&o)[MT][D / 8][4]) {
    constexpr int ROW = D + 16;
    const int lane = r * 4 + cq;
    bool any = false;
    for (int i = 0; i < D / 4; ++i) {            // lane's row: one key
        const uint32_t w = *reinterpret_cast<const uint32_t*>(vt + lane * ROW + i * 4);
        any |= ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0);
    }
    if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                for (int key = 0; key < 32; ++key)
                    if ((vt[key * ROW + (2 * cq + (i & 1)) * (D / 8) + j] & 0x7f) == 0x7f &&
                        key0 + key <= rpos[mt][i >> 1])
                        o[mt][j][i] = NAN;
    __syncwarp();
    for (int i = 0; i < D; ++i)
        if ((vt[lane * ROW + i] & 0x7f) == 0x7f) vt[lane * ROW + i] = 0;
    __syncwarp();
}

// Blocks of a kernel that fit an SM at once, its dynamic shared memory
// allowed first (0: error); asked once per kernel and device.
int blocks_per_sm(const void* kernel, int threads, int smem) {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, int> known;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> g(mu);
    auto at = known.find({kernel, dev});
    if (at != known.end()) return at->second;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess)
        return 0;
    known[{kernel, dev}] = n;
    return n;
}

// ---------------------------------------------------------------------------
// tensor-core kernel (D = 32, 64, 128)
// ---------------------------------------------------------------------------
// e4m3 values are exact in fp16, so the codes are converted (one instruction
// for two) and multiplied with mma.m16n8k16 on fp16, accumulating in fp32;
// the power-of-two scales stay outside: kscale multiplies the logits, vscale
// goes into the exponent of the weights.  Rows of a tile are (token, head)
// pairs of one K/V head, 16 or 32 of them.
//
// A block's four warps take the tile's keys 32 at a time in turn, each with a
// ring of shared-memory stages of its own filled by cp.async (no block-wide
// barrier inside the walk), its own running maximum, sum and output; they are
// joined through shared memory at the item's end.
//
// Fragments are read from shared memory without a transposition.  The feature
// order inside a dot product is free, so lane (r, c) = (lane / 4, lane % 4)
// takes features c*D/4 .. (c+1)*D/4 of key r, contiguous bytes, and Q is laid
// out to match; V's output columns are free likewise, so lane (r, c) takes
// features r*D/8 .. (r+1)*D/8 of its four keys.  Rows are padded by 16 bytes.
//
// Work is cut by keys: the items (request, K/V head, row tile; with a
// selection token, K/V head, head tile) are laid end to end in units of 128
// keys and each block takes an equal share, so a long request spreads over
// all blocks and short ones share them.  A share that ends inside an item
// leaves its part in the workspace; k_cache_join adds up the parts of each
// such item in order.
constexpr int kTileWarps = 4;
constexpr int kStep = 32;                       // keys per warp step
constexpr int kUnit = kStep * kTileWarps;       // keys per block and unit
constexpr float kPBase = 10.f;                  // weights are 2^(a - M + 10), a <= M + 5 before M moves
constexpr float kPSlack = 5.f;

// What a block leaves behind for the item it ends inside of (parts 0: none).
struct JoinDesc {
    int parts;      // blocks that hold a part of the item, this one first
    int row0;       // first row's token
    int head0;      // its first query head
    int q0, rows;   // (rows: valid rows; row q0 + i is token row0 + (q0 + i) / G ...)
};

struct TileWork {
    float* part_o;       // [2 * blocks][R][D]
    float2* part_ml;     // [2 * blocks][R]
    JoinDesc* join;      // [blocks]
};

template <int D> constexpr int tile_stages() { return D == 128 ? 3 : D == 64 ? 4 : 6; }
template <int D> constexpr int tile_row() { return D + 16; }
template <int D> constexpr int tile_smem() { return kTileWarps * tile_stages<D>() * 2 * kStep * tile_row<D>(); }

__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
// the part of (lo, hi) that pack_f16x2 leaves out, as fp16
__device__ __forceinline__ uint32_t rest_f16x2(float lo, float hi, uint32_t packed) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&packed));
    return pack_f16x2(lo - f.x, hi - f.y);
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory, or 16 zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int N> __device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint8_t* p) {
    if constexpr (N == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else if constexpr (N == 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else if constexpr (N == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// One item (or a block's part of it).
struct Item {
    int s, g;            // request, K/V head
    int t0;              // token row of the request's (selection: the item's) first row
    int q0, rows;        // first (token, head) row of the tile within the request, valid rows
    int n_keys;          // keys listed for the tile (selection: n_sel * page)
    int pos0;            // position of the token t0
    const int* sel;      // its selected pages, or null
};

// Requests' shares of the work, in units: u(s) units for each of
// Hkv * tiles(s) items.
struct Share {
    int n, len, tiles, units;
};
__device__ __forceinline__ Share share_of(const CacheAttn& a, int s, int R) {
    Share h;
    const int t0 = __ldg(a.r.tok_off + s);
    h.n = __ldg(a.r.tok_off + s + 1) - t0;
    const long long cap = static_cast<long long>(a.r.max_pages) * a.c.page;
    h.len = static_cast<int>(min(static_cast<long long>(max(__ldg(a.r.length + s), 0)), cap));
    h.tiles = h.n > 0 ? static_cast<int>((static_cast<long long>(h.n) * a.G + R - 1) / R) : 0;
    h.units = max(1, (h.len + kUnit - 1) / kUnit);
    return h;
}

// Per-lane facts on a warp's coming 32 steps (lane i: step i of the batch).
struct Ahead {
    int pid[2];        // page of each 16-key half
    int cnt;           // valid keys of the halves, 8 bits each
    float ks[2], vs[2];
};

template <typename TI, typename TO, int D, int MT, bool SPLITQ, bool SPLITP>
__global__ void __launch_bounds__(kTileWarps * 32, 2) k_cache_attn_tile(CacheAttn a, TileWork wk) {
    constexpr int R = 16 * MT, NST = tile_stages<D>(), ROW = tile_row<D>(), STAGE = 2 * kStep * ROW;
    constexpr int KW = D / 16;      // words of a lane's key part: D/4 bytes
    constexpr int VW = D / 32;      // words of a lane's value part: D/8 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm_m[kTileWarps][R], sm_l[kTileWarps][R];
    __shared__ long long sm_scan[kTileWarps];
    __shared__ long long sm_at;     // units before request sm_s
    __shared__ int sm_s;
    const unsigned full = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, cq = lane & 3;
    const CacheView& c = a.c;
    const int S = a.r.S, Hkv = c.Hkv, page = c.page;
    uint8_t* ring = smem + warp * NST * STAGE;
    const uint32_t ring_u = smem_u32(ring);

    // ---- this block's share [u0, u1) of all units -------------------------
    long long total;
    const int ht = a.sel ? (a.G + R - 1) / R : 0;      // head tiles (selection)
    const int usel = a.sel ? static_cast<int>((static_cast<long long>(a.n_sel) * page + kUnit - 1) / kUnit) : 0;
    const int per = (S + kTileWarps * 32 - 1) / (kTileWarps * 32);
    long long before = 0;
    if (a.sel) {
        total = static_cast<long long>(__ldg(a.r.tok_off + S)) * Hkv * ht * usel;
    } else {
        long long mine = 0;
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s >= S) break;
            const Share h = share_of(a, s, R);
            mine += static_cast<long long>(Hkv) * h.tiles * h.units;
        }
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(full, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sm_scan[warp] = x;
        __syncthreads();
        total = 0;
        before = x - mine;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) {
            if (w < warp) before += sm_scan[w];
            total += sm_scan[w];
        }
    }
    const long long blocks = min(static_cast<long long>(gridDim.x), total);
    if (tid == 0) wk.join[blockIdx.x].parts = 0;
    if (blockIdx.x >= blocks) return;
    const long long u0 = total * blockIdx.x / blocks, u1 = total * (blockIdx.x + 1) / blocks;
    int cur_s = 0;
    long long cur_at = 0;           // units before request cur_s
    if (!a.sel) {
        long long at = before;      // the thread whose requests hold u0 finds it
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s >= S) break;
            const Share h = share_of(a, s, R);
            const long long w = static_cast<long long>(Hkv) * h.tiles * h.units;
            if (at <= u0 && u0 < at + w) {
                sm_s = s;
                sm_at = at;
            }
            at += w;
            if (at > u0) break;
        }
        __syncthreads();
        cur_s = sm_s;
        cur_at = sm_at;
    }

    for (long long u = u0; u < u1;) {
        // ---- the item that unit u falls into ------------------------------
        Item it;
        int units;
        long long base;             // its first unit
        if (a.sel) {
            units = usel;
            const long long k = u / usel;
            base = k * usel;
            const int hti = static_cast<int>(k % ht);
            const long long tg = k / ht;
            it.g = static_cast<int>(tg % Hkv);
            it.t0 = static_cast<int>(tg / Hkv);
            it.s = request_of(a.r.tok_off, S, it.t0);
            it.pos0 = position_of(a.r, page, it.s, it.t0);
            it.q0 = hti * R;
            it.rows = min(R, a.G - it.q0);
            it.n_keys = it.pos0 < 0 ? 0 : a.n_sel * page;
            it.sel = a.sel + tg * a.n_sel;
        } else {
            Share h = share_of(a, cur_s, R);
            while (cur_at + static_cast<long long>(Hkv) * h.tiles * h.units <= u) {
                cur_at += static_cast<long long>(Hkv) * h.tiles * h.units;
                ++cur_s;
                h = share_of(a, cur_s, R);
            }
            units = h.units;
            const long long k = (u - cur_at) / units;
            base = cur_at + k * units;
            it.g = static_cast<int>(k / h.tiles);
            const int tile = static_cast<int>(k % h.tiles);
            it.s = cur_s;
            it.t0 = __ldg(a.r.tok_off + cur_s);
            it.q0 = tile * R;
            it.rows = min(R, h.n * a.G - it.q0);
            // position of the tile's last token, as position_of caps it
            const long long p0 = static_cast<long long>(__ldg(a.r.length + cur_s)) - h.n;
            const long long cap = static_cast<long long>(a.r.max_pages) * page - 1;
            it.pos0 = static_cast<int>(max(p0, -(1ll << 31)));
            it.n_keys = static_cast<int>(max(min(p0 + (it.q0 + it.rows - 1) / a.G, cap), -1ll)) + 1;
            it.sel = nullptr;
        }
        const int j0 = static_cast<int>(u - base);
        const int j1 = static_cast<int>(min(static_cast<long long>(units), j0 + (u1 - u)));
        const bool whole = j0 == 0 && j1 == units;
        const int capk = a.r.max_pages * page - 1;

        // ---- the rows' queries, as fp16 relative to a power of two per row --
        uint32_t qh[MT][KW][4];
        uint32_t ql[SPLITQ ? MT : 1][SPLITQ ? KW : 1][4];
        float cqs[MT][2];           // the power times scale * log2(e)
        int rpos[MT][2];            // the rows' positions
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = mt * 16 + half * 8 + r;
                const bool valid = row < it.rows;
                const int q = it.q0 + (valid ? row : 0);
                const int tok = a.sel ? 0 : q / a.G, hd = it.g * a.G + (a.sel ? q : q % a.G);
                const int64_t src = (static_cast<int64_t>(it.t0 + tok) * a.H + hd) * D + cq * (D / 4);
                const TI* Qp = static_cast<const TI*>(a.Q) + src;
                float x[D / 4];
                load_part<TI, D / 4>(Qp, a.q_vec != 0, x);
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < D / 4; ++i) {
                    if (!valid) x[i] = 0.f;
                    const float v = fabsf(x[i]);
                    if (v < INFINITY) amax = fmaxf(amax, v);
                }
                amax = fmaxf(amax, __shfl_xor_sync(full, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(full, amax, 2));
                // 2^e with amax / 2^e in [2^14, 2^15); at least 2^-112 so that its inverse is finite
                const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 14, 15);
                const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                cqs[mt][half] = __uint_as_float(static_cast<uint32_t>(e) << 23) * a.qscale;
                const long long p = static_cast<long long>(it.pos0) + tok;
                rpos[mt][half] = valid ? static_cast<int>(max(min(p, static_cast<long long>(capk)), -1ll)) : 0x7fffffff;
#pragma unroll
                for (int ks = 0; ks < KW; ++ks) {
                    const float x0 = x[4 * ks] * up, x1 = x[4 * ks + 1] * up, x2 = x[4 * ks + 2] * up, x3 = x[4 * ks + 3] * up;
                    qh[mt][ks][half] = pack_f16x2(x0, x1);
                    qh[mt][ks][half + 2] = pack_f16x2(x2, x3);
                    if constexpr (SPLITQ) {
                        ql[mt][ks][half] = rest_f16x2(x0, x1, qh[mt][ks][half]);
                        ql[mt][ks][half + 2] = rest_f16x2(x2, x3, qh[mt][ks][half + 2]);
                    }
                }
            }
        }
        int min_pos = 0x7fffffff;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) min_pos = min(min_pos, min(rpos[mt][0], rpos[mt][1]));
        min_pos = __reduce_min_sync(full, min_pos);

        float o[MT][D / 8][4], M[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            M[mt][0] = M[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
        }

        // ---- walk this warp's steps: first + 4 k, k < n -------------------
        const int first = j0 * kTileWarps + warp;
        const int end_step = min(j1 * kTileWarps, (it.n_keys + kStep - 1) / kStep);
        const int n = end_step > first ? (end_step - first + kTileWarps - 1) / kTileWarps : 0;
        const int* trow = a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages;
        auto look = [&](int k) {     // lane's step k of this warp
            Ahead h;
            h.cnt = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                h.pid[q] = 0;
                h.ks[q] = h.vs[q] = 1.f;
                const int key = (first + k * kTileWarps) * kStep + 16 * q;
                if (k < n && key < it.n_keys) {
                    int lp = key >> c.lp, m;
                    if (it.sel) {
                        lp = __ldg(it.sel + lp);
                        // (keys behind the token's own position are not listed)
                        m = lp < 0 || lp > (it.pos0 >> c.lp) ? 0
                            : min(16, it.pos0 + 1 - (lp << c.lp) - (key & (page - 1)));
                    } else {
                        m = min(16, it.n_keys - key);
                    }
                    if (m > 0) {
                        const int pid = __ldg(trow + lp);
                        if (static_cast<unsigned>(pid) < static_cast<unsigned>(c.pages)) {
                            const int64_t ph = static_cast<int64_t>(pid) * Hkv + it.g;
                            h.pid[q] = pid;
                            h.ks[q] = __ldg(c.kscale + ph);
                            h.vs[q] = __ldg(c.vscale + ph);
                            h.cnt |= m << (8 * q);
                        }
                    }
                }
            }
            return h;
        };
        auto issue = [&](const Ahead& h, int k) {    // step k's copies (k < n), into its stage
            const uint32_t dst = ring_u + (k % NST) * STAGE;
            const int cnt = __shfl_sync(full, h.cnt, k & 31);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int pid = __shfl_sync(full, h.pid[q], k & 31);
                const int m = (cnt >> (8 * q)) & 0xff;
                const int off = ((first + k * kTileWarps) * kStep + 16 * q) & (page - 1);
                const int64_t src = (((static_cast<int64_t>(pid) * Hkv + it.g) << c.lp) + off) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int ch = i * 32 + lane, row = ch / (D / 16), col = ch % (D / 16);
                    const bool ok = row < m;
                    const int64_t at = src + (ok ? ch * 16 : 0);
                    copy16(dst + (16 * q + row) * ROW + col * 16, c.k8 + at, ok);
                    copy16(dst + (kStep + 16 * q + row) * ROW + col * 16, c.v8 + at, ok);
                }
            }
        };
        Ahead now = look(lane), next;
        if (n > 32) next = look(32 + lane);
#pragma unroll
        for (int k = 0; k < NST - 1; ++k) {
            if (k < n) issue(now, k);
            copy_commit();
        }
        for (int k = 0; k < n; ++k) {
            if (k > 0 && (k & 31) == 0) {
                now = next;
                if (k + 32 < n) next = look(k + 32 + lane);
            }
            if (k + NST - 1 < n) {
                const int kk = k + NST - 1;
                issue((kk >> 5) != (k >> 5) ? next : now, kk);
            }
            copy_commit();
            copy_wait<NST - 1>();
            __syncwarp();
            const uint8_t* kt = ring + (k % NST) * STAGE;
            uint8_t* vt = ring + (k % NST) * STAGE + kStep * ROW;
            const int cnt = __shfl_sync(full, now.cnt, k & 31);
            const int key0 = (first + k * kTileWarps) * kStep;

            // logits
            float x[MT][4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) x[mt][nt][0] = x[mt][nt][1] = x[mt][nt][2] = x[mt][nt][3] = 0.f;
                uint32_t w[KW];
                lds_words<KW>(w, kt + (nt * 8 + r) * ROW + cq * (D / 4));
#pragma unroll
                for (int ks = 0; ks < KW; ++ks) {
                    uint32_t b0, b1;
                    e4m3x4_f16(w[ks], b0, b1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_f16(x[mt][nt], qh[mt][ks], b0, b1);
                        if constexpr (SPLITQ) mma_f16(x[mt][nt], ql[mt][ks], b0, b1);
                    }
                }
            }
            float ks2[2], lv[2], iv[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                ks2[q] = __shfl_sync(full, now.ks[q], k & 31);
                const float vs = __shfl_sync(full, now.vs[q], k & 31);
                lv[q] = static_cast<float>(static_cast<int>((__float_as_uint(vs) >> 23) & 0xff) - 127);
                iv[q] = __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
            }
            // a = logit + log2(vscale), -inf where the row does not see the key
            const bool diagonal = !it.sel && key0 + kStep - 1 > min_pos;
            if (cnt == 0x1010 && !diagonal) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[mt][nt][i] = fmaf(x[mt][nt][i], cqs[mt][i >> 1] * ks2[nt >> 1], lv[nt >> 1]);
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int col = (nt & 1) * 8 + 2 * cq + (i & 1);     // within the half
                            const bool see = col < ((cnt >> (8 * (nt >> 1))) & 0xff) &&
                                             (it.sel || key0 + (nt >> 1) * 16 + col <= rpos[mt][i >> 1]);
                            x[mt][nt][i] = see ? fmaf(x[mt][nt][i], cqs[mt][i >> 1] * ks2[nt >> 1], lv[nt >> 1]) : -INFINITY;
                        }
                if (diagonal) hide_nan<D, MT>(vt, rpos, key0, r, cq, o);
            }
            // the running maximum moves when a weight would pass 2^15
            bool move = false;
            float top[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float t = x[mt][0][2 * half];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) t = fmaxf(t, fmaxf(x[mt][nt][2 * half], x[mt][nt][2 * half + 1]));
                    top[mt][half] = t;
                    move |= t > M[mt][half] + kPSlack;
                }
            }
            if (__any_sync(full, move)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float t = top[mt][half];
                        t = fmaxf(t, __shfl_xor_sync(full, t, 1));
                        t = fmaxf(t, __shfl_xor_sync(full, t, 2));
                        t = fmaxf(t, M[mt][half]);
                        const float f = M[mt][half] == t ? 1.f : ex2(M[mt][half] - t);
                        M[mt][half] = t;
                        l[mt][half] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[mt][j][2 * half] *= f;
                            o[mt][j][2 * half + 1] *= f;
                        }
                    }
                }
            }
            // weights, their sums, and the products with V
            uint32_t ph[MT][2][4], pl[SPLITP ? MT : 1][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float m0 = (M[mt][0] == -INFINITY ? 0.f : M[mt][0]) - kPBase;
                const float m1 = (M[mt][1] == -INFINITY ? 0.f : M[mt][1]) - kPBase;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float (&p)[4] = x[mt][2 * q + b];
                        p[0] = ex2(p[0] - m0);
                        p[1] = ex2(p[1] - m0);
                        p[2] = ex2(p[2] - m1);
                        p[3] = ex2(p[3] - m1);
                        s0 += p[0] + p[1];
                        s1 += p[2] + p[3];
                        ph[mt][q][2 * b] = pack_f16x2(p[0], p[1]);
                        ph[mt][q][2 * b + 1] = pack_f16x2(p[2], p[3]);
                        if constexpr (SPLITP) {
                            pl[mt][q][2 * b] = rest_f16x2(p[0], p[1], ph[mt][q][2 * b]);
                            pl[mt][q][2 * b + 1] = rest_f16x2(p[2], p[3], ph[mt][q][2 * b + 1]);
                        }
                    }
                    l[mt][0] = fmaf(s0, iv[q], l[mt][0]);
                    l[mt][1] = fmaf(s1, iv[q], l[mt][1]);
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    lds_words<VW>(w[i], vt + (16 * q + 2 * cq + (i & 1) + (i >> 1) * 8) * ROW + r * (D / 8));
#pragma unroll
                for (int v = 0; v < VW; ++v) {
                    uint32_t b0[4], b1[4];
                    e4m3x4_f16(__byte_perm(w[0][v], w[1][v], 0x5140), b0[0], b0[1]);
                    e4m3x4_f16(__byte_perm(w[0][v], w[1][v], 0x7362), b0[2], b0[3]);
                    e4m3x4_f16(__byte_perm(w[2][v], w[3][v], 0x5140), b1[0], b1[1]);
                    e4m3x4_f16(__byte_perm(w[2][v], w[3][v], 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma_f16(o[mt][4 * v + i], ph[mt][q], b0[i], b1[i]);
                            if constexpr (SPLITP) mma_f16(o[mt][4 * v + i], pl[mt][q], b0[i], b1[i]);
                        }
                    }
                }
            }
            __syncwarp();    // (the stage is filled again in the next step)
        }
        copy_wait<0>();

        // ---- join the warps ------------------------------------------------
        float* os = reinterpret_cast<float*>(ring);      // [R][D] (R * D * 4 <= NST * STAGE)
        __syncwarp();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = mt * 16 + half * 8 + r;
                float t = l[mt][half];
                t += __shfl_xor_sync(full, t, 1);
                t += __shfl_xor_sync(full, t, 2);
                if (cq == 0) {
                    sm_m[warp][row] = M[mt][half];
                    sm_l[warp][row] = t;
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < D / 8; j += 4)
                        *reinterpret_cast<float4*>(os + row * D + (2 * cq + b) * (D / 8) + j) =
                            make_float4(o[mt][j][2 * half + b], o[mt][j + 1][2 * half + b], o[mt][j + 2][2 * half + b],
                                        o[mt][j + 3][2 * half + b]);
            }
        }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (j0 == 0 ? 1 : 0);
        for (int e = tid; e < it.rows * (D / 4); e += kTileWarps * 32) {
            const int row = e / (D / 4), d = (e % (D / 4)) * 4;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) m = fmaxf(m, sm_m[w][row]);
            const float mu = m == -INFINITY ? 0.f : m;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) {
                const float f = ex2(sm_m[w][row] - mu);
                const float4 x = *reinterpret_cast<const float4*>(smem + w * NST * STAGE + (row * D + d) * 4);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
                sum = fmaf(f, sm_l[w][row], sum);
            }
            if (whole) {
                const int q = it.q0 + row;
                const int tok = a.sel ? 0 : q / a.G, hd = it.g * a.G + (a.sel ? q : q % a.G);
                store_out<TO>(static_cast<TO*>(a.out), (static_cast<int64_t>(it.t0 + tok) * a.H + hd) * D + d, acc, sum,
                              a.o_vec != 0);
            } else {
                *reinterpret_cast<float4*>(wk.part_o + (static_cast<int64_t>(slot) * R + row) * D + d) = acc;
                if (d == 0) wk.part_ml[static_cast<int64_t>(slot) * R + row] = make_float2(m, sum);
            }
        }
        if (j0 == 0 && j1 < units && tid == 0) {
            const long long last = base + units;      // blocks up to the one that holds unit last - 1
            const long long cl = (last * blocks + total - 1) / total - 1;
            JoinDesc jd;
            jd.parts = static_cast<int>(cl) - static_cast<int>(blockIdx.x) + 1;
            jd.row0 = it.t0;
            jd.head0 = it.g * a.G;
            jd.q0 = it.q0;
            jd.rows = it.rows;
            wk.join[blockIdx.x] = jd;
        }
        __syncthreads();     // (the rings and sm_m are used again)
        u += j1 - j0;
    }
}

// Adds up the parts of the item that block blockIdx.x of the tile kernel ended
// inside of, row blockIdx.y: each warp takes every kJoinWarps-th part, lanes
// over the features; the warps' sums are added in warp order.  (A request
// alone is cut into as many parts as there are blocks for its head; with one
// warp a row this was 48 us for 76 parts, all of it latency.)
constexpr int kJoinWarps = 8;
template <typename TO, int D, int R>
__global__ void __launch_bounds__(kJoinWarps * 32) k_cache_join(CacheAttn a, TileWork wk) {
    __shared__ float s_acc[kJoinWarps][D], s_sum[kJoinWarps], s_top[kJoinWarps];
    const JoinDesc jd = wk.join[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    if (jd.parts == 0 || row >= jd.rows) return;
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * R + row; };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < jd.parts; i += kJoinWarps * 32) m = fmaxf(m, wk.part_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_top[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_top[w]);
    const float mu = m == -INFINITY ? 0.f : m;
    constexpr int V = D / 32;
    float acc[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
    for (int i = warp; i < jd.parts; i += kJoinWarps) {
        const float2 ml = wk.part_ml[slot(i)];
        const float* p = wk.part_o + slot(i) * D;
        const float f = ex2(ml.x - mu);
        sum = fmaf(f, ml.y, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(f, p[v * 32 + lane], acc[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp][v * 32 + lane] = acc[v];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float o = 0.f, total = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        o += s_acc[w][d];
        total += s_sum[w];
    }
    const int q = jd.q0 + row;
    const int tok = a.sel ? 0 : q / a.G, hd = jd.head0 + (a.sel ? q : q % a.G);
    store_elem(static_cast<TO*>(a.out), (static_cast<int64_t>(jd.row0 + tok) * a.H + hd) * D + d,
               total == 0.f ? 0.f : o / total);
}

// ---- host -------------------------------------------------------------------
template <typename TI, typename TO, int D, int MT, bool SPLITQ, bool SPLITP>
gtattn_status launch_tile(const CacheAttn& a, cudaStream_t s) {
    constexpr int R = 16 * MT, smem = tile_smem<D>();
    static_assert(R * D * 4 <= tile_stages<D>() * 2 * kStep * tile_row<D>(), "a warp's output fits its ring");
    auto kernel = k_cache_attn_tile<TI, TO, D, MT, SPLITQ, SPLITP>;
    const int per_sm = blocks_per_sm(reinterpret_cast<const void*>(kernel), kTileWarps * 32, smem);
    if (per_sm < 1) return GTATTN_ERR_CUDA;
    const int blocks = num_sms() * per_sm;
    // (an item of one unit is never cut)
    const int64_t keys = a.sel ? (int64_t)a.n_sel * a.c.page : (int64_t)a.r.max_pages * a.c.page;
    const bool cut = keys > kUnit;
    const unsigned rows = (unsigned)std::min<int64_t>(R, a.sel ? a.G : (int64_t)a.r.T * a.G);   // of a tile, at most
    TileWork wk{};
    const size_t n_o = cut ? sizeof(float) * 2 * blocks * R * D : 0, n_ml = cut ? sizeof(float2) * 2 * blocks * R : 0;
    void* ws = nullptr;
    GT_TRY(pool_alloc(&ws, n_o + n_ml + sizeof(JoinDesc) * blocks, s));
    wk.part_o = static_cast<float*>(ws);
    wk.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + n_o);
    wk.join = reinterpret_cast<JoinDesc*>(static_cast<char*>(ws) + n_o + n_ml);
    {
        ProfScope ps(GTATTN_KCAT_CACHE, cut ? 2 : 1, s);
        kernel<<<blocks, kTileWarps * 32, smem, s>>>(a, wk);
        if (cut) k_cache_join<TO, D, R><<<dim3(blocks, rows), kJoinWarps * 32, 0, s>>>(a, wk);
    }
    const cudaError_t e = cudaGetLastError();
    pool_free(ws, s);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}

template <int D> gtattn_status launch_tile_d(const CacheAttn& a, gtattn_dtype dtype, int mt, cudaStream_t s) {
    using B = __nv_bfloat16;
    if constexpr (D == 128) {      // (two tiles' registers do not fit)
        if (dtype == GTATTN_F32) return launch_tile<float, float, D, 1, true, true>(a, s);
        return dtype == GTATTN_BF16 ? launch_tile<B, B, D, 1, false, false>(a, s) : launch_tile<B, float, D, 1, false, true>(a, s);
    } else {
    if (dtype == GTATTN_F32) return launch_tile<float, float, D, 1, true, true>(a, s);
    if (dtype == GTATTN_BF16)
        return mt == 2 ? launch_tile<B, B, D, 2, false, false>(a, s) : launch_tile<B, B, D, 1, false, false>(a, s);
    return mt == 2 ? launch_tile<B, float, D, 2, false, true>(a, s) : launch_tile<B, float, D, 1, false, true>(a, s);
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
    // two row tiles a warp where requests bring more rows than one tile holds
    const int mt = !sel && T * a.G > 16 * S ? 2 : 1;
    if (a.c.pages > 0) switch (a.c.D) {
        case 32: return launch_tile_d<32>(a, dtype, mt, stream);
        case 64: return launch_tile_d<64>(a, dtype, mt, stream);
        case 128: return launch_tile_d<128>(a, dtype, mt, stream);
        default: break;
    }
    const int64_t items = T * H;
    const int blocks = (int)std::min<int64_t>(items, num_sms() * 16);
    ProfScope ps(GTATTN_KCAT_CACHE, 1, stream);
    if (dtype == GTATTN_F32)
        k_cache_attn_generic<float, float><<<blocks, kGenWarps * 32, 0, stream>>>(a, items);
    else if (dtype == GTATTN_BF16)
        k_cache_attn_generic<__nv_bfloat16, __nv_bfloat16><<<blocks, kGenWarps * 32, 0, stream>>>(a, items);
    else
        k_cache_attn_generic<__nv_bfloat16, float><<<blocks, kGenWarps * 32, 0, stream>>>(a, items);
    GT_CUDA(cudaGetLastError());
    return GTATTN_OK;
}
