// cache_tile.cuh -- attention over the 8-bit cache on the tensor cores, for one
// head width a source file (cache_tile32.cu and so on: they compile side by
// side).
#pragma once

#include <algorithm>
#include <mutex>

#include "cache_attn.cuh"

namespace gt {
namespace {

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
template <int D, int NT>
__device__ void hide_nan(uint8_t* vt, const int (&rpos)[NT][2], int key0, int r, int cq, float (&o)[D / 16][NT][4]) {
    constexpr int ROW = D + 16;
    const int lane = r * 4 + cq;
    bool any = false;
    for (int i = 0; i < D / 4; ++i) {            // lane's row: one key
        const uint32_t w = *reinterpret_cast<const uint32_t*>(vt + lane * ROW + i * 4);
        any |= ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0);
    }
    if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                for (int key = 0; key < 32; ++key)
                    if ((vt[key * ROW + r * (D / 8) + 2 * j + (i >> 1)] & 0x7f) == 0x7f && key0 + key <= rpos[nt][i & 1])
                        o[j][nt][i] = NAN;
    __syncwarp();
    for (int i = 0; i < D; ++i)
        if ((vt[lane * ROW + i] & 0x7f) == 0x7f) vt[lane * ROW + i] = 0;
    __syncwarp();
}

// Blocks of a kernel that fit an SM at once, its dynamic shared memory
// allowed first (0: error); asked once per kernel and device (and again where
// the table is full: nothing here allocates or throws).
int blocks_per_sm(const void* kernel, int threads, int smem) {
    struct Known {
        const void* kernel;
        int dev, n;
    };
    static std::mutex mu;
    static Known known[64];
    static int count = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> g(mu);
    for (int i = 0; i < count; ++i)
        if (known[i].kernel == kernel && known[i].dev == dev) return known[i].n;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess)
        return 0;
    if (count < 64) known[count++] = Known{kernel, dev, n};
    return n;
}

// ---------------------------------------------------------------------------
// tensor-core kernel (D = 32, 64, 128)
// ---------------------------------------------------------------------------
// e4m3 values are exact in fp16, so the codes are converted (one instruction
// for two) and multiplied with mma.m16n8k16 on fp16, accumulating in fp32;
// the power-of-two scales stay outside: kscale multiplies the logits, vscale
// goes into the exponent of the weights.  Rows of a tile are (token, head)
// pairs of one K/V head, 8 NT of them.
//
// Both products are formed transposed, keys (or features) along the 16 of the
// instruction and rows along its 8: logits^T = K Q^T, out^T = V^T weights^T.
// A token's few heads then fill the tile.  (With rows along the 16, half the
// registers and of the softmax's instructions went to rows that are not there:
// 206 registers at D = 128 against 157, so two warps a scheduler against
// three, whose waits could not be hidden: 121 us for the 64 requests below in
// this kernel, against 103.)  The weights, keys by rows as they come out, become the second
// product's operand by one 8 x 8 transposition each (movmatrix).
//
// A block's four warps take the tile's keys 32 at a time in turn, each with a
// ring of shared-memory stages of its own filled by cp.async (no block-wide
// barrier inside the walk), its own running maximum, sum and output; they are
// joined through shared memory at the item's end.
//
// Fragments are read from shared memory without a transposition.  The feature
// order inside a dot product is free, so lane (r, c) = (lane / 4, lane % 4)
// takes features c*D/4 .. (c+1)*D/4 of key r, contiguous bytes, and Q is laid
// out to match; out's features are free likewise, so lane (r, c) takes
// features r*D/8 .. (r+1)*D/8 of its four keys.  Rows are padded by 16 bytes:
// no bank conflicts.
//
// Work is cut by keys: an item (request, K/V head, row tile; with a selection
// token, K/V head, head tile) of more than lc units of 128 keys becomes tasks
// of lc units each, lc such that all items together make about kTasksPerBlock
// tasks for each resident block.  Blocks claim tasks from a counter: equal
// shares handed out beforehand left the SMs busy between 161 and 228 thousand
// cycles of 238 (they do not all get the same share of the memory).  Bound by
// memory: 64 requests of 500-8191 tokens, 32 heads over 8 of 128, 103 us in
// this kernel (5.5 TB/s of 6.8), 113 with the plan and the join; one request of
// 262150 tokens 57 and 69 us.  Where the cuts lie depends on the
// sizes alone, and k_cache_join adds up an item's parts in order, so results
// do not depend on who took what.
constexpr int kTileWarps = 4;
constexpr int kStep = 32;                       // keys per warp step
constexpr int kUnit = kStep * kTileWarps;       // keys per block and unit
constexpr float kPBase = 10.f;                  // weights are 2^(a - M + 10), a <= M + 5 before M moves
constexpr float kPSlack = 5.f;

constexpr int kTasksPerBlock = 4;

// One item.
struct Item {
    int s, g;            // request, K/V head
    int t0;              // token row of the request's (selection: the item's) first row
    int q0, rows;        // first (token, head) row of the tile within the request, valid rows
    int n_keys;          // keys listed for the tile (selection: n_sel * page)
    int pos0;            // position of the token t0
    int units;           // 128 keys each
};

// The cut.
struct TilePlan {
    int lc;              // units of a task
    unsigned tasks;
    unsigned multi;      // items of several tasks
    int most;            // the most tasks of one item
    unsigned next;       // tasks claimed beyond the blocks' own (two each, one in cache_tc.cu)
    int pad[3];
};
// A task, units [j0, j1) of an item, as the plan lists it.
struct alignas(16) Task {
    Item it;
    int j0, j1;
    int slot;            // where its part goes (below 0: it is the whole item)
    int parts;           // tasks of the item
    int pad[4];
};
constexpr int kTaskWords = sizeof(Task) / 4;
static_assert(kTaskWords == 16, "a half-warp reads a task");
struct TileWork {
    TilePlan* plan;      // null: as many blocks as items, of one unit each
    Task* list;          // every task
    Task* multi;         // the first task of every item of several
    int* pre;            // [3][S] tasks, partial results and items of several tasks before request s (S > kPlanHeld)
    float* part_o;       // [slots][R][D]
    float2* part_ml;     // [slots][R]
    int target;          // tasks aimed at
};

// resident blocks an SM the registers are cut for, and stages a warp's ring has
template <int D, int NT> constexpr int tile_blocks() { return D * NT <= 64 ? 4 : D * NT <= 128 ? 3 : 2; }
template <int D, int NT> constexpr int tile_stages() {      // (228 KB an SM; 3 KB a block for the rest)
    const int n = (228 * 1024 / tile_blocks<D, NT>() - 3 * 1024) / (kTileWarps * 2 * kStep * (D + 16));
    return n < 8 ? n : 8;
}
template <int D> constexpr int tile_row() { return D + 16; }
template <int D, int NT> constexpr int tile_smem() { return kTileWarps * tile_stages<D, NT>() * 2 * kStep * tile_row<D>(); }

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
// 8 x 8 transposition of 16-bit values, two a lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; or 16 zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool valid) {
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

// Requests' shares of the work, in units: u(s) units for each of
// Hkv * tiles(s) items.
struct Share {
    int n, len, tiles, units;
};
__device__ __forceinline__ Share share_of(const CacheAttn& a, int s, int R) {
    Share h;
    h.n = min(__ldg(a.r.tok_off + s + 1), a.r.T) - __ldg(a.r.tok_off + s);       // (rows past T do not exist)
    const long long cap = static_cast<long long>(a.r.max_pages) * a.c.page;
    h.len = static_cast<int>(min(static_cast<long long>(max(__ldg(a.r.length + s), 0)), cap));
    h.tiles = h.n > 0 ? static_cast<int>((static_cast<long long>(h.n) * a.G + R - 1) / R) : 0;
    h.units = max(1, (h.len + kUnit - 1) / kUnit);
    return h;
}

// Item k of request s (full attention), and item k of all (selection).
__device__ __forceinline__ Item item_full(const CacheAttn& a, int R, int s, unsigned k) {
    const Share h = share_of(a, s, R);
    Item it;
    it.s = s;
    it.g = static_cast<int>(k / h.tiles);       // tiles of one K/V head side by side: they read the same pages
    it.t0 = __ldg(a.r.tok_off + s);
    it.q0 = static_cast<int>(k % h.tiles) * R;
    it.rows = min(R, h.n * a.G - it.q0);
    const long long p0 = static_cast<long long>(__ldg(a.r.length + s)) - (__ldg(a.r.tok_off + s + 1) - it.t0);
    const long long cap = static_cast<long long>(a.r.max_pages) * a.c.page - 1;
    it.pos0 = static_cast<int>(max(p0, -(1ll << 31)));
    // up to the tile's last token, its position capped as position_of caps it
    it.n_keys = static_cast<int>(max(min(p0 + (it.q0 + it.rows - 1) / a.G, cap), -1ll)) + 1;
    it.units = h.units;
    return it;
}
__device__ __forceinline__ int sel_units(const CacheAttn& a) {
    return static_cast<int>((static_cast<long long>(a.n_sel) * a.c.page + kUnit - 1) / kUnit);
}
__device__ __forceinline__ Item item_sel(const CacheAttn& a, int R, unsigned k) {
    const unsigned ht = (a.G + R - 1) / R, tg = k / ht;
    Item it;
    it.g = static_cast<int>(tg % a.c.Hkv);
    it.t0 = static_cast<int>(tg / a.c.Hkv);
    it.s = request_of(a.r.tok_off, a.r.S, it.t0);
    it.pos0 = position_of(a.r, a.c.page, it.s, it.t0);
    it.q0 = static_cast<int>(k % ht) * R;
    it.rows = min(R, a.G - it.q0);
    it.n_keys = it.pos0 < 0 ? 0 : a.n_sel * a.c.page;
    it.units = sel_units(a);
    return it;
}

// Sum and exclusive prefix over a block.
constexpr int kPlanThreads = 256;
constexpr int kPlanHeld = 2048;     // requests whose prefixes fit shared memory
__device__ __forceinline__ long long plan_scan(long long v, long long* total) {
    __shared__ long long sums[kPlanThreads / 32];
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
    long long w = lane < static_cast<int>(blockDim.x >> 5) ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp > 0 ? before : 0) + x - v;
}

// Task `part` of an item's nch; slot: that of the item's first part.
__device__ __forceinline__ Task part_of(const Item& it, unsigned slot, int lc, int nch, unsigned part) {
    Task t{};
    t.it = it;
    t.j0 = static_cast<int>(part) * lc;
    t.j1 = static_cast<int>(min(static_cast<long long>(it.units), static_cast<long long>(t.j0) + lc));
    t.slot = nch > 1 ? static_cast<int>(slot + part) : -1;
    t.parts = nch;
    return t;
}

// The plan: how long a task is, and the list of them.  Every block adds up
// the requests' sizes by itself and then lists its share of the tasks (one
// block for all took 14 us for 2700 tasks, most of it the list).
__global__ void __launch_bounds__(kPlanThreads) k_cache_plan(CacheAttn a, TileWork wk, int R) {
    __shared__ int held[3 * kPlanHeld];
    __shared__ int s_most[kPlanThreads / 32];
    let_next_start();
    after_previous();
    const int S = a.r.S, tid = threadIdx.x;
    const long long x0 = static_cast<long long>(blockIdx.x) * kPlanThreads + tid;
    const long long dx = static_cast<long long>(gridDim.x) * kPlanThreads;
    const bool lead = blockIdx.x == 0 && tid == 0;
    if (a.sel) {
        const int units = sel_units(a);
        const long long items = static_cast<long long>(min(__ldg(a.r.tok_off + S), a.r.T)) * a.c.Hkv * ((a.G + R - 1) / R);
        const int lc = static_cast<int>(max((items * units + wk.target - 1) / wk.target, 1ll));
        const int nch = (units + lc - 1) / lc;
        if (lead) *wk.plan = TilePlan{lc, static_cast<unsigned>(items * nch), nch > 1 ? static_cast<unsigned>(items) : 0u, nch, 0u};
        for (long long x = x0; x < items * nch; x += dx) {
            const unsigned item = static_cast<unsigned>(x / nch), part = static_cast<unsigned>(x % nch);
            const Task t = part_of(item_sel(a, R, item), item * nch, lc, nch, part);
            wk.list[x] = t;
            if (nch > 1 && part == 0) wk.multi[item] = t;
        }
        return;
    }
    int* pre = S <= kPlanHeld ? held : wk.pre;     // (in global memory all blocks write the same)
    const int per = (S + kPlanThreads - 1) / kPlanThreads;
    const int s0 = static_cast<int>(min(static_cast<long long>(tid) * per, static_cast<long long>(S))), s1 = min(s0 + per, S);
    long long total = 0;
    int longest = 0;
    for (int s = s0; s < s1; ++s) {
        const Share h = share_of(a, s, R);
        total += static_cast<long long>(a.c.Hkv) * h.tiles * h.units;
        if (h.tiles) longest = max(longest, h.units);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((tid & 31) == 0) s_most[tid >> 5] = longest;
    long long all;
    plan_scan(total, &all);
    const int lc = static_cast<int>(max((all + wk.target - 1) / wk.target, 1ll));
    long long tasks = 0, slots = 0, multi = 0;
    for (int s = s0; s < s1; ++s) {
        const Share h = share_of(a, s, R);
        const long long items = static_cast<long long>(a.c.Hkv) * h.tiles, nch = (h.units + lc - 1) / lc;
        tasks += items * nch;
        if (nch > 1) {
            slots += items * nch;
            multi += items;
        }
    }
    long long all_t, all_s, all_m;
    tasks = plan_scan(tasks, &all_t);
    slots = plan_scan(slots, &all_s);
    multi = plan_scan(multi, &all_m);
    for (int s = s0; s < s1; ++s) {
        pre[s] = static_cast<int>(tasks);
        pre[S + s] = static_cast<int>(slots);
        pre[2 * S + s] = static_cast<int>(multi);
        const Share h = share_of(a, s, R);
        const long long items = static_cast<long long>(a.c.Hkv) * h.tiles, nch = (h.units + lc - 1) / lc;
        tasks += items * nch;
        if (nch > 1) {
            slots += items * nch;
            multi += items;
        }
    }
    __syncthreads();
    if (lead) {
        for (int w = 0; w < kPlanThreads / 32; ++w) longest = max(longest, s_most[w]);
        *wk.plan = TilePlan{lc, static_cast<unsigned>(all_t), static_cast<unsigned>(all_m), (longest + lc - 1) / lc, 0u};
    }
    for (long long x = x0; x < all_t; x += dx) {
        int lo = 0, hi = S;          // the last request whose tasks begin at or before x
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (static_cast<unsigned>(pre[m]) <= static_cast<unsigned>(x)) lo = m;
            else hi = m;
        }
        const unsigned in = static_cast<unsigned>(x) - static_cast<unsigned>(pre[lo]);
        const int nch = (share_of(a, lo, R).units + lc - 1) / lc;
        const unsigned item = in / nch, part = in % nch;
        const Task t = part_of(item_full(a, R, lo, item), static_cast<unsigned>(pre[S + lo]) + item * nch, lc, nch, part);
        wk.list[x] = t;
        if (nch > 1 && part == 0) wk.multi[static_cast<unsigned>(pre[2 * S + lo]) + item] = t;
    }
}

// The item that block b takes when there is no plan (at most one each, of one unit): the warp walks the requests.
__device__ __forceinline__ bool task_plain(const CacheAttn& a, int R, unsigned b, int lane, Task* t) {
    if (a.sel) {
        if (b >= static_cast<long long>(min(__ldg(a.r.tok_off + a.r.S), a.r.T)) * a.c.Hkv * ((a.G + R - 1) / R)) return false;
        t->it = item_sel(a, R, b);
    } else {
        long long before = 0;
        int s0 = 0;
        bool found = false;
        for (; s0 < a.r.S && !found; s0 += 32) {
            const long long items = s0 + lane < a.r.S ? static_cast<long long>(a.c.Hkv) * share_of(a, s0 + lane, R).tiles : 0;
            long long x = items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned m = __ballot_sync(0xffffffffu, before + x > b);
            if (m) {
                const int at = __ffs(m) - 1;
                const long long first = __shfl_sync(0xffffffffu, before + x - items, at);
                t->it = item_full(a, R, s0 + at, static_cast<unsigned>(b - first));
                found = true;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
        }
        if (!found) return false;
    }
    t->j0 = 0;
    t->j1 = t->it.units;
    t->slot = -1;
    t->parts = 1;
    return true;
}

// Per-lane facts on a warp's coming 32 steps (lane i: step i of the batch).
struct Ahead {
    int pid[2];        // page of each 16-key half
    int cnt;           // valid keys of the halves, 8 bits each
    float ks[2], vs[2];
};

// What a step's arithmetic needs beside the copies.
struct StepFacts {
    int cnt;             // as Ahead's
    float ks[2], vs[2];
};
// Where a warp's keys of a task are.
struct Reach {
    const int* row;      // the request's table
    const int* sel;
    int g, n_keys, pos0, first, n;
};
__device__ __forceinline__ int pt_first(const Task& t, int warp) { return t.j0 * kTileWarps + warp; }

// PAD: heads of c.D < D features, a multiple of 16: rows of them in memory, of
// D, zeros behind, in shared memory and registers.
template <typename TI, typename TO, int D, int NT, bool SPLITQ, bool SPLITP, bool PAD = false>
__global__ void __launch_bounds__(kTileWarps * 32, (tile_blocks<D, NT>())) k_cache_attn_tile(CacheAttn a, TileWork wk) {
    constexpr int R = 8 * NT, RJ = R < 16 ? R : 16, NST = tile_stages<D, NT>(), ROW = tile_row<D>(), STAGE = 2 * kStep * ROW;
    constexpr int OROW = D + 4;     // row stride of a warp's output in the join, in floats
    static_assert(RJ * OROW * 4 <= STAGE && NST >= 2, "RJ rows of a warp's output fit a stage");
    constexpr int KW = D / 16;      // words of a lane's key part: D/4 bytes
    constexpr int VW = D / 32;      // words of a lane's value part: D/8 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm_m[kTileWarps][RJ], sm_l[kTileWarps][RJ];
    __shared__ Task sm_task[3];     // tasks i, i + 1 and, being written, i + 2 of this block
    __shared__ int sm_more[3];
    __shared__ int sm_free[kTileWarps];
    __shared__ StepFacts sm_facts[kTileWarps][NST];
    const unsigned full = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, cq = lane & 3;
    const CacheView& c = a.c;
    const int Hkv = c.Hkv, page = c.page;
    const int width = PAD ? c.D : D;       // features of a head in memory
    uint8_t* ring = smem + warp * NST * STAGE;
    const uint32_t ring_u = smem_u32(ring);
    let_next_start();
    after_previous();

    const unsigned tasks = wk.plan ? wk.plan->tasks : 0;
    // Task i of this block (0 and 1: by its place in the grid, others claimed) goes to sm_task by way of warp 0's
    // registers: claimed when the block begins task i - 2, read a few steps later, put down at that task's end.
    // (Fetched in one go, the three dependent accesses held warp 0, and with it the block, up for 2 us a task.)
    auto claim = [&]() { return lane == 0 && wk.plan ? 2 * gridDim.x + atomicAdd(&wk.plan->next, 1u) : 0u; };
    auto task_word = [&](unsigned x) {       // lane i: word i of task x
        return lane < kTaskWords && x < tasks ? reinterpret_cast<const int*>(wk.list + x)[lane] : 0;
    };
    auto put = [&](int i, unsigned x, int word) {
        if (lane < kTaskWords) reinterpret_cast<int*>(&sm_task[i % 3])[lane] = word;
        if (lane == 0) sm_more[i % 3] = x < tasks;
    };
    if (warp == 0) {
        if (wk.plan) {
            const unsigned x1 = gridDim.x + blockIdx.x;
            const int w0 = task_word(blockIdx.x), w1 = task_word(x1);
            put(0, blockIdx.x, w0);
            put(1, x1, w1);
        } else {
            Task t{};
            const bool more = task_plain(a, R, blockIdx.x, lane, &t);
            if (lane == 0) {
                sm_task[0] = t;
                sm_more[0] = more;
                sm_more[1] = 0;
            }
        }
    }
    __syncthreads();

    // ---- the copies: the warp's steps of all its block's tasks, one stream --
    // A step of task i is 32 keys; this warp has the steps first + 4 k, k < n,
    // of it.  Copies run NST - 1 steps ahead of the arithmetic, also from a
    // task's last steps into the next task's first (whose place is known: it
    // was fetched while the block worked on the task before).
    const int dlane = (lane / (D / 16)) * ROW + (lane % (D / 16)) * 16;
    int issued = 0, done = 0;       // steps copied and used so far
    int pi = -1, pk = 0, pn = 0;    // the copies' task and step in it
    Reach pt{};                     // where that task's keys are
    Ahead cur{}, nxt{};             // facts on the steps pk / 32 * 32 + lane of it; on the first 32 of the next task
    int nxt_of = -1;
    auto reach = [&](int i) {
        const Task& t = sm_task[i % 3];
        Reach p;
        p.row = a.r.table + static_cast<int64_t>(t.it.s) * a.r.max_pages;
        p.sel = a.sel ? a.sel + (static_cast<int64_t>(t.it.t0) * Hkv + t.it.g) * a.n_sel : nullptr;
        p.g = t.it.g;
        p.n_keys = t.it.n_keys;
        p.pos0 = t.it.pos0;
        p.first = t.j0 * kTileWarps + warp;
        const int end = min(t.j1 * kTileWarps, (t.it.n_keys + kStep - 1) / kStep);
        p.n = end > p.first ? (end - p.first + kTileWarps - 1) / kTileWarps : 0;
        return p;
    };
    auto look = [&](const Reach& p, int k) {     // step k of the warp's steps
        Ahead h;
        h.cnt = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            h.pid[q] = 0;
            h.ks[q] = h.vs[q] = 1.f;
            const int key = (p.first + k * kTileWarps) * kStep + 16 * q;
            if (k < p.n && key < p.n_keys) {
                int lp = key >> c.lp, m;
                if (p.sel) {
                    lp = __ldg(p.sel + lp);
                    // (keys behind the token's own position are not listed)
                    m = lp < 0 || lp > (p.pos0 >> c.lp) ? 0 : min(16, p.pos0 + 1 - (lp << c.lp) - (key & (page - 1)));
                } else {
                    m = min(16, p.n_keys - key);
                }
                if (m > 0) {
                    const int pid = __ldg(p.row + lp);
                    if (static_cast<unsigned>(pid) < static_cast<unsigned>(c.pages)) {
                        const int64_t ph = static_cast<int64_t>(pid) * Hkv + p.g;
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
    // copies the next step, if it belongs to a task up to number `last`
    auto produce = [&](int last) {
        while (pk == pn) {
            if (pi >= last || !sm_more[(pi + 1) % 3]) return false;
            ++pi;
            pt = reach(pi);
            pn = pt.n;
            pk = 0;
            cur = nxt_of == pi ? nxt : look(pt, lane);
        }
        if (pk > 0 && (pk & 31) == 0) cur = look(pt, pk + lane);
        const int st = issued % NST, from = pk & 31;
        const uint32_t dst = ring_u + st * STAGE;
        const int cnt = __shfl_sync(full, cur.cnt, from);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int pid = __shfl_sync(full, cur.pid[q], from);
            const int m = (cnt >> (8 * q)) & 0xff;
            const int off = ((pt.first + pk * kTileWarps) * kStep + 16 * q) & (page - 1);
            const int64_t src = (((static_cast<int64_t>(pid) * Hkv + pt.g) << c.lp) + off) * width;
            // 16 rows of D bytes, contiguous: lane i's 16 bytes are in row i / (D / 16) and every 512 / D rows on
            const uint32_t to = dst + dlane + 16 * q * ROW;
            if (!PAD && m == 16) {
                const uint8_t* kp = c.k8 + src + lane * 16;
                const uint8_t* vp = c.v8 + src + lane * 16;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    copy16(to + i * (512 / D) * ROW, kp + i * 512);
                    copy16(to + i * (512 / D) * ROW + kStep * ROW, vp + i * 512);
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int row = lane / (D / 16) + i * (512 / D), col = lane % (D / 16) * 16;
                    const bool ok = row < m && (!PAD || col < width);
                    const int64_t at = src + (ok ? row * width + col : 0);
                    copy16_or_zero(to + i * (512 / D) * ROW, c.k8 + at, ok);
                    copy16_or_zero(to + i * (512 / D) * ROW + kStep * ROW, c.v8 + at, ok);
                }
            }
        }
        copy_commit();
        if (lane == from) sm_facts[warp][st] = StepFacts{cur.cnt, {cur.ks[0], cur.ks[1]}, {cur.vs[0], cur.vs[1]}};
        ++issued;
        ++pk;
        return true;
    };

    for (int i = 0; sm_more[i % 3]; ++i) {
        const Item it = sm_task[i % 3].it;
        const int out_slot = sm_task[i % 3].slot;
        const int n = reach(i).n;
        const int capk = a.r.max_pages * page - 1;
        while (issued - done < NST - 1 && produce(i + 1)) {}
        if (pi == i && sm_more[(i + 1) % 3]) {       // (used when the copies get there)
            nxt = look(reach(i + 1), lane);
            nxt_of = i + 1;
        }
        unsigned claimed = 0;
        int word = 0;
        if (warp == 0) claimed = claim();

        // ---- the rows' queries, as fp16 relative to a power of two per row --
        uint32_t qh[NT][KW][2];
        uint32_t ql[SPLITQ ? NT : 1][SPLITQ ? KW : 1][2];
        float cqs[NT][2];           // rows 8 nt + 2 cq + e: the power times scale * log2(e)
        int rpos[NT][2];            // and their positions
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool valid = nt * 8 + r < it.rows;
            const int q = it.q0 + (valid ? nt * 8 + r : 0);
            const int tok = a.sel ? 0 : q / a.G, hd = it.g * a.G + (a.sel ? q : q % a.G);
            const int64_t src = (static_cast<int64_t>(it.t0 + tok) * a.H + hd) * width + cq * (D / 4);
            float x[D / 4];
            if constexpr (PAD) {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) x[i] = cq * (D / 4) + i < width ? load_elem(static_cast<const TI*>(a.Q), src + i) : 0.f;
            } else {
                load_part<TI, D / 4>(static_cast<const TI*>(a.Q) + src, a.q_vec != 0, x);
            }
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
            const float down = __uint_as_float(static_cast<uint32_t>(e) << 23) * a.qscale;
            const long long p = static_cast<long long>(it.pos0) + tok;
            const int pos = valid ? static_cast<int>(max(min(p, static_cast<long long>(capk)), -1ll)) : 0x7fffffff;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                cqs[nt][i] = __shfl_sync(full, down, (2 * cq + i) * 4);
                rpos[nt][i] = __shfl_sync(full, pos, (2 * cq + i) * 4);
            }
#pragma unroll
            for (int ks = 0; ks < KW; ++ks) {
                const float x0 = x[4 * ks] * up, x1 = x[4 * ks + 1] * up, x2 = x[4 * ks + 2] * up, x3 = x[4 * ks + 3] * up;
                qh[nt][ks][0] = pack_f16x2(x0, x1);
                qh[nt][ks][1] = pack_f16x2(x2, x3);
                if constexpr (SPLITQ) {
                    ql[nt][ks][0] = rest_f16x2(x0, x1, qh[nt][ks][0]);
                    ql[nt][ks][1] = rest_f16x2(x2, x3, qh[nt][ks][1]);
                }
            }
        }
        int min_pos = 0x7fffffff;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) min_pos = min(min_pos, min(rpos[nt][0], rpos[nt][1]));
        min_pos = __reduce_min_sync(full, min_pos);

        float o[D / 16][NT][4], M[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            M[nt][0] = M[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.f;
        }

        // ---- walk the task's steps ------------------------------------------
        const int first = pt_first(sm_task[i % 3], warp);
        for (int k = 0; k < n; ++k) {
            if (warp == 0 && k == 2) {
                claimed = __shfl_sync(full, claimed, 0);
                word = task_word(claimed);
            }
            produce(i + 1);
            // all copies up to this step's: those of at most NST - 1 later steps may be under way
            if (issued - done - 1 >= NST - 1) copy_wait<NST - 1>();
            else if (NST > 2 && issued - done - 1 == NST - 2) copy_wait<(NST > 2 ? NST - 2 : 0)>();
            else copy_wait<0>();
            __syncwarp();
            const int st = done % NST;
            const StepFacts facts = sm_facts[warp][st];
            const int cnt = facts.cnt;
            const int key0 = (first + k * kTileWarps) * kStep;
            const uint8_t* kt = ring + st * STAGE;
            uint8_t* vt = ring + st * STAGE + kStep * ROW;

            // logits: keys 16 q + r (elements 0, 1) and + 8 (2, 3), rows 8 nt + 2 cq + (0, 1)
            float x[2][NT][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[q][nt][0] = x[q][nt][1] = x[q][nt][2] = x[q][nt][3] = 0.f;
                uint32_t w0[KW], w1[KW];
                lds_words<KW>(w0, kt + (q * 16 + r) * ROW + cq * (D / 4));
                lds_words<KW>(w1, kt + (q * 16 + 8 + r) * ROW + cq * (D / 4));
#pragma unroll
                for (int ks = 0; ks < KW; ++ks) {
                    uint32_t ka[4];
                    e4m3x4_f16(w0[ks], ka[0], ka[2]);
                    e4m3x4_f16(w1[ks], ka[1], ka[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(x[q][nt], ka, qh[nt][ks][0], qh[nt][ks][1]);
                        if constexpr (SPLITQ) mma_f16(x[q][nt], ka, ql[nt][ks][0], ql[nt][ks][1]);
                    }
                }
            }
            float lv[2], iv[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float vs = facts.vs[q];
                lv[q] = static_cast<float>(static_cast<int>((__float_as_uint(vs) >> 23) & 0xff) - 127);
                iv[q] = __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
            }
            // a = logit + log2(vscale), -inf where the row does not see the key
            const bool diagonal = !a.sel && key0 + kStep - 1 > min_pos;
            if (cnt == 0x1010 && !diagonal) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[q][nt][i] = fmaf(x[q][nt][i], cqs[nt][i & 1] * facts.ks[q], lv[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int col = (i >> 1) * 8 + r;     // within the half
                            const bool see = col < ((cnt >> (8 * q)) & 0xff) &&
                                             (a.sel || key0 + q * 16 + col <= rpos[nt][i & 1]);
                            x[q][nt][i] = see ? fmaf(x[q][nt][i], cqs[nt][i & 1] * facts.ks[q], lv[q]) : -INFINITY;
                        }
                if (diagonal) hide_nan<D, NT>(vt, rpos, key0, r, cq, o);
            }
            // the running maximum moves when a weight would pass 2^15
            bool move = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[nt][i] = fmaxf(fmaxf(x[0][nt][i], x[0][nt][i + 2]), fmaxf(x[1][nt][i], x[1][nt][i + 2]));
                    move |= top[nt][i] > M[nt][i] + kPSlack;
                }
            }
            if (__any_sync(full, move)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float t = top[nt][i];
                        t = fmaxf(t, __shfl_xor_sync(full, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(full, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(full, t, 16));
                        t = fmaxf(t, M[nt][i]);
                        const float f = M[nt][i] == t ? 1.f : ex2(M[nt][i] - t);
                        M[nt][i] = t;
                        l[nt][i] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[j][nt][i] *= f;
                            o[j][nt][i + 2] *= f;
                        }
                    }
                }
            }
            // weights, their sums, and the products with V
            uint32_t ph[2][NT][2], pl[2][SPLITP ? NT : 1][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = (M[nt][0] == -INFINITY ? 0.f : M[nt][0]) - kPBase;
                const float m1 = (M[nt][1] == -INFINITY ? 0.f : M[nt][1]) - kPBase;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float (&p)[4] = x[q][nt];
                    p[0] = ex2(p[0] - m0);
                    p[1] = ex2(p[1] - m1);
                    p[2] = ex2(p[2] - m0);
                    p[3] = ex2(p[3] - m1);
                    l[nt][0] = fmaf(p[0] + p[2], iv[q], l[nt][0]);
                    l[nt][1] = fmaf(p[1] + p[3], iv[q], l[nt][1]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t h = pack_f16x2(p[2 * b], p[2 * b + 1]);
                        ph[q][nt][b] = transpose8(h);
                        if constexpr (SPLITP) pl[q][nt][b] = transpose8(rest_f16x2(p[2 * b], p[2 * b + 1], h));
                    }
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
                    uint32_t va[2][4];         // features 4 v + (0, 1) and + (2, 3) of the lane's
                    e4m3x4_f16(__byte_perm(w[0][v], w[1][v], 0x5140), va[0][0], va[0][1]);
                    e4m3x4_f16(__byte_perm(w[0][v], w[1][v], 0x7362), va[1][0], va[1][1]);
                    e4m3x4_f16(__byte_perm(w[2][v], w[3][v], 0x5140), va[0][2], va[0][3]);
                    e4m3x4_f16(__byte_perm(w[2][v], w[3][v], 0x7362), va[1][2], va[1][3]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(o[2 * v + i][nt], va[i], ph[q][nt][0], ph[q][nt][1]);
                            if constexpr (SPLITP) mma_f16(o[2 * v + i][nt], va[i], pl[q][nt][0], pl[q][nt][1]);
                        }
                    }
                }
            }
            __syncwarp();    // (the stage is filled again in the next step)
            ++done;
        }

        if (warp == 0) {
            if (n <= 2) {
                claimed = __shfl_sync(full, claimed, 0);
                word = task_word(claimed);
            }
            put(i + 2, claimed, word);
        }

        // ---- join the warps, RJ rows at a time, each through its free stage --
        float* os = reinterpret_cast<float*>(ring + (issued % NST) * STAGE);
        if (lane == 0) sm_free[warp] = static_cast<int>(reinterpret_cast<uint8_t*>(os) - smem);
#pragma unroll
        for (int j0r = 0; j0r < R; j0r += RJ) {
            if (j0r > 0) __syncthreads();
#pragma unroll
            for (int n8 = 0; n8 < RJ / 8; ++n8) {
                const int nt = j0r / 8 + n8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = n8 * 8 + 2 * cq + i;
                    float t = l[nt][i];
                    t += __shfl_xor_sync(full, t, 4);
                    t += __shfl_xor_sync(full, t, 8);
                    t += __shfl_xor_sync(full, t, 16);
                    if (r == 0) {
                        sm_m[warp][row] = M[nt][i];
                        sm_l[warp][row] = t;
                    }
                    if (j0r + row < it.rows) {
                        float* to = os + row * OROW + r * (D / 8);
#pragma unroll
                        for (int j = 0; j < D / 16; j += 2)
                            *reinterpret_cast<float4*>(to + 2 * j) =
                                make_float4(o[j][nt][i], o[j][nt][i + 2], o[j + 1][nt][i], o[j + 1][nt][i + 2]);
                    }
                }
            }
            __syncthreads();
            for (int e = tid; e < min(RJ, it.rows - j0r) * (D / 4); e += kTileWarps * 32) {
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
                    const float4 x = *reinterpret_cast<const float4*>(smem + sm_free[w] + (row * OROW + d) * 4);
                    acc.x = fmaf(f, x.x, acc.x);
                    acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z);
                    acc.w = fmaf(f, x.w, acc.w);
                    sum = fmaf(f, sm_l[w][row], sum);
                }
                if (out_slot < 0) {
                    const int q = it.q0 + j0r + row;
                    const int tok = a.sel ? 0 : q / a.G, hd = it.g * a.G + (a.sel ? q : q % a.G);
                    if (!PAD || d < width)
                        store_out<TO>(static_cast<TO*>(a.out), (static_cast<int64_t>(it.t0 + tok) * a.H + hd) * width + d, acc, sum,
                                      a.o_vec != 0);
                } else {
                    const int64_t at = static_cast<int64_t>(out_slot) * R + j0r + row;
                    *reinterpret_cast<float4*>(wk.part_o + at * D + d) = acc;
                    if (d == 0) wk.part_ml[at] = make_float2(m, sum);
                }
            }
        }
        __syncthreads();     // (the free stages and sm_m are used again; the tasks up to i + 2 are there)
    }
    copy_wait<0>();
}

// Adds up the parts of the items that were cut.  Items of up to kJoinFew parts
// go to a block for every eight rows, a warp a row; of longer ones a block takes one row, its
// warps every kJoinWarps-th part, added in warp order (one request alone is
// cut into a part for every few hundred keys; with a warp a row that took
// 48 us for 76 parts, all of it latency).
constexpr int kJoinWarps = 8;
constexpr int kJoinFew = 16;
template <typename TO, int D, int R>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) k_cache_join(CacheAttn a, TileWork wk) {
    __shared__ float s_acc[kJoinWarps][D], s_sum[kJoinWarps], s_top[kJoinWarps];
    let_next_start();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned items = wk.plan->multi;
    const bool longer = wk.plan->most > kJoinFew;
    constexpr int V = D / 32;
    auto out_at = [&](const Item& it, int row) {
        const int x = it.q0 + row;
        const int tok = a.sel ? 0 : x / a.G, hd = it.g * a.G + (a.sel ? x : x % a.G);
        return (static_cast<int64_t>(it.t0 + tok) * a.H + hd) * a.c.D;      // (a.c.D < D: padded heads)
    };
    constexpr int GROUPS = R / kJoinWarps;
    for (unsigned long long j = blockIdx.x; j < static_cast<unsigned long long>(items) * GROUPS; j += gridDim.x) {
        const Task t = wk.multi[j / GROUPS];
        if (t.parts > kJoinFew) continue;
        const int row = static_cast<int>(j % GROUPS) * kJoinWarps + warp;
        if (row < t.it.rows) {
            const int64_t slot = static_cast<int64_t>(t.slot) * R + row;
            float2 ml = make_float2(-INFINITY, 0.f);       // lane i: part i
            if (lane < t.parts) ml = wk.part_ml[slot + lane * R];
            float top = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float f = ex2(ml.x - (top == -INFINITY ? 0.f : top));
            float acc[V], sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 8
            for (int i = 0; i < t.parts; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                sum = fmaf(fi, __shfl_sync(0xffffffffu, ml.y, i), sum);
                const float* p = wk.part_o + (slot + i * R) * D;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(fi, p[v * 32 + lane], acc[v]);
            }
            const int64_t at = out_at(t.it, row);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * 32 + lane < a.c.D)
                    store_elem(static_cast<TO*>(a.out), at + v * 32 + lane, sum == 0.f ? 0.f : acc[v] / sum);
        }
    }
    if (!longer) return;
    for (long long j = blockIdx.x; j < static_cast<long long>(items) * R; j += gridDim.x) {
        const Task t = wk.multi[j / R];
        const int row = static_cast<int>(j % R);
        if (t.parts <= kJoinFew || row >= t.it.rows) continue;       // (the same for the whole block)
        const int64_t slot = static_cast<int64_t>(t.slot) * R + row;
        float top = -INFINITY;
        for (int i = threadIdx.x; i < t.parts; i += kJoinWarps * 32)
            top = fmaxf(top, wk.part_ml[slot + static_cast<int64_t>(i) * R].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        __syncthreads();
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
        const float mu = top == -INFINITY ? 0.f : top;
        float acc[V], sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 8
        for (int i = warp; i < t.parts; i += kJoinWarps) {
            const int64_t at = slot + static_cast<int64_t>(i) * R;
            const float2 ml = wk.part_ml[at];
            const float* p = wk.part_o + at * D;
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
        if (d < a.c.D) {
            float o = 0.f, total = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                o += s_acc[w][d];
                total += s_sum[w];
            }
            store_elem(static_cast<TO*>(a.out), out_at(t.it, row) + d, total == 0.f ? 0.f : o / total);
        }
    }
}

// ---- host -------------------------------------------------------------------
// The plan, a kernel that works through it (tiles of R rows, D features), and
// the join of what was cut.  resident: blocks an SM, where the occupancy that
// CUDA reports is not it.
template <typename TO, int D, int R>
gtattn_status launch_planned(void (*kernel)(CacheAttn, TileWork), int threads, int smem, int tasks_per_block,
                             const CacheAttn& a, cudaStream_t s, int resident = 0) {
    int per_sm = blocks_per_sm(reinterpret_cast<const void*>(kernel), threads, smem);
    if (per_sm < 1) return GTATTN_ERR_CUDA;
    if (resident) per_sm = resident;
    const int blocks = num_sms() * per_sm;
    const int64_t rows_all = (int64_t)a.r.T * a.G;
    const int64_t keys = a.sel ? (int64_t)a.n_sel * a.c.page : (int64_t)a.r.max_pages * a.c.page;
    const int64_t items = a.sel ? (int64_t)a.r.T * a.c.Hkv * ((a.G + R - 1) / R)
                                : a.c.Hkv * ((rows_all + R - 1) / R + a.r.S);       // at most
    const bool cut = keys > kUnit;       // (an item of one unit is never cut)
    TileWork wk{};
    if (!cut && items <= blocks) {
        ProfScope ps(GTATTN_KCAT_CACHE, 1, s);
        GT_CUDA(launch_after(kernel, dim3((unsigned)items), threads, smem, s, a, wk));
        return GTATTN_OK;
    }
    wk.target = tasks_per_block * blocks;
    // items of several tasks have more than lc units: at most 2 * units / lc <= 2 * target parts in all
    const size_t slots = cut ? 2 * (size_t)wk.target : 0;
    const size_t n_o = sizeof(float) * slots * R * D, n_ml = sizeof(float2) * slots * R;
    const size_t n_list = sizeof(Task) * ((size_t)items + slots);
    const size_t n_multi = cut ? sizeof(Task) * (size_t)std::min<int64_t>(items, wk.target) : 0;
    const size_t n_pre = a.sel || a.r.S <= kPlanHeld ? 0 : 3 * sizeof(int) * (size_t)a.r.S;
    void* ws = nullptr;
    GT_TRY(pool_alloc(&ws, n_o + n_ml + n_list + sizeof(TilePlan) + n_multi + n_pre, s));
    char* at = static_cast<char*>(ws);
    wk.part_o = reinterpret_cast<float*>(at);
    wk.part_ml = reinterpret_cast<float2*>(at += n_o);
    wk.list = reinterpret_cast<Task*>(at += n_ml);
    wk.plan = reinterpret_cast<TilePlan*>(at += n_list);
    wk.multi = reinterpret_cast<Task*>(at += sizeof(TilePlan));
    wk.pre = reinterpret_cast<int*>(at += n_multi);
    cudaError_t e;
    {
        ProfScope ps(GTATTN_KCAT_CACHE, cut ? 3 : 2, s);
        const int64_t list = items + (int64_t)slots;        // tasks, at most
        e = launch_after(k_cache_plan, dim3((unsigned)std::min<int64_t>(num_sms(), (list + 2 * kPlanThreads - 1) / (2 * kPlanThreads))),
                         kPlanThreads, 0, s, a, wk, R);
        if (e == cudaSuccess)
            e = launch_after(kernel, dim3((unsigned)(cut ? blocks : std::min<int64_t>(blocks, items))), threads, smem, s, a, wk);
        if (cut && e == cudaSuccess)
            e = launch_after(k_cache_join<TO, D, R>, dim3((unsigned)std::min<int64_t>(items * R, num_sms() * 4)), kJoinWarps * 32, 0,
                             s, a, wk);
    }
    pool_free(ws, s);
    return e == cudaSuccess ? GTATTN_OK : cuda_status(e);
}

template <typename TI, typename TO, int D, int NT, bool SPLITQ, bool SPLITP>
gtattn_status launch_tile(const CacheAttn& a, cudaStream_t s) {
    return launch_planned<TO, D, 8 * NT>(k_cache_attn_tile<TI, TO, D, NT, SPLITQ, SPLITP>, kTileWarps * 32, tile_smem<D, NT>(),
                                         kTasksPerBlock, a, s);
}

template <int D, int NT> gtattn_status launch_tile_n(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (dtype == GTATTN_F32) return launch_tile<float, float, D, NT, true, true>(a, s);
    if (dtype == GTATTN_BF16) return launch_tile<B, B, D, NT, false, false>(a, s);
    return launch_tile<B, float, D, NT, false, true>(a, s);
}
// Heads of a.c.D < D features, 16 rows a tile.
template <int D> gtattn_status launch_tile_padded(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    using B = __nv_bfloat16;
    constexpr int threads = kTileWarps * 32, smem = tile_smem<D, 2>();
    if (dtype == GTATTN_F32)
        return launch_planned<float, D, 16>(k_cache_attn_tile<float, float, D, 2, true, true, true>, threads, smem, kTasksPerBlock, a, s);
    if (dtype == GTATTN_BF16)
        return launch_planned<B, D, 16>(k_cache_attn_tile<B, B, D, 2, false, false, true>, threads, smem, kTasksPerBlock, a, s);
    return launch_planned<float, D, 16>(k_cache_attn_tile<B, float, D, 2, false, true, true>, threads, smem, kTasksPerBlock, a, s);
}
// 8, 16 or 32 rows a tile, by the rows that a request brings per K/V head (32
// not at D = 128 nor, with its queries in two parts, in fp32: registers).
template <int D> gtattn_status launch_tile_d(const CacheAttn& a, gtattn_dtype dtype, int64_t rows, cudaStream_t s) {
    if (rows <= 8) return launch_tile_n<D, 1>(a, dtype, s);
    if constexpr (D < 128)
        if (rows > 16 && dtype != GTATTN_F32) {
            using B = __nv_bfloat16;
            return dtype == GTATTN_BF16 ? launch_tile<B, B, D, 4, false, false>(a, s)
                                        : launch_tile<B, float, D, 4, false, true>(a, s);
        }
    return launch_tile_n<D, 2>(a, dtype, s);
}

}  // namespace
}  // namespace gt
