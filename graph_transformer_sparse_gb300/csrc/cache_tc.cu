// cache_tc.cu -- attention over the 8-bit cache for many rows at once (a
// prompt's next piece), on the 5th-generation tensor cores: 128 rows a tile
// (tcgen05, accumulators in tensor memory), heads of 64 or 128, bf16 queries.
//
// A block of eight warps, two blocks an SM.  Warps 4-7 bring the keys: e4m3
// codes by 16-byte loads, converted to fp16 (exact) and stored in the
// 128-byte-swizzled layout that the products read.  Warps 0-3 are the rows, a
// thread each (= its lane of tensor memory): S_j = Q K_j^T comes out of tensor
// memory in pieces of 32 columns and goes back as weights in fp16 (with a
// second fp16 for the rest where the output is fp32), under the maximum so far;
// where that is not known yet or has become too small S_j is read twice.  Then one thread issues O += P_j V_j and S_(j+1),
// and everybody meets at its end; meanwhile warps 4-7 have stored tile j + 1.
// The other block of the SM works while this one waits.  Scales, the running
// maximum's slack and the cut of the work are those of cache_tile.cuh, and so
// are the parts that k_cache_join adds up.
//
// Bound by the softmax's instructions (per element two FMAs, a maximum, an
// exp2, half a conversion and an addition against 4 D product operations): 4
// requests adding 2000 tokens to 8000, 32 heads over 8 of 64, take 460 us
// (469 TFLOP/s; the tiles of cache_tile.cuh 937 us), 8000-token prompts of 16
// heads over 8 of 128 401 us (861).  From 64 rows a request and K/V head on:
// with 17 tokens of 4 heads both take 61 us, with 64 tokens 115 against 143.
// Every wait for the tensor cores is bounded: a block whose wait runs out
// records an error (gtattn_device_errors), waits for what it issued, frees its
// tensor memory and ends.
#include "cache_tile.cuh"
#include "tc.cuh"

namespace gt {
namespace {

__device__ int g_cache_errors;      // 1: a bounded wait gave up

constexpr int kTcThreads = 256;
constexpr int kTcRows = 128;
constexpr int kTcTasks = 2;         // tasks aimed at for each resident block
constexpr uint32_t kTcCols = 256;   // tensor memory of a block: S and P, then O
constexpr uint32_t kTcColO = 128;

template <int D> struct TcCfg {
    static constexpr int KT = D == 64 ? 128 : 64;             // keys a tile
    static constexpr int GR = KT / 16;                        // groups of 16 keys (one page, one scale)
    static constexpr int QB = kTcRows * D * 2, KB = KT * D * 2;
    // columns of the weights: beside S where they fit (S can then be read again), else over it
    static constexpr bool apart(bool split) { return D == 128 || !split; }
    static constexpr uint32_t col_p(bool split) { return !apart(split) ? 0u : D == 128 ? 64u : 192u; }
    static constexpr uint32_t col_step(bool split) { return apart(split) ? 16u : 32u; }     // 32 keys
    static constexpr uint32_t col_rest(bool split) { return apart(split) ? 32u : 16u; }     // their rests
    static constexpr int SMEM = QB + 4 * KB + 1024;           // Q, two stages of K and V, alignment
};

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                 "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// kind::f16 with fp16 A and B, fp32 D
constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// A 16-key group of a tile: page (below 0: none), valid keys, scales.
struct Group {
    int pid, cnt;
    float ks, vs;
};
// What the rows need of it: the keys' scale, log2 of the values' and its inverse.
struct alignas(16) GroupFacts {
    int cnt;
    float ks, lv, iv;
};
constexpr float kTcBase = 4.f;          // weights are 2^(a - M + 4) ...
constexpr float kTcSumLimit = 32768.f;  // ... and a tile's add up to this at most, or M moves

template <typename TO, int D, bool SPLITP>
__global__ void __launch_bounds__(kTcThreads, 2) k_cache_attn_tc(CacheAttn a, TileWork wk) {
    using C = TcCfg<D>;
    constexpr int KT = C::KT, GR = C::GR, KPW = KT / 4, GPW = KPW / 16;     // keys and groups of a loading warp
    constexpr int SUB = KT * 128;         // bytes between a key tile's 64-feature halves (D = 128)
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sQ = smem;
    auto sK = [&](int b) { return smem + C::QB + b * 2 * C::KB; };
    auto sV = [&](int b) { return smem + C::QB + b * 2 * C::KB + C::KB; };
    __shared__ Task sm_task[2];
    __shared__ int sm_more[2];
    __shared__ GroupFacts sm_group[2][GR];
    __shared__ int sm_page[2][GR];
    // per tile (j mod 3): keys whose value holds a NaN, where some row does not see them; written while tile
    // j - 1 is worked on, read with tile j, cleared with tile j + 1
    __shared__ uint32_t sm_nan[3][4];
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t s_tmem;
    const unsigned full = 0xffffffffu;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const CacheView& c = a.c;
    const bool rows_side = warp < 4;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&s_tmem)), "r"(kTcCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < 12) (&sm_nan[0][0])[tid] = 0;
    let_next_start();
    after_previous();
    const unsigned tasks = wk.plan ? wk.plan->tasks : 0;
    if (warp == 4) {
        if (wk.plan) {
            if (lane < kTaskWords && blockIdx.x < tasks)
                reinterpret_cast<int*>(&sm_task[0])[lane] = reinterpret_cast<const int*>(wk.list + blockIdx.x)[lane];
            if (lane == 0) sm_more[0] = blockIdx.x < tasks;
        } else {
            Task t{};
            const bool more = task_plain(a, kTcRows, blockIdx.x, lane, &t);
            if (lane == 0) {
                sm_task[0] = t;
                sm_more[0] = more;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr uint32_t idS = idesc_f16(128, KT, 0), idO = idesc_f16(128, D, 1);
    uint32_t waits = 0;          // commits waited for (the barrier's phase)
    bool failed = false;         // uniform over the block
    auto wait_mma = [&]() {
        const bool ok = mbar_wait(&bar, waits & 1);
        ++waits;
        tc_fence_after();
        return ok;
    };

    for (int i = 0; !failed && sm_more[i & 1]; ++i) {
        const Task task = sm_task[i & 1];
        const Item& it = task.it;
        const int key_b = task.j0 * kUnit;
        const int key_e = static_cast<int>(min(static_cast<long long>(it.n_keys), static_cast<long long>(task.j1) * kUnit));
        const int T = key_e > key_b ? (key_e - key_b + KT - 1) / KT : 0;
        const int cap = a.r.max_pages * c.page - 1;
        auto pos_of = [&](int row) {     // the position of tile row `row`'s token
            const long long p = static_cast<long long>(it.pos0) + (it.q0 + row) / a.G;
            return static_cast<int>(max(min(p, static_cast<long long>(cap)), -1ll));
        };
        const int* trow = a.r.table + static_cast<int64_t>(it.s) * a.r.max_pages;
        const int min_pos = pos_of(0);

        // ---- warps 4-7: keys ------------------------------------------------
        const int lw = warp - 4;
        auto look = [&](int j) {          // lane g < GPW: the warp's group g of tile j
            Group h{-1, 0, 1.f, 1.f};
            const int key = key_b + j * KT + lw * KPW + lane * 16;
            if (lane < GPW && j < T && key < key_e) {
                const int pid = __ldg(trow + (key >> c.lp));
                if (static_cast<unsigned>(pid) < static_cast<unsigned>(c.pages)) {
                    const int64_t ph = static_cast<int64_t>(pid) * c.Hkv + it.g;
                    h = Group{pid, min(16, key_e - key), __ldg(c.kscale + ph), __ldg(c.vscale + ph)};
                }
            }
            return h;
        };
        uint4 kr[4], vr[4];
        auto fetch = [&](const Group& h, int j) {      // the warp's KPW rows of tile j: 4 x 32 16-byte pieces of K and V
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int ch = x * 32 + lane, row = ch / (D / 16), col = ch % (D / 16);
                const int pid = __shfl_sync(full, h.pid, row / 16), cnt = __shfl_sync(full, h.cnt, row / 16);
                kr[x] = vr[x] = make_uint4(0u, 0u, 0u, 0u);
                if ((row & 15) < cnt) {
                    const int off = (key_b + j * KT + lw * KPW + row) & (c.page - 1);
                    const int64_t at = ((((static_cast<int64_t>(pid) * c.Hkv + it.g) << c.lp) + off) * D) + col * 16;
                    kr[x] = __ldg(reinterpret_cast<const uint4*>(c.k8 + at));
                    vr[x] = __ldg(reinterpret_cast<const uint4*>(c.v8 + at));
                }
            }
        };
        auto put8 = [&](unsigned char* tile, int row, int col8, uint32_t w0, uint32_t w1) {    // 8 codes, features 8 col8 ..
            uint4 h;
            e4m3x4_f16(w0, h.x, h.y);
            e4m3x4_f16(w1, h.z, h.w);
            *reinterpret_cast<uint4*>(tile + (col8 >> 3) * SUB + row * 128 + (((col8 & 7) ^ (row & 7)) << 4)) = h;
        };
        auto store = [&](const Group& h, int j) {
            const int b = j & 1;
            const bool diagonal = key_b + (j + 1) * KT - 1 > min_pos;
            if (lane < GPW) {
                const uint32_t e = __float_as_uint(h.vs) & 0x7f800000u;
                sm_page[b][lw * GPW + lane] = h.pid;
                sm_group[b][lw * GPW + lane] =
                    GroupFacts{h.cnt, h.ks, static_cast<float>(static_cast<int>(e >> 23) - 127), __uint_as_float((254u << 23) - e)};
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int ch = x * 32 + lane, row = ch / (D / 16), col = ch % (D / 16), key = lw * KPW + row;
                put8(sK(b), key, 2 * col, kr[x].x, kr[x].y);
                put8(sK(b), key, 2 * col + 1, kr[x].z, kr[x].w);
                if (diagonal) {           // (a NaN times a weight of 0 would reach rows that do not see it)
                    uint32_t* w = reinterpret_cast<uint32_t*>(&vr[x]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t n = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        if (n) {
                            w[k] &= ~((n >> 7) * 0xffu);
                            atomicOr(&sm_nan[j % 3][key >> 5], 1u << (key & 31));
                        }
                    }
                }
                put8(sV(b), key, 2 * col, vr[x].x, vr[x].y);
                put8(sV(b), key, 2 * col + 1, vr[x].z, vr[x].w);
            }
        };
        Group g0{}, g1{}, g2{};           // groups of the tile being fetched, and of the two after it
        if (!rows_side) {
            g0 = look(0);
            g1 = look(1);
            g2 = look(2);
            if (T > 0) {
                fetch(g0, 0);
                store(g0, 0);
            }
        }

        // ---- warps 0-3: rows ------------------------------------------------
        const int row = (warp & 3) * 32 + lane;
        const bool valid = row < it.rows;
        const int pos = valid ? pos_of(row) : 0x7fffffff;
        const int qrow = it.q0 + (valid ? row : 0);
        const int64_t at_out = (static_cast<int64_t>(it.t0 + qrow / a.G) * a.H + it.g * a.G + qrow % a.G) * D;
        float cq = 0.f, M = -INFINITY, l = 0.f;
        uint32_t poisoned[D / 32];        // features that a NaN reached
#pragma unroll
        for (int x = 0; x < D / 32; ++x) poisoned[x] = 0u;
        if (rows_side) {
            const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q) + at_out;
            float amax = 0.f;
#pragma unroll
            for (int d = 0; d < D; d += 8) {
                float x[8];
                load_part<__nv_bfloat16, 8>(Q + d, a.q_vec != 0, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float v = fabsf(x[k]);
                    if (v < INFINITY) amax = fmaxf(amax, v);
                }
            }
            // 2^e with amax / 2^e in [2^14, 2^15), as in cache_tile.cuh
            const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 14, 15);
            const float up = valid ? __uint_as_float(static_cast<uint32_t>(254 - e) << 23) : 0.f;
            cq = __uint_as_float(static_cast<uint32_t>(e) << 23) * a.qscale;
#pragma unroll
            for (int d = 0; d < D; d += 8) {
                float x[8];
                load_part<__nv_bfloat16, 8>(Q + d, a.q_vec != 0, x);
                if (!valid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = 0.f;
                }
                *reinterpret_cast<uint4*>(sQ + (d >> 6) * (kTcRows * 128) + row * 128 + ((((d >> 3) & 7) ^ (row & 7)) << 4)) =
                    make_uint4(pack_f16x2(x[0] * up, x[1] * up), pack_f16x2(x[2] * up, x[3] * up),
                               pack_f16x2(x[4] * up, x[5] * up), pack_f16x2(x[6] * up, x[7] * up));
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncthreads();
        const uint64_t dQ = smem_desc_sw128(su32(sQ), 16, 1024);
        auto issue_s = [&](int b) {       // S = Q K^T, by one thread
            const uint64_t dK = smem_desc_sw128(su32(sK(b)), 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_ss(tmem, dQ + (k >> 2) * ((kTcRows * 128) >> 4) + (k & 3) * 2, dK + (k >> 2) * (SUB >> 4) + (k & 3) * 2, idS,
                       k > 0);
        };
        if (warp == 4 && lane == 0 && T > 0) {
            tc_fence_after();
            issue_s(0);
            commit_one(&bar);
        }
        // the next task
        unsigned claimed = 0;
        if (warp == 4 && lane == 0 && wk.plan) claimed = gridDim.x + atomicAdd(&wk.plan->next, 1u);

        for (int j = 0; j < T; ++j) {
            const int b = j & 1;
            bool ok;
            if (!rows_side) {
                // tile j + 1: under way before S_j is there, stored after it (O += P_(j-1) V_(j-1) has then read its stage)
                g0 = g1;
                g1 = g2;
                if (j + 1 < T) fetch(g0, j + 1);
                g2 = look(j + 3);
                ok = wait_mma();
                if (j + 1 < T) store(g0, j + 1);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            } else {
                ok = wait_mma();
                const uint32_t tS = tmem + lane_base, tP = tS + C::col_p(SPLITP);
                const int key0 = key_b + j * KT;
                const int ahead = pos - key0;          // the row sees the tile's keys 0 .. ahead
                // a = logit + log2(vscale) of columns 32 x + 16 q .. + 15, -inf where the row does not see the key
                auto logits = [&](const uint32_t* s, const GroupFacts& g, int first, float* v) {
                    const float cs = cq * g.ks;
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = fmaf(__uint_as_float(s[k]), cs, g.lv);
                    const int see = min(g.cnt, ahead - first + 1);
                    if (see < 16) {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (k >= see) v[k] = -INFINITY;
                    }
                };
                // The maximum is looked for in a task's first tile, and where a tile's weights grow too large
                // under the one so far (or, where the weights take S's place, before it is known: always).
                bool look_top = j == 0 || !C::apart(SPLITP);
                for (;;) {
                    if (look_top) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int x = 0; x < KT / 32; ++x) {
                            uint32_t s[32];
                            tmem_ld32(tS + 32 * x, s);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float v[16];
                                logits(s + 16 * q, sm_group[b][2 * x + q], 32 * x + 16 * q, v);
#pragma unroll
                                for (int k = 0; k < 16; ++k) top = fmaxf(top, v[k]);
                            }
                        }
                        if (__any_sync(full, top > M + (C::apart(SPLITP) ? 0.f : kPSlack))) {
                            const float t = fmaxf(top, M), f = M == t ? 1.f : ex2(M - t);
                            M = t;
                            l *= f;
                            if (j > 0) {
#pragma unroll 1
                                for (int x = 0; x < D / 32; ++x) {
                                    uint32_t o[32];
                                    tmem_ld32(tmem + lane_base + kTcColO + 32 * x, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                    tmem_st32(tmem + lane_base + kTcColO + 32 * x, o);
                                }
                            }
                        }
                    }
                    const float mu = (M == -INFINITY ? 0.f : M) - kTcBase;
                    float sum = 0.f, scaled = 0.f;
#pragma unroll 1
                    for (int x = 0; x < KT / 32; ++x) {
                        uint32_t s[32];
                        tmem_ld32(tS + 32 * x, s);
                        tmem_ld_wait();
                        uint32_t p[SPLITP ? 32 : 16];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const GroupFacts g = sm_group[b][2 * x + q];
                            float v[16];
                            logits(s + 16 * q, g, 32 * x + 16 * q, v);
                            float s0 = 0.f, s1 = 0.f;
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                v[k] = ex2(v[k] - mu);
                                v[k + 1] = ex2(v[k + 1] - mu);
                                s0 += v[k];
                                s1 += v[k + 1];
                                const uint32_t h = pack_f16x2(v[k], v[k + 1]);
                                p[8 * q + k / 2] = h;
                                if constexpr (SPLITP) p[16 + 8 * q + k / 2] = rest_f16x2(v[k], v[k + 1], h);
                            }
                            s0 += s1;
                            sum += s0;
                            scaled = fmaf(s0, g.iv, scaled);
                        }
                        if constexpr (!SPLITP) {
                            tmem_st16(tP + C::col_step(false) * x, p);
                        } else if constexpr (C::apart(true)) {
                            tmem_st16(tP + C::col_step(true) * x, p);
                            tmem_st16(tP + C::col_step(true) * x + C::col_rest(true), p + 16);
                        } else {
                            tmem_st32(tP + C::col_step(true) * x, p);
                        }
                    }
                    const bool over = !look_top && !(sum <= kTcSumLimit);      // (a NaN: looked for once)
                    if (!__any_sync(full, over)) {
                        l += scaled;
                        break;
                    }
                    look_top = true;
                }
                tmem_st_wait();
                if (tid < 4) sm_nan[(j + 2) % 3][tid] = 0;
                const uint32_t* nan = sm_nan[j % 3];
                if (nan[0] | nan[1] | nan[2] | nan[3]) {
                    for (int k = 0; k < KT; ++k) {
                        if (!((nan[k >> 5] >> (k & 31)) & 1u) || !valid || key0 + k > pos) continue;
                        const int64_t ph = static_cast<int64_t>(sm_page[b][k >> 4]) * c.Hkv + it.g;
                        const uint8_t* v = c.v8 + ((ph << c.lp) + ((key0 + k) & (c.page - 1))) * D;
#pragma unroll
                        for (int d = 0; d < D; ++d)
                            if ((v[d] & 0x7f) == 0x7f) poisoned[d >> 5] |= 1u << (d & 31);
                    }
                }
            }
            tc_fence_before();
            failed = __syncthreads_or(!ok);
            if (failed) break;
            if (warp == 4 && lane == 0) {
                tc_fence_after();
                const uint64_t dV = smem_desc_sw128(su32(sV(b)), SUB, 1024);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k) {           // 16 keys: 8 columns of P, 16 rows of V
                    const uint32_t pa = tmem + C::col_p(SPLITP) + C::col_step(SPLITP) * (k >> 1) + 8 * (k & 1);
                    mma_ts(tmem + kTcColO, pa, dV + k * 128, idO, j > 0 || k > 0);
                    if constexpr (SPLITP) mma_ts(tmem + kTcColO, pa + C::col_rest(SPLITP), dV + k * 128, idO, 1u);
                }
                if (j + 1 < T) issue_s(b ^ 1);
                commit_one(&bar);
            }
        }
        if (failed) break;
        if (warp == 4) {
            const unsigned x = __shfl_sync(full, claimed, 0);
            const bool more = wk.plan && x < tasks;
            if (lane < kTaskWords && more)
                reinterpret_cast<int*>(&sm_task[(i + 1) & 1])[lane] = reinterpret_cast<const int*>(wk.list + x)[lane];
            if (lane == 0) sm_more[(i + 1) & 1] = more;
        }
        if (tid < 12) (&sm_nan[0][0])[tid] = 0;       // (all tiles' are read)
        bool ok = true;
        if (T > 0) ok = wait_mma();
        if (rows_side && __all_sync(full, ok)) {
            const float inv = task.slot < 0 ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                uint32_t o[32];
                if (T > 0) {
                    tmem_ld32(tmem + lane_base + kTcColO + 32 * x, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    if (!valid) break;
                    float4 y = make_float4(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv,
                                           __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
                    const uint32_t bad = poisoned[x] >> k;
                    if (bad & 1u) y.x = NAN;
                    if (bad & 2u) y.y = NAN;
                    if (bad & 4u) y.z = NAN;
                    if (bad & 8u) y.w = NAN;
                    if (task.slot < 0)
                        store_out<TO>(static_cast<TO*>(a.out), at_out + 32 * x + k, y, 1.f, a.o_vec != 0);
                    else
                        *reinterpret_cast<float4*>(wk.part_o + (static_cast<int64_t>(task.slot) * kTcRows + row) * D + 32 * x + k) = y;
                }
            }
            if (task.slot >= 0 && valid) wk.part_ml[static_cast<int64_t>(task.slot) * kTcRows + row] = make_float2(M, l);
        }
        tc_fence_before();
        failed = __syncthreads_or(!ok);
        tc_fence_after();
    }
    if (failed) {
        if (tid == 0) atomicOr(&g_cache_errors, 1);
        if (warp == 4 && lane == 0) {     // what was issued ends before its tensor memory goes
            commit_one(&bar);
            for (int x = 0; x < 2; ++x) mbar_wait(&bar, (waits + 1 + x) & 1, kTcWaitCycles / 4);      // (the one that ran out, and this)
        }
        __syncthreads();
    }
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcCols) : "memory");
    }
}

// (two blocks an SM: registers and shared memory are cut for that; the occupancy query says one of a kernel
// that allocates tensor memory, though two take half of it each)
template <int D> gtattn_status launch_tc(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (dtype == GTATTN_BF16)
        return launch_planned<B, D, kTcRows>(k_cache_attn_tc<B, D, false>, kTcThreads, TcCfg<D>::SMEM, kTcTasks, a, s, 2);
    return launch_planned<float, D, kTcRows>(k_cache_attn_tc<float, D, true>, kTcThreads, TcCfg<D>::SMEM, kTcTasks, a, s, 2);
}

}  // namespace

bool cache_tc_takes(const CacheAttn& a, gtattn_dtype dtype, int64_t rows) {
    return !a.sel && dtype != GTATTN_F32 && (a.c.D == 64 || a.c.D == 128) && rows >= kCacheTcMinRows;
}
gtattn_status cache_tc(const CacheAttn& a, gtattn_dtype dtype, cudaStream_t s) {
    return a.c.D == 64 ? launch_tc<64>(a, dtype, s) : launch_tc<128>(a, dtype, s);
}
cudaError_t cache_tc_errors(int* code, int reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_cache_errors, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && reset) e = cudaMemcpyToSymbol(g_cache_errors, &zero, sizeof(int));
    return e;
}
}  // namespace gt
