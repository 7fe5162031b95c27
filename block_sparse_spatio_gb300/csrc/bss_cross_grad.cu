// bss_cross_grad.cu -- gradients of the cross attention.
//
//   P = exp(scale q k^T - lse),  D = sum dO O,  dS = P (dO v^T - D)
//   dq = scale dS k,  dv = P^T dO,  dk = scale dS^T q
//
// Two kernels, each with its own P and dS (7 products of rows x keys x d where 5
// would do): one has the rows in TMEM's lanes and sums dq over the keys, the other
// the keys and sums dk and dv over the rows.  One kernel would need dq's sums over
// the key tiles in memory: atomics, whose order changes results, or a pass of their
// own.
//
// dq: a CTA takes items of (group, 128 rows, head); per key tile the products
// S(t+1), dQ(t), dP(t+1) follow one another, so that P(t+1) is made beneath dQ(t) and
// dP(t+1), dS(t) beneath S(t+1).  D is made here, once an item, and kept for the
// second kernel.
//
// dk, dv: the pairs of (key tile, row tile) of all heads lie in a line that is cut
// into equal runs, one a CTA, whatever the lengths; a key tile's products are S(t+1),
// dK(t), dP(t+1), dV(t+1) over its row tiles.  Where a run ends inside a key tile the
// sums go to the workspace in 32 bits, and a third kernel adds them in their order.
#include "bss_cross.cuh"

#include <cstring>
#include <type_traits>

namespace bss {
namespace {

constexpr int kThreads = 384;
constexpr int kElementwise = 256;  // threads 128 .. 383: a lane of TMEM and half of the columns
constexpr uint32_t kRegsControl = 72, kRegsElementwise = 208;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColA = 256, kColB = 384;  // S, dP, two accumulators

struct GradArgs {
    CUtensorMap q, dO, k, v;
    CrossShape s;
    int32_t tiles;      // of 128 rows in a group
    int32_t key_tiles;  // of 128 keys in a group
    int64_t items;      // of the first kernel
    int32_t blocks;     // of the second
    const uint16_t* O;
    uint16_t *dq, *dk, *dv;
    int64_t O_row, O_head, dq_row, dq_head;
    int64_t dk_group, dk_token, dk_head, dv_group, dv_token, dv_head;
    float scale;
    const float* lse;  // [heads][rows]
    float* delta;      // [heads][rows]
    int64_t* starts;   // [groups + 1]: pairs of key and row tiles in front of a group
    float* parts;      // [2 blocks][2][128][d]
    int* status;
};

// where half of a thread's columns lies, and 16 columns of an operand in TMEM: each
// half of the columns keeps its bf16 values at the start of its own 64
__device__ __forceinline__ uint32_t packed_col(int kk) { return static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8); }

__device__ __forceinline__ void store_packed(uint32_t at, const float (&v)[64]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = pack_bf16x2(v[32 * q + 2 * x], v[32 * q + 2 * x + 1]);
        BSS_TMEM_ST16(at + 16 * q, w);
    }
}

// A row's (or key's) accumulator columns [first, first + 32 NC) -> bf16 memory
template <int NC>
__device__ __forceinline__ void store_row(uint32_t at, uint16_t* to, float scale, bool live) {
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) {
        uint32_t o[32];
        BSS_TMEM_LD32(at + cc * 32, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    w[x] = pack_bf16x2(__uint_as_float(o[8 * u + 2 * x]) * scale, __uint_as_float(o[8 * u + 2 * x + 1]) * scale);
                reinterpret_cast<uint4*>(to + cc * 32)[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// ---------------------------------------------------------------- dq
constexpr int kKStages = 3, kVStages = 2;

template <int D>
struct DqSmem {
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kQ = 0, kDO = kTile, kK = 2 * kTile, kV = kK + kKStages * kTile;
    static constexpr uint32_t kDelta = kV + kVStages * kTile;  // float [2][2][128]
    static constexpr uint32_t kBar = kDelta + 2048;
    // q_full q_empty do_full do_empty k_full k_empty v_full v_empty s_full s_read dp_full ds_full dq_done[2] halves
    static constexpr uint32_t kBars = 4 + 2 * kKStages + 2 * kVStages + 7;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 16;
};

struct DqItem {
    int group, row0, rows, head, valid, n;
};

__device__ __forceinline__ DqItem dq_item(const GradArgs& a, int64_t i) {
    DqItem t;
    const int64_t rest = i / a.s.heads;
    t.head = static_cast<int>(i - rest * a.s.heads);
    t.group = static_cast<int>(rest / a.tiles);
    t.row0 = static_cast<int>(rest - static_cast<int64_t>(t.group) * a.tiles) * 128;
    t.rows = a.s.rows_of(t.group) - t.row0;
    t.valid = t.rows > 0 ? a.s.valid(t.group) : 0;
    t.n = (t.valid + kKeyTile - 1) / kKeyTile;
    return t;
}

// starts[], by one warp
__device__ __forceinline__ void count_pairs(const GradArgs& a) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int g0 = 0; g0 < a.s.groups; g0 += 32) {
        const int g = g0 + lane;
        int64_t n = 0;
        if (g < a.s.groups)
            n = static_cast<int64_t>((a.s.valid(g) + kKeyTile - 1) / kKeyTile) * ((a.s.rows_of(g) + 127) / 128) * a.s.heads;
        int64_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (g < a.s.groups) a.starts[g] = before + sum - n;
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) a.starts[a.s.groups] = before;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_dq_kernel(const __grid_constant__ GradArgs a) {
    using L = DqSmem<D>;
    constexpr int kChunks = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* q_empty = q_full + 1;
    uint64_t* do_full = q_empty + 1;
    uint64_t* do_empty = do_full + 1;
    uint64_t* k_full = do_empty + 1;
    uint64_t* k_empty = k_full + kKStages;
    uint64_t* v_full = k_empty + kKStages;
    uint64_t* v_empty = v_full + kVStages;
    uint64_t* s_full = v_empty + kVStages;
    uint64_t* s_read = s_full + 1;
    uint64_t* dp_full = s_read + 1;
    uint64_t* ds_full = dp_full + 1;
    uint64_t* dq_done = ds_full + 1;
    uint64_t* halves = dq_done + 2;  // both halves of a row's D are there
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(halves + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles could not be addressed
        record_status(a.status, BSS_ERR_CUDA);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1 + kElementwise / 32);
        for (int i = 0; i < kKStages; ++i) mbar_init(k_full + i, 1), mbar_init(k_empty + i, 1);
        for (int i = 0; i < kVStages; ++i) mbar_init(v_full + i, 1), mbar_init(v_empty + i, 1);
        mbar_init(s_full, 1);
        mbar_init(s_read, kElementwise);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, kElementwise);
        mbar_init(dq_done, 1);
        mbar_init(dq_done + 1, 1);
        mbar_init(halves, kElementwise);
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&a.q);
            tma_prefetch_desc(&a.dO);
            tma_prefetch_desc(&a.k);
            tma_prefetch_desc(&a.v);
            uint32_t items = 0, dos = 0, ks = 0, vs = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
                const DqItem t = dq_item(a, i);
                if (t.n == 0) continue;
                const int row = t.group * a.s.group_rows + t.row0;
                const int kv = t.head / a.s.share, g = a.s.shared_states ? 0 : t.group;
                if (items > 0) ok = mbar_wait(q_empty, (items - 1) & 1, a.status);
                if (!ok) break;
                mbar_arrive_expect_tx(q_full, L::kTile);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    tma_load_3d(smem + L::kQ + c * kChunkBytesSw128, &a.q, c * 64, row, t.head, q_full);
                ++items;
                for (int j = 0; ok && j < t.n; ++j) {
                    const uint32_t sk = ks % kKStages, sv = vs % kVStages;
                    if (ks >= kKStages) ok = mbar_wait(k_empty + sk, (ks / kKStages - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(k_full + sk, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_4d(smem + L::kK + sk * L::kTile + c * kChunkBytesSw128, &a.k, c * 64, j * kKeyTile, kv, g, k_full + sk);
                    ++ks;
                    if (j == 0) {
                        if (items > 1) ok = mbar_wait(do_empty, (items - 2) & 1, a.status);
                        if (!ok) break;
                        mbar_arrive_expect_tx(do_full, L::kTile);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            tma_load_3d(smem + L::kDO + c * kChunkBytesSw128, &a.dO, c * 64, row, t.head, do_full);
                        ++dos;
                    }
                    if (vs >= kVStages) ok = mbar_wait(v_empty + sv, (vs / kVStages - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(v_full + sv, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_4d(smem + L::kV + sv * L::kTile + c * kChunkBytesSw128, &a.v, c * 64, j * kKeyTile, kv, g, v_full + sv);
                    ++vs;
                }
            }
            // no copy may still be landing in shared memory at exit
            if (items > 0) mbar_wait(q_full, (items - 1) & 1, a.status);
            if (dos > 0) mbar_wait(do_full, (dos - 1) & 1, a.status);
            for (uint32_t f = ks > kKStages ? ks - kKStages : 0; f < ks; ++f)
                mbar_wait(k_full + f % kKStages, (f / kKStages) & 1, a.status);
            for (uint32_t f = vs > kVStages ? vs - kVStages : 0; f < vs; ++f)
                mbar_wait(v_full + f % kVStages, (f / kVStages) & 1, a.status);
        } else if (warp == 1) {
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint64_t d_q = desc_kmajor_sw128(base + L::kQ, 0), d_do = desc_kmajor_sw128(base + L::kDO, 0);
            const uint64_t d_k = desc_kmajor_sw128(base + L::kK, 0), d_v = desc_kmajor_sw128(base + L::kV, 0);
            const uint64_t d_kt = desc_mnmajor_sw128(base + L::kK, 0);
            constexpr uint64_t kTileStep = L::kTile >> 4;
            constexpr uint32_t idesc_dq = idesc_bf16_f32(128, D, 1);
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, a.status));
            };
            auto commit = [&](uint64_t* bar) {
                if (leader) tc_commit(bar);
            };
            auto product = [&](uint32_t col, uint64_t da, uint64_t db, int w) {  // 128 rows x w columns over d
                const uint32_t idesc = idesc_bf16_f32(128, 0, 0) | (static_cast<uint32_t>(w >> 3) << 17);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at = static_cast<uint64_t>((kk >> 2) * (kChunkBytesSw128 >> 4) + (kk & 3) * 2);
                        umma_ss(tmem + col, da + at, db + at, idesc, kk > 0);
                    }
                }
            };
            int64_t i = blockIdx.x;
            DqItem t;
            auto next_item = [&](int64_t from) {
                for (i = from; i < a.items; i += gridDim.x) {
                    t = dq_item(a, i);
                    if (t.n > 0) return true;
                }
                return false;
            };
            auto width = [](const DqItem& it, int j) {
                const int left = it.valid - j * kKeyTile;
                return left >= kKeyTile ? kKeyTile : (left + 15) & ~15;
            };
            uint32_t step = 0, items = 0;  // of the products below: dQ's
            // S of tile j of item `it`, which is step f
            auto issue_s = [&](const DqItem& it, int j, uint32_t f, uint32_t item) {
                const uint32_t st = f % kKStages;
                if (j == 0 && !wait(q_full, item & 1)) return false;
                if (!wait(k_full + st, (f / kKStages) & 1)) return false;
                const int w = width(it, j), left = it.valid - j * kKeyTile;
                if (left < w) clear_rows<D>(smem + L::kK + st * L::kTile, kChunkBytesSw128, left);
                if (f > 0 && !wait(s_read, (f - 1) & 1)) return false;
                tc_fence_after();
                product(kColS, d_q, d_k + st * kTileStep, w);
                commit(s_full);
                if (j == it.n - 1) commit(q_empty);
                return true;
            };
            auto issue_dp = [&](const DqItem& it, int j, uint32_t f, uint32_t item) {
                const uint32_t st = f % kVStages;
                if (j == 0 && !wait(do_full, item & 1)) return false;
                if (!wait(v_full + st, (f / kVStages) & 1)) return false;
                tc_fence_after();
                product(kColP, d_do, d_v + st * kTileStep, width(it, j));
                commit(dp_full);
                commit(v_empty + st);
                if (j == it.n - 1) commit(do_empty);
                return true;
            };
            bool more = next_item(i);
            bool ok = !more || (issue_s(t, 0, 0, 0) && issue_dp(t, 0, 0, 0));
            while (ok && more) {
                const DqItem cur = t;
                const uint32_t item = items;
                for (int j = 0; j < cur.n; ++j, ++step) {
                    DqItem nxt = cur;
                    int nj = j + 1;
                    uint32_t n_item = item;
                    bool has = true;
                    if (nj == cur.n) {
                        has = more = next_item(i + gridDim.x);
                        nxt = t, nj = 0, n_item = item + 1;
                    }
                    if (has && !(ok = issue_s(nxt, nj, step + 1, n_item))) break;
                    if (!(ok = wait(ds_full, step & 1))) break;
                    tc_fence_after();
                    const uint32_t st = step % kKStages;
                    if (leader) {
                        const int steps = width(cur, j) / 16;
                        for (int kk = 0; kk < steps; ++kk)
                            umma_ts(tmem + kColA + 128 * (item & 1), tmem + kColP + packed_col(kk),
                                    d_kt + st * kTileStep + static_cast<uint64_t>(kk * 128), idesc_dq, j > 0 || kk > 0);
                    }
                    commit(k_empty + st);
                    if (j == cur.n - 1) commit(dq_done + (item & 1));
                    if (has && !(ok = issue_dp(nxt, nj, step + 1, n_item))) break;
                }
                ++items;
            }
        } else if (warp == 2 && blockIdx.x == 0) {
            count_pairs(a);
        }
    } else {
        setmaxnreg_inc<kRegsElementwise>();
        const int half = (warp - 4) >> 2;
        const int r = threadIdx.x - 128 - half * 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + 64 * half, t_p = tmem + lanes + kColP + 64 * half;
        float* exchange = reinterpret_cast<float*>(smem + L::kDelta);
        const float c = a.s.scale_log2;
        uint32_t step = 0, items = 0;
        bool ok = true;
        // the item whose dq is still to be stored
        bool pending = false;
        uint16_t* out = nullptr;
        bool out_live = false;
        constexpr int kCols = D / 2;  // dq columns of a thread
        auto store_pending = [&]() {
            const uint32_t item = items - 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(dq_done + (item & 1), (item >> 1) & 1, a.status))) return false;
            tc_fence_after();
            store_row<kCols / 32>(tmem + lanes + kColA + 128 * (item & 1) + half * kCols, out, a.scale, out_live);
            pending = false;
            return true;
        };
        for (int64_t i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const DqItem t = dq_item(a, i);
            if (t.rows <= 0) continue;
            const bool live = r < t.rows;
            const int64_t row = static_cast<int64_t>(t.group) * a.s.group_rows + t.row0 + r;
            uint16_t* to = a.dq + row * a.dq_row + t.head * a.dq_head + half * kCols;
            if (t.n == 0) {
                if (live)
                    for (int u = 0; u < kCols / 8; ++u) reinterpret_cast<uint4*>(to)[u] = make_uint4(0, 0, 0, 0);
                continue;
            }
            // O of half of the channels, on its way while S and P are made
            uint4 o[kCols / 8];
            float lse2 = INFINITY;
            if (live) {
                const uint4* from = reinterpret_cast<const uint4*>(a.O + row * a.O_row + t.head * a.O_head + half * kCols);
#pragma unroll
                for (int u = 0; u < kCols / 8; ++u) o[u] = ld_row(from + u);
                lse2 = a.lse[static_cast<int64_t>(t.head) * a.s.rows + row] * 1.4426950408889634f;
            } else {
#pragma unroll
                for (int u = 0; u < kCols / 8; ++u) o[u] = make_uint4(0, 0, 0, 0);
            }
            float delta = 0.0f;
            for (int j = 0; j < t.n; ++j, ++step) {
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full, step & 1, a.status)))) break;
                tc_fence_after();
                const int left = t.valid - j * kKeyTile - half * 64;  // valid ones of this half's columns
                float p[64];
                {
                    uint32_t s[2][32];
                    BSS_TMEM_LD32(t_s, s[0]);
                    BSS_TMEM_LD32(t_s + 32, s[1]);
                    tmem_wait_ld();
                    tc_fence_before();
                    mbar_arrive(s_read);
                    const uint64_t c2 = f2_pack(c, c), nl2 = f2_pack(-lse2, -lse2);
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        float y0, y1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[x >> 4][2 * (x & 15)]), __uint_as_float(s[x >> 4][2 * (x & 15) + 1])), c2, nl2), y0, y1);
                        p[2 * x] = ex2_approx(y0);
                        p[2 * x + 1] = ex2_approx(y1);
                    }
                }
                if (j == 0) {
                    // D = sum dO O of the row: this half of the channels, then both
                    if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(do_full, items & 1, a.status)))) break;
                    float sum = 0.0f;
                    const uint8_t* from = smem + L::kDO + (D == 128 ? half * kChunkBytesSw128 : 0) + r * 128;
#pragma unroll
                    for (int u = 0; u < kCols / 8; ++u) {
                        const int unit = (D == 128 ? 0 : half * 4) + u;
                        const uint4 g = *reinterpret_cast<const uint4*>(from + ((unit ^ (r & 7)) << 4));
                        sum += dot(unpack_bf16<false>(g), unpack_bf16<false>(o[u]));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(do_empty);
                    float* x = exchange + (items & 1) * 256;
                    x[half * 128 + r] = sum;
                    mbar_arrive(halves);
                    if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(halves, items & 1, a.status)))) break;
                    delta = x[r] + x[128 + r];
                    if (half == 0 && live) a.delta[static_cast<int64_t>(t.head) * a.s.rows + row] = delta;
                }
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(dp_full, step & 1, a.status)))) break;
                tc_fence_after();
                {
                    uint32_t g[2][32];
                    BSS_TMEM_LD32(t_p, g[0]);
                    BSS_TMEM_LD32(t_p + 32, g[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 64; ++x) p[x] *= __uint_as_float(g[x >> 5][x & 31]) - delta;
                    if (left < 64) {
#pragma unroll
                        for (int x = 0; x < 64; ++x)
                            if (x >= left) p[x] = 0.0f;
                    }
                    store_packed(t_p, p);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(ds_full);
                if (j == 0 && pending && !(ok = store_pending())) break;
            }
            if (!ok) break;
            ++items;
            pending = true;
            out = to;
            out_live = live;
        }
        if (ok && pending) store_pending();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- dk, dv
constexpr int kQStages = 3, kDOStages = 2, kAuxStages = 2;

template <int D>
struct DkvSmem {
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kK = 0, kV = kTile, kQ = 2 * kTile, kDO = kQ + kQStages * kTile;
    static constexpr uint32_t kAux = kDO + kDOStages * kTile;  // lse in base 2, delta: float [stage][2][128]
    static constexpr uint32_t kBar = kAux + kAuxStages * 1024;
    // k_full k_empty v_full v_empty q_full q_empty do_full do_empty aux_full aux_empty s_full p_full dp_full ds_full sums
    static constexpr uint32_t kBars = 4 + 2 * kQStages + 2 * kDOStages + 2 * kAuxStages + 5;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 16;
};

// The run of a CTA, key tile by key tile.
struct Part {
    int group, kv, tile, valid;  // the key tile
    int per, row_tiles;          // its row tiles over all heads that share it, and those of one head
    int first, last;             // of this run
    int64_t end;                 // where the run goes on
};

__device__ __forceinline__ int64_t run_begin(const GradArgs& a, int64_t total, int b) {
    const int64_t each = total / a.blocks, rest = total - each * a.blocks;
    return each * b + (b < rest ? b : rest);
}

__device__ __forceinline__ Part part_at(const GradArgs& a, int64_t u, int64_t hi) {
    int lo_g = 0, hi_g = a.s.groups - 1;
    while (lo_g < hi_g) {  // the last group that starts at or in front of u, among those with pairs
        const int mid = (lo_g + hi_g + 1) >> 1;
        if (a.starts[mid] <= u) lo_g = mid;
        else hi_g = mid - 1;
    }
    Part p;
    p.group = lo_g;
    p.valid = a.s.valid(lo_g);
    const int tiles = (p.valid + kKeyTile - 1) / kKeyTile;
    p.row_tiles = (a.s.rows_of(lo_g) + 127) / 128;
    p.per = p.row_tiles * a.s.share;
    const int64_t local = u - a.starts[lo_g], seg = local / p.per;
    p.first = static_cast<int>(local - seg * p.per);
    p.kv = static_cast<int>(seg / tiles);
    p.tile = static_cast<int>(seg - static_cast<int64_t>(p.kv) * tiles);
    const int64_t seg_end = u - p.first + p.per;
    p.end = seg_end < hi ? seg_end : hi;
    p.last = p.first + static_cast<int>(p.end - u);
    return p;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_dkv_kernel(const __grid_constant__ GradArgs a) {
    using L = DkvSmem<D>;
    constexpr int kChunks = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* k_empty = k_full + 1;
    uint64_t* v_full = k_empty + 1;
    uint64_t* v_empty = v_full + 1;
    uint64_t* q_full = v_empty + 1;
    uint64_t* q_empty = q_full + kQStages;
    uint64_t* do_full = q_empty + kQStages;
    uint64_t* do_empty = do_full + kDOStages;
    uint64_t* aux_full = do_empty + kDOStages;
    uint64_t* aux_empty = aux_full + kAuxStages;
    uint64_t* s_full = aux_empty + kAuxStages;
    uint64_t* p_full = s_full + 1;
    uint64_t* dp_full = p_full + 1;
    uint64_t* ds_full = dp_full + 1;
    uint64_t* sums = ds_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sums + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t total = a.starts[a.s.groups];
    const int64_t lo = run_begin(a, total, blockIdx.x), hi = run_begin(a, total, blockIdx.x + 1);
    if (lo >= hi) return;
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles could not be addressed
        record_status(a.status, BSS_ERR_CUDA);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        mbar_init(v_full, 1);
        mbar_init(v_empty, 1);
        for (int i = 0; i < kQStages; ++i) mbar_init(q_full + i, 1), mbar_init(q_empty + i, 1);
        for (int i = 0; i < kDOStages; ++i) mbar_init(do_full + i, 1), mbar_init(do_empty + i, 1);
        for (int i = 0; i < kAuxStages; ++i) mbar_init(aux_full + i, 64), mbar_init(aux_empty + i, kElementwise);
        mbar_init(s_full, 1);
        mbar_init(p_full, kElementwise);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, kElementwise);
        mbar_init(sums, 1);
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // unit x of a part: its head and first row in the group
    auto head_of = [&](const Part& p, int x) { return p.kv * a.s.share + x / p.row_tiles; };
    auto row_of = [&](const Part& p, int x) { return (x % p.row_tiles) * 128; };

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&a.q);
            tma_prefetch_desc(&a.dO);
            tma_prefetch_desc(&a.k);
            tma_prefetch_desc(&a.v);
            uint32_t parts = 0, vs = 0, qs = 0, dos = 0;
            bool ok = true;
            for (int64_t u = lo; ok && u < hi;) {
                const Part p = part_at(a, u, hi);
                const int g = a.s.shared_states ? 0 : p.group;
                if (parts > 0) ok = mbar_wait(k_empty, (parts - 1) & 1, a.status);
                if (!ok) break;
                mbar_arrive_expect_tx(k_full, L::kTile);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    tma_load_4d(smem + L::kK + c * kChunkBytesSw128, &a.k, c * 64, p.tile * kKeyTile, p.kv, g, k_full);
                ++parts;
                for (int x = p.first; x < p.last; ++x) {
                    const uint32_t sq = qs % kQStages, sd = dos % kDOStages;
                    const int row = p.group * a.s.group_rows + row_of(p, x), head = head_of(p, x);
                    if (qs >= kQStages) ok = mbar_wait(q_empty + sq, (qs / kQStages - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(q_full + sq, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(smem + L::kQ + sq * L::kTile + c * kChunkBytesSw128, &a.q, c * 64, row, head, q_full + sq);
                    ++qs;
                    if (x == p.first) {
                        if (parts > 1) ok = mbar_wait(v_empty, (parts - 2) & 1, a.status);
                        if (!ok) break;
                        mbar_arrive_expect_tx(v_full, L::kTile);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            tma_load_4d(smem + L::kV + c * kChunkBytesSw128, &a.v, c * 64, p.tile * kKeyTile, p.kv, g, v_full);
                        ++vs;
                    }
                    if (dos >= kDOStages) ok = mbar_wait(do_empty + sd, (dos / kDOStages - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(do_full + sd, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(smem + L::kDO + sd * L::kTile + c * kChunkBytesSw128, &a.dO, c * 64, row, head, do_full + sd);
                    ++dos;
                }
                u = p.end;
            }
            // no copy may still be landing in shared memory at exit
            if (parts > 0) mbar_wait(k_full, (parts - 1) & 1, a.status);
            if (vs > 0) mbar_wait(v_full, (vs - 1) & 1, a.status);
            for (uint32_t f = qs > kQStages ? qs - kQStages : 0; f < qs; ++f)
                mbar_wait(q_full + f % kQStages, (f / kQStages) & 1, a.status);
            for (uint32_t f = dos > kDOStages ? dos - kDOStages : 0; f < dos; ++f)
                mbar_wait(do_full + f % kDOStages, (f / kDOStages) & 1, a.status);
        } else if (warp == 1) {
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint64_t d_k = desc_kmajor_sw128(base + L::kK, 0), d_v = desc_kmajor_sw128(base + L::kV, 0);
            const uint64_t d_q = desc_kmajor_sw128(base + L::kQ, 0), d_do = desc_kmajor_sw128(base + L::kDO, 0);
            const uint64_t d_qt = desc_mnmajor_sw128(base + L::kQ, 0), d_dot = desc_mnmajor_sw128(base + L::kDO, 0);
            constexpr uint64_t kTileStep = L::kTile >> 4;
            constexpr uint32_t idesc_sum = idesc_bf16_f32(128, D, 1);
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, a.status));
            };
            auto commit = [&](uint64_t* bar) {
                if (leader) tc_commit(bar);
            };
            auto rows_in = [&](const Part& p, int x) {
                const int left = a.s.rows_of(p.group) - row_of(p, x);
                return left < 128 ? left : 128;
            };
            auto product = [&](uint32_t col, uint64_t da, uint64_t db, int w) {
                const uint32_t idesc = idesc_bf16_f32(128, 0, 0) | (static_cast<uint32_t>(w >> 3) << 17);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at = static_cast<uint64_t>((kk >> 2) * (kChunkBytesSw128 >> 4) + (kk & 3) * 2);
                        umma_ss(tmem + col, da + at, db + at, idesc, kk > 0);
                    }
                }
            };
            auto sum_up = [&](uint32_t col, uint32_t from, uint64_t db, int w, bool add) {
                if (leader)
                    for (int kk = 0; kk < w / 16; ++kk)
                        umma_ts(tmem + col, tmem + from + packed_col(kk), db + static_cast<uint64_t>(kk * 128), idesc_sum, add || kk > 0);
            };
            // a cursor over the run's units
            Part p = part_at(a, lo, hi);
            int x = p.first;
            uint32_t part = 0;
            // S, dP and dV of unit f at the cursor
            auto issue_s = [&](uint32_t f) {
                const uint32_t st = f % kQStages;
                if (x == p.first && !wait(k_full, part & 1)) return false;
                if (!wait(q_full + st, (f / kQStages) & 1)) return false;
                const int n = rows_in(p, x);
                if (n & 15) clear_rows<D>(smem + L::kQ + st * L::kTile, kChunkBytesSw128, n);
                tc_fence_after();
                product(kColS, d_k, d_q + st * kTileStep, (n + 15) & ~15);
                commit(s_full);
                if (x == p.last - 1) commit(k_empty);
                return true;
            };
            auto issue_dp = [&](uint32_t f) {
                const uint32_t st = f % kDOStages;
                if (x == p.first && !wait(v_full, part & 1)) return false;
                if (!wait(do_full + st, (f / kDOStages) & 1)) return false;
                const int n = rows_in(p, x);
                if (n & 15) clear_rows<D>(smem + L::kDO + st * L::kTile, kChunkBytesSw128, n);
                tc_fence_after();
                product(kColP, d_v, d_do + st * kTileStep, (n + 15) & ~15);
                commit(dp_full);
                if (x == p.last - 1) commit(v_empty);
                return true;
            };
            auto issue_dv = [&](uint32_t f) {
                const uint32_t st = f % kDOStages;
                if (!wait(p_full, f & 1)) return false;
                tc_fence_after();
                sum_up(kColA, kColS, d_dot + st * kTileStep, (rows_in(p, x) + 15) & ~15, x > p.first);
                commit(do_empty + st);
                return true;
            };
            bool ok = issue_s(0) && issue_dp(0) && issue_dv(0);
            const uint32_t units = static_cast<uint32_t>(hi - lo);
            for (uint32_t f = 0; ok && f < units; ++f) {
                const int w = (rows_in(p, x) + 15) & ~15;
                const bool add = x > p.first, last = x == p.last - 1, more = f + 1 < units;
                if (last) {
                    if (more) {
                        p = part_at(a, p.end, hi);
                        x = p.first;
                        ++part;
                    }
                } else {
                    ++x;
                }
                if (more && !(ok = issue_s(f + 1))) break;
                if (!(ok = wait(ds_full, f & 1))) break;
                tc_fence_after();
                sum_up(kColB, kColP, d_qt + (f % kQStages) * kTileStep, w, add);
                commit(q_empty + f % kQStages);
                if (last) commit(sums);
                if (more && !(ok = issue_dp(f + 1) && issue_dv(f + 1))) break;
            }
        } else if (warp >= 2) {
            // what the rows of a unit bring to their columns
            const int i = static_cast<int>(threadIdx.x) - 64;
            float* aux = reinterpret_cast<float*>(smem + L::kAux);
            uint32_t f = 0;
            bool ok = true;
            for (int64_t u = lo; ok && u < hi;) {
                const Part p = part_at(a, u, hi);
                const int rows = a.s.rows_of(p.group);
                for (int x = p.first; x < p.last; ++x, ++f) {
                    const uint32_t st = f % kAuxStages;
                    const int r = row_of(p, x) + i;
                    const int64_t at = static_cast<int64_t>(head_of(p, x)) * a.s.rows + static_cast<int64_t>(p.group) * a.s.group_rows + r;
                    float v[4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const bool live = r + 64 * y < rows;
                        v[y] = live ? a.lse[at + 64 * y] * 1.4426950408889634f : INFINITY;
                        v[2 + y] = live ? a.delta[at + 64 * y] : 0.0f;
                    }
                    if (f >= kAuxStages) ok = mbar_wait(aux_empty + st, (f / kAuxStages - 1) & 1, a.status);
                    if (!ok) break;
                    aux[st * 256 + i] = -v[0];
                    aux[st * 256 + 64 + i] = -v[1];
                    aux[st * 256 + 128 + i] = -v[2];
                    aux[st * 256 + 192 + i] = -v[3];
                    mbar_arrive(aux_full + st);
                }
                u = p.end;
            }
        }
    } else {
        setmaxnreg_inc<kRegsElementwise>();
        const int half = (warp - 4) >> 2;
        const int r = threadIdx.x - 128 - half * 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + 64 * half, t_p = tmem + lanes + kColP + 64 * half;
        const float* aux = reinterpret_cast<const float*>(smem + L::kAux) + half * 64;
        const float c = a.s.scale_log2;
        const uint64_t c2 = f2_pack(c, c);
        uint32_t f = 0, part = 0;
        bool ok = true;
        for (int64_t u = lo; ok && u < hi; ++part) {
            const Part t = part_at(a, u, hi);
            const int key = t.tile * kKeyTile + r;
            const bool live = key < t.valid;
            for (int x = t.first; x < t.last; ++x, ++f) {
                const uint32_t st = f % kAuxStages;
                float p[64];
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(aux_full + st, (f / kAuxStages) & 1, a.status)))) break;
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full, f & 1, a.status)))) break;
                tc_fence_after();
                {
                    uint32_t s[2][32];
                    BSS_TMEM_LD32(t_s, s[0]);
                    BSS_TMEM_LD32(t_s + 32, s[1]);
                    tmem_wait_ld();
                    const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(aux + st * 256);
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const ulonglong2 l = l2[y];
                        const uint32_t* v = &s[y >> 3][4 * (y & 7)];
                        float y0, y1, y2, y3;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[0]), __uint_as_float(v[1])), c2, l.x), y0, y1);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2]), __uint_as_float(v[3])), c2, l.y), y2, y3);
                        p[4 * y] = ex2_approx(y0);
                        p[4 * y + 1] = ex2_approx(y1);
                        p[4 * y + 2] = ex2_approx(y2);
                        p[4 * y + 3] = ex2_approx(y3);
                    }
#pragma unroll
                    for (int y = 0; y < 64; ++y) p[y] = live ? p[y] : 0.0f;
                    store_packed(t_s, p);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full);
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(dp_full, f & 1, a.status)))) break;
                tc_fence_after();
                {
                    uint32_t g[2][32];
                    BSS_TMEM_LD32(t_p, g[0]);
                    BSS_TMEM_LD32(t_p + 32, g[1]);
                    tmem_wait_ld();
                    const ulonglong2* d2 = reinterpret_cast<const ulonglong2*>(aux + st * 256 + 128);
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const ulonglong2 d = d2[y];
                        const uint32_t* v = &g[y >> 3][4 * (y & 7)];
                        float y0, y1, y2, y3;
                        f2_unpack(f2_add(f2_pack(__uint_as_float(v[0]), __uint_as_float(v[1])), d.x), y0, y1);
                        f2_unpack(f2_add(f2_pack(__uint_as_float(v[2]), __uint_as_float(v[3])), d.y), y2, y3);
                        p[4 * y] *= y0;
                        p[4 * y + 1] *= y1;
                        p[4 * y + 2] *= y2;
                        p[4 * y + 3] *= y3;
                    }
                    // a masked state's values may be anything
#pragma unroll
                    for (int y = 0; y < 64; ++y) p[y] = live ? p[y] : 0.0f;
                    store_packed(t_p, p);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(ds_full);
                mbar_arrive(aux_empty + st);
            }
            if (!ok) break;
            // the key tile's sums: half 0 has dv, half 1 dk
            if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(sums, part & 1, a.status)))) break;
            tc_fence_after();
            const uint32_t acc = tmem + lanes + (half == 0 ? kColA : kColB);
            if (t.first == 0 && t.last == t.per) {
                uint16_t* to = half == 0 ? a.dv + t.group * a.dv_group + key * a.dv_token + t.kv * a.dv_head
                                         : a.dk + t.group * a.dk_group + key * a.dk_token + t.kv * a.dk_head;
                store_row<D / 32>(acc, to, half == 0 ? 1.0f : a.scale, key < a.s.keys);
            } else {
                const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (t.first > 0 ? 0 : 1);
                float* to = a.parts + ((slot * 2 + half) * 128 + r) * D;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    BSS_TMEM_LD32(acc + cc * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        reinterpret_cast<uint4*>(to + cc * 32)[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
            }
            tc_fence_before();
            u = t.end;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- sums of parts, zeros
// Block (b, y): the key tile in which run b ends, if it also begins there: the parts
// of runs b, b + 1, ... in their order.  Key tiles without a valid state: zeros.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ GradArgs a) {
    const int64_t total = a.starts[a.s.groups];
    const int b = blockIdx.x;
    const int64_t lo = run_begin(a, total, b), hi = run_begin(a, total, b + 1);
    if (lo < hi) {
        // the part that ends the run
        Part p = part_at(a, hi - 1, hi);
        const int64_t seg = hi - 1 - p.first;  // where its key tile begins
        if (seg >= lo && seg + p.per > hi) {
            int ends = b + 1;  // the run that holds the key tile's end
            while (run_begin(a, total, ends + 1) < seg + p.per) ++ends;
            constexpr int kVectors = 2 * 128 * D / 8;
            for (int i = blockIdx.y * 256 + threadIdx.x; i < kVectors; i += gridDim.y * 256) {
                float v[8], w[8];
                auto fetch = [&](int64_t slot, float (&to)[8]) {
                    const float4* from = reinterpret_cast<const float4*>(a.parts + slot * 2 * 128 * D) + 2 * i;
                    const float4 x = from[0], y = from[1];
                    to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w, to[4] = y.x, to[5] = y.y, to[6] = y.z, to[7] = y.w;
                };
                fetch(2 * static_cast<int64_t>(b) + 1, v);
                for (int run = b + 1; run <= ends; ++run) {
                    fetch(2 * static_cast<int64_t>(run), w);
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] += w[x];
                }
                const int which = i / (128 * D / 8), r = i / (D / 8) % 128, c = i % (D / 8) * 8;
                const int key = p.tile * kKeyTile + r;
                if (key >= a.s.keys) continue;
                uint16_t* to = which == 0 ? a.dv + p.group * a.dv_group + key * a.dv_token + p.kv * a.dv_head
                                          : a.dk + p.group * a.dk_group + key * a.dk_token + p.kv * a.dk_head;
                const float scale = which == 0 ? 1.0f : a.scale;
                *reinterpret_cast<uint4*>(to + c) = make_uint4(pack2(v[0] * scale, v[1] * scale), pack2(v[2] * scale, v[3] * scale),
                                                               pack2(v[4] * scale, v[5] * scale), pack2(v[6] * scale, v[7] * scale));
            }
        }
    }
    if (a.s.lengths == nullptr) return;
    const int64_t tiles = static_cast<int64_t>(a.s.groups) * a.key_tiles * a.s.kv_heads;
    for (int64_t i = blockIdx.x + static_cast<int64_t>(blockIdx.y) * gridDim.x; i < tiles; i += static_cast<int64_t>(gridDim.x) * gridDim.y) {
        const int64_t rest = i / a.s.kv_heads;
        const int kv = static_cast<int>(i - rest * a.s.kv_heads);
        const int g = static_cast<int>(rest / a.key_tiles), first = static_cast<int>(rest - static_cast<int64_t>(g) * a.key_tiles) * kKeyTile;
        if (first < a.s.valid(g)) continue;
        for (int e = threadIdx.x; e < 2 * 128 * D / 8; e += 256) {
            const int which = e / (128 * D / 8), key = first + e / (D / 8) % 128, c = e % (D / 8) * 8;
            if (key >= a.s.keys) continue;
            uint16_t* to = which == 0 ? a.dv + g * a.dv_group + key * a.dv_token + kv * a.dv_head
                                      : a.dk + g * a.dk_group + key * a.dk_token + kv * a.dk_head;
            *reinterpret_cast<uint4*>(to + c) = make_uint4(0, 0, 0, 0);
        }
    }
}

template <int D>
bss_status launch_backward(GradArgs& a, cudaStream_t stream) {
    auto dq = cross_dq_kernel<D>;
    auto dkv = cross_dkv_kernel<D>;
    int blocks;
    bss_status st = resident_blocks(reinterpret_cast<const void*>(dq), kThreads, DqSmem<D>::kBytes, &blocks);
    if (st == BSS_OK) st = resident_blocks(reinterpret_cast<const void*>(dkv), kThreads, DkvSmem<D>::kBytes, &blocks);
    if (st != BSS_OK) return st;
    const int64_t grid = a.items < num_sms() ? a.items : num_sms();
    dq<<<static_cast<unsigned>(grid), kThreads, DqSmem<D>::kBytes, stream>>>(a);
    if ((st = cuda_check(cudaGetLastError(), "query gradient launch")) != BSS_OK) return st;
    dkv<<<static_cast<unsigned>(a.blocks), kThreads, DkvSmem<D>::kBytes, stream>>>(a);
    if ((st = cuda_check(cudaGetLastError(), "key gradient launch")) != BSS_OK) return st;
    cross_join_kernel<D><<<dim3(static_cast<unsigned>(a.blocks), 8), 256, 0, stream>>>(a);
    return cuda_check(cudaGetLastError(), "key gradient sums launch");
}

int64_t aligned_up(int64_t v) { return (v + 255) / 256 * 256; }

struct Plan {
    int64_t delta_at, starts_at, parts_at, bytes;
    int32_t tiles, key_tiles, blocks;
};

// rows_per_group at most rows
Plan plan_of(const bss_cross_grads& a) {
    Plan p;
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    p.tiles = static_cast<int32_t>((a.rows_per_group + 127) / 128);
    p.key_tiles = static_cast<int32_t>((static_cast<int64_t>(a.keys) + kKeyTile - 1) / kKeyTile);
    const double pairs = static_cast<double>(groups) * p.tiles * p.key_tiles * a.heads;
    p.blocks = pairs < num_sms() ? static_cast<int32_t>(pairs) : num_sms();
    p.delta_at = 0;
    p.starts_at = aligned_up(a.rows * a.heads * 4);
    p.parts_at = p.starts_at + aligned_up((groups + 1) * 8);
    p.bytes = p.parts_at + 2ll * p.blocks * 2 * 128 * a.head_dim * 4;
    return p;
}

bss_status check_grads(bss_cross_grads& a) {
    const bss_status st = check_cross_sizes(a.rows, &a.rows_per_group, a.heads, a.kv_heads, a.head_dim, a.keys, a.softmax_scale, a.lengths);
    if (st != BSS_OK) return st;
    if (a.lse == nullptr) return set_error(BSS_ERR_INVALID_ARG, "lse is NULL");
    return BSS_OK;
}

}  // namespace
}  // namespace bss

extern "C" {

bss_status bss_cross_attention_backward_workspace(const bss_cross_grads* args, int64_t* bytes) {
    using namespace bss;
    clear_error();
    if (bytes == nullptr) return set_error(BSS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_cross_grads a = *args;
    const bss_status st = check_grads(a);
    if (st != BSS_OK) return st;
    *bytes = plan_of(a).bytes;
    return BSS_OK;
}

bss_status bss_cross_attention_backward(const bss_cross_grads* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_cross_grads p = *args;
    bss_status st = check_grads(p);
    if (st != BSS_OK) return st;
    const Plan plan = plan_of(p);
    const int64_t groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
    Operand t[11];
    if ((st = check_row_heads(&t[0], p.dO, "dO", p.rows, p.heads, p.head_dim, false)) != BSS_OK ||
        (st = check_row_heads(&t[1], p.q, "q", p.rows, p.heads, p.head_dim, false)) != BSS_OK ||
        (st = check_row_heads(&t[2], p.O, "O", p.rows, p.heads, p.head_dim, false)) != BSS_OK ||
        (st = check_states(&t[3], p.k, "k", groups, p.keys, p.kv_heads, p.head_dim, false)) != BSS_OK ||
        (st = check_states(&t[4], p.v, "v", groups, p.keys, p.kv_heads, p.head_dim, false)) != BSS_OK ||
        (st = check_run(&t[5], p.lengths, "lengths", 4 * groups, 4, false)) != BSS_OK ||
        (st = check_run(&t[6], p.lse, "lse", 4 * p.rows * p.heads, 4, false)) != BSS_OK ||
        (st = check_row_heads(&t[7], p.dq, "dq", p.rows, p.heads, p.head_dim, true)) != BSS_OK ||
        (st = check_states(&t[8], p.dk, "dk", groups, p.keys, p.kv_heads, p.head_dim, true)) != BSS_OK ||
        (st = check_states(&t[9], p.dv, "dv", groups, p.keys, p.kv_heads, p.head_dim, true)) != BSS_OK ||
        (st = check_run(&t[10], p.workspace, "workspace", plan.bytes, 16, true)) != BSS_OK ||
        (st = check_workspace(p.workspace, p.workspace_bytes, plan.bytes)) != BSS_OK ||
        (st = check_outputs(t, 11)) != BSS_OK)
        return st;
    if (groups > 1 && (p.k.group_stride == 0 || p.v.group_stride == 0))
        return set_error(BSS_ERR_UNSUPPORTED, "gradients of states shared by several groups: give one group");
    GradArgs a;
    memset(&a, 0, sizeof(a));
    if ((st = row_heads_map(&a.q, p.q, p.rows, p.heads, p.head_dim, kHalfRows)) != BSS_OK ||
        (st = row_heads_map(&a.dO, p.dO, p.rows, p.heads, p.head_dim, kHalfRows)) != BSS_OK ||
        (st = states_map(&a.k, p.k, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK ||
        (st = states_map(&a.v, p.v, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK)
        return st;
    a.s = cross_shape(p.rows, p.rows_per_group, p.heads, p.kv_heads, p.head_dim, p.keys, p.softmax_scale, p.lengths,
                      p.k.group_stride);
    a.tiles = plan.tiles, a.key_tiles = plan.key_tiles, a.blocks = plan.blocks;
    a.items = groups * plan.tiles * p.heads;
    a.O = static_cast<const uint16_t*>(p.O.data);
    a.dq = static_cast<uint16_t*>(p.dq.data);
    a.dk = static_cast<uint16_t*>(p.dk.data);
    a.dv = static_cast<uint16_t*>(p.dv.data);
    auto stride = [](int64_t extent, int64_t s) { return extent > 1 ? s : 0; };
    a.O_row = stride(p.rows, p.O.token_stride), a.O_head = stride(p.heads, p.O.head_stride);
    a.dq_row = stride(p.rows, p.dq.token_stride), a.dq_head = stride(p.heads, p.dq.head_stride);
    a.dk_group = stride(groups, p.dk.group_stride), a.dk_token = stride(p.keys, p.dk.token_stride);
    a.dk_head = stride(p.kv_heads, p.dk.head_stride);
    a.dv_group = stride(groups, p.dv.group_stride), a.dv_token = stride(p.keys, p.dv.token_stride);
    a.dv_head = stride(p.kv_heads, p.dv.head_stride);
    a.scale = p.softmax_scale > 0.0f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim));
    a.lse = p.lse;
    char* ws = static_cast<char*>(p.workspace);
    a.delta = reinterpret_cast<float*>(ws + plan.delta_at);
    a.starts = reinterpret_cast<int64_t*>(ws + plan.starts_at);
    a.parts = reinterpret_cast<float*>(ws + plan.parts_at);
    a.status = device_status_ptr();
    if (a.status == nullptr) return set_error(BSS_ERR_CUDA, "cannot resolve the device status word");
    return p.head_dim == 128 ? launch_backward<128>(a, stream) : launch_backward<64>(a, stream);
}

}  // extern "C"
