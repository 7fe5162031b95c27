// bss_cross_grad.cu -- gradients of the cross attention.
//
//   P = exp(scale q k^T - lse),  D = sum dO O,  dS = P (dO v^T - D)
//   dq = scale dS k,  dv = P^T dO,  dk = scale dS^T q
//
// Two kernels, each with its own P and dS (7 products of rows x keys x d where 5
// would do): one has the rows in TMEM's lanes and sums dq over the keys, the other
// the keys and sums dk and dv over the rows.  One kernel would have to bring dq's sums
// over the key tiles together: in memory by atomics, whose order changes results, or by a
// pass of their own; or, for a few key tiles, in the shared memory of a cluster that holds
// one a CTA, in a fixed order, which has not been built.
//
// dq: a CTA takes items of (group, 128 rows, head); per key tile the products
// S(t+1), dP(t+1), dQ(t) follow one another (two dP in TMEM), so that the P and dS of a
// tile are made beneath the products of its neighbours.  D is made here, once an item,
// and kept for the second kernel.
//
// dk, dv: the row tiles of all key heads lie in a line that is cut into equal runs, one
// a team of CTAs; each CTA of a team has a key tile of its own, so that the team reads
// a row tile about once from memory (single CTAs cutting the line of all pairs of
// tiles read 1.58 GB for 75,600 x 10 x 128 over 512 states instead of 0.4).  A tile's
// products are S(t+1), dK(t), dP(t+1), dV(t+1).  Where a run ends inside a head's rows
// the sums go to the workspace in 32 bits, and a third kernel adds them in their order.
// With a few rows neither: one kernel without tiles, in 32 bits.
//
// P and dS are rounded to bf16 on the way to their products (the tensor cores take both
// operands in one type), dS once more beside the result's own rounding: errors are 1.4
// times those of a gradient in 32 bits that is rounded at its store.
//
// 75,600 x 10 x 128 over 512 states: 538 us (920 TFLOP/s of five products, 1,290 of the seven
// made): dq 251, dk and dv 257, their sums 14 (one by one).  Both are bound by shared memory: dq moves
// 240 KB a step (1,920 cycles at 128 bytes) beneath 1,536 cycles of products, dk and dv 256
// KB and the rows' statistics (over 2,048 cycles) beneath 2,048.
#include "bss_cross.cuh"

#include <cstring>
#include <type_traits>

namespace bss {
namespace {

constexpr int kThreads = 384;
constexpr int kElementwise = 256;  // threads 128 .. 383: a lane of TMEM and half of the columns
// Registers of the second kernel: 128 x 120 + 256 x 184 = 62,464 of the launch's 384 x 168 = 64,512.
constexpr uint32_t kRegsControl = 120, kRegsElementwise = 184;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColA = 256, kColB = 384;  // S, dP, two sums (or a second dP and one)

struct GradArgs {
    CUtensorMap q, dO, k, v;
    CrossShape s;
    int32_t tiles;      // of 128 rows in a group
    int32_t key_tiles;  // of 128 keys in a group
    int32_t items;      // of the first kernel
    int32_t blocks;     // of the second
    FastDiv by_tiles;
    const uint16_t* O;
    uint16_t *dq, *dk, *dv;
    int64_t O_row, O_head, dq_row, dq_head;
    int64_t dk_group, dk_token, dk_head, dv_group, dv_token, dv_head;
    float scale;
    const float* lse;  // [heads][rows]
    float* delta;      // [heads][rows]
    int64_t* starts;   // [groups + 1]: row tiles of all key heads in front of a group; [groups + 1]: most key tiles
    float* parts;      // [2 blocks][2][128][d]
    int4* joins;       // [blocks]: group (or -1), key head, key tile and further parts of what a CTA leaves to be joined
    int* status;
};

// where half of a thread's columns lies, and 16 columns of an operand in TMEM: each
// half of the columns keeps its bf16 values at the start of its own 64
__device__ __forceinline__ uint32_t packed_col(int kk) { return static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8); }

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// A row's lse in base 2.  Without a score above minus infinity its P is 0: an lse of plus
// infinity makes it so.
__device__ __forceinline__ float lse_base2(float lse) { return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f; }

__device__ __forceinline__ void store_packed(uint32_t at, const float (&v)[64]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = pack_bf16x2(v[32 * q + 2 * x], v[32 * q + 2 * x + 1]);
        BSS_TMEM_ST16(at + 16 * q, w);
    }
}

// ---------------------------------------------------------------- dq
// d[g][n] += sum over 16 channels of a[g][c] b[n][c] for 8 rows each: lane 4 g + i gets
// n = 2 i and 2 i + 1.
__device__ __forceinline__ void add_rows_product(float (&d)[2], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
    float unused0 = 0.0f, unused1 = 0.0f;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(unused0), "+f"(unused1)
                 : "r"(a0), "r"(0u), "r"(a1), "r"(b0), "r"(b1));
}

// Threads: 4 warps of control (loads, products), 4 that make D, 8 elementwise.
// Registers: 128 x (88 + 152 + 2 x 136) = the launch's 512 x 128.
constexpr int kDqThreads = 512, kAuxThreads = 128;
constexpr uint32_t kDqRegsControl = 88, kDqRegsAux = 152, kDqRegsElementwise = 136;
constexpr int kKStages = 3, kVStages = 2;

template <int D>
struct DqSmem {
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kQ = 0, kDO = kTile, kK = 2 * kTile, kV = kK + kKStages * kTile;
    static constexpr uint32_t kAux = kV + kVStages * kTile;  // D, lse in base 2: float [item & 1][2][128]
    static constexpr uint32_t kBar = kAux + 2048;
    // q_full q_empty do_full do_empty k_full k_empty v_full v_empty s_full s_read dp_full[2] ds_full[2] dq_done
    // dq_read aux_full[2] aux_empty[2] cleared
    static constexpr uint32_t kBars = 4 + 2 * kKStages + 2 * kVStages + 13;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 16;
};

struct DqItem {
    int group, row0, rows, head, valid, n;
};

__device__ __forceinline__ DqItem dq_item(const GradArgs& a, int i) {
    DqItem t;
    const int rest = a.s.by_heads.div(i);
    t.head = i - rest * a.s.heads;
    t.group = a.by_tiles.div(rest);
    t.row0 = (rest - t.group * a.tiles) * 128;
    t.rows = a.s.rows_of(t.group) - t.row0;
    t.valid = t.rows > 0 ? a.s.valid(t.group) : 0;
    t.n = (t.valid + kKeyTile - 1) / kKeyTile;
    return t;
}

// starts[], by one warp
__device__ __forceinline__ void count_rows(const GradArgs& a) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    int most = 0;
    for (int g0 = 0; g0 < a.s.groups; g0 += 32) {
        const int g = g0 + lane;
        int64_t n = 0;
        if (g < a.s.groups) {
            const int tiles = (a.s.valid(g) + kKeyTile - 1) / kKeyTile;
            n = tiles > 0 ? static_cast<int64_t>((a.s.rows_of(g) + 127) / 128) * a.s.heads : 0;
            most = tiles > most ? tiles : most;
        }
        int64_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (g < a.s.groups) a.starts[g] = before + sum - n;
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
        a.starts[a.s.groups] = before;
        a.starts[a.s.groups + 1] = most;
    }
}

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1) cross_dq_kernel(const __grid_constant__ GradArgs a) {
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
    uint64_t* ds_full = dp_full + 2;
    uint64_t* dq_done = ds_full + 2;
    uint64_t* dq_read = dq_done + 1;
    uint64_t* aux_full = dq_read + 1;
    uint64_t* aux_empty = aux_full + 2;
    uint64_t* cleared = aux_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cleared + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles could not be addressed
        record_status(a.status, BSS_ERR_CUDA);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1 + kAuxThreads / 32);
        for (int i = 0; i < kKStages; ++i) mbar_init(k_full + i, 1), mbar_init(k_empty + i, 1);
        for (int i = 0; i < kVStages; ++i) mbar_init(v_full + i, 1), mbar_init(v_empty + i, 1);
        mbar_init(cleared, 32);
        mbar_init(s_full, 1);
        mbar_init(s_read, kElementwise);
        mbar_init(dp_full, 1);
        mbar_init(dp_full + 1, 1);
        mbar_init(ds_full, kElementwise);
        mbar_init(ds_full + 1, kElementwise);
        mbar_init(dq_done, 1);
        mbar_init(dq_read, kAuxThreads);
        for (int i = 0; i < 2; ++i) mbar_init(aux_full + i, kAuxThreads), mbar_init(aux_empty + i, kElementwise);
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    cudaGridDependencySynchronize();

    if (warp < 4) {
        setmaxnreg_dec<kDqRegsControl>();
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&a.q);
            tma_prefetch_desc(&a.dO);
            tma_prefetch_desc(&a.k);
            tma_prefetch_desc(&a.v);
            uint32_t items = 0, dos = 0, ks = 0, vs = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
                const DqItem t = dq_item(a, i);
                if (t.n == 0) continue;
                const int row = t.group * a.s.group_rows + t.row0;
                const int kv = a.s.by_share.div(t.head), g = a.s.shared_states ? 0 : t.group;
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
            const uint32_t d_q = desc_lo_kmajor(base + L::kQ), d_do = desc_lo_kmajor(base + L::kDO);
            const uint32_t d_k = desc_lo_kmajor(base + L::kK), d_v = desc_lo_kmajor(base + L::kV);
            const uint32_t d_kt = desc_lo_mnmajor(base + L::kK);
            constexpr uint32_t kTileStep = L::kTile >> 4;
            constexpr uint32_t idesc_dq = idesc_bf16_f32(128, D, 1);
            // (no vote: only the leader's MMAs and commits count)
            auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, a.status); };
            auto commit = [&](uint64_t* bar) {
                if (leader) tc_commit(bar);
            };
            auto product = [&](uint32_t col, uint32_t da, uint32_t db, int w) {  // 128 rows x w columns over d
                const uint32_t idesc = idesc_bf16_f32(128, 0, 0) | (static_cast<uint32_t>(w >> 3) << 17);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (kk >> 2) * (kChunkBytesSw128 >> 4) + (kk & 3) * 2;
                        umma_ss(tmem + col, desc_of(da + at), desc_of(db + at), idesc, kk > 0);
                    }
                }
            };
            int i = blockIdx.x;
            auto next_item = [&](DqItem& t) {  // the next one with keys, from i on
                for (; i < a.items; i += gridDim.x) {
                    t = dq_item(a, i);
                    if (t.n > 0) {
                        i += gridDim.x;
                        return true;
                    }
                }
                return false;
            };
            auto width = [](const DqItem& it, int j) {
                const int left = it.valid - j * kKeyTile;
                return left >= kKeyTile ? kKeyTile : (left + 15) & ~15;
            };
            uint32_t clears = 0;
            // S of tile j of an item, which is step f
            auto issue_s = [&](const DqItem& it, int j, uint32_t f, uint32_t item) {
                const uint32_t st = f % kKStages;
                if (j == 0 && !wait(q_full, item & 1)) return false;
                if (!wait(k_full + st, (f / kKStages) & 1)) return false;
                const int w = width(it, j), left = it.valid - j * kKeyTile;
                if (left < w && it.valid < a.s.keys && !clear_rows<D>(smem + L::kK + st * L::kTile, left, cleared, clears, a.status)) return false;
                if (f > 0 && !wait(s_read, (f - 1) & 1)) return false;
                tc_fence_after();
                product(kColS, d_q, d_k + st * kTileStep, w);
                commit(s_full);
                if (j == it.n - 1) commit(q_empty);
                return true;
            };
            // dP into the buffer that dQ(f - 2), issued before, has read
            auto issue_dp = [&](const DqItem& it, int j, uint32_t f, uint32_t item) {
                const uint32_t st = f % kVStages;
                if (j == 0 && !wait(do_full, item & 1)) return false;
                if (!wait(v_full + st, (f / kVStages) & 1)) return false;
                tc_fence_after();
                product(kColP + 128 * (f & 1), d_do, d_v + st * kTileStep, width(it, j));
                commit(dp_full + (f & 1));
                commit(v_empty + st);
                if (j == it.n - 1) commit(do_empty);
                return true;
            };
            DqItem cur, nxt;
            uint32_t step = 0, item = 0;
            bool more = next_item(cur);
            bool ok = !more || (issue_s(cur, 0, 0, 0) && issue_dp(cur, 0, 0, 0));
            while (ok && more) {
                more = next_item(nxt);
                for (int j = 0; j < cur.n; ++j, ++step) {
                    const bool last = j == cur.n - 1;
                    if (!last) {
                        if (!(ok = issue_s(cur, j + 1, step + 1, item) && issue_dp(cur, j + 1, step + 1, item))) break;
                    } else if (more) {
                        if (!(ok = issue_s(nxt, 0, step + 1, item + 1) && issue_dp(nxt, 0, step + 1, item + 1))) break;
                    }
                    if (!(ok = wait(ds_full + (step & 1), (step >> 1) & 1))) break;
                    if (j == 0 && item > 0 && !(ok = wait(dq_read, (item - 1) & 1))) break;  // the sums of the item before
                    tc_fence_after();
                    const uint32_t st = step % kKStages;
                    const int w = width(cur, j);
                    const uint32_t from = tmem + kColP + 128 * (step & 1), db = d_kt + st * kTileStep;
                    if (w == kKeyTile) {  // unrolled: 38 cycles a product of 16 keys instead of 110
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_ts(tmem + kColB, from + packed_col(kk), desc_of(db + kk * 128), idesc_dq, j > 0 || kk > 0);
                        }
                    } else if (leader) {
                        for (int kk = 0; kk < w / 16; ++kk)
                            umma_ts(tmem + kColB, from + packed_col(kk), desc_of(db + kk * 128), idesc_dq, j > 0 || kk > 0);
                    }
                    commit(k_empty + st);
                    if (last) commit(dq_done);
                }
                cur = nxt;
                ++item;
            }
        } else if (warp == 2 && blockIdx.x == 0) {
            count_rows(a);
        }
    } else if (warp < 8) {
        setmaxnreg_inc<kDqRegsAux>();
        {
            // D = sum dO O of an item's rows, and the sums of dq to memory.  dO is in shared
            // memory; O and lse come from memory an item ahead, into registers.  (Both from
            // memory: beside 224 KiB of shared memory the loads in flight have little room in
            // L1, and 64 KiB an item took 7,500 cycles, more than a tile's products.)  8 rows'
            // sums are the diagonal of a small matrix product: lane 4 g + c has 8 channels of
            // every 32 of row g, the same ones for both operands.
            constexpr int kParts = D / 32;  // 16-byte units of a lane and row
            float* aux = reinterpret_cast<float*>(smem + L::kAux);
            const int w = warp - 4, g = lane >> 2;  // 32 rows a warp
            uint32_t items = 0;
            bool ok = true;
            auto first_row = [&](const DqItem& t) { return static_cast<int64_t>(t.group) * a.s.group_rows + t.row0 + w * 32; };
            int i = blockIdx.x;
            auto next_item = [&](DqItem& t) {  // the next one with keys; the rows of those without get zeros
                for (; i < a.items; i += gridDim.x) {
                    t = dq_item(a, i);
                    if (t.n > 0) {
                        i += gridDim.x;
                        return true;
                    }
                    uint16_t* to = a.dq + first_row(t) * a.dq_row + t.head * a.dq_head;
                    for (int e = lane; e < 32 * (D / 8); e += 32)
                        if (w * 32 + e / (D / 8) < t.rows)
                            *reinterpret_cast<uint4*>(to + e / (D / 8) * a.dq_row + e % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
                }
                return false;
            };
            uint4 o[4][kParts];
            float lse = 0.0f;
            auto fetch = [&](const DqItem& t) {
                const int64_t row0 = first_row(t);
                const int rows = t.rows - w * 32;  // of this warp's 32; rows that do not exist: another one in their place
                const uint16_t* o0 = a.O + t.head * a.O_head + (lane & 3) * 8;
                lse = lane < rows ? lse_base2(a.lse[static_cast<int64_t>(t.head) * a.s.rows + row0 + lane]) : INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t r = rows > 0 ? row0 + min(8 * k + g, rows - 1) : row0 - w * 32;
#pragma unroll
                    for (int c = 0; c < kParts; ++c) o[k][c] = ld_row(o0 + r * a.O_row + 32 * c);
                }
            };
            auto store_last = [&](const DqItem& t) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(dq_done, (items - 1) & 1, a.status))) return false;
                tc_fence_after();
                // out of TMEM at once: the next item's first sums wait for it
                uint4 u[D / 8];
                read_rows<D>(u, tmem + (static_cast<uint32_t>(w * 32) << 16) + kColB, a.scale);
                tc_fence_before();
                mbar_arrive(dq_read);
                write_rows<D / 8>(u, a.dq + first_row(t) * a.dq_row + t.head * a.dq_head, a.dq_row, t.rows - w * 32);
                return true;
            };
            DqItem t, nxt, last;
            bool more = next_item(t);
            if (more) fetch(t);
            while (ok && more) {
                const uint32_t buf = items & 1;
                if (items >= 2 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(aux_empty + buf, (items / 2 - 1) & 1, a.status)))) break;
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(do_full, items & 1, a.status)))) break;
                float* x = aux + buf * 256 + w * 32;
                float* delta = a.delta + static_cast<int64_t>(t.head) * a.s.rows + first_row(t);
                float d[4][2] = {};
#pragma unroll
                for (int c = 0; c < kParts; ++c) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 8 * k + g, unit = 4 * c + (lane & 3);
                        const uint4 u = *reinterpret_cast<const uint4*>(smem + L::kDO + (unit >> 3) * kChunkBytesSw128 + (w * 32 + r) * 128 +
                                                                        (((unit & 7) ^ (r & 7)) << 4));
                        add_rows_product(d[k], u.x, u.y, o[k][c].x, o[k][c].y);
                        add_rows_product(d[k], u.z, u.w, o[k][c].z, o[k][c].w);
                    }
                }
                if ((lane & 3) == (g >> 1)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 8 * k + g;
                        const float sum = g & 1 ? d[k][1] : d[k][0];
                        x[r] = sum;
                        if (w * 32 + r < t.rows) delta[r] = sum;
                    }
                }
                x[128 + lane] = lse;
                mbar_arrive(aux_full + buf);
                __syncwarp();
                if (lane == 0) mbar_arrive(do_empty);
                if (items > 0 && !(ok = store_last(last))) break;
                more = next_item(nxt);
                if (more) fetch(nxt);
                ++items;
                last = t;
                t = nxt;
            }
            if (ok && items > 0) store_last(last);
        }
    } else {
        setmaxnreg_inc<kDqRegsElementwise>();
        const int half = (warp - 8) >> 2;
        const int r = threadIdx.x - 256 - half * 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + 64 * half, t_p = tmem + lanes + kColP + 64 * half;
        const float* aux = reinterpret_cast<const float*>(smem + L::kAux);
        const float c = a.s.scale_log2;
        uint32_t step = 0, items = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const DqItem t = dq_item(a, i);
            if (t.n == 0) continue;
            const float* x = aux + (items & 1) * 256 + r;
            if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(aux_full + (items & 1), (items >> 1) & 1, a.status)))) break;
            const float lse2 = x[128];
            const uint64_t nd2 = f2_pack(-x[0], -x[0]);
            mbar_arrive(aux_empty + (items & 1));
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
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(dp_full + (step & 1), (step >> 1) & 1, a.status)))) break;
                tc_fence_after();
                {
                    const uint32_t at = t_p + 128 * (step & 1);
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t g[32];
                        BSS_TMEM_LD32(at + 32 * cc, g);
                        tmem_wait_ld();
                        float* v = p + 32 * cc;
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            f2_unpack(f2_mul(f2_pack(v[2 * x], v[2 * x + 1]),
                                             f2_add(f2_pack(__uint_as_float(g[2 * x]), __uint_as_float(g[2 * x + 1])), nd2)),
                                      v[2 * x], v[2 * x + 1]);
                        if (left < 64) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (32 * cc + x >= left) v[x] = 0.0f;
                        }
                        uint32_t w[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) w[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
                        BSS_TMEM_ST16(at + 16 * cc, w);  // columns that are read already
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                // (two barriers: the next tile's dS may be there before this one's is taken)
                mbar_arrive(ds_full + (step & 1));
            }
            ++items;
        }
    }

    tc_fence_before();
    __syncwarp();
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
    // cleared
    static constexpr uint32_t kBars = 4 + 2 * kQStages + 2 * kDOStages + 2 * kAuxStages + 6;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 16;
};

// A CTA's share: a run of the line of row tiles, for one key tile (or, with more of
// them than CTAs, every so many).  Part: the run's piece of a key head's rows.
struct Part {
    int group, kv, tile, valid, rows;  // the key tile; rows of the group
    int per;                           // row tiles of the head, over all heads that share it
    int first, last;                   // of this piece
    int64_t end;                       // where the run goes on
};

struct Share {
    int64_t lo, hi, at;
    int tile, step, tiles;  // this CTA's key tiles: tile, tile + step, ... below tiles
};

__device__ __forceinline__ int64_t run_begin(int64_t total, int teams, int team) {
    const int64_t each = total / teams, rest = total - each * teams;
    return each * team + (team < rest ? team : rest);
}

// Teams of CTAs: one a key tile each; at most as many as there are row tiles.
__device__ __forceinline__ int teams_of(const GradArgs& a, int64_t total, int tiles) {
    const int64_t teams = tiles > 0 && tiles <= a.blocks ? a.blocks / tiles : 1;
    return static_cast<int>(teams < total ? teams : (total > 0 ? total : 1));
}

__device__ __forceinline__ Share share_of(const GradArgs& a, int block) {
    const int64_t total = a.starts[a.s.groups];
    Share s;
    s.tiles = static_cast<int>(a.starts[a.s.groups + 1]);
    const int teams = teams_of(a, total, s.tiles);
    s.step = s.tiles <= a.blocks ? s.tiles : a.blocks;
    const int team = s.step > 0 ? block / s.step : teams;
    s.tile = team < teams ? block - team * s.step : s.tiles;
    if (team < teams) s.lo = run_begin(total, teams, team), s.hi = run_begin(total, teams, team + 1);
    else s.lo = s.hi = 0;
    s.at = s.lo;
    return s;
}

__device__ __forceinline__ Part part_at(const GradArgs& a, int64_t u, int64_t hi) {
    int lo_g = 0, hi_g = a.s.groups - 1;
    while (lo_g < hi_g) {  // the last group that starts at or in front of u: it has row tiles
        const int mid = (lo_g + hi_g + 1) >> 1;
        if (a.starts[mid] <= u) lo_g = mid;
        else hi_g = mid - 1;
    }
    Part p;
    p.group = lo_g;
    p.valid = a.s.valid(lo_g);
    p.rows = a.s.rows_of(lo_g);
    p.per = (p.rows + 127) / 128 * a.s.share;
    const int64_t local = u - a.starts[lo_g];
    p.kv = static_cast<int>(local / p.per);
    p.first = static_cast<int>(local - static_cast<int64_t>(p.kv) * p.per);
    const int64_t seg_end = u - p.first + p.per;
    p.end = seg_end < hi ? seg_end : hi;
    p.last = p.first + static_cast<int>(p.end - u);
    return p;
}

// The share's next part with valid keys.
__device__ __forceinline__ bool next_part(const GradArgs& a, Share& s, Part& p) {
    while (s.tile < s.tiles) {
        while (s.at < s.hi) {
            p = part_at(a, s.at, s.hi);
            s.at = p.end;
            p.tile = s.tile;
            if (s.tile * kKeyTile < p.valid) return true;
        }
        s.tile += s.step;
        s.at = s.lo;
    }
    return false;
}

// The head's rows in which a CTA's run ends, if they also begin there: its own part is
// the first, the same key tile's CTAs in the teams behind have the others.  (With more
// key tiles than CTAs there is one team, and no part of a head's rows.)
__device__ __forceinline__ int4 to_join(const GradArgs& a, const Share& s) {
    const int64_t total = a.starts[a.s.groups];
    const int teams = teams_of(a, total, s.tiles);
    if (teams > 1 && s.lo < s.hi) {
        const Part p = part_at(a, s.hi - 1, s.hi);
        const int64_t begin = s.hi - 1 - p.first, end = begin + p.per;
        if (begin >= s.lo && end > s.hi && s.tile * kKeyTile < p.valid) {
            const int team = blockIdx.x / s.step;
            int last = team + 1;  // the team that has the head's last rows
            while (run_begin(total, teams, last + 1) < end) ++last;
            return make_int4(p.group, p.kv, s.tile, last - team);
        }
    }
    return make_int4(-1, 0, 0, 0);
}

// A row tile: its head and first row in the group.
struct RowTile {
    int head, row0;
    __device__ __forceinline__ void begin(const GradArgs& a, const Part& p) {
        const int tiles = (p.rows + 127) / 128, h = p.first / tiles;
        head = p.kv * a.s.share + h;
        row0 = (p.first - h * tiles) * 128;
    }
    __device__ __forceinline__ void next(const Part& p) {
        row0 += 128;
        if (row0 >= p.rows) row0 = 0, ++head;
    }
};

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
    uint64_t* cleared = sums + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cleared + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cudaGridDependencySynchronize();
    Share share = share_of(a, blockIdx.x);
    Part p;
    const bool works = next_part(a, share, p), placed = (smem_u32(smem) & 1023u) == 0;
    if (!works || !placed) {
        if (!placed) record_status(a.status, BSS_ERR_CUDA);  // the swizzled tiles could not be addressed
        if (threadIdx.x == 0) a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
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
        mbar_init(cleared, 32);
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    RowTile tile;
    bool more = true;
    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&a.q);
            tma_prefetch_desc(&a.dO);
            tma_prefetch_desc(&a.k);
            tma_prefetch_desc(&a.v);
            uint32_t parts = 0, vs = 0, qs = 0, dos = 0;
            bool ok = true;
            for (; ok && more; more = next_part(a, share, p)) {
                const int g = a.s.shared_states ? 0 : p.group;
                if (parts > 0) ok = mbar_wait(k_empty, (parts - 1) & 1, a.status);
                if (!ok) break;
                mbar_arrive_expect_tx(k_full, L::kTile);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    tma_load_4d(smem + L::kK + c * kChunkBytesSw128, &a.k, c * 64, p.tile * kKeyTile, p.kv, g, k_full);
                ++parts;
                tile.begin(a, p);
                for (int x = p.first; x < p.last; ++x, tile.next(p)) {
                    const uint32_t sq = qs % kQStages, sd = dos % kDOStages;
                    const int row = p.group * a.s.group_rows + tile.row0;
                    if (qs >= kQStages) ok = mbar_wait(q_empty + sq, (qs / kQStages - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(q_full + sq, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(smem + L::kQ + sq * L::kTile + c * kChunkBytesSw128, &a.q, c * 64, row, tile.head, q_full + sq);
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
                        tma_load_3d(smem + L::kDO + sd * L::kTile + c * kChunkBytesSw128, &a.dO, c * 64, row, tile.head, do_full + sd);
                    ++dos;
                }
            }
            // no copy may still be landing in shared memory at exit
            if (parts > 0) mbar_wait(k_full, (parts - 1) & 1, a.status);
            if (vs > 0) mbar_wait(v_full, (vs - 1) & 1, a.status);
            for (uint32_t f = qs > kQStages ? qs - kQStages : 0; f < qs; ++f)
                mbar_wait(q_full + f % kQStages, (f / kQStages) & 1, a.status);
            for (uint32_t f = dos > kDOStages ? dos - kDOStages : 0; f < dos; ++f)
                mbar_wait(do_full + f % kDOStages, (f / kDOStages) & 1, a.status);
        } else if (warp == 0 && lane == 1) {
            a.joins[blockIdx.x] = to_join(a, share);
        } else if (warp == 1) {
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint32_t d_k = desc_lo_kmajor(base + L::kK), d_v = desc_lo_kmajor(base + L::kV);
            const uint32_t d_q = desc_lo_kmajor(base + L::kQ), d_do = desc_lo_kmajor(base + L::kDO);
            const uint32_t d_qt = desc_lo_mnmajor(base + L::kQ), d_dot = desc_lo_mnmajor(base + L::kDO);
            constexpr uint32_t kTileStep = L::kTile >> 4;
            constexpr uint32_t idesc_sum = idesc_bf16_f32(128, D, 1);
            // (no vote: only the leader's MMAs and commits count)
            auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, a.status); };
            auto commit = [&](uint64_t* bar) {
                if (leader) tc_commit(bar);
            };
            // (a whole tile's products apart: nothing of theirs is computed at run time)
            auto product = [&](uint32_t col, uint32_t da, uint32_t db, int w) {
                const uint32_t idesc = idesc_bf16_f32(128, 0, 0) | (static_cast<uint32_t>(w >> 3) << 17);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (kk >> 2) * (kChunkBytesSw128 >> 4) + (kk & 3) * 2;
                        umma_ss(tmem + col, desc_of(da + at), desc_of(db + at), idesc, kk > 0);
                    }
                }
            };
            auto sum_up = [&](uint32_t col, uint32_t from, uint32_t db, int w, bool add) {
                if (w == 128) {
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_ts(tmem + col, tmem + from + packed_col(kk), desc_of(db + kk * 128), idesc_sum, add || kk > 0);
                    }
                } else if (leader) {
                    for (int kk = 0; kk < w / 16; ++kk)
                        umma_ts(tmem + col, tmem + from + packed_col(kk), desc_of(db + kk * 128), idesc_sum, add || kk > 0);
                }
            };
            // the row tile at the cursor, number f of the share
            uint32_t part = 0, clears = 0;
            int x = p.first;
            tile.begin(a, p);
            // behind the last row of all a load gives zeros; behind another group's there are rows
            auto last_rows = [&]() { return p.group == a.s.groups - 1; };
            auto rows_now = [&]() { return p.rows - tile.row0 < 128 ? p.rows - tile.row0 : 128; };
            auto issue_s = [&](uint32_t f) {
                const uint32_t st = f % kQStages;
                if (x == p.first && !wait(k_full, part & 1)) return false;
                if (!wait(q_full + st, (f / kQStages) & 1)) return false;
                const int n = rows_now();
                if ((n & 15) && !last_rows() && !clear_rows<D>(smem + L::kQ + st * L::kTile, n, cleared, clears, a.status)) return false;
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
                const int n = rows_now();
                if ((n & 15) && !last_rows() && !clear_rows<D>(smem + L::kDO + st * L::kTile, n, cleared, clears, a.status)) return false;
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
                sum_up(kColA, kColS, d_dot + st * kTileStep, (rows_now() + 15) & ~15, x > p.first);
                commit(do_empty + st);
                return true;
            };
            bool ok = issue_s(0) && issue_dp(0) && issue_dv(0);
            for (uint32_t f = 0; ok && more; ++f) {
                const int w = (rows_now() + 15) & ~15;
                const bool add = x > p.first, last = x == p.last - 1;
                if (last) {
                    more = next_part(a, share, p);
                    if (more) {
                        x = p.first;
                        tile.begin(a, p);
                        ++part;
                    }
                } else {
                    ++x;
                    tile.next(p);
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
            for (; ok && more; more = next_part(a, share, p)) {
                tile.begin(a, p);
                for (int x = p.first; x < p.last; ++x, ++f, tile.next(p)) {
                    const uint32_t st = f % kAuxStages;
                    const int r = tile.row0 + i;
                    const int64_t at = static_cast<int64_t>(tile.head) * a.s.rows + static_cast<int64_t>(p.group) * a.s.group_rows + r;
                    float v[4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const bool live = r + 64 * y < p.rows;
                        v[y] = live ? lse_base2(a.lse[at + 64 * y]) : INFINITY;
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
        Part& t = p;
        uint32_t f = 0, part = 0;
        bool ok = true;
        for (; ok && more; more = next_part(a, share, t), ++part) {
            const int key = t.tile * kKeyTile + r;
            const bool live = key < t.valid;
            for (int x = t.first; x < t.last; ++x, ++f) {
                const uint32_t st = f % kAuxStages;
                float w[64];
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
                        w[4 * y] = ex2_approx(y0);
                        w[4 * y + 1] = ex2_approx(y1);
                        w[4 * y + 2] = ex2_approx(y2);
                        w[4 * y + 3] = ex2_approx(y3);
                    }
#pragma unroll
                    for (int y = 0; y < 64; ++y) w[y] = live ? w[y] : 0.0f;
                    store_packed(t_s, w);
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
                        w[4 * y] *= y0;
                        w[4 * y + 1] *= y1;
                        w[4 * y + 2] *= y2;
                        w[4 * y + 3] *= y3;
                    }
                    // a masked state's values may be anything
#pragma unroll
                    for (int y = 0; y < 64; ++y) w[y] = live ? w[y] : 0.0f;
                    store_packed(t_p, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(ds_full);
                mbar_arrive(aux_empty + st);
            }
            if (!ok) break;
            // the key tile's sums: half 0 has dv, half 1 dk.  A masked state's are zeros, also
            // where a row's dO or q is no number: 0 times it would not be.
            if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(sums, part & 1, a.status)))) break;
            tc_fence_after();
            const uint32_t acc = tmem + lanes + (half == 0 ? kColA : kColB);
            if (t.first == 0 && t.last == t.per) {
                const int key0 = t.tile * kKeyTile + (warp & 3) * 32;
                uint16_t* to = half == 0 ? a.dv + t.group * a.dv_group + key0 * a.dv_token + t.kv * a.dv_head
                                         : a.dk + t.group * a.dk_group + key0 * a.dk_token + t.kv * a.dk_head;
                store_rows<D>(acc, to, half == 0 ? a.dv_token : a.dk_token, a.s.keys - key0, half == 0 ? 1.0f : a.scale, live);
            } else {
                // [16 bytes of the channels][key]: the join reads them so
                const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (t.first > 0 ? 0 : 1);
                uint4* to = reinterpret_cast<uint4*>(a.parts + (slot * 2 + half) * 128 * D) + r;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    BSS_TMEM_LD32(acc + cc * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        to[(cc * 8 + y) * 128] = live ? make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]) : make_uint4(0, 0, 0, 0);
                }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- sums of parts, zeros
// Block (b, y): the parts that begin with CTA b's, in their order.  Key tiles without a
// valid state: zeros.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ GradArgs a) {
    cudaGridDependencySynchronize();
    const int4 join = a.joins[blockIdx.x];
    if (join.x >= 0) {
        const int tiles = static_cast<int>(a.starts[a.s.groups + 1]), step = tiles <= a.blocks ? tiles : a.blocks;
        // a thread sums 8 channels of a key: neighbours in a warp are neighbouring keys
        constexpr int kVectors = 2 * 128 * D / 8;
        for (int i = blockIdx.y * 256 + threadIdx.x; i < kVectors; i += gridDim.y * 256) {
            const int which = i / (128 * D / 8), r = i % 128, c = i / 128 % (D / 8);
            float v[8], w[8];
            auto fetch = [&](int64_t slot, float (&to)[8]) {
                const float4* from = reinterpret_cast<const float4*>(a.parts + (slot * 2 + which) * 128 * D) + 2 * c * 128 + r;
                const float4 x = from[0], y = from[128];
                to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w, to[4] = y.x, to[5] = y.y, to[6] = y.z, to[7] = y.w;
            };
            fetch(2 * static_cast<int64_t>(blockIdx.x) + 1, v);
#pragma unroll 4
            for (int k = 1; k <= join.w; ++k) {
                fetch(2 * (static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(k) * step), w);
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] += w[x];
            }
            const int key = join.z * kKeyTile + r;
            if (key >= a.s.keys) continue;
            uint16_t* to = which == 0 ? a.dv + join.x * a.dv_group + key * a.dv_token + join.y * a.dv_head
                                      : a.dk + join.x * a.dk_group + key * a.dk_token + join.y * a.dk_head;
            const float scale = which == 0 ? 1.0f : a.scale;
            *reinterpret_cast<uint4*>(to + 8 * c) = make_uint4(pack2(v[0] * scale, v[1] * scale), pack2(v[2] * scale, v[3] * scale),
                                                               pack2(v[4] * scale, v[5] * scale), pack2(v[6] * scale, v[7] * scale));
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

// ---------------------------------------------------------------- few rows
// A few rows a group (a token, a handful of queries) fill no tile: everything in 32 bits,
// eight lanes a key with d / 8 channels each, four keys a warp at once.  The first blocks
// have dq, one a row and head, and go over all its keys; the others have dk and dv of 64
// keys each and go over the rows of all heads that share them.  No sums between blocks, no
// workspace.  Bound by a key's chain of load, two sums of eight lanes and an exponential.
// Taken for a few rows of a key head and few pairs of rows and keys (us on the device, without
// and with tiles): 10 heads x 128, one row over 512 / 2,048 states 6.2 / 16.3 and 18.9 / 37.1, 8
// rows 12.5 / 26.7 and 18.9 / 37.0, 16 rows 17.8 / 50.5 and 19.0 / 36.9; 40 heads, 8 rows over 512
// (2^17.3 pairs) 30.7 and 23.1.  A call by itself takes 19 us instead of 34: one launch instead
// of three, and no workspace.
constexpr int kFewRows = 16;
constexpr int64_t kFewPairs = 1 << 17;

struct FewGradArgs {
    CrossShape s;
    const uint16_t *q, *dO, *O, *k, *v;
    uint16_t *dq, *dk, *dv;
    int64_t q_row, q_head, dO_row, dO_head, O_row, O_head, dq_row, dq_head;
    int64_t k_group, k_token, k_head, v_group, v_token, v_head;
    int64_t dk_group, dk_token, dk_head, dv_group, dv_token, dv_head;
    float scale;
    const float* lse;  // [heads][rows]
    int32_t dq_blocks, key_blocks;
};

template <int D>
__global__ void __launch_bounds__(kFewThreads) cross_few_kernel(const __grid_constant__ FewGradArgs a) {
    constexpr int N = D / 64;
    __shared__ float sums[kFewWarps][D];
    const int warp = threadIdx.x >> 5, unit = threadIdx.x & 7, slot = (threadIdx.x >> 3) & 3;
    cudaGridDependencySynchronize();
    if (static_cast<int>(blockIdx.x) < a.dq_blocks) {
        const int row = blockIdx.x / a.s.heads, h = blockIdx.x - row * a.s.heads, kv = h / a.s.share;
        const int group = row / a.s.group_rows, n = a.s.valid(group);
        float q[8 * N], g[8 * N], x[8 * N], sum[8 * N] = {};
        load_part<N>(a.O + row * a.O_row + h * a.O_head, unit, x);
        load_part<N>(a.dO + row * a.dO_row + h * a.dO_head, unit, g);
        load_part<N>(a.q + row * a.q_row + h * a.q_head, unit, q);
        const float delta = dot_part<N>(g, x), lse = lse_base2(a.lse[static_cast<int64_t>(h) * a.s.rows + row]);
        const uint16_t* k = a.k + group * a.k_group + kv * a.k_head;
        const uint16_t* v = a.v + group * a.v_group + kv * a.v_head;
#pragma unroll 2
        for (int first = warp * 4; first < n; first += kFewWarps * 4) {
            const int64_t key = min(first + slot, n - 1);
            float y[8 * N];
            load_part<N>(k + key * a.k_token, unit, x);
            load_part<N>(v + key * a.v_token, unit, y);
            const float s = dot_part<N>(q, x), dp = dot_part<N>(g, y);
            const float p = ex2_approx(fmaf(s, a.s.scale_log2, -lse)), ds = p * (dp - delta);
            if (first + slot < n)
#pragma unroll
                for (int i = 0; i < 8 * N; ++i) sum[i] = fmaf(ds, x[i], sum[i]);
        }
#pragma unroll
        for (int i = 0; i < 8 * N; ++i) {
            sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 8);
            sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 16);
            if (slot == 0) sums[warp][8 * (unit + 8 * (i / 8)) + i % 8] = sum[i];
        }
        __syncthreads();
        if (threadIdx.x < 8) {
#pragma unroll
            for (int i = 0; i < 8 * N; ++i) {
                sum[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < kFewWarps; ++w) sum[i] += sums[w][8 * (unit + 8 * (i / 8)) + i % 8];
            }
            store_part<N>(a.dq + row * a.dq_row + h * a.dq_head, unit, sum, a.scale);
        }
        return;
    }
    const int block = blockIdx.x - a.dq_blocks, rest = block / a.key_blocks;
    const int group = rest / a.s.kv_heads, kv = rest - group * a.s.kv_heads, n = a.s.valid(group);
    const int64_t key = (block - rest * a.key_blocks) * (kFewWarps * 4) + warp * 4 + slot;
    const bool live = key < n;
    float k[8 * N] = {}, v[8 * N] = {}, dk[8 * N] = {}, dv[8 * N] = {};
    if (live) {
        load_part<N>(a.k + group * a.k_group + key * a.k_token + kv * a.k_head, unit, k);
        load_part<N>(a.v + group * a.v_group + key * a.v_token + kv * a.v_head, unit, v);
    }
    const int row0 = group * a.s.group_rows, rows = a.s.rows_of(group), pairs = n > 0 ? rows * a.s.share : 0;
#pragma unroll 2
    for (int i = 0; i < pairs; ++i) {
        const int h = kv * a.s.share + i / rows, row = row0 + i % rows;
        float q[8 * N], g[8 * N], o[8 * N];
        load_part<N>(a.q + row * a.q_row + h * a.q_head, unit, q);
        load_part<N>(a.dO + row * a.dO_row + h * a.dO_head, unit, g);
        load_part<N>(a.O + row * a.O_row + h * a.O_head, unit, o);
        const float lse = lse_base2(a.lse[static_cast<int64_t>(h) * a.s.rows + row]);
        const float s = dot_part<N>(q, k), dp = dot_part<N>(g, v), delta = dot_part<N>(g, o);
        const float p = ex2_approx(fmaf(s, a.s.scale_log2, -lse)), ds = p * (dp - delta);
#pragma unroll
        for (int c = 0; c < 8 * N; ++c) {
            dk[c] = fmaf(ds, q[c], dk[c]);
            dv[c] = fmaf(p, g[c], dv[c]);
        }
    }
    if (key >= a.s.keys) return;
    if (!live)
#pragma unroll
        for (int c = 0; c < 8 * N; ++c) dk[c] = dv[c] = 0.0f;
    store_part<N>(a.dk + group * a.dk_group + key * a.dk_token + kv * a.dk_head, unit, dk, a.scale);
    store_part<N>(a.dv + group * a.dv_group + key * a.dv_token + kv * a.dv_head, unit, dv, 1.0f);
}

template <int D>
bss_status launch_backward(GradArgs& a, cudaStream_t stream) {
    auto dq = cross_dq_kernel<D>;
    auto dkv = cross_dkv_kernel<D>;
    int blocks;
    bss_status st = resident_blocks(reinterpret_cast<const void*>(dq), kDqThreads, DqSmem<D>::kBytes, &blocks);
    if (st == BSS_OK) st = resident_blocks(reinterpret_cast<const void*>(dkv), kThreads, DkvSmem<D>::kBytes, &blocks);
    if (st != BSS_OK) return st;
    const int grid = a.items < num_sms() ? a.items : num_sms();
    st = launch_behind_with(dq, dim3(static_cast<unsigned>(grid)), kDqThreads, DqSmem<D>::kBytes, 1, stream, "query gradient launch", a);
    if (st == BSS_OK)
        st = launch_behind_with(dkv, dim3(static_cast<unsigned>(a.blocks)), kThreads, DkvSmem<D>::kBytes, 1, stream, "key gradient launch", a);
    if (st == BSS_OK)
        st = launch_behind_with(cross_join_kernel<D>, dim3(static_cast<unsigned>(a.blocks), 8), 256, 0, 1, stream,
                                "key gradient sums launch", a);
    return st;
}

int64_t aligned_up(int64_t v) { return (v + 255) / 256 * 256; }

struct Plan {
    int64_t delta_at, starts_at, joins_at, parts_at, bytes;
    int32_t tiles, key_tiles, blocks;
    bool few;
};


// rows_per_group at most rows
Plan plan_of(const bss_cross_grads& a) {
    Plan p;
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    p.few = a.rows_per_group * (a.heads / a.kv_heads) <= kFewRows && a.rows * a.heads <= kFewPairs / a.keys;
    p.tiles = static_cast<int32_t>((a.rows_per_group + 127) / 128);
    p.key_tiles = static_cast<int32_t>((static_cast<int64_t>(a.keys) + kKeyTile - 1) / kKeyTile);
    const double pairs = static_cast<double>(groups) * p.tiles * p.key_tiles * a.heads;
    p.blocks = pairs < num_sms() ? static_cast<int32_t>(pairs) : num_sms();
    p.delta_at = 0;
    p.starts_at = aligned_up(a.rows * a.heads * 4);
    p.joins_at = p.starts_at + aligned_up((groups + 2) * 8);
    p.parts_at = p.joins_at + aligned_up(p.blocks * 16ll);
    p.bytes = p.few ? 0 : p.parts_at + 2ll * p.blocks * 2 * 128 * a.head_dim * 4;
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
    auto stride = [](int64_t extent, int64_t s) { return extent > 1 ? s : 0; };
    const CrossShape shape = cross_shape(p.rows, p.rows_per_group, p.heads, p.kv_heads, p.head_dim, p.keys, p.softmax_scale,
                                         p.lengths, p.k.group_stride);
    const float scale = p.softmax_scale > 0.0f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim));
    if (plan.few) {
        FewGradArgs f;
        memset(&f, 0, sizeof(f));
        f.s = shape, f.scale = scale, f.lse = p.lse;
        auto rows_of = [&](const bss_token_tensor& t, auto*& to, int64_t& row, int64_t& head) {
            to = static_cast<uint16_t*>(t.data), row = stride(p.rows, t.token_stride), head = stride(p.heads, t.head_stride);
        };
        auto states_of = [&](const bss_state_tensor& t, auto*& to, int64_t& group, int64_t& token, int64_t& head) {
            to = static_cast<uint16_t*>(t.data), group = stride(groups, t.group_stride);
            token = stride(p.keys, t.token_stride), head = stride(p.kv_heads, t.head_stride);
        };
        rows_of(p.q, f.q, f.q_row, f.q_head);
        rows_of(p.dO, f.dO, f.dO_row, f.dO_head);
        rows_of(p.O, f.O, f.O_row, f.O_head);
        rows_of(p.dq, f.dq, f.dq_row, f.dq_head);
        states_of(p.k, f.k, f.k_group, f.k_token, f.k_head);
        states_of(p.v, f.v, f.v_group, f.v_token, f.v_head);
        states_of(p.dk, f.dk, f.dk_group, f.dk_token, f.dk_head);
        states_of(p.dv, f.dv, f.dv_group, f.dv_token, f.dv_head);
        f.dq_blocks = static_cast<int32_t>(p.rows * p.heads);
        f.key_blocks = static_cast<int32_t>((p.keys + kFewWarps * 4ll - 1) / (kFewWarps * 4));
        const unsigned blocks = static_cast<unsigned>(f.dq_blocks + groups * p.kv_heads * f.key_blocks);
        return launch_behind(p.head_dim == 128 ? cross_few_kernel<128> : cross_few_kernel<64>, dim3(blocks), kFewThreads, stream,
                             "few rows' gradient launch", f);
    }
    const int64_t items = groups * plan.tiles * p.heads;
    if (items > 0x7FFFFFFF - 4096) return set_error(BSS_ERR_UNSUPPORTED, "too many rows and heads");
    GradArgs a;
    memset(&a, 0, sizeof(a));
    if ((st = row_heads_map(&a.q, p.q, p.rows, p.heads, p.head_dim, kHalfRows)) != BSS_OK ||
        (st = row_heads_map(&a.dO, p.dO, p.rows, p.heads, p.head_dim, kHalfRows)) != BSS_OK ||
        (st = states_map(&a.k, p.k, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK ||
        (st = states_map(&a.v, p.v, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK)
        return st;
    a.s = shape;
    a.tiles = plan.tiles, a.key_tiles = plan.key_tiles, a.blocks = plan.blocks;
    a.items = static_cast<int32_t>(items);
    a.by_tiles = FastDiv(static_cast<uint32_t>(plan.tiles));
    a.O = static_cast<const uint16_t*>(p.O.data);
    a.dq = static_cast<uint16_t*>(p.dq.data);
    a.dk = static_cast<uint16_t*>(p.dk.data);
    a.dv = static_cast<uint16_t*>(p.dv.data);
    a.O_row = stride(p.rows, p.O.token_stride), a.O_head = stride(p.heads, p.O.head_stride);
    a.dq_row = stride(p.rows, p.dq.token_stride), a.dq_head = stride(p.heads, p.dq.head_stride);
    a.dk_group = stride(groups, p.dk.group_stride), a.dk_token = stride(p.keys, p.dk.token_stride);
    a.dk_head = stride(p.kv_heads, p.dk.head_stride);
    a.dv_group = stride(groups, p.dv.group_stride), a.dv_token = stride(p.keys, p.dv.token_stride);
    a.dv_head = stride(p.kv_heads, p.dv.head_stride);
    a.scale = scale;
    a.lse = p.lse;
    char* ws = static_cast<char*>(p.workspace);
    a.delta = reinterpret_cast<float*>(ws + plan.delta_at);
    a.starts = reinterpret_cast<int64_t*>(ws + plan.starts_at);
    a.joins = reinterpret_cast<int4*>(ws + plan.joins_at);
    a.parts = reinterpret_cast<float*>(ws + plan.parts_at);
    a.status = device_status_ptr();
    if (a.status == nullptr) return set_error(BSS_ERR_CUDA, "cannot resolve the device status word");
    return p.head_dim == 128 ? launch_backward<128>(a, stream) : launch_backward<64>(a, stream);
}

}  // extern "C"
