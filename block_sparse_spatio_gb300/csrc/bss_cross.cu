// bss_cross.cu -- attention of the video's tokens over an encoder's states of
// another length (forward).
//
//   S = q k^T,  P = exp(scale S - m),  l = sum P,  O = P v / l,  lse = m + ln l
//
// for the valid keys of a row's group.  One CTA takes items of (group, 256 rows,
// head) in turn; an item's rows are two halves of 128, whose softmaxes alternate
// with each other's MMAs:
//   warp 0        loads Q of each half, K and V tiles of 128 keys (two stages each)
//   warp 1        issues S_1(j) PV_0(j) S_0(j+1) PV_1(j): each half's softmax has the
//                 other half's two products to work in.  S_0 of the next item follows
//                 the last S_0 of this one, so the tensor cores do not wait for the
//                 end of an item.
//   warps 4..7    bring O / l and lse of a finished half to memory, while
//   warps 8..15   go on with the softmax of the next item, one thread a row (when they
//                 stored O themselves an item of 4 key tiles took 16,000 cycles, a third
//                 of them stores and waits for the last product).
// TMEM: S_h at 128 h (P_h as bf16 over its first 64 columns), O_h at 256 + 128 h.
// A row's reference is the maximum of its first tile, moved only when the sum of a
// later tile's P passes 2^16 (then O and l are rescaled), or when no score so far was
// above minus infinity.
// P is rounded to bf16 on the way to its product, because the tensor cores take both
// operands in one type and 32-bit ones at an eighth of the rate; l sums the unrounded P.
//
// 75,600 x 10 x 128 over 512 states, lse kept: 156 us (1,270 TFLOP/s).  A further key tile
// costs 31.9 us (1,554 TFLOP/s, 90% of what cuBLAS sustains under the power limit; a step of both
// halves moves 272 KB of shared memory, 2,125 cycles at 128 bytes, beneath 2,048 cycles
// of products), the ends of the items 18 us.  Over 128 states 69 us, of which Q and O alone are 59 at a copy's rate.
#include "bss_cross.cuh"

#include <cstring>
#include <type_traits>

namespace bss {
namespace {

constexpr int kThreads = 512;
constexpr int kStages = 2;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
constexpr float kSumLimit = 65536.0f;
// Registers: 128 x (64 + 96 + 2 x 176) = the launch's 512 x 128.
constexpr uint32_t kRegsControl = 64, kRegsStore = 96, kRegsSoftmax = 176;

// A tile of queries holds rows of its group alone, zeros behind them: the next group's may
// be written over by another CTA at that moment (O over q), and a row's large scores move
// the references of its whole warp.  Hence a dimension of groups in the map of those that
// have all of group_rows rows, and a map of its own for a shorter last one.
struct CrossArgs {
    CUtensorMap q, q_rest, k, v, o;
    CrossShape s;
    int32_t whole;  // groups of group_rows rows
    int32_t tiles;  // of 256 rows in a group
    int32_t items;
    FastDiv by_tiles;
    uint16_t* O;
    int64_t O_row, O_head;
    float* lse;
    int* status;
};

template <int D>
struct CrossSmem {
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = 2 * kTile;
    static constexpr uint32_t kV = kK + kStages * kTile;
    static constexpr uint32_t kO = kV + kStages * kTile;  // 32 rows of each of the storing warps
    static constexpr uint32_t kSums = kO + kTile;         // l: float [half][item & 1][128]
    static constexpr uint32_t kBar = kSums + 2048;
    // q_full[2] q_empty[2] k_full k_empty v_full v_empty [kStages] s_full[2] p_full[2] o_done[2] o_final[2] o_read[2]
    // l_full[2][2] cleared
    static constexpr uint32_t kBars = 4 + 4 * kStages + 15;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 16;
};

struct Item {
    int group, row0, rows, head, valid, n;  // row0, rows: the item's rows within the group
    bool two;                               // the second half has rows
};

__device__ __forceinline__ Item item_at(const CrossArgs& a, int i) {
    Item t;
    const int rest = a.s.by_heads.div(i);
    t.head = i - rest * a.s.heads;
    t.group = a.by_tiles.div(rest);
    t.row0 = (rest - t.group * a.tiles) * 256;
    t.rows = a.s.rows_of(t.group) - t.row0;
    t.valid = t.rows > 0 ? a.s.valid(t.group) : 0;
    t.n = (t.valid + kKeyTile - 1) / kKeyTile;
    t.two = t.rows > kHalfRows;
    return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_forward_kernel(const __grid_constant__ CrossArgs a) {
    using L = CrossSmem<D>;
    constexpr int kChunks = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles could not be addressed
        record_status(a.status, BSS_ERR_CUDA);
        return;
    }
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* q_empty = q_full + 2;
    uint64_t* k_full = q_empty + 2;
    uint64_t* k_empty = k_full + kStages;
    uint64_t* v_full = k_empty + kStages;
    uint64_t* v_empty = v_full + kStages;
    uint64_t* s_full = v_empty + kStages;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 2;
    uint64_t* o_final = o_done + 2;
    uint64_t* o_read = o_final + 2;
    uint64_t* l_full = o_read + 2;
    uint64_t* cleared = l_full + 4;  // (l_full: by half and item & 1)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cleared + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 128);
            mbar_init(o_done + i, 1);
            mbar_init(o_final + i, 1);
            mbar_init(o_read + i, 128);
            mbar_init(l_full + i, 128);
            mbar_init(l_full + 2 + i, 128);
        }
        mbar_init(cleared, 32);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
            mbar_init(v_full + i, 1);
            mbar_init(v_empty + i, 1);
        }
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    cudaGridDependencySynchronize();

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&a.q);
            tma_prefetch_desc(&a.k);
            tma_prefetch_desc(&a.v);
            uint32_t fills = 0, q_fills[2] = {0, 0};
            uint32_t k_issued = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
                const Item t = item_at(a, i);
                if (t.n == 0) continue;
                const bool rest = t.group >= a.whole;
                const CUtensorMap* q = rest ? &a.q_rest : &a.q;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !t.two) break;
                    if (q_fills[h] > 0) ok = mbar_wait(q_empty + h, (q_fills[h] - 1) & 1, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(q_full + h, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_4d(smem + L::kQ + h * L::kTile + c * kChunkBytesSw128, q, c * 64, t.row0 + h * kHalfRows, t.head,
                                    rest ? 0 : t.group, q_full + h);
                    ++q_fills[h];
                }
                const int kv = a.s.by_share.div(t.head), g = a.s.shared_states ? 0 : t.group;
                for (int j = 0; ok && j < t.n; ++j, ++fills) {
                    const uint32_t st = fills % kStages, parity = (fills / kStages - 1) & 1;
                    if (fills >= kStages) ok = mbar_wait(k_empty + st, parity, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(k_full + st, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_4d(smem + L::kK + st * L::kTile + c * kChunkBytesSw128, &a.k, c * 64, j * kKeyTile, kv, g,
                                    k_full + st);
                    k_issued = fills + 1;
                    if (fills >= kStages) ok = mbar_wait(v_empty + st, parity, a.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(v_full + st, L::kTile);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_4d(smem + L::kV + st * L::kTile + c * kChunkBytesSw128, &a.v, c * 64, j * kKeyTile, kv, g,
                                    v_full + st);
                }
            }
            // no copy may still be landing in shared memory at exit
            for (int h = 0; h < 2; ++h)
                if (q_fills[h] > 0) mbar_wait(q_full + h, (q_fills[h] - 1) & 1, a.status);
            for (uint32_t f = k_issued > kStages ? k_issued - kStages : 0; f < k_issued; ++f)
                mbar_wait(k_full + f % kStages, (f / kStages) & 1, a.status);
            for (uint32_t f = fills > kStages ? fills - kStages : 0; f < fills; ++f)
                mbar_wait(v_full + f % kStages, (f / kStages) & 1, a.status);
        } else if (warp == 1) {
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint32_t dq = desc_lo_kmajor(base + L::kQ), dk = desc_lo_kmajor(base + L::kK);
            const uint32_t dv = desc_lo_mnmajor(base + L::kV);
            constexpr uint32_t kTileStep = L::kTile >> 4;
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
            // (no vote: only the leader's MMAs and commits count)
            auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, a.status); };
            auto commit = [&](uint64_t* bar) {
                if (leader) tc_commit(bar);
            };
            // keys of a tile rounded up to what an MMA takes
            auto width = [](const Item& t, int j) {
                const int left = t.valid - j * kKeyTile;
                return left >= kKeyTile ? kKeyTile : (left + 15) & ~15;
            };
            auto issue_s = [&](int h, uint32_t st, int w) {
                const uint32_t idesc = idesc_bf16_f32(128, 0, 0) | (static_cast<uint32_t>(w >> 3) << 17);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (kk >> 2) * (kChunkBytesSw128 >> 4) + (kk & 3) * 2;
                        umma_ss(tmem + kColS + 128 * h, desc_of(dq + h * kTileStep + at), desc_of(dk + st * kTileStep + at), idesc, kk > 0);
                    }
                }
            };
            auto issue_pv = [&](int h, uint32_t st, int w, bool add) {
                const uint32_t o = tmem + kColO + 128 * h, p = tmem + kColS + 128 * h, b = dv + st * kTileStep;
                if (leader) {  // unrolled: a loop takes 110 cycles a product of 16 keys, which lasts 64
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk * 16 < w) umma_ts(o, p + kk * 8, desc_of(b + kk * 128), idesc_pv, add || kk > 0);
                }
            };
            uint32_t fills = 0, clears = 0;               // K and V tiles taken
            uint32_t q_taken[2] = {0, 0}, p_taken[2] = {0, 0}, items[2] = {0, 0};
            int i = blockIdx.x;
            Item t;
            auto next_item = [&](int from) {  // the first one with keys
                for (i = from; i < a.items; i += gridDim.x) {
                    t = item_at(a, i);
                    if (t.n > 0) return true;
                }
                return false;
            };
            // the first S_0 of item t, whose K tile is fill f
            auto begin_item = [&](uint32_t f) {
                const uint32_t st = f % kStages;
                if (!wait(q_full + 0, q_taken[0]++ & 1) || !wait(k_full + st, (f / kStages) & 1)) return false;
                tc_fence_after();
                issue_s(0, st, width(t, 0));
                commit(s_full + 0);
                if (t.n == 1) commit(q_empty + 0);
                return true;
            };
            bool more = next_item(i), ok = true;
            if (more) ok = begin_item(0);
            while (ok && more) {
                const Item cur = t;
                for (int j = 0; j < cur.n; ++j, ++fills) {
                    const uint32_t st = fills % kStages, parity = (fills / kStages) & 1;
                    const int w = width(cur, j);
                    if (cur.two) {
                        if (j == 0 && !(ok = wait(q_full + 1, q_taken[1]++ & 1))) break;
                        tc_fence_after();
                        issue_s(1, st, w);
                        commit(s_full + 1);
                        if (j == cur.n - 1) commit(q_empty + 1);
                    }
                    commit(k_empty + st);  // both halves' S
                    if (!(ok = wait(v_full + st, parity))) break;
                    const int left = cur.valid - j * kKeyTile;
                    // (behind the last state of all a load gives zeros)
                    if (left < w && cur.valid < a.s.keys && !(ok = clear_rows<D>(smem + L::kV + st * L::kTile, left, cleared, clears, a.status))) break;
                    if (!(ok = wait(p_full + 0, p_taken[0]++ & 1))) break;
                    // an item's first product: the O before has been read
                    if (j == 0 && items[0]++ > 0 && !(ok = wait(o_read + 0, items[0] & 1))) break;
                    tc_fence_after();
                    issue_pv(0, st, w, j > 0);
                    commit(o_done + 0);
                    if (j == cur.n - 1) commit(o_final + 0);
                    if (j + 1 < cur.n) {
                        const uint32_t f = fills + 1;
                        if (!(ok = wait(k_full + f % kStages, (f / kStages) & 1))) break;
                        tc_fence_after();
                        issue_s(0, f % kStages, width(cur, j + 1));
                        commit(s_full + 0);
                        if (j + 1 == cur.n - 1) commit(q_empty + 0);
                    } else {
                        more = next_item(i + gridDim.x);
                        if (more && !(ok = begin_item(fills + 1))) break;
                    }
                    if (cur.two) {
                        if (!(ok = wait(p_full + 1, p_taken[1]++ & 1))) break;
                        if (j == 0 && items[1]++ > 0 && !(ok = wait(o_read + 1, items[1] & 1))) break;
                        tc_fence_after();
                        issue_pv(1, st, w, j > 0);
                        commit(o_done + 1);
                        if (j == cur.n - 1) commit(o_final + 1);
                    }
                    commit(v_empty + st);
                }
            }
        }
    } else if (warp < 8) {
        setmaxnreg_dec<kRegsStore>();
        const int w = warp - 4, r = threadIdx.x - 128;
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        const float* sums = reinterpret_cast<const float*>(smem + L::kSums) + r;
        uint8_t* mine = smem + L::kO + w * (32 * D * 2);  // 64 columns of 32 rows, 128 bytes a row, twice over for 128
        uint32_t items[2] = {0, 0};
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const Item t = item_at(a, i);
            if (t.rows <= 0) continue;
#pragma unroll 1
            for (int h = 0; h < (t.two ? 2 : 1); ++h) {
                const int row0 = t.row0 + h * kHalfRows + w * 32, rows = t.row0 + t.rows - row0;  // the warp's, in the group
                const int64_t first = static_cast<int64_t>(t.group) * a.s.group_rows + row0;
                uint16_t* out = a.O + first * a.O_row + t.head * a.O_head;
                if (t.n == 0) {  // no states
                    for (int e = lane; e < 32 * (D / 8); e += 32)
                        if (e / (D / 8) < rows) *reinterpret_cast<uint4*>(out + e / (D / 8) * a.O_row + e % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
                    if (a.lse != nullptr && lane < rows) a.lse[static_cast<int64_t>(t.head) * a.s.rows + first + lane] = -INFINITY;
                    continue;
                }
                const uint32_t n = h == 0 ? items[0]++ : items[1]++;
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(l_full + 2 * h + (n & 1), (n >> 1) & 1, a.status)))) break;
                const float l = sums[(h * 2 + (n & 1)) * 128];
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if (lane == 0) tma_store_wait_read_all();  // the store before has read its rows
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_final + h, n & 1, a.status)))) break;
                tc_fence_after();
                const uint32_t t_o = tmem + lanes + kColO + 128 * h;
#pragma unroll
                for (int c = 0; c < D; c += 64) {
                    uint4 u[8];
                    read_rows<64>(u, t_o + c, inv);
                    if (c + 64 == D) {
                        tc_fence_before();
                        mbar_arrive(o_read + h);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(mine + c * 64 + lane * 128 + ((k ^ (lane & 7)) << 4)) = u[k];
                }
                if (rows >= 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int c = 0; c < D; c += 64) tma_store_3d(&a.o, mine + c * 64, c, static_cast<int>(first), t.head);
                        tma_store_commit();
                    }
                } else {  // what lies behind the group's last row is another's
                    __syncwarp();
                    for (int e = lane; e < 32 * (D / 8); e += 32) {
                        const int row = e / (D / 8), unit = e % (D / 8);
                        if (row < rows)
                            *reinterpret_cast<uint4*>(out + row * a.O_row + unit * 8) =
                                *reinterpret_cast<const uint4*>(mine + (unit >> 3) * 4096 + row * 128 + (((unit & 7) ^ (row & 7)) << 4));
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) tma_store_wait_read_all();
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        const int h = (warp - 8) >> 2;
        const int r = threadIdx.x - 256 - h * 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + 128 * h, t_o = tmem + lanes + kColO + 128 * h;
        float* sums = reinterpret_cast<float*>(smem + L::kSums) + h * 256 + r;
        uint32_t items = 0;
        const float c = a.s.scale_log2;
        uint32_t steps = 0;  // tiles of this half so far
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const Item t = item_at(a, i);
            if (t.rows <= h * kHalfRows || t.n == 0) continue;
            float m = 0.0f, l = 0.0f;
            for (int j = 0; j < t.n; ++j, ++steps) {
                if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full + h, steps & 1, a.status)))) break;
                tc_fence_after();
                const int left = t.valid - j * kKeyTile;
                auto pass = [&](auto masked_tag) -> bool {
                    constexpr bool MASKED = decltype(masked_tag)::value;
                    // 64 columns at a time, twice over for the first tile's maximum
                    uint32_t pk[64];
                    auto load = [&](uint32_t (&s)[2][32], int hf) {
                        BSS_TMEM_LD32(t_s + 64 * hf, s[0]);
                        BSS_TMEM_LD32(t_s + 64 * hf + 32, s[1]);
                        tmem_wait_ld();
                        if constexpr (MASKED) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int valid = left - 64 * hf - 32 * q;
                                if (valid < 32) {
#pragma unroll
                                    for (int x = 0; x < 32; ++x)
                                        if (x >= valid) s[q][x] = 0xFF800000u;  // minus infinity
                                }
                            }
                        }
                    };
                    if (j == 0) {
                        float mx[4];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t s[2][32];
                            load(s, hf);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float& top = mx[2 * hf + q];
                                top = __uint_as_float(s[q][0]);
#pragma unroll
                                for (int x = 1; x < 32; ++x) top = fmaxf(top, __uint_as_float(s[q][x]));
                            }
                        }
                        m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                    }
                    const float ref = m == -INFINITY ? 0.0f : m;
                    const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-ref, -ref);
                    uint64_t sum_a = 0ull, sum_b = 0ull;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t s[2][32];
                        load(s, hf);
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            float y0, y1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[x >> 4][2 * (x & 15)]), __uint_as_float(s[x >> 4][2 * (x & 15) + 1])), c2, nm2), y0, y1);
                            const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                            if (x & 1) sum_b = f2_add(sum_b, f2_pack(p0, p1));
                            else sum_a = f2_add(sum_a, f2_pack(p0, p1));
                            pk[32 * hf + x] = pack_bf16x2(p0, p1);
                        }
                    }
                    float a0, a1, b0, b1;
                    f2_unpack(sum_a, a0, a1);
                    f2_unpack(sum_b, b0, b1);
                    const float sum = (a0 + a1) + (b0 + b1);
                    if (j > 0 && __any_sync(0xFFFFFFFFu, sum > kSumLimit || m == -INFINITY)) return false;
                    l += sum;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) BSS_TMEM_ST16(t_s + 16 * q4, (pk + 16 * q4));
                    return true;
                };
                const bool done = left >= kKeyTile ? pass(std::false_type()) : pass(std::true_type());
                if (!done) {
                    // the reference moves: the tile's maximum, then O and l by what it moved
                    float top = -INFINITY;
#pragma unroll 1
                    for (int cc = 0; cc < 4 && cc * 32 < left; ++cc) {
                        uint32_t s[32];
                        BSS_TMEM_LD32(t_s + 32 * cc, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (cc * 32 + x < left) top = fmaxf(top, __uint_as_float(s[x]));
                    }
                    const float m_new = fmaxf(top * c, m);
                    const float alpha = m_new == m ? 1.0f : ex2_approx(m - m_new);
                    const float ref = m_new == -INFINITY ? 0.0f : m_new;
                    // PV_h(j-1) was issued before S_h(j): it has completed
                    if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done + h, (steps - 1) & 1, a.status)))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        BSS_TMEM_LD32(t_o + cc * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                        BSS_TMEM_ST32(t_o + cc * 32, o);
                    }
                    float sum = 0.0f;
#pragma unroll 1
                    for (int cc = 0; cc < 4 && cc * 32 < left; ++cc) {
                        uint32_t s[32], pk[16];
                        BSS_TMEM_LD32(t_s + 32 * cc, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float x0 = cc * 32 + 2 * x < left ? __uint_as_float(s[2 * x]) : -INFINITY;
                            const float x1 = cc * 32 + 2 * x + 1 < left ? __uint_as_float(s[2 * x + 1]) : -INFINITY;
                            const float p0 = ex2_approx(fmaf(x0, c, -ref)), p1 = ex2_approx(fmaf(x1, c, -ref));
                            sum += p0 + p1;
                            pk[x] = pack_bf16x2(p0, p1);
                        }
                        BSS_TMEM_ST16(t_s + 16 * cc, pk);
                    }
                    l = l * alpha + sum;
                    m = m_new;
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + h);
            }
            if (!ok) break;
            // (the buffer before last: its O was read before this item's products began)
            sums[(items & 1) * 128] = l;
            mbar_arrive(l_full + 2 * h + (items & 1));
            ++items;
            if (a.lse != nullptr && h * kHalfRows + r < t.rows)
                a.lse[static_cast<int64_t>(t.head) * a.s.rows + static_cast<int64_t>(t.group) * a.s.group_rows + t.row0 + h * kHalfRows + r] =
                    l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
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

// ---------------------------------------------------------------- few rows
// A few rows a group fill no tile: a block takes a row and head, in 32 bits, eight lanes a
// key, eight keys a warp at once; every eight lanes keep their own maximum and sums, which
// are brought to one maximum at the end, in a fixed order.  Taken while every row and head
// has an SM.  Heads of 128 over 64 / 512 / 2,048 / 8,192 states, us on the device, without
// tiles and with: 10 rows and heads 2.7 / 5.3 / 14.6 / 51 and 4.8 / 8.1 / 22.5 / 80, 80 of
// them 2.8 / 5.5 / 14.9 / 52 and 4.9 / 8.2 / 22.5 / 80, 150 of them 2.8 / 5.6 / 15.2 / 52 and
// 5.0 / 8.3 / 22.7 / 80; 160 of them, a second round of blocks, 10.2 over 512 and 8.4.  Tiles
// would be faster only where each row has states of its own that leave L2 together (150 rows and
// heads, 2,048 states each, 157 MB: 30.1 and 27.5); 32 bits are kept there.  Bound by a round's
// chain of load, sum of eight lanes and exponentials (0.4 us for 128 keys).
struct FewArgs {
    CrossShape s;
    const uint16_t *q, *k, *v;
    uint16_t* O;
    int64_t q_row, q_head, O_row, O_head, k_group, k_token, k_head, v_group, v_token, v_head;
    float* lse;
};

template <int D>
__global__ void __launch_bounds__(kFewThreads) cross_few_forward_kernel(const __grid_constant__ FewArgs a) {
    constexpr int N = D / 64;
    __shared__ float sums[kFewWarps][D], tops[kFewWarps], totals[kFewWarps];
    const int warp = threadIdx.x >> 5, unit = threadIdx.x & 7, slot = (threadIdx.x >> 3) & 3;
    cudaGridDependencySynchronize();
    const int row = blockIdx.x / a.s.heads, h = blockIdx.x - row * a.s.heads, kv = h / a.s.share;
    const int group = row / a.s.group_rows, n = a.s.valid(group);
    float q[8 * N], sum[8 * N] = {}, m = -INFINITY, l = 0.0f;
    load_part<N>(a.q + row * a.q_row + h * a.q_head, unit, q);
    const uint16_t* k = a.k + group * a.k_group + kv * a.k_head;
    const uint16_t* v = a.v + group * a.v_group + kv * a.v_head;
    for (int first = warp * 8; first < n; first += kFewWarps * 8) {
        float x[2][8 * N], y[2][8 * N], s[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t key = min(first + 4 * j + slot, n - 1);
            load_part<N>(k + key * a.k_token, unit, x[j]);
            load_part<N>(v + key * a.v_token, unit, y[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j] = dot_part<N>(q, x[j]) * a.s.scale_log2;
            if (first + 4 * j + slot >= n) s[j] = -INFINITY;
        }
        const float top = fmaxf(m, fmaxf(s[0], s[1])), ref = top == -INFINITY ? 0.0f : top;
        const float alpha = ex2_approx(m - ref);
        m = top;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < 8 * N; ++i) sum[i] *= alpha;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float p = ex2_approx(s[j] - ref);
            l += p;
            if (first + 4 * j + slot < n)
#pragma unroll
                for (int i = 0; i < 8 * N; ++i) sum[i] = fmaf(p, y[j][i], sum[i]);
        }
    }
    float top = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
    const float part = ex2_approx(m - (top == -INFINITY ? 0.0f : top));
    l *= part;
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) {
        sum[i] *= part;
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 8);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 16);
        if (slot == 0) sums[warp][8 * (unit + 8 * (i / 8)) + i % 8] = sum[i];
    }
    if (slot == 0 && unit == 0) tops[warp] = top, totals[warp] = l;
    __syncthreads();
    if (threadIdx.x >= 8) return;
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, tops[w]);
    const float ref = top == -INFINITY ? 0.0f : top;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) sum[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
        const float of = ex2_approx(tops[w] - ref);
        l = fmaf(of, totals[w], l);
#pragma unroll
        for (int i = 0; i < 8 * N; ++i) sum[i] = fmaf(of, sums[w][8 * (unit + 8 * (i / 8)) + i % 8], sum[i]);
    }
    store_part<N>(a.O + row * a.O_row + h * a.O_head, unit, sum, l == 0.0f ? 0.0f : 1.0f / l);
    if (a.lse != nullptr && unit == 0)
        a.lse[static_cast<int64_t>(h) * a.s.rows + row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
}

template <int D>
bss_status launch_forward(CrossArgs& a, cudaStream_t stream) {
    auto kernel = cross_forward_kernel<D>;
    int blocks;
    const bss_status st = resident_blocks(reinterpret_cast<const void*>(kernel), kThreads, CrossSmem<D>::kBytes, &blocks);
    if (st != BSS_OK) return st;
    const int grid = a.items < num_sms() ? a.items : num_sms();
    return launch_behind_with(kernel, dim3(static_cast<unsigned>(grid)), kThreads, CrossSmem<D>::kBytes, 1, stream,
                              "cross attention launch", a);
}

}  // namespace

// ---------------------------------------------------------------- checks of both passes
bss_status check_cross_sizes(int64_t rows, int64_t* rows_per_group, int32_t heads, int32_t kv_heads, int32_t head_dim,
                             int32_t keys, float softmax_scale, const int32_t* lengths) {
    if (rows <= 0 || *rows_per_group <= 0) return set_error(BSS_ERR_INVALID_ARG, "rows and rows_per_group must be positive");
    if (rows > 0x7FFFFFFF - 256) return set_error(BSS_ERR_UNSUPPORTED, "rows must be below 2^31 - 256");
    if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0)
        return set_error(BSS_ERR_INVALID_ARG, "kv_heads must divide heads (got %d, %d)", heads, kv_heads);
    if (heads > 65535) return set_error(BSS_ERR_UNSUPPORTED, "more than 65535 heads");
    if (head_dim != 64 && head_dim != 128)
        return set_error(BSS_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", head_dim);
    if (keys <= 0) return set_error(BSS_ERR_INVALID_ARG, "keys must be positive");
    if (keys > 0x7FFFFFFF - 256) return set_error(BSS_ERR_UNSUPPORTED, "keys must be below 2^31 - 256");
    if (!std::isfinite(softmax_scale)) return set_error(BSS_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (!is_aligned(lengths, 4)) return set_error(BSS_ERR_INVALID_ARG, "lengths must be 4-byte aligned");
    if (*rows_per_group > rows) *rows_per_group = rows;
    return BSS_OK;
}

bss_status check_row_heads(Operand* o, const bss_token_tensor& t, const char* name, int64_t rows, int32_t heads, int32_t d,
                           bool output) {
    o->p = t.data;
    o->name = name;
    o->output = output;
    if (t.data == nullptr) return set_error(BSS_ERR_INVALID_ARG, "%s is NULL", name);
    if (!is_aligned(t.data, 16)) return set_error(BSS_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    const int64_t ts = rows > 1 ? t.token_stride : 8, hs = heads > 1 ? t.head_stride : 8;
    if (ts % 8 != 0 || hs % 8 != 0 || ts <= 0 || hs <= 0 || ts > kMaxRowStride || hs > kMaxStateStride)
        return set_error(BSS_ERR_INVALID_ARG,
                         "%s: strides must be positive multiples of 8 elements, a token's at most 2^28, a head's 2^38", name);
    o->r = region_3d(t.data, rows, ts, heads, hs, d, 2);
    if (output && o->r.self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s: rows or heads overlap", name);
    return BSS_OK;
}

bss_status check_states(Operand* o, const bss_state_tensor& t, const char* name, int64_t groups, int64_t keys, int32_t heads,
                        int32_t d, bool output) {
    o->p = t.data;
    o->name = name;
    o->output = output;
    if (t.data == nullptr) return set_error(BSS_ERR_INVALID_ARG, "%s is NULL", name);
    if (!is_aligned(t.data, 16)) return set_error(BSS_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    int64_t gs = t.group_stride, ts = t.token_stride, hs = t.head_stride;
    if (!output && gs == 0) groups = 1;
    if (groups <= 1) gs = 8;
    if (keys <= 1) ts = 8;
    if (heads <= 1) hs = 8;
    if (gs % 8 != 0 || ts % 8 != 0 || hs % 8 != 0 || gs <= 0 || ts <= 0 || hs <= 0 || ts > kMaxRowStride ||
        hs > kMaxStateStride || gs > kMaxStateStride)
        return set_error(BSS_ERR_INVALID_ARG,
                         "%s: strides must be positive multiples of 8 elements, a token's at most 2^28, the others 2^38", name);
    // the last byte's address must exist
    const unsigned __int128 end = static_cast<unsigned __int128>(groups - 1) * gs + static_cast<unsigned __int128>(keys - 1) * ts +
                                  static_cast<unsigned __int128>(heads - 1) * hs + d;
    if (end > (static_cast<unsigned __int128>(1) << 50)) return set_error(BSS_ERR_INVALID_ARG, "%s: strides too large", name);
    // two of the four dimensions taken as one where they can be
    if (heads <= 1 || hs == d) {
        o->r = region_3d(t.data, groups, gs, keys, ts, static_cast<int64_t>(heads) * d, 2);
    } else if (keys <= 1 || ts == d) {
        o->r = region_3d(t.data, groups, gs, heads, hs, keys * d, 2);
    } else if (groups <= 1 || gs == keys * ts) {
        o->r = region_3d(t.data, groups * keys, ts, heads, hs, d, 2);
    } else {
        if (output) return set_error(BSS_ERR_UNSUPPORTED, "%s: groups, tokens and heads all apart", name);
        o->r = region_2d(t.data, 1, 0, static_cast<int64_t>(end), 2);
    }
    if (output && o->r.self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s: groups, tokens or heads overlap", name);
    return BSS_OK;
}

CrossShape cross_shape(int64_t rows, int64_t rows_per_group, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t keys,
                       float softmax_scale, const int32_t* lengths, int64_t group_stride) {
    CrossShape s;
    s.rows = static_cast<int32_t>(rows);
    s.group_rows = static_cast<int32_t>(rows_per_group);
    s.groups = static_cast<int32_t>((rows + rows_per_group - 1) / rows_per_group);
    s.heads = heads, s.kv_heads = kv_heads, s.share = heads / kv_heads;
    s.keys = keys;
    s.shared_states = group_stride == 0 || s.groups == 1;
    s.lengths = lengths;
    s.by_heads = FastDiv(static_cast<uint32_t>(heads));
    s.by_share = FastDiv(static_cast<uint32_t>(s.share));
    s.scale_log2 = (softmax_scale > 0.0f ? softmax_scale : 1.0f / sqrtf(static_cast<float>(head_dim))) * 1.4426950408889634f;
    return s;
}

bss_status row_heads_map(CUtensorMap* map, const bss_token_tensor& t, int64_t rows, int32_t heads, int32_t d, int box) {
    const uint64_t ts = static_cast<uint64_t>(rows > 1 ? t.token_stride : 8) * 2;
    const uint64_t hs = static_cast<uint64_t>(heads > 1 ? t.head_stride : 8) * 2;
    return encode_tmap_3d(map, t.data, d, rows, heads, ts, hs, 64, box);
}

bss_status states_map(CUtensorMap* map, const bss_state_tensor& t, int64_t groups, int64_t keys, int32_t heads, int32_t d,
                      int box) {
    if (t.group_stride == 0) groups = 1;
    return encode_tmap_4d(map, t.data,
                          {static_cast<uint64_t>(d), static_cast<uint64_t>(keys), static_cast<uint64_t>(heads),
                           static_cast<uint64_t>(groups)},
                          {static_cast<uint64_t>(t.token_stride) * 2, static_cast<uint64_t>(t.head_stride) * 2,
                           static_cast<uint64_t>(t.group_stride) * 2},
                          64, box);
}

}  // namespace bss

extern "C" {

bss_status bss_cross_attention(const bss_cross_args* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_cross_args p = *args;
    bss_status st = check_cross_sizes(p.rows, &p.rows_per_group, p.heads, p.kv_heads, p.head_dim, p.keys, p.softmax_scale, p.lengths);
    if (st != BSS_OK) return st;
    const int64_t groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
    Operand t[6];
    if ((st = check_row_heads(&t[0], p.q, "q", p.rows, p.heads, p.head_dim, false)) != BSS_OK ||
        (st = check_states(&t[1], p.k, "k", groups, p.keys, p.kv_heads, p.head_dim, false)) != BSS_OK ||
        (st = check_states(&t[2], p.v, "v", groups, p.keys, p.kv_heads, p.head_dim, false)) != BSS_OK ||
        (st = check_run(&t[3], p.lengths, "lengths", 4 * groups, 4, false)) != BSS_OK ||
        (st = check_row_heads(&t[4], p.O, "O", p.rows, p.heads, p.head_dim, true)) != BSS_OK ||
        (st = check_run(&t[5], p.lse, "lse", 4 * p.rows * p.heads, 4, true)) != BSS_OK)
        return st;
    // over q only element by element (with as many rows as heads a transposed view has the same bytes)
    if ((p.rows <= 1 || p.O.token_stride == p.q.token_stride) && (p.heads <= 1 || p.O.head_stride == p.q.head_stride)) t[4].over = 0;
    if ((st = check_outputs(t, 6)) != BSS_OK) return st;
    if ((p.k.group_stride == 0) != (p.v.group_stride == 0) && groups > 1)
        return set_error(BSS_ERR_UNSUPPORTED, "k and v must both be shared by the groups, or neither");
    const CrossShape shape = cross_shape(p.rows, p.rows_per_group, p.heads, p.kv_heads, p.head_dim, p.keys, p.softmax_scale,
                                         p.lengths, p.k.group_stride);
    auto stride = [](int64_t extent, int64_t s) { return extent > 1 ? s : 0; };
    if (p.rows * p.heads <= num_sms()) {
        FewArgs f;
        memset(&f, 0, sizeof(f));
        f.s = shape, f.lse = p.lse;
        f.q = static_cast<const uint16_t*>(p.q.data), f.O = static_cast<uint16_t*>(p.O.data);
        f.k = static_cast<const uint16_t*>(p.k.data), f.v = static_cast<const uint16_t*>(p.v.data);
        f.q_row = stride(p.rows, p.q.token_stride), f.q_head = stride(p.heads, p.q.head_stride);
        f.O_row = stride(p.rows, p.O.token_stride), f.O_head = stride(p.heads, p.O.head_stride);
        f.k_group = stride(groups, p.k.group_stride), f.v_group = stride(groups, p.v.group_stride);
        f.k_token = stride(p.keys, p.k.token_stride), f.v_token = stride(p.keys, p.v.token_stride);
        f.k_head = stride(p.kv_heads, p.k.head_stride), f.v_head = stride(p.kv_heads, p.v.head_stride);
        return launch_behind(p.head_dim == 128 ? cross_few_forward_kernel<128> : cross_few_forward_kernel<64>,
                             dim3(static_cast<unsigned>(p.rows * p.heads)), kFewThreads, stream, "few rows' attention launch", f);
    }
    const int64_t tiles = (p.rows_per_group + 255) / 256, items = groups * tiles * p.heads;
    if (items > 0x7FFFFFFF - 4096) return set_error(BSS_ERR_UNSUPPORTED, "too many rows and heads");
    CrossArgs a;
    memset(&a, 0, sizeof(a));
    const int64_t whole = p.rows / p.rows_per_group, rest = p.rows - whole * p.rows_per_group;
    auto queries_map = [&](CUtensorMap* map, int64_t group, int64_t rows, int64_t groups) {
        const uint64_t row = static_cast<uint64_t>(stride(p.rows, p.q.token_stride)) * 2;
        return encode_tmap_4d(map, static_cast<const char*>(p.q.data) + group * p.rows_per_group * row,
                              {static_cast<uint64_t>(p.head_dim), static_cast<uint64_t>(rows), static_cast<uint64_t>(p.heads),
                               static_cast<uint64_t>(groups)},
                              {row, static_cast<uint64_t>(p.q.head_stride) * 2, static_cast<uint64_t>(p.rows_per_group) * row}, 64,
                              kHalfRows);
    };
    if ((st = queries_map(&a.q, 0, p.rows_per_group, whole)) != BSS_OK ||
        (rest > 0 && (st = queries_map(&a.q_rest, whole, rest, 1)) != BSS_OK) ||
        (st = row_heads_map(&a.o, p.O, p.rows, p.heads, p.head_dim, 32)) != BSS_OK ||
        (st = states_map(&a.k, p.k, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK ||
        (st = states_map(&a.v, p.v, groups, p.keys, p.kv_heads, p.head_dim, kKeyTile)) != BSS_OK)
        return st;
    a.s = shape;
    a.whole = static_cast<int32_t>(whole);
    a.tiles = static_cast<int32_t>(tiles);
    a.items = static_cast<int32_t>(items);
    a.by_tiles = FastDiv(static_cast<uint32_t>(a.tiles));
    a.O = static_cast<uint16_t*>(p.O.data);
    a.O_row = stride(p.rows, p.O.token_stride);
    a.O_head = stride(p.heads, p.O.head_stride);
    a.lse = p.lse;
    a.status = device_status_ptr();
    if (a.status == nullptr) return set_error(BSS_ERR_CUDA, "cannot resolve the device status word");
    return p.head_dim == 128 ? launch_forward<128>(a, stream) : launch_forward<64>(a, stream);
}

}  // extern "C"
