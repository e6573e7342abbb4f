// paged_prefill_tc.cu -- attention of several new tokens per sequence over a
// paged K/V cache on the tcgen05 tensor cores (the same function as
// paged_prefill.cu, for calls with rows enough to fill its tiles).
//
// One CTA holds two 128-row query tiles A and B of one (sequence, kv head).  The G
// query heads of a kv head share its keys, so a tile's rows are (token, head)
// pairs, row r = token r / G, head r % G: a tile spans 128 / G tokens, so little
// of its last key tile lies beyond the causal border, and each K / V tile that
// TMA brings serves all heads of the group.  Per key tile of 128 keys and query
// tile: S = Q K^T into TMEM, one thread per row takes p = 2^(s - m) and writes P
// (bf16 / f16) back to TMEM, O += P V accumulates there.  The reference maximum m
// moves (and O, l are rescaled) only when a tile's maximum passes it by more than
// 2^8.  While one tile's rows are exponentiated the tensor cores work for the
// other.
//
// K and V tiles are read from the pages as they lie, one TMA box (64 elements x
// up to 128 rows of a page) at a time, 128-byte swizzled: as K-major operand of
// the first product, and as MN-major operand of the second (V needs no
// transposed copy).  Boxes of pages that no row sees point beyond the pool, which
// TMA fills with zeros without reading anything; so does a bad page number.  In
// the tiles at the edges (the last one, the ends of the sinks and the window's
// start) the MMA warp zeroes the V rows that no row sees, since 0 * NaN from a
// stale row would not be 0.
//
// P is rounded to the cache's type, bf16 2^-9 of each weight at most, which in a
// sum over keys of mixed sign is about the output's own rounding; l is summed
// from the unrounded weights in f32.
//
// Warps 0-3: tile A; warps 4-7: tile B (a warp reads the TMEM lanes of its index
// mod 4); warp 8: TMA producer; warp 9: TMEM allocation, edge rows, MMA issue;
// warps 10 and 11 only complete the warpgroup that gives up registers.  A row's
// 128 scores stand in registers at once: their maximum, then one fused
// multiply-add and one exponential each, so a thread needs more registers (200)
// than the other warps (104).  Every mbarrier wait is bounded; a timeout raises
// EMBER_ERR_TIMEOUT, the CTA drains its copies and frees TMEM.
#include <cudaTypedefs.h>

#include "paged.cuh"
#include "tc_common.cuh"

namespace ember {

namespace {

constexpr int PT_THREADS = 384;
constexpr int PT_TMA = 8, PT_MMA = 9;   // warps
constexpr int PT_REGS_ROW = 200, PT_REGS_REST = 104;   // 256 * 200 + 128 * 104 = 384 * 168, the launch's share
constexpr int PT_ROWS = 128;   // rows of a query tile
constexpr int PT_KEYS = 128;   // keys of a tile

template <int DP>
struct PtSmem {
    static constexpr int KB = DP / 64;                    // 64-element blocks of a row
    static constexpr int TILE = KB * 128 * 128;           // Q tile, K tile or V tile
    static constexpr int NSTG = DP == 64 ? 4 : 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = 2 * TILE;               // stage: K tile, V tile
    static constexpr int OFF_BAR = OFF_KV + NSTG * 2 * TILE;
    static constexpr int TOTAL = OFF_BAR + 256 + 1024;    // + barriers, + alignment slack
    // TMEM columns: S_A, S_B (128 f32 each), O_A, O_B (DP f32 each); P (128
    // values, two to a column) in its own columns for DP 64, over S for DP 128
    static constexpr bool ALIAS = DP == 128;
    static constexpr uint32_t COL_S = 0, COL_O = 256;
    static constexpr uint32_t col_p(int t) { return ALIAS ? COL_S + t * 128 : 384 + t * 64; }
};

// Descriptor of an MN-major operand written by TMA with the 128-byte swizzle:
// 64 elements of M/N to a 128-byte row, 8-row groups of K 1024 bytes apart
// (stride offset), the next 64 elements `lead` bytes further (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lead) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3ffffu) >> 4);
    d |= (uint64_t)(lead >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
constexpr uint32_t IDESC_B_MN = 1u << 16;   // B is MN-major

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

template <class E, int DP>
__global__ void __launch_bounds__(PT_THREADS, 1)
    k_paged_prefill_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       PagedPrefillArgs a) {
    using L = PtSmem<DP>;
    constexpr int NSTG = L::NSTG;
    extern __shared__ uint8_t pt_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pt_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
    uint64_t* q_full = bar + 0;
    uint64_t* s_full = bar + 1;     // [2] per query tile
    uint64_t* p_full = bar + 3;     // [2]
    uint64_t* o_full = bar + 5;     // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 7);
    int* sflag = reinterpret_cast<int*>(bar + 8);   // [0] failed, [1] tiles issued, [2] tiles consumed
    uint64_t* kv_full = bar + 10;   // [NSTG]
    uint64_t* kv_empty = bar + 16;  // [NSTG]
    uint64_t* s_free = bar + 22;    // [2] the row values of S are in registers (P beside S only)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.c.D, G = a.NH / a.c.NKV, g = blockIdx.y;
    const int QT = PT_ROWS / G;                        // tokens of a query tile
    pdl_wait();
    // the last tiles see the most keys: they go first
    const int x = (int)(gridDim.x - 1 - blockIdx.x);
    const RowTile tile = find_row_tile(a, 2 * QT, x, x == 0 && g == 0 && warp == 0);
    if (tile.b < 0) return;
    const SeqRows sr = seq_rows(a, tile.b, false);
    const int i0 = tile.i * 2 * QT;                    // first token of tile A
    const int tokens = min(2 * QT, sr.nq - i0);
    const int pos0 = sr.len - sr.nq + i0;              // its position (negative: sees nothing)
    // keys that some row sees: [first, end) and [0, sinks); in tiles of 128
    const int end = pos0 + tokens;
    const int first = a.window > 0 ? max(0, pos0 + 1 - a.window) : 0;
    const int sinks = min(a.sinks, first);
    const int ns = (sinks + PT_KEYS - 1) / PT_KEYS;
    const int wb = max(first / PT_KEYS, ns);
    const int nkt = end <= 0 ? 0 : ns + max(0, (end + PT_KEYS - 1) / PT_KEYS - wb);
    auto key0_of = [&](int j) { return PT_KEYS * (j < ns ? j : wb + j - ns); };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 256);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 128);
            mbar_init(&s_free[t], 128);
            mbar_init(&o_full[t], 1);
        }
        for (int s = 0; s < NSTG; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        sflag[0] = 0;
        sflag[1] = 0;
        sflag[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == PT_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= PT_TMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PT_REGS_REST));
    if (warp == PT_TMA) {   // ------------------------------------- TMA producer
        const int P = 1 << a.c.page_shift;
        const int box = min(P, PT_KEYS);               // rows of a box
        const int boxes = PT_KEYS / box;               // of a tile: lane i < boxes copies box i
        auto look_up = [&](int j) {                    // the lane's page of tile j; n_pages reads as zeros
            const int k0 = key0_of(j) + lane * box;
            if (lane >= boxes || k0 >= end || (k0 + box <= first && k0 >= sinks)) return a.c.n_pages;
            const int page = a.c.table[(size_t)sr.seq * a.c.width + (k0 >> a.c.page_shift)];
            if (page >= 0 && page < a.c.n_pages) return page;
            raise_status(a.status, EMBER_ERR_INVALID_ARG);
            return a.c.n_pages;
        };
        int page = nkt > 0 ? look_up(0) : 0;
        int issued = 0;
        bool fail = false;
        for (; issued < nkt; ++issued) {
            const int s = issued % NSTG;
            if (issued >= NSTG && !mbar_wait(&kv_empty[s], (uint32_t)(issued / NSTG - 1) & 1u)) fail = true;
            if (__any_sync(FULL_MASK, fail)) {
                fail = true;
                break;
            }
            if (lane == 0) mbar_expect_tx(&kv_full[s], 2 * L::TILE);
            __syncwarp();
            if (lane < boxes) {
                const int row = (key0_of(issued) + lane * box) & (P - 1);
                uint8_t* kd = sm + L::OFF_KV + s * 2 * L::TILE + lane * box * 128;
#pragma unroll
                for (int kb = 0; kb < L::KB; ++kb) {
                    tma_load_4d(kd + kb * 128 * 128, &tmK, kb * 64, row, g, page, &kv_full[s]);
                    tma_load_4d(kd + L::TILE + kb * 128 * 128, &tmV, kb * 64, row, g, page, &kv_full[s]);
                }
            }
            if (issued + 1 < nkt) page = look_up(issued + 1);
        }
        if (lane == 0) {
            if (fail) sflag[0] = 1;
            sflag[1] = issued;
        }
    } else if (warp == PT_MMA) {   // ------------------------------ MMA issuer
        constexpr uint32_t type = E::bf16 ? idesc_bf16(0, 0) : idesc_f16(0, 0);
        constexpr uint32_t idS = type | idesc_f16(PT_ROWS, PT_KEYS);
        constexpr uint32_t idO = type | idesc_f16(PT_ROWS, DP) | IDESC_B_MN;
        auto mma_s = [&](int t, int s) {   // S_t = Q_t . K(stage s)^T
            const uint32_t q0 = smem_u32(sm + L::OFF_Q + t * L::TILE);
            const uint32_t k0 = smem_u32(sm + L::OFF_KV + s * 2 * L::TILE);
#pragma unroll
            for (int kb = 0; kb < L::KB; ++kb)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16(tmem + L::COL_S + t * 128, sdesc_sw128(q0 + kb * 128 * 128 + k * 32),
                              sdesc_sw128(k0 + kb * 128 * 128 + k * 32), idS, (kb | k) ? 1u : 0u);
            umma_commit(&s_full[t]);
        };
        auto mma_pv = [&](int t, int s, bool acc) {   // O_t += P_t (TMEM) . V(stage s)
            const uint32_t v0 = smem_u32(sm + L::OFF_KV + s * 2 * L::TILE + L::TILE);
#pragma unroll
            for (int k = 0; k < PT_KEYS / 16; ++k)
                umma_f16_ts(tmem + L::COL_O + t * DP, tmem + L::col_p(t) + k * 8,
                            sdesc_mn_sw128(v0 + k * 16 * 128, 128 * 128), idO, (acc || k) ? 1u : 0u);
            umma_commit(&o_full[t]);
        };
        // waits for K and V of tile j; V rows that nobody sees become zeros
        auto kv_ready = [&](int j) {
            const int s = j % NSTG;
            if (!mbar_wait(&kv_full[s], (uint32_t)(j / NSTG) & 1u)) return false;
            const int key0 = key0_of(j);
            if (key0 + PT_KEYS > end || (key0 < first && key0 + PT_KEYS > sinks)) {
                uint8_t* v = sm + L::OFF_KV + s * 2 * L::TILE + L::TILE;
                for (int i = lane; i < PT_KEYS * 8 * L::KB; i += 32) {   // a 16-byte piece of a row each
                    const int r = i / (8 * L::KB), c = i % (8 * L::KB), key = key0 + r;
                    if (key >= end || (key < first && key >= sinks))
                        *reinterpret_cast<uint4*>(v + (c >> 3) * 128 * 128 + r * 128 + (c & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            return true;
        };
        bool ok = mbar_wait(q_full, 0) && (nkt == 0 || kv_ready(0));
        ok = __all_sync(FULL_MASK, ok);
        int j = 0;
        if (ok && nkt > 0 && lane == 0) {
            tc_fence_after();
            mma_s(0, 0);
            mma_s(1, 0);
        }
        __syncwarp();
        for (; ok && j < nkt; ++j) {
            const int s = j % NSTG;
            const bool more = j + 1 < nkt;
            const int s1 = (j + 1) % NSTG;
            bool in = true;
            if (L::ALIAS) {
                // P lies over S: P . V(j) of a query tile goes before its S(j + 1)
                // (MMAs of one thread run in the order of issue)
                in = mbar_wait(&p_full[0], (uint32_t)j & 1u);
                if (!__all_sync(FULL_MASK, in)) break;
                if (lane == 0) {
                    tc_fence_after();
                    mma_pv(0, s, j > 0);
                }
                __syncwarp();
                if (more) {
                    in = kv_ready(j + 1);
                    if (!__all_sync(FULL_MASK, in)) break;
                    if (lane == 0) {
                        tc_fence_after();
                        mma_s(0, s1);
                    }
                    __syncwarp();
                }
                in = mbar_wait(&p_full[1], (uint32_t)j & 1u);
                if (!__all_sync(FULL_MASK, in)) break;
                if (lane == 0) {
                    tc_fence_after();
                    mma_pv(1, s, j > 0);
                    if (more) mma_s(1, s1);
                }
            } else {
                // S(j + 1) as soon as the rows of S(j) are in registers, while they
                // are exponentiated
                if (more) {
                    in = kv_ready(j + 1);
                    if (!__all_sync(FULL_MASK, in)) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        in = in && mbar_wait(&s_free[t], (uint32_t)j & 1u);
                        if (!__all_sync(FULL_MASK, in)) break;
                        if (lane == 0) {
                            tc_fence_after();
                            mma_s(t, s1);
                        }
                        __syncwarp();
                    }
                    if (!__all_sync(FULL_MASK, in)) break;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    in = in && mbar_wait(&p_full[t], (uint32_t)j & 1u);
                    if (!__all_sync(FULL_MASK, in)) break;
                    if (lane == 0) {
                        tc_fence_after();
                        mma_pv(t, s, j > 0);
                    }
                    __syncwarp();
                }
                if (!__all_sync(FULL_MASK, in)) break;
            }
            if (lane == 0) umma_commit(&kv_empty[s]);
            __syncwarp();
        }
        if (lane == 0) {
            if (!ok || j < nkt) sflag[0] = 1;
            sflag[2] = j;
        }
    }
    } else {   // -------------------------------------------------- softmax warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PT_REGS_ROW));
        constexpr float RESCALE = 8.f;
        const int t = warp >> 2;                      // query tile: 0 = A, 1 = B
        const int qw = warp & 3;                      // TMEM lane quarter of this warp
        const int r = qw * 32 + lane;                 // row within the tile
        const int tok = t * QT + r / G, h = r % G;    // token of the pair, head of the group
        const bool live = r < QT * G && tok < tokens;
        const int qp = pos0 + min(tok, tokens - 1);   // its position (rows that are not live: the last one's)
        const long long row = sr.row0 + i0 + tok;
        {   // the row's q into its swizzled tile (rows that are not live: zeros); a
            // negative scale becomes its sign, so that the largest score is the largest product
            const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
            const uint4* q = reinterpret_cast<const uint4*>(a.q + row * a.ld_q + (long long)(g * G + h) * D);
            uint8_t* d = sm + L::OFF_Q + t * L::TILE + r * 128;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
                uint4 v = live && c * 8 < D ? __ldcg(q + c) : make_uint4(0u, 0u, 0u, 0u);
                v.x ^= sign;
                v.y ^= sign;
                v.z ^= sign;
                v.w ^= sign;
                *reinterpret_cast<uint4*>(d + (c >> 3) * 128 * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(q_full);
        }
        const uint32_t lane_off = (uint32_t)(qw * 32) << 16;
        const uint32_t tS = tmem + L::COL_S + t * 128 + lane_off;
        const uint32_t tO = tmem + L::COL_O + t * DP + lane_off;
        const uint32_t tP = tmem + L::col_p(t) + lane_off;
        const float sc = fabsf(a.scale) * LOG2E;
        float m = SOFTMAX_FLOOR, l = 0.f;             // reference maximum (of s * sc), sum of 2^(s sc - m)
        bool ok = true;
        for (int j = 0; j < nkt; ++j) {
            if (!mbar_wait(&s_full[t], (uint32_t)j & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t v[PT_KEYS];                      // the row's products, then its weights
#pragma unroll
            for (int c = 0; c < PT_KEYS; c += 32) tmem_ld32(tS + c, v + c);
            tmem_ld_wait();
            if (!L::ALIAS) {
                tc_fence_before();
                mbar_arrive(&s_free[t]);
            }
            // column c is visible when c < hi and (c >= lo or c < sk)
            const int key0 = key0_of(j);
            const int hi = qp - key0 + 1;
            const int lo = a.window > 0 ? qp - a.window + 1 - key0 : 0;
            const int sk = a.sinks - key0;
            if (!__all_sync(FULL_MASK, hi >= PT_KEYS && (lo <= 0 || sk >= PT_KEYS))) {
#pragma unroll
                for (int c = 0; c < PT_KEYS; ++c)
                    if (!(c < hi && (c >= lo || c < sk))) v[c] = 0xff800000u;   // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < PT_KEYS; c += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx[i] = fmaxf(mx[i], fmaxf(__uint_as_float(v[c + 2 * i]), __uint_as_float(v[c + 2 * i + 1])));
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            // the reference moves (and O, l are rescaled) only when the tile's
            // maximum passes it by more than RESCALE (log2 units): weights stay
            // below 2^RESCALE
            const bool move = mt > m + RESCALE;
            const bool any_move = __any_sync(FULL_MASK, move);
            float corr = 1.f;
            if (any_move) {
                const float mnew = move ? mt : m;
                corr = ex2(m - mnew);
                l *= corr;
                m = mnew;
            }
            float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < PT_KEYS; c += 2) {
                const float p0 = ex2(fmaf(__uint_as_float(v[c]), sc, -m));
                const float p1 = ex2(fmaf(__uint_as_float(v[c + 1]), sc, -m));
                rs[(c >> 1) & 3] += p0 + p1;
                v[c >> 1] = E::pack(p0, p1);
            }
            if (j > 0) {   // P . V(j - 1) must be complete before O is touched or P is rewritten
                if (!mbar_wait(&o_full[t], (uint32_t)(j - 1) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (any_move) {
#pragma unroll 1
                    for (int c0 = 0; c0 < DP; c0 += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + c0, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                        tmem_st16(tO + c0, o);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < PT_KEYS / 2; c += 16) tmem_st16(tP + c, v + c);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[t]);
            l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        }
        if (ok && nkt > 0 && !mbar_wait(&o_full[t], (uint32_t)(nkt - 1) & 1u)) ok = false;
        if (!ok) sflag[0] = 1;
        tc_fence_after();
        if (ok) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t* out = a.out + row * a.ld_out + (long long)(g * G + h) * D;
#pragma unroll
            for (int c0 = 0; c0 < DP; c0 += 32) {
                if (c0 >= D) break;
                uint32_t o[32];
                if (nkt > 0) {
                    tmem_ld32(tO + c0, o);
                    tmem_ld_wait();
                }
                if (live) {
#pragma unroll
                    for (int d = 0; d < 32; d += 8) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (nkt > 0 && l != 0.f) {
                            w.x = E::pack(__uint_as_float(o[d]) * inv, __uint_as_float(o[d + 1]) * inv);
                            w.y = E::pack(__uint_as_float(o[d + 2]) * inv, __uint_as_float(o[d + 3]) * inv);
                            w.z = E::pack(__uint_as_float(o[d + 4]) * inv, __uint_as_float(o[d + 5]) * inv);
                            w.w = E::pack(__uint_as_float(o[d + 6]) * inv, __uint_as_float(o[d + 7]) * inv);
                        }
                        if (c0 + d < D) *reinterpret_cast<uint4*>(out + c0 + d) = w;
                    }
                }
            }
            if (a.lse && live) a.lse[row * a.NH + g * G + h] = l == 0.f ? -INFINITY : m * LN2 + logf(l);
        }
    }

    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if (threadIdx.x == 0 && sflag[0]) raise_status(a.status, EMBER_ERR_TIMEOUT);
    if (warp == PT_TMA && lane == 0 && sflag[0]) {
        // drain K/V copies issued but never consumed by the MMA warp
        for (int j = sflag[2]; j < sflag[1]; ++j) (void)mbar_wait(&kv_full[j % NSTG], (uint32_t)(j / NSTG) & 1u);
    }
    if (warp == PT_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

template <class E, int DP>
cudaError_t launch_dp(const void* mk, const void* mv, const PagedPrefillArgs& a, cudaStream_t s) {
    auto k = k_paged_prefill_tc<E, DP>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PtSmem<DP>::TOTAL);
    if (e != cudaSuccess) return e;
    const int per = 2 * (PT_ROWS / (a.NH / a.c.NKV));
    const dim3 grid((unsigned)(((long long)a.n + per - 1) / per + a.B), a.c.NKV);
    return launch_k(k, grid, dim3(PT_THREADS), PtSmem<DP>::TOTAL, s, *reinterpret_cast<const CUtensorMap*>(mk),
                    *reinterpret_cast<const CUtensorMap*>(mv), a);
}

}  // namespace

bool paged_prefill_maps(const PagedView& c, void* mk, void* mv) {
    const uint64_t dims[4] = {(uint64_t)c.D, 1ull << c.page_shift, (uint64_t)c.NKV, (uint64_t)c.n_pages};
    const uint64_t strides[3] = {(uint64_t)c.row_stride * 2, (uint64_t)c.head_stride * 2, (uint64_t)c.page_stride * 2};
    const uint32_t box[4] = {64u, (1u << c.page_shift) < 128u ? 1u << c.page_shift : 128u, 1u, 1u};
    return encode_map_bf16(mk, c.k, 4, dims, strides, box) && encode_map_bf16(mv, c.v, 4, dims, strides, box);
}

cudaError_t launch_paged_prefill_tc(const PagedPrefillArgs& a, const void* mk, const void* mv, cudaStream_t s) {
    if (a.c.bf16) return a.c.D <= 64 ? launch_dp<ElemBf16, 64>(mk, mv, a, s) : launch_dp<ElemBf16, 128>(mk, mv, a, s);
    return a.c.D <= 64 ? launch_dp<ElemF16, 64>(mk, mv, a, s) : launch_dp<ElemF16, 128>(mk, mv, a, s);
}

}  // namespace ember
