// adapters.cu -- a projection that all requests share, with the low-rank adapter of each
// row's own beside it:  y_i = W x_i + bias + s_a B_a (A_a x_i),  a = ids[i].
//
// Bound: for few rows the bytes of W and of the adapters that the rows name, for many rows
// the products.  Two launches: the first takes t_i = s_a A_a x_i (k_adapter with LOW, for
// little work k_adapter_rows), the second y (k_adapter without); the second starts with
// the first and streams W and x meanwhile, and waits for t only when it has come to the
// adapters.
//
// k_adapter is one tcgen05 kernel for both.  A tile is 128 rows of W (or the R rows of one A_a) by
// up to NT rows of x: the weights are the M = 128 operand, so that a few rows of x waste no
// tensor work and W streams through at the memory's rate.  The adapters of a tile's rows
// are further blocks along K: B_a's 128 rows against t, where t stands as zeros for the
// rows that have another adapter.  Only the columns from an adapter's first to its last row
// in the tile are multiplied, so rows of one request that stand together cost what they
// must, and rows in any order are right.  Each adapter is read once a tile.
//
// t goes in as the sum of two values of x's type (bf16 2^-17 relative; f16 2^-22 or 2^-25
// absolute), so that its rounding does not count beside the output's own; that costs a few
// products of K = 16 more.
//
// Few tiles split K and the adapters over the CTAs of a cluster, which join their f32 sums
// through distributed shared memory in rank order: no atomics, no workspace but t, equal
// calls give equal bits.  Many tiles run persistently, one CTA an SM, the next tile's
// products under the last one's output.
//
// Warp 0: copies; warp 1: TMEM and products; warps 2-5: output; the others: which adapters a
// tile has, and t's tiles.  Every wait is bounded; a timeout raises EMBER_ERR_TIMEOUT, the
// CTA drains its copies and frees TMEM.
#include <cudaTypedefs.h>

#include "paged.cuh"
#include "rounds.h"
#include "tc_common.cuh"

namespace ember {

namespace {

// Warps that write t's tiles, and threads of a CTA, by the tile's width.  Wide tiles of rows in any
// order are bound by that writing (256 rows of 40 adapters of rank 16 on 4096 30 us, with four warps
// 37; 777 rows of 9 of rank 32 27 and 37); narrow ones only have more threads to start (128 rows of
// 8 adapters of rank 16 on 4096 16 us, with eight 18.5).
constexpr int ad_builders(int nt) { return nt > 128 ? 8 : 4; }
constexpr int ad_threads(int nt) { return 192 + 32 * ad_builders(nt); }
constexpr int AD_M = 128;                        // rows of W in a tile
constexpr int AD_BK = 64;                        // K of a block
constexpr int AD_SLICE = 32;                     // rows of x that are put out at a time
constexpr int AD_LD = AD_M + 4;                  // their distance in shared memory, floats
// f32 outputs: the tensor cores' sums lose a little at every step, in proportion to the steps, so an
// accumulator takes at most AD_FOLD blocks of K (48 steps) before the output warps add it to a sum in
// TMEM, rounded to nearest, under the next blocks' products where there is room for a second
// accumulator.  4096 rows at K 8192: off by 0.76e-6 of the norm in 145 us; 16 blocks 1.1e-6 in 138, 8
// blocks 0.57e-6 in 157, one accumulator 9.3e-6 in 116.  The first launch's, whose t's rounding to two terms is of the same size, likewise.  Outputs of 16 bits do without: their own rounding is 1.6e-3 or 2e-4.
constexpr int AD_FOLD = 12;

template <int NT, bool LOW>
struct AdSmem {
    static constexpr int A_BYTES = AD_M * 128, X_BYTES = NT * 128, STAGE = A_BYTES + X_BYTES;
    // as many as fit, since W has to be on its way (five stages of 16 KB of W on 128 SMs, 2 us from
    // asking to having: 5 TB/s); the first launch's small ones leave room for other CTAs
    static constexpr int STAGES = LOW ? (NT == 128 ? 6 : 4) : NT == 256 ? 4 : NT == 128 ? 6 : NT == 64 ? 8 : NT == 32 ? 9 : 10;
    // an adapter's block in a stage: 16 ranks of 128 rows of B, and both terms of t's
    static constexpr int SLAB_A = AD_M * 32, SLAB_T = NT * 32, SLABS = STAGE / (SLAB_A + 2 * SLAB_T);
    static constexpr int OFF_T = SLABS * SLAB_A;
    static constexpr int OUT = AD_SLICE * AD_LD * 4;
    static constexpr int OFF_OUT = STAGES * STAGE;
    static constexpr int OFF_LIST = OFF_OUT + OUT;           // [2][NT] entries
    static constexpr int OFF_IDS = OFF_LIST + 2 * NT * 16;   // [2][NT]
    static constexpr int OFF_RUNS = OFF_IDS + 2 * NT * 4;    // [NT]
    static constexpr int OFF_WORD = OFF_RUNS + NT * 16;      // a bit for each row
    static constexpr int OFF_BAR = OFF_WORD + 32;
    static constexpr int BARS = 32 * STAGES + 96;
    static constexpr int TOTAL = OFF_BAR + BARS + 1024;      // + alignment slack
    static_assert(TOTAL <= 232448, "shared memory of a CTA");
    static_assert(STAGES * STAGE >= NT * AD_LD * 4, "the cluster's sums, the last tile's output");
};

// An adapter of a tile and the columns [c0, c1) of the tile, multiples of 16, that hold its rows.
struct alignas(16) AdEntry {
    int adapter;
    uint16_t c0, c1;
    float scale;
};

// Shared-memory descriptor of a K-major tile with the 32-byte swizzle: rows of 32 bytes (16
// ranks), 8-row groups 256 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(256 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)6 << 61;
}

// The adapters of rows [row0, row0 + a.nt) of ids, in the order in which they come first, by the
// ad_builders(NT) warps together; their number.  Neighbouring rows with one adapter are a run; each
// thread compares its run with all others.  (A search for one adapter after another took 0.15 us
// for each, a comparison of 256 rows with one another 8 us.)
struct alignas(16) AdRun {
    int adapter;
    uint16_t c0, c1;                             // its rows
    float scale;
};
template <int NT>
__device__ __forceinline__ int list_adapters(const AdapterArgs& a, int row0, AdEntry* list, int* s_ids, AdRun* runs, uint32_t* s_word) {
    constexpr int T = 32 * ad_builders(NT), PER = (NT + T - 1) / T, WORDS = (NT + 31) / 32;
    const int tid = threadIdx.x - (ad_threads(NT) - T), lane = tid & 31;
    auto sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(T) : "memory"); };
    // the place of this thread's k-th element among those whose flag is set, by a ballot a warp
    auto count = [&](const bool (&flag)[PER], int (&at)[PER]) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const unsigned m = __ballot_sync(FULL_MASK, flag[k]);
            if (lane == 0 && k * T + tid < NT) s_word[(k * T + tid) / 32] = m;
        }
        sync();
        int n = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) at[k] = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            const uint32_t m = s_word[w];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int own = (k * T + tid) / 32;
                at[k] += w < own ? __popc(m) : w == own ? __popc(m & ((1u << lane) - 1u)) : 0;
            }
            n += __popc(m);
        }
        sync();
        return n;
    };
    float scale[PER];
    bool flag[PER];
    int at[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int c = k * T + tid, row = row0 + c;
        int x = c < a.nt && row < a.n ? a.ids[row] : -1;
        if (x >= a.n_adapters) {
            raise_status(a.status, EMBER_ERR_INVALID_ARG);
            x = -1;
        }
        if (c < NT) s_ids[c] = max(x, -1);
        scale[k] = x >= 0 && a.scale ? a.scale[x] : 1.f;
    }
    sync();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int c = k * T + tid;
        flag[k] = c < NT && s_ids[c] >= 0 && (c == 0 || s_ids[c - 1] != s_ids[c]);
    }
    const int n_runs = count(flag, at);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int c = k * T + tid;
        if (c >= NT || s_ids[c] < 0) continue;
        if (flag[k]) {
            runs[at[k]].adapter = s_ids[c];
            runs[at[k]].c0 = (uint16_t)c;
            runs[at[k]].scale = scale[k];
        }
        if (c + 1 == NT || s_ids[c + 1] != s_ids[c]) runs[at[k] + flag[k] - 1].c1 = (uint16_t)(c + 1);
    }
    sync();
    int last[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int r = k * T + tid;
        flag[k] = r < n_runs;
        last[k] = 0;
        if (!flag[k]) continue;
        const int x = runs[r].adapter;
        for (int q = 0; q < n_runs; ++q)
            if (runs[q].adapter == x) {
                flag[k] = flag[k] && q >= r;
                last[k] = runs[q].c1;
            }
    }
    const int n = count(flag, at);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (!flag[k]) continue;
        const AdRun r = runs[k * T + tid];
        list[at[k]] = AdEntry{r.adapter, (uint16_t)(r.c0 & ~15), (uint16_t)((last[k] + 15) & ~15), r.scale};
    }
    sync();
    return n;
}

// The blocks of a CTA's entries one after another: 16 ranks of an entry, then the next 16, then
// the entry `step` further on.  (Divisions took the thread that issues products longer than they.)
struct Block {
    const AdEntry* entry;
    int slab, slabs, step;
    __device__ __forceinline__ Block(const AdEntry* e, int n, int by) : entry(e), slab(0), slabs(n), step(by) {}
    __device__ __forceinline__ void next() {
        if (++slab == slabs) {
            slab = 0;
            entry += step;
        }
    }
};

// ---- values that are not finite ----
// A product of a tile's adapter takes in neighbouring rows with others as zeros, and zero times an
// infinity of B is not zero.  So where an output is not finite the outputs that B may have spoilt are
// taken again, each from its own row and adapter alone: those that are not finite, of rows of W for
// which some adapter of the tile's rows has a value in B that is not.  One operation an output sees to
// it where all is finite.  With a row of x that is not, whose outputs rightly are not either, a look at
// the tile's B: 64 rows of 40 adapters of rank 16 on 2048 x 16384 22 -> 30 us, 777 rows of 9 of rank 32
// 22 -> 26.  With one of those 40 b's infinite all over 570 us (an output and warp after another 850).
__device__ __forceinline__ bool odd16(uint32_t x, bool bf16) { return bf16 ? (x & 0x7f80) == 0x7f80 : (x & 0x7c00) == 0x7c00; }
template <bool BF16>
__device__ __forceinline__ bool any_odd(const uint4& v) {
    bool odd = false;
    for (uint32_t u : {v.x, v.y, v.z, v.w}) odd |= odd16(u, BF16) | odd16(u >> 16, BF16);
    return odd;
}
struct AdMend {
    int ids[256], named[256], n_named;   // the tile's rows' adapters, and each of them once
    uint32_t rows[AD_M / 32];            // of W, a bit each
};
// Outputs [lo, hi) of a tile in eights (row c of x, rows f .. f + 7 of W: c * 16 + f / 8), by the whole CTA.
template <class E>
__device__ __noinline__ void take_again(const AdapterArgs& a, int row0, int m0, int lo, int hi, AdMend* s) {
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int rows = min(a.nt, a.n - row0), RP = (a.R + 15) & ~15;
    __syncthreads();
    for (int c = tid; c < rows; c += T) {
        const int x = a.ids[row0 + c];
        s->ids[c] = x >= 0 && x < a.n_adapters ? x : -1;
    }
    if (tid < AD_M / 32) s->rows[tid] = 0;
    if (tid == 0) s->n_named = 0;
    __syncthreads();
    for (int c = tid; c < rows; c += T) {
        const int id = s->ids[c];
        bool seen = id < 0;
#pragma unroll 8
        for (int k = 0; k < c; ++k) seen |= s->ids[k] == id;
        if (!seen) s->named[atomicAdd(&s->n_named, 1)] = id;   // (in no order: only marks follow)
    }
    __syncthreads();
    const int pieces = min(AD_M, a.N - m0) * (a.R / 8), all = s->n_named * pieces;   // of 16 bytes, side by side for an adapter
    for (int i0 = tid; i0 < all; i0 += 8 * T) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * T;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (i < all)
                v[k] = __ldg(reinterpret_cast<const uint4*>(a.lb + ((long long)s->named[i / pieces] * a.N + m0) * a.R) + i % pieces);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (any_odd<E::bf16>(v[k])) {
                const int m = (i0 + k * T) % pieces / (a.R / 8);
                atomicOr(&s->rows[m / 32], 1u << (m % 32));
            }
    }
    __syncthreads();
    const auto marks = [&](int g) { return s->rows[g / 4] >> (g % 4 * 8) & 0xffu; };   // of rows 8 g .. 8 g + 7
    const unsigned groups = __ballot_sync(FULL_MASK, lane < AD_M / 8 && marks(lane) != 0);
    const int ng = __popc(groups);
    for (int e = warp; e < rows * ng; e += T / 32) {
        const int c = e / ng, g = (int)__fns(groups, 0, e % ng + 1), i = c * (AD_M / 8) + g;
        if (i < lo || i >= hi) continue;
        const int row = row0 + c, m = m0 + 8 * g, id = s->ids[c];
        float* o32 = static_cast<float*>(a.out) + row * a.ld_out + m;
        uint16_t* o16 = static_cast<uint16_t*>(a.out) + row * a.ld_out + m;
        bool odd = false;
        if (lane < 8 && (marks(g) >> lane & 1u))
            odd = a.out_f32 ? (__float_as_uint(__ldcg(o32 + lane)) & 0x7f800000u) == 0x7f800000u : odd16(__ldcg(o16 + lane), E::bf16);
        if (!__any_sync(FULL_MASK, odd)) continue;
        // all eight, for one latency
        float y[8], u[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        const uint4 *x = reinterpret_cast<const uint4*>(a.x + row * a.ld_x), *w = reinterpret_cast<const uint4*>(a.w + (long long)m * a.K);
        for (int k = lane; k < a.K / 8; k += 32) {
            uint4 q[8];
            const uint4 xk = __ldg(x + k);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = __ldg(w + (long long)j * (a.K / 8) + k);
            unpack8w<!E::bf16>(xk, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                unpack8w<!E::bf16>(q[j], v);
#pragma unroll
                for (int d = 0; d < 8; ++d) y[j] = fmaf(u[d], v[d], y[j]);
            }
        }
        if (id >= 0)
            for (int r = lane; r < a.R; r += 32) {
                const uint16_t* t = a.t + (long long)row * 2 * RP + r / 16 * 32 + r % 16;
                const uint32_t two = (uint32_t)__ldcg(t) | (uint32_t)__ldcg(t + 16) << 16;
                const float t1 = E::lo(two), tr = odd16(two & 0xffff, E::bf16) ? t1 : t1 + E::hi(two);   // (an infinity's second term is no number)
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(E::lo((uint32_t)a.lb[((long long)id * a.N + m + j) * a.R + r]), tr, y[j]);
            }
        float mine = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sum = warp_sum(y[j]);
            if (lane == j) mine = sum;
        }
        if (odd) {
            if (a.bias) mine += E::lo((uint32_t)a.bias[m + lane]);
            if (a.out_f32) o32[lane] = mine;
            else o16[lane] = (uint16_t)E::pack(mine, 0.f);
        }
    }
}

// Eight sums of a row of x.  First launch: ranks r .. r + 7 of its adapter, as two terms (and
// zeros for the ranks that fill up a product); second: outputs m .. m + 7.  True: beyond f16.
template <class E>
__device__ __forceinline__ bool store_low(const AdapterArgs& a, int row, int r, float scale, float (&y)[8]) {
    const int RP = (a.R + 15) & ~15;
    uint16_t* t = a.t + (long long)row * 2 * RP + r / 16 * 32 + r % 16;   // both terms of 16 ranks side by side
    uint32_t hi[4], lo[4];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float u = y[2 * j] * scale, v = y[2 * j + 1] * scale;
        if (!E::bf16) bad |= f16_out_of_range(u) | f16_out_of_range(v);
        hi[j] = E::pack(u, v);
        lo[j] = E::pack(u - E::lo(hi[j]), v - E::hi(hi[j]));
    }
    *reinterpret_cast<uint4*>(t) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(t + 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (r + 8 == a.R && a.R < RP) {
        *reinterpret_cast<uint4*>(t + 8) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(t + 24) = make_uint4(0u, 0u, 0u, 0u);
    }
    return bad;
}
template <class E>
__device__ __forceinline__ void store_out(const AdapterArgs& a, int row, int m, const float (&y)[8]) {
    if (a.out_f32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * a.ld_out + m);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.ld_out + m) =
            make_uint4(E::pack(y[0], y[1]), E::pack(y[2], y[3]), E::pack(y[4], y[5]), E::pack(y[6], y[7]));
    }
}

// (Two CTAs to an SM where they have room: one of each launch.)
template <class E, int NT, bool LOW, bool FOLD>
__global__ void __launch_bounds__(ad_threads(NT), NT <= 128 && !FOLD ? 2 : 1)
    k_adapter(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ AdapterArgs a) {
    using L = AdSmem<NT, LOW>;
    constexpr int S = L::STAGES;
    // TMEM: two accumulators, which take turns, or one and two and the sum
    constexpr int ACCS = FOLD && NT > 128 ? 1 : 2;
    constexpr uint32_t COLS = FOLD && NT <= 128 ? 4 * NT : 2 * NT;
    static_assert(COLS >= 32 && COLS <= 512 && (ACCS + FOLD) * NT <= COLS, "TMEM");
    extern __shared__ uint8_t ad_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ad_raw) + 1023) & ~uintptr_t(1023));
    float* s_out = reinterpret_cast<float*>(sm + L::OFF_OUT);
    AdEntry* s_list = reinterpret_cast<AdEntry*>(sm + L::OFF_LIST);
    int* s_ids = reinterpret_cast<int*>(sm + L::OFF_IDS);
    AdRun* s_runs = reinterpret_cast<AdRun*>(sm + L::OFF_RUNS);
    uint32_t* s_word = reinterpret_cast<uint32_t*>(sm + L::OFF_WORD);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
    uint64_t* full = bar;                // [S] a stage's copies have landed
    uint64_t* empty = bar + S;           // [S] its products are done
    uint64_t* t_go = bar + 2 * S;        // [S] t's tile may be written there
    uint64_t* t_full = bar + 3 * S;      // [S] it is
    uint64_t* acc_full = bar + 4 * S;    // [2]
    uint64_t* acc_empty = acc_full + 2;  // [2]
    uint64_t* list_full = acc_empty + 2; // [2]
    uint64_t* list_empty = list_full + 2;
    int* s_count = reinterpret_cast<int*>(list_empty + 2);   // [2] entries of the lists
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_count + 2);
    int* sflag = reinterpret_cast<int*>(tmem_slot + 1);      // [0] failed, [1] stages issued, [2] consumed, [3] an output is not finite
    static_assert((4 * S + 8) * 8 + 7 * 4 <= L::BARS, "barriers");
    static_assert(sizeof(AdMend) <= S * L::STAGE, "over the stages");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int CL = a.splits, rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;   // CTAs of a cluster
    const int nk = (a.K + AD_BK - 1) / AD_BK;
    const int start = (int)blockIdx.x / CL, stride = (int)gridDim.x / CL;
    const int RP = (a.R + 15) & ~15;                          // ranks with those that fill up a product
    const int slabs = RP / 16;                                // blocks of an adapter

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&t_go[s], 1);
            mbar_init(&t_full[s], ad_builders(NT));
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
            mbar_init(&list_full[b], 1);
            mbar_init(&list_empty[b], 2 + ad_builders(NT));   // copies, products, builders
        }
        sflag[0] = sflag[1] = sflag[2] = sflag[3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // The second launch starts once every CTA of the first has come past its wait: what came
    // before both is complete for it too.
    if (LOW) {
        pdl_wait();
        pdl_trigger();
        if (warp >= 6) {                         // the CTA's one row tile
            const int n = list_adapters<NT>(a, start % a.row_tiles * a.nt, s_list, s_ids, s_runs, s_word);
            if (warp == 6 && lane == 0) s_count[0] = n;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Its tiles.  Second launch: the cluster's start, start + stride, ..; with a cluster of several
    // it is one, whose K they share.  First launch: a tile holds as many of the list's adapters as
    // have room in 128 rows, the cluster has every step-th of its row tile's, and as many CTAs as
    // there are for each share one's K.
    const int P = LOW ? AD_M / a.R : 1;
    const int step = LOW ? stride / a.row_tiles : 1, first_tile = LOW ? start / a.row_tiles : 0;
    const int have = LOW ? max(0, ((s_count[0] + P - 1) / P - first_tile + step - 1) / step)
                         : max(0, (a.row_tiles * a.col_tiles - start + stride - 1) / stride);
    int C = CL;                                  // CTAs that share a tile
    if (LOW)
        while (C > 1 && have * C > CL) C /= 2;
    const int part = rank % C, first_of = rank / C, every = LOW ? CL / C : 1;
    const int tiles = LOW ? max(0, (have - first_of + every - 1) / every) : have;
    const int kb0 = (int)((long long)nk * part / C), kb1 = (int)((long long)nk * (part + 1) / C);
    // A tile alone has both accumulators, and each gets half of K: half the steps lose half (777 rows,
    // K 1024, f32 outputs: off by 0.66e-6 of their norm in 22.1 us, in one accumulator 1.2e-6 in 21.5).
    // Whatever the outputs' type, so that the narrow ones are the f32 ones rounded up to K 1024.
    const bool two = !LOW && !FOLD && tiles == 1 && kb1 - kb0 >= 2;
    const int mid = two ? (kb0 + kb1) / 2 : kb1;
    // A tile's products are one run of blocks in one accumulator, or several in turn.
    const int runs = FOLD ? max(1, (kb1 - kb0 + AD_FOLD - 1) / AD_FOLD) : 1;
    // sums c .. c + 15 of this thread's row: an accumulator's and, if there are some, those at `more`
    auto sums_of = [&](uint32_t acc, bool some, uint32_t more, int c, float (&y)[16]) {
        uint32_t r[16], q[16];
        tmem_ld16(acc + c, r);
        if (some) tmem_ld16(more + c, q);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(r[i]) + (some ? __uint_as_float(q[i]) : 0.f);
    };
    struct Tile {
        int row0, m0, e0;                        // first row of x, first row of W, first entry (first launch)
    };
    auto tile_of = [&](int li) {
        Tile t;
        const int i = start + li * stride;
        t.row0 = i % a.row_tiles * a.nt;
        t.m0 = LOW ? 0 : i / a.row_tiles * AD_M;
        t.e0 = LOW ? (first_tile + (first_of + li * every) * step) * P : 0;
        return t;
    };
    // Blocks of a tile's adapters that are this CTA's (entries part, part + C, ..); a stage holds SLABS.
    auto blocks_of = [&](int n) { return n > part ? (n - part + C - 1) / C * slabs : 0; };
    // Sums m .. m + 7 of row c of x: whether anybody wants them, and where they go.
    auto wanted = [&](const Tile& t, int c, int m) {
        if (!LOW) return t.m0 + m < a.N;
        const int e = t.e0 + m / a.R;
        return m < P * a.R && e < s_count[0] && s_list[e].adapter == s_ids[c];
    };
    bool bad = false;                            // f16: t beyond its range
    float probe[4] = {0.f, 0.f, 0.f, 0.f};       // NaN once an output was not finite (four: a chain of one took 0.5 us)
    auto store = [&](const Tile& t, int c, int m, float (&y)[8]) {
        if (LOW) bad |= store_low<E>(a, t.row0 + c, m % a.R, s_list[t.e0 + m / a.R].scale, y);
        else store_out<E>(a, t.row0 + c, t.m0 + m, y);
    };

    if (warp == 0) {
        if (lane == 0) {   // ---------------- copies
            int g = 0;                           // stages so far
            bool ok = true;
            auto slot = [&](int& s) {
                s = g % S;
                ok = g < S || mbar_wait(&empty[s], ((uint32_t)(g / S) & 1u) ^ 1u);
                return ok;
            };
            for (int li = 0; li < tiles && ok; ++li) {
                const Tile t = tile_of(li);
                int s;
                for (int kb = kb0; kb < kb1 && slot(s); ++kb, ++g) {
                    uint8_t* p = sm + s * L::STAGE;
                    const int n = LOW ? min(P, s_count[0] - t.e0) : 0;
                    mbar_expect_tx(&full[s], (LOW ? n * a.R * 128 : L::A_BYTES) + a.nt * 128);
                    if (!LOW) tma_load_2d(p, &tmW, kb * AD_BK, t.m0, &full[s]);
                    for (int e = 0; e < n; ++e)
                        tma_load_3d(p + e * a.R * 128, &tmW, kb * AD_BK, 0, s_list[t.e0 + e].adapter, &full[s]);
                    tma_load_2d(p + L::A_BYTES, &tmX, kb * AD_BK, t.row0, &full[s]);
                }
                if (LOW || !ok) continue;
                const int b = li & 1;
                ok = mbar_wait(&list_full[b], (uint32_t)(li >> 1) & 1u);
                const int all = ok ? blocks_of(s_count[b]) : 0;
                Block at(s_list + b * NT + part, slabs, C);
                for (int f = 0; f < all && slot(s); f += L::SLABS, ++g) {
                    const int m = min(L::SLABS, all - f);
                    mbar_expect_tx(&full[s], m * L::SLAB_A);
                    for (int i = 0; i < m; ++i, at.next())
                        tma_load_3d(sm + s * L::STAGE + i * L::SLAB_A, &tmB, at.slab * 16, t.m0, at.entry->adapter, &full[s]);
                    mbar_arrive(&t_go[s]);
                }
                if (ok) mbar_arrive(&list_empty[b]);
            }
            if (!ok) sflag[0] = 1;
            sflag[1] = g;
        }
    } else if (warp == 1) {
        if (lane == 0) {   // ---------------- products
            constexpr uint32_t type = E::bf16 ? idesc_bf16(0, 0) : idesc_f16(0, 0);
            const uint32_t id_x = type | idesc_f16(AD_M, a.nt);
            int g = 0;
            uint32_t t_phase = 0;                // of t_full, a bit a slot
            bool ok = true;
            for (int li = 0; li < tiles && ok; ++li) {
                const int b = li & 1;
                int run = li * runs, kr = kb0;   // this run's number of all and its first block
                auto begin = [&] {
                    ok = run < ACCS || mbar_wait(&acc_empty[run % ACCS], ((uint32_t)(run / ACCS) & 1u) ^ 1u);
                    tc_fence_after();
                    return ok;
                };
                if (!begin()) break;
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    if (FOLD && kb == kr + AD_FOLD) {
                        umma_commit(&acc_full[run % ACCS]);
                        ++run;
                        kr = kb;
                        if (!begin()) break;
                    }
                    const uint32_t acc = tmem + (uint32_t)(run % ACCS * NT);
                    const int s = g % S;
                    if (!(ok = mbar_wait(&full[s], (uint32_t)(g / S) & 1u))) break;
                    tc_fence_after();
                    const uint32_t w = smem_u32(sm + s * L::STAGE), x = w + L::A_BYTES;
#pragma unroll
                    for (int k = 0; k < AD_BK / 16; ++k)
                        umma_bf16(kb < mid ? acc : acc + NT, sdesc_sw128(w + k * 32), sdesc_sw128(x + k * 32), id_x,
                                  (kb != kr && kb != mid) || k > 0);
                    umma_commit(&empty[s]);
                }
                if (!LOW && ok) {
                    const uint32_t acc = tmem + (uint32_t)(run % ACCS * NT);
                    ok = mbar_wait(&list_full[b], (uint32_t)(li >> 1) & 1u);
                    const int all = ok ? blocks_of(s_count[b]) : 0;
                    Block next(s_list + b * NT + part, slabs, C);
                    for (int f = 0; f < all; f += L::SLABS, ++g) {
                        const int s = g % S;
                        ok = mbar_wait(&full[s], (uint32_t)(g / S) & 1u) && mbar_wait(&t_full[s], t_phase >> s & 1u);
                        if (!ok) break;
                        t_phase ^= 1u << s;
                        tc_fence_after();
                        const uint64_t w = sdesc_sw32(smem_u32(sm + s * L::STAGE)), u = sdesc_sw32(smem_u32(sm + s * L::STAGE + L::OFF_T));
#pragma unroll 1
                        for (int i = 0; i < min(L::SLABS, all - f); ++i, next.next()) {
                            const int c0 = next.entry->c0;
                            const uint32_t id = type | idesc_f16(AD_M, next.entry->c1 - c0);
                            const uint64_t t = u + (i * 2 * L::SLAB_T >> 4) + c0 * 2;   // (rows of 32 bytes)
                            umma_bf16(acc + c0, w + (i * L::SLAB_A >> 4), t, id, 1);
                            umma_bf16(acc + c0, w + (i * L::SLAB_A >> 4), t + (L::SLAB_T >> 4), id, 1);
                        }
                        umma_commit(&empty[s]);
                    }
                    if (ok) mbar_arrive(&list_empty[b]);
                }
                if (ok) umma_commit(&acc_full[run % ACCS]);
            }
            if (!ok) sflag[0] = 1;
            sflag[2] = g;
        }
    } else if (warp >= 6) {
        if (!LOW) {   // -------------- which adapters a tile has, and t's tiles
            const int builder = warp - 6;
            int g = 0;                           // stages so far
            uint32_t go_phase = 0;
            bool waited = false;
            // (all of them see the phases: a wait names one by its parity alone)
            auto ready = [&](int li) { return li < 2 || mbar_wait(&list_empty[li & 1], ((uint32_t)(li >> 1) & 1u) ^ 1u); };
            auto all_of_us = [](bool ok) {
                uint32_t all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all)
                             : "r"((uint32_t)ok), "n"(32 * ad_builders(NT))
                             : "memory");
                return all != 0;
            };
            auto build = [&](int li) {
                bool ok = true;
                const int b = li & 1;
                const Tile t = tile_of(li);
                const int n = list_adapters<NT>(a, t.row0, s_list + b * NT, s_ids + b * NT, s_runs, s_word);
                if (builder == 0 && lane == 0) {
                    s_count[b] = n;
                    mbar_arrive(&list_full[b]);
                }
                const int* ids = s_ids + b * NT;
                g += kb1 - kb0;
                if (!waited) {                   // t is the first launch's
                    pdl_wait();
                    waited = true;
                }
                const int all = blocks_of(n);
                // One tile, and t's rows fit where its output will be staged: they are fetched at
                // once, and writing a block is a matter of shared memory.  (The two places have a
                // pointer each: a load that is of one space by name must never see the other's address.)
                const uint4* rows_t = reinterpret_cast<const uint4*>(a.t + (long long)t.row0 * 2 * RP);
                const uint4* kept_t = reinterpret_cast<const uint4*>(s_out);
                const int rows = min(a.nt, a.n - t.row0);
                const bool kept = tiles == 1 && all > 0 && rows * RP * 4 <= L::OUT;
                if (kept) {
                    const int tid = threadIdx.x - (ad_threads(NT) - 32 * ad_builders(NT));
                    for (int i = tid; i < rows * (RP / 4); i += 32 * ad_builders(NT))
                        reinterpret_cast<uint4*>(s_out)[i] = __ldcg(rows_t + i);
                    asm volatile("bar.sync 2, %0;" ::"n"(32 * ad_builders(NT)) : "memory");
                }
                Block next(s_list + b * NT + part, slabs, C);
                for (int f = 0; f < all; f += L::SLABS, ++g) {
                    const int s = g % S, m = min(L::SLABS, all - f);
                    // Pieces of 32 rows of a block, 16 ranks of both terms of each row, or zeros: the
                    // builders' in turn, the first one asked for before the stage is free.
                    int p = builder, i = 0, c = 0;   // this builder's piece: of block i, column c
                    const AdEntry* en = nullptr;
                    int slab = 0;
                    auto find = [&] {                // false: there is none
                        for (; i < m; ++i, next.next()) {
                            const int wide = (next.entry->c1 - next.entry->c0 + 31) / 32;
                            if (p < wide) {
                                en = next.entry;
                                slab = next.slab;
                                c = en->c0 + 32 * p + lane;
                                return true;
                            }
                            p -= wide;
                        }
                        return false;
                    };
                    uint4 v[4];
                    auto ask = [&] {
                        const bool own = c < en->c1 && ids[c] == en->adapter;
                        const int from = c * (RP / 4) + slab * 4;
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = make_uint4(0u, 0u, 0u, 0u);
                        if (own && kept)
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] = kept_t[from + q];
                        if (own && !kept)
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] = __ldcg(rows_t + from + q);
                    };
                    bool some = find();
                    if (some) ask();
                    if (!(ok = __all_sync(FULL_MASK, mbar_wait(&t_go[s], go_phase >> s & 1u)))) break;   // (all lanes or none)
                    go_phase ^= 1u << s;
                    while (some) {
                        uint8_t* dst = sm + s * L::STAGE + L::OFF_T + i * 2 * L::SLAB_T + c * 32;
                        if (c < en->c1)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                *reinterpret_cast<uint4*>(dst + (q >> 1) * L::SLAB_T + (((q & 1) ^ (c >> 2 & 1)) << 4)) = v[q];
                        p += ad_builders(NT);
                        some = find();
                        if (some) ask();
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&t_full[s]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&list_empty[b]);
                return ok;
            };
            if (!rounds_together(tiles, ready, all_of_us, build)) sflag[0] = 1;
            if (!waited) pdl_wait();             // this grid ends after the first one, whatever happens
        }
    } else {   // ---------------- output, warps 2..5
        const int quad = warp & 3, tid = threadIdx.x - 64;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t sum = tmem + ACCS * NT + lane_off;
        for (int li = 0; li < tiles; ++li) {
            const Tile t = tile_of(li);
            const int rows = min(a.nt, a.n - t.row0);
            int run = li * runs;
            auto next_run = [&] {                // false for all four warps, which the barriers below need, or none
                const uint32_t ok = mbar_wait(&acc_full[run % ACCS], (uint32_t)(run / ACCS) & 1u);
                uint32_t all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all)
                             : "r"(ok)
                             : "memory");
                tc_fence_after();
                return all != 0;
            };
            // every run but the last is added to the sum, and its accumulator is free again
            constexpr int FOLD_COLS = NT < 32 ? NT : 32;
            bool ok = next_run();
            for (int k = 0; FOLD && ok && k + 1 < runs; ++k) {
                const uint32_t acc = tmem + (uint32_t)(run % ACCS * NT) + lane_off;
#pragma unroll 1
                for (int c = 0; c < rows; c += FOLD_COLS) {
                    uint32_t x[FOLD_COLS], y[FOLD_COLS];
#pragma unroll
                    for (int i = 0; i < FOLD_COLS; i += 16) {
                        tmem_ld16(acc + c + i, x + i);
                        if (k > 0) tmem_ld16(sum + c + i, y + i);
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < FOLD_COLS; ++i)
                        if (k > 0) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
#pragma unroll
                    for (int i = 0; i < FOLD_COLS; i += 16) tmem_st16(sum + c + i, x + i);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[run % ACCS]);
                ++run;
                ok = next_run();
            }
            if (!ok) {
                sflag[0] = 1;
                break;
            }
            const int b = run % ACCS;
            const uint32_t acc = tmem + (uint32_t)(b * NT) + lane_off;
            const bool some = two || (FOLD && runs > 1);   // sums beside the accumulator's
            const uint32_t more = FOLD ? sum : acc + NT;
            if (C > 1) {                         // the whole tile, joined below
                float* dst = reinterpret_cast<float*>(sm) + quad * 32 + lane;
                for (int c = 0; c < rows; c += 16) {
                    float y[16];
                    sums_of(acc, some, more, c, y);
#pragma unroll
                    for (int i = 0; i < 16; ++i) dst[(c + i) * AD_LD] = y[i];
                }
                break;
            }
            if (!LOW) {
                // Through shared memory and TMA: while other tiles follow, slices of 16 rows of x, two
                // in turn; the last tile at once over the stages, which nothing needs any more.
                const int m = t.m0 + quad * 32 + lane;   // this thread's row of W
                const bool last = li + 1 == tiles;
                const int row_bytes = AD_M * (a.out_f32 ? 4 : 2);
                float add = 0.f;
                if (a.bias && m < a.N) add = E::bf16 ? bf16_to_f32(a.bias[m]) : __half2float(__ushort_as_half(a.bias[m]));
                auto put_out = [&](const uint8_t* buf, int c) {   // (clipped to what there is)
                    tma_store_2d(&tmOut, buf, t.m0, t.row0 + c);
                    bulk_commit();
                };
                for (int c = 0; c < rows; c += 16) {
                    float y[16];
                    sums_of(acc, some, more, c, y);
                    if (c + 16 >= rows) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[b]);
                    }
                    uint8_t* buf = last ? sm + c * row_bytes : sm + L::OFF_OUT + (c >> 4 & 1) * (16 * AD_M * 4);
                    if (!last) {
                        if (tid == 0) bulk_wait_read<1>();   // the slice before the last one has left
                        asm volatile("bar.sync 1, 128;" ::: "memory");
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) probe[i & 3] = fmaf(y[i], 0.f, probe[i & 3]);
                    if (a.out_f32) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            reinterpret_cast<float*>(buf)[i * AD_M + quad * 32 + lane] = y[i] + add;
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            reinterpret_cast<uint16_t*>(buf)[i * AD_M + quad * 32 + lane] = (uint16_t)E::pack(y[i] + add, 0.f);
                    }
                    if (!last) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        asm volatile("bar.sync 1, 128;" ::: "memory");
                        if (tid == 0) put_out(buf, c);
                    } else if ((c & 48) == 48 || c + 16 >= rows) {   // 64 rows' worth
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        asm volatile("bar.sync 1, 128;" ::: "memory");
                        if (tid == 0)
                            for (int d = c & ~63; d <= c; d += 16) put_out(sm + d * row_bytes, d);
                    }
                }
                if (!last && tid == 0) {
                    bulk_wait_read<0>();         // the next tile begins with the first slice's place again
                }
                continue;
            }
            const int f = tid % 16 * 8;          // this thread's 8 ranks
            for (int c = 0; c < rows; c += AD_SLICE) {
                float y[AD_SLICE / 16][16];
                sums_of(acc, some, more, c, y[0]);
                if (NT >= AD_SLICE) sums_of(acc, some, more, c + 16, y[1]);
                if (c + AD_SLICE >= rows) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[b]);
                }
#pragma unroll
                for (int i = 0; i < AD_SLICE; ++i)
                    if (NT >= AD_SLICE || i < 16) s_out[i * AD_LD + quad * 32 + lane] = y[i / 16][i % 16];
                asm volatile("bar.sync 1, 128;" ::: "memory");
                for (int i = tid / 16; i < min(AD_SLICE, rows - c); i += 8) {
                    if (!wanted(t, c + i, f)) continue;
                    const float4* p = reinterpret_cast<const float4*>(s_out + i * AD_LD + f);
                    const float4 u = p[0], v = p[1];
                    float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                    store(t, c + i, f, y);
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
        }
        if (!LOW && tid == 0) bulk_wait<0>();    // every output copy complete before the end
    }
    __syncwarp();

    if (C > 1) {   // ---------------- the cluster's sums, a share of the tile for each CTA
        cluster_sync_all();
        if (tiles > 0) {                         // (the same for all that share it)
            const Tile t = tile_of(0);
            const int rows = min(a.nt, a.n - t.row0);
            const uint32_t at = smem_u32(sm);
            const int all = rows * (AD_M / 8), lo = (int)((long long)all * part / C), hi = (int)((long long)all * (part + 1) / C);
            for (int i = lo + (int)threadIdx.x; i < hi; i += ad_threads(NT)) {
                const int c = i / (AD_M / 8), f = i % (AD_M / 8) * 8;
                if (!wanted(t, c, f)) continue;  // (most of the first launch's)
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = 0.f;
                float4 v[8][2];                  // asked for at once: one after another they took 0.3 us each
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (p < C) {
                        v[p][0] = ld_cluster4(at + (c * AD_LD + f) * 4, rank - part + p);
                        v[p][1] = ld_cluster4(at + (c * AD_LD + f + 4) * 4, rank - part + p);
                    }
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (p < C)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            y[4 * h] += v[p][h].x;
                            y[4 * h + 1] += v[p][h].y;
                            y[4 * h + 2] += v[p][h].z;
                            y[4 * h + 3] += v[p][h].w;
                        }
                if (!LOW && a.bias) {
                    float add[8];
                    unpack8w<!E::bf16>(*reinterpret_cast<const uint4*>(a.bias + t.m0 + f), add);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] += add[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) probe[j & 3] = fmaf(y[j], 0.f, probe[j & 3]);
                store(t, c, f, y);
            }
        }
        cluster_sync_all();                      // no CTA leaves while its shared memory is read
    }
    if (bad) raise_status(a.status, EMBER_ERR_RANGE);
    if (!LOW && (probe[0] + probe[1]) + (probe[2] + probe[3]) != 0.f) sflag[3] = 1;
    if (!LOW) pdl_trigger();

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sflag[0]) {
        raise_status(a.status, EMBER_ERR_TIMEOUT);
        for (int g = max(sflag[2], sflag[1] - S); g < sflag[1]; ++g)   // copies in flight
            (void)mbar_wait(&full[g % S], (uint32_t)(g / S) & 1u);
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS));
    }
    if constexpr (!LOW) {
        if (sflag[3] && !sflag[0]) {             // (the outputs are written, and nothing is left in flight)
            pdl_wait();
            for (int li = 0; li < tiles; ++li) {
                const Tile t = tile_of(li);
                const int all = min(a.nt, a.n - t.row0) * (AD_M / 8);
                take_again<E>(a, t.row0, t.m0, (int)((long long)all * part / C), (int)((long long)all * (part + 1) / C),
                              reinterpret_cast<AdMend*>(sm));
            }
        }
    }
}

// The first launch for little work: a CTA for eight ranks of a row, its warps for a part of K each.
// No list of adapters, no tensor memory, no cluster: one row on rank 8 has t 2 us sooner.  A is
// read for each row that names it, from L2, which is what bounds it: 2 n R K bytes.
constexpr int AR_WARPS = 4, AR_RANKS = 8;
template <class E>
__global__ void __launch_bounds__(AR_WARPS * 32) k_adapter_rows(AdapterArgs a, const uint16_t* x, long long ld_x, const uint16_t* la) {
    __shared__ float s_sum[AR_WARPS][AR_RANKS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = a.R / AR_RANKS, row = (int)(blockIdx.x / groups), r = (int)(blockIdx.x % groups) * AR_RANKS;
    pdl_wait();
    pdl_trigger();
    const int id = a.ids[row];
    if (id >= a.n_adapters && threadIdx.x == 0) raise_status(a.status, EMBER_ERR_INVALID_ARG);
    if (id < 0 || id >= a.n_adapters) return;
    const float scale = a.scale ? a.scale[id] : 1.f;
    const uint4* xp = reinterpret_cast<const uint4*>(x + row * ld_x);
    const uint4* ap = reinterpret_cast<const uint4*>(la + ((long long)id * a.R + r) * a.K);
    float sum[AR_RANKS];
#pragma unroll
    for (int k = 0; k < AR_RANKS; ++k) sum[k] = 0.f;
    const int pieces = a.K / 8;
#pragma unroll 2
    for (int i = warp * 32 + lane; i < pieces; i += AR_WARPS * 32) {
        uint4 w[AR_RANKS];
        const uint4 v = xp[i];
#pragma unroll
        for (int k = 0; k < AR_RANKS; ++k) w[k] = __ldg(ap + (long long)k * pieces + i);
        float u[8];
        unpack8w<!E::bf16>(v, u);
#pragma unroll
        for (int k = 0; k < AR_RANKS; ++k) {
            float y[8];
            unpack8w<!E::bf16>(w[k], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[k] = fmaf(u[j], y[j], sum[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < AR_RANKS; ++k) sum[k] = warp_sum(sum[k]);
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < AR_RANKS; ++k) s_sum[warp][k] = sum[k];
    __syncthreads();
    if (threadIdx.x == 0) {
        float y[AR_RANKS];
#pragma unroll
        for (int k = 0; k < AR_RANKS; ++k) {
            y[k] = 0.f;
#pragma unroll
            for (int w = 0; w < AR_WARPS; ++w) y[k] += s_sum[w][k];
        }
        if (store_low<E>(a, row, r, scale, y)) raise_status(a.status, EMBER_ERR_RANGE);
    }
}

template <class E, int NT, bool LOW, bool FOLD>
cudaError_t launch_form(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& b, const CUtensorMap& o, const AdapterArgs& a,
                      int grid, cudaStream_t s) {
    constexpr int SMEM = AdSmem<NT, LOW>::TOTAL;
    auto k = k_adapter<E, NT, LOW, FOLD>;
    static OncePerDevice once;
    const cudaError_t e = once([&] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e != cudaSuccess) return e;
    if (a.splits > 1) return launch_cluster_k(k, dim3(grid), dim3(ad_threads(NT)), SMEM, a.splits, s, w, x, b, o, a);
    return launch_k(k, dim3(grid), dim3(ad_threads(NT)), SMEM, s, w, x, b, o, a);
}
template <class E, int NT, bool LOW>
cudaError_t launch_nt(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& b, const CUtensorMap& o, const AdapterArgs& a,
                      int grid, bool fold, cudaStream_t s) {
    if (fold) return launch_form<E, NT, LOW, true>(w, x, b, o, a, grid, s);
    return launch_form<E, NT, LOW, false>(w, x, b, o, a, grid, s);
}
template <class E, bool LOW>
cudaError_t launch_low(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& b, const CUtensorMap& o, const AdapterArgs& a,
                       int grid, bool fold, cudaStream_t s) {
    if (a.nt <= 16) return launch_nt<E, 16, LOW>(w, x, b, o, a, grid, fold, s);
    if (a.nt <= 32) return launch_nt<E, 32, LOW>(w, x, b, o, a, grid, fold, s);
    if (a.nt <= 64) return launch_nt<E, 64, LOW>(w, x, b, o, a, grid, fold, s);
    if (a.nt <= 128) return launch_nt<E, 128, LOW>(w, x, b, o, a, grid, fold, s);
    if constexpr (!LOW) return launch_nt<E, 256, LOW>(w, x, b, o, a, grid, fold, s);
    return cudaErrorInvalidValue;
}
template <class E>
cudaError_t launch_rows(const AdapterArgs& a, const AdapterRows& r, cudaStream_t s) {
    // an SM set to little shared memory takes no CTA of the second launch before this one's are gone
    static OncePerDevice once;
    const cudaError_t e = once([] {
        return cudaFuncSetAttribute(k_adapter_rows<E>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    return launch_k(k_adapter_rows<E>, dim3((unsigned)a.n * (a.R / AR_RANKS)), dim3(AR_WARPS * 32), 0, s, a, r.x, r.ld_x, r.a);
}
template <class E>
cudaError_t launch_type(const AdapterMaps& m, AdapterArgs a, const AdapterPlan& p, const AdapterRows& r, cudaStream_t s) {
    const auto& mw = *reinterpret_cast<const CUtensorMap*>(m.w);
    const auto& mx = *reinterpret_cast<const CUtensorMap*>(m.x);
    const auto& ma = *reinterpret_cast<const CUtensorMap*>(m.a);
    const auto& mb = *reinterpret_cast<const CUtensorMap*>(m.b);
    const auto& mxl = *reinterpret_cast<const CUtensorMap*>(m.x_low);
    const auto& mo = *reinterpret_cast<const CUtensorMap*>(m.out);
    a.row_tiles = p.low_row_tiles;
    a.col_tiles = 1;
    a.splits = p.low_splits;
    a.nt = p.low_nt;
    const cudaError_t e = p.low_grid ? launch_low<E, true>(ma, mxl, ma, ma, a, p.low_grid, p.low_fold, s)
                                     : launch_rows<E>(a, r, s);
    if (e != cudaSuccess) return e;
    a.row_tiles = p.row_tiles;
    a.col_tiles = p.col_tiles;
    a.splits = p.splits;
    a.nt = p.nt;
    return launch_low<E, false>(mw, mx, mb, mo, a, p.grid, p.fold, s);
}

// Multiplications n R K of k_adapter_rows at most, twice as many from 16 adapters on, since the
// tcgen05 kernel has a tile for every two (rank 64) that a row tile names, whatever their rows.  On
// 4096 inputs and outputs (bf16, rows in any order), by rows and with tcgen05: 64 rows of rank 32 on
// 40 adapters 16 and 25 us; 128 rows of rank 64 on 8 adapters (2^25) 21 and 28; 256 rows of rank 64
// (2^26) on 2 adapters 32 and 29, on 8 36 and 36, on 32 47 and 58; twice that on 8 adapters 46 and
// 42, on 64 93 and 126, but 70 and 57 where each adapter's rows stand together.
constexpr int AR_MOST = 1 << 25, AR_ADAPTERS = 16;

// Cycles of a block's products, 4 of M = 128, N = nt, K = 16: no less than 112 each.
int block_cycles(int nt) { return max(450, nt * 8 / 3); }

}  // namespace

AdapterPlan adapter_plan(int n, int N, int K, int R, int n_adapters, bool out_f32, int sms) {
    AdapterPlan p{};
    const int nk = (K + AD_BK - 1) / AD_BK;
    p.col_tiles = (N + AD_M - 1) / AD_M;
    // The tile and the split that end first, by rounds of tiles over the SMs.  Few rows: one row
    // tile, K split until the SMs are full.  Many rows: any multiple of 16 rows up to 256, so that
    // 4096 rows of 16 column tiles are 304 tiles of 224 rows, two rounds of 152, not 256 of 256.
    long long best = -1;
    for (int nt = min(256, (n + 15) & ~15); nt >= 16; nt -= 16) {
        const int rt = (n + nt - 1) / nt;
        if (rt > 1 && nt < 128) break;
        for (int c = 1; c <= 8 && c <= nk; c *= 2) {
            const long long tiles = (long long)rt * p.col_tiles;
            if (c > 1 && tiles * c > sms) break;
            const long long rounds = (tiles * c + sms - 1) / sms;
            // (a tile alone has half of its blocks in each accumulator)
            const bool fold = out_f32 && (nk + c - 1) / c > AD_FOLD * (rounds == 1 ? 2 : 1);
            const long long cost = rounds * ((nk + c - 1) / c) * block_cycles(nt) + rounds * 8 * nt + (c > 1 ? 2000 : 0);
            if (best < 0 || cost < best) {
                best = cost;
                p.nt = nt;
                p.splits = c;
                p.fold = fold;
                p.row_tiles = rt;
                p.grid = (int)(c > 1 ? tiles * c : min(tiles, (long long)sms));
            }
        }
        if (rt == 1) break;
    }
    if ((double)n * R * K <= (double)AR_MOST * (min(n_adapters, n) >= AR_ADAPTERS ? 2 : 1)) return p;
    p.low_nt = min((n + 15) & ~15, 128);
    p.low_row_tiles = (n + p.low_nt - 1) / p.low_nt;
    const int most = (min(n_adapters, p.low_nt) + AD_M / R - 1) / (AD_M / R);   // tiles of a row tile
    // A CTA for each SM.  How many adapters a row tile has is known on the device: its clusters share
    // them out.
    p.low_fold = out_f32 && nk > AD_FOLD;
    p.low_splits = 1;
    while (p.low_splits < 8 && nk >= 2 * p.low_splits && p.low_row_tiles * p.low_splits * 2 <= sms) p.low_splits *= 2;
    const int clusters = max(1, min(most, sms / (p.low_splits * p.low_row_tiles)));
    p.low_grid = p.low_row_tiles * clusters * p.low_splits;
    return p;
}

size_t adapter_ws(int n, int R) { return (size_t)n * 2 * ((R + 15) & ~15) * sizeof(uint16_t); }

bool adapter_maps(const AdapterArgs& a, const AdapterPlan& p, const AdapterRows& r, AdapterMaps& m) {
    const uint64_t K = a.K, N = a.N, R = a.R, n = a.n;
    const uint64_t wd[2] = {K, N}, xd[2] = {K, n}, ad[3] = {K, R, (uint64_t)a.n_adapters}, bd[3] = {R, N, (uint64_t)a.n_adapters};
    const uint64_t ws[1] = {K * 2}, xs[1] = {(uint64_t)r.ld_x * 2}, as[2] = {K * 2, K * R * 2}, bs[2] = {R * 2, R * N * 2};
    const uint32_t wb[2] = {AD_BK, AD_M}, xb[2] = {AD_BK, (uint32_t)p.nt}, xl[2] = {AD_BK, (uint32_t)p.low_nt};
    const uint32_t ab[3] = {AD_BK, (uint32_t)a.R, 1}, bb[3] = {16, AD_M, 1};
    return encode_map_bf16(m.w, r.w, 2, wd, ws, wb) && encode_map_bf16(m.x, r.x, 2, xd, xs, xb) &&
           encode_map_bf16_sw32(m.b, r.b, 3, bd, bs, bb) && (p.splits > 1 || encode_map_rows(m.out, a.out, a.out_f32, N, n, a.ld_out, AD_M, 16)) &&
           (!p.low_grid || (encode_map_bf16(m.x_low, r.x, 2, xd, xs, xl) && encode_map_bf16(m.a, r.a, 3, ad, as, ab)));
}

cudaError_t launch_adapter(const AdapterMaps& m, const AdapterArgs& a, const AdapterPlan& p, const AdapterRows& r, bool bf16,
                           cudaStream_t s) {
    return bf16 ? launch_type<ElemBf16>(m, a, p, r, s) : launch_type<ElemF16>(m, a, p, r, s);
}

}  // namespace ember
