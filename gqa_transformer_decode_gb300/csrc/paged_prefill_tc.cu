// paged_prefill_tc.cu -- attention of several new tokens per sequence over a
// paged K/V cache on the tcgen05 tensor cores (the same function as
// paged_prefill.cu, for calls with rows enough to fill its tiles).
//
// One CTA holds two 128-row query tiles A and B of one (sequence, kv head).  The G
// query heads of a kv head share its keys, so a tile's rows are (token, head)
// pairs, row r = token r / G, head r % G: a tile spans 128 / G tokens, so little
// of its last key tile lies beyond the causal border, and each K / V tile that
// TMA brings serves all heads of the group.  Per key tile of 64 keys and query
// tile: S = Q K^T into TMEM, one thread per row takes p = 2^(s - m) and writes P
// (bf16 / f16) back to TMEM, O += P V accumulates there.  The reference maximum m
// moves (and O, l are rescaled, the tile done again) only when a row's weights of a
// tile sum to more than 2^15, so that most tiles need no maximum at all.  S has two
// buffers for each query tile, so the products of the next key tile are ready before
// a row's thread asks for them, and the two query tiles' threads and the tensor
// cores wait for one another only when one of them has fallen a whole tile behind.
// (With one buffer of 128 keys, P over it, a step was the sum of both products and
// the exponentials, 3.8 k cycles for 128 keys; a product of 64 columns takes 45
// cycles, of 128 columns 64.)
//
// K and V tiles are read from the pages as they lie, one TMA box (64 elements x
// up to 128 rows of a page) at a time, 128-byte swizzled: as K-major operand of
// the first product, and as MN-major operand of the second (V needs no
// transposed copy).  Boxes of pages that no row sees point beyond the pool, which
// TMA fills with zeros without reading anything; so does a bad page number.  In
// the tiles at the edges (the last one, the ends of the sinks and the window's
// start) a warp zeroes the V rows that no row sees, since 0 * NaN from a
// stale row would not be 0.
//
// P is rounded once to the cache's type, bf16 by 2^-8 of each weight at most, f16 by
// 2^-11, which in a sum over keys of mixed sign is about the output's own rounding
// (error against 64 bits 0.0022 and 0.00029, the bare rounding's 0.0016 and 0.00021).
// A second term, as decode has it, is another P V product: at head_dim 128, which
// the tensor pipe bounds, 512 cycles more on the 1263 of a step.  PT_SHARED takes it, since
// a decode step's outputs are not to be less exact for the prefix being shared; prefill
// does not.  l is summed from the unrounded weights in f32.
//
// CTAs are persistent: one whose last copies are issued asks the hardware to
// cancel a CTA that has not started yet (clusterlaunchcontrol) and takes over
// that one's tiles, so the next pair's Q, K and first products run under this
// one's epilogue, and the pairs still go to whichever SM is free.  Barrier phases
// and ring slots count on across the pairs.
//
// A call with few pairs splits their keys instead (SPLIT): the CTAs of a cluster
// share a pair's key tiles, leave (m, l, O) of its rows in their shared memory and
// join a share of the rows each through distributed shared memory.
//
// Measured: a 2048-token prompt, 32 heads on 8 of 64, 27.4 us (627 TFLOP/s of
// the products it cannot do without), one of 8000 tokens 296 us (885); five chunks of up
// to 1000 tokens on up to 5000 keys, 16 on 8 of 128, f16, 67 us (1200); 8192 tokens
// under a window of 1024, 68 us (945).  For 64 keys and both query tiles the products
// take 1263 cycles at head_dim 128 and 640 at 64 with nothing else running, the
// exponentials with their sums and rounding 540.  A step takes about 1330 at head_dim
// 128: the products.  At 64 it takes 1370: a row's thread waits for its scores, loads
// them (150 cycles each), works on them (under 900, two warps a scheduler) and hands
// the weights over (150), one after the other.  The copy and MMA warps' own
// instructions matter as much as the products: each must pass a tile in less than that.
// The tensor pipe is active for 65 % of the cycles in the chunks, whose longest tile
// pairs (87 key tiles) set the time, 52 % under the window and 27 % in the prompt.
//
// The same kernel takes the shared prefixes of ember_paged_decode_shared (PT_SHARED): a
// "sequence" is then a group of one-token rows, all of which see the group's prefix, and
// the key tiles of all (pair, kv head)s form a line of which CTA c takes the c-th equal
// share, as in paged_decode.cu.  What a CTA has of a pair it leaves as (m, l, O) of the
// pair's rows, which paged_shared.cu joins with the rows' own keys.
//
// Warps 0-3: tile A; warps 4-7: tile B (a warp reads the TMEM lanes of its index
// mod 4); warp 8: TMA producer; warp 9: TMEM allocation; warps
// 9 and 10: MMA issue for tile A and for tile B, so that neither's waiting holds
// up the other's products; warp 11: edge rows.  A row's 64 scores, and at the end
// its output, stand in registers at once, so a row's thread needs more of them
// (200) than the other warps (104).  Every mbarrier wait is bounded; a timeout
// raises EMBER_ERR_TIMEOUT, the CTA drains its copies and frees TMEM.
#include <algorithm>
#include <climits>

#include <cudaTypedefs.h>

#include "paged_groups.cuh"
#include "rounds.h"
#include "tc_common.cuh"

namespace ember {

namespace {

constexpr int PT_THREADS = 384;
constexpr int PT_TMA = 8, PT_MMA = 9, PT_EDGE = 11;   // warps (PT_MMA and the one after it: tiles A and B)
constexpr int PT_REGS_ROW = 200, PT_REGS_REST = 104;   // 256 * 200 + 128 * 104 = 384 * 168, the launch's share
constexpr int PT_ROWS = 128;   // rows of a query tile
constexpr int PT_PARTS = 8;    // CTAs of a cluster at most
// A pair's keys: by one CTA, or shared out over a cluster, or over the line.
enum PtForm : int { PT_WHOLE = 0, PT_SPLIT = 1, PT_SHARED = 2 };

template <int DP>
struct PtSmem {
    static constexpr int KB = DP / 64;                    // 64-element blocks of a row
    static constexpr int QTILE = KB * PT_ROWS * 128;      // a Q tile
    static constexpr int TILE = KB * PT_KEYS * 128;       // a K or V tile
    static constexpr int NS = DP == 64 ? 16 : 10;         // ring slots, a K or a V tile each
    static constexpr int OFF_Q = 0;                       // Q of tile A, of tile B
    static constexpr int OFF_KV = 2 * QTILE;
    static constexpr int OFF_BAR = OFF_KV + NS * TILE;
    static constexpr int TOTAL = OFF_BAR + 640 + 1024;    // + barriers, + alignment slack
    static_assert(TOTAL <= 232448, "shared memory of a CTA");
    static_assert(2 * PT_ROWS * (DP * 4 + 8) <= OFF_BAR, "the split form's rows");
    // TMEM columns: two S buffers of 64 f32 for each query tile, the weights P (64
    // values, two to a column) over the first half of theirs, their second terms over
    // the other; O_A, O_B (DP f32 each)
    static constexpr uint32_t col_s(int t, int b) { return t * 128 + b * 64; }
    static constexpr uint32_t col_o(int t) { return 256 + t * DP; }
};

// Low words of the operands' descriptors (the high word is the same for all:
// 8-row groups 1024 bytes apart, version 1, 128-byte swizzle).  K-major: rows of
// 128 bytes along K.  MN-major: 64 elements of M/N to a 128-byte row, the next 64
// `lead` bytes further.  Steps along K are added to the low word.
constexpr uint32_t DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr & 0x3ffffu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t lead) {
    return (saddr & 0x3ffffu) >> 4 | (lead >> 4) << 16;
}
// D (+)= A B^T, A in shared memory or in tensor memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"((uint32_t)acc), "n"(DESC_HI));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"((uint32_t)acc), "n"(DESC_HI));
}
// one lane of the warp, the same one each time
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(FULL_MASK, x, 0); }
constexpr uint32_t IDESC_B_MN = 1u << 16;   // B is MN-major

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// two f32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    uint64_t r, u, v, w;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(y.x), "f"(y.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(z.x), "f"(z.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(u), "l"(v), "l"(w));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r, u, v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(y.x), "f"(y.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(u), "l"(v));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
// bits 0 .. n - 1
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Four neighbouring lanes exchange the four 16-byte pieces that each holds of its row, so that
// together they write 64 bytes of one row after another instead of 16 of four rows each:
// afterwards q[i] is piece lane % 4 of row i of the four.
__device__ __forceinline__ void transpose_four(uint4 (&q)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    auto swap = [&](uint4& x, uint4& y, bool upper, int d) {   // lanes d apart: my y for its x
        const uint4 give = upper ? x : y;
        uint4 got;
        got.x = __shfl_xor_sync(FULL_MASK, give.x, d);
        got.y = __shfl_xor_sync(FULL_MASK, give.y, d);
        got.z = __shfl_xor_sync(FULL_MASK, give.z, d);
        got.w = __shfl_xor_sync(FULL_MASK, give.w, d);
        if (upper) x = got;
        else y = got;
    };
    swap(q[0], q[1], odd, 1);
    swap(q[2], q[3], odd, 1);
    swap(q[0], q[2], high, 2);
    swap(q[1], q[3], high, 2);
}
// The rows that those four lanes' pointers stand for.
template <class T>
__device__ __forceinline__ void rows_of_four(T* own, T* (&rows)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rows[i] = reinterpret_cast<T*>(__shfl_sync(FULL_MASK, (unsigned long long)own, (threadIdx.x & 28) | i));
}

// What one CTA index stands for: the pair of query tiles of one kv head.
struct PtPair {
    int g, seq, row0, tokens, pos0;   // kv head, table row, first query row, tokens, position of the first
    int end, first, sinks;            // keys that some row sees: [first, end) and [0, sinks)
    int ns, wb, j0, nkt;              // key tiles: of the sinks, first of the window; this CTA's first and number (-1: no such pair)
    int slot;                         // PT_SHARED: where its partials go
    __device__ __forceinline__ int key0(int j) const { return PT_KEYS * (j0 + j < ns ? j0 + j : wb + j0 + j - ns); }
};
// pair: its number among `pairs`; the keys in `parts` shares, of which the part-th.
__device__ __forceinline__ PtPair pt_pair(const PagedPrefillArgs& a, int QT, unsigned pair, unsigned pairs, int part,
                                          int parts, bool reporter) {
    PtPair p;
    // the last tiles see the most keys: those of all kv heads go first
    const int x = (int)(pairs - 1 - pair) / a.c.NKV;
    p.g = (int)(pairs - 1 - pair) % a.c.NKV;
    p.nkt = -1;
    p.tokens = 0;
    const RowTile tile = find_row_tile(a, 2 * QT, x, reporter && x == 0 && p.g == 0);
    if (tile.b < 0) return p;
    const SeqRows sr = seq_rows(a, tile.b, false);
    const int i0 = tile.i * 2 * QT;
    p.seq = sr.seq;
    p.row0 = sr.row0 + i0;
    p.tokens = min(2 * QT, sr.nq - i0);
    p.pos0 = sr.len - sr.nq + i0;                      // negative: sees nothing
    p.end = p.pos0 + p.tokens;
    p.first = a.window > 0 ? max(0, p.pos0 + 1 - a.window) : 0;
    p.sinks = min(a.sinks, p.first);
    p.ns = (p.sinks + PT_KEYS - 1) / PT_KEYS;
    p.wb = max(p.first / PT_KEYS, p.ns);
    const int all = p.end <= 0 ? 0 : p.ns + max(0, (p.end + PT_KEYS - 1) / PT_KEYS - p.wb);
    p.j0 = (int)((long long)all * part / parts);
    p.nkt = (int)((long long)all * (part + 1) / parts) - p.j0;
    return p;
}

// ---- PT_SHARED ----
__device__ __forceinline__ PtGroups pt_groups(const PagedPrefillArgs& a, int QT) {
    return PtGroups{a.cu, a.shared, a.seqs, a.lens, a.B, a.n, a.c.n_seqs, a.c.NKV, 2 * QT, (long long)a.c.width << a.c.page_shift};
}
// The line's length and a CTA's share of it; one warp of the grid leaves what the join needs
// to find a pair's partials: the share, then each group's first slot and place in the line.
__device__ __forceinline__ void pt_line(const PagedPrefillArgs& a, const PtGroups& gs, bool leave, unsigned& each, unsigned& lo, unsigned& hi) {
    const int lane = threadIdx.x & 31;
    unsigned pairs = 0, rows = 0, line = 0;
    int2* head = reinterpret_cast<int2*>(a.ws);
    float own = 0.f;           // the rows' own keys, about
    for (int b = lane; b < a.n; b += 32) own += max(0, a.lens[b]);
    for (int g0 = 0; g0 < a.B; g0 += 32) {
        unsigned row0, line0;
        const PtGroup r = pt_scan(gs, g0, pairs, rows, line, row0, line0);
        own -= (float)r.nq * r.keys;
        const int g = g0 + lane;
        if (leave && g < a.B) head[1 + g] = make_int2((int)row0, (int)line0);
    }
    own = fmaxf(0.f, warp_sum(own));
    const int sms = prefix_sms(line, pairs, own * a.c.NKV * a.c.D * 4.f, gridDim.x);
    each = max((unsigned)PT_SHARE, (line + sms - 1) / max(1, sms));
    if (leave && lane == 0) head[0] = make_int2((int)each, (int)line);
    lo = min(line, blockIdx.x * each);
    hi = min(line, lo + each);
}
// The pair at place `at` of the line and the key tiles that the CTA has of it from there on.
__device__ __forceinline__ PtPair pt_shared(const PtGroups& a, int QT, unsigned at, unsigned hi) {
    PtPair p;
    p.nkt = -1;
    p.tokens = 0;
    if (at >= hi) return p;
    unsigned pairs = 0, rows = 0, line = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
        unsigned row0, line0;
        const PtGroup mine = pt_scan(a, g0, pairs, rows, line, row0, line0);
        const unsigned hit =
            __ballot_sync(FULL_MASK, at >= line0 && at - line0 < (unsigned)mine.nx * a.NKV * (unsigned)mine.tiles);
        if (!hit) continue;
        const int src = __ffs(hit) - 1;
        const PtGroup r = pt_group(a, g0 + src);
        const unsigned off = at - __shfl_sync(FULL_MASK, line0, src);
        // a kv head's pairs side by side: they read the same keys at about the same time
        const int pi = (int)(off / (unsigned)r.tiles), x = pi % r.nx;
        p.g = pi / r.nx;
        p.seq = r.seq;
        p.row0 = r.row0 + x * 2 * QT;
        p.tokens = min(2 * QT, r.nq - x * 2 * QT);
        p.pos0 = 0;
        p.end = r.keys;
        p.first = p.sinks = p.ns = p.wb = 0;
        p.j0 = (int)(off % (unsigned)r.tiles);
        p.nkt = (int)min((unsigned)(r.tiles - p.j0), hi - at);
        // a slot for each of the pair's rows, after those of all pairs before, and a pair's rows further for
        // each CTA: pairs and CTAs both only rise along the line, one of them at each step, so no two share one
        p.slot = (int)__shfl_sync(FULL_MASK, row0, src) + p.g * r.nq + x * 2 * QT + (int)blockIdx.x * 2 * QT;
        break;
    }
    return p;
}

// Asks for a CTA that has not started; 16 bytes of answer, counted on bar.
__device__ __forceinline__ void try_cancel(uint32_t answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The answer: whether there was one, and its index in the grid.
__device__ __forceinline__ bool cancelled(uint32_t answer, unsigned& cta) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(answer)
        : "memory");
    cta = x;
    return ok != 0;
}

template <class E, int DP, int FORM>
__global__ void __launch_bounds__(PT_THREADS, 1)
    k_paged_prefill_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, PagedPrefillArgs a) {
    using L = PtSmem<DP>;
    constexpr int NS = L::NS;
    constexpr bool SPLIT = FORM == PT_SPLIT, SHARED = FORM == PT_SHARED;
    constexpr int TERMS = SHARED ? 2 : 1;              // values of the type that a weight is the sum of
    extern __shared__ uint8_t pt_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pt_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
    uint64_t* s_full = bar + 0;     // [query tile][buffer]
    uint64_t* p_full = bar + 4;     // [query tile][buffer]
    uint64_t* o_full = bar + 8;     // [query tile][buffer]: P . V of that buffer's tile is complete
    uint64_t* o_free = bar + 12;    // [query tile] O of a finished pair is in registers
    uint64_t* q_full = bar + 14;
    uint64_t* q_empty = bar + 15;
    uint64_t* next_full = bar + 16;   // [2] answer of the it-th request in answers[it % 2]
    uint64_t* next_empty = bar + 18;  // [2]
    uint64_t* answers = bar + 20;     // [2] of 16 bytes
    uint64_t* kv_full = bar + 24;     // [NS]: slot i % NS holds K (i even) or V (i odd) of the (i / 2)-th key tile
    uint64_t* kv_empty = bar + 40;    // [NS]
    uint64_t* v_raw = bar + 56;       // [NS / 2] V as it came, before the edge warp has seen it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 64);
    int* sflag = reinterpret_cast<int*>(bar + 65);   // failed
    // A wait names a phase by its parity, so whoever waits on a barrier sees every
    // one of its phases in turn.

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);    // the warps of a query tile
            mbar_init(&o_full[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&o_free[t], 4);
            mbar_init(&next_full[t], 1);
            mbar_init(&next_empty[t], 12);   // the warps that read the answer
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);               // both MMA warps
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 2);
            if (i & 1) mbar_init(&v_raw[i >> 1], 1);
        }
        sflag[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == PT_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    const int D = a.c.D, G = a.NH / a.c.NKV;
    const int QT = PT_ROWS / G;                        // tokens of a query tile
    const int parts = SPLIT ? a.parts : 1, part = SPLIT ? (int)(blockIdx.x % parts) : 0;   // (a cluster's CTAs)
    unsigned first_pair = blockIdx.x / parts, pairs_all = gridDim.x / parts;
    pdl_wait();
    if (SHARED) {   // (then these are the CTA's share of the line)
        pdl_trigger();   // the rows' own keys do not need this grid's results
        unsigned each;
        pt_line(a, pt_groups(a, QT), blockIdx.x == 0 && warp == 0, each, first_pair, pairs_all);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // By a whole warp: true once every lane's barrier has completed its phase, false after
    // the bounded time.  (The first try, nearly always the last, is a poll and a vote: a
    // loop of each lane's own took 300 cycles of a step's 2000.)
    auto wait_at = [&](uint32_t addr, uint32_t parity) {
        if (__all_sync(FULL_MASK, mbar_try_wait(addr, parity))) return true;
        const long long t0 = clock64();
        while (!__all_sync(FULL_MASK, mbar_try_wait(addr, parity)))
            if (__any_sync(FULL_MASK, clock64() - t0 > TC_WAIT_CYCLES)) return false;
        return true;
    };
    auto wait_all = [&](uint64_t* b, int parity) { return wait_at(smem_u32(b), (uint32_t)parity & 1u); };
    // the CTA index (SHARED: the place in the line) after the it-th pair's: false when there is none left (or, ok = false, no answer)
    auto take_next = [&](int it, unsigned& cta, bool& ok, int nkt) {
        if (SPLIT) return false;
        if (SHARED) return walk_on(cta, nkt, pairs_all);
        if (!wait_all(&next_full[it & 1], it >> 1)) {
            ok = false;
            return false;
        }
        const bool got = cancelled(smem_u32(answers + 2 * (it & 1)), cta);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&next_empty[it & 1]);
        return got;
    };

    auto pair_at = [&](unsigned cta, bool reporter) {
        if constexpr (SHARED) return pt_shared(pt_groups(a, QT), QT, cta, pairs_all);
        else return pt_pair(a, QT, cta, pairs_all, part, parts, reporter);
    };

    if (warp >= PT_TMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PT_REGS_REST));
    if (warp == PT_TMA) {   // ------------------------------------- TMA producer
        const int P = 1 << a.c.page_shift;
        const int box = min(P, PT_KEYS);               // rows of a box
        const int boxes = PT_KEYS / box;               // of a tile: lane i < boxes looks up box i's page
        unsigned cta = first_pair;
        int issued = 0, pairs = 0, it = 0;             // slots and pairs with keys so far
        // The slots of K(j) and V(j) are waited for together (a wait for the phase before a
        // barrier's first passes), and one lane issues a tile's copies: with a wait, a page
        // and a choice of map for each of the two, this warp's 2000 cycles a tile set the
        // kernel's pace, the copies themselves take 330.
        int slot = 0;
        uint32_t empty = 1;
        const uint32_t empty_at = smem_u32(kv_empty);
        bool ok = true, asked = false;
        for (;; ++it) {
            PtPair p = pair_at(cta, part == 0);
            if (p.nkt > 0) {
                // The page of the lane's box of tile j, if some row sees its keys.  What it
                // loads is looked at two tiles later, so that nothing waits for it.
                struct Entry {
                    int page;
                    bool seen;
                };
                auto look_up = [&](int j) {
                    Entry e{0, false};
                    if (j >= p.nkt) return e;
                    const int k0 = p.key0(j) + lane * box;
                    e.seen = lane < boxes && k0 < p.end && (k0 + box > p.first || k0 < p.sinks);
                    if (e.seen) e.page = a.c.table[(size_t)p.seq * a.c.width + (k0 >> a.c.page_shift)];
                    return e;
                };
                Entry e0 = look_up(0), e1 = look_up(1);
                if (SHARED) {                          // (asked for beside the pages)
                    p.end = min(p.end, pt_seen(pt_groups(a, QT), p.row0, p.tokens));
                    e0.seen &= p.key0(0) + lane * box < p.end;
                    e1.seen &= p.key0(1) + lane * box < p.end;
                }
                const int g = uniform(p.g);
                ok = pairs == 0 || wait_all(q_empty, pairs - 1);
                if (!ok) break;
                if (lane == 0) {                       // tokens beyond the sequence's: whatever follows, or zeros
                    mbar_expect_tx(q_full, 2 * L::KB * QT * G * 128);
                    for (int t = 0; t < 2; ++t)
                        for (int kb = 0; kb < L::KB; ++kb)
                            tma_load_3d(sm + L::OFF_Q + t * L::QTILE + kb * PT_ROWS * 128, &tmQ, kb * 64, p.g * G,
                                        p.row0 + t * QT, q_full);
                }
                ++pairs;
                for (int j = 0; j < p.nkt; ++j, issued += 2) {
                    bool known = e0.page >= 0 && e0.page < a.c.n_pages;
                    if (e0.seen && !known) raise_status(a.status, EMBER_ERR_INVALID_ARG);
                    const int page = e0.seen && known ? e0.page : a.c.n_pages;   // n_pages reads as zeros
                    e0 = e1;
                    e1 = look_up(j + 2);
                    int pages[PT_KEYS / 16];
#pragma unroll
                    for (int i = 0; i < PT_KEYS / 16; ++i) pages[i] = __shfl_sync(FULL_MASK, page, i);
                    const int s = uniform(slot), row = uniform(p.key0(j) & (P - 1));   // (0 where a tile has several boxes)
                    if (!(ok = wait_at(empty_at + (s + (lane & 1)) * 8, empty))) break;
                    if (elect_one()) {
                        uint64_t *kf = &kv_full[s], *vf = &v_raw[s >> 1];
                        uint8_t* d = sm + L::OFF_KV + s * L::TILE;
                        mbar_expect_tx(kf, L::TILE);
#pragma unroll
                        for (int i = 0; i < PT_KEYS / 16; ++i)
                            if (i < boxes)
#pragma unroll
                                for (int kb = 0; kb < L::KB; ++kb)
                                    tma_load_4d(d + kb * PT_KEYS * 128 + i * box * 128, &tmK, kb * 64, row, g, pages[i], kf);
                        mbar_expect_tx(vf, L::TILE);
#pragma unroll
                        for (int i = 0; i < PT_KEYS / 16; ++i)
                            if (i < boxes)
#pragma unroll
                                for (int kb = 0; kb < L::KB; ++kb)
                                    tma_load_4d(d + L::TILE + kb * PT_KEYS * 128 + i * box * 128, &tmV, kb * 64, row, g,
                                                pages[i], vf);
                    }
                    __syncwarp();
                    if ((slot += 2) == NS) slot = 0, empty ^= 1;
                }
                if (!ok) break;
            }
            // asked for only now, a ring's worth of tiles before the pair ends: a CTA
            // that asked at its start would hold work that another could begin first
            if (FORM == PT_WHOLE) {
                ok = it < 2 || wait_all(&next_empty[it & 1], (it >> 1) - 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_expect_tx(&next_full[it & 1], 16);
                    try_cancel(smem_u32(answers + 2 * (it & 1)), &next_full[it & 1]);
                }
                __syncwarp();
                asked = true;
            }
            if (!take_next(it, cta, ok, p.nkt)) break;
            asked = false;
        }
        if (!ok && lane == 0) {
            sflag[0] = 1;
            // what is in flight lands before the block ends
            if (asked) (void)mbar_wait(&next_full[it & 1], (uint32_t)(it >> 1) & 1u);
            if (pairs) (void)mbar_wait(q_full, (uint32_t)(pairs - 1) & 1u);
            for (int i = max(0, issued - NS); i < issued; ++i)
                (void)mbar_wait(i & 1 ? &v_raw[i % NS >> 1] : &kv_full[i % NS], (uint32_t)(i / NS) & 1u);
        }
    } else if (warp == PT_EDGE) {   // ----------------------------- V rows that nobody sees become zeros
        unsigned cta = first_pair;
        int base = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            PtPair p = pair_at(cta, false);
            const int nkt = max(0, p.nkt);
            if (SHARED && nkt > 0) p.end = min(p.end, pt_seen(pt_groups(a, QT), p.row0, p.tokens));
            for (int j = 0; ok && j < nkt; ++j) {
                const int i = 2 * (base + j) + 1, s = i % NS, key0 = p.key0(j);
                ok = wait_all(&v_raw[s >> 1], i / NS);
                if (ok && (key0 + PT_KEYS > p.end || (key0 < p.first && key0 + PT_KEYS > p.sinks))) {
                    const uint32_t v = smem_u32(sm + L::OFF_KV + s * L::TILE);
                    auto zero = [&](int r0, int r1) {   // rows [r0, r1): 16 bytes a lane
#pragma unroll 4
                        for (int e = max(r0, 0) * 8 * L::KB + lane; e < min(r1, PT_KEYS) * 8 * L::KB; e += 32)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             v + (L::KB == 1 ? e * 16
                                                             : ((e >> 3) & 1) * (PT_KEYS * 128) + (e >> 4) * 128 + (e & 7) * 16)),
                                         "r"(0)
                                         : "memory");
                    };
                    zero(p.sinks - key0, p.first - key0);
                    zero(p.end - key0, PT_KEYS);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (ok && lane == 0) mbar_arrive(&kv_full[s]);
            }
            if (!ok) break;
            base += nkt;
            if (!take_next(it, cta, ok, p.nkt)) break;
        }
        if (!ok && lane == 0) sflag[0] = 1;
    } else {   // -------------------------------------------------- MMA issuers, one for each query tile
        const int t = warp - PT_MMA;
        constexpr uint32_t type = E::bf16 ? idesc_bf16(0, 0) : idesc_f16(0, 0);
        constexpr uint32_t idS = type | idesc_f16(PT_ROWS, PT_KEYS);
        constexpr uint32_t idO = type | idesc_f16(PT_ROWS, DP) | IDESC_B_MN;
        // Issuing is the tensor pipe's pace-maker when a product takes 45 to 64 cycles:
        // operands are warp-uniform, descriptors one addition each.
        const uint32_t tm = uniform(tmem);
        const uint32_t kv0 = uniform(smem_u32(sm + L::OFF_KV));
        const uint32_t col_s = tm + uniform(t * 128), col_o = tm + uniform(L::col_o(t));
        const uint32_t dq = uniform(desc_k(smem_u32(sm + L::OFF_Q + t * L::QTILE)));
        const uint32_t dk0 = uniform(desc_k(kv0)), dv0 = uniform(desc_mn(kv0, PT_KEYS * 128));
        const uint32_t p_at = smem_u32(&p_full[2 * t]), o_at = smem_u32(&o_full[2 * t]), s_at = smem_u32(&s_full[2 * t]);
        const uint32_t free_at = smem_u32(&o_free[t]), full_at = smem_u32(kv_full), empty_at = smem_u32(kv_empty);
        auto commit = [](uint32_t at) {
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(at) : "memory");
        };
        auto mma_s = [&](uint32_t c, uint32_t dk) {   // S = Q . K^T
#pragma unroll
            for (int kb = 0; kb < L::KB; ++kb)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(c, dq + ((kb * PT_ROWS * 128 + k * 32) >> 4), dk + ((kb * PT_KEYS * 128 + k * 32) >> 4), idS, kb | k);
        };
        auto mma_pv = [&](uint32_t c, uint32_t dv, bool acc) {   // O += P (TMEM) . V
#pragma unroll
            for (int i = 0; i < TERMS; ++i)
#pragma unroll
                for (int k = 0; k < PT_KEYS / 16; ++k)
                    mma_ts(col_o, c + i * (PT_KEYS / 2) + k * 8, dv + ((k * 16 * 128) >> 4), idO, acc || i || k);
        };
        // one lane issues f() after everything the warp has waited for
        auto issue = [&](auto f) {
            if (elect_one()) {
                tc_fence_after();
                f();
            }
            __syncwarp();
        };
        unsigned cta = first_pair;
        int base = 0, pairs = 0;   // key tiles and pairs with keys so far
        int mine = 0, with = 0;    // those in which this query tile has tokens
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const PtPair p = pair_at(cta, false);
            const int nkt = max(0, p.nkt);
            auto slot_full = [&](int i) { return &kv_full[i % NS]; };
            if (nkt > 0 && !(ok = wait_all(q_full, pairs))) break;
            if (t * QT >= p.tokens) {
                // no tokens: the other tile alone, this warp only hands its half of the slots back
                for (int i = 2 * base; ok && i < 2 * (base + nkt); ++i) {
                    ok = wait_all(slot_full(i), i / NS);
                    if (ok && lane == 0) mbar_arrive(&kv_empty[i % NS]);
                }
                if (ok && nkt > 0 && lane == 0) mbar_arrive(q_empty);
            } else {
                // S of the pair's key tile j; then K (after the last one Q) is free
                auto first_s = [&](int j) {
                    const int n = base + j;
                    if (!(ok = wait_all(slot_full(2 * n), 2 * n / NS))) return;
                    const uint32_t b = uniform((mine + j) & 1), dk = dk0 + uniform(2 * n % NS) * (L::TILE >> 4);
                    issue([&] {
                        mma_s(col_s + b * 64, dk);
                        commit(s_at + b * 8);
                        umma_commit(&kv_empty[2 * n % NS]);
                        if (j + 1 == nkt) umma_commit(q_empty);
                    });
                };
                if (nkt > 0) first_s(0);
                if (ok && nkt > 1) first_s(1);
                // What a step waits for and its operands are carried along, not computed: the
                // pipe idles from the end of one step's issue to the start of the next.
                int sv = (2 * base + 1) % NS, sk = (2 * base + 4) % NS;   // slots of V(j) and K(j + 2), their phases
                uint32_t vp = (2 * base + 1) / NS & 1, kp = (2 * base + 4) / NS & 1, buf = mine & 1, pp = mine >> 1 & 1;
                const int role = lane & 3;
                for (int j = 0; j < nkt; ++j) {
                    // P . V(j) frees the buffer that S(j + 2) takes (MMAs of one thread run
                    // in the order of issue), and S(j + 1) is there already
                    const bool more = j + 2 < nkt;
                    // P(j), V(j), K(j + 2) and, before a pair's first P . V, the end of the
                    // pair before's use of O: a lane each, so that one poll sees them all
                    uint32_t at = p_at + buf * 8, parity = pp;
                    if (role == 1) at = full_at + sv * 8, parity = vp;
                    if (role == 2 && more) at = full_at + sk * 8, parity = kp;
                    if (role == 3 && j == 0 && with > 0) at = free_at, parity = (with - 1) & 1;
                    const uint32_t c = col_s + uniform(buf) * 64, dv = dv0 + uniform(sv) * (L::TILE >> 4),
                                   dk = dk0 + uniform(sk) * (L::TILE >> 4);
                    const uint32_t o_bar = o_at + buf * 8, s_bar = s_at + buf * 8, v_bar = empty_at + sv * 8, k_bar = empty_at + sk * 8;
                    if (!(ok = wait_at(at, parity))) break;
                    issue([&] {
                        mma_pv(c, dv, j > 0);
                        commit(o_bar);
                        commit(v_bar);
                        if (more) {
                            mma_s(c, dk);
                            commit(s_bar);
                            commit(k_bar);
                            if (j + 3 == nkt) umma_commit(q_empty);
                        }
                    });
                    pp ^= buf;
                    buf ^= 1;
                    if ((sv += 2) >= NS) sv -= NS, vp ^= 1;
                    if ((sk += 2) >= NS) sk -= NS, kp ^= 1;
                }
                mine += nkt;
                with += nkt > 0;
            }
            if (!ok) break;
            base += nkt;
            pairs += nkt > 0;
            if (!take_next(it, cta, ok, p.nkt)) break;
        }
        if (!ok && lane == 0) sflag[0] = 1;
    }
    } else {   // -------------------------------------------------- softmax warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PT_REGS_ROW));
        constexpr float MOST = 32768.f;               // f16 weights stay finite
        const int t = warp >> 2;                      // query tile: 0 = A, 1 = B
        const int qw = warp & 3;                      // TMEM lane quarter of this warp
        const int r = qw * 32 + lane;                 // row within the tile
        const int tok = t * QT + r / G, h = r % G;    // token of the pair, head of the group
        const uint32_t lane_off = (uint32_t)(qw * 32) << 16;
        const uint32_t tO = tmem + L::col_o(t) + lane_off;
        const float sc = a.scale * LOG2E;             // > 0
        unsigned cta = first_pair;
        int base = 0;                                 // key tiles so far
        bool ok = true;
        PtPair pair;                                  // (SPLIT: the one pair)
        for (int it = 0; ok; ++it) {
        const PtPair p = pair_at(cta, false);
        const int nkt = t * QT < p.tokens ? max(0, p.nkt) : 0;   // (without tokens the tile has no products either)
        const bool live = p.nkt >= 0 && r < QT * G && tok < p.tokens;
        int qp = p.pos0 + min(tok, p.tokens - 1);         // its position (rows that are not live: the last one's)
        if (SHARED && p.nkt >= 0) qp = min(p.end, a.lens[p.row0 + min(tok, p.tokens - 1)]) - 1;   // its last key here
        float m = SOFTMAX_FLOOR, l = 0.f;             // reference maximum (of s * sc) less LIFT, sum of 2^(s sc - m)
        for (int j = 0; j < nkt; ++j) {
            const int n = base + j;
            const uint32_t tS = tmem + L::col_s(t, n & 1) + lane_off;
            uint32_t v[PT_KEYS];                      // the row's products, then its weights
            uint32_t left[PT_KEYS / 2];               // (two terms) what their rounding left
            // S(n); and P . V(n - 2), complete before it, for its phase to be seen
            const bool odd_lane = n >= 2 && (lane & 1);
            if (!wait_all((odd_lane ? o_full : s_full) + 2 * t + (n & 1), odd_lane ? (n >> 1) - 1 : n >> 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // column c is visible when c < hi and (c >= lo or c < sk)
            const int key0 = p.key0(j);
            const int hi = qp - key0 + 1;
            const int lo = a.window > 0 ? qp - a.window + 1 - key0 : 0;
            const int sk = a.sinks - key0;
            const bool whole = __all_sync(FULL_MASK, hi >= PT_KEYS && (lo <= 0 || sk >= PT_KEYS));
            auto scores = [&]() {                     // the row's products, -inf where hidden
#pragma unroll
                for (int c = 0; c < PT_KEYS; c += 32) tmem_ld32(tS + c, v + c);
                tmem_ld_wait();
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < PT_KEYS / 32; ++k) {   // a bit a column: no branches
                        const uint32_t see = below(hi - 32 * k) & (~below(lo - 32 * k) | below(sk - 32 * k));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[32 * k + i] = (see >> i) & 1u ? v[32 * k + i] : 0xff800000u;
                    }
                }
            };
            auto largest = [&]() {                    // of the row's scores
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < PT_KEYS; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = max3(mx[i], __uint_as_float(v[c + 2 * i]), __uint_as_float(v[c + 2 * i + 1]));
                return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sc;
            };
            auto weigh = [&]() {                      // scores -> weights, packed; their sum
                const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
                float2 rs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) rs[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < PT_KEYS; c += 2) {
                    float2 w = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, m2);
                    w.x = ex2(w.x);
                    w.y = ex2(w.y);
                    rs[(c >> 1) & 3] = add2(rs[(c >> 1) & 3], w);
                    const uint32_t x = TERMS == 2 && E::bf16 ? __byte_perm(__float_as_uint(w.x), __float_as_uint(w.y), 0x7632)
                                                             : E::pack(w.x, w.y);   // (cut off: the second term has the rest)
                    v[c >> 1] = x;
                    if (TERMS == 2) {
                        const float2 y = add2(w, make_float2(-E::lo(x), -E::hi(x)));
                        left[c >> 1] = E::pack(y.x, y.y);
                    }
                }
                const float2 r2 = add2(add2(rs[0], rs[1]), add2(rs[2], rs[3]));
                return r2.x + r2.y;
            };
            // The reference maximum is looked for only while a row has none, and when the
            // tile's weights against the old one sum to more than MOST: until then every
            // weight is exact to the same relative rounding, and within f16's range.
            // (Rows that are not live hold anything and ask for nothing.)
            scores();
            const bool look = live && m == SOFTMAX_FLOOR;
            if (__any_sync(FULL_MASK, look)) m = look ? fmaxf(m, largest() - E::LIFT) : m;
            float sum = weigh();
            const bool move = live && !(sum <= MOST);
            const bool any_move = __any_sync(FULL_MASK, move);
            float corr = 1.f;
            if (any_move) {
                scores();                             // (S is whole until P is stored)
                const float mnew = move ? fmaxf(m, largest() - E::LIFT) : m;
                corr = ex2(m - mnew);
                l *= corr;
                m = mnew;
                sum = weigh();
            }
            if (any_move && j > 0) {   // O is touched: P . V(j - 1) must be complete
                if (!wait_all(&o_full[2 * t + ((n - 1) & 1)], (n - 1) >> 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < DP; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c0, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                    tmem_st16(tO + c0, o);
                    tmem_st16(tO + c0 + 16, o + 16);
                }
            }
            // over S(j), all of it read; P . V(j - 2), the last reader here, was issued before S(j)
#pragma unroll
            for (int c = 0; c < PT_KEYS / 2; c += 16) {
                tmem_st16(tS + c, v + c);
                if (TERMS == 2) tmem_st16(tS + PT_KEYS / 2 + c, left + c);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + (n & 1)]);
            l += sum;
        }
        if (SPLIT) {   // the rows as they are into shared memory; joined below
            if (ok && nkt > 0) {
                const int last = base + nkt - 1;
                ok = wait_all(&o_full[2 * t + (last & 1)], last >> 1);
                tc_fence_after();
            }
            // both query tiles' products are complete: nothing reads Q, K or V any more
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const int at = t * PT_ROWS + r;
            float* mine = reinterpret_cast<float*>(sm) + at * DP;
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                if (nkt > 0) {
                    tmem_ld32(tO + c, o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4*>(mine + 4 * (((c + i) / 4) ^ (r & 7))) =
                        nkt > 0 ? make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]) : make_uint4(0u, 0u, 0u, 0u);
            }
            reinterpret_cast<float2*>(sm + 2 * PT_ROWS * DP * 4)[at] = make_float2(m, l);
            pair = p;
            break;
        }
        if (SHARED) {   // the rows as they are; joined by another kernel
            const size_t at = (size_t)(unsigned)p.slot * G + t * QT * G + r;   // (slots are of a token's G rows)
            const bool store = live && at < (size_t)a.slots * G;
            float* own = store ? a.ws + a.ws_head + at * D : nullptr;
            if (ok && nkt > 0) {
                const int last = base + nkt - 1;
                ok = wait_all(&o_full[2 * t + (last & 1)], last >> 1);
                tc_fence_after();
                if (ok) {
                    // (16 bytes of 32 rows each at a time took 4 us for rows of 64, 8 us for 128)
                    float* rows[4];
                    rows_of_four(own, rows);
#pragma unroll
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            uint4 q[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) q[k] = make_uint4(o[i + 4 * k], o[i + 4 * k + 1], o[i + 4 * k + 2], o[i + 4 * k + 3]);
                            transpose_four(q);
                            const int d = c + i + 4 * (lane & 3);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (rows[k] && d < D) *reinterpret_cast<uint4*>(rows[k] + d) = q[k];
                        }
                    }
                    if (store)
                        reinterpret_cast<float2*>(a.ws + a.ws_head + (size_t)a.slots * G * D)[at] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[t]);
                }
            }
            if (!ok) break;
            base += nkt;
            if (!take_next(it, cta, ok, p.nkt)) break;
            continue;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t w[DP / 2];                           // the row of the output
#pragma unroll
        for (int c = 0; c < DP / 2; ++c) w[c] = 0u;
        if (ok && nkt > 0) {
            const int last = base + nkt - 1;
            ok = wait_all(&o_full[2 * t + (last & 1)], last >> 1);
            tc_fence_after();
            if (ok) {
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t x = E::pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        w[c / 2 + i] = l == 0.f ? 0u : x;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[t]);
            }
        }
        if (!ok) break;
        {
            const long long row = p.row0 + tok;
            uint16_t* own = live ? a.out + row * a.ld_out + (long long)(p.g * G + h) * D : nullptr;
            uint16_t* rows[4];
            rows_of_four(own, rows);
#pragma unroll
            for (int c0 = 0; c0 < DP; c0 += 32) {
                if (c0 >= D) break;
                uint4 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t* x = w + c0 / 2 + 4 * i;
                    q[i] = make_uint4(x[0], x[1], x[2], x[3]);
                }
                transpose_four(q);
                const int c = c0 + 8 * (lane & 3);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rows[i] && c < D) *reinterpret_cast<uint4*>(rows[i] + c) = q[i];
            }
            if (a.lse && live) a.lse[row * a.NH + p.g * G + h] = l == 0.f ? -INFINITY : m * LN2 + logf(l);
        }
        base += nkt;
        if (!take_next(it, cta, ok, p.nkt)) break;
        }
        if (!ok) sflag[0] = 1;
        if (SPLIT) {
            cluster_sync_all();
            // rows [part, part + 1) * 256 / parts, eight dimensions a thread
            const uint32_t o_at = smem_u32(sm), ml_at = o_at + 2 * PT_ROWS * DP * 4;
            const int rows = 2 * PT_ROWS / parts;
            for (int e = threadIdx.x; e < rows * (DP / 8); e += 256) {
                const int at = part * rows + e / (DP / 8), c = e % (DP / 8), rr = at % PT_ROWS;
                const int tk = at / PT_ROWS * QT + rr / G, hh = rr % G;
                if (rr >= QT * G || tk >= pair.tokens || c * 8 >= D) continue;
                float mx = SOFTMAX_FLOOR, sum = 0.f, acc[8];
                float2 ml[PT_PARTS];
#pragma unroll
                for (int i = 0; i < PT_PARTS; ++i)
                    if (i < parts) {
                        ml[i] = ld_cluster2(ml_at + at * 8, i);
                        mx = fmaxf(mx, ml[i].x);
                    }
#pragma unroll
                for (int d = 0; d < 8; ++d) acc[d] = 0.f;
#pragma unroll
                for (int i = 0; i < PT_PARTS; ++i)
                    if (i < parts) {
                        const float f = ex2(ml[i].x - mx);
                        sum = fmaf(ml[i].y, f, sum);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float4 x = ld_cluster4(o_at + (at * DP + 4 * ((2 * c + q) ^ (rr & 7))) * 4, i);
                            acc[4 * q] = fmaf(x.x, f, acc[4 * q]);
                            acc[4 * q + 1] = fmaf(x.y, f, acc[4 * q + 1]);
                            acc[4 * q + 2] = fmaf(x.z, f, acc[4 * q + 2]);
                            acc[4 * q + 3] = fmaf(x.w, f, acc[4 * q + 3]);
                        }
                    }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int d = 0; d < 8; ++d) acc[d] = sum == 0.f ? 0.f : acc[d] * inv;
                const long long row = pair.row0 + tk;
                *reinterpret_cast<uint4*>(a.out + row * a.ld_out + (long long)(pair.g * G + hh) * D + c * 8) =
                    make_uint4(E::pack(acc[0], acc[1]), E::pack(acc[2], acc[3]), E::pack(acc[4], acc[5]), E::pack(acc[6], acc[7]));
                if (a.lse && c == 0)
                    a.lse[row * a.NH + pair.g * G + hh] = sum == 0.f ? -INFINITY : mx * LN2 + logf(sum);
            }
            cluster_sync_all();                       // no CTA leaves while another reads its shared memory
        }
    }
    if (SPLIT && warp >= PT_TMA) {
        cluster_sync_all();
        cluster_sync_all();
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sflag[0]) raise_status(a.status, EMBER_ERR_TIMEOUT);
    if (warp == PT_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

template <class E, int DP>
cudaError_t launch_dp(const PagedPrefillMaps& m, PagedPrefillArgs a, int sms, cudaStream_t s) {
    constexpr int SMEM = PtSmem<DP>::TOTAL;
    const int per = 2 * (PT_ROWS / (a.NH / a.c.NKV));
    const unsigned pairs = (unsigned)((((long long)a.n + per - 1) / per + a.B) * a.c.NKV);
    // CTAs of a cluster that share a pair's keys: as many as leave every one an SM and
    // two key tiles.  (`pairs` is the most there can be; about B / 2 of them are not.)
    const long long about = max((long long)a.B, a.n / per + a.B / 2ll) * a.c.NKV;
    const long long keys = (long long)a.c.width << a.c.page_shift;
    const long long seen = a.window > 0 ? min(keys, (long long)a.window + a.sinks + per) : keys;
    a.parts = 1;
    while (a.parts < PT_PARTS && about * a.parts * 2 <= sms && seen >= 4ll * a.parts * PT_KEYS) a.parts *= 2;
    const auto& mq = *reinterpret_cast<const CUtensorMap*>(m.q);
    const auto& mk = *reinterpret_cast<const CUtensorMap*>(m.k);
    const auto& mv = *reinterpret_cast<const CUtensorMap*>(m.v);
    if (a.parts > 1) {
        auto k = k_paged_prefill_tc<E, DP, PT_SPLIT>;
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        return launch_cluster_k(k, dim3(pairs * a.parts), dim3(PT_THREADS), SMEM, a.parts, s, mq, mk, mv, a);
    }
    auto k = k_paged_prefill_tc<E, DP, PT_WHOLE>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(pairs), dim3(PT_THREADS), SMEM, s, mq, mk, mv, a);
}

template <class E, int DP>
cudaError_t launch_shared(const PagedPrefillMaps& m, const PagedPrefillArgs& a, int sms, cudaStream_t s) {
    constexpr int SMEM = PtSmem<DP>::TOTAL;
    auto k = k_paged_prefill_tc<E, DP, PT_SHARED>;
    static OncePerDevice once;
    const cudaError_t e = once([&] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(sms), dim3(PT_THREADS), SMEM, s, *reinterpret_cast<const CUtensorMap*>(m.q),
                    *reinterpret_cast<const CUtensorMap*>(m.k), *reinterpret_cast<const CUtensorMap*>(m.v), a);
}

}  // namespace

PagedSharedWs paged_shared_ws(int B, int n_groups, int NH, int NKV, int D, int sms) {
    const int per = 2 * (PT_ROWS / (NH / NKV));
    PagedSharedWs w;
    w.head = (2 * (1 + n_groups) + 3) & ~3;
    w.slots = (int)std::min<long long>((long long)B * NKV + (long long)sms * per, INT_MAX);
    w.rows_per_pair = per;
    w.floats = w.head + (size_t)w.slots * (NH / NKV) * (D + 2);
    return w;
}

cudaError_t launch_paged_shared(const PagedPrefillArgs& a, const PagedPrefillMaps& m, int sms, cudaStream_t s) {
    if (a.c.bf16) return a.c.D <= 64 ? launch_shared<ElemBf16, 64>(m, a, sms, s) : launch_shared<ElemBf16, 128>(m, a, sms, s);
    return a.c.D <= 64 ? launch_shared<ElemF16, 64>(m, a, sms, s) : launch_shared<ElemF16, 128>(m, a, sms, s);
}

bool paged_prefill_maps(const PagedPrefillArgs& a, PagedPrefillMaps& m) {
    const PagedView& c = a.c;
    const int G = a.NH / c.NKV, per = 2 * (PT_ROWS / G);
    if ((((long long)a.n + per - 1) / per + a.B) * c.NKV > 0x7fffffffll) return false;   // the grid
    const uint64_t qd[3] = {(uint64_t)c.D, (uint64_t)a.NH, (uint64_t)a.n};
    const uint64_t qs[2] = {(uint64_t)c.D * 2, (uint64_t)a.ld_q * 2};
    const uint32_t qb[3] = {64u, (uint32_t)G, (uint32_t)(PT_ROWS / G)};
    const uint64_t dims[4] = {(uint64_t)c.D, 1ull << c.page_shift, (uint64_t)c.NKV, (uint64_t)c.n_pages};
    const uint64_t strides[3] = {(uint64_t)c.row_stride * 2, (uint64_t)c.head_stride * 2, (uint64_t)c.page_stride * 2};
    const uint32_t box[4] = {64u, (1u << c.page_shift) < (unsigned)PT_KEYS ? 1u << c.page_shift : (unsigned)PT_KEYS, 1u, 1u};
    return encode_map_bf16(m.q, a.q, 3, qd, qs, qb) && encode_map_bf16(m.k, c.k, 4, dims, strides, box) &&
           encode_map_bf16(m.v, c.v, 4, dims, strides, box);
}

cudaError_t launch_paged_prefill_tc(const PagedPrefillArgs& a, const PagedPrefillMaps& m, int sms, cudaStream_t s) {
    if (a.c.bf16) return a.c.D <= 64 ? launch_dp<ElemBf16, 64>(m, a, sms, s) : launch_dp<ElemBf16, 128>(m, a, sms, s);
    return a.c.D <= 64 ? launch_dp<ElemF16, 64>(m, a, sms, s) : launch_dp<ElemF16, 128>(m, a, sms, s);
}

}  // namespace ember
