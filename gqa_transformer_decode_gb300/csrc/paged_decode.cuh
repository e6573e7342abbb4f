// paged_decode.cuh -- what the one-token attentions share (paged_decode.cu, paged_shared.cu):
// which blocks of keys a row reads, and a block's products and softmax in a warp's registers.
#pragma once

#include <climits>

#include "paged.cuh"

namespace ember {

namespace {

constexpr int PD_WARPS = 4;
constexpr int PD_THREADS = PD_WARPS * 32;
constexpr int PD_STAGES = 2;         // ring stages of a warp
constexpr int pd_ctas_per_sm(int ht) { return ht == 1 ? 3 : 2; }   // registers: 168 or 255 a thread
// Keys of a block: 8 KB of K and V rows either way.
template <int DP>
constexpr int PD_KEYS = DP == 64 ? 32 : 16;

// What a row's keys lie in: its own pages, or those of its group's prefix up to `from` and
// its own from there on, or its own from there on alone (the prefix is another kernel's).
enum PdShare : int { PD_OWN = 0, PD_SHARED = 1, PD_TAIL = 2 };

// Blocks of one sequence: [0, ns) hold its sinks, the rest its window.
struct SeqBlocks {
    int n, ns, wb;       // blocks, blocks of the sinks, first block of the window
    int end, first, sinks;
    int from, prefix;    // PD_SHARED: keys below `from` are those of table row `prefix`
    bool zero;           // nothing visible: the output is zero (PD_TAIL: the row is valid)
    __device__ __forceinline__ int index(int i) const { return i < ns ? i : wb + i - ns; }
};

// The last group that does not begin behind the row, for N rows at once: seven places of the
// interval at a step, asked for together (one place at a step, a row after another: 1024 rows in 64
// groups on 2 kv heads of 64 70 us, so 63).  Whatever the array holds, a row's answer is below n_groups, and the same each time.
template <int N>
__device__ __forceinline__ void find_groups(const PagedDecodeArgs& a, const int (&b)[N], int (&lo)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) lo[e] = 0;
    for (int n = a.n_groups; n > 1;) {
        const int step = (n + 7) / 8;
        int at[N][7];
#pragma unroll
        for (int e = 0; e < N; ++e)
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                const int i = lo[e] + (j + 1) * step;
                at[e][j] = i < a.n_groups ? a.groups[i] : INT_MAX;
            }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            int c = 0;
#pragma unroll
            for (int j = 0; j < 7; ++j) c += at[e][j] <= b[e];
            lo[e] += c * step;
        }
        n = step;
    }
}

// The prefix of row b, found in group lo, if it is in that group and the prefix is valid: its shared keys and
// their table row.
__device__ __forceinline__ int shared_prefix(const PagedDecodeArgs& a, int b, int lo, int& from, int& prefix) {
    const int r0 = a.groups[lo], r1 = a.groups[lo + 1];
    from = a.shared[lo];
    prefix = a.prefixes[lo];
    if (r0 < 0 || r0 > b || b >= r1 || r1 > a.B) return EMBER_ERR_INVALID_ARG;
    if (prefix < 0 || prefix >= a.c.n_seqs) return EMBER_ERR_INVALID_ARG;
    if (from < 0 || from > ((long long)a.c.width << a.c.page_shift)) return EMBER_ERR_CAPACITY;
    return EMBER_OK;
}

template <int KEYS, int SHARE>
__device__ __forceinline__ SeqBlocks seq_blocks(const PagedDecodeArgs& a, int b, int seq, int len, int group, bool report) {
    SeqBlocks r;
    r.n = 0;
    r.ns = r.wb = r.end = r.first = r.sinks = r.from = r.prefix = 0;
    r.zero = false;
    if (seq < 0) return r;                                   // padding: the row is left as it is
    if (seq >= a.c.n_seqs) {
        if (report) raise_status(a.status, EMBER_ERR_INVALID_ARG);
        return r;
    }
    if (len < 0 || len > ((long long)a.c.width << a.c.page_shift)) {
        if (report) raise_status(a.status, EMBER_ERR_CAPACITY);
        return r;
    }
    if (SHARE != PD_OWN) {
        const int e = shared_prefix(a, b, group, r.from, r.prefix);
        if (e != EMBER_OK) {
            if (report) raise_status(a.status, e);
            return r;
        }
    }
    if (SHARE == PD_TAIL) {
        r.zero = true;
        r.end = len;
        r.first = min(r.from, len);
        r.wb = r.first / KEYS;
        r.n = r.first < len ? (len + KEYS - 1) / KEYS - r.wb : 0;
        return r;
    }
    if (len == 0) {
        r.zero = true;
        return r;
    }
    const Visible v(len - 1, a.window, a.sinks);
    r.end = v.end;
    r.first = v.first;
    r.sinks = v.sinks;
    r.ns = (v.sinks + KEYS - 1) / KEYS;
    r.wb = max(v.first / KEYS, r.ns);
    r.n = r.ns + (v.end + KEYS - 1) / KEYS - r.wb;
    return r;
}

template <int KEYS, int SHARE>
__device__ __forceinline__ SeqBlocks seq_blocks(const PagedDecodeArgs& a, int b, bool report) {
    int row[1] = {b}, group[1] = {0};
    const int seq = a.seqs ? a.seqs[b] : b, len = a.lens[b];
    if (SHARE != PD_OWN) find_groups(a, row, group);
    return seq_blocks<KEYS, SHARE>(a, b, seq, len, group[0], report);
}

// Every warp by itself: the line's length, and in which sequence block `x`
// (known once the length is: at(total)) lies.  Four sequences a lane, 128 at a time.
constexpr int PD_SCAN = 4;
template <int KEYS, int SHARE>
__device__ __forceinline__ unsigned scan_chunk(const PagedDecodeArgs& a, int b0, bool report, int (&n)[PD_SCAN],
                                               unsigned& before) {
    const int lane = threadIdx.x & 31;
    unsigned own = 0;
    int seq[PD_SCAN], len[PD_SCAN], row[PD_SCAN], group[PD_SCAN];
#pragma unroll
    for (int e = 0; e < PD_SCAN; ++e) {
        const int b = b0 + PD_SCAN * lane + e;
        seq[e] = b >= a.B ? -1 : a.seqs ? a.seqs[b] : b;
        len[e] = b >= a.B ? 0 : a.lens[b];
        row[e] = b;
        group[e] = 0;
    }
    if (SHARE != PD_OWN) find_groups(a, row, group);
#pragma unroll
    for (int e = 0; e < PD_SCAN; ++e) {
        n[e] = seq_blocks<KEYS, SHARE>(a, row[e], seq[e], len[e], group[e], report).n;
        own += n[e];
    }
    unsigned incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += y;
    }
    before = incl - own;
    return __shfl_sync(FULL_MASK, incl, 31);
}

// A place in the line: block `i` of kv head g of sequence b.
struct Place {
    int b, g, i;
    SeqBlocks s;
};

template <int DP, int HT>
struct PdSmem {
    static constexpr int TILE = PD_KEYS<DP> * DP * 2;             // one K (or V) block
    static constexpr int RING = PD_WARPS * PD_STAGES * 2 * TILE;
    static constexpr int ROW = DP + 4;                            // a head's O row in the merge: no bank conflicts
    static constexpr int SCR = 2 * 8 * HT * ROW * 4;              // O of two warps
    static constexpr int TOTAL = RING + SCR;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// One warp's attention of a group's heads over blocks of keys.  HT: tiles of 8 query heads (1 up
// to G = 8, else 2).
template <class E, int DP, int HT>
struct PdState {
    static constexpr int KEYS = PD_KEYS<DP>, NSUB = KEYS / 16, KS = DP / 16;
    uint32_t qb[HT][KS][2];
    // O^T: rows (dimensions) 16 i + g4 and + 8, columns (heads) 8 t + 2 q4 and + 1
    float o[HT][KS][4];
    float m[HT][2], l[HT][2];            // of heads 8 t + 2 q4 + e, m less LIFT; l over this lane's keys
    // q of the group's heads as B fragments (columns >= G zero); nothing seen yet
    __device__ __forceinline__ void begin(const uint16_t* q, int G, int D) {
        const int lane = threadIdx.x & 31, g4 = lane >> 2, q4 = lane & 3;
#pragma unroll
        for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = 8 * t + g4, col = 16 * kk + 8 * e + 2 * q4;
                    qb[t][kk][e] = h < G && col < D ? *reinterpret_cast<const uint32_t*>(q + h * D + col) : 0u;
                }
#pragma unroll
        for (int t = 0; t < HT; ++t) {
#pragma unroll
            for (int i = 0; i < KS; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
            m[t][0] = m[t][1] = SOFTMAX_FLOOR;
            l[t][0] = l[t][1] = 0.f;
        }
    }
    // the block of keys key0 .. whose K and V tiles stand at kt and vt; sc: scale log2 e
    __device__ __forceinline__ void block(uint32_t kt, uint32_t vt, int key0, const SeqBlocks& x, float sc) {
        const int lane = threadIdx.x & 31, g4 = lane >> 2;
        const int mi = lane >> 3, r8 = lane & 7;
        float s[NSUB][HT][4];            // S^T: keys g4 and g4 + 8 of each 16
#pragma unroll
        for (int u = 0; u < NSUB; ++u)
#pragma unroll
            for (int t = 0; t < HT; ++t) s[u][t][0] = s[u][t][1] = s[u][t][2] = s[u][t][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int u = 0; u < NSUB; ++u) {
                uint32_t ka[4];
                ldsm4(kt + q_off<DP>(16 * u + (mi & 1) * 8 + r8, 2 * kk + (mi >> 1)), ka[0], ka[1], ka[2], ka[3]);
#pragma unroll
                for (int t = 0; t < HT; ++t) E::mma(s[u][t], ka, qb[t][kk][0], qb[t][kk][1]);
            }
        // every key of the block visible: below the end, and all in the window or all among the sinks
        const bool whole = key0 + KEYS <= x.end && (key0 >= x.first || key0 + KEYS <= x.sinks);
        bool up = false;
#pragma unroll
        for (int u = 0; u < NSUB; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bool in = true;
                if (!whole) {
                    const int key = key0 + 16 * u + g4 + 8 * (i >> 1);
                    in = key < x.end && (key >= x.first || key < x.sinks);
                }
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    s[u][t][i] = in ? s[u][t][i] * sc : -INFINITY;
                    up |= s[u][t][i] > m[t][i & 1] + (8.f + E::LIFT);
                }
            }
        if (__any_sync(FULL_MASK, up)) {
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = -INFINITY;
#pragma unroll
                    for (int u = 0; u < NSUB; ++u) x = fmaxf(x, fmaxf(s[u][t][e], s[u][t][e + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, d));
                    x = fmaxf(m[t][e], x - E::LIFT);
                    const float f = ex2(m[t][e] - x);
                    m[t][e] = x;
                    l[t][e] *= f;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[t][i][e] *= f;
                        o[t][i][e + 2] *= f;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < NSUB; ++u) {
            uint32_t pb[HT][2], pr[HT][2];   // P^T as B fragments: keys 2 q4, + 1 (and + 8) of head g4
#pragma unroll
            for (int t = 0; t < HT; ++t) {
                float (&p)[4] = s[u][t];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = ex2(p[i] - m[t][i & 1]);
                l[t][0] += p[0] + p[2];
                l[t][1] += p[1] + p[3];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x = E::pack(p[2 * e], p[2 * e + 1]);
                    pb[t][e] = transpose8x8(x);
                    // what the rounding left
                    pr[t][e] = transpose8x8(E::pack(p[2 * e] - E::lo(x), p[2 * e + 1] - E::hi(x)));
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                uint32_t va[4];
                ldsm4t(vt + q_off<DP>(16 * u + (mi >> 1) * 8 + r8, 2 * i + (mi & 1)), va[0], va[1], va[2], va[3]);
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    E::mma(o[t][i], va, pb[t][0], pb[t][1]);
                    E::mma(o[t][i], va, pr[t][0], pr[t][1]);
                }
            }
        }
    }
    // l of the heads, over all the lanes' keys
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(FULL_MASK, l[t][e], d);
    }
};

}  // namespace

}  // namespace ember
