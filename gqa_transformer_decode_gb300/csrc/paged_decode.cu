// paged_decode.cu -- attention of one new token per sequence over a paged K/V
// cache: out = sum_j softmax_j(scale q . k_j) v_j over the keys that the
// sequence's last position sees (all of them, or a window and a few first
// tokens), and optionally lse = log sum_j exp(scale q . k_j).
//
// Bound: the bytes of the visible K and V rows, each read once for the G query
// heads that share a kv head.  So the heads of a group are the rows of one
// 16-row matrix product (rows >= G are zero) and a warp takes 16 keys at a
// time: S = Q K^T, one pass with the running maximum and sum of each row, and
// O += P V, all in registers (mma.m16n8k16, f32 accumulators).
//
// Work split: the visible keys of every (sequence, kv head) form a list of
// 16-key blocks, the lists of all sequences stand one behind the other, and
// CTA c takes the c-th equal share of that whole line, so a ragged batch and
// one long sequence both keep every SM busy to the end.  A CTA's warps take
// its blocks in turn; each warp streams its own blocks through a ring of
// cp.async copies that runs on across sequence boundaries.  A (sequence, kv
// head) whose blocks lie in one CTA is finished there; otherwise its CTAs leave
// (m, l, O) partials that a second small kernel joins in CTA order, so the
// result depends on the lengths and the device only.
//
// Blocks start at multiples of 16 keys and pages hold a multiple of 16 rows,
// so a block lies in one page.  Rows that the query does not see are filled
// with zeros by the copy itself, never read: whatever a page holds beyond a
// sequence's end, NaN among it, has no effect, and table entries of pages
// without a visible key are not looked at.
//
// P is the second product's operand.  For f16 it is rounded to f16 (2^-12
// relative).  bf16 would cost 2^-9, as much as the output's own rounding, so
// there P goes in as the sum of two bf16 values: the products are far from
// bounding this kernel.
#include "paged.cuh"

namespace ember {

namespace {

constexpr int PD_WARPS = 4;
constexpr int PD_THREADS = PD_WARPS * 32;
constexpr int PD_KEYS = 16;          // keys of a block
constexpr int PD_STAGES = 3;         // ring stages of a warp
constexpr int PD_MIN_BLOCKS = 8;     // blocks of a CTA at least (two per warp)
constexpr int PD_CTAS_PER_SM = 2;

// Blocks of one sequence: [0, ns) hold its sinks, the rest its window.
struct SeqBlocks {
    int n, ns, wb;       // blocks, blocks of the sinks, first block of the window
    int end, first, sinks;
    bool zero;           // nothing visible: the output is zero
    __device__ __forceinline__ int key0(int i) const { return PD_KEYS * (i < ns ? i : wb + i - ns); }
};

__device__ __forceinline__ SeqBlocks seq_blocks(const PagedDecodeArgs& a, int b, bool report) {
    SeqBlocks r;
    r.n = 0;
    r.ns = r.wb = r.end = r.first = r.sinks = 0;
    r.zero = false;
    const int seq = a.seqs ? a.seqs[b] : b;
    if (seq < 0) return r;                                   // padding: the row is left as it is
    if (seq >= a.c.n_seqs) {
        if (report) raise_status(a.status, EMBER_ERR_INVALID_ARG);
        return r;
    }
    const int len = a.lens[b];
    if (len < 0 || len > ((long long)a.c.width << a.c.page_shift)) {
        if (report) raise_status(a.status, EMBER_ERR_CAPACITY);
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
    r.ns = (v.sinks + PD_KEYS - 1) / PD_KEYS;
    r.wb = max(v.first / PD_KEYS, r.ns);
    r.n = r.ns + (v.end + PD_KEYS - 1) / PD_KEYS - r.wb;
    return r;
}

// Sum over the block's threads and exclusive prefix (s holds PD_WARPS + 1 ints).
__device__ __forceinline__ int block_scan(int v, int* s, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < PD_WARPS; ++w) {
        if (w < warp) base += s[w];
        total += s[w];
    }
    return base + incl - v;
}

// Blocks of the whole line divided over `ctas` CTAs: CTA c takes [lo(c), lo(c + 1)).
struct Shares {
    long long total;     // blocks of all (sequence, kv head)s
    int ctas;            // CTAs that take part
    __device__ __forceinline__ Shares(long long t, int grid) {
        total = t;
        const long long most = (t + PD_MIN_BLOCKS - 1) / PD_MIN_BLOCKS;
        ctas = (int)min((long long)grid, max(1ll, most));
    }
    __device__ __forceinline__ long long lo(int c) const { return total * c / ctas; }
    // the CTA whose share holds block x
    __device__ __forceinline__ int holder(long long x) const {
        return (int)(((x + 1) * ctas - 1) / total);
    }
};

// A place in the line: block `i` of kv head g of sequence b.
struct Place {
    int b, g, i;
    SeqBlocks s;
};

template <int DP>
struct PdSmem {
    static constexpr int TILE = PD_KEYS * DP * 2;                // one K (or V) block
    static constexpr int RING = PD_WARPS * PD_STAGES * 2 * TILE;
    static constexpr int SCR = 16 * DP * 4;                       // the merge's O rows
    static constexpr int TOTAL = RING + SCR;
};

template <class E, int DP>
__global__ void __launch_bounds__(PD_THREADS, PD_CTAS_PER_SM) k_paged_decode(PagedDecodeArgs a) {
    constexpr int KS = DP / 16, NT = DP / 8, C8 = DP / 8;
    using L = PdSmem<DP>;
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ int s_scan[PD_WARPS];
    __shared__ int s_find[4];
    __shared__ float s_m[PD_WARPS][16], s_l[PD_WARPS][16];
    float* s_o = reinterpret_cast<float*>(sm + L::RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV;
    pdl_wait();
    pdl_trigger();   // after the wait: the join kernel may then read the caller's lengths at once

    // ---- the whole line's length, and this CTA's first place in it ----
    long long line = 0;
    for (int b0 = 0; b0 < a.B; b0 += PD_THREADS) {
        const int b = b0 + tid;
        int n = 0, total;
        if (b < a.B) n = seq_blocks(a, b, blockIdx.x == 0).n;
        block_scan(n, s_scan, total);
        line += total;
    }
    line *= NKV;
    // rows of sequences without keys
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (seq_blocks(a, b, false).zero) {
            uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (long long)b * a.ld_out);
            for (int e = tid; e < a.NH * D / 2; e += PD_THREADS) o[e] = 0u;
            if (a.lse)
                for (int e = tid; e < a.NH; e += PD_THREADS) a.lse[(long long)b * a.NH + e] = -INFINITY;
        }
    if (line == 0) return;
    const Shares share(line, gridDim.x);
    if ((int)blockIdx.x >= share.ctas) return;
    const long long lo = share.lo(blockIdx.x), hi = share.lo(blockIdx.x + 1);
    {
        long long run = 0;
        for (int b0 = 0; b0 < a.B; b0 += PD_THREADS) {
            const int b = b0 + tid;
            int n = 0, total;
            if (b < a.B) n = seq_blocks(a, b, false).n;
            const long long at = run + (long long)block_scan(n, s_scan, total) * NKV;
            if (n > 0 && at <= lo && lo < at + (long long)n * NKV) {
                s_find[0] = b;
                s_find[1] = (int)((lo - at) / n);
                s_find[2] = (int)((lo - at) % n);
            }
            run += (long long)total * NKV;
        }
        __syncthreads();
    }
    Place cur;
    cur.b = s_find[0];
    cur.g = s_find[1];
    cur.i = s_find[2];
    cur.s = seq_blocks(a, cur.b, false);

    auto advance = [&](Place& p, int by) {   // to the block `by` further on (inside the line)
        p.i += by;
        while (p.i >= p.s.n) {
            p.i -= p.s.n;
            if (++p.g == NKV) {
                p.g = 0;
                do p.s = seq_blocks(a, ++p.b, false);
                while (p.s.n == 0 && p.b + 1 < a.B);
            }
        }
    };

    // ---- copies: warp w takes blocks lo + w, lo + w + PD_WARPS, ... ----
    const int mine = (int)max(0ll, (hi - lo - warp + PD_WARPS - 1) / PD_WARPS);
    uint8_t* ring = sm + warp * (PD_STAGES * 2 * L::TILE);
    const uint32_t ring_u = sa_u32(ring);
    Place ld = cur;
    int ld_page = 0;
    auto page_of = [&](const Place& p) {
        const int seq = a.seqs ? a.seqs[p.b] : p.b;
        return a.c.table[(size_t)seq * a.c.width + (p.s.key0(p.i) >> a.c.page_shift)];
    };
    if (mine > 0) {
        advance(ld, warp);
        ld_page = page_of(ld);
    }
    auto issue = [&](int j) {                // the warp's j-th block -> stage j % PD_STAGES
        if (j < mine) {
            const uint32_t kd = ring_u + (uint32_t)(j % PD_STAGES) * 2 * L::TILE, vd = kd + L::TILE;
            const int key0 = ld.s.key0(ld.i);
            const bool ok = ld_page >= 0 && ld_page < a.c.n_pages;   // a bad page reads as zeros
            if (!ok && lane == 0) raise_status(a.status, EMBER_ERR_INVALID_ARG);
            const long long base = ok ? (long long)ld_page * a.c.page_stride + (long long)ld.g * a.c.head_stride +
                                            (long long)(key0 & ((1 << a.c.page_shift) - 1)) * a.c.row_stride
                                      : 0;
            const int c = lane % C8;
#pragma unroll
            for (int r = lane / C8; r < PD_KEYS; r += 32 / C8) {
                const int key = key0 + r;
                const bool in = ok && c * 8 < D && key < ld.s.end && (key >= ld.s.first || key < ld.s.sinks);
                const long long off = in ? base + (long long)r * a.c.row_stride + c * 8 : 0;
                cp_async16(kd + q_off<DP>(r, c), a.c.k + off, in);
                cp_async16(vd + q_off<DP>(r, c), a.c.v + off, in);
            }
            if (j + 1 < mine) {
                advance(ld, PD_WARPS);
                ld_page = page_of(ld);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < PD_STAGES - 1; ++j) issue(j);

    // ---- segments: the CTA's blocks of one (sequence, kv head) after another ----
    const float sc = a.scale * LOG2E;
    int j = 0;                               // the warp's next block
    long long at = lo;                       // the line's block at the segment's start
    while (at < hi) {
        const int seg = (int)min((long long)(cur.s.n - cur.i), hi - at);   // its blocks in this CTA
        // q of the group's heads as A fragments (rows >= G zero)
        uint32_t qa[KS][4];
        const uint16_t* q = a.q + (long long)cur.b * a.ld_q + (long long)cur.g * G * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = g4 + (e & 1) * 8, col = 16 * kk + (e >> 1) * 8 + 2 * q4;
                qa[kk][e] = row < G && col < D ? *reinterpret_cast<const uint32_t*>(q + row * D + col) : 0u;
            }
        float o[NT][4];
#pragma unroll
        for (int dn = 0; dn < NT; ++dn) o[dn][0] = o[dn][1] = o[dn][2] = o[dn][3] = 0.f;
        float m0 = SOFTMAX_FLOOR, m1 = SOFTMAX_FLOOR, l0 = 0.f, l1 = 0.f;   // rows g4, g4 + 8
        const long long seg_end = at + seg;
        for (; lo + warp + (long long)j * PD_WARPS < seg_end; ++j) {
            const int blk = cur.i + (int)(lo + warp + (long long)j * PD_WARPS - at);
            issue(j + PD_STAGES - 1);
            cp_async_wait<PD_STAGES - 1>();
            __syncwarp();
            const uint32_t kt = ring_u + (uint32_t)(j % PD_STAGES) * 2 * L::TILE, vt = kt + L::TILE;
            const int key0 = cur.s.key0(blk);
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            const int mi = lane >> 3;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                uint32_t b0, b1, b2, b3;
                ldsm4(kt + q_off<DP>((mi >> 1) * 8 + (lane & 7), 2 * kk + (mi & 1)), b0, b1, b2, b3);
                E::mma(s[0], qa[kk], b0, b1);
                E::mma(s[1], qa[kk], b2, b3);
            }
            float mx0 = m0, mx1 = m1;
            // every key of the block visible: below the end, and all in the window or all among the sinks
            const bool whole = key0 + PD_KEYS <= cur.s.end && (key0 >= cur.s.first || key0 + PD_KEYS <= cur.s.sinks);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nt][i] *= sc;
                    if (!whole) {
                        const int key = key0 + nt * 8 + 2 * q4 + (i & 1);
                        if (key >= cur.s.end || (key < cur.s.first && key >= cur.s.sinks)) s[nt][i] = -INFINITY;
                    }
                    if (i < 2) mx0 = fmaxf(mx0, s[nt][i]);
                    else mx1 = fmaxf(mx1, s[nt][i]);
                }
            mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, 2));
            const float sc0 = ex2(m0 - mx0), sc1 = ex2(m1 - mx1);
            float p[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[nt][i] = ex2(s[nt][i] - (i < 2 ? mx0 : mx1));
            l0 = l0 * sc0 + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
            l1 = l1 * sc1 + ((p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
            m0 = mx0;
            m1 = mx1;
#pragma unroll
            for (int dn = 0; dn < NT; ++dn) {
                o[dn][0] *= sc0; o[dn][1] *= sc0;
                o[dn][2] *= sc1; o[dn][3] *= sc1;
            }
            const uint32_t pa[4] = {E::pack(p[0][0], p[0][1]), E::pack(p[0][2], p[0][3]), E::pack(p[1][0], p[1][1]),
                                    E::pack(p[1][2], p[1][3])};
            uint32_t pr[4];
            if (E::bf16) {                   // what the first rounding left
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pr[i] = E::pack(p[i >> 1][2 * (i & 1)] - E::lo(pa[i]), p[i >> 1][2 * (i & 1) + 1] - E::hi(pa[i]));
            }
#pragma unroll
            for (int dn = 0; dn < NT; dn += 2) {
                uint32_t r0, r1, r2, r3;
                ldsm4t(vt + q_off<DP>((mi & 1) * 8 + (lane & 7), dn + (mi >> 1)), r0, r1, r2, r3);
                E::mma(o[dn], pa, r0, r1);
                E::mma(o[dn + 1], pa, r2, r3);
                if (E::bf16) {
                    E::mma(o[dn], pr, r0, r1);
                    E::mma(o[dn + 1], pr, r2, r3);
                }
            }
            __syncwarp();                    // the stage is read: the next copy may fill it
        }

        // ---- merge the warps' states, in warp order ----
        l0 += __shfl_xor_sync(FULL_MASK, l0, 1);
        l0 += __shfl_xor_sync(FULL_MASK, l0, 2);
        l1 += __shfl_xor_sync(FULL_MASK, l1, 1);
        l1 += __shfl_xor_sync(FULL_MASK, l1, 2);
        __syncthreads();                     // the previous segment's merge is read
        if (q4 == 0) {
            s_m[warp][g4] = m0;
            s_m[warp][g4 + 8] = m1;
            s_l[warp][g4] = l0;
            s_l[warp][g4 + 8] = l1;
        }
        __syncthreads();
        float M0 = SOFTMAX_FLOOR, M1 = SOFTMAX_FLOOR, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
            M0 = fmaxf(M0, s_m[v][g4]);
            M1 = fmaxf(M1, s_m[v][g4 + 8]);
        }
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
            L0 += s_l[v][g4] * ex2(s_m[v][g4] - M0);
            L1 += s_l[v][g4 + 8] * ex2(s_m[v][g4 + 8] - M1);
        }
        const float f0 = ex2(m0 - M0), f1 = ex2(m1 - M1);
        for (int v = 0; v < PD_WARPS; ++v) {
            if (warp == v) {
#pragma unroll
                for (int dn = 0; dn < NT; ++dn)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = g4 + 8 * h;
                        if (row < G) {
                            float2* d = reinterpret_cast<float2*>(s_o + row * DP + dn * 8 + 2 * q4);
                            float2 x = v ? *d : make_float2(0.f, 0.f);
                            x.x = fmaf(o[dn][2 * h], h ? f1 : f0, x.x);
                            x.y = fmaf(o[dn][2 * h + 1], h ? f1 : f0, x.y);
                            *d = x;
                        }
                    }
            }
            __syncthreads();
        }
        const bool complete = seg == cur.s.n;
        if (warp == 0 && q4 == 0) {          // the rows' m and l of the whole segment
            s_m[0][g4] = M0;
            s_m[0][g4 + 8] = M1;
            s_l[0][g4] = L0;
            s_l[0][g4 + 8] = L1;
        }
        __syncthreads();
        if (complete) {
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (long long)cur.b * a.ld_out + (long long)cur.g * G * D);
            for (int e = tid; e < G * D / 2; e += PD_THREADS) {
                const int row = e / (D / 2), d = 2 * (e - row * (D / 2));
                const float l = s_l[0][row];
                const float inv = l == 0.f ? 0.f : 1.f / l;
                out[e] = E::pack(s_o[row * DP + d] * inv, s_o[row * DP + d + 1] * inv);
            }
            if (a.lse && tid < G)
                a.lse[(long long)cur.b * a.NH + cur.g * G + tid] =
                    s_l[0][tid] == 0.f ? -INFINITY : s_m[0][tid] * LN2 + logf(s_l[0][tid]);
        } else {
            // slot 0: the segment reaches back to the CTA's first block, slot 1: it begins inside
            float* ws = a.ws + (size_t)(2 * blockIdx.x + (at == lo ? 0 : 1)) * G * (D + 2);
            for (int e = tid; e < G * (D + 2); e += PD_THREADS) {
                const int row = e / (D + 2), d = e - row * (D + 2);
                ws[e] = d == 0 ? s_m[0][row] : d == 1 ? s_l[0][row] : s_o[row * DP + d - 2];
            }
        }
        at = seg_end;
        if (at < hi) advance(cur, seg);      // on to the next (sequence, kv head)
    }
    cp_async_wait<0>();
}

// Joins the partials of each (sequence, kv head) that several CTAs share:
// block (g, b), in CTA order.
template <class E>
__global__ void __launch_bounds__(PD_THREADS) k_paged_join(PagedDecodeArgs a, int grid) {
    __shared__ int s_scan[PD_WARPS];
    __shared__ float s_M[16], s_L[16];
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV;
    // The first kernel triggers after its own wait, so what the caller passed
    // is complete here; its partials are after pdl_wait.
    long long before = 0, line = 0;
    for (int b0 = 0; b0 < a.B; b0 += PD_THREADS) {
        const int x = b0 + tid;
        const int n = x < a.B ? seq_blocks(a, x, false).n : 0;
        int total, upto;
        block_scan(x < b ? n : 0, s_scan, upto);
        block_scan(n, s_scan, total);
        before += upto;
        line += total;
    }
    pdl_wait();                              // on every path: what follows in the stream waits for this kernel only
    pdl_trigger();
    const int n = seq_blocks(a, b, false).n;
    if (n == 0) return;
    const Shares share(line * NKV, grid);
    const long long s0 = before * NKV + (long long)g * n, s1 = s0 + n;
    const int c0 = share.holder(s0), c1 = share.holder(s1 - 1);
    if (c0 == c1) return;                    // finished by that CTA
    auto slot = [&](int c) {
        return a.ws + (size_t)(2 * c + (s0 <= share.lo(c) ? 0 : 1)) * G * (D + 2);
    };
    if (tid < G) {
        float M = SOFTMAX_FLOOR, L = 0.f;
        for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(slot(c) + tid * (D + 2)));
        for (int c = c0; c <= c1; ++c) {
            const float* p = slot(c) + tid * (D + 2);
            L += __ldcg(p + 1) * ex2(__ldcg(p) - M);
        }
        s_M[tid] = M;
        s_L[tid] = L;
    }
    __syncthreads();
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (long long)b * a.ld_out + (long long)g * G * D);
    for (int e = tid; e < G * D / 2; e += PD_THREADS) {
        const int row = e / (D / 2), d = 2 * (e - row * (D / 2));
        float x = 0.f, y = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float* p = slot(c) + row * (D + 2);
            const float f = ex2(__ldcg(p) - s_M[row]);
            x = fmaf(__ldcg(p + 2 + d), f, x);
            y = fmaf(__ldcg(p + 3 + d), f, y);
        }
        const float inv = s_L[row] == 0.f ? 0.f : 1.f / s_L[row];
        out[e] = E::pack(x * inv, y * inv);
    }
    if (a.lse && tid < G)
        a.lse[(long long)b * a.NH + g * G + tid] = s_L[tid] == 0.f ? -INFINITY : s_M[tid] * LN2 + logf(s_L[tid]);
}

template <class E, int DP>
cudaError_t launch_dp(const PagedDecodeArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(k_paged_decode<E, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PdSmem<DP>::TOTAL);
    if (e != cudaSuccess) return e;
    const int grid = sms * PD_CTAS_PER_SM;
    const cudaError_t r = launch_k(k_paged_decode<E, DP>, dim3(grid), dim3(PD_THREADS), PdSmem<DP>::TOTAL, s, a);
    if (r != cudaSuccess) return r;
    return launch_k(k_paged_join<E>, dim3(a.c.NKV, a.B), dim3(PD_THREADS), 0, s, a, grid);
}

}  // namespace

size_t paged_decode_ws(int NKV, int G, int D, int sms) {
    (void)NKV;
    return (size_t)sms * PD_CTAS_PER_SM * 2 * G * (D + 2) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int sms, cudaStream_t s) {
    if (a.c.bf16) return a.c.D <= 64 ? launch_dp<ElemBf16, 64>(a, sms, s) : launch_dp<ElemBf16, 128>(a, sms, s);
    return a.c.D <= 64 ? launch_dp<ElemF16, 64>(a, sms, s) : launch_dp<ElemF16, 128>(a, sms, s);
}

}  // namespace ember
