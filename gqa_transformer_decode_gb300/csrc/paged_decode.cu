// paged_decode.cu -- attention of one new token per sequence over a paged K/V
// cache: out = sum_j softmax_j(scale q . k_j) v_j over the keys that the
// sequence's last position sees (all of them, or a window and a few first
// tokens), and optionally lse = log sum_j exp(scale q . k_j).
//
// Bound: the bytes of the visible K and V rows, each read once for the G query
// heads that share a kv head.  So the heads of a group are the 8 (or 2 x 8)
// columns of the products and 16 keys, or 16 dimensions, their rows: S^T = K Q^T,
// one pass with a running maximum and sum per head, O^T += V^T P^T, all in
// registers (mma.m16n8k16, f32 accumulators; P^T becomes an operand by
// movmatrix).  With the heads as the 16 rows half the work was on rows that most
// groups lack.  The maximum that scores are taken against moves (and O, l are
// rescaled) only when a score passes it by more than 2^8, so that most blocks
// need one vote instead of a reduction over the lanes.
//
// Work split, two ways:
//   line     the visible keys of every (sequence, kv head) form a list of blocks,
//            the lists of all sequences stand one behind the other, and CTA c
//            takes the c-th equal share of that whole line, so a ragged batch
//            and one long sequence both keep every SM busy to the end.  A CTA's
//            warps take its blocks in turn; each warp streams its own blocks
//            through a ring of cp.async copies that runs on across sequence
//            boundaries.  A (sequence, kv head) whose blocks lie in one CTA is
//            finished there; otherwise its CTAs leave (m, l, O) partials that a
//            second small kernel joins in CTA order.
//   cluster  for short sequences (few ones: longer): the CTAs of one thread-block
//            cluster share one (sequence, kv head) and join through distributed shared
//            memory, with no scan of the lengths, no workspace and no second kernel.
// Either way the result depends on the inputs, the form and the device only.
//
// Blocks start at multiples of 16 keys and pages hold a multiple of 16 rows,
// so a block lies in one page.  Rows that the query does not see are filled
// with zeros by the copy itself, never read: whatever a page holds beyond a
// sequence's end, NaN among it, has no effect, and table entries of pages
// without a visible key are not looked at.
//
// Measured: 64 sequences of 64 to 4096 keys, 32 heads on 8 of 64 (269 MB of K and V
// rows), 55 us, 4.9 TB/s; one of 131071 keys, 32 on 8 of 128, f16 (537 MB), 89 us, 6.0
// TB/s (a copy moves 6.7).  Of the 55 us the first data arrive 5 us after the start
// (lengths, page numbers and rows are three loads that depend on one another), the
// CTAs end between 34 and 48 us, and the join with its launch takes 5.
//
// P, the second product's operand, goes in as the sum of two values of the cache's
// type (bf16 2^-16 relative, f16 2^-22 or 2^-32 of the largest): one would add as much error as the output's
// own rounding, and the products are far from bounding this kernel.
#include "paged_decode.cuh"

namespace ember {

namespace {

constexpr int PD_MIN_BLOCKS = 8;     // blocks of a CTA at least (two per warp)
constexpr int PD_MAX_CLUSTER = 8;     // CTAs of a cluster (a power of two)
constexpr int PD_CLUSTER_BLOCKS = 8;  // blocks of a warp in cluster form at most
constexpr int PJ_PARTS = 8;           // partials of a (sequence, kv head) from which a block joins a single head
constexpr int PD_MAX_CTAS = 512;     // grid at most (the join's weights stand in shared memory)

// Blocks of the whole line divided over `ctas` CTAs: CTA c takes [lo(c), lo(c + 1)).
// (The launcher keeps the line below 2^30 blocks.)
struct Shares {
    unsigned total, ctas, each;
    __device__ __forceinline__ Shares(unsigned t, unsigned grid) {
        total = t;
        const unsigned most = (t + PD_MIN_BLOCKS - 1) / PD_MIN_BLOCKS;
        each = (t + min(grid, most) - 1) / min(grid, most);
        ctas = (t + each - 1) / each;
    }
    __device__ __forceinline__ unsigned lo(unsigned c) const { return min(total, c * each); }
};

// The workspace: a record for each CTA of the grid, then two partials for each.
__device__ __forceinline__ float* partials(const PagedDecodeArgs& a, int grid) { return a.ws + 4 * (size_t)grid; }

// HT: tiles of 8 query heads (1 up to G = 8, else 2)
template <class E, int DP, int HT, bool CLUSTER, int SHARE>
__global__ void __launch_bounds__(PD_THREADS, pd_ctas_per_sm(HT)) k_paged_decode(PagedDecodeArgs a) {
    constexpr int KEYS = PD_KEYS<DP>, NSUB = KEYS / 16;
    constexpr int KS = DP / 16, C8 = DP / 8;
    using L = PdSmem<DP, HT>;
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ float s_m[PD_WARPS][8 * HT], s_l[PD_WARPS][8 * HT], s_M[8 * HT], s_L[8 * HT];
    float* s_o = reinterpret_cast<float*>(sm + L::RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV;
    pdl_wait();

    auto zero_row = [&](int b, int h0, int h1) {       // heads [h0, h1) of a sequence without keys
        uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (long long)b * a.ld_out);
        for (int e = h0 * D / 2 + tid; e < h1 * D / 2; e += PD_THREADS) o[e] = 0u;
        if (a.lse)
            for (int e = h0 + tid; e < h1; e += PD_THREADS) a.lse[(long long)b * a.NH + e] = -INFINITY;
    };

    // What the join finds: a record of each (sequence, kv head) or, where these are
    // more than the CTAs, of each CTA's last one: {b, g, partials (0: nothing to
    // join), first CTA * 2 + its slot}.
    int4* record = reinterpret_cast<int4*>(a.ws);
    auto no_keys = [&]() {                             // sequences without blocks, shared out over the CTAs
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            const SeqBlocks s = seq_blocks<KEYS, SHARE>(a, b, false);
            if (s.zero) zero_row(b, 0, a.NH);
            if (a.by_pair && s.n == 0)
                for (int g = tid; g < NKV; g += PD_THREADS) record[b * NKV + g] = make_int4(0, 0, 0, 0);
        }
    };

    // ---- this CTA's blocks [lo, hi) and the first one's place ----
    unsigned lo, hi;
    Place cur;
    if (CLUSTER) {
        cur.b = blockIdx.z;
        cur.g = blockIdx.y;
        cur.s = seq_blocks<KEYS, SHARE>(a, cur.b, blockIdx.x == 0 && cur.g == 0 && tid == 0);
        if (cur.s.n == 0) {                            // so for the whole cluster
            if (cur.s.zero && blockIdx.x == 0) zero_row(cur.b, cur.g * G, (cur.g + 1) * G);
            return;
        }
        // a block for each warp at least; CTAs left over join in with nothing, so that a
        // smaller cluster (a table with room for fewer blocks) gives the same bits
        const unsigned each = max(PD_WARPS, (cur.s.n + a.split - 1) / a.split);
        lo = min((unsigned)cur.s.n, blockIdx.x * each);
        hi = min((unsigned)cur.s.n, lo + each);
        cur.i = (int)lo;
    } else {
        int n[PD_SCAN];
        unsigned line = 0, before = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32 * PD_SCAN) line += scan_chunk<KEYS, SHARE>(a, b0, blockIdx.x == 0 && warp == 0, n, before);
        line *= NKV;
        const Shares share(max(1u, line), gridDim.x);
        if (line == 0 || blockIdx.x >= share.ctas) {
            pdl_trigger();
            if (!a.by_pair && tid == 0) record[blockIdx.x] = make_int4(0, 0, 0, 0);
            no_keys();
            return;
        }
        lo = share.lo(blockIdx.x);
        hi = share.lo(blockIdx.x + 1);
        unsigned run = 0;
        for (int b0 = 0;; b0 += 32 * PD_SCAN) {
            // one chunk: its counts are still in the registers
            const unsigned total = a.B <= 32 * PD_SCAN ? line / NKV : scan_chunk<KEYS, SHARE>(a, b0, false, n, before);
            if (lo < run + total * NKV) {
                unsigned at = run + before * NKV;
                int b = -1;
                unsigned first = 0;
#pragma unroll
                for (int e = 0; e < PD_SCAN; ++e) {
                    if (lo >= at && lo < at + (unsigned)n[e] * NKV) {
                        b = b0 + PD_SCAN * lane + e;
                        first = at;
                    }
                    at += (unsigned)n[e] * NKV;
                }
                const int src = __ffs(__ballot_sync(FULL_MASK, b >= 0)) - 1;
                cur.b = __shfl_sync(FULL_MASK, b, src);
                cur.s = seq_blocks<KEYS, SHARE>(a, cur.b, false);
                const unsigned x = lo - __shfl_sync(FULL_MASK, first, src);
                cur.g = (int)(x / (unsigned)cur.s.n);
                cur.i = (int)(x - (unsigned)cur.g * (unsigned)cur.s.n);
                break;
            }
            run += total * NKV;
        }
    }

    auto advance = [&](Place& p, int by) {   // to the block `by` further on (inside the line)
        p.i += by;
        while (p.i >= p.s.n) {
            p.i -= p.s.n;
            if (++p.g == NKV) {
                p.g = 0;
                do p.s = seq_blocks<KEYS, SHARE>(a, ++p.b, false);
                while (p.s.n == 0 && p.b + 1 < a.B);
            }
        }
    };

    // ---- copies: warp w takes blocks lo + w, lo + w + PD_WARPS, ... ----
    const int mine = ((int)(hi - lo) - warp + PD_WARPS - 1) / PD_WARPS;
    uint8_t* ring = sm + warp * (PD_STAGES * 2 * L::TILE);
    const uint32_t ring_u = sa_u32(ring);
    Place ld = cur;
    int ld_page[NSUB];                       // pages of its 16-key parts, looked up one block ahead
    int ld_before[NSUB];                     // PD_SHARED: those of the part's keys below `from`
    auto look_up = [&]() {
        const int seq = a.seqs ? a.seqs[ld.b] : ld.b;
        const int key0 = KEYS * ld.s.index(ld.i);
#pragma unroll
        for (int u = 0; u < NSUB; ++u) {
            const int k0 = key0 + 16 * u;    // a part that nobody sees has no page
            const bool any = k0 < ld.s.end && (k0 + 16 > ld.s.first || k0 < ld.s.sinks);
            const bool own = SHARE == PD_OWN || (k0 + 16 > ld.s.from && ld.s.end > ld.s.from);
            ld_page[u] = any && own ? a.c.table[(size_t)seq * a.c.width + (k0 >> a.c.page_shift)] : 0;
            if (SHARE == PD_SHARED)
                ld_before[u] = any && k0 < ld.s.from ? a.c.table[(size_t)ld.s.prefix * a.c.width + (k0 >> a.c.page_shift)] : 0;
        }
    };
    if (mine > 0) {
        advance(ld, warp);
        look_up();
    }
    auto issue = [&](int j) {                // the warp's j-th block -> stage j % PD_STAGES
        if (j < mine) {
            const uint32_t kd = ring_u + (uint32_t)(j % PD_STAGES) * 2 * L::TILE, vd = kd + L::TILE;
            const int key0 = KEYS * ld.s.index(ld.i);
            const int c = lane % C8;
#pragma unroll
            for (int u = 0; u < NSUB; ++u) {
                const int k0 = key0 + 16 * u;
                const bool ok = ld_page[u] >= 0 && ld_page[u] < a.c.n_pages;   // a bad page reads as zeros
                if (!ok && lane == 0) raise_status(a.status, EMBER_ERR_INVALID_ARG);
                const long long in_page =
                    (long long)ld.g * a.c.head_stride + (long long)(k0 & ((1 << a.c.page_shift) - 1)) * a.c.row_stride + c * 8;
                const long long base = ok ? (long long)ld_page[u] * a.c.page_stride + in_page : 0;
                bool ok_before = true;
                long long before = 0;
                if (SHARE == PD_SHARED) {
                    ok_before = ld_before[u] >= 0 && ld_before[u] < a.c.n_pages;
                    if (!ok_before && lane == 0) raise_status(a.status, EMBER_ERR_INVALID_ARG);
                    before = ok_before ? (long long)ld_before[u] * a.c.page_stride + in_page : 0;
                }
#pragma unroll
                for (int i = 0; i < 16 * C8 / 32; ++i) {
                    const int r = lane / C8 + i * (32 / C8);
                    const int key = k0 + r;
                    const bool shared = SHARE == PD_SHARED && key < ld.s.from;
                    const bool in =
                        (shared ? ok_before : ok) && c * 8 < D && key < ld.s.end && (key >= ld.s.first || key < ld.s.sinks);
                    const long long off = in ? (shared ? before : base) + (long long)r * a.c.row_stride : 0;
                    cp_async16(kd + q_off<DP>(16 * u + r, c), a.c.k + off, in);
                    cp_async16(vd + q_off<DP>(16 * u + r, c), a.c.v + off, in);
                }
            }
            if (j + 1 < mine) {
                advance(ld, PD_WARPS);
                look_up();
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < PD_STAGES - 1; ++j) issue(j);

    // ---- segments: the CTA's blocks of one (sequence, kv head) after another ----
    const float sc = a.scale * LOG2E;
    int j = 0;                               // the warp's next block
    unsigned at = lo;                        // the line's block at the segment's start
    do {
        const int seg = min(cur.s.n - cur.i, (int)(hi - at));   // its blocks in this CTA (0: a cluster's CTA without work)
        PdState<E, DP, HT> st;
        st.begin(a.q + (long long)cur.b * a.ld_q + (long long)cur.g * G * D, G, D);
        auto &o = st.o;
        auto &m = st.m, &l = st.l;
        const unsigned seg_end = at + seg;
        for (; lo + warp + j * PD_WARPS < seg_end; ++j) {
            const int blk = cur.i + (int)(lo + warp + j * PD_WARPS - at);
            issue(j + PD_STAGES - 1);
            cp_async_wait<PD_STAGES - 1>();
            __syncwarp();
            const uint32_t kt = ring_u + (uint32_t)(j % PD_STAGES) * 2 * L::TILE, vt = kt + L::TILE;
            const int key0 = KEYS * cur.s.index(blk);
            st.block(kt, vt, key0, cur.s, sc);
            __syncwarp();                    // the stage is read: the next copy may fill it
        }

        // ---- merge the warps' states: 2 and 3 into 0 and 1, then 1 into 0 ----
        st.end();
        __syncthreads();                     // the previous segment's output is written
        if (g4 == 0) {
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s_m[warp][8 * t + 2 * q4 + e] = m[t][e];
                    s_l[warp][8 * t + 2 * q4 + e] = l[t][e];
                }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * t + 2 * q4 + e;
                float M = s_m[0][h];
#pragma unroll
                for (int v = 1; v < PD_WARPS; ++v) M = fmaxf(M, s_m[v][h]);
                const float f = ex2(m[t][e] - M);
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[t][i][e] *= f;
                    o[t][i][e + 2] *= f;
                }
            }
        auto store_o = [&](int buf) {
            float* d = s_o + buf * 8 * HT * L::ROW;
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        d[(8 * t + 2 * q4 + (e & 1)) * L::ROW + 16 * i + g4 + 8 * (e >> 1)] = o[t][i][e];
        };
        auto add_o = [&](int buf) {
            const float* d = s_o + buf * 8 * HT * L::ROW;
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[t][i][e] += d[(8 * t + 2 * q4 + (e & 1)) * L::ROW + 16 * i + g4 + 8 * (e >> 1)];
        };
        if (warp >= 2) store_o(warp - 2);
        __syncthreads();
        if (warp < 2) add_o(warp);
        if (warp == 1) store_o(1);
        __syncthreads();
        if (warp == 0) {
            add_o(1);
            store_o(0);
        }
        if (warp == 1 && lane < 8 * HT) {    // the heads' m and l of the whole segment
            float M = s_m[0][lane], S = 0.f;
#pragma unroll
            for (int v = 1; v < PD_WARPS; ++v) M = fmaxf(M, s_m[v][lane]);
#pragma unroll
            for (int v = 0; v < PD_WARPS; ++v) S += s_l[v][lane] * ex2(s_m[v][lane] - M);
            s_M[lane] = M;
            s_L[lane] = S;
        }
        __syncthreads();
        if (CLUSTER) break;
        const bool complete = seg == cur.s.n;
        if (complete) {
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (long long)cur.b * a.ld_out + (long long)cur.g * G * D);
            for (int e = tid; e < G * D / 2; e += PD_THREADS) {
                const int row = e / (D / 2), d = 2 * (e - row * (D / 2));
                const float l = s_L[row];
                const float inv = l == 0.f ? 0.f : 1.f / l;
                out[e] = E::pack(s_o[row * L::ROW + d] * inv, s_o[row * L::ROW + d + 1] * inv);
            }
            if (a.lse && tid < G)
                a.lse[(long long)cur.b * a.NH + cur.g * G + tid] =
                    s_L[tid] == 0.f ? -INFINITY : s_M[tid] * LN2 + logf(s_L[tid]);
        } else {
            // slot 0: the segment reaches back to the CTA's first block, slot 1: it begins inside
            float* ws = partials(a, gridDim.x) + (size_t)(2 * blockIdx.x + (at == lo ? 0 : 1)) * G * (D + 2);
            for (int e = tid; e < G * (D + 2); e += PD_THREADS) {
                const int row = e / (D + 2), d = e - row * (D + 2);
                ws[e] = d == 0 ? s_M[row] : d == 1 ? s_L[row] : s_o[row * L::ROW + d - 2];
            }
        }
        // a segment that begins here and that later CTAs go on with is this CTA's last
        // (hi - lo is then every CTA's share)
        if (tid == 0 && (a.by_pair ? cur.i == 0 : seg_end == hi)) {
            const int parts =
                cur.i == 0 && !complete ? (int)((at + cur.s.n - 1) / (hi - lo)) - (int)blockIdx.x + 1 : 0;
            record[a.by_pair ? cur.b * NKV + cur.g : blockIdx.x] =
                make_int4(cur.b, cur.g, parts, 2 * blockIdx.x + (at == lo ? 0 : 1));
        }
        at = seg_end;
        if (at >= hi) break;
        advance(cur, seg);                   // on to the next (sequence, kv head)
    } while (true);
    cp_async_wait<0>();
    pdl_trigger();                           // late: the join's blocks would take issue slots meanwhile
    if (!CLUSTER) {
        no_keys();
        return;
    }

    // ---- cluster: every CTA joins a share of the group's output ----
    cluster_sync_all();
    const uint32_t um = sa_u32(s_M), ul = sa_u32(s_L), uo = sa_u32(s_o);
    const unsigned C = gridDim.x;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (long long)cur.b * a.ld_out + (long long)cur.g * G * D);
    for (int e = blockIdx.x * PD_THREADS + tid; e < G * D / 2; e += C * PD_THREADS) {
        const int row = e / (D / 2), d = 2 * (e - row * (D / 2));
        float cm[PD_MAX_CLUSTER], cl[PD_MAX_CLUSTER], M = SOFTMAX_FLOOR, S = 0.f;
        float2 co[PD_MAX_CLUSTER], x = make_float2(0.f, 0.f);
#pragma unroll
        for (unsigned r = 0; r < PD_MAX_CLUSTER; ++r)
            if (r < C) {
                cm[r] = ld_cluster(um + 4 * row, r);
                cl[r] = ld_cluster(ul + 4 * row, r);
                co[r] = ld_cluster2(uo + 4 * (row * L::ROW + d), r);
            }
#pragma unroll
        for (unsigned r = 0; r < PD_MAX_CLUSTER; ++r)
            if (r < C) M = fmaxf(M, cm[r]);
#pragma unroll
        for (unsigned r = 0; r < PD_MAX_CLUSTER; ++r)
            if (r < C) {
                const float f = ex2(cm[r] - M);
                S = fmaf(cl[r], f, S);
                x.x = fmaf(co[r].x, f, x.x);
                x.y = fmaf(co[r].y, f, x.y);
            }
        const float inv = S == 0.f ? 0.f : 1.f / S;
        out[e] = E::pack(x.x * inv, x.y * inv);
        if (a.lse && d == 0)
            a.lse[(long long)cur.b * a.NH + cur.g * G + row] = S == 0.f ? -INFINITY : M * LN2 + logf(S);
    }
    cluster_sync_all();                      // no CTA leaves while another reads its shared memory
}

// Joins the partials of each (sequence, kv head) that several CTAs share, in
// CTA order.  Block (r, y) reads record r and joins heads [y * heads, (y + 1) *
// heads) of its group.  Threads take four dimensions each and the partials in
// turn; they ask for their first values together with the (m, l) of all partials,
// of which a warp for each head then finds the weights.
constexpr int PJ_WARPS = 8;
constexpr int PJ_THREADS = PJ_WARPS * 32;
constexpr int PJ_AHEAD = 4;

template <class E>
__global__ void __launch_bounds__(PJ_THREADS) k_paged_join(PagedDecodeArgs a, int grid, int heads) {
    __shared__ float s_w[16][PD_MAX_CTAS];                 // [head][partial]
    __shared__ float s_inv[16];
    __shared__ float4 s_o[PJ_THREADS];
    const int h0 = blockIdx.y * heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.c.D, G = a.NH / a.c.NKV;
    pdl_wait();
    pdl_trigger();
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(a.ws) + blockIdx.x);
    const int b = rec.x, g = rec.y, parts = rec.z, c0 = rec.w >> 1;
    // (what another call wrote into a workspace that two share by mistake is not followed out of the buffers)
    if (parts <= 0 || c0 < 0 || c0 >= grid || parts > grid - c0 || b < 0 || b >= a.B || g < 0 || g >= a.c.NKV) return;
    // partial i: slot 0 of its CTA, but slot 1 of the first when the segment begins inside it
    const float* base = partials(a, grid) + (size_t)h0 * (D + 2);
    const size_t slot = (size_t)G * (D + 2);
    auto part = [&](int h, int i) {
        return base + (2 * (size_t)(c0 + i) + (i == 0 ? rec.w & 1 : 0)) * slot + (size_t)h * (D + 2);
    };
    const int quads = heads * (D / 4);                      // four dimensions of a head each
    const int wide = min(quads, PJ_THREADS), turns = PJ_THREADS / wide;   // threads of a partial, partials at a time
    const int t0 = tid / wide;
    auto value = [&](int q, int i) {
        const int h = q / (D / 4), d = 4 * (q - h * (D / 4));
        const float2* p = reinterpret_cast<const float2*>(part(h, i) + 2 + d);
        const float2 u = __ldcg(p), v = __ldcg(p + 1);
        return make_float4(u.x, u.y, v.x, v.y);
    };
    float4 ahead[PJ_AHEAD];
#pragma unroll
    for (int k = 0; k < PJ_AHEAD; ++k)
        if (t0 < turns && t0 + k * turns < parts) ahead[k] = value(tid % wide, t0 + k * turns);
    for (int h = warp; h < heads; h += PJ_WARPS) {
        float M = SOFTMAX_FLOOR;
        float2 ml[2];                                       // the lane's first two partials
        for (int i = lane, k = 0; i < parts; i += 32, ++k) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(part(h, i)));
            if (k == 0) ml[0] = x;
            if (k == 1) ml[1] = x;
            M = fmaxf(M, x.x);
        }
        M = warp_max(M);
        float L = 0.f;
        for (int i = lane, k = 0; i < parts; i += 32, ++k) {
            const float2 x = k == 0 ? ml[0] : k == 1 ? ml[1] : __ldcg(reinterpret_cast<const float2*>(part(h, i)));
            const float f = ex2(x.x - M);
            s_w[h][i] = f;
            L += x.y * f;
        }
        L = warp_sum(L);
        if (lane == 0) {
            s_inv[h] = L == 0.f ? 0.f : 1.f / L;
            if (a.lse) a.lse[(long long)b * a.NH + g * G + h0 + h] = L == 0.f ? -INFINITY : M * LN2 + logf(L);
        }
    }
    __syncthreads();
    for (int q0 = 0; q0 < quads; q0 += PJ_THREADS) {
        const int q = q0 + tid % wide, h = q / (D / 4), d = 4 * (q - h * (D / 4));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4& x, int i) {
            const float f = s_w[h][i];
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
        };
        if (q < quads && t0 < turns) {
#pragma unroll
            for (int k = 0; k < PJ_AHEAD; ++k)
                if (t0 + k * turns < parts) add(q0 == 0 ? ahead[k] : value(q, t0 + k * turns), t0 + k * turns);
#pragma unroll 4
            for (int i = t0 + PJ_AHEAD * turns; i < parts; i += turns) add(value(q, i), i);
        }
        if (turns > 1) {
            s_o[tid] = o;
            __syncthreads();
            if (t0 == 0)
                for (int t = 1; t < turns; ++t) {
                    const float4 y = s_o[tid + t * wide];
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                }
        }
        if (q < quads && t0 == 0) {
            const float inv = s_inv[h];
            uint2* out = reinterpret_cast<uint2*>(a.out + (long long)b * a.ld_out + (long long)(g * G + h0 + h) * D + d);
            *out = make_uint2(E::pack(o.x * inv, o.y * inv), E::pack(o.z * inv, o.w * inv));
        }
    }
}

int pd_grid_full(int sms, int G) { return min(PD_MAX_CTAS, sms * pd_ctas_per_sm(G <= 8 ? 1 : 2)); }

// How a call is split: by the most blocks that its table and window allow.
struct PdPlan {
    int cluster, split;   // CTAs of a cluster (0: the line), and that share a long sequence
    int grid;             // the line's CTAs
};
PdPlan pd_plan(const PagedView& c, int B, int NH, int window, int sinks, int sms) {
    const int G = NH / c.NKV, KEYS = c.D <= 64 ? PD_KEYS<64> : PD_KEYS<128>;
    const long long keys = (long long)c.width << c.page_shift;
    // (a window's blocks: its own, one more at each end that it cuts, one that the sinks cut)
    const long long seen = window > 0 ? min(keys, (long long)window + sinks + 3 * KEYS) : keys;
    const long long blocks = (seen + KEYS - 1) / KEYS, pairs = (long long)B * c.NKV;
    // A cluster has no second kernel, but only its own CTAs: 14 heads on 2 of 64,
    // cluster and line, 4.5 and 8.6 us for 500 keys, 7.4 and 10.5 for 4000, 11.4 and
    // 10.8 for 8000, 19.2 and 11.6 for 16000.  With clusters on most of the chip the
    // line's even shares win earlier: 28 sequences of 2000 keys 12.1 and 13.8 us, of
    // 4000 keys 20.5 and 19.8, of 8000 keys 32.5 and 28.6.  Past a full chip a sequence
    // has one CTA, for as many blocks as in the full one: 400 sequences of 100 keys 11.7
    // and 13.5 us, 800 25.3 and 29.3, 1600 44.8 and 47.7, 900 of 480 keys 50.3 and 49.3;
    // 200 sequences of 250 keys on 8 kv heads 23.8 and 34.3.
    const int full = pd_grid_full(sms, G);
    int split = PD_MAX_CLUSTER;
    while (split > 1 && pairs * split > full) split /= 2;
    const int per_warp = pairs * split * 2 <= full ? PD_CLUSTER_BLOCKS : PD_CLUSTER_BLOCKS / 2;
    if (blocks <= split * PD_WARPS * per_warp) {
        int C = 1;
        while (C < split && C * PD_WARPS < blocks) C *= 2;
        return {C, split, 0};
    }
    return {0, 0, (int)min((long long)full, (blocks * pairs + PD_MIN_BLOCKS - 1) / PD_MIN_BLOCKS)};
}

template <class E, int DP, int HT, int SHARE>
cudaError_t launch_ht(PagedDecodeArgs a, int sms, cudaStream_t s) {
    constexpr int SMEM = PdSmem<DP, HT>::TOTAL;
    const PdPlan plan = pd_plan(a.c, a.B, a.NH, a.window, a.sinks, sms);
    a.split = plan.split;
    if (plan.cluster) {
        auto k = k_paged_decode<E, DP, HT, true, SHARE>;
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        return launch_cluster_k(k, dim3(plan.cluster, a.c.NKV, a.B), dim3(PD_THREADS), SMEM, plan.cluster, s, a);
    }
    auto k = k_paged_decode<E, DP, HT, false, SHARE>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    a.by_pair = (long long)a.B * a.c.NKV < plan.grid;
    const cudaError_t r = launch_k(k, dim3(plan.grid), dim3(PD_THREADS), SMEM, s, a);
    if (r != cudaSuccess || plan.grid == 1) return r;
    // A block joins a group's heads, since most records say that there is nothing to
    // do; but one head where few (sequence, kv head)s have many partials.
    const int G = a.NH / a.c.NKV, records = a.by_pair ? a.B * a.c.NKV : plan.grid - 1;
    const int heads = (long long)a.B * a.c.NKV * PJ_PARTS < plan.grid ? 1 : G;
    return launch_k(k_paged_join<E>, dim3(records, G / heads), dim3(PJ_THREADS), 0, s, a, plan.grid, heads);
}

template <class E, int DP>
cudaError_t launch_dp(const PagedDecodeArgs& a, int sms, cudaStream_t s) {
    if (a.groups) return a.NH / a.c.NKV <= 8 ? launch_ht<E, DP, 1, PD_SHARED>(a, sms, s) : launch_ht<E, DP, 2, PD_SHARED>(a, sms, s);
    return a.NH / a.c.NKV <= 8 ? launch_ht<E, DP, 1, PD_OWN>(a, sms, s) : launch_ht<E, DP, 2, PD_OWN>(a, sms, s);
}

}  // namespace

size_t paged_decode_ws(const PagedView& c, int B, int NH, int window, int sinks, int sms) {
    const PdPlan plan = pd_plan(c, B, NH, window, sinks, sms);
    return plan.cluster ? 0 : (size_t)plan.grid * (4 + 2 * (size_t)(NH / c.NKV) * (c.D + 2)) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int sms, cudaStream_t s) {
    if (a.c.bf16) return a.c.D <= 64 ? launch_dp<ElemBf16, 64>(a, sms, s) : launch_dp<ElemBf16, 128>(a, sms, s);
    return a.c.D <= 64 ? launch_dp<ElemF16, 64>(a, sms, s) : launch_dp<ElemF16, 128>(a, sms, s);
}

}  // namespace ember
