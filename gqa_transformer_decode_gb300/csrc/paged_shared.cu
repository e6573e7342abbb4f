// paged_shared.cu -- attention of one new token per sequence where groups of sequences share a
// long prefix: out = softmax over the prefix's keys and the row's own, each prefix read once for
// all rows of its group.
//
// Softmax over two sets of keys is joined from each set's maximum, sum and weighted values.  So
// three launches:
//   k_paged_prefill_tc<.., PT_SHARED>   the prefixes: the group's (row, head) pairs are the rows
//                    of matrix products on tcgen05, which is where the work is (4 D flops a key
//                    for each query head, against 4 D bytes a key and kv head)
//   k_shared_tail    the rows' own keys, as in paged_decode.cu, bound by their bytes
//   k_shared_join    the two
// The second needs nothing of the first: it starts as the first one's CTAs leave their SMs, some
// of them at once in small calls (paged_groups.cuh), and ends after it.  The third starts when the
// second is through.
//
// Tails are short and many (a few hundred keys for each of hundreds of rows and kv heads), so a
// warp, not a CTA, is what takes a share of the line of blocks: it works on its blocks alone and
// leaves what it has of a (row, kv head) as one partial, with no other warp to wait for, and the
// join adds up the few partials of each.  With shares for CTAs, whose warps merge their states
// once for each (row, kv head), 64 rows of one block each on 8 kv heads took as long as 64 of 256
// keys.
//
// Calls of little work, or of groups of one or two rows, read each row's keys once for each row
// instead (paged_decode.cu, PD_SHARED), which is one launch.
#include "paged_decode.cuh"
#include "paged_groups.cuh"

namespace ember {

namespace {

// The workspace of k_shared_tail: {first slot, partials} for each (row, kv head), then the
// partials, [G][D + 2] floats each: m, l, sums.  What warp w has of pair p lies in slot p + w,
// which no other has: along the line p and w only rise, one of them at each step.
__device__ __forceinline__ float* tail_partials(const PagedDecodeArgs& a) { return a.ws + ((2 * (size_t)a.B * a.c.NKV + 3) & ~(size_t)3); }

template <class E, int DP, int HT>
__global__ void __launch_bounds__(PD_THREADS, pd_ctas_per_sm(HT)) k_shared_tail(PagedDecodeArgs a) {
    constexpr int KEYS = PD_KEYS<DP>, NSUB = KEYS / 16, KS = DP / 16, C8 = DP / 8;
    using L = PdSmem<DP, HT>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV;
    const unsigned W = blockIdx.x * PD_WARPS + warp;
    int2* record = reinterpret_cast<int2*>(a.ws);

    // (no wait: this grid starts when all CTAs of the prefixes' are past theirs, and everything
    // before that one is then complete)
    int n[PD_SCAN];
    unsigned line = 0, before = 0;
    constexpr int CHUNK = 32 * PD_SCAN;
    // One chunk of rows each warp scans for itself; of more, the warps take turns and hand each
    // other the totals (1024 rows in 64 groups on 2 kv heads of 64: 35 us; all by itself 63).
    const bool one = a.B <= CHUNK;
    unsigned* totals = reinterpret_cast<unsigned*>(sm);
    static_assert(4 * (65536 / CHUNK) <= L::RING, "65535 rows");
    for (int c = one ? 0 : warp; c * CHUNK < a.B; c += PD_WARPS) {
        // one warp of the grid: errors, and rows without blocks
        const bool report = c % gridDim.x == blockIdx.x && (!one || warp == 0);
        const unsigned t = scan_chunk<KEYS, PD_TAIL>(a, c * CHUNK, report, n, before);
        if (one) line = t;
        else if (lane == 0) totals[c] = t;
        for (int e = 0; report && e < PD_SCAN; ++e) {
            const int b = c * CHUNK + PD_SCAN * lane + e;
            if (b < a.B && n[e] == 0)
                for (int g = 0; g < NKV; ++g) record[(size_t)b * NKV + g] = make_int2(0, 0);
        }
    }
    if (!one) {
        __syncthreads();
        for (int c = lane; c * CHUNK < a.B; c += 32) line += totals[c];
        line = __reduce_add_sync(FULL_MASK, line);
    }
    line *= NKV;
    // as many CTAs as have room on the SMs that the prefixes leave
    const PtGroups gs{a.groups, a.shared, a.prefixes, a.lens, a.n_groups, a.B, a.c.n_seqs, NKV, a.prefix_rows,
                      (long long)a.c.width << a.c.page_shift};
    unsigned pairs = 0, rows = 0, tiles = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
        unsigned row0, line0;
        (void)pt_scan(gs, g0, pairs, rows, tiles, row0, line0);
    }
    const int per_sm = pd_ctas_per_sm(HT), sms = (int)gridDim.x / per_sm;
    const int beside = prefix_sms(tiles, pairs, (float)line * (KEYS * DP * 4), sms);
    const unsigned NW = PD_WARPS * (unsigned)per_sm * (beside < sms ? sms - beside : sms);
    const unsigned each = max(1u, (line + NW - 1) / NW);
    const unsigned lo = min(line, W * each), hi = min(line, lo + each);
    int chunk = 0;                               // that the warp's share begins in
    unsigned run = 0;
    if (!one) {
        if (lo < hi)
            while (lo >= run + totals[chunk] * NKV) run += totals[chunk++] * NKV;
        __syncthreads();                         // the ring may be filled
    }
    if (lo < hi) {
        Place cur;
        if (!one)                                // (else its counts are still in the registers)
            (void)scan_chunk<KEYS, PD_TAIL>(a, chunk * CHUNK, false, n, before);
        {
            unsigned at = run + before * NKV, first = 0;
            int b = -1;
#pragma unroll
            for (int e = 0; e < PD_SCAN; ++e) {
                if (lo >= at && lo < at + (unsigned)n[e] * NKV) {
                    b = chunk * CHUNK + PD_SCAN * lane + e;
                    first = at;
                }
                at += (unsigned)n[e] * NKV;
            }
            const int src = __ffs(__ballot_sync(FULL_MASK, b >= 0)) - 1;
            cur.b = __shfl_sync(FULL_MASK, b, src);
            cur.s = seq_blocks<KEYS, PD_TAIL>(a, cur.b, false);
            const unsigned x = lo - __shfl_sync(FULL_MASK, first, src);
            cur.g = (int)(x / (unsigned)cur.s.n);
            cur.i = (int)(x - (unsigned)cur.g * (unsigned)cur.s.n);
        }
        auto next_pair = [&](Place& p) {         // (inside the line)
            p.i = 0;
            if (++p.g == NKV) {
                p.g = 0;
                do p.s = seq_blocks<KEYS, PD_TAIL>(a, ++p.b, false);
                while (p.s.n == 0 && p.b + 1 < a.B);
            }
        };

        // ---- copies, a block ahead ----
        const int mine = (int)(hi - lo);
        const uint32_t ring = sa_u32(sm + warp * (PD_STAGES * 2 * L::TILE));
        Place ld = cur;
        int page[NSUB];                          // of its 16-key parts, looked up one block ahead
        auto look_up = [&]() {
            const int seq = a.seqs ? a.seqs[ld.b] : ld.b;
#pragma unroll
            for (int u = 0; u < NSUB; ++u) {
                const int k0 = KEYS * ld.s.index(ld.i) + 16 * u;
                page[u] = k0 < ld.s.end && k0 + 16 > ld.s.first ? a.c.table[(size_t)seq * a.c.width + (k0 >> a.c.page_shift)] : 0;
            }
        };
        look_up();
        auto issue = [&](int j) {
            if (j < mine) {
                const uint32_t kd = ring + (uint32_t)(j % PD_STAGES) * 2 * L::TILE, vd = kd + L::TILE;
                const int key0 = KEYS * ld.s.index(ld.i), c = lane % C8;
#pragma unroll
                for (int u = 0; u < NSUB; ++u) {
                    const int k0 = key0 + 16 * u;
                    const bool ok = page[u] >= 0 && page[u] < a.c.n_pages;   // a bad page reads as zeros
                    if (!ok && lane == 0) raise_status(a.status, EMBER_ERR_INVALID_ARG);
                    const long long base =
                        ok ? (long long)page[u] * a.c.page_stride + (long long)ld.g * a.c.head_stride +
                                 (long long)(k0 & ((1 << a.c.page_shift) - 1)) * a.c.row_stride + c * 8
                           : 0;
#pragma unroll
                    for (int i = 0; i < 16 * C8 / 32; ++i) {
                        const int r = lane / C8 + i * (32 / C8), key = k0 + r;
                        const bool in = ok && c * 8 < D && key < ld.s.end && key >= ld.s.first;
                        const long long off = in ? base + (long long)r * a.c.row_stride : 0;
                        cp_async16(kd + q_off<DP>(16 * u + r, c), a.c.k + off, in);
                        cp_async16(vd + q_off<DP>(16 * u + r, c), a.c.v + off, in);
                    }
                }
                if (j + 1 < mine) {
                    if (++ld.i >= ld.s.n) next_pair(ld);
                    look_up();
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int j = 0; j < PD_STAGES - 1; ++j) issue(j);

        // ---- the warp's blocks of one (row, kv head) after another ----
        const float sc = a.scale * LOG2E;
        PdState<E, DP, HT> st;
        for (int j = 0; j < mine;) {
            const int seg = min(cur.s.n - cur.i, mine - j);
            st.begin(a.q + (long long)cur.b * a.ld_q + (long long)cur.g * G * D, G, D);
            for (int e = 0; e < seg; ++e, ++j) {
                issue(j + PD_STAGES - 1);
                cp_async_wait<PD_STAGES - 1>();
                __syncwarp();
                const uint32_t kt = ring + (uint32_t)(j % PD_STAGES) * 2 * L::TILE;
                st.block(kt, kt + L::TILE, KEYS * cur.s.index(cur.i + e), cur.s, sc);
                __syncwarp();                    // the stage is read: the next copy may fill it
            }
            st.end();
            const size_t pair = (size_t)cur.b * NKV + cur.g;
            float* out = tail_partials(a) + (pair + W) * G * (D + 2);
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = 8 * t + 2 * q4 + e;
                    if (h >= G) continue;
                    if (g4 == 0) *reinterpret_cast<float2*>(out + h * (D + 2)) = make_float2(st.m[t][e], st.l[t][e]);
#pragma unroll
                    for (int i = 0; i < KS; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (16 * i + 8 * r < D) out[h * (D + 2) + 2 + 16 * i + g4 + 8 * r] = st.o[t][i][e + 2 * r];
                }
            // the pair's first warp knows how many there are: all have the same share
            if (cur.i == 0 && lane == 0)
                record[pair] = make_int2((int)(pair + W), (int)((lo + j - seg + cur.s.n - 1) / each) - (int)W + 1);
            if (j < mine) next_pair(cur);
        }
        cp_async_wait<0>();
    }
    pdl_trigger();
    pdl_wait();                                  // this grid ends after the prefixes'
}

// Joins what the two have left of a row's kv head: block (kv head, row).  Threads take four
// dimensions each and the partials in turn.
constexpr int SJ_AHEAD = 4;                      // partials asked for at a time

template <class E, int SJ_THREADS>
__global__ void __launch_bounds__(SJ_THREADS) k_shared_join(PagedDecodeArgs a, int warps) {
    __shared__ float4 s_o[SJ_THREADS];
    __shared__ float2 s_ml[SJ_THREADS];
    const int tid = threadIdx.x;
    const int g = blockIdx.x, b = blockIdx.y;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV;
    // What the call got may be read before the wait (the kernels before began after it was complete).
    int row[1] = {b}, of[1];
    find_groups(a, row, of);
    const int group = of[0];
    const SeqBlocks s = seq_blocks<16, PD_TAIL>(a, b, a.seqs ? a.seqs[b] : b, a.lens[b], group, false);
    int pi = 0, at = 0;                          // the pair of row tiles among its group's, the row's slot
    if (s.zero && s.from > 0) {
        const int row0 = a.groups[group], nq = a.groups[group + 1] - row0, i = b - row0;
        pi = g * ((nq + a.prefix_rows - 1) / a.prefix_rows) + i / a.prefix_rows;
        at = g * nq + i;
    }
    pdl_wait();
    if (!s.zero) return;                         // the row is left as it is
    const size_t pair = (size_t)b * NKV + g;
    const int2* head = reinterpret_cast<const int2*>(a.prefix);
    const int2 line = __ldcg(head), first = __ldcg(head + 1 + group), rec = __ldcg(reinterpret_cast<const int2*>(a.ws) + pair);
    // (what another call wrote into a workspace that two share by mistake is not followed out of the buffers)
    int np = 0, slot0 = 0;                       // the prefix's partials: those of neighbouring CTAs
    if (s.from > 0) {
        const unsigned tiles = (unsigned)(s.from + 63) / 64, each = max(1, line.x), p0 = (unsigned)first.y + (unsigned)pi * tiles;
        np = (int)((p0 + tiles - 1) / each - p0 / each) + 1;
        const long long s0 = (long long)first.x + at + (long long)(p0 / each) * a.prefix_rows;
        if (s0 < 0 || np < 0 || s0 + (long long)(np - 1) * a.prefix_rows >= a.prefix_slots) np = 0;
        else slot0 = (int)s0;
    }
    int no = rec.y;                              // the row's own
    const int slots = a.B * NKV + warps;
    if (no < 0 || no > slots || rec.x < 0 || rec.x > slots - no) no = 0;
    const float* own = tail_partials(a) + (size_t)rec.x * G * (D + 2);
    const float* sums = a.prefix + a.prefix_head + (size_t)slot0 * G * D;
    const float2* ml = reinterpret_cast<const float2*>(a.prefix + a.prefix_head + (size_t)a.prefix_slots * G * D) + (size_t)slot0 * G;
    const size_t apart = (size_t)a.prefix_rows * G;   // from one CTA's partial to the next one's
    const int parts = np + no;
    // Each thread takes four dimensions of a head and every turns-th partial, four at a time, against
    // a maximum of its own; the threads of one place are joined at the end.
    const int quads = G * (D / 4), wide = min(quads, SJ_THREADS), turns = SJ_THREADS / wide, t0 = tid / wide;
    for (int q0 = 0; q0 < quads; q0 += wide) {
        const int q = q0 + tid % wide, h = q / (D / 4), d = 4 * (q - h * (D / 4));
        float M = SOFTMAX_FLOOR, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float f, const float4& x) {
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
        };
        auto move = [&](float to) {
            const float f = ex2(M - to);
            l *= f;
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            M = to;
        };
        if (q < quads && t0 < turns)
            for (int i0 = t0; i0 < parts; i0 += SJ_AHEAD * turns) {
                float2 s2[SJ_AHEAD];
                float4 x[SJ_AHEAD];
                float top = M;
#pragma unroll
                for (int k = 0; k < SJ_AHEAD; ++k) {
                    const int i = i0 + k * turns;
                    s2[k] = make_float2(SOFTMAX_FLOOR, 0.f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < np) {
                        s2[k] = __ldcg(ml + i * apart + h);
                        x[k] = __ldcg(reinterpret_cast<const float4*>(sums + (i * apart + h) * D + d));
                    } else if (i < parts) {
                        const float2* p = reinterpret_cast<const float2*>(own + ((size_t)(i - np) * G + h) * (D + 2));
                        const float2 u = __ldcg(p + 1 + d / 2), v = __ldcg(p + 2 + d / 2);
                        s2[k] = __ldcg(p);
                        x[k] = make_float4(u.x, u.y, v.x, v.y);
                    }
                }
#pragma unroll
                for (int k = 0; k < SJ_AHEAD; ++k) top = fmaxf(top, s2[k].x);
                if (top > M) move(top);
#pragma unroll
                for (int k = 0; k < SJ_AHEAD; ++k) {
                    const float f = ex2(s2[k].x - M);
                    l = fmaf(s2[k].y, f, l);
                    add(f, x[k]);
                }
            }
        if (turns > 1) {
            __syncthreads();
            s_o[tid] = o;
            s_ml[tid] = make_float2(M, l);
            __syncthreads();
            if (t0 == 0)
                for (int t = 1; t < turns; ++t) {
                    const float2 y = s_ml[tid + t * wide];
                    if (y.x > M) move(y.x);
                    const float f = ex2(y.x - M);
                    l = fmaf(y.y, f, l);
                    add(f, s_o[tid + t * wide]);
                }
        }
        if (q < quads && t0 == 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint2* out = reinterpret_cast<uint2*>(a.out + (long long)b * a.ld_out + (long long)(g * G + h) * D + d);
            *out = make_uint2(E::pack(o.x * inv, o.y * inv), E::pack(o.z * inv, o.w * inv));
            if (a.lse && d == 0) a.lse[(long long)b * a.NH + g * G + h] = l == 0.f ? -INFINITY : M * LN2 + logf(l);
        }
    }
}

// A call reads each row's keys once for each row (paged_decode.cu, PD_SHARED) up to so many bytes of
// keys and values: one group on 8 kv heads of 128 with 36 MB 15.9 us so and 19.3 apart, 52 MB 18.0
// and 19.3, 69 MB 19.5 and 20.0, 143 MB 26.9 and 20.5; and with fewer than three rows a group on
// average: 64 rows of 4096 shared and 200 own keys take 149 us so, apart 114 in groups of 2 and 86
// in groups of 3; but 1024 rows of 256 and 64 keys 246 so, apart 382 in groups of 2, 249 of 3 and
// 212 of 4.
constexpr double PD_TOGETHER = 72e6;
constexpr int PD_APART_ROWS = 3;

struct SharedPlan {
    bool apart;                                  // the prefixes by themselves
    int grid;                                    // k_shared_tail's
    size_t tail_floats;
    PagedSharedWs prefix;
};
SharedPlan shared_plan(const PagedView& c, int B, int NH, int n_groups, int sms) {
    SharedPlan p{};
    const int G = NH / c.NKV;
    const long long keys = (long long)c.width << c.page_shift;
    p.apart = (double)B * c.NKV * keys * c.D * 4 > PD_TOGETHER && n_groups <= B / PD_APART_ROWS;
    p.grid = sms * pd_ctas_per_sm(G <= 8 ? 1 : 2);
    p.tail_floats = ((2 * (size_t)B * c.NKV + 3) & ~(size_t)3) + ((size_t)B * c.NKV + (size_t)p.grid * PD_WARPS) * G * (c.D + 2);
    p.tail_floats = (p.tail_floats + 3) & ~(size_t)3;
    p.prefix = paged_shared_ws(B, n_groups, NH, c.NKV, c.D, sms);
    return p;
}

template <class E, int DP, int HT>
cudaError_t launch_ht(PagedDecodeArgs a, const PagedPrefillArgs& p, const PagedPrefillMaps& maps, const SharedPlan& plan, int sms,
                      cudaStream_t s) {
    constexpr int SMEM = PdSmem<DP, HT>::RING;
    cudaError_t e = launch_paged_shared(p, maps, sms, s);
    if (e != cudaSuccess) return e;
    auto k = k_shared_tail<E, DP, HT>;
    static OncePerDevice once;
    e = once([&] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e != cudaSuccess) return e;
    e = launch_k(k, dim3(plan.grid), dim3(PD_THREADS), SMEM, s, a);
    if (e != cudaSuccess) return e;
    // all blocks at once: 1024 of 256 threads take two rounds of 4 us
    const dim3 grid(a.c.NKV, a.B);
    if ((long long)a.c.NKV * a.B <= 4 * sms) return launch_k(k_shared_join<E, 256>, grid, dim3(256), 0, s, a, plan.grid * PD_WARPS);
    return launch_k(k_shared_join<E, 128>, grid, dim3(128), 0, s, a, plan.grid * PD_WARPS);
}
template <class E>
cudaError_t launch_type(const PagedDecodeArgs& a, const PagedPrefillArgs& p, const PagedPrefillMaps& m, const SharedPlan& plan,
                        int sms, cudaStream_t s) {
    if (a.NH / a.c.NKV <= 8) return a.c.D <= 64 ? launch_ht<E, 64, 1>(a, p, m, plan, sms, s) : launch_ht<E, 128, 1>(a, p, m, plan, sms, s);
    return a.c.D <= 64 ? launch_ht<E, 64, 2>(a, p, m, plan, sms, s) : launch_ht<E, 128, 2>(a, p, m, plan, sms, s);
}

}  // namespace

size_t paged_decode_shared_ws(const PagedView& c, int B, int NH, int n_groups, int sms) {
    const SharedPlan p = shared_plan(c, B, NH, n_groups, sms);
    const size_t together = paged_decode_ws(c, B, NH, 0, 0, sms);   // (also for scales that are not positive)
    return p.apart ? max(together, (p.tail_floats + p.prefix.floats) * sizeof(float)) : together;
}

cudaError_t launch_paged_decode_shared(PagedDecodeArgs a, int sms, cudaStream_t s) {
    const SharedPlan plan = shared_plan(a.c, a.B, a.NH, a.n_groups, sms);
    PagedPrefillArgs p{};
    p.c = a.c;
    p.q = a.q;
    p.ld_q = a.ld_q;
    p.n = a.B;
    p.B = a.n_groups;
    p.NH = a.NH;
    PagedPrefillMaps maps;
    // (the row threads of the prefixes' kernel take scores against a maximum of the products: scale > 0)
    if (!plan.apart || !(a.scale > 0.f) || !paged_prefill_maps(p, maps)) return launch_paged_decode(a, sms, s);
    p.seqs = a.prefixes;
    p.cu = a.groups;
    p.lens = a.lens;
    p.scale = a.scale;
    p.status = a.status;
    p.shared = a.shared;
    p.ws = a.ws + plan.tail_floats;
    p.ws_head = plan.prefix.head;
    p.slots = plan.prefix.slots;
    a.prefix = p.ws;
    a.prefix_head = plan.prefix.head;
    a.prefix_slots = plan.prefix.slots;
    a.prefix_rows = plan.prefix.rows_per_pair;
    return a.c.bf16 ? launch_type<ElemBf16>(a, p, maps, plan, sms, s) : launch_type<ElemF16>(a, p, maps, plan, sms, s);
}

}  // namespace ember
