// paged_prefill.cu -- attention of several new tokens per sequence over a
// paged K/V cache: the query rows cu[b] .. cu[b + 1] of sequence b are its last
// positions, each sees the keys at or before it (or a window of them and a few
// first tokens), out = softmax(scale Q K^T) V and lse = log sum exp.
//
// This kernel serves short sequences, and what the tcgen05 kernel
// (paged_prefill_tc.cu) does not take: a scale that is not positive.  The G query
// heads of a kv head share its keys, so a tile's rows are (token, head) pairs: row
// r = token r / G, head r % G.  One CTA holds 64 rows of one kv head, 16 to a
// warp, and walks the keys in tiles of 64 that cp.async copies (zero fill for keys
// no row sees) stage two deep in shared memory.  Bound by latency: 4 sequences
// of 9 new tokens, 14 heads on 2, in 4.3 us.
//
// The weights go into the second product as the sum of two values of the cache's type
// (bf16 2^-16 relative, f16 2^-22), as in decode: with one the output's error would be
// 1.35 times its own rounding's.  The second product of f16 costs 10 % (64 sequences of
// 20 tokens on 100 keys, 16 heads on 8 of 128, 20.7 -> 22.3 us, as bf16).
#include "paged.cuh"

namespace ember {

namespace {

constexpr int PP_THREADS = 128;
constexpr int PP_ROWS = 64;
constexpr int PP_KEYS = 64;
constexpr int PP_SMALL_KEYS = 128;   // keys that the table holds for a sequence
constexpr int PP_SMALL_ROWS = 64;    // new tokens of a sequence, on average

template <int DP>
struct PpSmem {
    static constexpr int TILE = PP_KEYS * DP * 2;
    static constexpr int TOTAL = 4 * TILE;      // two stages of K and V
};

template <class E, int DP>
__global__ void __launch_bounds__(PP_THREADS) k_paged_prefill(PagedPrefillArgs a) {
    constexpr int KS = DP / 16, NT = DP / 8, C8 = DP / 8;
    using L = PpSmem<DP>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;
    const int D = a.c.D, NKV = a.c.NKV, G = a.NH / NKV, g = blockIdx.y;
    const int QT = PP_ROWS / G;
    pdl_wait();
    pdl_trigger();

    const RowTile tile = find_row_tile(a, QT, (int)blockIdx.x, blockIdx.x == 0 && g == 0 && warp == 0);
    const int b = tile.b;
    if (b < 0) return;
    const SeqRows sr = seq_rows(a, b, false);
    const int i0 = tile.i * QT;                       // first token of the tile
    const int tokens = min(QT, sr.nq - i0);
    const int pos0 = sr.len - sr.nq + i0;                // its position (negative: sees nothing)
    const int pos1 = pos0 + tokens - 1;

    // rows g4 and g4 + 8 of the warp
    int pos[2], tok[2], head[2];
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + g4 + 8 * h;
        tok[h] = r / G;
        head[h] = r - tok[h] * G;
        live[h] = tok[h] < tokens;
        pos[h] = live[h] ? pos0 + tok[h] : -1;
    }
    uint32_t qa[KS][4];
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int h = e & 1, col = 16 * kk + (e >> 1) * 8 + 2 * q4;
            const uint16_t* q = a.q + (long long)(sr.row0 + i0 + tok[h]) * a.ld_q + (long long)(g * G + head[h]) * D;
            qa[kk][e] = live[h] && col < D ? *reinterpret_cast<const uint32_t*>(q + col) : 0u;
        }

    // ---- key tiles that some row sees: those of the sinks, then the window's ----
    const int end = pos1 + 1;                            // keys at or beyond it are hidden from all
    const int first = a.window > 0 ? max(0, pos0 + 1 - a.window) : 0;
    const int sinks = min(a.sinks, first);
    const int ns = (sinks + PP_KEYS - 1) / PP_KEYS;
    const int wb = max(first / PP_KEYS, ns);
    const int nt_all = end <= 0 ? 0 : ns + max(0, (end + PP_KEYS - 1) / PP_KEYS - wb);
    auto key0_of = [&](int t) { return PP_KEYS * (t < ns ? t : wb + t - ns); };
    auto issue = [&](int t) {
        if (t < nt_all) {
            const uint32_t kd = sa_u32(sm) + (uint32_t)(t & 1) * 2 * L::TILE, vd = kd + L::TILE;
            const int key0 = key0_of(t);
            for (int e = tid; e < PP_KEYS * C8; e += PP_THREADS) {
                const int r = e / C8, c = e % C8, key = key0 + r;
                bool in = key < end && (key >= first || key < sinks) && c * 8 < D;
                long long off = 0;
                if (in) {
                    const int page = a.c.table[(size_t)sr.seq * a.c.width + (key >> a.c.page_shift)];
                    if (page < 0 || page >= a.c.n_pages) {
                        in = false;                      // a bad page reads as zeros
                        raise_status(a.status, EMBER_ERR_INVALID_ARG);
                    } else {
                        off = (long long)page * a.c.page_stride + (long long)g * a.c.head_stride +
                              (long long)(key & ((1 << a.c.page_shift) - 1)) * a.c.row_stride + c * 8;
                    }
                }
                cp_async16(kd + q_off<DP>(r, c), a.c.k + off, in);
                cp_async16(vd + q_off<DP>(r, c), a.c.v + off, in);
            }
        }
        cp_async_commit();
    };

    const float sc = a.scale * LOG2E;
    float o[NT][4];
#pragma unroll
    for (int dn = 0; dn < NT; ++dn) o[dn][0] = o[dn][1] = o[dn][2] = o[dn][3] = 0.f;
    float m[2] = {SOFTMAX_FLOOR, SOFTMAX_FLOOR}, l[2] = {0.f, 0.f};
    issue(0);
    for (int t = 0; t < nt_all; ++t) {
        issue(t + 1);
        cp_async_wait<1>();
        __syncthreads();
        const uint32_t kt = sa_u32(sm) + (uint32_t)(t & 1) * 2 * L::TILE, vt = kt + L::TILE;
        const int mi = lane >> 3;
        const int key0 = key0_of(t);
        float s[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int nt = 0; nt < 8; nt += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm4(kt + q_off<DP>(nt * 8 + (mi >> 1) * 8 + (lane & 7), 2 * kk + (mi & 1)), b0, b1, b2, b3);
                E::mma(s[nt], qa[kk], b0, b1);
                E::mma(s[nt + 1], qa[kk], b2, b3);
            }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = i >> 1, key = key0 + nt * 8 + 2 * q4 + (i & 1);
                const bool in = key <= pos[h] && (a.window <= 0 || key > pos[h] - a.window || key < a.sinks);
                s[nt][i] = in ? s[nt][i] * sc : -INFINITY;
                mx[h] = fmaxf(mx[h], s[nt][i]);
            }
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(FULL_MASK, mx[h], 1));
            mx[h] = fmaxf(m[h], fmaxf(mx[h], __shfl_xor_sync(FULL_MASK, mx[h], 2)) - E::LIFT);
            f[h] = ex2(m[h] - mx[h]);
            m[h] = mx[h];
            l[h] *= f[h];
        }
#pragma unroll
        for (int dn = 0; dn < NT; ++dn)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[dn][i] *= f[i >> 1];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nt][i] = ex2(s[nt][i] - m[i >> 1]);
                l[i >> 1] += s[nt][i];
            }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {                 // 16 keys each
            uint32_t pa[4], pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = s[2 * ks + (i >> 1)][2 * (i & 1)], y = s[2 * ks + (i >> 1)][2 * (i & 1) + 1];
                pa[i] = E::pack(x, y);
                pr[i] = E::pack(x - E::lo(pa[i]), y - E::hi(pa[i]));   // what the rounding left
            }
#pragma unroll
            for (int dn = 0; dn < NT; dn += 2) {
                uint32_t r0, r1, r2, r3;
                ldsm4t(vt + q_off<DP>(ks * 16 + (mi & 1) * 8 + (lane & 7), dn + (mi >> 1)), r0, r1, r2, r3);
                E::mma(o[dn], pa, r0, r1);
                E::mma(o[dn + 1], pa, r2, r3);
                E::mma(o[dn], pr, r0, r1);
                E::mma(o[dn + 1], pr, r2, r3);
            }
        }
        __syncthreads();                                 // the stage is read
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(FULL_MASK, l[h], 1);
        l[h] += __shfl_xor_sync(FULL_MASK, l[h], 2);
        if (!live[h]) continue;
        const long long row = sr.row0 + i0 + tok[h];
        const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
        uint16_t* out = a.out + row * a.ld_out + (long long)(g * G + head[h]) * D;
#pragma unroll
        for (int dn = 0; dn < NT; ++dn) {
            const int col = dn * 8 + 2 * q4;
            if (col < D) *reinterpret_cast<uint32_t*>(out + col) = E::pack(o[dn][2 * h] * inv, o[dn][2 * h + 1] * inv);
        }
        if (a.lse && q4 == 0)
            a.lse[row * a.NH + g * G + head[h]] = l[h] == 0.f ? -INFINITY : m[h] * LN2 + logf(l[h]);
    }
}

template <class E, int DP>
cudaError_t launch_dp(const PagedPrefillArgs& a, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(k_paged_prefill<E, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PpSmem<DP>::TOTAL);
    if (e != cudaSuccess) return e;
    const int qt = PP_ROWS / (a.NH / a.c.NKV);
    const dim3 grid((unsigned)(((long long)a.n + qt - 1) / qt + a.B), a.c.NKV);
    return launch_k(k_paged_prefill<E, DP>, grid, dim3(PP_THREADS), PpSmem<DP>::TOTAL, s, a);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedPrefillArgs& a, int sms, cudaStream_t s) {
    // Short sequences only, where filling the tcgen05 kernel's pipeline costs more than
    // the whole attention.  14 heads on 2 of 64, here and there: 20 new tokens each of 256
    // sequences 18.5 and 27.7 us, 4 sequences of 9 tokens 4.3 and 5.5, 60 of 64 sequences
    // 10.1 and 11.4, but 100 of 64 sequences 14.0 and 13.7; 32 on 8: 20 of 256 sequences
    // 68 and 91, 60 of 64 27.7 and 24.5, 100 of 64 55 and 38.  With keys for more than two
    // of its tiles the other kernel wins at any size: 2 tokens on 200 keys 9.4 and 7.1 us,
    // of 64 sequences on 1000 keys 33 and 15 us.
    const bool small = ((long long)a.c.width << a.c.page_shift) <= PP_SMALL_KEYS && a.n <= PP_SMALL_ROWS * (long long)a.B;
    PagedPrefillMaps maps;
    // (the tcgen05 kernel takes the largest product for the largest score: scale > 0)
    if (!small && a.scale > 0.f && paged_prefill_maps(a, maps)) return launch_paged_prefill_tc(a, maps, sms, s);
    if (a.c.bf16) return a.c.D <= 64 ? launch_dp<ElemBf16, 64>(a, s) : launch_dp<ElemBf16, 128>(a, s);
    return a.c.D <= 64 ? launch_dp<ElemF16, 64>(a, s) : launch_dp<ElemF16, 128>(a, s);
}

}  // namespace ember
