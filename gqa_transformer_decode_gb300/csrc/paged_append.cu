// paged_append.cu -- new tokens into a paged K/V cache: per-head RMSNorm of q
// and k (optional), rotate-half RoPE, one rounding to the cache's type, and
// the store of the K and V rows into their sequences' pages.
//
// For each head row x of D values and the token's position p:
//   y_i = x_i * rsqrt(mean(x^2) + eps) * w_i          (q and k, when normed)
//   z_i = y_i c_i - y_{i+D/2} s_i,  z_{i+D/2} = y_{i+D/2} c_i + y_i s_i
// with c, s the f32 tables' row p; V rows are only rounded.  Everything is f32
// until the one rounding at the store.  The rotation rounds each product and
// sum separately (rope_pair), so K rows appended from the same f32 values
// equal ember_rope_store's bit for bit.
//
// A thread owns eight pairs (i, i + D/2) of a head: two 16-byte pieces of the
// stored row (and two or four loads of 16 bytes), so the rotation needs no
// exchange and the norm's sum of squares is a shuffle over the head's D/16
// lanes.  A block takes whole tokens (threadIdx.y; x runs over the token's heads).
// Its first rows are asked for before the position and the page number, which only
// the rotation and the stores need, and each next item's before this one is
// worked on.  Few tokens: a thread for each item, since the time is the loads'
// latency.  Once the items fill the chip, 64 threads a token go through its heads
// in turn and keep its cos / sin in registers (9725 normed bf16 tokens of 16 + 8 +
// 8 heads of 128: 29 us against 45 with a thread for each item, which runs out of
// issue slots; 4096 f32 tokens of 32 + 8 + 8 heads of 64, outputs in L2: 11.6 against
// 12.3 us).
//
// Bound: bytes; each input is read once and each output written once.  The
// 4096-token prompt takes 14.2 us where all of them pass HBM (5.4 TB/s, 80 % of a
// copy's rate), 11.6 where the outputs stay in L2; the normed one 29.9 us, 5.4 TB/s,
// bound by its instructions.
#include "paged.cuh"

namespace ember {

namespace {

constexpr int AP_THREADS = 256, AP_FEW_THREADS = 64;
constexpr int AP_MANY = 152 * 2048;   // items: threads of a full chip

__device__ __forceinline__ void load8_f32(const float* p, float* f) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// Eight source elements as they come, and widened (each is read once: evict first).
struct SrcF32 {
    struct Raw { float4 a, b; };
    __device__ __forceinline__ static Raw load(const void* base, long long off) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
        return {__ldcs(p), __ldcs(p + 1)};
    }
    __device__ __forceinline__ static void widen(const Raw& r, float* f) {
        f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
        f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
    }
};
struct SrcBf16 {
    using Raw = uint4;
    __device__ __forceinline__ static Raw load(const void* base, long long off) {
        return __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off));
    }
    __device__ __forceinline__ static void widen(const Raw& r, float* f) { unpack8(r, f); }
};
struct SrcF16 {
    using Raw = uint4;
    __device__ __forceinline__ static Raw load(const void* base, long long off) { return SrcBf16::load(base, off); }
    __device__ __forceinline__ static void widen(const Raw& r, float* f) { unpack8_f16(r, f); }
};

template <class E>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(E::pack(f[0], f[1]), E::pack(f[2], f[3]), E::pack(f[4], f[5]), E::pack(f[6], f[7]));
}

template <class S, class E, int D>
__global__ void __launch_bounds__(AP_THREADS, 4) k_paged_append(PagedAppendArgs a) {
    constexpr int H2 = D / 2, TPH = D / 16;                  // threads of a head
    const int NKV = a.c.NKV, nq = a.q ? a.NH : 0;
    const int per_tok = (nq + 2 * NKV) * TPH;
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    pdl_wait();
    if (t >= a.n) return;
    // item r: eight pairs of one head of q, then k, then v
    auto place = [&](int r, int& kind, int& g) {
        const int head = r / TPH;
        kind = head < nq ? 0 : head < nq + NKV ? 1 : 2;
        g = kind == 0 ? head : kind == 1 ? head - nq : head - nq - NKV;
    };
    const int i0 = (threadIdx.x % TPH) * 8;                  // elements i0.. and H2 + i0.. of every head
    auto fetch = [&](int r, typename S::Raw& x, typename S::Raw& y) {
        int kind, g;
        place(r, kind, g);
        const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const long long off = (long long)t * (kind == 0 ? a.ld_q : kind == 1 ? a.ld_k : a.ld_v) + g * D + i0;
        x = S::load(src, off);
        y = S::load(src, off + H2);
    };
    int r = threadIdx.x;
    typename S::Raw x, y;
    fetch(r, x, y);
    const int seq = a.seqs[t], pos = a.positions[t];
    if (seq < 0) return;                                     // padding
    int err = 0, page = 0;
    if (seq >= a.c.n_seqs) err = EMBER_ERR_INVALID_ARG;
    else if (pos < 0 || (pos >> a.c.page_shift) >= a.c.width || pos >= a.n_pos) err = EMBER_ERR_CAPACITY;
    float c[8], s[8];
    if (!err) {
        page = a.c.table[(size_t)seq * a.c.width + (pos >> a.c.page_shift)];
        load8_f32(a.cos_t + (long long)pos * H2 + i0, c);
        load8_f32(a.sin_t + (long long)pos * H2 + i0, s);
        if (page < 0 || page >= a.c.n_pages) err = EMBER_ERR_INVALID_ARG;
    }
    if (err) {                                               // the whole token is skipped
        if (r == 0) raise_status(a.status, err);
        return;
    }
    const long long at = (long long)page * a.c.page_stride + (long long)(pos & ((1 << a.c.page_shift) - 1)) * a.c.row_stride + i0;
    uint16_t* q_row = a.q_out + (long long)t * a.ld_out + i0;
    while (true) {
        float v[8], w[8];
        S::widen(x, v);
        S::widen(y, w);
        int kind, g;
        place(r, kind, g);
        r += blockDim.x;
        if (r < per_tok) fetch(r, x, y);                     // the next item's, while this one is worked on
        if (kind < 2) {
            const uint16_t* nw = kind == 0 ? a.q_norm : a.k_norm;
            if (nw) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += v[e] * v[e] + w[e] * w[e];
                const unsigned lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
                const unsigned group = ((1u << TPH) - 1u) << (lane & ~(unsigned)(TPH - 1));
#pragma unroll
                for (int o = TPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                const float ri = rsqrtf(ss * (1.f / D) + a.eps);
                float n[8];
                unpack8(*reinterpret_cast<const uint4*>(nw + i0), n);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * ri * n[e];
                unpack8(*reinterpret_cast<const uint4*>(nw + H2 + i0), n);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = w[e] * ri * n[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float r0, r1;
                rope_pair(v[e], w[e], c[e], s[e], r0, r1);
                v[e] = r0;
                w[e] = r1;
            }
        }
        uint16_t* dst = kind == 0 ? q_row + g * D : (kind == 1 ? a.c.k : a.c.v) + at + (long long)g * a.c.head_stride;
        *reinterpret_cast<uint4*>(dst) = pack8<E>(v);
        *reinterpret_cast<uint4*>(dst + H2) = pack8<E>(w);
        if (r >= per_tok) break;
    }
    pdl_trigger();
}

template <class S, int D>
cudaError_t launch_d(const PagedAppendArgs& a, cudaStream_t s) {
    const int per_tok = ((a.q ? a.NH : 0) + 2 * a.c.NKV) * (D / 16);
    // a token's heads in turn once the tokens fill the chip, else all of them at once
    const int threads = (long long)a.n * per_tok >= AP_MANY ? AP_FEW_THREADS : AP_THREADS;
    const int x = per_tok < threads ? per_tok : threads, y = threads / x;
    const dim3 grid((unsigned)(((long long)a.n + y - 1) / y)), block(x, y);
    return a.c.bf16 ? launch_k(k_paged_append<S, ElemBf16, D>, grid, block, 0, s, a)
                    : launch_k(k_paged_append<S, ElemF16, D>, grid, block, 0, s, a);
}
template <class S>
cudaError_t launch_src(const PagedAppendArgs& a, cudaStream_t s) {
    if (a.c.D <= 32) return a.c.D == 16 ? launch_d<S, 16>(a, s) : launch_d<S, 32>(a, s);
    return a.c.D == 64 ? launch_d<S, 64>(a, s) : launch_d<S, 128>(a, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    if (a.src == 0) return launch_src<SrcF32>(a, s);
    return a.src == 1 ? launch_src<SrcBf16>(a, s) : launch_src<SrcF16>(a, s);
}

}  // namespace ember
