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
// A thread owns eight pairs (i, i + D/2) of one head: two 16-byte pieces of
// the stored row (and two or four loads of 16 bytes), so the rotation needs no
// exchange and the norm's sum of squares is a shuffle over the head's D/16
// lanes.  A block takes whole tokens, so that the position, the table entry and
// the cos / sin row are read once per token into L1.
// Bound: bytes; each input is read once and each output written once.
#include "paged.cuh"

namespace ember {

namespace {

constexpr int AP_THREADS = 256;

struct SrcF32 {
    __device__ __forceinline__ static void load8(const void* base, long long off, float* f) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
        const float4 a = p[0], b = p[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
struct SrcBf16 {
    __device__ __forceinline__ static void load8(const void* base, long long off, float* f) {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off), f);
    }
};
struct SrcF16 {
    __device__ __forceinline__ static void load8(const void* base, long long off, float* f) {
        unpack8_f16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off), f);
    }
};

template <class E>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(E::pack(f[0], f[1]), E::pack(f[2], f[3]), E::pack(f[4], f[5]), E::pack(f[6], f[7]));
}

template <class S, class E>
__global__ void __launch_bounds__(AP_THREADS) k_paged_append(PagedAppendArgs a, int tokens_per_block) {
    const int D = a.c.D, H2 = D / 2;
    const int tph = D / 16;                                  // threads of a head
    const int nq = a.q ? a.NH : 0;
    const int per_tok = (nq + 2 * a.c.NKV) * tph;
    const int t0 = blockIdx.x * tokens_per_block;
    const int items = min(tokens_per_block, a.n - t0) * per_tok;
    const unsigned lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (int it = threadIdx.x; it < items; it += AP_THREADS) {
        const int tt = it / per_tok;
        const int r = it - tt * per_tok;
        const int head = r / tph, i0 = (r - head * tph) * 8;  // elements i0.. and H2 + i0..
        const int t = t0 + tt;
        const int seq = a.seqs[t], pos = a.positions[t];
        if (seq < 0) continue;                                // padding
        int err = 0;
        if (seq >= a.c.n_seqs) err = EMBER_ERR_INVALID_ARG;
        else if (pos < 0 || (pos >> a.c.page_shift) >= a.c.width || pos >= a.n_pos) err = EMBER_ERR_CAPACITY;
        int page = 0;
        if (!err) {
            page = a.c.table[(size_t)seq * a.c.width + (pos >> a.c.page_shift)];
            if (page < 0 || page >= a.c.n_pages) err = EMBER_ERR_INVALID_ARG;
        }
        if (err) {                                            // the whole token is skipped
            if (r == 0) raise_status(a.status, err);
            continue;
        }
        const int kind = head < nq ? 0 : head < nq + a.c.NKV ? 1 : 2;   // q, k, v
        const int g = kind == 0 ? head : kind == 1 ? head - nq : head - nq - a.c.NKV;
        const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const long long ld = kind == 0 ? a.ld_q : kind == 1 ? a.ld_k : a.ld_v;
        const long long off = (long long)t * ld + (long long)g * D + i0;
        float x[8], y[8];
        S::load8(src, off, x);
        S::load8(src, off + H2, y);
        if (kind < 2) {
            const uint16_t* nw = kind == 0 ? a.q_norm : a.k_norm;
            if (nw) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
                const unsigned group = ((1u << tph) - 1u) << (lane & ~(unsigned)(tph - 1));
                for (int o = tph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                const float ri = rsqrtf(ss / (float)D + a.eps);
                float w[8];
                unpack8(*reinterpret_cast<const uint4*>(nw + i0), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * ri * w[e];
                unpack8(*reinterpret_cast<const uint4*>(nw + H2 + i0), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = y[e] * ri * w[e];
            }
            float c[8], s[8];
            SrcF32::load8(a.cos_t, (long long)pos * H2 + i0, c);
            SrcF32::load8(a.sin_t, (long long)pos * H2 + i0, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float r0, r1;
                rope_pair(x[e], y[e], c[e], s[e], r0, r1);
                x[e] = r0;
                y[e] = r1;
            }
        }
        uint16_t* dst;
        if (kind == 0) {
            dst = a.q_out + (long long)t * a.ld_out + (long long)g * D;
        } else {
            const int row = pos & ((1 << a.c.page_shift) - 1);
            dst = (kind == 1 ? a.c.k : a.c.v) + (long long)page * a.c.page_stride + (long long)g * a.c.head_stride +
                  (long long)row * a.c.row_stride;
        }
        *reinterpret_cast<uint4*>(dst + i0) = pack8<E>(x);
        *reinterpret_cast<uint4*>(dst + H2 + i0) = pack8<E>(y);
    }
}

template <class S>
cudaError_t launch_src(const PagedAppendArgs& a, cudaStream_t s) {
    const int per_tok = ((a.q ? a.NH : 0) + 2 * a.c.NKV) * (a.c.D / 16);
    const int tpb = per_tok >= AP_THREADS ? 1 : AP_THREADS / per_tok;
    const dim3 grid((unsigned)(((long long)a.n + tpb - 1) / tpb));
    return a.c.bf16 ? launch_k(k_paged_append<S, ElemBf16>, grid, dim3(AP_THREADS), 0, s, a, tpb)
                    : launch_k(k_paged_append<S, ElemF16>, grid, dim3(AP_THREADS), 0, s, a, tpb);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    if (a.src == 0) return launch_src<SrcF32>(a, s);
    return a.src == 1 ? launch_src<SrcBf16>(a, s) : launch_src<SrcF16>(a, s);
}

}  // namespace ember
