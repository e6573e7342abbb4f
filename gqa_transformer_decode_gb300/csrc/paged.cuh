// paged.cuh -- device helpers shared by the paged-cache kernels: element
// types, cp.async copies with zero fill, warp matrix products on bf16 or f16
// operands, and which keys of a paged sequence a query sees.
#pragma once

#include <cuda_bf16.h>

#include "kernels.h"
#include "mma_common.cuh"

namespace ember {

// Cache element types.  Values are computed in f32 and rounded once, to
// nearest even, when they are stored.
// LIFT: softmax weights go into the second product as 2^(s - max + LIFT).  Below 2^-14
// an f16 has a fixed step of 2^-24, so without a lift 250000 keys of weight 2^-25.1
// each, 0.7 % of the sum beside one key of weight 1, would round to nothing; lifted,
// a weight is off by at most 2^-32 of the largest one.
struct ElemBf16 {
    static constexpr bool bf16 = true;
    static constexpr float LIFT = 0.f;
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ __forceinline__ static float lo(uint32_t u) { return bf16_lo(u); }
    __device__ __forceinline__ static float hi(uint32_t u) { return bf16_hi(u); }
    // c += a (16x16) * b (16x8), f32 accumulators
    __device__ __forceinline__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
struct ElemF16 {
    static constexpr bool bf16 = false;
    static constexpr float LIFT = 7.f;
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
    __device__ __forceinline__ static float lo(uint32_t u) { return __half2float(__ushort_as_half((uint16_t)u)); }
    __device__ __forceinline__ static float hi(uint32_t u) { return __half2float(__ushort_as_half((uint16_t)(u >> 16))); }
    __device__ __forceinline__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        mma16816(c, a, b0, b1);
    }
};

// 16 bytes from global to shared memory, or 16 zero bytes when !valid (the
// source is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- thread-block clusters: shared memory at the same address in another CTA ----
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.f32 %0, [r];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr, uint32_t rank) {
    float2 v;
    asm volatile(
        "{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [r];\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync_all() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// Keys of one sequence that a query at position pos sees: all of [0, pos], or
// under a window the last `window` of them and the first `sinks`.
struct Visible {
    int end;    // pos + 1: keys at or beyond it are hidden
    int first;  // first key of the window (0 without one)
    int sinks;  // keys below it are visible too
    __device__ __forceinline__ Visible(int pos, int window, int n_sinks) {
        end = pos + 1;
        first = window > 0 ? max(0, end - window) : 0;
        sinks = min(n_sinks, first);
    }
    __device__ __forceinline__ bool sees(int key) const { return key < end && (key >= first || key < sinks); }
};

// The scores' running maximum starts at a finite value below every score that
// counts, so that a row which has seen no key yet (or only scores of -inf)
// never forms inf - inf.
constexpr float SOFTMAX_FLOOR = -3.0e38f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// ---- prefill: query rows of a ragged batch ----
// One sequence's query rows and keys; nq == 0 when it has none or is invalid.
struct SeqRows {
    int row0, nq, len, seq;
};
__device__ __forceinline__ SeqRows seq_rows(const PagedPrefillArgs& a, int b, bool report) {
    SeqRows r{0, 0, 0, 0};
    r.seq = a.seqs ? a.seqs[b] : b;
    if (r.seq < 0) return r;
    const int r0 = a.cu[b], r1 = a.cu[b + 1];
    const int len = a.lens[b];
    int err = 0;
    if (r.seq >= a.c.n_seqs || r0 < 0 || r1 < r0 || r1 > a.n) err = EMBER_ERR_INVALID_ARG;
    else if (len < 0 || len > ((long long)a.c.width << a.c.page_shift)) err = EMBER_ERR_CAPACITY;
    if (err) {
        if (report) raise_status(a.status, err);
        return r;
    }
    r.row0 = r0;
    r.nq = r1 - r0;
    r.len = len;
    return r;
}

// The x-th tile of `tokens` query tokens over all sequences: its sequence and
// its number there (sequence -1: there are fewer tiles).  Every warp finds it by
// itself, 32 sequences at a time.
struct RowTile {
    int b, i;
};
__device__ __forceinline__ RowTile find_row_tile(const PagedPrefillArgs& a, int tokens, int x, bool report) {
    const int lane = threadIdx.x & 31;
    RowTile r{-1, 0};
    long long run = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = b0 + lane < a.B ? (seq_rows(a, b0 + lane, report).nq + tokens - 1) / tokens : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += y;
        }
        const long long at = run + incl - n;
        const unsigned hit = __ballot_sync(FULL_MASK, n > 0 && at <= x && x < at + n);
        if (hit && r.b < 0) {
            const int src = __ffs(hit) - 1;
            r.b = b0 + src;
            r.i = __shfl_sync(FULL_MASK, (int)(x - at), src);
            if (!report) break;              // the reporting warp looks at every sequence
        }
        run += __shfl_sync(FULL_MASK, incl, 31);
    }
    return r;
}

}  // namespace ember
