// logprobs.cu -- from rows of logits l, with x = l / temperature: the log probability
// x_i - log sum_j e^{x_j} of a given token and its rank, the entropy
// -sum_j p_j log p_j, and the `top` largest logits with their log probabilities.
//
// Bound: one read of the logits.  So everything comes out of one pass: each thread keeps
// a running maximum m of its logits, S = sum e^{(l - m) / t} and U = sum e^{(l - m) / t}
// (l - m), rescaled when m moves (at most a few times a row), and the entropy is
// log S - U / (S t), two terms of one sign; the given token's logit is read first, so
// that its rank is a count on the way.
//
// The largest `top` <= 32 come out of the same pass by a threshold that rises: the
// threads form 32 groups, whose maxima so far are 32 different elements, so that the
// top-th largest of these maxima is a lower bound of the top-th largest logit.  The
// number of a 16-byte vector with an element at or above the bound goes into a list (a
// few hundred of a row of 150000 do), everything else costs nothing, since the maximum of
// a vector is taken for m anyway.  In the end these vectors are read again, and their
// elements above the last bound ordered by counting.  Rows that overflow the list
// (thousands of equal largest logits) or hold a NaN are searched value by value, slowly
// but right.
//
// A row is split over the CTAs of a cluster while that leaves CTAs idle otherwise, and
// joined through distributed shared memory: one launch, no workspace, no atomics on
// global memory; equal calls give equal bits.
#include "kernels.h"
#include "paged.cuh"

namespace ember {

namespace {

// Threads of a CTA, T: 512 while the rows are few, whose ends (joining, ordering) then take half the
// time (64 rows of 128256 f32, top 20: 18.0 us, with 256 20.9), else 256, whose rows end one under
// another's loads (2048 rows of 151936 bf16, top 10: 143 us, with 512 167).  1024 threads of an SM either way.
constexpr int lp_per_sm(int T) { return 1024 / T; }
constexpr int LP_AHEAD = 4;                     // vectors of 16 bytes in flight for each thread
constexpr int LP_TOP = EMBER_LOGPROBS_MAX_TOP;
constexpr int LP_CLUSTER = 8;                   // CTAs of a row at most
constexpr int LP_HITS = 2048;                   // vectors looked at again at most
// A group (T / 32 lanes) without elements leaves no bound, but then there are less than T vectors (of 8) and the ends.
constexpr int lp_list(int T) { return 8 * (T + 2); }
static_assert(LP_TOP == 32, "one group's maximum for each of the largest");
// In the fast pass every logit counts as at least LP_LOW: -inf then has the weight 0 and
// gives no inf - inf.  A row whose largest logit is not within +-LP_LOW goes the slow way.
constexpr float LP_LOW = -1e30f;

// the larger of two and of three, NaN if any is
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y, float z) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// Element types.  largest: of a 16-byte vector, at least LP_LOW, NaN if one is; unpack: its
// elements as floats that are at least LP_LOW; above: how many are larger than x (EQUAL: or equal),
// x of the type, in pairs (1.0 for each; with conversions first it took twice as long).
struct LogitF32 {
    static constexpr int VEC = 4;
    using T = float;
    static constexpr uint32_t NONE = 0xff800000u;   // -inf
    __device__ __forceinline__ static float one(float x) { return x; }
    __device__ __forceinline__ static float largest(const uint4& w) {
        return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z)), __uint_as_float(w.w), LP_LOW);
    }
    __device__ __forceinline__ static void unpack(const uint4& w, float* x) {
        x[0] = max_nan(__uint_as_float(w.x), LP_LOW), x[1] = max_nan(__uint_as_float(w.y), LP_LOW);
        x[2] = max_nan(__uint_as_float(w.z), LP_LOW), x[3] = max_nan(__uint_as_float(w.w), LP_LOW);
    }
    template <bool EQUAL>
    __device__ __forceinline__ static int above(const uint4& w, float x) {
        auto one = [&](uint32_t u) { return (int)(EQUAL ? __uint_as_float(u) >= x : __uint_as_float(u) > x); };
        return one(w.x) + one(w.y) + one(w.z) + one(w.w);
    }
};
struct LogitBf16 {
    static constexpr int VEC = 8;
    using T = uint16_t;
    static constexpr uint32_t NONE = 0xff80ff80u;
    __device__ __forceinline__ static float one(uint16_t x) { return bf16_to_f32(x); }
    __device__ __forceinline__ static float largest(const uint4& w) {
        const uint32_t m = max_bf16x2(max_bf16x2(w.x, w.y), max_bf16x2(w.z, w.w));
        return max_nan(bf16_lo(m), bf16_hi(m), LP_LOW);
    }
    __device__ __forceinline__ static void unpack(uint4 w, float* x) {
        constexpr uint32_t low = 0xf14af14au;       // -1.0003e30: the largest bf16 that is not above LP_LOW
        unpack8(make_uint4(max_bf16x2(w.x, low), max_bf16x2(w.y, low), max_bf16x2(w.z, low), max_bf16x2(w.w, low)), x);
    }
    template <bool EQUAL>
    __device__ __forceinline__ static int above(const uint4& w, float x) {
        const __nv_bfloat162 t = __float2bfloat162_rn(x);
        auto two = [&](uint32_t u) {
            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&u);
            return EQUAL ? __hge2(v, t) : __hgt2(v, t);
        };
        const __nv_bfloat162 n = __hadd2(__hadd2(two(w.x), two(w.y)), __hadd2(two(w.z), two(w.w)));
        return (int)(__low2float(n) + __high2float(n));
    }
};
struct LogitF16 {
    static constexpr int VEC = 8;
    using T = uint16_t;
    static constexpr uint32_t NONE = 0xfc00fc00u;
    __device__ __forceinline__ static float one(uint16_t x) { return __half2float(__ushort_as_half(x)); }
    __device__ __forceinline__ static float largest(const uint4& w) {
        const uint32_t m = max_f16x2(max_f16x2(w.x, w.y), max_f16x2(w.z, w.w));
        return max_nan(one((uint16_t)m), one((uint16_t)(m >> 16)), LP_LOW);
    }
    __device__ __forceinline__ static void unpack(const uint4& w, float* x) {
        unpack8_f16(w, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = max_nan(x[e], LP_LOW);
    }
    template <bool EQUAL>
    __device__ __forceinline__ static int above(const uint4& w, float x) {
        const __half2 t = __float2half2_rn(x);
        auto two = [&](uint32_t u) {
            const __half2 v = *reinterpret_cast<const __half2*>(&u);
            return EQUAL ? __hge2(v, t) : __hgt2(v, t);
        };
        const __half2 n = __hadd2(__hadd2(two(w.x), two(w.y)), __hadd2(two(w.z), two(w.w)));
        return (int)(__low2float(n) + __high2float(n));
    }
};

// two f32 operations in one instruction
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// the value that argmax_key made the key's high word from (NaN for the highest)
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t u = (uint32_t)(k >> 32);
    if (u == 0xffffffffu) return __uint_as_float(0x7fffffffu);
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// A row's maximum, S and U (see above) and the count that the rank is made of.
struct Sums {
    float m, s, u;
    int above;
    __device__ __forceinline__ void move(float to, float c2) {   // to a larger maximum
        const float f = ex2((m - to) * c2);
        u = f == 0.f ? 0.f : f * fmaf(s, m - to, u);   // (without weight m - to may be of any size)
        s *= f;
        m = to;
    }
};

// The sums of N neighbouring lanes joined: all to the largest maximum first, then plain sums, in
// one order for all of them.
template <int N>
__device__ __forceinline__ Sums join_lanes(Sums q, float c2) {
    float m = q.m;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
    if (m > q.m) q.move(m, c2);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        q.s += __shfl_xor_sync(FULL_MASK, q.s, o);
        q.u += __shfl_xor_sync(FULL_MASK, q.u, o);
        q.above += __shfl_xor_sync(FULL_MASK, q.above, o);
    }
    return q;
}
// Over the whole CTA (s_sums: one a warp).
template <int T>
__device__ __noinline__ Sums join_all(Sums q, float c2, Sums* s_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    q = join_lanes<32>(q, c2);
    __syncthreads();
    if (lane == 0) s_sums[warp] = q;
    __syncthreads();
    return join_lanes<T / 32>(s_sums[lane % (T / 32)], c2);
}

// Leaves the maximum of this thread's group so far, from g, the thread's.
template <int T>
__device__ __forceinline__ void leave_maximum(float g, float* s_group) {
    constexpr int GROUP = T / 32;
#pragma unroll
    for (int o = 1; o < GROUP; o <<= 1) g = fmaxf(g, __shfl_xor_sync(FULL_MASK, g, o));
    if (threadIdx.x % GROUP == 0) *(volatile float*)(s_group + threadIdx.x / GROUP) = g;
}
// A lower bound of the top-th largest logit from the groups' maxima as they are (each a
// lower bound of what it will be): the top-th largest of them, sorted by a whole warp.
__device__ __noinline__ float raised_bound(const float* s_group, int top) {
    const int lane = threadIdx.x & 31;
    float v = *(const volatile float*)(s_group + lane);
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size / 2; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(FULL_MASK, v, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0);   // of the two goes to the lower lane, in the end
            v = larger ? fmaxf(v, y) : fminf(v, y);
        }
    return fmaxf(LP_LOW, __shfl_sync(FULL_MASK, v, top - 1));
}

// Puts each key of s_keys[0 .. n) that is among the `top` largest into its place: the number of
// larger ones (0: no key).  Four lanes count for a key.
template <int T>
__device__ __noinline__ void order_keys(const unsigned long long* s_keys, int n, int top, unsigned long long* s_top) {
    for (int i0 = 0; i0 < n; i0 += T / 4) {
        const int i = i0 + (int)threadIdx.x / 4;
        const unsigned long long x = i < n ? s_keys[i] : 0ull;
        int larger = 0;
#pragma unroll 4
        for (int k = threadIdx.x & 3; k < n; k += 4) larger += s_keys[k] > x;
        larger += __shfl_xor_sync(FULL_MASK, larger, 1);
        larger += __shfl_xor_sync(FULL_MASK, larger, 2);
        if (x != 0 && larger < top && (threadIdx.x & 3) == 0) s_top[larger] = x;
    }
}

// The slow ways, over elements [i0, i1) of a row, by the whole CTA.
struct Search {
    unsigned long long best[32];
    int found[32];
};
// Adds to s_top[have ..] the largest elements of values below that of the key `before` (first: there
// is none), in order, until there are `top`: finds the largest, then in one walk all that equal it.
template <class L, int T>
__device__ __noinline__ int take_largest(const typename L::T* row, int i0, int i1, unsigned long long before, bool first,
                                         int have, int top, unsigned long long* s_top, Search& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    while (have < top) {
        unsigned long long best = 0;
        const float limit = key_value(before);
        if (first || limit != limit) {
            for (int i = i0 + tid; i < i1; i += T) {
                const unsigned long long k = argmax_key(L::one(row[i]), (uint32_t)i);
                if ((first || k < before) && k > best) best = k;
            }
        } else {                                     // what a mask has left few of: by value alone, the walk from the start
            float m = -INFINITY;
            bool any = false;
#pragma unroll 8
            for (int i = i0 + tid; i < i1; i += T) {
                const float x = L::one(row[i]);
                any |= x < limit;
                m = fmaxf(m, x < limit ? x : -INFINITY);
            }
            if (any) best = argmax_key(m, (uint32_t)i0);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(FULL_MASK, best, o);
            best = y > best ? y : best;
        }
        __syncthreads();
        if (lane == 0) s.best[warp] = best;
        __syncthreads();
        for (int w = 0; w < (T / 32); ++w) best = s.best[w] > best ? s.best[w] : best;
        if (best == 0) return have;                  // no more of them (a key is never 0)
        const uint32_t value = (uint32_t)(best >> 32);
        for (int j = argmax_key_index(best); j < i1 && have < top; j += T) {
            const int i = j + tid;
            const unsigned long long k = i < i1 ? argmax_key(L::one(row[i]), (uint32_t)i) : 0ull;
            const bool same = i < i1 && (uint32_t)(k >> 32) == value;
            const unsigned m = __ballot_sync(FULL_MASK, same);
            __syncthreads();
            if (lane == 0) s.found[warp] = __popc(m);
            __syncthreads();
            int at = have + __popc(m & ((1u << lane) - 1u));
            for (int w = 0; w < (T / 32); ++w) {
                if (w < warp) at += s.found[w];
                have += s.found[w];
            }
            if (same && at < top) s_top[at] = k;
        }
        before = (unsigned long long)value << 32;    // below all of this value
        first = false;
    }
    return top;
}
// Sums of a row of any values; above: how many stand before element id, less id.
template <class L, int T>
__device__ __noinline__ Sums sum_slowly(const typename L::T* row, int i0, int i1, int id, float xi, float c2, Sums* s_sums) {
    Sums q{-INFINITY, 0.f, 0.f, 0};
    const unsigned long long mine = id >= 0 ? argmax_key(xi, (uint32_t)id) : 0ull;
    for (int i = i0 + (int)threadIdx.x; i < i1; i += T) {
        const float x = L::one(row[i]);
        if (id >= 0) q.above += (argmax_key(x, (uint32_t)i) > mine) - (i < id);
        if (x > q.m) q.move(x, c2);
        const float d = fmaxf(x - q.m, LP_LOW), p = x == -INFINITY ? 0.f : ex2(d * c2);
        q.s += p;
        q.u = fmaf(p, d, q.u);
    }
    return join_all<T>(q, c2, s_sums);
}

template <class L, int T>
__global__ void __launch_bounds__(T, lp_per_sm(T)) k_logprobs(LogprobsArgs a) {
    constexpr int VEC = L::VEC, LP_LIST = lp_list(T);
    using Elem = typename L::T;
    __shared__ unsigned long long s_list[LP_LIST];
    __shared__ unsigned long long s_top[LP_TOP], s_all[LP_CLUSTER * LP_TOP];
    __shared__ float s_group[32];
    __shared__ Sums s_sums[T / 32], s_part;
    __shared__ int s_hit[LP_HITS], s_hits, s_count, s_nan;
    __shared__ Search s_search;
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned C = a.cluster, part = blockIdx.x % C;
    const long long r = blockIdx.x / C;
    const int top = a.top;
    if (tid == 0) s_hits = s_count = s_nan = 0;
    if (tid < LP_TOP) s_top[tid] = 0;
    if (tid < 32) s_group[tid] = -INFINITY;
    pdl_wait();

    // Vector j of the row holds elements first + j * VEC ..: the 0th ends where the row's
    // memory is aligned, so it and the last one may be partly or wholly outside.
    const Elem* row = static_cast<const Elem*>(a.logits) + r * a.ldl;
    const int ahead = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(Elem);   // elements before it
    const int first = ahead - VEC;
    const int vectors = 1 + (int)(((long long)a.V - ahead + VEC - 1) / VEC);
    const int lo = (int)((long long)vectors * part / C), hi = (int)((long long)vectors * (part + 1) / C);
    const int whole_lo = max(lo, 1), whole_hi = min(hi, 1 + (a.V - ahead) / VEC);   // (V < ahead: none)
    const uint4* at = reinterpret_cast<const uint4*>(row + first);                 // vector 0
    const float c2 = LOG2E / a.t;

    const int id = a.ids ? a.ids[r] : -1;
    const bool given = id >= 0 && id < a.V;
    const float xi = given ? L::one(row[id]) : 0.f;
    const int jid = given ? (id - first) / VEC : -1;                               // its vector

    Sums q{LP_LOW, 0.f, 0.f, 0};
    bool nan = false;
    float bound = LP_LOW;                        // of the top-th largest logit, from below
    auto raise = [&]() { bound = raised_bound(s_group, top); };
    // Lists element i of value x if it may be among the largest.
    auto list = [&](float x, int i) {
        if (!(x >= bound && x > LP_LOW)) return;
        const int n = atomicAdd(&s_count, 1);
        if (n < LP_LIST) s_list[n] = argmax_key(x, (uint32_t)i);
    };
    // The same in the batch that the given token's vector lies in or stands between.
    auto count_around = [&](const uint4 (&w)[LP_AHEAD], int j) {
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k)
            if (j + k * T < whole_hi)            // (-inf stands beyond the part, which may equal xi)
                q.above += j + k * T < jid ? L::template above<true>(w[k], xi) : L::template above<false>(w[k], xi);
        if ((jid - j) % T == 0 && jid >= whole_lo && jid < whole_hi)   // its own vector: equal ones before it (read again)
            for (int i = first + jid * VEC; i < id; ++i) q.above += L::one(row[i]) == xi;
    };
    // the row's ends, an element for each of the first threads
    const int j_end = tid < VEC ? 0 : vectors - 1, i_end = first + j_end * VEC + tid % VEC;
    const bool has_end = tid < 2 * VEC && j_end >= lo && j_end < hi && (j_end < whole_lo || j_end >= whole_hi) &&
                         (tid < VEC || j_end > 0) && i_end >= 0 && i_end < a.V;
    const float x_end = has_end ? L::one(row[i_end]) : 0.f;
    uint4 next[LP_AHEAD];
    const uint4 none = make_uint4(L::NONE, L::NONE, L::NONE, L::NONE);
#pragma unroll
    for (int k = 0; k < LP_AHEAD; ++k) {
        const int j = whole_lo + tid + k * T;
        next[k] = j < whole_hi ? ld_stream(at + j) : none;
    }
    __syncthreads();
    if (top > 0) {                               // a first bound before anything is listed
        float g = LP_LOW;
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) g = fmaxf(g, L::largest(next[k]));   // (a NaN is left out here, and found below)
        leave_maximum<T>(g, s_group);
        __syncthreads();
        raise();
        q.m = g;
    }
    const uint64_t k2 = pair(c2, c2);
    for (int j0 = whole_lo; j0 < whole_hi; j0 += LP_AHEAD * T) {
        // what has to be decided once for a batch, then its exponentials without a branch; vectors
        // beyond the part are -inf
        uint4 w[LP_AHEAD];
        float big[LP_AHEAD];
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            const int jn = j0 + tid + (k + LP_AHEAD) * T;
            w[k] = next[k];
            next[k] = jn < whole_hi ? ld_stream(at + jn) : none;
            big[k] = L::largest(w[k]);
        }
        float most = max_nan(max_nan(big[0], big[1], big[2]), big[3]);
        static_assert(LP_AHEAD == 4, "the batch's largest");
        if (!(most <= q.m)) {
            if (most != most) {
                nan = true;
                most = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));   // (the row goes the slow way)
            }
            if (most > q.m) q.move(most, c2);
        }
        const int j = j0 + tid;
        if (given && most >= xi) {               // larger ones, before the given token equal ones too
            if (j + (LP_AHEAD - 1) * T < min(jid, whole_hi)) {
#pragma unroll
                for (int k = 0; k < LP_AHEAD; ++k) q.above += L::template above<true>(w[k], xi);
            } else if (j > jid) {
#pragma unroll
                for (int k = 0; k < LP_AHEAD; ++k) q.above += L::template above<false>(w[k], xi);
            } else {
                count_around(w, j);
            }
        }
        bool listed = false;
        if (top > 0 && most >= bound)
#pragma unroll
            for (int k = 0; k < LP_AHEAD; ++k)
                if (big[k] >= bound && big[k] > LP_LOW) {   // (beyond the part all are LP_LOW)
                    const int n = atomicAdd(&s_hits, 1);
                    if (n < LP_HITS) s_hit[n] = j + k * T;
                    listed = true;
                }
        const uint64_t m2 = pair(-q.m, -q.m);
        uint64_t s = 0ull, u = 0ull;
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            float x[VEC];
            L::unpack(w[k], x);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const uint64_t d = add2(pair(x[e], x[e + 1]), m2);
                float2 p = halves(mul2(d, k2));
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                const uint64_t p2 = pair(p.x, p.y);
                s = add2(s, p2);
                u = fma2(p2, d, u);
            }
        }
        const float2 s1 = halves(s), u1 = halves(u);
        q.s += s1.x + s1.y;
        q.u += u1.x + u1.y;
        if (top > 0 && __any_sync(FULL_MASK, listed)) {
            leave_maximum<T>(q.m, s_group);
            __syncwarp();
            raise();
        }
    }
    if (has_end) {
        const float v = max_nan(x_end, LP_LOW);
        if (v != v) nan = true;
        else if (v > q.m) q.move(v, c2);
        if (given) q.above += x_end > xi || (x_end == xi && i_end < id);
        if (top > 0) list(v, i_end);
        const float d = v - q.m, p = ex2(d * c2);
        q.s += p;
        q.u = fmaf(p, d, q.u);
    }
    if (nan) s_nan = 1;
    if (top > 0) leave_maximum<T>(q.m, s_group);
    q = join_all<T>(q, c2, s_sums);

    // ---- this part's largest above LP_LOW, in order ----
    const int i_lo = max(0, first + lo * VEC), i_hi = (int)min((long long)a.V, first + (long long)hi * VEC);
    if (top > 0) {
        raise();                                 // (of the whole part)
        const int hits = s_hits;
        if (hits <= LP_HITS)
            for (int h = tid; h < hits; h += T) {
                const int j = s_hit[h];
                float x[VEC];
                L::unpack(ld_stream(at + j), x);
#pragma unroll
                for (int e = 0; e < VEC; ++e) list(x[e], first + j * VEC + e);
            }
        __syncthreads();
        const int listed = s_count;
        if (s_nan || hits > LP_HITS || listed > LP_LIST) {
            take_largest<L, T>(row, i_lo, i_hi, 0ull, true, 0, top, s_top, s_search);
            __syncthreads();
            if (tid < top && s_top[tid] <= argmax_key(LP_LOW, 0u)) s_top[tid] = 0;
        } else {
            order_keys<T>(s_list, listed, top, s_top);
        }
    }
    if (tid == 0) s_part = q;
    pdl_trigger();

    // ---- the parts' joined in the first CTA ----
    if (C > 1) {
        cluster_sync_all();
        if (part == 0) {
            const uint32_t sums = sa_u32(&s_part), keys = sa_u32(s_top);
            Sums y{LP_LOW, 0.f, 0.f, 0};
            if (lane < (int)C) {
                y.m = ld_cluster(sums, lane);
                y.s = ld_cluster(sums + 4, lane);
                y.u = ld_cluster(sums + 8, lane);
                y.above = __float_as_int(ld_cluster(sums + 12, lane));
            }
            q = join_lanes<LP_CLUSTER>(y, c2);
            q.m = __shfl_sync(FULL_MASK, q.m, 0);
            q.s = __shfl_sync(FULL_MASK, q.s, 0);
            q.u = __shfl_sync(FULL_MASK, q.u, 0);
            q.above = __shfl_sync(FULL_MASK, q.above, 0);
            for (int i = tid; i < (int)C * top; i += T) {
                const float2 k = ld_cluster2(keys + 8 * (i % top), i / top);
                s_all[i] = (unsigned long long)__float_as_uint(k.y) << 32 | __float_as_uint(k.x);
            }
            if (tid > 0 && tid < (int)C && __float_as_int(ld_cluster(sa_u32(&s_nan), tid)) != 0) s_nan = 1;
        }
        // no CTA leaves while its shared memory is read
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        if (part != 0) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            return;
        }
        __syncthreads();
        if (tid < top) s_top[tid] = 0;
        __syncthreads();
        order_keys<T>(s_all, (int)C * top, top, s_top);
    }
    __syncthreads();

    // ---- what the fast pass leaves out ----
    const bool has_nan = s_nan != 0;
    if (has_nan || !(q.m > LP_LOW && q.m < -LP_LOW))
        q = sum_slowly<L, T>(row, 0, a.V, given ? id : -1, xi, c2, s_sums);
    else if (given)
        q.above -= id;                           // (sum_slowly's count)
    if (top > 0) {
        const int have = __syncthreads_count(tid < top && s_top[min(tid, LP_TOP - 1)] != 0);
        if (have < top) take_largest<L, T>(row, 0, a.V, have > 0 ? s_top[have - 1] : 0ull, have == 0, have, top, s_top, s_search);
        __syncthreads();
    }

    // ---- the row's outputs ----
    const bool flat = q.m == -INFINITY && !has_nan;                // every logit -inf: uniform, as the sampler has it
    const bool undefined = has_nan || q.m == INFINITY;
    const float log_s = flat ? logf((float)a.V) : logf(q.s);
    auto logprob = [&](float x) {
        if (undefined) return __int_as_float(0x7fffffff);
        return flat ? -log_s : (x - q.m) / a.t - log_s;
    };
    if (tid == 0) {
        if (a.logprob) a.logprob[r] = given ? logprob(xi) : __int_as_float(0x7fffffff);
        if (a.rank) a.rank[r] = given ? q.above + id : -1;
        if (a.entropy) a.entropy[r] = undefined ? __int_as_float(0x7fffffff) : flat ? log_s : log_s - q.u / (q.s * a.t);
    }
    if (tid < top) {
        const unsigned long long k = s_top[tid];
        a.top_ids[r * top + tid] = argmax_key_index(k);
        a.top_logprobs[r * top + tid] = logprob(key_value(k));
    }
    if (C > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

template <class L, int T>
cudaError_t launch_threads(LogprobsArgs a, int sms, cudaStream_t s) {
    // As many CTAs of a row as leave every one its place and a first batch.
    a.cluster = 1;
    while (a.cluster < LP_CLUSTER && (long long)a.n * a.cluster * 2 <= lp_per_sm(T) * sms && a.V >= 2 * a.cluster * L::VEC * T)
        a.cluster *= 2;
    const dim3 grid((unsigned)(a.n * (long long)a.cluster));
    if (a.cluster > 1) return launch_cluster_k(k_logprobs<L, T>, grid, dim3(T), 0, a.cluster, s, a);
    return launch_k(k_logprobs<L, T>, grid, dim3(T), 0, s, a);
}
template <class L>
cudaError_t launch_type(const LogprobsArgs& a, int sms, cudaStream_t s) {
    return a.n <= sms ? launch_threads<L, 512>(a, sms, s) : launch_threads<L, 256>(a, sms, s);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, int sms, cudaStream_t s) {
    if (a.dtype == EMBER_F32) return launch_type<LogitF32>(a, sms, s);
    return a.dtype == EMBER_BF16 ? launch_type<LogitBf16>(a, sms, s) : launch_type<LogitF16>(a, sms, s);
}

}  // namespace ember
