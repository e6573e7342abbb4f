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
// top-th largest of these maxima is a lower bound of the top-th largest logit.  An
// element at or above the bound goes into a list in shared memory (a few hundred of a
// row of 150000 do), everything else costs nothing, since the maximum of a vector is
// taken for m anyway.  The list is then ordered by counting.  Rows that overflow it
// (thousands of equal largest logits) or hold a NaN are searched once for each of the
// `top`, slowly but right.
//
// A row is split over the CTAs of a cluster while that leaves CTAs idle otherwise, and
// joined through distributed shared memory: one launch, no workspace, no atomics on
// global memory; equal calls give equal bits.
#include "kernels.h"
#include "paged.cuh"

namespace ember {

namespace {

constexpr int LP_THREADS = 512;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_GROUP = LP_THREADS / 32;       // lanes of a group: 32 groups
constexpr int LP_AHEAD = 4;                     // vectors of 16 bytes in flight for each thread
constexpr int LP_TOP = EMBER_LOGPROBS_MAX_TOP;
constexpr int LP_CLUSTER = 8;                   // CTAs of a row at most
// An empty group leaves no bound, but then fewer than LP_THREADS + 1 vectors of 8.
constexpr int LP_LIST = 8 * (LP_THREADS + 1);
static_assert(LP_TOP == 32, "one group's maximum for each of the largest");

struct LogitF32 {
    static constexpr int VEC = 4;
    using T = float;
    __device__ __forceinline__ static float one(float x) { return x; }
    __device__ __forceinline__ static void unpack(const uint4& w, float* x) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
};
struct LogitBf16 {
    static constexpr int VEC = 8;
    using T = uint16_t;
    __device__ __forceinline__ static float one(uint16_t x) { return bf16_to_f32(x); }
    __device__ __forceinline__ static void unpack(const uint4& w, float* x) { unpack8(w, x); }
};
struct LogitF16 {
    static constexpr int VEC = 8;
    using T = uint16_t;
    __device__ __forceinline__ static float one(uint16_t x) { return __half2float(__ushort_as_half(x)); }
    __device__ __forceinline__ static void unpack(const uint4& w, float* x) { unpack8_f16(w, x); }
};

// the larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
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
        const float f = m == -INFINITY ? 0.f : ex2((m - to) * c2);
        u = f == 0.f ? 0.f : f * fmaf(s, m - to, u);   // (without weight m - to may be of any size)
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o, float c2) {
        if (o.m > m) move(o.m, c2);
        else if (m > o.m) o.move(m, c2);
        s += o.s;
        u += o.u;
        above += o.above;
    }
};

template <class L>
__global__ void __launch_bounds__(LP_THREADS, 2) k_logprobs(LogprobsArgs a) {
    constexpr int VEC = L::VEC;
    using T = typename L::T;
    __shared__ unsigned long long s_list[LP_LIST];
    __shared__ unsigned long long s_top[LP_TOP];
    __shared__ unsigned long long s_all[LP_CLUSTER * LP_TOP];
    __shared__ float s_group[32];
    __shared__ Sums s_sums[LP_WARPS], s_part;
    __shared__ int s_count, s_nan, s_kept;
    __shared__ unsigned long long s_best[LP_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned C = a.cluster, part = blockIdx.x % C;
    const long long r = blockIdx.x / C;
    const int top = a.top;
    if (tid == 0) s_count = s_nan = s_kept = 0;
    if (tid < LP_TOP) s_top[tid] = 0;
    pdl_wait();

    // Vector j of the row holds elements first + j * VEC ..: the 0th ends where the row's
    // memory is aligned, so it and the last one may be partly or wholly outside.
    const T* row = static_cast<const T*>(a.logits) + r * a.ldl;
    const int ahead = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);   // elements before it
    const int first = ahead - VEC;
    const int vectors = 1 + (int)(((long long)a.V - ahead + VEC - 1) / VEC);
    const int lo = (int)((long long)vectors * part / C), hi = (int)((long long)vectors * (part + 1) / C);
    const float c2 = LOG2E / a.t;

    const int id = a.ids ? a.ids[r] : -1;
    const bool given = id >= 0 && id < a.V;
    const float xi = given ? L::one(row[id]) : 0.f;
    const int jid = given ? (id - first) / VEC : 0;

    auto whole = [&](int j) { return j > 0 && first + (j + 1) * VEC <= a.V; };
    auto fetch = [&](int j) {                    // its bits; elements outside are -inf
        if (j < hi && whole(j)) return ld_stream(reinterpret_cast<const uint4*>(row + first + (long long)j * VEC));
        constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<L, LogitF16>::value ? 0xfc00fc00u : 0xff80ff80u;
        uint4 w = make_uint4(none, none, none, none);
        if (j < hi) {
            uint32_t b[4] = {none, none, none, none};
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = first + j * VEC + e;
                if (i < 0 || i >= a.V) continue;
                if constexpr (sizeof(T) == 4) b[e] = __float_as_uint(row[i]);
                else b[e / 2] = e & 1 ? (b[e / 2] & 0xffffu) | (uint32_t)row[i] << 16 : (b[e / 2] & 0xffff0000u) | row[i];
            }
            w = make_uint4(b[0], b[1], b[2], b[3]);
        }
        return w;
    };

    Sums q{-INFINITY, 0.f, 0.f, 0};
    bool nan = false;
    float bound = -INFINITY;                     // of the top-th largest logit, from below
    // The bound from the groups' maxima as they are (each a lower bound of what it will be);
    // g: this thread's maximum.
    auto raise = [&](float g) {
#pragma unroll
        for (int o = 1; o < LP_GROUP; o <<= 1) g = fmaxf(g, __shfl_xor_sync(FULL_MASK, g, o));
        volatile float* group = s_group;
        if (lane % LP_GROUP == 0) group[tid / LP_GROUP] = g;
        __syncwarp();
        const float v = group[lane];
        int before = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float w = __shfl_sync(FULL_MASK, v, i);
            before += w > v || (w == v && i < lane);
        }
        const unsigned at = __ballot_sync(FULL_MASK, before == top - 1);
        bound = __shfl_sync(FULL_MASK, v, __ffs(at) - 1);
    };

    uint4 next[LP_AHEAD];
#pragma unroll
    for (int k = 0; k < LP_AHEAD; ++k) next[k] = fetch(lo + tid + k * LP_THREADS);
    if (tid < 32) s_group[tid] = -INFINITY;
    __syncthreads();
    if (top > 0) {                               // a first bound before anything is listed
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            float x[VEC];
            L::unpack(next[k], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) q.m = fmaxf(q.m, x[e]);
        }
        raise(q.m);
        __syncthreads();
        raise(q.m);
    }
    for (int j0 = lo; j0 < hi; j0 += LP_AHEAD * LP_THREADS) {
        bool listed = false;
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            const int j = j0 + tid + k * LP_THREADS;
            const uint4 w = next[k];
            next[k] = fetch(j + LP_AHEAD * LP_THREADS);
            if (j >= hi) continue;
            float x[VEC];
            L::unpack(w, x);
            float big = x[0];
#pragma unroll
            for (int e = 1; e < VEC; ++e) big = max_nan(big, x[e]);
            if (!(big <= q.m)) {
                if (big != big) {
                    nan = true;
                    big = q.m;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) big = fmaxf(big, x[e]);
                }
                if (big > q.m) q.move(big, c2);
            }
            if (top > 0 && big >= bound) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (x[e] >= bound && x[e] > -INFINITY) {
                        const int at = atomicAdd(&s_count, 1);
                        if (at < LP_LIST) s_list[at] = argmax_key(x[e], (uint32_t)(first + j * VEC + e));
                        listed = true;
                    }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // (-inf has no weight, and -inf - -inf is not a number: both end at the floor)
                const float d = fmaxf(x[e] - q.m, -1e30f);
                const float p = ex2(d * c2);
                q.s += p;
                q.u = fmaf(p, d, q.u);
            }
            if (given) {                         // elements that stand before the given one: larger, or equal and earlier
                if (j == jid || j == 0) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int i = first + j * VEC + e;
                        q.above += i < 0 || i >= a.V ? 0 : i < id ? -(x[e] < xi) : x[e] > xi;
                    }
                } else if (j < jid) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) q.above -= x[e] < xi;
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) q.above += x[e] > xi;
                }
            }
        }
        if (top > 0 && __any_sync(FULL_MASK, listed)) raise(q.m);
    }
    if (nan) s_nan = 1;
    const float largest = q.m;                   // of this thread
    if (top > 0) raise(largest);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sums y;
        y.m = __shfl_xor_sync(FULL_MASK, q.m, o);
        y.s = __shfl_xor_sync(FULL_MASK, q.s, o);
        y.u = __shfl_xor_sync(FULL_MASK, q.u, o);
        y.above = __shfl_xor_sync(FULL_MASK, q.above, o);
        // in the same order on both sides, so that all lanes hold the same sum
        if (lane & o) {
            y.join(q, c2);
            q = y;
        } else {
            q.join(y, c2);
        }
    }
    if (lane == 0) s_sums[warp] = q;
    __syncthreads();
    q = s_sums[0];
    for (int w = 1; w < LP_WARPS; ++w) q.join(s_sums[w], c2);
    const bool has_nan = s_nan != 0;

    // every element of this part by its key, NaN above all others
    auto each = [&](auto f) {
        const int i0 = max(0, first + lo * VEC), i1 = (int)min((long long)a.V, first + (long long)hi * VEC);
        for (int i = i0 + tid; i < i1; i += LP_THREADS) f(argmax_key(L::one(row[i]), (uint32_t)i));
    };
    if (given && (has_nan || xi != xi)) {        // the count by keys; id is added below
        const unsigned long long mine = argmax_key(xi, (uint32_t)id);
        int n = 0;
        each([&](unsigned long long k) {
            const int i = argmax_key_index(k);
            n += (k > mine) - (i < id);
        });
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(FULL_MASK, n, o);
        __syncthreads();
        if (lane == 0) s_sums[warp].above = n;
        __syncthreads();
        q.above = 0;
        for (int w = 0; w < LP_WARPS; ++w) q.above += s_sums[w].above;
    }
    if (tid == 0) s_part = q;

    // ---- this part's largest, in order, without -inf ----
    if (top > 0) {
        const int listed = s_count;
        if (has_nan || listed > LP_LIST) {
            unsigned long long before = ~0ull;
            const unsigned long long least = argmax_key(-INFINITY, 0u);   // (0u: the highest key of -inf)
            for (int k = 0; k < top; ++k) {
                unsigned long long best = 0;
                each([&](unsigned long long x) {
                    if ((k == 0 || x < before) && x > least && x > best) best = x;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long y = __shfl_xor_sync(FULL_MASK, best, o);
                    best = y > best ? y : best;
                }
                __syncthreads();
                if (lane == 0) s_best[warp] = best;
                __syncthreads();
                for (int w = 0; w < LP_WARPS; ++w) best = s_best[w] > best ? s_best[w] : best;
                if (tid == 0) s_top[k] = best;
                if (best == 0) break;            // no more of them (the same for all threads)
                before = best;
            }
        } else {
            // what lies below the last bound goes, then each element's place is the number of larger ones
            // (the highest index has the lowest key of its value)
            raise(largest);
            const unsigned long long least = argmax_key(bound, 0xffffffffu);
            unsigned long long keep[LP_LIST / LP_THREADS + 1];
#pragma unroll
            for (int k = 0; k < LP_LIST / LP_THREADS + 1; ++k) {
                const int i = tid + k * LP_THREADS;
                keep[k] = i < listed ? s_list[i] : 0ull;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < LP_LIST / LP_THREADS + 1; ++k)
                if (keep[k] != 0 && keep[k] >= least) s_list[atomicAdd(&s_kept, 1)] = keep[k];
            __syncthreads();
            const int kept = s_kept;
            for (int i = tid; i < kept; i += LP_THREADS) {
                const unsigned long long x = s_list[i];
                int larger = 0;
                for (int k = 0; k < kept; ++k) larger += s_list[k] > x;
                if (larger < top) s_top[larger] = x;
            }
        }
    }
    pdl_trigger();

    // ---- the parts' joined in the first CTA ----
    if (C > 1) {
        cluster_sync_all();
        if (part == 0) {
            const uint32_t at = sa_u32(&s_part), keys = sa_u32(s_top);
            for (unsigned p = 1; p < C; ++p) {
                Sums y;
                y.m = ld_cluster(at, p);
                y.s = ld_cluster(at + 4, p);
                y.u = ld_cluster(at + 8, p);
                y.above = __float_as_int(ld_cluster(at + 12, p));
                q.join(y, c2);
            }
            for (int i = tid; i < (int)C * top; i += LP_THREADS) {
                const float2 k = ld_cluster2(keys + 8 * (i % top), i / top);
                s_all[i] = (unsigned long long)__float_as_uint(k.y) << 32 | __float_as_uint(k.x);
            }
            if (tid == 0)
                for (unsigned p = 1; p < C; ++p)
                    if (__float_as_int(ld_cluster(sa_u32(&s_nan), p)) != 0) s_nan = 1;
        }
        cluster_sync_all();                      // no CTA leaves while its shared memory is read
        if (part != 0) return;
        if (tid < top) s_top[tid] = 0;
        __syncthreads();
        for (int i = tid; i < (int)C * top; i += LP_THREADS) {
            const unsigned long long x = s_all[i];
            if (x == 0) continue;
            int larger = 0;
            for (int k = 0; k < (int)C * top; ++k) larger += s_all[k] > x;
            if (larger < top) s_top[larger] = x;
        }
    }
    __syncthreads();

    // ---- the row's outputs ----
    const bool flat = q.m == -INFINITY && !s_nan;                  // every logit -inf: uniform, as the sampler has it
    const bool bad = s_nan || q.m == INFINITY;                     // no distribution
    const float log_s = flat ? logf((float)a.V) : logf(q.s);
    auto logprob = [&](float x) {
        if (bad) return __int_as_float(0x7fffffff);
        return flat ? -log_s : (x - q.m) / a.t - log_s;
    };
    if (tid == 0) {
        if (a.logprob) a.logprob[r] = given ? logprob(xi) : __int_as_float(0x7fffffff);
        if (a.rank) a.rank[r] = given ? q.above + id : -1;
        if (a.entropy) a.entropy[r] = bad ? __int_as_float(0x7fffffff) : flat ? log_s : log_s - q.u / (q.s * a.t);
    }
    if (warp == 0 && top > 0) {
        const unsigned long long k = lane < top ? s_top[lane] : 0ull;
        int have = __popc(__ballot_sync(FULL_MASK, k != 0));
        if (k != 0) {
            a.top_ids[r * top + lane] = argmax_key_index(k);
            a.top_logprobs[r * top + lane] = logprob(key_value(k));
        }
        // fewer than `top` above -inf: the first of the others, which stand among the first 64
        for (int i0 = 0; have < top && i0 < a.V; i0 += 32) {
            const int i = i0 + lane;
            const bool none = i < a.V && L::one(row[i]) == -INFINITY;
            const unsigned m = __ballot_sync(FULL_MASK, none);
            const int at = have + __popc(m & ((1u << lane) - 1u));
            if (none && at < top) {
                a.top_ids[r * top + at] = i;
                a.top_logprobs[r * top + at] = logprob(-INFINITY);
            }
            have += __popc(m);
        }
    }
}

template <class L>
cudaError_t launch_type(LogprobsArgs a, int sms, cudaStream_t s) {
    // As many CTAs of a row as leave every one its place (two on an SM) and a first batch.
    a.cluster = 1;
    while (a.cluster < LP_CLUSTER && (long long)a.n * a.cluster * 2 <= 2 * sms &&
           a.V >= 2 * a.cluster * L::VEC * LP_THREADS)
        a.cluster *= 2;
    const dim3 grid((unsigned)(a.n * (long long)a.cluster));
    if (a.cluster > 1) return launch_cluster_k(k_logprobs<L>, grid, dim3(LP_THREADS), 0, a.cluster, s, a);
    return launch_k(k_logprobs<L>, grid, dim3(LP_THREADS), 0, s, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, int sms, cudaStream_t s) {
    if (a.dtype == EMBER_F32) return launch_type<LogitF32>(a, sms, s);
    return a.dtype == EMBER_BF16 ? launch_type<LogitBf16>(a, sms, s) : launch_type<LogitF16>(a, sms, s);
}

}  // namespace ember
