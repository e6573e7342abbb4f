// paged_groups.cuh -- the line of key tiles of shared prefixes, as the prefixes' kernel
// (paged_prefill_tc.cu, PT_SHARED) and the rows' own (paged_shared.cu) see it, and which SMs
// take which.
#pragma once

#include "paged.cuh"

namespace ember {

namespace {

constexpr int PT_KEYS = 64;    // keys of a tile
constexpr int PT_SHARE = 4;    // key tiles of a CTA at least

// Groups cu[g] .. cu[g + 1] - 1 of n rows that read keys[g] keys of table row seqs[g].
struct PtGroups {
    const int32_t *cu, *keys, *seqs, *lens;
    int n_groups, n, n_seqs, NKV, rows_per_pair;
    long long most;            // keys that the table has room for
};
// The rows of a group in pairs of tiles and its key tiles; none if it is invalid (the rows' own
// kernel reports that) or has no prefix.
struct PtGroup {
    int row0, nq, keys, seq, nx, tiles;
};
__device__ __forceinline__ PtGroup pt_group(const PtGroups& a, int g) {
    PtGroup r{0, 0, 0, 0, 0, 0};
    if (g >= a.n_groups) return r;
    const int r0 = a.cu[g], r1 = a.cu[g + 1], keys = a.keys[g], seq = a.seqs[g];
    if (seq < 0 || seq >= a.n_seqs || r0 < 0 || r1 <= r0 || r1 > a.n || keys <= 0 || keys > a.most) return r;
    r.row0 = r0;
    r.nq = r1 - r0;
    r.keys = keys;
    r.seq = seq;
    r.nx = (r.nq + a.rows_per_pair - 1) / a.rows_per_pair;
    r.tiles = (keys + PT_KEYS - 1) / PT_KEYS;
    return r;
}
// The keys that some of the rows sees, for a whole warp: the longest length.  (Rows of padding count:
// to look whether a row is one, in an array that nothing else here needs, took 2 us.)
__device__ __forceinline__ int pt_seen(const PtGroups& a, int row0, int rows) {
    int seen = 0;
    for (int i = row0 + (int)(threadIdx.x & 31); i < row0 + rows; i += 32) {
        const int len = a.lens[i];
        if (len <= a.most) seen = max(seen, len);
    }
    return __reduce_max_sync(FULL_MASK, seen);
}
// Where 32 groups' rows (each for every kv head) and key tiles begin, each lane its own group's, after
// those of `rows` and `line` before; both are moved on, and the number of pairs.
__device__ __forceinline__ PtGroup pt_scan(const PtGroups& a, int g0, unsigned& pairs, unsigned& rows, unsigned& line,
                                           unsigned& row0, unsigned& line0) {
    const int lane = threadIdx.x & 31;
    const PtGroup r = pt_group(a, g0 + lane);
    const unsigned np = (unsigned)r.nx * a.NKV, nr = (unsigned)r.nq * a.NKV, nl = np * (unsigned)r.tiles;
    pairs += __reduce_add_sync(FULL_MASK, np);
    row0 = nr;
    line0 = nl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(FULL_MASK, row0, o), y = __shfl_up_sync(FULL_MASK, line0, o);
        if (lane >= o) {
            row0 += x;
            line0 += y;
        }
    }
    const unsigned all_r = __shfl_sync(FULL_MASK, row0, 31), all_l = __shfl_sync(FULL_MASK, line0, 31);
    row0 += rows - nr;
    line0 += line - nl;
    rows += all_r;
    line += all_l;
    return r;
}

// SMs for the prefixes' products; the others are for the rows' own keys, which then run beside
// them.  That pays while both are short and made of latencies: 64 rows on 8192 keys and up to 512
// of their own 30.7 us, one kernel after the other 33.3.  With more than PT_APART tiles an SM a
// share that is off costs more than latencies do: five documents of 75 rows 77 us beside each
// other, 56 after each other; 256 rows of 32 heads on 8 of 64 on 16384 keys 134 and 95; though 128
// rows of 32 on 8 of 128 on 32768 104 and 115.
// In proportion to what each would take one SM: a key tile of a pair 1700 cycles, a pair four
// tiles more, and a CTA's SM reads 40 bytes a cycle when not all SMs do.  (64 rows on 8192 keys and
// 512 of their own 29.6 us so, with 1350 or 2300 cycles 30.5.)
constexpr unsigned PT_APART = 12;
__device__ __forceinline__ int prefix_sms(unsigned tiles, unsigned pairs, float tail_bytes, int sms) {
    if (tiles == 0) return 0;
    if (!(tail_bytes > 0.f) || tiles > PT_APART * sms) return sms;
    const float w1 = (tiles + 4.f * pairs) * 1700.f, w2 = tail_bytes * (1.f / 40.f);
    return min(sms - 1, max(1, (int)(sms * (w1 / (w1 + w2)) + 0.5f)));
}

}  // namespace

}  // namespace ember
