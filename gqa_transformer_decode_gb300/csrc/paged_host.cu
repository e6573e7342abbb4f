// paged_host.cu -- the C entry points of the paged K/V cache operators:
// argument checks before any device work, then one or two launches.
#include "entry.h"

using namespace ember;

namespace {

__global__ void k_take_status(int* status, int* taken) {
    pdl_wait();
    *taken = atomicExch(status, 0);
}

// The checks every operator shares; fills the kernels' view of the cache.
ember_status check_cache(const ember_paged_kv* kv, PagedView& c) {
    if (!kv) PG_FAIL(EMBER_ERR_INVALID_ARG, "kv is NULL");
    if (!kv->k || !kv->v || !kv->table) PG_FAIL(EMBER_ERR_INVALID_ARG, "NULL pages or table");
    if (kv->dtype != EMBER_BF16 && kv->dtype != EMBER_F16)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "cache dtype must be EMBER_BF16 or EMBER_F16");
    if (kv->n_pages <= 0 || kv->n_kv_heads <= 0 || kv->n_seqs <= 0 || kv->table_width <= 0)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "n_pages, n_kv_heads, n_seqs and table_width must be > 0");
    const int D = kv->head_dim, P = kv->page_size;
    if (D != 16 && D != 32 && D != 64 && D != 128)
        PG_FAIL(EMBER_ERR_UNSUPPORTED, "head_dim must be 16, 32, 64 or 128");
    if (P < 16 || P > 1024 || (P & (P - 1)))
        PG_FAIL(EMBER_ERR_UNSUPPORTED, "page_size must be a power of two from 16 to 1024");
    if ((long long)kv->table_width * P > (1ll << 30))
        PG_FAIL(EMBER_ERR_UNSUPPORTED, "table_width * page_size > 2^30");
    if (!aligned16(kv->k) || !aligned16(kv->v) || (reinterpret_cast<uintptr_t>(kv->table) & 3))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "pages must be 16-byte aligned, the table 4-byte aligned");
    if (kv->row_stride < D || kv->head_stride < D || kv->page_stride < D || kv->row_stride % 8 ||
        kv->head_stride % 8 || kv->page_stride % 8)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "strides must be multiples of 8 elements and at least head_dim");
    c.k = static_cast<uint16_t*>(kv->k);
    c.v = static_cast<uint16_t*>(kv->v);
    c.table = kv->table;
    c.n_pages = kv->n_pages;
    c.page_shift = 0;
    while ((1 << c.page_shift) < P) ++c.page_shift;
    c.NKV = kv->n_kv_heads;
    c.D = D;
    c.n_seqs = kv->n_seqs;
    c.width = kv->table_width;
    c.page_stride = kv->page_stride;
    c.head_stride = kv->head_stride;
    c.row_stride = kv->row_stride;
    c.bf16 = kv->dtype == EMBER_BF16;
    return EMBER_OK;
}

ember_status check_heads(const ember_paged_kv* kv, int32_t n_heads) {
    if (n_heads <= 0 || n_heads % kv->n_kv_heads)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "n_heads must be a positive multiple of n_kv_heads");
    if (n_heads / kv->n_kv_heads > 16) PG_FAIL(EMBER_ERR_UNSUPPORTED, "GQA group > 16");
    if ((long long)n_heads * kv->head_dim > (1 << 20)) PG_FAIL(EMBER_ERR_UNSUPPORTED, "n_heads * head_dim > 2^20");
    return EMBER_OK;
}

// Checks that the two attentions share; window 0 when it hides nothing.
ember_status check_attention(const ember_paged_kv* kv, int32_t rows, int32_t n_heads, const void* q, int64_t ld_q,
                             const void* out, int64_t ld_out, const int32_t* lens, int32_t& window, int32_t& sinks,
                             float scale) {
    ember_status st = check_heads(kv, n_heads);
    if (st != EMBER_OK) return st;
    if (rows < 0 || rows > (1 << 30)) PG_FAIL(EMBER_ERR_INVALID_ARG, "bad number of rows");
    if (window < 0 || sinks < 0) PG_FAIL(EMBER_ERR_INVALID_ARG, "window and sinks must be >= 0");
    if (!(scale - scale == 0.f)) PG_FAIL(EMBER_ERR_INVALID_ARG, "scale must be finite");
    if (window >= (long long)kv->table_width * kv->page_size) window = 0;
    if (window == 0) sinks = 0;
    if (rows == 0) return EMBER_OK;
    if (!lens) PG_FAIL(EMBER_ERR_INVALID_ARG, "lens is NULL");
    st = check_rows("q", q, ld_q, (int64_t)n_heads * kv->head_dim);
    if (st != EMBER_OK) return st;
    return check_rows("out", out, ld_out, (int64_t)n_heads * kv->head_dim);
}

// Attention of one token per sequence; a.groups and what goes with it are set.
ember_status decode(const ember_paged_kv* kv, PagedDecodeArgs& a, const void* q, int64_t ld_q, int32_t B, int32_t n_heads,
                    const int32_t* seqs, const int32_t* lens, int32_t window, int32_t sinks, float scale, void* out,
                    int64_t ld_out, float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                    ember_stream_t stream) {
    ember_status st = check_cache(kv, a.c);
    if (st != EMBER_OK) return st;
    st = check_attention(kv, B, n_heads, q, ld_q, out, ld_out, lens, window, sinks, scale);
    if (st != EMBER_OK) return st;
    if (B == 0) return EMBER_OK;
    if (B > 65535) PG_FAIL(EMBER_ERR_UNSUPPORTED, "B > 65535");
    if (!seqs && B > kv->n_seqs) PG_FAIL(EMBER_ERR_INVALID_ARG, "B > n_seqs without seqs");
    if ((st = check_words("seqs, lens, lse and status", seqs, lens, lse, status)) != EMBER_OK) return st;
    if (kv->n_kv_heads > 65535 ||
        (double)B * kv->n_kv_heads * ((double)kv->table_width * kv->page_size / 16) > (double)(1 << 30))
        PG_FAIL(EMBER_ERR_UNSUPPORTED, "B * n_kv_heads * table_width * page_size > 2^34");
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return cuda_failed("no device", e);
    const size_t need = a.groups ? paged_decode_shared_ws(a.c, B, n_heads, a.n_groups, sms)
                                 : paged_decode_ws(a.c, B, n_heads, window, sinks, sms);
    if ((need && !workspace) || !aligned16(workspace))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "workspace must be given and 16-byte aligned");
    if (workspace_bytes < need) PG_FAIL(EMBER_ERR_CAPACITY, "workspace smaller than its query answers");
    a.q = static_cast<const uint16_t*>(q);
    a.ld_q = ld_q;
    a.B = B;
    a.NH = n_heads;
    a.seqs = seqs;
    a.lens = lens;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ld_out = ld_out;
    a.lse = lse;
    a.ws = static_cast<float*>(workspace);
    a.status = status;
    e = a.groups ? launch_paged_decode_shared(a, sms, (cudaStream_t)stream) : launch_paged_decode(a, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_failed("decode launch failed", e);
    return EMBER_OK;
}

}  // namespace

extern "C" {

ember_status ember_paged_append(const ember_paged_kv* kv, const void* q, const void* k, const void* v,
                                int32_t src_dtype, int64_t ld_q, int64_t ld_k, int64_t ld_v, int32_t n,
                                int32_t n_heads, const int32_t* seqs, const int32_t* positions,
                                const uint16_t* q_norm, const uint16_t* k_norm, float eps, const float* cos_t,
                                const float* sin_t, int32_t n_pos, void* q_out, int64_t ld_out, int32_t* status,
                                ember_stream_t stream) {
    PagedAppendArgs a{};
    ember_status st = check_cache(kv, a.c);
    if (st != EMBER_OK) return st;
    if (n < 0 || n > (1 << 30)) PG_FAIL(EMBER_ERR_INVALID_ARG, "bad number of tokens");
    if (src_dtype != EMBER_F32 && src_dtype != EMBER_BF16 && src_dtype != EMBER_F16)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "src_dtype must be EMBER_F32, EMBER_BF16 or EMBER_F16");
    if (!(eps >= 0.f)) PG_FAIL(EMBER_ERR_INVALID_ARG, "eps must be >= 0");
    if (n_pos <= 0) PG_FAIL(EMBER_ERR_INVALID_ARG, "n_pos must be > 0");
    if (n == 0) return EMBER_OK;
    if (!seqs || !positions) PG_FAIL(EMBER_ERR_INVALID_ARG, "seqs or positions is NULL");
    if ((st = check_words("seqs, positions and status", seqs, positions, status)) != EMBER_OK) return st;
    if (!cos_t || !sin_t || !aligned16(cos_t) || !aligned16(sin_t))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "cos_t and sin_t must be given and 16-byte aligned");
    if (!aligned16(q_norm) || !aligned16(k_norm))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "q_norm and k_norm must be 16-byte aligned");
    const int64_t kvd = (int64_t)kv->n_kv_heads * kv->head_dim;
    if (kvd > (1 << 20)) PG_FAIL(EMBER_ERR_UNSUPPORTED, "n_kv_heads * head_dim > 2^20");   // (as n_heads with q)
    if ((st = check_rows("k", k, ld_k, kvd)) != EMBER_OK) return st;
    if ((st = check_rows("v", v, ld_v, kvd)) != EMBER_OK) return st;
    if ((q == nullptr) != (q_out == nullptr)) PG_FAIL(EMBER_ERR_INVALID_ARG, "q and q_out go together");
    if (q) {
        if ((st = check_heads(kv, n_heads)) != EMBER_OK) return st;
        const int64_t qd = (int64_t)n_heads * kv->head_dim;
        if ((st = check_rows("q", q, ld_q, qd)) != EMBER_OK) return st;
        if ((st = check_rows("q_out", q_out, ld_out, qd)) != EMBER_OK) return st;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.src = src_dtype;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.n = n;
    a.NH = q ? n_heads : 0;
    a.seqs = seqs;
    a.positions = positions;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.cos_t = cos_t;
    a.sin_t = sin_t;
    a.n_pos = n_pos;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.ld_out = ld_out;
    a.status = status;
    const cudaError_t e = launch_paged_append(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_failed("append launch failed", e);
    return EMBER_OK;
}

size_t ember_paged_decode_workspace(const ember_paged_kv* kv, int32_t B, int32_t n_heads) {
    PagedView c;
    int sms = 0;
    if (B <= 0 || B > 65535 || check_cache(kv, c) != EMBER_OK || check_heads(kv, n_heads) != EMBER_OK) return 0;
    if (device_sms(&sms) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return paged_decode_ws(c, B, n_heads, 0, 0, sms);
}

ember_status ember_paged_decode(const ember_paged_kv* kv, const void* q, int64_t ld_q, int32_t B, int32_t n_heads,
                                const int32_t* seqs, const int32_t* lens, int32_t window, int32_t sinks, float scale,
                                void* out, int64_t ld_out, float* lse, void* workspace, size_t workspace_bytes,
                                int32_t* status, ember_stream_t stream) {
    PagedDecodeArgs a{};
    return decode(kv, a, q, ld_q, B, n_heads, seqs, lens, window, sinks, scale, out, ld_out, lse, workspace, workspace_bytes,
                  status, stream);
}

size_t ember_paged_decode_shared_workspace(const ember_paged_kv* kv, int32_t B, int32_t n_heads, int32_t n_groups) {
    PagedView c;
    int sms = 0;
    if (B <= 0 || B > 65535 || n_groups <= 0 || n_groups > B || check_cache(kv, c) != EMBER_OK || check_heads(kv, n_heads) != EMBER_OK)
        return 0;
    if (device_sms(&sms) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return paged_decode_shared_ws(c, B, n_heads, n_groups, sms);
}

ember_status ember_paged_decode_shared(const ember_paged_kv* kv, const void* q, int64_t ld_q, int32_t B, int32_t n_heads,
                                       const int32_t* seqs, const int32_t* lens, const int32_t* groups,
                                       const int32_t* shared, const int32_t* prefixes, int32_t n_groups, float scale,
                                       void* out, int64_t ld_out, float* lse, void* workspace, size_t workspace_bytes,
                                       int32_t* status, ember_stream_t stream) {
    PagedDecodeArgs a{};
    if (B > 0) {
        if (n_groups <= 0 || n_groups > B) PG_FAIL(EMBER_ERR_INVALID_ARG, "n_groups must be in [1, B]");
        if (!groups || !shared || !prefixes) PG_FAIL(EMBER_ERR_INVALID_ARG, "groups, shared or prefixes is NULL");
        const ember_status st = check_words("groups, shared and prefixes", groups, shared, prefixes);
        if (st != EMBER_OK) return st;
        a.groups = groups;
        a.shared = shared;
        a.prefixes = prefixes;
        a.n_groups = n_groups;
    }
    return decode(kv, a, q, ld_q, B, n_heads, seqs, lens, 0, 0, scale, out, ld_out, lse, workspace, workspace_bytes, status,
                  stream);
}

ember_status ember_paged_prefill(const ember_paged_kv* kv, const void* q, int64_t ld_q, int32_t n, int32_t B,
                                 int32_t n_heads, const int32_t* seqs, const int32_t* cu, const int32_t* lens,
                                 int32_t window, int32_t sinks, float scale, void* out, int64_t ld_out, float* lse,
                                 int32_t* status, ember_stream_t stream) {
    PagedPrefillArgs a{};
    ember_status st = check_cache(kv, a.c);
    if (st != EMBER_OK) return st;
    if (B < 0) PG_FAIL(EMBER_ERR_INVALID_ARG, "B < 0");
    st = check_attention(kv, B == 0 ? 0 : n, n_heads, q, ld_q, out, ld_out, lens, window, sinks, scale);
    if (st != EMBER_OK) return st;
    if (n == 0 || B == 0) return EMBER_OK;
    if (!cu) PG_FAIL(EMBER_ERR_INVALID_ARG, "cu is NULL");
    if (B > 65535 || kv->n_kv_heads > 65535) PG_FAIL(EMBER_ERR_UNSUPPORTED, "B > 65535 or n_kv_heads > 65535");
    if (!seqs && B > kv->n_seqs) PG_FAIL(EMBER_ERR_INVALID_ARG, "B > n_seqs without seqs");
    if ((st = check_words("seqs, cu, lens, lse and status", seqs, cu, lens, lse, status)) != EMBER_OK) return st;
    a.q = static_cast<const uint16_t*>(q);
    a.ld_q = ld_q;
    a.n = n;
    a.B = B;
    a.NH = n_heads;
    a.seqs = seqs;
    a.cu = cu;
    a.lens = lens;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ld_out = ld_out;
    a.lse = lse;
    a.status = status;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return cuda_failed("no device", e);
    e = launch_paged_prefill(a, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_failed("prefill launch failed", e);
    return EMBER_OK;
}

ember_status ember_paged_take_status(int32_t* status, int32_t* taken, ember_stream_t stream) {
    if (!status || !taken) PG_FAIL(EMBER_ERR_INVALID_ARG, "status or taken is NULL");
    const ember_status st = check_words("status and taken", status, taken);
    if (st != EMBER_OK) return st;
    const cudaError_t e = launch_k(k_take_status, dim3(1), dim3(1), 0, (cudaStream_t)stream, status, taken);
    if (e != cudaSuccess) return cuda_failed("status launch failed", e);
    return EMBER_OK;
}

}  // extern "C"
