// rows_host.cu -- the C entry points of the operators on rows that need no cache: log
// probabilities, projections with adapters.  Argument checks before any device work, then
// one or two launches.
#include "entry.h"

using namespace ember;

extern "C" {

ember_status ember_logprobs(const void* logits, int32_t dtype, int32_t n, int32_t V, int64_t ldl, float temperature,
                            const int32_t* ids, int32_t top, float* logprob, int32_t* rank, float* entropy,
                            int32_t* top_ids, float* top_logprobs, ember_stream_t stream) {
    if (dtype != EMBER_F32 && dtype != EMBER_BF16 && dtype != EMBER_F16)
        PG_FAIL(EMBER_ERR_INVALID_ARG, "dtype must be EMBER_F32, EMBER_BF16 or EMBER_F16");
    if (n < 0 || n > (1 << 30)) PG_FAIL(EMBER_ERR_INVALID_ARG, "bad number of rows");
    if (V <= 0 || V > (1 << 30)) PG_FAIL(EMBER_ERR_INVALID_ARG, "V must be in [1, 2^30]");
    if (ldl < V) PG_FAIL(EMBER_ERR_INVALID_ARG, "ldl < V");
    if (!(temperature >= 1e-6f && temperature <= 1e6f)) PG_FAIL(EMBER_ERR_INVALID_ARG, "temperature must be in [1e-6, 1e6]");
    if (top < 0 || top > V) PG_FAIL(EMBER_ERR_INVALID_ARG, "top must be in [0, V]");
    if (top > EMBER_LOGPROBS_MAX_TOP) PG_FAIL(EMBER_ERR_UNSUPPORTED, "top > %d", EMBER_LOGPROBS_MAX_TOP);
    if (n == 0) return EMBER_OK;
    if (top > 0 && (!top_ids || !top_logprobs)) PG_FAIL(EMBER_ERR_INVALID_ARG, "top_ids or top_logprobs is NULL");
    if (!ids && (logprob || rank)) PG_FAIL(EMBER_ERR_INVALID_ARG, "logprob and rank need ids");
    if (!logits) PG_FAIL(EMBER_ERR_INVALID_ARG, "logits is NULL");
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == EMBER_F32 ? 4 : 2))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "logits must be aligned to their elements");
    const ember_status st = check_words("ids and outputs", ids, logprob, rank, entropy, top_ids, top_logprobs);
    if (st != EMBER_OK) return st;
    LogprobsArgs a{};
    a.logits = logits;
    a.dtype = dtype;
    a.n = n;
    a.V = V;
    a.ldl = ldl;
    a.t = temperature;
    a.ids = ids;
    a.top = top;
    a.logprob = logprob;
    a.rank = rank;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return cuda_failed("no device", e);
    e = launch_logprobs(a, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_failed("logprobs launch failed", e);
    return EMBER_OK;
}

size_t ember_adapter_workspace(int32_t n, int32_t rank) {
    if (n <= 0 || n > (1 << 30) || rank < 8 || rank > 128 || rank % 8) return 0;
    return adapter_ws(n, rank);
}

ember_status ember_adapter_project(const ember_adapters* ad, const void* x, int64_t ld_x, const void* w, const void* bias,
                                   int32_t dtype, int32_t n, int32_t N, int32_t K, const int32_t* ids, void* out,
                                   int32_t out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                   int32_t* status, ember_stream_t stream) {
    if (!ad) PG_FAIL(EMBER_ERR_INVALID_ARG, "adapters is NULL");
    if (dtype != EMBER_BF16 && dtype != EMBER_F16) PG_FAIL(EMBER_ERR_INVALID_ARG, "dtype must be EMBER_BF16 or EMBER_F16");
    if (out_dtype != dtype && out_dtype != EMBER_F32) PG_FAIL(EMBER_ERR_INVALID_ARG, "out_dtype must be dtype or EMBER_F32");
    if (n < 0 || n > (1 << 30)) PG_FAIL(EMBER_ERR_INVALID_ARG, "bad number of rows");
    if (N <= 0 || K <= 0 || N % 8 || K % 8) PG_FAIL(EMBER_ERR_INVALID_ARG, "N and K must be positive multiples of 8");
    if (N > (1 << 28) || K > (1 << 28)) PG_FAIL(EMBER_ERR_UNSUPPORTED, "N or K > 2^28");
    if (ad->n_adapters <= 0) PG_FAIL(EMBER_ERR_INVALID_ARG, "n_adapters must be > 0");
    if (ad->rank <= 0 || ad->rank % 8) PG_FAIL(EMBER_ERR_INVALID_ARG, "rank must be a positive multiple of 8");
    if (ad->rank > 128) PG_FAIL(EMBER_ERR_UNSUPPORTED, "rank > 128");
    if (n == 0) return EMBER_OK;
    if (!ad->a || !ad->b || !aligned16(ad->a) || !aligned16(ad->b))
        PG_FAIL(EMBER_ERR_INVALID_ARG, "a and b must be given and 16-byte aligned");
    if (!w || !aligned16(w) || !aligned16(bias)) PG_FAIL(EMBER_ERR_INVALID_ARG, "w must be given, w and bias 16-byte aligned");
    if (!ids) PG_FAIL(EMBER_ERR_INVALID_ARG, "ids is NULL");
    ember_status st = check_words("scale, ids and status", ad->scale, ids, status);
    if (st != EMBER_OK) return st;
    if ((st = check_rows("x", x, ld_x, K)) != EMBER_OK) return st;
    if ((st = check_rows("out", out, ld_out, N)) != EMBER_OK) return st;
    if (ld_x > (1ll << 36) || ld_out > (1ll << 36)) PG_FAIL(EMBER_ERR_UNSUPPORTED, "row stride of x or out > 2^36");
    if (!workspace || !aligned16(workspace)) PG_FAIL(EMBER_ERR_INVALID_ARG, "workspace must be given and 16-byte aligned");
    if (workspace_bytes < adapter_ws(n, ad->rank))
        PG_FAIL(EMBER_ERR_CAPACITY, "workspace smaller than ember_adapter_workspace");
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return cuda_failed("no device", e);
    AdapterArgs a{};
    a.ids = ids;
    a.n = n;
    a.N = N;
    a.K = K;
    a.R = ad->rank;
    a.n_adapters = ad->n_adapters;
    a.scale = ad->scale;
    a.bias = static_cast<const uint16_t*>(bias);
    a.x = static_cast<const uint16_t*>(x);
    a.ld_x = ld_x;
    a.w = static_cast<const uint16_t*>(w);
    a.lb = static_cast<const uint16_t*>(ad->b);
    a.t = static_cast<uint16_t*>(workspace);
    a.out = out;
    a.ld_out = ld_out;
    a.out_f32 = out_dtype == EMBER_F32;
    a.status = status;
    const AdapterPlan plan = adapter_plan(n, N, K, a.R, a.n_adapters, a.out_f32, sms);
    const AdapterRows rows{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), static_cast<const uint16_t*>(ad->a),
                           static_cast<const uint16_t*>(ad->b), ld_x};
    AdapterMaps maps;
    if (!adapter_maps(a, plan, rows, maps))
        PG_FAIL(EMBER_ERR_UNSUPPORTED, "the driver takes no tensor map of these sizes and strides");
    e = launch_adapter(maps, a, plan, rows, dtype == EMBER_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_failed("adapter launch failed", e);
    return EMBER_OK;
}

}  // extern "C"
