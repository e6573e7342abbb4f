// rows_host.cu -- the C entry points of the operators on rows that need no cache:
// log probabilities.  Argument checks before any device work, then one launch.
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

}  // extern "C"
