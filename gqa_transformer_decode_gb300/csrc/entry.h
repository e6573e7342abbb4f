// entry.h -- what the operators' C entry points share: answering errors, and checks
// of arguments before any device work.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace ember {

#define PG_FAIL(st, ...) return set_error(st, __VA_ARGS__)

// Answers a CUDA error, and takes it off the thread's record: the next caller that
// looks there would take it for its own.
inline ember_status cuda_failed(const char* what, cudaError_t e) {
    cudaGetLastError();
    PG_FAIL(EMBER_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int PG_MAX_DEVICES = 64;

// SMs of the current device (asked once per device).
inline cudaError_t device_sms(int* sms) {
    static std::atomic<int> known[PG_MAX_DEVICES];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < PG_MAX_DEVICES && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < PG_MAX_DEVICES) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Index arrays, lse and the status word: loads and atomics of 4 bytes.
template <class... P>
ember_status check_words(const char* which, const P*... p) {
    if (((reinterpret_cast<uintptr_t>(p) | ...) & 3) != 0) PG_FAIL(EMBER_ERR_INVALID_ARG, "%s must be 4-byte aligned", which);
    return EMBER_OK;
}

inline ember_status check_rows(const char* what, const void* p, int64_t ld, int64_t cols) {
    if (!p) PG_FAIL(EMBER_ERR_INVALID_ARG, "%s is NULL", what);
    if (!aligned16(p)) PG_FAIL(EMBER_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
    if (ld < cols || ld % 8) PG_FAIL(EMBER_ERR_INVALID_ARG, "row stride of %s must be a multiple of 8 and cover a row", what);
    return EMBER_OK;
}

}  // namespace ember
