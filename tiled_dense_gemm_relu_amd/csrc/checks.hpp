// Argument checks and launches shared by the C entry points of gemm_relu_groups.h
// and gemm_relu_blocks.h.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_relu.h"
#include "device.hpp"
#include "kernel_table.hpp"

namespace gemm_relu_hip {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// One matrix (or stack of matrices) argument.
struct Span {
    const void* p;
    int64_t bytes;
};

inline bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Checks shared by all entry points: inputs and outputs present, aligned, and
// no output (or the workspace) sharing bytes with anything else.
inline int check_spans(const Span* in, int n_in, const Span* words, int n_words, const Span* out, int n_out)
{
    for (int i = 0; i < n_in; ++i) {
        if (in[i].bytes > 0 && !in[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (in[i].bytes > 0 && !aligned(in[i].p, 2)) return GEMM_RELU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n_words; ++i) {
        if (words[i].bytes > 0 && !words[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (words[i].bytes > 0 && !aligned(words[i].p, 4)) return GEMM_RELU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n_out; ++i) {
        if (out[i].bytes > 0 && !out[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (out[i].bytes > 0 && !aligned(out[i].p, 2)) return GEMM_RELU_ERR_MISALIGNED;
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return GEMM_RELU_ERR_ALIAS;
        for (int j = 0; j < n_words; ++j)
            if (overlaps(out[i].p, out[i].bytes, words[j].p, words[j].bytes)) return GEMM_RELU_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return GEMM_RELU_ERR_ALIAS;
    }
    return GEMM_RELU_OK;
}

inline int check_workspace(void* workspace, int64_t bytes, int64_t need)
{
    if (need == 0) return GEMM_RELU_OK;
    return !workspace || bytes < need || !aligned(workspace, 256) ? GEMM_RELU_ERR_WORKSPACE : GEMM_RELU_OK;
}

// Whether one launch can have that many workgroups: their threads are counted in 32 bits.
inline bool launchable(int64_t blocks, int threads) { return blocks <= int64_t(UINT32_MAX) / threads; }

inline int enqueue(const void* fn, dim3 grid, int threads, void** args, hipStream_t stream, size_t lds = 0)
{
    const hipError_t err = hipLaunchKernel(fn, grid, dim3((unsigned)threads), args, lds, stream);
    return err == hipSuccess ? GEMM_RELU_OK : GEMM_RELU_ERR_LAUNCH;
}

inline int zero_fill(void* p, int64_t halves, hipStream_t stream)
{
    if (halves <= 0) return GEMM_RELU_OK;
    size_t count = (size_t)halves;
    void* args[] = {&p, &count};
    return enqueue(zero_fill_kernel(), dim3((unsigned)std::min<int64_t>(ceil_div(halves, 256), 65536)), 256, args, stream);
}

}  // namespace gemm_relu_hip
