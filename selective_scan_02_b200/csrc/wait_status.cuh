// wait_status.cuh -- where the operators' kernels note that a bounded wait ran out: the error word of the call's workspace,
// and a word of this device's that outlives the workspace (one for each file that includes this).
#pragma once

#include <cuda_runtime.h>

#include "wait_words.h"

namespace ss2d {

static __device__ int g_wait_ran_out;

__device__ __forceinline__ void wait_ran_out(int *err)
{
    atomicExch(err, 1);
    atomicExch(&g_wait_ran_out, 1);
}

// Adds to *out whether the current device's word of this file was set, and clears it if it was.  Waits for the stream.
static cudaError_t take_wait_ran_out(bool *out, cudaStream_t s)
{
    int flag = 0;
    const int none = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&flag, g_wait_ran_out, sizeof(flag), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || flag == 0)
        return e;
    *out = true;
    e = cudaMemcpyToSymbolAsync(g_wait_ran_out, &none, sizeof(none), 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace ss2d
