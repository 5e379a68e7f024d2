// wait_words.h -- the files that note bounded waits in a word of the device's (wait_status.cuh, internal).
#pragma once

#include <cuda_runtime.h>

namespace ss2d {

// Each adds to *out whether its word on the current device was set, and clears it if it was.  Waits for the stream.
cudaError_t matmul_fp8_wait_ran_out(bool *out, cudaStream_t s);
cudaError_t linear_chunked_wait_ran_out(bool *out, cudaStream_t s);
cudaError_t diag_wait_ran_out(bool *out, cudaStream_t s);

}  // namespace ss2d
