// device_free.h -- giving a handle's device memory back.
#pragma once

#include <cuda_runtime.h>

// cudaFree() that a stream capture under way on this or another thread allows: handles are also
// closed by Python's garbage collector, at any time, and a plain cudaFree() would fail, keep the
// memory and end the capture with an error. (What is freed is not part of the capture.)
inline void kvr_device_free(void *p) {
    if (p == nullptr) return;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    cudaFree(p);
    if (relaxed) cudaThreadExchangeStreamCaptureMode(&mode);
    cudaGetLastError();
}
