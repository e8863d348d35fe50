// block_host.cuh -- host-side odds and ends of the operators around the
// convolution, and what their translation units call of one another.
#pragma once
#include <cuda_runtime.h>

#include "ccv3d.h"
#include "elem.cuh"

namespace ccv3d {

constexpr int kSms = 148;  // B200
typedef __nv_bfloat16 bf16;

inline ccv3d_status launched() { return cudaGetLastError() == cudaSuccess ? CCV3D_OK : CCV3D_ERR_CUDA; }
inline bool known(ccv3d_dtype t) { return t == CCV3D_BF16 || t == CCV3D_FP32; }
inline size_t size_of(ccv3d_dtype t) { return t == CCV3D_BF16 ? 2 : 4; }
inline long long up(long long a, long long b) { return (a + b - 1) / b; }

// Reads and clears this translation unit's status word after the work queued on
// `stream`; `v` keeps an error it already holds.
static inline cudaError_t take_status(int* v, cudaStream_t stream) {
    int mine = 0;
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&mine, g_block_status, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && mine != 0) {
        e = cudaMemcpyToSymbolAsync(g_block_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                                    stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    if (*v == 0) *v = mine;
    return e;
}

}  // namespace ccv3d
