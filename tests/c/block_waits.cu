// block_waits.cu -- the bounded waits of the operators around the convolution,
// made to run out: the kernels of the library, compiled with a short limit and
// with a bulk copy that leaves one of its calls out, so that the barrier it
// would have completed never does.  One block, so that calls come in order.
#define kWaitLimitNs kLibraryWaitLimitNs
#include "params.h"
#undef kWaitLimitNs
#define bulk_g2s library_bulk_g2s
#include "bulk.cuh"
#undef bulk_g2s

namespace ccv3d {
constexpr uint64_t kWaitLimitNs = 20000000ull;  // 20 ms
__device__ int g_left_out, g_issued;            // the copy left out (-1: none), copies asked for
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                         uint32_t bar) {
    if (atomicAdd(&g_issued, 1) != g_left_out) library_bulk_g2s(dst, src, bytes, bar);
}
}  // namespace ccv3d

#include "norm_launch.cuh"
#include "pointwise_simt.cuh"

using namespace ccv3d;

namespace {

// Runs f; returns the status the kernel recorded (-1: a CUDA error), and the copies it asked for.
template <typename F>
int with_copy_left_out(int which, int* issued, F&& f) {
    int zero = 0, status = 0;
    if (cudaMemcpyToSymbol(g_left_out, &which, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_issued, &zero, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_block_status, &zero, sizeof(int)) != cudaSuccess)
        return -1;
    f();
    if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyFromSymbol(issued, g_issued, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&status, g_block_status, sizeof(int)) != cudaSuccess)
        return -1;
    return status;
}

constexpr int kC = 96;  // channels: four threads a row, three units each

}  // namespace

#define API extern "C" __attribute__((visibility("default")))

// Rows of a tile and stages of the ring, forward or backward.
API void tile_shape(int backward, long long rows, int* tile_rows, int* stages) {
    const RowShape r = row_shape(kC, true, 3);
    const TileLaunch l = backward ? tile_launch(r, kC, 2, rows, 4, 3, 52 * 1024, 512)
                                  : tile_launch(r, kC, 2, rows, 2, 4, 20 * 1024, 768);
    *tile_rows = l.t.rows;
    *stages = l.t.stages;
}

// h_out = h + rms(b), y = rms(h_out)
API int norm_forward(const void* h, const void* b, void* h_out, void* y, long long rows, int left_out,
                     int* issued) {
    const NormFwd p = {h, b, nullptr, nullptr, nullptr, nullptr, nullptr, h_out, y, rows, rows, kC,
                       kNormRms, kNormRms, kActNone, 1e-6f, 1.0f, 1.0f / kC};
    const TileLaunch l = tile_launch(row_shape(kC, true, 3), kC, 2, rows, 2, 4, 20 * 1024, 768);
    return with_copy_left_out(left_out, issued, [&] {
        allow_smem<norm_fwd_tiles<bf16_t, true, 4, 3, true>>();
        norm_fwd_tiles<bf16_t, true, 4, 3, true><<<1, l.threads, l.smem>>>(p, l.t);
    });
}

API int norm_backward(const void* h, const void* b, const void* dy, const void* dh_out, void* dh,
                      void* db, float* part, long long rows, int left_out, int* issued) {
    const NormBwd p = {h, b, nullptr, nullptr, nullptr, nullptr, nullptr, dy, dh_out, dh, db, part,
                       rows, rows, 1, 1, 1, kC, kNormRms, kNormRms, kActNone, 1e-6f, 1.0f, 1.0f / kC};
    const TileLaunch l = tile_launch(row_shape(kC, true, 3), kC, 2, rows, 4, 3, 52 * 1024, 512);
    return with_copy_left_out(left_out, issued, [&] {
        allow_smem<norm_bwd_tiles<bf16_t, true, 4, 3, kBwdRms>>();
        norm_bwd_tiles<bf16_t, true, 4, 3, kBwdRms><<<1, l.threads, l.smem>>>(p, l.t);
    });
}

// out [M, 8] = x [M, K] w [8, K]^T, M <= 8
API int few_rows_product(const void* x, const void* w, void* out, int M, int K, int left_out,
                         int* issued) {
    const PwOut o = {nullptr, nullptr, out, nullptr, nullptr, M, 8, kActNone};
    return with_copy_left_out(left_out, issued, [&] {
        pw_rows_mma_kernel<1><<<1, 256>>>(static_cast<const bf16_t*>(x),
                                          static_cast<const bf16_t*>(w), K, o);
    });
}
