// block_ranges.cu -- the range checks of the operators around the convolution:
// kernels of the bounds-checked build (compile with -DCCV3D_CHECKED), launched
// with more blocks or gate rows than their parameters allow for.  The buffers
// behind the parameters are larger than those say, so that nothing is out of
// range in memory, whatever is checked.
#include "norm_launch.cuh"
#include "qcache.cuh"

using namespace ccv3d;

namespace {

// Runs f; the status its kernel recorded, or -1 after a CUDA error.
template <typename F>
int status_of(F&& f) {
    int zero = 0, status = 0;
    if (cudaMemcpyToSymbol(g_block_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    f();
    if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyFromSymbol(&status, g_block_status, sizeof(int)) != cudaSuccess)
        return -1;
    return status;
}

QCacheJob job(int C, int fmt, int px, int slots, int frames) {
    QCacheJob j = {};
    j.pixels = px;
    j.N = 1;
    j.C = C;
    j.groups = (C + 31) / 32;
    j.code_bytes = fmt == kQE2m1 ? (C + 1) / 2 : C;
    j.slots = slots;
    j.T = j.frames = frames;
    return j;
}

}  // namespace

#define API extern "C" __attribute__((visibility("default")))

// A cache of one batch entry, written or read as if it had `entries`.
API int cache_write(const void* x, void* codes, void* scales, int C, int fmt, int px, int slots,
                    int frames, int entries) {
    QCacheJob j = job(C, fmt, px, slots, frames);
    j.src = x;
    j.codes = static_cast<uint8_t*>(codes);
    j.scales = static_cast<uint8_t*>(scales);
    const dim3 grid((unsigned)up((long long)px * 4 * j.groups, kQThreads * kQUnits), frames * entries);
    return status_of([&] {
        if (C % 32 == 0) qcache_write_kernel<bf16_t, 8, true><<<grid, kQThreads>>>(j, fmt);
        else if (C % 8 == 0) qcache_write_kernel<bf16_t, 8, false><<<grid, kQThreads>>>(j, fmt);
        else qcache_write_kernel<bf16_t, 1, false><<<grid, kQThreads>>>(j, fmt);
    });
}
API int cache_read(void* out, void* codes, void* scales, int C, int fmt, int px, int slots,
                   int frames, int entries) {
    QCacheJob j = job(C, fmt, px, slots, frames);
    j.dst = out;
    j.codes = static_cast<uint8_t*>(codes);
    j.scales = static_cast<uint8_t*>(scales);
    const dim3 grid((unsigned)up((long long)px * ((C + 7) / 8), kQThreads * kQUnits), frames * entries);
    return status_of([&] {
        if (C % 32 == 0) qcache_read_kernel<bf16_t, 8, true><<<grid, kQThreads>>>(j, fmt);
        else if (C % 8 == 0) qcache_read_kernel<bf16_t, 8, false><<<grid, kQThreads>>>(j, fmt);
        else qcache_read_kernel<bf16_t, 1, false><<<grid, kQThreads>>>(j, fmt);
    });
}

// h_out = h + gate * b, y = rms(h_out); gate_rows need not divide the rows.
// C = 96 in tiles, C = 1024 a block a row.
API int norm_forward(const void* h, const void* b, const void* gate, void* h_out, void* y, int C,
                     long long rows, long long gate_rows) {
    const NormFwd p = {h, b, gate, nullptr, nullptr, nullptr, nullptr, h_out, y, rows, gate_rows, C,
                       kNormRms, kNormNone, kActNone, 1e-6f, 1.0f, 1.0f / C};
    const RowShape r = row_shape(C, true, 3);
    return status_of([&] {
        if (C == 96) norm_fwd_run<bf16_t, true, true, 4, 3>(p, r, nullptr);
        else norm_fwd_run<bf16_t, true, true, 0, 1>(p, r, nullptr);
    });
}
// Gradients, with blocks for `groups` gate groups where the parameters have one.
API int norm_backward(const void* h, const void* b, const void* gate, const void* dy,
                      const void* dh_out, void* dh, void* db, float* part, int C, long long rows,
                      int groups) {
    const NormBwd p = {h, b, gate, nullptr, nullptr, nullptr, nullptr, dy, dh_out, dh, db, part,
                       rows, rows, 1, 1, 1, C, kNormRms, kNormNone, kActNone, 1e-6f, 1.0f, 1.0f / C};
    const RowShape r = row_shape(C, true, 3);
    return status_of([&] {
        if (C == 96) {
            const TileLaunch l = tile_launch(r, C, 2, rows, 4, 3, 52 * 1024, 512);
            allow_smem<norm_bwd_tiles<bf16_t, true, 4, 3, kBwdRms>>();
            norm_bwd_tiles<bf16_t, true, 4, 3, kBwdRms><<<groups, l.threads, l.smem>>>(p, l.t);
        } else {
            norm_bwd_rows<bf16_t, true, 1, false><<<groups, r.threads>>>(p);
        }
    });
}
