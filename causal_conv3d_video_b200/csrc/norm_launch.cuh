// norm_launch.cuh -- launch shapes and launches of the norms (norm.cuh).  The
// templates are instantiated for bf16 in norm_bf16.cu and for fp32 in
// norm_fp32.cu, which compile beside one another.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_host.cuh"
#include "norm.cuh"

namespace ccv3d {

// Threads that share a row (0: the block's) and eight-channel units a thread.
// Within a warp the least idle of the shapes the kernels are built for (the
// decoder's widths, three times a power of two, leave no thread idle), of
// equals the one with the fewest threads a row (the fewest shuffles); single-channel loads (C not a
// multiple of 8) want 16 threads side by side.  Wider rows take a block each.
struct RowShape {
    int tpr, units, threads;
};
inline RowShape row_shape(int C, bool vec, int max_units) {
    const int n = (int)up(C, 8);
    RowShape best = {0, n > 512 ? 2 : 1, 0};
    best.threads = (int)up(up(n, best.units), 32) * 32;
    int cover = 1 << 30;
    for (int u = 1; u <= max_units; ++u)
        for (int tpr = vec ? 4 : 16; tpr <= 32; tpr *= 2)
            if (tpr * u >= n && tpr * u <= cover) {
                cover = tpr * u;
                best = {tpr, u, 0};
            }
    return best;
}

// Tiles of rows for the staged kernels: about `want` bytes of all tensors a
// stage, whole passes of the block, and no more rows than there are.  Long rows
// (fp32 at the decoder's wide layers) take blocks of fewer threads, so that a
// pass stays near that size too.
struct TileLaunch {
    TileShape t;
    int threads, blocks_per_sm;
    size_t smem;
};
inline TileLaunch tile_launch(const RowShape& r, int C, int e, long long rows, int tensors, int vectors,
                       int want, int threads_per_sm) {
    TileLaunch l;
    const int row = C * e;
    l.threads = kTileThreads;
    while (l.threads > 64 && (long long)tensors * row * (l.threads / r.tpr) > want) l.threads /= 2;
    const int pass = l.threads / r.tpr;
    long long passes =
        std::max<long long>(1, (long long)want * l.threads / kTileThreads / ((long long)tensors * row * pass));
    // (short calls: about four tiles a block, so that the blocks end together)
    passes = std::max<long long>(1, std::min(passes, rows / ((long long)pass * kSms * 8)));
    l.t.rows = (int)passes * pass;
    l.t.cap = (l.t.rows * row + 16 + 127) / 128 * 128;
    l.t.vec_len = r.tpr * r.units * 8;
    l.t.stages = (long long)tensors * l.t.cap * 3 <= 100 * 1024 ? 3 : 2;
    l.smem = (size_t)l.t.stages * tensors * l.t.cap + (size_t)vectors * l.t.vec_len * 4 + l.t.stages * 8;
    // (the column sums' buffer of the backward pass, a row a warp, is the idle ring)
    l.smem = std::max(l.smem, (size_t)(l.threads / 32) * C * 4);
    l.blocks_per_sm = (int)std::max<size_t>(
        1, std::min<size_t>(threads_per_sm / l.threads, 227 * 1024 / (l.smem + 1024)));
    return l;
}

// Dynamic shared memory of up to kBytes for a kernel, once per device.
template <auto* K, int kBytes = 200 * 1024>
void allow_smem() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
        cudaGetLastError();
        return;
    }
    if (done[dev].load(std::memory_order_acquire)) return;
    cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    cudaGetLastError();
    done[dev].store(true, std::memory_order_release);
}

// Blocks of K with that many threads (a multiple of 32, at most 512) that an SM
// holds at once: a grid that walks its rows takes exactly as many, since a part
// of a second wave would cost a whole one.
template <auto* K>
int blocks_an_sm(int threads) {
    static std::atomic<int> known[17];
    std::atomic<int>& k = known[threads / 32];
    int n = k.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, K, threads, 0) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        k.store(n, std::memory_order_relaxed);
    }
    return n;
}

template <typename T, bool V, bool B, int TPR, int NU>
void norm_fwd_run(const NormFwd& p, const RowShape& r, cudaStream_t st) {
    if constexpr (TPR == 0) {
        const int grid = (int)std::min<long long>(
            p.rows, (long long)kSms * blocks_an_sm<norm_fwd_rows<T, V, NU, B>>(r.threads));
        norm_fwd_rows<T, V, NU, B><<<grid, r.threads, 0, st>>>(p);
    } else {
        const TileLaunch l = tile_launch(r, p.C, sizeof(T), p.rows, B ? 2 : 1, 4, 20 * 1024, 768);
        const int grid = (int)std::min<long long>(up(p.rows, l.t.rows), kSms * l.blocks_per_sm);
        allow_smem<norm_fwd_tiles<T, V, TPR, NU, B>>();
        norm_fwd_tiles<T, V, TPR, NU, B><<<grid, l.threads, l.smem, st>>>(p, l.t);
    }
}

// Launch shape of the backward pass: blocks per gate group.
struct BwdShape {
    RowShape row;
    TileLaunch tile;
    long long groups, group_rows;
    int blocks_per_group;
    int sums;  // column sums the kernel takes: 2 or 4
};
inline BwdShape bwd_shape(const ccv3d_norm_desc* d, bool gated, int form) {
    BwdShape b = {};
    // (the wide-row kernel has one form for means and biases)
    b.row = row_shape(d->C, d->C % 8 == 0, 3);
    b.sums = form == kBwdBiased || (form != kBwdRms && b.row.tpr == 0) ? 4 : 2;
    b.groups = gated ? d->rows / d->gate_rows : 1;
    b.group_rows = gated ? d->gate_rows : d->rows;
    long long steps = b.group_rows, blocks;
    if (b.row.tpr == 0) {
        blocks = (long long)kSms * std::max(1, 512 / b.row.threads);
    } else {
        b.tile = tile_launch(b.row, d->C, (int)size_of(d->dtype), b.group_rows, 4, 3, 52 * 1024,
                             bwd_blocks(form, b.row.units) * kTileThreads);
        blocks = kSms * b.tile.blocks_per_sm;
        steps = up(b.group_rows, b.tile.t.rows);
    }
    b.blocks_per_group = (int)std::min(steps, std::max<long long>(1, blocks / b.groups));
    return b;
}

template <typename T, bool V, int F, int TPR, int NU>
void norm_bwd_run(const NormBwd& p, const BwdShape& s, cudaStream_t st) {
    const int grid = (int)(s.groups * s.blocks_per_group);
    if constexpr (TPR == 0) {
        norm_bwd_rows<T, V, NU, F != kBwdRms><<<grid, s.row.threads, 0, st>>>(p);
    } else {
        allow_smem<norm_bwd_tiles<T, V, TPR, NU, F>>();
        norm_bwd_tiles<T, V, TPR, NU, F><<<grid, s.tile.threads, s.tile.smem, st>>>(p, s.tile.t);
    }
}

// Calls f with the constants (TPR, units) of a shape.
template <bool V, typename F>
void with_shape(const RowShape& r, F&& f) {
    auto units = [&](auto tpr) {
        if (r.units == 1) f(tpr, std::integral_constant<int, 1>());
        else if (r.units == 2) f(tpr, std::integral_constant<int, 2>());
        else if constexpr (decltype(tpr)::value != 0) f(tpr, std::integral_constant<int, 3>());
    };
    switch (r.tpr) {
        case 4: if constexpr (V) units(std::integral_constant<int, 4>()); break;
        case 8: if constexpr (V) units(std::integral_constant<int, 8>()); break;
        case 16: units(std::integral_constant<int, 16>()); break;
        case 32: units(std::integral_constant<int, 32>()); break;
        default: units(std::integral_constant<int, 0>());
    }
}

template <typename T, bool V, bool B>
void norm_fwd_shape(const NormFwd& p, cudaStream_t st) {
    // few rows (under two an SM): a block each, without the ring's start-up
    // (one row of 768: 3.3 us against 5.7)
    const RowShape r = row_shape(p.C, V, p.rows < 2 * kSms ? 0 : 3);
    with_shape<V>(r, [&](auto tpr, auto nu) { norm_fwd_run<T, V, B, tpr(), nu()>(p, r, st); });
}
template <typename T, bool V, int F>
void norm_bwd_shape(const NormBwd& p, const BwdShape& s, cudaStream_t st) {
    with_shape<V>(s.row, [&](auto tpr, auto nu) {
        norm_bwd_run<T, V, F, tpr(), nu()>(p, s, st);
    });
}

template <typename T>
void norm_fwd_type(const NormFwd& p, cudaStream_t st) {
    if (p.C % 8 == 0)
        p.b != nullptr ? norm_fwd_shape<T, true, true>(p, st) : norm_fwd_shape<T, true, false>(p, st);
    else
        p.b != nullptr ? norm_fwd_shape<T, false, true>(p, st)
                       : norm_fwd_shape<T, false, false>(p, st);
}
template <typename T, bool V>
void norm_bwd_form(const NormBwd& p, const BwdShape& s, int form, cudaStream_t st) {
    if (form == kBwdRms) norm_bwd_shape<T, V, kBwdRms>(p, s, st);
    else if (form == kBwdMeans) norm_bwd_shape<T, V, kBwdMeans>(p, s, st);
    else norm_bwd_shape<T, V, kBwdBiased>(p, s, st);
}
template <typename T>
void norm_bwd_type(const NormBwd& p, const BwdShape& s, int form, cudaStream_t st) {
    if (p.C % 8 == 0) norm_bwd_form<T, true>(p, s, form, st);
    else norm_bwd_form<T, false>(p, s, form, st);
}

// The backward pass, and (f) the parameter gradients from its partials.
template <typename T>
void norm_backward_type(const NormBwd& p, const BwdShape& s, int form, const NormFin* f,
                        cudaStream_t st) {
    norm_bwd_type<T>(p, s, form, st);
    if (f == nullptr) return;
    const dim3 grid((unsigned)up(p.C, kFinCols), (unsigned)std::min<long long>(s.groups, 32768));
    const dim3 block(kFinCols, kFinRows);
    norm_fin_group_kernel<T><<<grid, block, 0, st>>>(*f);
    if (s.groups > 1) norm_fin_all_kernel<T><<<grid.x, block, 0, st>>>(*f);
}

void norm_forward_bf16(const NormFwd& p, cudaStream_t st);
void norm_forward_fp32(const NormFwd& p, cudaStream_t st);
void norm_backward_bf16(const NormBwd& p, const BwdShape& s, int form, const NormFin* f,
                        cudaStream_t st);
void norm_backward_fp32(const NormBwd& p, const BwdShape& s, int form, const NormFin* f,
                        cudaStream_t st);
cudaError_t norm_status_bf16(int* v, cudaStream_t st);
cudaError_t norm_status_fp32(int* v, cudaStream_t st);

}  // namespace ccv3d
