// ccv3d_block.cu -- C ABI of the operators around the convolution: block norms
// (ccv3d_norm_*), the 1x1x1 product (ccv3d_pointwise_*) and the quantised ring
// cache (ccv3d_qcache_*).  Argument checks, launch shapes and launches; the
// kernels and the mathematics are in the headers (the norms' launches in
// norm_launch.cuh, compiled for each type in norm_bf16.cu and norm_fp32.cu).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "ccv3d.h"
#include "block_host.cuh"
#include "elem.cuh"
#include "norm_launch.cuh"
#include "pointwise_simt.cuh"
#include "pointwise_tc.cuh"
#include "qcache.cuh"

using namespace ccv3d;

namespace {

// The buffers of a call: every one 16-byte aligned, no written one
// overlapping another.  NULL and empty buffers are left out.
struct Buffers {
    struct One { uintptr_t at; size_t bytes; bool written; };
    One b[24];
    int n = 0;
    bool aligned = true, alias = false;
    void add(const void* p, size_t bytes, bool written) {
        if (p == nullptr || bytes == 0) return;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (a & 15u) aligned = false;
        for (int i = 0; i < n; ++i)
            if ((written || b[i].written) && a < b[i].at + b[i].bytes && b[i].at < a + bytes)
                alias = true;
        b[n++] = {a, bytes, written};
    }
    void in(const void* p, size_t bytes) { add(p, bytes, false); }
    void out(const void* p, size_t bytes) { add(p, bytes, true); }
    ccv3d_status check() const {
        return !aligned ? CCV3D_ERR_ALIGNMENT : (alias ? CCV3D_ERR_ALIAS : CCV3D_OK);
    }
};

// ------------------------------------------------------------------- norms
ccv3d_status check_norm(const ccv3d_norm_desc* d) {
    if (d == nullptr) return CCV3D_ERR_INVALID;
    if (!known(d->dtype) || d->pre < CCV3D_NORM_NONE || d->pre > CCV3D_NORM_LAYER ||
        d->post < CCV3D_NORM_NONE || d->post > CCV3D_NORM_LAYER || d->act < CCV3D_ACT_NONE ||
        d->act > CCV3D_ACT_GELU)
        return CCV3D_ERR_UNSUPPORTED;
    if (d->rows < 0 || d->C < 1 || !(d->eps > 0.0f) || !std::isfinite(d->eps) ||
        !std::isfinite(d->scale))
        return CCV3D_ERR_INVALID;
    if (d->C > CCV3D_NORM_MAX_C || d->rows > (1LL << 46) / d->C) return CCV3D_ERR_UNSUPPORTED;
    return CCV3D_OK;
}

bool gate_fits(const ccv3d_norm_desc* d, const void* gate) {
    return gate == nullptr || (d->gate_rows >= 1 && d->rows % d->gate_rows == 0);
}

// --------------------------------------------------------------- pointwise
ccv3d_status check_pointwise(const ccv3d_pointwise_desc* d) {
    if (d == nullptr) return CCV3D_ERR_INVALID;
    if (!known(d->dtype) || d->act < CCV3D_ACT_NONE || d->act > CCV3D_ACT_GELU)
        return CCV3D_ERR_UNSUPPORTED;
    if (d->pixels < 0 || d->Cin < 1 || d->Cout < 1) return CCV3D_ERR_INVALID;
    if (d->pixels > 0x7fffffffLL - 256 || d->Cin > 65536 || d->Cout > 65536)
        return CCV3D_ERR_UNSUPPORTED;
    return CCV3D_OK;
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// Shape of a product on FFMA: the tile (128 x 128, 64 x 64, 128 x 32 or 32 x 128)
// and the splits of the reduction with the shortest time on the fullest SM
// (blocks on one SM share its time), in FMAs at about 83 a cycle and SM for the
// largest tile; the others' count 1.5 times (half the FMAs per shared-memory
// read).  Splits are of at least 8 steps of 16; joining them is a launch and two
// trips of the partials.
struct SimtShape {
    int tm, tn, splits;
    long long tiles, k_per_split;
};
SimtShape simt_shape(long long M, long long N, long long K) {
    constexpr int kTiles[4][2] = {{128, 128}, {64, 64}, {128, 32}, {32, 128}};
    SimtShape best = {};
    double cost = 1e300;
    for (const auto& t : kTiles) {
        const long long tiles = up(M, t[0]) * up(N, t[1]);
        // (the last two: a block an SM, and two)
        const int fill = (int)std::max<long long>(1, kSms / tiles);
        for (const int want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 256, 512, fill, 2 * fill}) {
            if (want > 1 && (want > up(K, 128) || tiles * want > 8 * kSms)) continue;
            const long long per = up(up(K, want), kPwK) * kPwK;
            const int splits = (int)std::max<long long>(1, up(K, per));
            double c = std::ceil((double)tiles * splits / kSms) * (double)t[0] * t[1] * (per + 32) *
                       (t[0] == 128 && t[1] == 128 ? 1.0 : 1.5);
            if (splits > 1) c += 83.0 * (4000.0 + (double)splits * M * N * 8.0 / 3500.0);
            if (c < cost) {
                cost = c;
                best = {t[0], t[1], splits, tiles, per};
            }
        }
    }
    return best;
}
size_t simt_ws(long long M, long long N, long long K) {
    const int s = simt_shape(M, N, K).splits;
    return s > 1 ? pad256((size_t)s * M * up(N, 4) * 4 * 4) : 0;
}

// Column sums of dP: chunks of rows, one row of partials each.
struct SumShape {
    int tpr, col_blocks;
    long long chunk, chunks;
};
SumShape sum_shape(long long M, int N) {
    SumShape s;
    const int n = (int)up(N, 8);
    s.tpr = 4;
    while (s.tpr < 32 && s.tpr < n) s.tpr *= 2;
    s.col_blocks = (int)up(n, s.tpr);
    const long long rows = 256 / s.tpr;  // side by side in a block
    const long long want = std::max<long long>(1, kSms * 8LL / s.col_blocks);
    s.chunk = std::max(up(M, want), rows * 4);
    s.chunks = std::max<long long>(1, up(M, s.chunk));
    return s;
}

// ---- tensor-core products
// Shape of D(m, n) = sum over K on pw_tc_kernel.
struct TcShape {
    int BN, tiles_m, tiles_n, kblocks, splits, kb_per_split, stages, chunk, n_bufs, n_pres, res_bufs,
        n_acc, tmem_cols, ldp;
    size_t smem, ws;
};

// Tile width and splits by the cost of the slowest pair, in SM cycles: a 64-deep
// step of a 256 x BN tile takes about max(500, 2.64 BN), a tile's epilogue about
// 12 BN beside the next tile's steps, a split reduction's partials two trips at
// 3500 bytes a cycle and a launch of 4000.  Measured steps, one tile on each of
// the 74 pairs, operands in L2: BN 32 438 cycles, 64 491, 96 498, 128 505, 160
// 531, 192 533, 224 574, 256 658.  (Calls of one to four rows of tiles take about
// 450 too, so the floor is not the pairs' share of L2.)
TcShape tc_shape(long long M, int N, long long K, bool b_mn, bool res, bool pre) {
    TcShape s = {};
    s.tiles_m = (int)up(M, kPtRows);
    s.kblocks = (int)up(K, kPtK);
    s.ldp = (int)up(N, 4) * 4;
    double best = 1e300;
    const int pairs = kSms / 2;
    for (int bn = 32; bn <= 256; bn += 32) {
        if (bn > 32 && bn - 32 >= N) break;
        const int tn = (int)up(N, bn);
        const long long tiles = (long long)s.tiles_m * tn;
        for (int want = 1; want <= 128; want *= 2) {
            const int per = (int)up(s.kblocks, want), splits = (int)up(s.kblocks, per);
            if (want > 1 && (per < 4 || tiles * want / 2 >= pairs)) break;
            const double step = std::max(500.0, 2.64 * bn), epi = 12.0 * bn;
            const double waves = (double)up(tiles * splits, pairs);
            double cost = waves * std::max(per * step, epi) + std::min(per * step, epi);
            if (splits > 1) cost += 4000.0 + (double)splits * M * N * 8.0 / 3500.0;
            if (cost < best * 0.999) {
                best = cost;
                s.BN = bn;
                s.tiles_n = tn;
                s.splits = splits;
                s.kb_per_split = per;
            }
        }
    }
    const bool parts = s.splits > 1;
    // staging: two buffers in turn a warp, for out and for pre; with pre and a
    // residual 32-column chunks, so that four operand stages are left
    // (partials: 32 fp32 columns, as many bytes as 64 of bf16)
    s.chunk = !parts && (s.BN % 64 != 0 || (res && pre)) ? 32 : 64;
    s.n_bufs = 2;
    s.n_pres = parts || !pre ? 0 : 2;
    s.res_bufs = parts || !res || N % 8 != 0 ? 0 : kPtResBufs;
    s.stages = 10;
    while (s.stages > 2 &&
           pt_smem(b_mn, s.BN, s.stages, s.chunk, s.n_bufs + s.n_pres, s.res_bufs) > 227 * 1024)
        --s.stages;
    s.smem = pt_smem(b_mn, s.BN, s.stages, s.chunk, s.n_bufs + s.n_pres, s.res_bufs);
    s.n_acc = std::min(kPtAccs, 512 / s.BN);
    s.tmem_cols = 32;
    while (s.tmem_cols < s.n_acc * s.BN) s.tmem_cols *= 2;
    s.ws = parts ? pad256((size_t)s.splits * M * s.ldp * 4) : 0;
    return s;
}

// Bytes of an operand of `rows` rows copied to rows of a multiple of 8 (0:
// its rows are that already).
size_t pack_bytes(long long rows, int C) {
    return C % 8 == 0 ? 0 : pad256((size_t)rows * up(C, 8) * 8 * 2);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// Map of a [rows][ld] bf16 matrix in boxes of `inner` x `outer` elements;
// elements past `cols` (<= ld) of a row are read as 0 and not written.
bool encode2d(CUtensorMap* m, const void* base, long long rows, int cols, int ld, int inner,
              int outer) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)inner, (cuuint32_t)outer}, es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                       strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of fp32 partials [splits][M][ldp] in boxes of 32 x 32 of one split.
bool encode_partials(CUtensorMap* m, float* base, int splits, long long M, int ldp) {
    const cuuint64_t dims[3] = {(cuuint64_t)ldp, (cuuint64_t)M, (cuuint64_t)splits};
    const cuuint64_t strides[2] = {(cuuint64_t)ldp * 4, (cuuint64_t)M * ldp * 4};
    const cuuint32_t box[3] = {32, 32, 1}, es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void set_tc_attrs() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
        cudaGetLastError();
        return;
    }
    if (done[dev].load(std::memory_order_acquire)) return;
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaFuncSetAttribute(pw_tc_kernel<false, false>, attr, 227 * 1024);
    cudaFuncSetAttribute(pw_tc_kernel<false, true>, attr, 227 * 1024);
    cudaFuncSetAttribute(pw_tc_kernel<true, true>, attr, 227 * 1024);
    cudaGetLastError();
    done[dev].store(true, std::memory_order_release);
}

const void* packed(const void* src, long long rows, int C, uint8_t*& at, cudaStream_t st) {
    if (C % 8 == 0) return src;
    const int Cp = (int)up(C, 8) * 8;
    bf16* dst = reinterpret_cast<bf16*>(at);
    at += pack_bytes(rows, C);
    const long long n = rows * (Cp / 8);
    pw_pack_kernel<<<(unsigned)std::min<long long>(up(n, 256), kSms * 16LL), 256, 0, st>>>(
        static_cast<const bf16*>(src), dst, rows, C, Cp);
    return dst;
}

// D = sum_k A B with the forward epilogue `o` (no bias, residual or pre for
// gradients).  A: [M][K] rows of lda, or (A_MN) [K][M]; B likewise with N.
template <bool A_MN, bool B_MN>
ccv3d_status run_tc(const void* A, int lda, const void* B, int ldb, long long M, int N,
                    long long K, const PwOut& o, float* partial, cudaStream_t st) {
    if (encode_fn() == nullptr) return CCV3D_ERR_CUDA;
    const TcShape s = tc_shape(M, N, K, B_MN, o.residual != nullptr, o.pre != nullptr);
    PtParams p;
    std::memset(&p, 0, sizeof(p));
    const bool direct = N % 8 != 0;
    bool ok = A_MN ? encode2d(&p.tm_a, A, K, (int)M, lda, 64, 64)
                   : encode2d(&p.tm_a, A, M, (int)K, lda, 64, 128);
    ok = ok && (B_MN ? encode2d(&p.tm_b, B, K, N, ldb, 64, 64)
                     : encode2d(&p.tm_b, B, N, (int)K, ldb, 64, s.BN / 2));
    const int ch = s.chunk;
    if (s.splits > 1) {
        p.partial = true;
        ok = ok && encode_partials(&p.tm_out, partial, s.splits, M, s.ldp);
    } else {
        p.bias = static_cast<const bf16*>(o.bias);
        p.residual = static_cast<const bf16*>(o.residual);
        p.out = static_cast<bf16*>(o.out);
        p.pre = static_cast<bf16*>(o.pre);
        p.act = o.act;
        p.direct = direct;
        if (!direct) {
            ok = ok && encode2d(&p.tm_out, o.out, M, N, N, ch, 32);
            if (o.residual != nullptr) ok = ok && encode2d(&p.tm_res, o.residual, M, N, N, ch, 128);
            if (o.pre != nullptr) ok = ok && encode2d(&p.tm_pre, o.pre, M, N, N, ch, 32);
        }
    }
    if (!ok) return CCV3D_ERR_CUDA;
    p.M = M;
    p.N = N;
    p.tiles_m = s.tiles_m;
    p.tiles_n = s.tiles_n;
    p.BN = s.BN;
    p.kblocks = s.kblocks;
    p.splits = s.splits;
    p.kb_per_split = s.kb_per_split;
    p.stages = s.stages;
    p.chunk = s.chunk;
    p.n_acc = s.n_acc;
    p.n_bufs = s.n_bufs;
    p.n_pres = s.n_pres;
    p.res_bufs = s.res_bufs;
    p.tmem_cols = s.tmem_cols;
    p.wait_limit_ns = kWaitLimitNs;
    set_tc_attrs();
    const long long total = (long long)s.tiles_m * s.tiles_n * s.splits;
    if (total > 0x7fffffffLL / 8) return CCV3D_ERR_UNSUPPORTED;
    const int pairs = (int)std::min<long long>(total, kSms / 2), grid = 2 * pairs;
    p.step_n = pairs % s.tiles_n;
    p.step_m = pairs / s.tiles_n % s.tiles_m;
    p.step_s = pairs / s.tiles_n / s.tiles_m;
    pw_tc_kernel<A_MN, B_MN><<<grid, kPtThreads, s.smem, st>>>(p);
    if (s.splits > 1) {
        const long long blocks = std::min<long long>(up(M * (s.ldp / 4), 256), kSms * 16LL);
        pw_join_kernel<bf16><<<(unsigned)blocks, 256, 0, st>>>(partial, s.splits, s.ldp, o);
    }
    return launched();
}

// Rows up to which the warp-level kernel takes a bf16 product whose Cin is a
// multiple of 8.  Us of 16 rows on it and of 17 on the tensor-core kernel with its
// reduction split: 384 -> 1152 3.1 and 6.0, 1024 -> 4096 4.7 and 10.0, 4096 ->
// 1024 7.8 and 9.9, 4096 -> 4096 12.8 and 16.9, 2048 -> 8192 13.5 and 16.6, 8192
// -> 2048 17.4 and 17.4; 32 rows on it take 23 at 4096 x 4096.
constexpr int kMmaRows = 16;
bool few_rows(const ccv3d_pointwise_desc* d) {
    return d->pixels <= kPwFewRows ||
           (d->dtype == CCV3D_BF16 && d->Cin % 8 == 0 && d->pixels <= kMmaRows);
}

// Workspaces, in the order of their parts.  Forward: packed x and w, partials.
struct FwdWs {
    size_t packs, parts, total;
};
FwdWs forward_ws(const ccv3d_pointwise_desc* d) {
    FwdWs w = {};
    const long long M = d->pixels;
    if (few_rows(d)) return w;
    if (d->dtype == CCV3D_FP32) {
        w.parts = simt_ws(M, d->Cout, d->Cin);
    } else {
        w.packs = pack_bytes(M, d->Cin) + pack_bytes(d->Cout, d->Cin);
        // (a residual or pre changes the buffers, not the splits)
        w.parts = tc_shape(M, d->Cout, d->Cin, false, false, false).ws;
    }
    w.total = w.packs + w.parts;
    return w;
}

// Backward: dP, column sums, packed x and w, partials (of dx, then of dw).
struct BwdWs {
    size_t dp, sums, packs, parts, total;
};
bool makes_dp(const ccv3d_pointwise_desc* d) {
    return d->act != CCV3D_ACT_NONE || (d->dtype == CCV3D_BF16 && d->Cout % 8 != 0);
}
// Elements of a row of dP.
int dp_row(const ccv3d_pointwise_desc* d) {
    return d->dtype == CCV3D_BF16 ? (int)up(d->Cout, 8) * 8 : d->Cout;
}
BwdWs backward_ws(const ccv3d_pointwise_desc* d) {
    BwdWs w = {};
    const long long M = d->pixels;
    w.dp = makes_dp(d) ? pad256((size_t)M * dp_row(d) * size_of(d->dtype)) : 0;
    w.sums = pad256((size_t)sum_shape(M, d->Cout).chunks * d->Cout * 4);
    if (d->dtype == CCV3D_FP32) {
        w.parts = std::max(simt_ws(M, d->Cin, d->Cout), simt_ws(d->Cout, d->Cin, M));
    } else {
        w.packs = pack_bytes(M, d->Cin) + pack_bytes(d->Cout, d->Cin);
        w.parts = std::max(tc_shape(M, d->Cin, d->Cout, true, false, false).ws,
                           tc_shape(d->Cout, d->Cin, M, true, false, false).ws);
    }
    w.total = w.dp + w.sums + w.packs + w.parts;
    return w;
}

// D = A B^T on FFMA, fp32.
template <bool AK, bool BK>
ccv3d_status run_simt(const void* A, const void* B, long long lda, long long ldb, long long M,
                      int N, long long K, PwOut o, float* partial, cudaStream_t st) {
    PwSimt p;
    p.A = A;
    p.B = B;
    p.sam = AK ? lda : 1;
    p.sak = AK ? 1 : lda;
    p.sbn = BK ? ldb : 1;
    p.sbk = BK ? 1 : ldb;
    p.M = M;
    p.N = N;
    p.K = K;
    p.vec = lda % 4 == 0 && ldb % 4 == 0;
    const SimtShape s = simt_shape(M, N, K);
    p.splits = s.splits;
    p.k_per_split = s.k_per_split;
    p.ldp = (int)up(N, 4) * 4;
    p.a_elems = (AK ? M : K) * lda;
    p.b_elems = (BK ? N : K) * ldb;
    p.o = o;
    p.o.partial = p.splits > 1 ? partial : nullptr;
    if (s.tiles > 0x7fffffffLL) return CCV3D_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)s.tiles, 1, p.splits);
    // more than one chain: room for the sums of whole ones
    const bool chains = std::min(K, s.k_per_split) > kPwChain;
    auto run = [&](auto tm, auto tn) {
        if (chains) {
            allow_smem<pw_simt_kernel<float, AK, BK, tm(), tn(), true>, tm() * tn() * 4>();
            pw_simt_kernel<float, AK, BK, tm(), tn(), true><<<grid, 256, tm() * tn() * 4, st>>>(p);
        } else {
            pw_simt_kernel<float, AK, BK, tm(), tn(), false><<<grid, 256, 0, st>>>(p);
        }
    };
    const std::integral_constant<int, 128> i128;
    const std::integral_constant<int, 64> i64;
    const std::integral_constant<int, 32> i32;
    if (s.tm == 32) run(i32, i128);
    else if (s.tn == 128) run(i128, i128);
    else if (s.tn == 64) run(i64, i64);
    else run(i128, i32);
    if (p.splits > 1) {
        const long long blocks = std::min<long long>(up(M * (p.ldp / 4), 256), kSms * 16LL);
        pw_join_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(partial, p.splits, p.ldp, o);
    }
    return launched();
}

template <typename T, int MR, int CPW>
void run_rows(const T* x, const T* w, int K, const PwOut& o, cudaStream_t st) {
    const unsigned grid = (unsigned)up(o.N, CPW);
    // (bf16 rows of multiples of 8 are pw_rows_mma_kernel's)
    if constexpr (sizeof(T) == 4) {
        if (K % 8 == 0) {
            pw_rows_kernel<T, MR, CPW, true><<<grid, 256, 0, st>>>(x, w, K, o);
            return;
        }
    }
    pw_rows_kernel<T, MR, CPW, false><<<grid, 256, 0, st>>>(x, w, K, o);
}

template <typename T>
ccv3d_status forward_type(const ccv3d_pointwise_desc* d, const void* x, const void* w,
                          const PwOut& o, void* ws, cudaStream_t st) {
    const long long M = d->pixels;
    if (few_rows(d)) {
        const T *xt = static_cast<const T*>(x), *wt = static_cast<const T*>(w);
        if constexpr (sizeof(T) == 2) {
            if (d->Cin % 8 == 0) {
                const unsigned grid = (unsigned)up(o.N, 8);
                if (M <= 8) pw_rows_mma_kernel<1><<<grid, 256, 0, st>>>(xt, wt, d->Cin, o);
                else pw_rows_mma_kernel<2><<<grid, 256, 0, st>>>(xt, wt, d->Cin, o);
                return launched();
            }
        }
        if (M == 1) run_rows<T, 1, 1>(xt, wt, d->Cin, o, st);
        else if (M <= 4) run_rows<T, 4, 2>(xt, wt, d->Cin, o, st);
        else run_rows<T, 8, 2>(xt, wt, d->Cin, o, st);
        return launched();
    }
    if constexpr (sizeof(T) == 4) {
        return run_simt<true, true>(x, w, d->Cin, d->Cin, d->pixels, d->Cout, d->Cin, o,
                                    static_cast<float*>(ws), st);
    } else {
        uint8_t* at = static_cast<uint8_t*>(ws);
        const void* A = packed(x, d->pixels, d->Cin, at, st);
        const void* B = packed(w, d->Cout, d->Cin, at, st);
        const int ld = (int)up(d->Cin, 8) * 8;
        return run_tc<false, false>(A, ld, B, ld, d->pixels, d->Cout, d->Cin, o,
                                    reinterpret_cast<float*>(at), st);
    }
}

template <typename T>
ccv3d_status backward_type(const ccv3d_pointwise_desc* d, const void* x, const void* w,
                           const void* pre, const void* dout, void* dx, void* dw, void* dbias,
                           void* ws, cudaStream_t st) {
    const long long M = d->pixels;
    const int K = d->Cin, N = d->Cout, ldp = dp_row(d);
    const BwdWs b = backward_ws(d);
    uint8_t* at = static_cast<uint8_t*>(ws);
    T* dp = reinterpret_cast<T*>(at);
    float* sums = reinterpret_cast<float*>(at + b.dp);
    uint8_t* packs = at + b.dp + b.sums;
    float* parts = reinterpret_cast<float*>(packs + b.packs);
    const bool make = makes_dp(d) && (dx != nullptr || dw != nullptr);
    if (make || dbias != nullptr) {
        const SumShape s = sum_shape(M, N);
        const dim3 grid(s.col_blocks, (unsigned)s.chunks);
        const T* tp = static_cast<const T*>(pre);
        const T* td = static_cast<const T*>(dout);
        float* cs = dbias != nullptr ? sums : nullptr;
        T* tdp = make ? dp : nullptr;
        if (N % 8 == 0)
            pw_dact_kernel<T, true><<<grid, 256, 0, st>>>(tp, td, tdp, cs, M, N, ldp, d->act,
                                                         s.tpr, s.chunk);
        else
            pw_dact_kernel<T, false><<<grid, 256, 0, st>>>(tp, td, tdp, cs, M, N, ldp, d->act,
                                                          s.tpr, s.chunk);
        if (dbias != nullptr)
            pw_colsum_kernel<T><<<(unsigned)up(N, 32), dim3(32, 32), 0, st>>>(
                sums, (int)s.chunks, N, static_cast<T*>(dbias));
        if (launched() != CCV3D_OK) return CCV3D_ERR_CUDA;
    }
    const void* dP = make ? dp : dout;
    PwOut o = {};
    o.act = CCV3D_ACT_NONE;
    ccv3d_status r = CCV3D_OK;
    if (dx != nullptr) {
        o.out = dx;
        o.M = M;
        o.N = K;
        if constexpr (sizeof(T) == 4) {
            r = run_simt<true, false>(dP, w, N, K, M, K, N, o, parts, st);
        } else {
            const void* B = packed(w, N, K, packs, st);
            r = run_tc<false, true>(dP, ldp, B, (int)up(K, 8) * 8, M, K, N, o, parts, st);
        }
    }
    if (r == CCV3D_OK && dw != nullptr) {
        o.out = dw;
        o.M = N;
        o.N = K;
        if constexpr (sizeof(T) == 4) {
            r = run_simt<false, false>(dP, x, N, K, N, K, M, o, parts, st);
        } else {
            const void* B = packed(x, M, K, packs, st);
            r = run_tc<true, true>(dP, ldp, B, (int)up(K, 8) * 8, N, K, M, o, parts, st);
        }
    }
    return r;
}

// ------------------------------------------------------------ quantised cache
ccv3d_status check_qcache(const ccv3d_qcache_desc* d) {
    if (d == nullptr) return CCV3D_ERR_INVALID;
    if (!known(d->dtype) || d->format < CCV3D_Q_INT8 || d->format > CCV3D_Q_E2M1)
        return CCV3D_ERR_UNSUPPORTED;
    if (d->N < 0 || d->C < 1 || d->H < 1 || d->W < 1 || d->ring_slots < 1)
        return CCV3D_ERR_INVALID;
    if (d->C > 65536 || (long long)d->H * d->W > 0x7fffffffLL ||
        (long long)d->N * d->ring_slots > 0x7fffffffLL ||
        (double)d->N * d->ring_slots * d->H * d->W * d->C > 1e13)
        return CCV3D_ERR_UNSUPPORTED;
    return CCV3D_OK;
}

QCacheJob qcache_job(const ccv3d_qcache_desc* d) {
    QCacheJob j = {};
    j.pixels = (long long)d->H * d->W;
    j.N = d->N;
    j.C = d->C;
    j.groups = (d->C + kQGroup - 1) / kQGroup;
    j.code_bytes = d->format == CCV3D_Q_E2M1 ? (d->C + 1) / 2 : d->C;
    j.slots = d->ring_slots;
    return j;
}

// Whole frames on the grid's second axis (at most CCV3D_QCACHE_MAX_FRAMES of them).
dim3 qcache_grid(const QCacheJob& j, long long threads_a_pixel) {
    return dim3((unsigned)up(j.pixels * threads_a_pixel, kQThreads * kQUnits),
                (unsigned)(j.N * j.frames));
}

template <typename T>
void qcache_write_run(const QCacheJob& j, int fmt, cudaStream_t st) {
    const dim3 grid = qcache_grid(j, 4LL * j.groups);
    if (j.C % 32 == 0) qcache_write_kernel<T, 8, true><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 8 == 0) qcache_write_kernel<T, 8, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 4 == 0) qcache_write_kernel<T, 4, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 2 == 0) qcache_write_kernel<T, 2, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else qcache_write_kernel<T, 1, false><<<grid, kQThreads, 0, st>>>(j, fmt);
}
template <typename T>
void qcache_read_run(const QCacheJob& j, int fmt, cudaStream_t st) {
    const dim3 grid = qcache_grid(j, up(j.C, 8));
    if (j.C % 32 == 0) qcache_read_kernel<T, 8, true><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 8 == 0) qcache_read_kernel<T, 8, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 4 == 0) qcache_read_kernel<T, 4, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else if (j.C % 2 == 0) qcache_read_kernel<T, 2, false><<<grid, kQThreads, 0, st>>>(j, fmt);
    else qcache_read_kernel<T, 1, false><<<grid, kQThreads, 0, st>>>(j, fmt);
}

}  // namespace

extern "C" {

ccv3d_status ccv3d_norm_forward(const ccv3d_norm_desc* d, const void* h, const void* b,
                                const void* gate, const void* post_w, const void* post_bias,
                                const void* pre_w, const void* pre_bias, void* h_out, void* y,
                                cudaStream_t stream) {
    const ccv3d_status c = check_norm(d);
    if (c != CCV3D_OK) return c;
    const bool pre = d->pre != CCV3D_NORM_NONE, post = d->post != CCV3D_NORM_NONE;
    if (!gate_fits(d, gate)) return CCV3D_ERR_INVALID;
    if (d->rows == 0) return CCV3D_OK;  // (empty tensors have NULL addresses)
    if ((b == nullptr && (!pre || post || gate != nullptr || h_out != nullptr)) ||
        (!post && (post_w != nullptr || post_bias != nullptr)) ||
        (!pre && (pre_w != nullptr || pre_bias != nullptr || y != nullptr)))
        return CCV3D_ERR_INVALID;
    if (h == nullptr || (b != nullptr && h_out == nullptr) || (pre && y == nullptr))
        return CCV3D_ERR_INVALID;
    const size_t e = size_of(d->dtype), vec = d->C * e, all = (size_t)d->rows * vec;
    Buffers bufs;
    if (h != h_out) bufs.in(h, all);  // the stream may be updated in place
    bufs.in(b, all);
    if (gate != nullptr) bufs.in(gate, (size_t)(d->rows / d->gate_rows) * vec);
    for (const void* v : {post_w, post_bias, pre_w, pre_bias}) bufs.in(v, vec);
    bufs.out(h_out, all);
    bufs.out(y, all);
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    const NormFwd p = {h, b, gate, post_w, post_bias, pre_w, pre_bias, h_out, y,
                       d->rows, gate != nullptr ? d->gate_rows : d->rows, d->C, d->pre, d->post, d->act,
                       d->eps, d->scale, 1.0f / (float)d->C};
    d->dtype == CCV3D_BF16 ? norm_forward_bf16(p, stream) : norm_forward_fp32(p, stream);
    return launched();
}

size_t ccv3d_norm_workspace(const ccv3d_norm_desc* d) {
    if (check_norm(d) != CCV3D_OK || d->rows == 0) return 0;
    // with a gate or without one, with biases or without: the largest of them
    long long slots = 0;
    for (int call = 0; call < 6; ++call) {
        const bool gated = call & 1;
        if (gated && (d->gate_rows < 1 || d->rows % d->gate_rows != 0)) continue;
        const BwdShape b = bwd_shape(d, gated, call / 2);
        slots = std::max(slots, b.groups * b.blocks_per_group * b.sums);
    }
    return (size_t)slots * d->C * sizeof(float);
}

ccv3d_status ccv3d_norm_backward(const ccv3d_norm_desc* d, const void* h_out, const void* b,
                                 const void* gate, const void* post_w, const void* post_bias,
                                 const void* pre_w, const void* pre_bias, const void* dy,
                                 const void* dh_out, void* dh, void* db, void* dgate,
                                 void* dpost_w, void* dpost_bias, void* dpre_w, void* dpre_bias,
                                 void* ws, size_t ws_bytes, cudaStream_t stream) {
    const ccv3d_status c = check_norm(d);
    if (c != CCV3D_OK) return c;
    const bool pre = d->pre != CCV3D_NORM_NONE, post = d->post != CCV3D_NORM_NONE;
    if (!gate_fits(d, gate)) return CCV3D_ERR_INVALID;
    const size_t e = size_of(d->dtype), vec = d->C * e, all = (size_t)d->rows * vec;
    if (d->rows == 0) {  // sums over no rows
        for (void* v : {dpost_w, dpost_bias, dpre_w, dpre_bias})
            if (v != nullptr && cudaMemsetAsync(v, 0, vec, stream) != cudaSuccess) {
                cudaGetLastError();
                return CCV3D_ERR_CUDA;
            }
        return CCV3D_OK;
    }
    if ((b == nullptr && (!pre || post || gate != nullptr || db != nullptr)) ||
        (!post && (post_w != nullptr || post_bias != nullptr)) ||
        (!pre && (pre_w != nullptr || pre_bias != nullptr || dy != nullptr)) ||
        (gate == nullptr && dgate != nullptr) || (post_w == nullptr && dpost_w != nullptr) ||
        (post_bias == nullptr && dpost_bias != nullptr) ||
        (pre_w == nullptr && dpre_w != nullptr) || (pre_bias == nullptr && dpre_bias != nullptr))
        return CCV3D_ERR_INVALID;
    if ((pre && (h_out == nullptr || dy == nullptr)) || (dy == nullptr && dh_out == nullptr))
        return CCV3D_ERR_INVALID;
    const bool sums = dgate != nullptr || dpost_w != nullptr || dpost_bias != nullptr ||
                      dpre_w != nullptr || dpre_bias != nullptr;
    const size_t need = sums ? ccv3d_norm_workspace(d) : 0;
    if (sums && ws == nullptr) return CCV3D_ERR_INVALID;
    if (ws_bytes < need) return CCV3D_ERR_SCRATCH_LIMIT;
    const size_t gates = gate != nullptr ? (size_t)(d->rows / d->gate_rows) * vec : 0;
    Buffers bufs;
    for (const void* v : {h_out, b, dy, dh_out}) bufs.in(v, all);
    for (const void* v : {post_w, post_bias, pre_w, pre_bias}) bufs.in(v, vec);
    bufs.in(gate, gates);
    bufs.out(dh, all);
    bufs.out(db, all);
    bufs.out(dgate, gates);
    for (const void* v : {dpost_w, dpost_bias, dpre_w, dpre_bias}) bufs.out(v, vec);
    bufs.out(ws, need);
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    // bias gradients, and dgate, to which post_bias adds, want the sums of du and G
    const int form = pre_bias != nullptr || post_bias != nullptr ? kBwdBiased
                     : d->pre == CCV3D_NORM_LAYER || d->post == CCV3D_NORM_LAYER ? kBwdMeans
                                                                                 : kBwdRms;
    const BwdShape s = bwd_shape(d, gate != nullptr, form);
    const long long slots = s.groups * s.blocks_per_group;
    if (slots > 0x7fffffffLL) return CCV3D_ERR_UNSUPPORTED;
    const NormBwd p = {h_out, b, gate, post_w, post_bias, pre_w, pre_bias, dy, dh_out, dh, db,
                       sums ? static_cast<float*>(ws) : nullptr, d->rows, s.group_rows, s.groups,
                       slots, s.blocks_per_group, d->C, d->pre, d->post, d->act, d->eps, d->scale,
                       1.0f / (float)d->C};
    float* part = static_cast<float*>(ws);
    const NormFin f = {part, part, gate, post_w, post_bias, dgate, dpost_w, dpost_bias, dpre_w,
                       dpre_bias, s.groups, slots, s.blocks_per_group, d->C, s.sums == 4 ? 1 : 0,
                       b != nullptr ? 1 : 0, d->scale};
    d->dtype == CCV3D_BF16 ? norm_backward_bf16(p, s, form, sums ? &f : nullptr, stream)
                           : norm_backward_fp32(p, s, form, sums ? &f : nullptr, stream);
    return launched();
}

ccv3d_status ccv3d_pointwise_workspace(const ccv3d_pointwise_desc* d, size_t* forward_bytes,
                                       size_t* backward_bytes) {
    if (forward_bytes) *forward_bytes = 0;
    if (backward_bytes) *backward_bytes = 0;
    const ccv3d_status c = check_pointwise(d);
    if (c != CCV3D_OK) return c;
    if (d->pixels == 0) return CCV3D_OK;
    if (forward_bytes)
        *forward_bytes = forward_ws(d).total;
    if (backward_bytes) *backward_bytes = backward_ws(d).total;
    return CCV3D_OK;
}

ccv3d_status ccv3d_pointwise_forward(const ccv3d_pointwise_desc* d, const void* x, const void* w,
                                     const void* bias, const void* residual, void* out, void* pre,
                                     void* ws, size_t ws_bytes, cudaStream_t stream) {
    size_t need = 0;
    const ccv3d_status c = ccv3d_pointwise_workspace(d, &need, nullptr);
    if (c != CCV3D_OK) return c;
    if (d->pixels == 0) return CCV3D_OK;
    if (x == nullptr || w == nullptr || out == nullptr || (need > 0 && ws == nullptr))
        return CCV3D_ERR_INVALID;
    if (ws_bytes < need) return CCV3D_ERR_SCRATCH_LIMIT;
    const size_t e = size_of(d->dtype), o_bytes = (size_t)d->pixels * d->Cout * e;
    Buffers bufs;
    bufs.in(x, (size_t)d->pixels * d->Cin * e);
    bufs.in(w, (size_t)d->Cout * d->Cin * e);
    bufs.in(bias, (size_t)d->Cout * e);
    if (residual != out) bufs.in(residual, o_bytes);  // the stream may be updated in place
    bufs.out(out, o_bytes);
    bufs.out(pre, o_bytes);
    bufs.out(ws, need);
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    PwOut o = {bias, residual, out, pre, nullptr, d->pixels, d->Cout, d->act};
    return d->dtype == CCV3D_BF16 ? forward_type<bf16>(d, x, w, o, ws, stream)
                                  : forward_type<float>(d, x, w, o, ws, stream);
}

ccv3d_status ccv3d_pointwise_backward(const ccv3d_pointwise_desc* d, const void* x, const void* w,
                                      const void* pre, const void* dout, void* dx, void* dw,
                                      void* dbias, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
    size_t need = 0;
    const ccv3d_status c = ccv3d_pointwise_workspace(d, nullptr, &need);
    if (c != CCV3D_OK) return c;
    const size_t e = size_of(d->dtype);
    if (d->pixels == 0) {
        cudaError_t r = cudaSuccess;
        if (dw != nullptr) r = cudaMemsetAsync(dw, 0, (size_t)d->Cout * d->Cin * e, stream);
        if (r == cudaSuccess && dbias != nullptr)
            r = cudaMemsetAsync(dbias, 0, (size_t)d->Cout * e, stream);
        if (r != cudaSuccess) cudaGetLastError();
        return r == cudaSuccess ? CCV3D_OK : CCV3D_ERR_CUDA;
    }
    if (dout == nullptr || (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) ||
        (pre != nullptr) != (d->act != CCV3D_ACT_NONE) || (need > 0 && ws == nullptr))
        return CCV3D_ERR_INVALID;
    if (ws_bytes < need) return CCV3D_ERR_SCRATCH_LIMIT;
    const size_t x_bytes = (size_t)d->pixels * d->Cin * e, w_bytes = (size_t)d->Cout * d->Cin * e,
                 o_bytes = (size_t)d->pixels * d->Cout * e;
    Buffers bufs;
    bufs.in(x, x_bytes);
    bufs.in(w, w_bytes);
    bufs.in(pre, o_bytes);
    bufs.in(dout, o_bytes);
    bufs.out(dx, x_bytes);
    bufs.out(dw, w_bytes);
    bufs.out(dbias, (size_t)d->Cout * e);
    bufs.out(ws, need);
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    return d->dtype == CCV3D_BF16
               ? backward_type<bf16>(d, x, w, pre, dout, dx, dw, dbias, ws, stream)
               : backward_type<float>(d, x, w, pre, dout, dx, dw, dbias, ws, stream);
}

ccv3d_status ccv3d_qcache_sizes(const ccv3d_qcache_desc* d, size_t* code_bytes,
                                size_t* scale_bytes) {
    if (code_bytes) *code_bytes = 0;
    if (scale_bytes) *scale_bytes = 0;
    const ccv3d_status c = check_qcache(d);
    if (c != CCV3D_OK) return c;
    const QCacheJob j = qcache_job(d);
    const size_t px = (size_t)d->N * d->ring_slots * j.pixels;
    if (code_bytes) *code_bytes = px * j.code_bytes;
    if (scale_bytes) *scale_bytes = px * j.groups;
    return CCV3D_OK;
}

ccv3d_status ccv3d_qcache_write(const ccv3d_qcache_desc* d, const void* x, int T_x, int first,
                                int frames, int slot, void* codes, void* scales,
                                cudaStream_t stream) {
    size_t cb = 0, sb = 0;
    const ccv3d_status c = ccv3d_qcache_sizes(d, &cb, &sb);
    if (c != CCV3D_OK) return c;
    if (T_x < 0 || first < 0 || frames < 0 || frames > T_x - first || frames > d->ring_slots ||
        slot < 0 || slot >= d->ring_slots)
        return CCV3D_ERR_INVALID;
    if ((long long)d->N * frames == 0) return CCV3D_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr) return CCV3D_ERR_INVALID;
    if ((long long)d->N * frames > CCV3D_QCACHE_MAX_FRAMES) return CCV3D_ERR_UNSUPPORTED;
    QCacheJob j = qcache_job(d);
    Buffers bufs;
    bufs.in(x, (size_t)d->N * T_x * j.pixels * d->C * size_of(d->dtype));
    bufs.out(codes, cb);
    bufs.out(scales, sb);
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    j.src = x;
    j.codes = static_cast<uint8_t*>(codes);
    j.scales = static_cast<uint8_t*>(scales);
    j.T = T_x;
    j.first = first;
    j.frames = frames;
    j.slot = slot;
    d->dtype == CCV3D_BF16 ? qcache_write_run<bf16>(j, d->format, stream)
                           : qcache_write_run<float>(j, d->format, stream);
    return launched();
}

ccv3d_status ccv3d_qcache_read(const ccv3d_qcache_desc* d, const void* codes, const void* scales,
                               int head, int frames, void* out, cudaStream_t stream) {
    size_t cb = 0, sb = 0;
    const ccv3d_status c = ccv3d_qcache_sizes(d, &cb, &sb);
    if (c != CCV3D_OK) return c;
    if (frames < 0 || frames > d->ring_slots || head < 0 || head >= d->ring_slots)
        return CCV3D_ERR_INVALID;
    if ((long long)d->N * frames == 0) return CCV3D_OK;
    if (out == nullptr || codes == nullptr || scales == nullptr) return CCV3D_ERR_INVALID;
    if ((long long)d->N * frames > CCV3D_QCACHE_MAX_FRAMES) return CCV3D_ERR_UNSUPPORTED;
    QCacheJob j = qcache_job(d);
    Buffers bufs;
    bufs.in(codes, cb);
    bufs.in(scales, sb);
    bufs.out(out, (size_t)d->N * frames * j.pixels * d->C * size_of(d->dtype));
    const ccv3d_status k = bufs.check();
    if (k != CCV3D_OK) return k;
    j.dst = out;
    j.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    j.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
    j.frames = frames;
    j.slot = head;
    d->dtype == CCV3D_BF16 ? qcache_read_run<bf16>(j, d->format, stream)
                           : qcache_read_run<float>(j, d->format, stream);
    return launched();
}

ccv3d_status ccv3d_block_get_status(cudaStream_t stream) {
    int v = 0;
    cudaError_t e = take_status(&v, stream);
    if (e == cudaSuccess) e = norm_status_bf16(&v, stream);
    if (e == cudaSuccess) e = norm_status_fp32(&v, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CCV3D_ERR_CUDA;
    }
    return static_cast<ccv3d_status>(v);
}

}  // extern "C"
