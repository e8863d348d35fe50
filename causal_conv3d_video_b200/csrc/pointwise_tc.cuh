// pointwise_tc.cuh -- the 1x1x1 convolution and its gradients on the tensor
// cores: one persistent kernel for D(m, n) = sum_k A(m, k) B(n, k), bf16
// operands, fp32 accumulation, with the epilogue fused.
//
// The operands are read where they lie.  Forward, A = x and B = w, have k
// innermost ("k-major"); dx has A = dP k-major and B = w with n innermost; dw
// has both A = dP and B = x with m and n innermost ("mn-major").  An mn-major
// tile is loaded as 64 (m or n) x 64 (k) boxes, the layout the MMA's
// transposed operand form reads, so nothing is transposed in memory.
//
// A CTA pair (cta_group::2) computes 256 x BN tiles, k in blocks of 64: each
// CTA loads its 128 rows of A and half of the columns of B (a TMA ring), the
// even CTA issues M = 256 MMAs, accumulators are double-buffered in TMEM so a
// tile's epilogue overlaps the next tile's loads and MMAs.  One pair per SM
// pair walks the tiles, columns fastest, so that neighbouring pairs share rows
// of A in L2.  Long reductions over few tiles (dw, few rows) are split; the
// fp32 partials are joined, in order, by a second launch.
//
// Epilogue: eight warps, two for each 32 of the CTA's 128 rows, each on its
// own, 64 (or 32) columns at a time, the two taking turns: TMEM -> registers,
// + bias, activation, + residual, one rounding to bf16, into a swizzled
// shared-memory buffer, TMA store.  One more warp runs ahead of them with the
// residual (TMA, a ring of chunks of all 128 rows) and the tiles' bias, so that
// no global-memory latency is left in a chunk: with each warp fetching its own
// residual and bias, a chunk took 2500 cycles, most of them waiting.  A chunk's
// shared-memory reads are all issued before its writes: interleaved, the bias
// reads alone waited 1750 cycles.
#pragma once
#include "elem.cuh"
#include "epilogue.cuh"
#include "kwalk.cuh"
#include "pointwise_simt.cuh"
#include "ptx.cuh"

namespace ccv3d {

constexpr int kPtEpiWarps = 8;
// warp 0: operand loads, 1: MMAs, 2: residual and bias, 4-11: the epilogue
// (a warp reads the TMEM lanes of its number modulo 4)
constexpr int kPtThreads = 128 + 32 * kPtEpiWarps;
constexpr int kPtResBufs = 4;    // chunks of the residual's ring
constexpr int kPtAccs = 4;       // most accumulators (TMEM holds 512 columns)
constexpr int kPtRows = 256;     // rows of a pair's tile
constexpr int kPtK = 64;
constexpr int kPtA = 128 * kPtK * 2;     // bytes of A a CTA and stage
constexpr int kPtBox = 64 * kPtK * 2;    // one mn-major box

struct PtParams {
    CUtensorMap tm_a, tm_b, tm_out, tm_res, tm_pre;  // tm_out: of the partials where there are
    const bf16_t* bias;
    const bf16_t* residual;  // direct: plain loads and stores instead of TMA
    bf16_t *out, *pre;
    bool partial;            // D goes to fp32 partials [split][M][ldp] and nothing else
    long long M;
    int N, act, direct;
    int tiles_m, tiles_n, BN, kblocks, splits, kb_per_split, stages, tmem_cols;
    int chunk;               // columns the epilogue moves at a time: 64 or 32
    int n_bufs, n_pres;      // staging buffers of an epilogue warp
    int res_bufs;            // kPtResBufs, or 0 without a ring
    int n_acc;               // accumulators in TMEM, 2 to kPtAccs
    int step_n, step_m, step_s;  // number of pairs, in tiles of the walk
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ void pt_load_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                             int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void pt_load(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void pt_store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1,
                                            int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void pt_store(const CUtensorMap* m, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1) : "memory");
}
// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool pt_elect() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ uint32_t pt_mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive on another CTA's barrier.  No wider than CTA scope: what has to be
// ordered before it are this warp's TMEM loads, which tcgen05.wait::ld and the
// tcgen05 fence have completed; a cluster-scope release waited 3000 to 5000
// cycles for the warp's outstanding stores.
__device__ __forceinline__ void pt_arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Shared-memory descriptor of an mn-major tile of 64 x 64 boxes (128-byte
// swizzle): 64 (m or n) elements are contiguous, 8-row groups of k are 1024
// bytes apart (stride offset), the next 64 of m or n one box on (leading
// offset).
__device__ __forceinline__ uint64_t pt_desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kPtBox >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

__host__ __device__ constexpr int pt_b_bytes(bool mn, int bn) {
    return mn ? ((bn / 2 + 63) / 64) * kPtBox : (bn / 2) * kPtK * 2;
}
__host__ __device__ constexpr size_t pt_smem(bool b_mn, int bn, int stages, int chunk,
                                             int bufs, int res_bufs) {  // chunk: bytes / 2 of a row
    return 1024 + (size_t)stages * (kPtA + pt_b_bytes(b_mn, bn)) +
           (size_t)chunk * 2 * (kPtEpiWarps * 32 * bufs + 128 * res_bufs) +
           (size_t)bn * 4 * 2 + (size_t)(2 * stages + 2 * kPtAccs + 4 + 2 * kPtResBufs) * 8 + 16;
}

// A role's walk over its pair's work items: item i = (split, m, n), n fastest,
// i = pair, pair + G, ...; the step G is split into the three counters once on
// the host, so that a step is additions with carries.
struct PtWalk {
    int n, m, split, it, left;
    __device__ __forceinline__ PtWalk(const PtParams& p, int pair, int G) {
        const int total = p.tiles_m * p.tiles_n * p.splits;
        n = pair % p.tiles_n;
        const int r = pair / p.tiles_n;
        m = r % p.tiles_m;
        split = r / p.tiles_m;
        it = 0;
        left = (total - pair + G - 1) / G;
    }
    __device__ __forceinline__ void next(const PtParams& p) {
        n += p.step_n;
        m += p.step_m;
        split += p.step_s;
        if (n >= p.tiles_n) {
            n -= p.tiles_n;
            ++m;
        }
        if (m >= p.tiles_m) {
            m -= p.tiles_m;
            ++split;
        }
        ++it;
        --left;
    }
    __device__ __forceinline__ int kb0(const PtParams& p) const { return split * p.kb_per_split; }
    __device__ __forceinline__ int kb1(const PtParams& p) const {
        return min(kb0(p) + p.kb_per_split, p.kblocks);
    }
};

struct PtShared {
    uint8_t* staging;     // [epilogue warps][n_bufs + n_pres][32 rows][chunk]
    uint8_t* res;         // [res_bufs][128 rows][chunk]
    float* bias;          // [2][BN]
    uint64_t *acc_full, *acc_empty, *bias_full, *bias_empty, *res_full, *res_empty;
};

// The warp that runs ahead of the epilogue: the bias of each tile (two tiles)
// and its residual chunks (res_bufs chunks).
template <int kCh>
__device__ __forceinline__ void pt_ahead(const PtParams& p, const PtShared& sh, int pair, int G,
                                         uint32_t rank, int lane) {
    constexpr uint32_t kBytes = 128 * kCh * 2;
    if (p.partial) return;
    const int nch = p.BN / kCh;
    Ring ring;
    int issued = 0;
    bool ok = true;
    for (PtWalk w(p, pair, G); w.left > 0; w.next(p)) {
        if (p.bias != nullptr) {
            const int b = w.it & 1;
            if (w.it >= 2 && !mbar_wait(smem_u32(&sh.bias_empty[b]), (uint32_t)(((w.it >> 1) & 1) ^ 1),
                                        &g_block_status, p.wait_limit_ns))
                ok = false;
            for (int i = lane; i < p.BN; i += 32) {
                const int c = w.n * p.BN + i;
                sh.bias[b * p.BN + i] = c < p.N ? (float)p.bias[c] : 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.bias_full[b]));
        }
        if (p.res_bufs > 0 && lane == 0) {
            const int r0 = w.m * kPtRows + (int)rank * 128;
            for (int c = 0; c < nch; ++c, ++issued) {
                const uint32_t bar = smem_u32(&sh.res_full[ring.st]);
                if (issued >= p.res_bufs && !mbar_wait(smem_u32(&sh.res_empty[ring.st]), ring.ph ^ 1u,
                                                       &g_block_status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                // (a box outside the matrix is zeros)
                mbar_arrive_expect_tx(bar, kBytes);
                pt_load(smem_u32(sh.res + ring.st * kBytes), &p.tm_res, bar,
                        w.n * p.BN + c * kCh, r0);
                ring.next(p.res_bufs);
            }
        }
        if (__any_sync(0xffffffffu, !ok)) return;
    }
}

// A chunk of 32 rows between a staging buffer and a matrix whose rows are no
// multiple of 16 bytes (no tensor map): row by row with the lanes along the
// columns, two columns a lane where rows start on 4 bytes; several rows' reads
// before their writes.
template <int kCh, bool kLoad>
__device__ __forceinline__ void pt_direct(const bf16_t* src, bf16_t* dst, uint8_t* buf,
                                          const PtParams& p, int r0, int c0, bool in, int lane) {
    constexpr int kRowB = kCh * 2;
    const bf16_t* base = kLoad ? src : dst;
    const long long bytes = p.M * p.N * 2;
    const int rows = in ? (int)min(32LL, p.M - r0) : 0;
    auto at = [&](int r, int c) { return buf + r * kRowB + (swizzled_chunk<kRowB>(c >> 3, r) << 4) + (c & 7) * 2; };
    if ((p.N & 1) == 0) {
        constexpr int kLanes = kCh / 2, kRows = 32 / kLanes;  // rows side by side in a warp
        const int c = lane % kLanes * 2, sub = lane / kLanes;
        if (c0 + c >= p.N) return;
#pragma unroll 8
        for (int r = sub; r < 32; r += kRows) {
            const long long i = ((long long)r0 + r) * p.N + c0 + c;
            const bool ok = r < rows && in_bounds(&g_block_status, base + i, 4, base, bytes);
            if constexpr (kLoad)
                *reinterpret_cast<uint32_t*>(at(r, c)) =
                    ok ? *reinterpret_cast<const uint32_t*>(src + i) : 0u;
            else if (ok)
                *reinterpret_cast<uint32_t*>(dst + i) = *reinterpret_cast<const uint32_t*>(at(r, c));
        }
    } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
#pragma unroll
            for (int c = lane; c < kCh; c += 32) {
                const long long i = ((long long)r0 + r) * p.N + c0 + c;
                const bool ok = r < rows && c0 + c < p.N &&
                                in_bounds(&g_block_status, base + i, 2, base, bytes);
                if constexpr (kLoad)
                    *reinterpret_cast<bf16_t*>(at(r, c)) = ok ? src[i] : bf16_t(0.0f);
                else if (ok)
                    dst[i] = *reinterpret_cast<const bf16_t*>(at(r, c));
            }
    }
}

// The epilogue of one warp: every second chunk of kCh columns of its 32 rows.
// kPart: chunks of 32 columns go out as fp32 partials.
template <int kCh, bool kPart>
__device__ __forceinline__ void pt_epilogue(const PtParams& p, const PtShared& sh, uint32_t tmem,
                                            int pair, int G, uint32_t rank, bool leader, int warp,
                                            int lane) {
    constexpr int kRowB = kPart ? 128 : kCh * 2, kBuf = 32 * kRowB;
    static_assert(!kPart || kCh == 32, "partials: 32 fp32 columns are a 128-byte row");
    const int q = warp & 3, wid = warp - 4, set = wid >> 2;
    const int nch = p.BN / kCh;
    uint8_t* bufs = sh.staging + (size_t)wid * kBuf * (p.n_bufs + p.n_pres);
    uint8_t* pres = bufs + (size_t)p.n_bufs * kBuf;
    const uint32_t empty_leader = pt_mapa(smem_u32(sh.acc_empty), 0);
    const bool biased = !kPart && p.bias != nullptr;
    int turn = 0;  // staging buffer
    int first = 0;  // chunks of the tiles before this one
    Ring acc;
    bool ok = true;
    for (PtWalk w(p, pair, G); w.left > 0; w.next(p), first += nch, acc.next(p.n_acc)) {
        const int b = w.it & 1;  // bias buffer
        const int r0 = w.m * kPtRows + (int)rank * 128 + q * 32;  // M < 2^31 - 256
        const int c_set = (set + first) & 1;
        if (biased && ok && !mbar_wait(smem_u32(&sh.bias_full[b]), (uint32_t)((w.it >> 1) & 1),
                                       &g_block_status, p.wait_limit_ns))
            ok = false;
        if (ok && !mbar_wait(smem_u32(&sh.acc_full[acc.st]), acc.ph, &g_block_status,
                             p.wait_limit_ns))
            ok = false;
        tc_fence_after();
        const uint32_t tacc = tmem + (uint32_t)(acc.st * p.BN) + ((uint32_t)(q * 32) << 16);
        const float* bias = sh.bias + b * p.BN;
        auto drained = [&]() {  // this warp has read the accumulator (and the bias)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(smem_u32(&sh.acc_empty[acc.st]));
                else pt_arrive_remote(empty_leader + (uint32_t)(acc.st * 8));
                if (biased) mbar_arrive(smem_u32(&sh.bias_empty[b]));
            }
        };
        if (c_set >= nch) drained();
        for (int c = c_set; c < nch; c += 2) {
            const int c0 = w.n * p.BN + c * kCh;
            const bool in = r0 < p.M && c0 < p.N;
            uint32_t v[kCh];
            __syncwarp();  // lanes left a wait or lane 0's stores: the load wants them together
#pragma unroll
            for (int i = 0; i < kCh / 16; ++i)
                tmem_ld_32x32b_x16(tacc + (uint32_t)(c * kCh + i * 16),
                                   *reinterpret_cast<uint32_t(*)[16]>(&v[i * 16]));
            tmem_ld_wait();
            if (biased) {
#pragma unroll
                for (int i = 0; i < kCh; i += 4) {
                    const float4 t = *reinterpret_cast<const float4*>(bias + c * kCh + i);
                    v[i] = __float_as_uint(__uint_as_float(v[i]) + t.x);
                    v[i + 1] = __float_as_uint(__uint_as_float(v[i + 1]) + t.y);
                    v[i + 2] = __float_as_uint(__uint_as_float(v[i + 2]) + t.z);
                    v[i + 3] = __float_as_uint(__uint_as_float(v[i + 3]) + t.w);
                }
            }
            if (c + 2 >= nch) drained();
            // the store before the last one has been read: its buffer is free
            if (lane == 0) bulk_wait_group_read1();
            __syncwarp();
            uint8_t* buf = bufs + turn * kBuf;
            if constexpr (kPart) {
#pragma unroll
                for (int i = 0; i < kCh / 4; ++i)
                    *reinterpret_cast<uint4*>(buf + lane * kRowB +
                                              (swizzled_chunk<kRowB>(i, lane) << 4)) =
                        make_uint4(v[i * 4], v[i * 4 + 1], v[i * 4 + 2], v[i * 4 + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (in && ok) pt_store_3d(&p.tm_out, smem_u32(buf), c0, r0, w.split);
                    bulk_commit_group();
                }
                turn ^= 1;
                continue;
            }
            uint8_t* pre = pres + turn * kBuf;
            if (p.pre != nullptr) {
#pragma unroll
                for (int i = 0; i < kCh / 8; ++i) {
                    float t[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) t[k] = __uint_as_float(v[i * 8 + k]);
                    *reinterpret_cast<uint4*>(pre + lane * kRowB +
                                              (swizzled_chunk<kRowB>(i, lane) << 4)) =
                        pack8<bf16_t, true>(t).a;
                }
            }
            if (p.act == kActSilu) {
#pragma unroll
                for (int i = 0; i < kCh; ++i)
                    v[i] = __float_as_uint(act_of<bf16_t>(__uint_as_float(v[i]), kActSilu));
            } else if (p.act == kActGelu) {
#pragma unroll
                for (int i = 0; i < kCh; ++i)
                    v[i] = __float_as_uint(act_of<bf16_t>(__uint_as_float(v[i]), kActGelu));
            }
            if (p.residual != nullptr) {
                const uint8_t* src = buf;
                const int j = first + c, slot = j % kPtResBufs;
                if (p.res_bufs > 0) {
                    if (ok && !mbar_wait(smem_u32(&sh.res_full[slot]),
                                         (uint32_t)((j / kPtResBufs) & 1), &g_block_status,
                                         p.wait_limit_ns))
                        ok = false;
                    src = sh.res + (size_t)(slot * 4 + q) * kBuf;
                } else {
                    pt_direct<kCh, true>(p.residual, nullptr, buf, p, r0, c0, in, lane);
                    __syncwarp();
                }
                Raw8<bf16_t, true> res[kCh / 8];
#pragma unroll
                for (int i = 0; i < kCh / 8; ++i)
                    res[i].a = *reinterpret_cast<const uint4*>(
                        src + lane * kRowB + (swizzled_chunk<kRowB>(i, lane) << 4));
#pragma unroll
                for (int i = 0; i < kCh / 8; ++i) {
                    float t[8];
                    unpack8<bf16_t, true>(res[i], t);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[i * 8 + k] = __float_as_uint(__uint_as_float(v[i * 8 + k]) + t[k]);
                }
                if (p.res_bufs > 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.res_empty[slot]));
                }
            }
#pragma unroll
            for (int i = 0; i < kCh / 8; ++i) {
                float t[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) t[k] = __uint_as_float(v[i * 8 + k]);
                *reinterpret_cast<uint4*>(buf + lane * kRowB +
                                          (swizzled_chunk<kRowB>(i, lane) << 4)) =
                    pack8<bf16_t, true>(t).a;
            }
            if (!p.direct) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (in && ok) {
                        pt_store(&p.tm_out, smem_u32(buf), c0, r0);
                        if (p.pre != nullptr) pt_store(&p.tm_pre, smem_u32(pre), c0, r0);
                    }
                    bulk_commit_group();
                }
            } else {
                __syncwarp();
                pt_direct<kCh, false>(nullptr, p.out, buf, p, r0, c0, in && ok, lane);
                if (p.pre != nullptr)
                    pt_direct<kCh, false>(nullptr, p.pre, pre, p, r0, c0, in && ok, lane);
                __syncwarp();
            }
            turn ^= 1;
        }
    }
    if (lane == 0) bulk_wait_group0();  // stores complete before the block exits
}

template <bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPtThreads, 1)
pw_tc_kernel(const __grid_constant__ PtParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = p.stages, BN = p.BN, hB = BN / 2;
    const int kB = pt_b_bytes(B_MN, BN);
    uint8_t* sA = smem;
    uint8_t* sB = smem + (size_t)stages * kPtA;
    uint8_t* staging = sB + (size_t)stages * kB;
    PtShared sh;
    sh.staging = staging;
    sh.res = staging + (size_t)kPtEpiWarps * 32 * p.chunk * 2 * (p.n_bufs + p.n_pres);
    sh.bias = reinterpret_cast<float*>(sh.res + (size_t)128 * p.chunk * 2 * p.res_bufs);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(sh.bias + 2 * BN);
    uint64_t* empty_bar = full_bar + stages;
    sh.acc_full = empty_bar + stages;      // [kPtAccs]
    sh.acc_empty = sh.acc_full + kPtAccs;  // [kPtAccs], used in the even CTA
    sh.bias_full = sh.acc_empty + kPtAccs;
    sh.bias_empty = sh.bias_full + 2;
    sh.res_full = sh.bias_empty + 2;   // [kPtResBufs]
    sh.res_empty = sh.res_full + kPtResBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sh.res_empty + kPtResBufs);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, G = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int b = 0; b < kPtAccs; ++b) {
            mbar_init(smem_u32(&sh.acc_full[b]), 1);
            mbar_init(smem_u32(&sh.acc_empty[b]), 2 * kPtEpiWarps);  // of both CTAs
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sh.bias_full[b]), 1);
            mbar_init(smem_u32(&sh.bias_empty[b]), kPtEpiWarps);
        }
        for (int b = 0; b < kPtResBufs; ++b) {
            mbar_init(smem_u32(&sh.res_full[b]), 1);
            mbar_init(smem_u32(&sh.res_empty[b]), 4);  // the four warps whose turn the chunk is
        }
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_a);
        tma_prefetch_desc(&p.tm_b);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), (uint32_t)p.tmem_cols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = 2u * (uint32_t)(kPtA + kB);
            Ring ring;
            int issued = 0;
            bool ok = true;
            for (PtWalk t(p, pair, G); t.left > 0 && ok; t.next(p)) {
                const int m0 = t.m * kPtRows + (int)rank * 128;
                const int n0 = t.n * BN + (int)rank * hB;
                const int kb1 = t.kb1(p);
                for (int kb = t.kb0(p); kb < kb1; ++kb, ++issued) {
                    if (issued >= stages && !mbar_wait(smem_u32(&empty_bar[ring.st]), ring.ph ^ 1u,
                                                       &g_block_status, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t local = smem_u32(&full_bar[ring.st]);
                    if (leader) mbar_arrive_expect_tx(local, bytes);
                    const uint32_t fb = pair_leader_addr(local);
                    const uint32_t a = smem_u32(sA + ring.st * kPtA);
                    const uint32_t b = smem_u32(sB + ring.st * kB);
                    if constexpr (A_MN) {
                        pt_load_pair(a, &p.tm_a, fb, m0, kb * kPtK);
                        pt_load_pair(a + kPtBox, &p.tm_a, fb, m0 + 64, kb * kPtK);
                    } else {
                        pt_load_pair(a, &p.tm_a, fb, kb * kPtK, m0);
                    }
                    if constexpr (B_MN) {
                        for (int c = 0; c < hB; c += 64)
                            pt_load_pair(b + (c >> 6) * kPtBox, &p.tm_b, fb, n0 + c, kb * kPtK);
                    } else {
                        pt_load_pair(b, &p.tm_b, fb, kb * kPtK, n0);
                    }
                    ring.next(stages);
                }
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // The whole warp walks the loop and one elected lane issues: the
            // descriptors stay in uniform registers, as the MMA takes them.
            const uint32_t idesc = idesc_bf16_m256((uint32_t)BN) | (A_MN ? 1u << 15 : 0u) |
                                   (B_MN ? 1u << 16 : 0u);
            // 16 of k further on: 32 bytes of a k-major row, two 1024-byte groups mn-major
            constexpr uint32_t a_step = A_MN ? 2048 >> 4 : 32 >> 4;
            constexpr uint32_t b_step = B_MN ? 2048 >> 4 : 32 >> 4;
            const uint64_t a0 = A_MN ? pt_desc_mn(smem_u32(sA)) : smem_desc_kmajor(smem_u32(sA), 128);
            const uint64_t b0 = B_MN ? pt_desc_mn(smem_u32(sB)) : smem_desc_kmajor(smem_u32(sB), 128);
            Ring ring, acc;
            bool ok = true;
            for (PtWalk t(p, pair, G); t.left > 0 && ok; t.next(p), acc.next(p.n_acc)) {
                const int kb0 = t.kb0(p), kb1 = t.kb1(p);
                if (t.it >= p.n_acc) ok = mbar_wait(smem_u32(&sh.acc_empty[acc.st]), acc.ph ^ 1u,
                                                    &g_block_status, p.wait_limit_ns);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc.st * BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = mbar_wait(smem_u32(&full_bar[ring.st]), ring.ph, &g_block_status,
                                   p.wait_limit_ns);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = a0 + (uint64_t)((ring.st * kPtA) >> 4);
                    const uint64_t bd = b0 + (uint64_t)((ring.st * kB) >> 4);
                    if (pt_elect()) {
#pragma unroll
                        for (int kk = 0; kk < kPtK / 16; ++kk)
                            umma_bf16_pair(d, a + a_step * kk, bd + b_step * kk, idesc,
                                           kb == kb0 && kk == 0 ? 0u : 1u);
                        umma_commit_pair(smem_u32(&empty_bar[ring.st]), (uint16_t)0x3);
                        if (kb + 1 == kb1)
                            umma_commit_pair(smem_u32(&sh.acc_full[acc.st]), (uint16_t)0x3);
                    }
                    __syncwarp();
                    ring.next(stages);
                }
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        if (p.chunk == 64) pt_ahead<64>(p, sh, pair, G, rank, lane);
        else pt_ahead<32>(p, sh, pair, G, rank, lane);
    } else if (warp >= 4) {
        if (p.partial)
            pt_epilogue<32, true>(p, sh, tmem_base, pair, G, rank, leader, warp, lane);
        else if (p.chunk == 64)
            pt_epilogue<64, false>(p, sh, tmem_base, pair, G, rank, leader, warp, lane);
        else
            pt_epilogue<32, false>(p, sh, tmem_base, pair, G, rank, leader, warp, lane);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // the peer's shared memory and barriers stay alive until both are done
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, (uint32_t)p.tmem_cols);
    }
}

// Rows of C elements copied to rows of Cp (a multiple of 8, the rest zeros):
// TMA needs row strides of 16 bytes.
__global__ void __launch_bounds__(256) pw_pack_kernel(const bf16_t* src, bf16_t* dst, long long rows,
                                                      int C, int Cp) {
    const long long n = rows * (Cp / 8), step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const long long r = i / (Cp / 8);
        const int c0 = (int)(i - r * (Cp / 8)) * 8;
        Raw8<bf16_t, false> raw;
        float f[8];
        if (!in_bounds(&g_block_status, src + r * C, C * 2LL, src, rows * C * 2)) continue;
        load8<bf16_t, false>(raw, src + r * C, c0, 1, C);
        unpack8<bf16_t, false>(raw, f);
        if (in_bounds(&g_block_status, dst + r * Cp + c0, 16, dst, rows * Cp * 2))
            *reinterpret_cast<uint4*>(dst + r * Cp + c0) = pack8<bf16_t, true>(f).a;
    }
}

}  // namespace ccv3d
