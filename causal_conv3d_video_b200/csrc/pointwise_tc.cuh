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
// Epilogue: each of four warps owns 32 rows of the CTA's 128 and works alone,
// 64 (or 32) columns at a time: TMEM -> registers, + bias, activation,
// + residual, one rounding to bf16, into a swizzled shared-memory buffer, TMA
// store.  The residual chunk was loaded by TMA into that same buffer up to
// two chunks ahead.
#pragma once
#include "elem.cuh"
#include "epilogue.cuh"
#include "kwalk.cuh"
#include "pointwise_simt.cuh"
#include "ptx.cuh"

namespace ccv3d {

constexpr int kPtThreads = 192;  // warp 0: loads, warp 1: MMAs, warps 2-5: epilogue
constexpr int kPtRows = 256;     // rows of a pair's tile
constexpr int kPtK = 64;
constexpr int kPtA = 128 * kPtK * 2;     // bytes of A a CTA and stage
constexpr int kPtBox = 64 * kPtK * 2;    // one mn-major box

struct PtParams {
    CUtensorMap tm_a, tm_b, tm_out, tm_res, tm_pre;
    const bf16_t* bias;
    const bf16_t* residual;  // direct: plain loads and stores instead of TMA
    bf16_t *out, *pre;
    float* partial;          // not NULL: fp32 partials [split][M][ldp] only
    long long M;
    int N, ldp, act, direct;
    int tiles_m, tiles_n, BN, kblocks, splits, kb_per_split, stages, n_bufs, tmem_cols;
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
__device__ __forceinline__ void pt_store(const CUtensorMap* m, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ uint32_t pt_mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void pt_arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
                 : "memory");
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
__host__ __device__ constexpr int pt_chunk(int bn) { return bn % 64 == 0 ? 64 : 32; }
__host__ __device__ constexpr size_t pt_smem(bool b_mn, int bn, int stages, int n_bufs, bool pre) {
    return 1024 + (size_t)stages * (kPtA + pt_b_bytes(b_mn, bn)) +
           (size_t)4 * 32 * pt_chunk(bn) * 2 * (n_bufs + (pre ? 2 : 0)) + (size_t)bn * 4 +
           (size_t)(2 * stages + 4 + 16) * 8 + 16;
}

struct PtItem {
    int m, n, split, kb0, kb1;  // tile of 256 rows, tile of BN columns
};
__device__ __forceinline__ PtItem pt_item(const PtParams& p, int i) {
    PtItem t;
    t.n = i % p.tiles_n;
    i /= p.tiles_n;
    t.m = i % p.tiles_m;
    t.split = i / p.tiles_m;
    t.kb0 = t.split * p.kb_per_split;
    t.kb1 = min(t.kb0 + p.kb_per_split, p.kblocks);
    return t;
}

// One chunk of kCh columns of a warp's 32 rows (lane = row): registers u from
// TMEM, then everything up to the store.
template <int kCh>
__device__ __forceinline__ void pt_epilogue(const PtParams& p, uint32_t tacc, int pair, int G,
                                            int total, uint32_t rank, bool leader, int warp,
                                            int lane, uint8_t* staging, float* bias_s,
                                            uint64_t* acc_full, uint64_t* acc_empty,
                                            uint64_t* res_bar) {
    constexpr int kRowB = kCh * 2, kBuf = 32 * kRowB;
    const int q = warp & 3, etid = threadIdx.x - 64;
    const int nb = p.n_bufs, nch = p.BN / kCh;
    uint8_t* bufs = staging + (size_t)q * kBuf * nb;
    uint8_t* pres = staging + (size_t)4 * kBuf * nb + (size_t)q * kBuf * 2;
    uint64_t* bars = res_bar + q * 4;  // one per residual buffer
    const uint32_t empty_leader = pt_mapa(smem_u32(acc_empty), 0);
    const bool res_tma = p.residual != nullptr && !p.direct && p.partial == nullptr;
    const int items = (total - pair + G - 1) / G;  // of this pair
    const int chunks = items * nch;
    // chunk j of this warp: whether it lies in D at all, and where
    auto place = [&](int j, int& r0, int& c0) {
        const PtItem t = pt_item(p, pair + (j / nch) * G);
        const long long r = (long long)t.m * kPtRows + rank * 128 + q * 32;
        r0 = (int)r;  // M < 2^31 - 256
        c0 = t.n * p.BN + (j % nch) * kCh;
        return r < p.M && c0 < p.N;
    };
    auto fetch = [&](int j) {  // lane 0: residual chunk j into its buffer
        int r0, c0;
        if (j >= chunks || !place(j, r0, c0)) return;
        const uint32_t bar = smem_u32(&bars[j & 3]);
        mbar_arrive_expect_tx(bar, kBuf);
        pt_load(smem_u32(bufs + (j & 3) * kBuf), &p.tm_res, bar, c0, r0);
    };
    uint32_t phases = 0;  // parity of each residual buffer's next completion
    if (res_tma && lane == 0) {
        fetch(0);
        fetch(1);
    }
    bool ok = true;
    int bias_tile = -1;
    for (int it = 0, j = 0; it < items; ++it) {
        const PtItem t = pt_item(p, pair + it * G);
        const int b = it & 1;
        if (ok && !mbar_wait(smem_u32(&acc_full[b]), (uint32_t)((it >> 1) & 1), &g_block_status,
                             p.wait_limit_ns))
            ok = false;
        tc_fence_after();
        if (t.n != bias_tile && p.partial == nullptr) {  // (uniform over the four warps)
            epi_bar();
            for (int i = etid; i < p.BN; i += 128) {
                const int c = t.n * p.BN + i;
                bias_s[i] = p.bias != nullptr && c < p.N ? (float)p.bias[c] : 0.0f;
            }
            epi_bar();
            bias_tile = t.n;
        }
        for (int c = 0; c < nch; ++c, ++j) {
            int r0, c0;
            const bool inside = place(j, r0, c0);
            uint32_t v[kCh];
            __syncwarp();  // lanes left a wait or lane 0's stores: the load wants them together
#pragma unroll
            for (int i = 0; i < kCh / 16; ++i)
                tmem_ld_32x32b_x16(tacc + (uint32_t)(b * p.BN) + ((uint32_t)(q * 32) << 16) +
                                       (uint32_t)(c * kCh + i * 16),
                                   *reinterpret_cast<uint32_t(*)[16]>(&v[i * 16]));
            tmem_ld_wait();
            if (c == nch - 1) {  // this accumulator is drained: back to the MMAs
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(smem_u32(&acc_empty[b]));
                    else pt_arrive_remote(empty_leader + (uint32_t)(b * 8));
                }
            }
            if (p.partial != nullptr) {
                const long long row = (long long)r0 + lane;
                if (inside && ok && row < p.M) {
                    float* dst = p.partial + ((long long)t.split * p.M + row) * p.ldp + c0;
#pragma unroll
                    for (int i = 0; i < kCh; i += 4)
                        if (c0 + i < p.ldp &&
                            in_bounds(&g_block_status, dst + i, 16, p.partial,
                                      (long long)p.splits * p.M * p.ldp * 4))
                            *reinterpret_cast<uint4*>(dst + i) =
                                make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
                continue;
            }
            // buffers: all but the last chunk's store have been read
            if (lane == 0) {
                bulk_wait_group_read1();
                if (res_tma) fetch(j + 2);
            }
            __syncwarp();
            uint8_t* buf = bufs + (nb == 4 ? (j & 3) : (j & 1)) * kBuf;
            uint8_t* row_b = buf + lane * kRowB;
            if (res_tma && inside) {
                const int k = j & 3;
                if (ok && !mbar_wait(smem_u32(&bars[k]), (phases >> k) & 1u, &g_block_status,
                                     p.wait_limit_ns))
                    ok = false;
                phases ^= 1u << k;
            } else if (p.residual != nullptr && p.direct) {
                // row by row, lanes along the columns
                for (int r = 0; r < 32; ++r)
#pragma unroll
                    for (int i = lane; i < kCh; i += 32) {
                        const long long row = (long long)r0 + r;
                        const bf16_t x = inside && row < p.M && c0 + i < p.N
                                             ? p.residual[row * p.N + c0 + i] : bf16_t(0.0f);
                        *reinterpret_cast<bf16_t*>(buf + r * kRowB +
                                                   (swizzled_chunk<kRowB>(i >> 3, r) << 4) +
                                                   (i & 7) * 2) = x;
                    }
                __syncwarp();
            }
            uint8_t* row_p = pres + (j & 1) * kBuf + lane * kRowB;
#pragma unroll
            for (int i = 0; i < kCh / 8; ++i) {
                float u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    u[k] = __uint_as_float(v[i * 8 + k]) + bias_s[c * kCh + i * 8 + k];
                const int at = swizzled_chunk<kRowB>(i, lane) << 4;
                if (p.pre != nullptr)
                    *reinterpret_cast<uint4*>(row_p + at) = pack8<bf16_t, true>(u).a;
                if (p.act != kActNone)
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[k] = act_of<bf16_t>(u[k], p.act);
                if (p.residual != nullptr) {
                    Raw8<bf16_t, true> r;
                    r.a = *reinterpret_cast<const uint4*>(row_b + at);
                    float f[8];
                    unpack8<bf16_t, true>(r, f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[k] += f[k];
                }
                *reinterpret_cast<uint4*>(row_b + at) = pack8<bf16_t, true>(u).a;
            }
            if (!p.direct) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && inside && ok) {
                    pt_store(&p.tm_out, smem_u32(buf), c0, r0);
                    if (p.pre != nullptr) pt_store(&p.tm_pre, smem_u32(pres + (j & 1) * kBuf), c0, r0);
                }
                if (lane == 0) bulk_commit_group();
            } else {
                __syncwarp();
                for (int r = 0; r < 32; ++r)
#pragma unroll
                    for (int i = lane; i < kCh; i += 32) {
                        const long long row = (long long)r0 + r, at = row * p.N + c0 + i;
                        if (!inside || !ok || row >= p.M || c0 + i >= p.N) continue;
                        const int off = r * kRowB + (swizzled_chunk<kRowB>(i >> 3, r) << 4) + (i & 7) * 2;
                        if (!in_bounds(&g_block_status, p.out + at, 2, p.out, p.M * p.N * 2)) continue;
                        p.out[at] = *reinterpret_cast<const bf16_t*>(buf + off);
                        if (p.pre != nullptr)
                            p.pre[at] = *reinterpret_cast<const bf16_t*>(pres + (j & 1) * kBuf + off);
                    }
                __syncwarp();
            }
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
    const int kB = pt_b_bytes(B_MN, BN), ch = pt_chunk(BN);
    uint8_t* sA = smem;
    uint8_t* sB = smem + (size_t)stages * kPtA;
    uint8_t* staging = sB + (size_t)stages * kB;
    float* bias_s = reinterpret_cast<float*>(
        staging + (size_t)4 * 32 * ch * 2 * (p.n_bufs + (p.pre != nullptr ? 2 : 0)));
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(bias_s + BN);
    uint64_t* empty_bar = full_bar + stages;
    uint64_t* acc_full = empty_bar + stages;  // [2]
    uint64_t* acc_empty = acc_full + 2;       // [2], used in the even CTA
    uint64_t* res_bar = acc_empty + 2;        // [4 warps][4]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_bar + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, G = gridDim.x >> 1;
    const int total = p.tiles_m * p.tiles_n * p.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 8);  // four epilogue warps of both CTAs
        }
        for (int b = 0; b < 16; ++b) mbar_init(smem_u32(&res_bar[b]), 1);
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
            for (int i = pair; i < total && ok; i += G) {
                const PtItem t = pt_item(p, i);
                const int m0 = t.m * kPtRows + (int)rank * 128;
                const int n0 = t.n * BN + (int)rank * hB;
                for (int kb = t.kb0; kb < t.kb1; ++kb, ++issued) {
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
        if (lane == 0 && leader) {
            const uint32_t idesc = idesc_bf16_m256((uint32_t)BN) | (A_MN ? 1u << 15 : 0u) |
                                   (B_MN ? 1u << 16 : 0u);
            // 16 of k further on: 32 bytes of a k-major row, two 1024-byte groups mn-major
            constexpr uint32_t a_step = A_MN ? 2048 >> 4 : 32 >> 4;
            constexpr uint32_t b_step = B_MN ? 2048 >> 4 : 32 >> 4;
            const uint64_t a0 = A_MN ? pt_desc_mn(smem_u32(sA)) : smem_desc_kmajor(smem_u32(sA), 128);
            const uint64_t b0 = B_MN ? pt_desc_mn(smem_u32(sB)) : smem_desc_kmajor(smem_u32(sB), 128);
            Ring ring;
            bool ok = true;
            for (int i = pair, it = 0; i < total && ok; i += G, ++it) {
                const PtItem t = pt_item(p, i);
                const int b = it & 1;
                if (it >= 2 && !mbar_wait(smem_u32(&acc_empty[b]), (uint32_t)(((it >> 1) & 1) ^ 1),
                                          &g_block_status, p.wait_limit_ns))
                    break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(b * BN);
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!mbar_wait(smem_u32(&full_bar[ring.st]), ring.ph, &g_block_status,
                                   p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = a0 + (uint64_t)((ring.st * kPtA) >> 4);
                    const uint64_t bd = b0 + (uint64_t)((ring.st * kB) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kPtK / 16; ++kk)
                        umma_bf16_pair(d, a + a_step * kk, bd + b_step * kk, idesc,
                                       kb == t.kb0 && kk == 0 ? 0u : 1u);
                    umma_commit_pair(smem_u32(&empty_bar[ring.st]), (uint16_t)0x3);
                    ring.next(stages);
                }
                umma_commit_pair(smem_u32(&acc_full[b]), (uint16_t)0x3);
            }
        }
        __syncwarp();
    } else {
        if (ch == 64)
            pt_epilogue<64>(p, tmem_base, pair, G, total, rank, leader, warp, lane, staging, bias_s,
                            acc_full, acc_empty, res_bar);
        else
            pt_epilogue<32>(p, tmem_base, pair, G, total, rank, leader, warp, lane, staging, bias_s,
                            acc_full, acc_empty, res_bar);
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
        load8<bf16_t, false>(raw, src + r * C, c0, 1, C);
        unpack8<bf16_t, false>(raw, f);
        *reinterpret_cast<uint4*>(dst + r * Cp + c0) = pack8<bf16_t, true>(f).a;
    }
}

}  // namespace ccv3d
