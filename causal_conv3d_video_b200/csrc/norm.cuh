// norm.cuh -- the norms before and after a block, fused with the block's gate
// and residual scale, and their gradients.
//
// A row is the C channels of one pixel.  norm(v) = (v - mu) * rstd * w + bias
// with mu = 0, rstd = 1 / sqrt(mean(v^2) + eps) (RMS), or mu = mean(v),
// rstd = 1 / sqrt(mean((v - mu)^2) + eps) (layer norm).  Forward:
//     h_out = round(h + scale * gate * post(b)),   y = act(pre(h_out)).
// y is taken from the stored (rounded) h_out, so the fused call gives the
// bits of the two halves called one after the other, and the backward pass,
// which starts from the stored h_out, is the derivative of what ran.
//
// Backward, with n and m the normalised rows of h_out and b, u = n w + bias:
//     du = dy act'(u),  dn = du w,
//     G = dh_out + rstd (dn - n mean(dn n) [- mean(dn)]),    dh = G,
//     dm = scale gate G post_w,  db = rstd_b (dm - m mean(dm m) [- mean(dm)]).
// All parameter gradients come from four column sums: sum du n and sum du,
// and per gate row sum G m and sum G (dgate = scale (post_w sum G m +
// post_bias sum G), dpost_w = scale sum_gates gate sum G m).  The rows'
// gradients are rounded once; the sums stay in fp32 registers over a block's
// rows, then go through fp32 partials that a second launch adds in a fixed
// order: no atomics, the same bits every run.
//
// HBM-bound (2 to 4 tensors moved forward, 4 to 6 backward): a row is read
// once and stays in registers.  TPR threads share a row (a power of two within
// a warp, or the whole block for wide rows), so that the row statistics are a
// few shuffles and each thread keeps a fixed set of channels, whose column sums
// it owns.
//   * Rows within a warp's share (the decoder's widths): blocks walk tiles of
//     rows; one thread has the next tiles copied to shared memory (bulk copies
//     on an mbarrier ring, rows are contiguous) while all work on this one, so
//     that the bytes in flight do not hang on registers or occupancy, and an
//     odd channel count costs no unaligned global loads.  The vectors (gate,
//     weights, biases, with the residual scale multiplied in) are in shared
//     memory as fp32.
//   * Wider rows: a block a row, loads straight to registers, the next row's
//     in flight while this one is worked on.
#pragma once
#include "elem.cuh"
#include "bulk.cuh"
#include "params.h"

namespace ccv3d {

struct NormFwd {
    const void *h, *b, *gate, *post_w, *post_bias, *pre_w, *pre_bias;
    void *h_out, *y;
    long long rows, gate_rows;
    int C, pre, post, act;
    float eps, scale, inv_c;
};

struct NormBwd {
    const void *h, *b, *gate, *post_w, *post_bias, *pre_w, *pre_bias, *dy, *dh_out;
    void *dh, *db;
    float* part;             // [quantity][gate groups x blocks per group][C]
    long long rows, group_rows;  // rows that share a gate row (all of them without a gate)
    long long groups, slots;     // gate groups; groups x blocks per group
    int blocks_per_group;
    int C, pre, post, act;
    float eps, scale, inv_c;
};

// Sum of K values over the threads of a row, the same bits in each of them.
// TPR = 0: over the block, through shared memory; two buffers in turn, so one
// barrier a sum is enough.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[4][32], int& turn) {
    constexpr int kSpan = TPR == 0 ? 32 : TPR;
#pragma unroll
    for (int o = kSpan / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (TPR == 0) {
        static_assert(K <= 4, "row_sum: at most four values");
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) red[turn][k][warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = lane < nw ? red[turn][k][lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            v[k] = s;
        }
        turn ^= 1;
    }
}

// First channel and channel step of unit u of row-thread `lane`.
template <bool V>
__device__ __forceinline__ int unit_c0(int u, int lane, int tpr) {
    return V ? (u * tpr + lane) * 8 : u * 8 * tpr + lane;
}

// Normalise the NU units of a row in place (v -> (v - mu) * rstd; channels
// past C end as 0); returns rstd.
template <bool V, int TPR, int NU>
__device__ __forceinline__ float normalise(float (&v)[NU][8], int kind, int lane, int tpr, int C,
                                           float eps, float inv_c, float (*red)[4][32],
                                           int& turn) {
    if (kind == kNormLayer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += v[u][i];
        row_sum<TPR, 1>(s, red, turn);
        const float mu = s[0] * inv_c;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] = (V ? c0 : c0 + i * tpr) < C ? v[u][i] - mu : 0.0f;
        }
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[0] = fmaf(v[u][i], v[u][i], q[0]);
    row_sum<TPR, 1>(q, red, turn);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_c, eps));
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= rstd;
    return rstd;
}

// Channels c0 .. of a weight vector as fp32; `otherwise` where there is none,
// 0 past C (so that idle lanes add nothing to a row's sums).
template <typename T, bool V>
__device__ __forceinline__ void weights8(float (&f)[8], const T* w, float otherwise, int c0,
                                         int step, int C) {
    if (w != nullptr) {
        Raw8<T, V> r;
        load8<T, V>(r, w, c0, step, C);
        unpack8<T, V>(r, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (V ? c0 : c0 + i * step) < C ? otherwise : 0.0f;
    }
}

// The wide-row form, one block a row (TPR = 0).  kB: there is a block output b
// (its norm, gate and scale); otherwise only the norm and activation of h.
template <typename T, bool V, int NU, bool kB>
__global__ void __launch_bounds__(512) norm_fwd_rows(
    const __grid_constant__ NormFwd p) {
    __shared__ float red[2][4][32];
    int turn = 0;
    constexpr int TPR = 0;
    const int tpr = (int)blockDim.x, lane = (int)threadIdx.x;
    const int C = p.C;
    const long long tensor = p.rows * C * (long long)sizeof(T), stride = gridDim.x;
    const T *h = static_cast<const T*>(p.h), *b = static_cast<const T*>(p.b);
    // (checked build) the row at element `at` of a tensor lies in it
    auto fits = [&](const void* base, long long at) {
        return in_bounds(&g_block_status, static_cast<const T*>(base) + at,
                         (long long)C * sizeof(T), base, tensor);
    };
    // what each thread keeps of the vectors
    float w[NU][8], wb[NU][8], g[NU][8], gb[NU][8];
    long long gate_row = -1;
    auto gates = [&](long long row) {  // scale * gate * post_w, scale * gate * post_bias
        const T* gate = static_cast<const T*>(p.gate);
        if (gate != nullptr && index_ok(&g_block_status, row, p.rows / p.gate_rows)) gate += row * C;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
            float t[8];
            weights8<T, V>(t, gate, 1.0f, c0, tpr, C);
            weights8<T, V>(g[u], static_cast<const T*>(p.post_w), 1.0f, c0, tpr, C);
            weights8<T, V>(gb[u], static_cast<const T*>(p.post_bias), 0.0f, c0, tpr, C);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] *= p.scale;
                g[u][i] *= t[i];
                gb[u][i] *= t[i];
            }
        }
        gate_row = row;
    };
    if (p.y != nullptr)
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            weights8<T, V>(w[u], static_cast<const T*>(p.pre_w), 1.0f, unit_c0<V>(u, lane, tpr),
                           tpr, C);
            weights8<T, V>(wb[u], static_cast<const T*>(p.pre_bias), 0.0f,
                           unit_c0<V>(u, lane, tpr), tpr, C);
        }
    auto load = [&](long long row, Raw8<T, V> (&rh)[NU], Raw8<T, V> (&rb)[NU]) {
        const bool ok = row < p.rows;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
            if (ok && fits(h, row * C)) load8<T, V>(rh[u], h + row * C, c0, tpr, C);
            else zero8<T, V>(rh[u]);
            if constexpr (kB) {
                if (ok && fits(b, row * C)) load8<T, V>(rb[u], b + row * C, c0, tpr, C);
                else zero8<T, V>(rb[u]);
            }
        }
    };
    long long row = blockIdx.x;
    Raw8<T, V> rh[NU], rb[NU];
    load(row, rh, rb);
    for (; row < p.rows; row += stride) {
        Raw8<T, V> nh[NU], nb[NU];
        load(row + stride, nh, nb);
        const long long at = row * C;
        float v[NU][8];
#pragma unroll
        for (int u = 0; u < NU; ++u) unpack8<T, V>(rh[u], v[u]);
        if constexpr (kB) {
            const long long gr = p.gate != nullptr ? row / p.gate_rows : 0;
            if (gr != gate_row) gates(gr);
            float m[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) unpack8<T, V>(rb[u], m[u]);
            if (p.post != kNormNone)
                normalise<V, TPR, NU>(m, p.post, lane, tpr, C, p.eps, p.inv_c, red, turn);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c0 = unit_c0<V>(u, lane, tpr);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] += fmaf(m[u][i], g[u][i], gb[u][i]);
                const Raw8<T, V> r = pack8<T, V>(v[u]);
                if (fits(p.h_out, at)) store8<T, V>(r, static_cast<T*>(p.h_out) + at, c0, tpr, C);
                unpack8<T, V>(r, v[u]);  // the stored value is what the norm reads
            }
        }
        if (p.y != nullptr) {
            normalise<V, TPR, NU>(v, p.pre, lane, tpr, C, p.eps, p.inv_c, red, turn);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = fmaf(v[u][i], w[u][i], wb[u][i]);
                if (p.act != kActNone)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = act_of<T>(v[u][i], p.act);
                if (fits(p.y, at))
                    store8<T, V>(pack8<T, V>(v[u]), static_cast<T*>(p.y) + at,
                                 unit_c0<V>(u, lane, tpr), tpr, C);
            }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            rh[u] = nh[u];
            if constexpr (kB) rb[u] = nb[u];
        }
    }
}

// A block's column sums -> its slot of the partials.  colbuf (TPR > 0): [warps][C].
template <bool V, int TPR, int NU, int kQ>
__device__ __forceinline__ void store_colsums(const NormBwd& p, const float (&acc)[kQ][NU][8],
                                              int lane, int tpr, float* colbuf) {
    if (p.part == nullptr) return;
    const int C = p.C;
    const long long part_bytes = (long long)kQ * p.slots * C * 4;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        float* out = p.part + ((long long)q * p.slots + blockIdx.x) * C;
        const bool fits = in_bounds(&g_block_status, out, (long long)C * 4, p.part, part_bytes);
        if constexpr (TPR == 0) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c0 = unit_c0<V>(u, lane, tpr), c = V ? c0 + i : c0 + i * tpr;
                    if (c < C && fits) out[c] = acc[q][u][i];
                }
        } else {
            // rows of one warp by shuffles, then the warps through shared memory
            const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
            __syncthreads();
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a = acc[q][u][i];
#pragma unroll
                    for (int o = 16; o >= TPR; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
                    const int c0 = unit_c0<V>(u, lane, tpr), c = V ? c0 + i : c0 + i * tpr;
                    if (wl < TPR && c < C) colbuf[warp * C + c] = a;
                }
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += blockDim.x) {
                float a = 0.0f;
                for (int w = 0; w < (int)(blockDim.x >> 5); ++w) a += colbuf[w * C + c];
                if (fits) out[c] = a;
            }
        }
    }
}

// Gradients of the rows, and the column sums over this block's rows: block
// (group, j) takes every blocks_per_group-th step of the group's rows, from
// its j-th.  kGen: a layer norm or a bias is there (row means, sums of du and
// G); without it the RMS-only arithmetic is a third shorter.
template <typename T, bool V, int NU, bool kGen>
__global__ void __launch_bounds__(512) norm_bwd_rows(
    const __grid_constant__ NormBwd p) {
    __shared__ float red[2][4][32];
    int turn = 0;
    constexpr int kQ = kGen ? 4 : 2;
    constexpr int TPR = 0;
    const int tpr = (int)blockDim.x, lane = (int)threadIdx.x;
    const int C = p.C;
    const long long tensor = p.rows * C * (long long)sizeof(T);
    float acc[kQ][NU][8] = {};
    const long long group = blockIdx.x / p.blocks_per_group;
    const int part_of = (int)(blockIdx.x % p.blocks_per_group);
    const long long row0 = group * p.group_rows, row1 = row0 + p.group_rows;
    const bool has_pre = p.dy != nullptr, has_b = p.b != nullptr;
    const long long gate_at = index_ok(&g_block_status, group, p.groups) ? group * C : 0;
    float w[NU][8], wb[NU][8], g[NU][8];  // pre_w, pre_bias, scale * gate * post_w
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int c0 = unit_c0<V>(u, lane, tpr);
        weights8<T, V>(w[u], static_cast<const T*>(p.pre_w), 1.0f, c0, tpr, C);
        if constexpr (kGen)
            weights8<T, V>(wb[u], static_cast<const T*>(p.pre_bias), 0.0f, c0, tpr, C);
        float t[8];
        weights8<T, V>(t, p.gate == nullptr ? nullptr : static_cast<const T*>(p.gate) + gate_at, 1.0f,
                       c0, tpr, C);
        weights8<T, V>(g[u], static_cast<const T*>(p.post_w), 1.0f, c0, tpr, C);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[u][i] *= p.scale * t[i];
    }
    struct Row {
        Raw8<T, V> h[NU], y[NU], g[NU], b[NU];
    };
    // (checked build) the row at element `at` of a tensor lies in it; each tensor
    // by itself, since the call may go without any of them
    auto fits = [&](const void* base, long long at) {
        return in_bounds(&g_block_status, static_cast<const T*>(base) + at,
                         (long long)C * sizeof(T), base, tensor);
    };
    auto load = [&](long long row, Row& r) {
        const long long at = row * C;
        const bool ok = row < row1;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
            zero8<T, V>(r.h[u]); zero8<T, V>(r.y[u]); zero8<T, V>(r.g[u]); zero8<T, V>(r.b[u]);
            if (!ok) continue;
            if (has_pre && fits(p.h, at) && fits(p.dy, at)) {
                load8<T, V>(r.h[u], static_cast<const T*>(p.h) + at, c0, tpr, C);
                load8<T, V>(r.y[u], static_cast<const T*>(p.dy) + at, c0, tpr, C);
            }
            if (p.dh_out != nullptr && fits(p.dh_out, at))
                load8<T, V>(r.g[u], static_cast<const T*>(p.dh_out) + at, c0, tpr, C);
            if (has_b && fits(p.b, at))
                load8<T, V>(r.b[u], static_cast<const T*>(p.b) + at, c0, tpr, C);
        }
    };
    const long long stride = p.blocks_per_group;
    long long row = row0 + part_of;
    Row cur;
    load(row, cur);
    for (; row < row1; row += stride) {
        Row next;
        load(row + stride, next);
        const long long at = row * C;
        float G[NU][8];
#pragma unroll
        for (int u = 0; u < NU; ++u) unpack8<T, V>(cur.g[u], G[u]);
        if (has_pre) {
            float n[NU][8], d[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                unpack8<T, V>(cur.h[u], n[u]);
                unpack8<T, V>(cur.y[u], d[u]);
            }
            const float rstd = normalise<V, TPR, NU>(n, kGen ? p.pre : kNormRms, lane, tpr, C,
                                                     p.eps, p.inv_c, red, turn);
            float s[kGen ? 2 : 1] = {};
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                if (p.act == kActSilu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[u][i] *= act_grad_of<T>(kGen ? fmaf(n[u][i], w[u][i], wb[u][i])
                                                       : n[u][i] * w[u][i], kActSilu);
                } else if (p.act == kActGelu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[u][i] *= act_grad_of<T>(kGen ? fmaf(n[u][i], w[u][i], wb[u][i])
                                                       : n[u][i] * w[u][i], kActGelu);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[0][u][i] = fmaf(d[u][i], n[u][i], acc[0][u][i]);
                    if constexpr (kGen) acc[2][u][i] += d[u][i];
                    d[u][i] *= w[u][i];
                    s[0] = fmaf(d[u][i], n[u][i], s[0]);
                    if constexpr (kGen) s[1] += d[u][i];
                }
            }
            row_sum<TPR, kGen ? 2 : 1>(s, red, turn);
            const float a = -s[0] * p.inv_c;
            float mean = 0.0f;
            if constexpr (kGen) mean = p.pre == kNormLayer ? s[1] * p.inv_c : 0.0f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[u][i] = fmaf(rstd, fmaf(n[u][i], a, kGen ? d[u][i] - mean : d[u][i]), G[u][i]);
        }
        if (p.dh != nullptr && fits(p.dh, at))
#pragma unroll
            for (int u = 0; u < NU; ++u)
                store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.dh) + at,
                             unit_c0<V>(u, lane, tpr), tpr, C);
        if (has_b) {
            float m[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) unpack8<T, V>(cur.b[u], m[u]);
            float rstd = 1.0f;
            if (p.post != kNormNone)
                rstd = normalise<V, TPR, NU>(m, kGen ? p.post : kNormRms, lane, tpr, C, p.eps,
                                             p.inv_c, red, turn);
            float s[kGen ? 2 : 1] = {};
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[1][u][i] = fmaf(G[u][i], m[u][i], acc[1][u][i]);
                    // (past C, G may hold a row's mean: m and g are 0 there, and the
                    // sums of those columns are not written)
                    if constexpr (kGen) acc[3][u][i] += G[u][i];
                    G[u][i] *= g[u][i];
                    s[0] = fmaf(G[u][i], m[u][i], s[0]);
                    if constexpr (kGen) s[1] += G[u][i];
                }
            if (p.db != nullptr) {
                if (p.post != kNormNone) {
                    row_sum<TPR, kGen ? 2 : 1>(s, red, turn);
                    const float a = -s[0] * p.inv_c;
                    float mean = 0.0f;
                    if constexpr (kGen) mean = p.post == kNormLayer ? s[1] * p.inv_c : 0.0f;
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            G[u][i] = rstd * fmaf(m[u][i], a, kGen ? G[u][i] - mean : G[u][i]);
                }
                if (fits(p.db, at))
#pragma unroll
                    for (int u = 0; u < NU; ++u)
                        store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.db) + at,
                                     unit_c0<V>(u, lane, tpr), tpr, C);
            }
        }
        cur = next;
    }
    store_colsums<V, TPR, NU, kQ>(p, acc, lane, tpr, nullptr);
}

// ------------------------------------------------- rows within a warp's share
constexpr int kTileThreads = 256;  // at most

// Tiles of rows in shared memory.  A tile's bytes start at the 16-byte
// boundary at or before its first row; what a bulk copy cannot take at a
// tensor's very end (under 16 bytes) is copied by the threads.
struct TileShape {
    int rows;        // rows of a tile
    int cap;         // bytes of a tile and tensor in shared memory
    int stages, vec_len;  // vec_len: channels the block's threads cover, the vectors' length
};

struct TileSpan {
    long long from;  // byte of the tensor the copy starts at (a multiple of 16)
    int off;         // of the tile's first row in the copy
    int bulk, tail;  // bytes copied in bulk, bytes after them
};
__device__ __forceinline__ TileSpan tile_span(long long row0, long long row1, int row_bytes,
                                              long long tensor) {
    TileSpan t;
    const long long b0 = row0 * row_bytes, b1 = row1 * row_bytes;
    t.from = b0 & ~15LL;
    t.off = (int)(b0 - t.from);
    const long long end = (b1 + 15) & ~15LL;
    t.bulk = (int)((end <= tensor ? end : b1 & ~15LL) - t.from);
    t.tail = (int)(b1 - t.from) - t.bulk;
    if (t.tail < 0) t.tail = 0;
    return t;
}

// Start the copies of a tile's nT tensors (one thread).
template <int nT>
__device__ __forceinline__ void tile_issue(const TileSpan& t, const void* const (&src)[nT],
                                           uint8_t* stage, int cap, uint32_t bar,
                                           long long tensor) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < nT; ++k) n += src[k] != nullptr;
    mbar_arrive_expect_tx(bar, (uint32_t)(n * t.bulk));
    if (t.bulk == 0) return;
#pragma unroll
    for (int k = 0; k < nT; ++k) {
        if (src[k] == nullptr) continue;
        const uint8_t* from = static_cast<const uint8_t*>(src[k]) + t.from;
        // checked build: a range outside the tensor is recorded and read from its start
        if (!in_bounds(&g_block_status, from, t.bulk, src[k], tensor))
            from = static_cast<const uint8_t*>(src[k]);
        bulk_g2s(smem_u32(stage + (size_t)k * cap), from, (uint32_t)t.bulk, bar);
    }
}
// The bytes after the bulk copies (all threads; uniform).
template <int nT>
__device__ __forceinline__ void tile_tail(const TileSpan& t, const void* const (&src)[nT],
                                          uint8_t* stage, int cap, long long tensor) {
    if (t.tail == 0) return;
    if ((int)threadIdx.x < t.tail)
#pragma unroll
        for (int k = 0; k < nT; ++k)
            if (src[k] != nullptr &&
                index_ok(&g_block_status, t.from + t.bulk + (int)threadIdx.x, tensor))
                stage[(size_t)k * cap + t.bulk + threadIdx.x] =
                    static_cast<const uint8_t*>(src[k])[t.from + t.bulk + threadIdx.x];
    __syncthreads();
}

// Waits for a tile; false from the first wait that ran out on.  After that the
// thread stores nothing, and issues nothing where it is the issuing one; `waits`
// counts down from the number of stages, a wait each that ran out, so that the
// tiles issued before are all waited for (the stages - 1 that follow: no copy
// lands in shared memory that has become another block's) and the waits for the
// ones never issued end soon.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t ph, int stages, int& waits) {
    if (waits > 0 && !mbar_wait(smem_u32(bar), ph, &g_block_status, kWaitLimitNs)) --waits;
    return waits == stages;
}

// Eight channels of a vector kept in shared memory, as pairs.
__device__ __forceinline__ void vec8(f2 (&f)[4], const float* s, bool vec, int c0, int step) {
    if (vec) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s + c0);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(s + c0 + 4);
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2_make(s[c0 + 2 * i * step], s[c0 + (2 * i + 1) * step]);
    }
}

template <typename T>
__device__ __forceinline__ float vec_at(const void* p, int c, int C, float otherwise) {
    return c >= C ? 0.0f : (p == nullptr ? otherwise : (float)static_cast<const T*>(p)[c]);
}

// Unit u of a staged row, in registers (zeros for a row that is not there).
template <typename T, bool V, int TPR>
__device__ __forceinline__ void tile_unit(f2 (&v)[4], const uint8_t* at, int u, int lane, int C,
                                          bool ok) {
    Raw8<T, V> r;
    if (ok) load8<T, V>(r, reinterpret_cast<const T*>(at), unit_c0<V>(u, lane, TPR), TPR, C);
    else zero8<T, V>(r);
    unpack8<T, V>(r, v);
}

// normalise() on pairs, within a warp's share.
template <bool V, int TPR, int NU>
__device__ __forceinline__ float normalise2(f2 (&v)[NU][4], int kind, int lane, int C, float eps,
                                            float inv_c) {
    int turn = 0;
    if (kind == kNormLayer) {
        f2 t = f2_all(0.0f);
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) t = f2_add(t, v[u][i]);
        float s[1] = {f2_sum(t)};
        row_sum<TPR, 1>(s, nullptr, turn);
        const f2 mu = f2_all(-s[0] * inv_c);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, TPR);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[u][i] = f2_add(v[u][i], mu);
                if constexpr (V) {
                    if (c0 >= C) v[u][i] = f2_all(0.0f);
                } else {
                    float a, b;
                    f2_get(v[u][i], a, b);
                    v[u][i] = f2_make(c0 + 2 * i * TPR < C ? a : 0.0f,
                                      c0 + (2 * i + 1) * TPR < C ? b : 0.0f);
                }
            }
        }
    }
    f2 t = f2_all(0.0f);
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) t = f2_fma(v[u][i], v[u][i], t);
    float q[1] = {f2_sum(t)};
    row_sum<TPR, 1>(q, nullptr, turn);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_c, eps));
    const f2 r2 = f2_all(rstd);
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = f2_mul(v[u][i], r2);
    return rstd;
}

template <typename T, bool V, int TPR, int NU, bool kB>
__global__ void __launch_bounds__(kTileThreads, 3) norm_fwd_tiles(
    const __grid_constant__ NormFwd p, const __grid_constant__ TileShape sh) {
    extern __shared__ __align__(128) uint8_t tile_smem[];
    constexpr int nT = kB ? 2 : 1;
    const int rpp = (int)blockDim.x / TPR;  // rows a pass
    const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR, C = p.C;
    const int row_bytes = C * (int)sizeof(T);
    const long long tensor = p.rows * row_bytes;
    const long long tiles = (p.rows + sh.rows - 1) / sh.rows;
    uint8_t* ring = tile_smem;
    const size_t stage_bytes = (size_t)nT * sh.cap;
    float* vecs = reinterpret_cast<float*>(ring + sh.stages * stage_bytes);  // w, wb, g, gb
    const int L = sh.vec_len;
    uint64_t* full = reinterpret_cast<uint64_t*>(vecs + 4 * L);
    const void* src[nT];
    src[0] = p.h;
    if constexpr (kB) src[1] = p.b;
    auto span = [&](long long t) {
        const long long r0 = t * sh.rows;
        return tile_span(r0, min(r0 + sh.rows, p.rows), row_bytes, tensor);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < sh.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        fence_mbar_init();
        for (int s = 0; s < sh.stages; ++s) {
            const long long t = blockIdx.x + (long long)s * gridDim.x;
            if (t < tiles)
                tile_issue<nT>(span(t), src, ring + s * stage_bytes, sh.cap, smem_u32(&full[s]), tensor);
        }
    }
    for (int c = threadIdx.x; c < L; c += blockDim.x) {
        vecs[c] = vec_at<T>(p.pre_w, c, C, 1.0f);
        vecs[L + c] = vec_at<T>(p.pre_bias, c, C, 0.0f);
        // one gate for all rows: with the scale and the post norm's vectors
        const float g = p.scale * (p.gate_rows >= p.rows ? vec_at<T>(p.gate, c, C, 1.0f) : 1.0f);
        vecs[2 * L + c] = g * vec_at<T>(p.post_w, c, C, 1.0f);
        vecs[3 * L + c] = g * vec_at<T>(p.post_bias, c, C, 0.0f);
    }
    __syncthreads();
    // (checked build) the row at element `at` of a tensor lies in it
    auto fits = [&](const void* base, long long at) {
        return in_bounds(&g_block_status, static_cast<const T*>(base) + at, row_bytes, base, tensor);
    };
    const bool gated = kB && p.gate != nullptr && p.gate_rows < p.rows;
    const bool post_bias = p.post_bias != nullptr, pre_bias = p.pre_bias != nullptr;
    int st = 0;
    uint32_t ph = 0;
    int waits = sh.stages;  // (see tile_wait)
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        const bool live = tile_wait(&full[st], ph, sh.stages, waits);
        uint8_t* stage = ring + st * stage_bytes;
        const TileSpan sp = span(t);
        tile_tail<nT>(sp, src, stage, sh.cap, tensor);
        const int n = (int)min((long long)sh.rows, p.rows - t * sh.rows);
        for (int r0 = 0; r0 < n; r0 += rpp) {
            const int r = r0 + sub;
            const bool ok = live && r < n;
            const long long row = t * sh.rows + r, at = row * C;
            const uint8_t* in = stage + sp.off + (size_t)r * row_bytes;
            f2 v[NU][4];
#pragma unroll
            for (int u = 0; u < NU; ++u) tile_unit<T, V, TPR>(v[u], in, u, lane, C, ok);
            if constexpr (kB) {
                f2 m[NU][4];
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    tile_unit<T, V, TPR>(m[u], in + sh.cap, u, lane, C, ok);
                if (p.post != kNormNone)
                    normalise2<V, TPR, NU>(m, p.post, lane, C, p.eps, p.inv_c);
                const long long gate_row = gated && ok ? row / p.gate_rows : 0;
                const T* gate = static_cast<const T*>(p.gate) +
                                (index_ok(&g_block_status, gate_row, p.rows / p.gate_rows) ? gate_row * C : 0);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const int c0 = unit_c0<V>(u, lane, TPR);
                    f2 f[4];
                    vec8(f, vecs + 2 * L, V, c0, TPR);
#pragma unroll
                    for (int i = 0; i < 4; ++i) m[u][i] = f2_mul(m[u][i], f[i]);
                    if (post_bias) {
                        vec8(f, vecs + 3 * L, V, c0, TPR);
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[u][i] = f2_add(m[u][i], f[i]);
                    }
                    if (gated) {
                        Raw8<T, V> r;
                        load8<T, V>(r, gate, c0, TPR, C);
                        unpack8<T, V>(r, f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[u][i] = f2_mul(m[u][i], f[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[u][i] = f2_add(v[u][i], m[u][i]);
                    const Raw8<T, V> o = pack8<T, V>(v[u]);
                    if (ok && fits(p.h_out, at)) store8<T, V>(o, static_cast<T*>(p.h_out) + at, c0, TPR, C);
                    unpack8<T, V>(o, v[u]);  // the stored value is what the norm reads
                }
            }
            if (p.y != nullptr) {
                normalise2<V, TPR, NU>(v, p.pre, lane, C, p.eps, p.inv_c);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const int c0 = unit_c0<V>(u, lane, TPR);
                    f2 f[4];
                    vec8(f, vecs, V, c0, TPR);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[u][i] = f2_mul(v[u][i], f[i]);
                    if (pre_bias) {
                        vec8(f, vecs + L, V, c0, TPR);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[u][i] = f2_add(v[u][i], f[i]);
                    }
                    if (p.act == kActSilu) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[u][i] = f2_act<T>(v[u][i], kActSilu);
                    } else if (p.act == kActGelu) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[u][i] = f2_act<T>(v[u][i], kActGelu);
                    }
                    if (ok && fits(p.y, at))
                        store8<T, V>(pack8<T, V>(v[u]), static_cast<T*>(p.y) + at, c0, TPR, C);
                }
            }
        }
        __syncthreads();  // every thread is done with the stage
        if (threadIdx.x == 0 && live) {
            const long long nt = t + (long long)sh.stages * gridDim.x;
            if (nt < tiles)
                tile_issue<nT>(span(nt), src, stage, sh.cap, smem_u32(&full[st]), tensor);
        }
        if (++st == sh.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
}

// kForm: kBwdRms, RMS norms without biases (two column sums, no row means);
// kBwdMeans, a layer norm is there; kBwdBiased, a bias is (four column sums:
// du and G too).
constexpr int kBwdRms = 0, kBwdMeans = 1, kBwdBiased = 2;
// 256-thread blocks an SM: four column sums of two or three units take more than
// 128 registers a thread (spilled at two blocks: 398 us against 230 for 900000 x
// 96, two layer norms with biases).
__host__ __device__ constexpr int bwd_blocks(int form, int units) {
    return form == kBwdBiased && units > 1 ? 1 : 2;
}
template <typename T, bool V, int TPR, int NU, int kForm>
__global__ void __launch_bounds__(kTileThreads, bwd_blocks(kForm, NU)) norm_bwd_tiles(
    const __grid_constant__ NormBwd p, const __grid_constant__ TileShape sh) {
    extern __shared__ __align__(128) uint8_t tile_smem[];
    constexpr int nT = 4, kQ = kForm == kBwdBiased ? 4 : 2;
    constexpr bool kMean = kForm != kBwdRms, kBias = kForm == kBwdBiased;
    const int rpp = (int)blockDim.x / TPR;  // rows a pass
    const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR, C = p.C;
    const int row_bytes = C * (int)sizeof(T);
    const long long tensor = p.rows * row_bytes;
    const long long group = blockIdx.x / p.blocks_per_group;
    const int part_of = (int)(blockIdx.x % p.blocks_per_group);
    const long long row0 = group * p.group_rows, row1 = row0 + p.group_rows;
    const long long tiles = (p.group_rows + sh.rows - 1) / sh.rows;
    uint8_t* ring = tile_smem;
    const size_t stage_bytes = (size_t)nT * sh.cap;
    float* vecs = reinterpret_cast<float*>(ring + sh.stages * stage_bytes);  // pre_w, pre_bias, g
    const int L = sh.vec_len;
    uint64_t* full = reinterpret_cast<uint64_t*>(vecs + 3 * L);
    const bool has_pre = p.dy != nullptr, has_b = p.b != nullptr;
    const void* src[nT] = {has_pre ? p.h : nullptr, p.dy, p.dh_out, p.b};
    auto span = [&](long long t) {
        const long long r0 = row0 + t * sh.rows;
        return tile_span(r0, min(r0 + sh.rows, row1), row_bytes, tensor);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < sh.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        fence_mbar_init();
        for (int s = 0; s < sh.stages; ++s) {
            const long long t = part_of + (long long)s * p.blocks_per_group;
            if (t < tiles)
                tile_issue<nT>(span(t), src, ring + s * stage_bytes, sh.cap, smem_u32(&full[s]), tensor);
        }
    }
    // (checked build) the row at element `at` of a tensor lies in it
    auto fits = [&](const void* base, long long at) {
        return in_bounds(&g_block_status, static_cast<const T*>(base) + at, row_bytes, base, tensor);
    };
    const T* gate = static_cast<const T*>(p.gate);
    if (gate != nullptr && index_ok(&g_block_status, group, p.groups)) gate += group * C;
    for (int c = threadIdx.x; c < L; c += blockDim.x) {
        vecs[c] = vec_at<T>(p.pre_w, c, C, 1.0f);
        vecs[L + c] = vec_at<T>(p.pre_bias, c, C, 0.0f);
        vecs[2 * L + c] = p.scale * vec_at<T>(gate, c, C, 1.0f) * vec_at<T>(p.post_w, c, C, 1.0f);
    }
    __syncthreads();
    f2 acc[kQ][NU][4];
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][u][i] = f2_all(0.0f);
    int st = 0;
    uint32_t ph = 0;
    int waits = sh.stages;  // (see tile_wait)
    for (long long t = part_of; t < tiles; t += p.blocks_per_group) {
        const bool live = tile_wait(&full[st], ph, sh.stages, waits);
        uint8_t* stage = ring + st * stage_bytes;
        const TileSpan sp = span(t);
        tile_tail<nT>(sp, src, stage, sh.cap, tensor);
        const int n = (int)min((long long)sh.rows, p.group_rows - t * sh.rows);
        for (int r0 = 0; r0 < n; r0 += rpp) {
            const int r = r0 + sub;
            const bool ok = live && r < n;
            const long long at = (row0 + t * sh.rows + r) * C;
            const uint8_t* in = stage + sp.off + (size_t)r * row_bytes;
            // two arrays of the row's channels: v is h, then b; G is dy and what
            // comes of it, then the gradient of the stream and what comes of that
            f2 v[NU][4], G[NU][4];
            if (has_pre) {
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    tile_unit<T, V, TPR>(v[u], in, u, lane, C, ok);
                    tile_unit<T, V, TPR>(G[u], in + sh.cap, u, lane, C, ok);
                }
                const float rstd = normalise2<V, TPR, NU>(v, kMean ? p.pre : kNormRms, lane, C,
                                                          p.eps, p.inv_c);
                f2 s0 = f2_all(0.0f), s1 = f2_all(0.0f);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const int c0 = unit_c0<V>(u, lane, TPR);
                    f2 w[4], wb[4];
                    vec8(w, vecs, V, c0, TPR);
                    if constexpr (kBias) vec8(wb, vecs + L, V, c0, TPR);
                    auto slope = [&](int kind) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f2 a = kBias ? f2_fma(v[u][i], w[i], wb[i]) : f2_mul(v[u][i], w[i]);
                            G[u][i] = f2_mul(G[u][i], f2_act_grad<T>(a, kind));
                        }
                    };
                    if (p.act == kActSilu) slope(kActSilu);
                    else if (p.act == kActGelu) slope(kActGelu);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[0][u][i] = f2_fma(G[u][i], v[u][i], acc[0][u][i]);
                        if constexpr (kBias) acc[2][u][i] = f2_add(acc[2][u][i], G[u][i]);
                        G[u][i] = f2_mul(G[u][i], w[i]);
                        s0 = f2_fma(G[u][i], v[u][i], s0);
                        if constexpr (kMean) s1 = f2_add(s1, G[u][i]);
                    }
                }
                float s[kMean ? 2 : 1];
                s[0] = f2_sum(s0);
                if constexpr (kMean) s[1] = f2_sum(s1);
                int turn = 0;
                row_sum<TPR, kMean ? 2 : 1>(s, nullptr, turn);
                const f2 a = f2_all(-s[0] * p.inv_c), r2 = f2_all(rstd);
                f2 mean = f2_all(0.0f);
                if constexpr (kMean) mean = f2_all(p.pre == kNormLayer ? -s[1] * p.inv_c : 0.0f);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    f2 g[4];
                    tile_unit<T, V, TPR>(g, in + 2 * sh.cap, u, lane, C, ok && p.dh_out != nullptr);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        G[u][i] = f2_fma(r2, f2_fma(v[u][i], a, kMean ? f2_add(G[u][i], mean) : G[u][i]),
                                         g[i]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    tile_unit<T, V, TPR>(G[u], in + 2 * sh.cap, u, lane, C, ok);
            }
            if (p.dh != nullptr && ok && fits(p.dh, at))
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.dh) + at,
                                 unit_c0<V>(u, lane, TPR), TPR, C);
            if (has_b) {
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    tile_unit<T, V, TPR>(v[u], in + 3 * sh.cap, u, lane, C, ok);
                float rstd = 1.0f;
                if (p.post != kNormNone)
                    rstd = normalise2<V, TPR, NU>(v, kMean ? p.post : kNormRms, lane, C, p.eps,
                                                  p.inv_c);
                f2 s0 = f2_all(0.0f), s1 = f2_all(0.0f);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    f2 g[4];
                    vec8(g, vecs + 2 * L, V, unit_c0<V>(u, lane, TPR), TPR);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[1][u][i] = f2_fma(G[u][i], v[u][i], acc[1][u][i]);
                        // (past C, G may hold a row's mean: v and g are 0 there, and the
                        // sums of those columns are not written)
                        if constexpr (kBias) acc[3][u][i] = f2_add(acc[3][u][i], G[u][i]);
                        G[u][i] = f2_mul(G[u][i], g[i]);
                        s0 = f2_fma(G[u][i], v[u][i], s0);
                        if constexpr (kMean) s1 = f2_add(s1, G[u][i]);
                    }
                }
                if (p.db != nullptr) {
                    if (p.post != kNormNone) {
                        float s[kMean ? 2 : 1];
                        s[0] = f2_sum(s0);
                        if constexpr (kMean) s[1] = f2_sum(s1);
                        int turn = 0;
                        row_sum<TPR, kMean ? 2 : 1>(s, nullptr, turn);
                        const f2 a = f2_all(-s[0] * p.inv_c), r2 = f2_all(rstd);
                        f2 mean = f2_all(0.0f);
                        if constexpr (kMean) mean = f2_all(p.post == kNormLayer ? -s[1] * p.inv_c : 0.0f);
#pragma unroll
                        for (int u = 0; u < NU; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                G[u][i] = f2_mul(r2, f2_fma(v[u][i], a,
                                                            kMean ? f2_add(G[u][i], mean) : G[u][i]));
                    }
                    if (ok && fits(p.db, at))
#pragma unroll
                        for (int u = 0; u < NU; ++u)
                            store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.db) + at,
                                         unit_c0<V>(u, lane, TPR), TPR, C);
                }
            }
        }
        __syncthreads();  // every thread is done with the stage
        if (threadIdx.x == 0 && live) {
            const long long nt = t + (long long)sh.stages * p.blocks_per_group;
            if (nt < tiles)
                tile_issue<nT>(span(nt), src, stage, sh.cap, smem_u32(&full[st]), tensor);
        }
        if (++st == sh.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    if (!__syncthreads_and(waits == sh.stages)) return;  // a wait ran out
    float sums[kQ][NU][8];
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_get(acc[q][u][i], sums[q][u][2 * i], sums[q][u][2 * i + 1]);
    // (the ring is idle: every copy was waited for)
    store_colsums<V, TPR, NU, kQ>(p, sums, lane, TPR, reinterpret_cast<float*>(ring));
}

struct NormFin {
    const float* part;
    float* part_out;  // the group's sums, at its first slot (several groups)
    const void *gate, *post_w, *post_bias;
    void *dgate, *dpost_w, *dpost_bias, *dpre_w, *dpre_bias;
    long long groups, slots;
    int blocks_per_group, C, has_bias, has_b;
    float scale;
};

template <typename T>
__device__ __forceinline__ void put(void* dst, long long i, float v) {
    if (dst == nullptr) return;
    if constexpr (sizeof(T) == 2) static_cast<T*>(dst)[i] = __float2bfloat16_rn(v);
    else static_cast<T*>(dst)[i] = v;
}
template <typename T>
__device__ __forceinline__ float get(const void* src, long long i, float otherwise) {
    return src == nullptr ? otherwise : (float)static_cast<const T*>(src)[i];
}

// Sums over `n` partial rows, `stride` rows apart, of column c of the nq
// quantities: 8 columns a block (few columns leave few blocks, so a block's 128
// thread rows go down the partials), in a fixed order; every thread of a column
// has them.
constexpr int kFinCols = 8, kFinRows = 128;
__device__ __forceinline__ void fin_sums(const float* src, long long slots, int nq, long long n,
                                         long long stride, int c, int C, float (&s)[4],
                                         float (*buf)[32][kFinCols]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = 0.0f;
    if (c < C) {
#pragma unroll 2
        for (long long i = threadIdx.y; i < n; i += kFinRows)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < nq && index_ok(&g_block_status, i * stride, slots))
                    s[q] += src[(q * slots + i * stride) * C + c];
    }
    const int t = threadIdx.y * kFinCols + threadIdx.x;  // a warp: 4 rows of 8 columns
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        s[q] += __shfl_xor_sync(0xffffffffu, s[q], 8);
        s[q] += __shfl_xor_sync(0xffffffffu, s[q], 16);
        if ((t & 31) < kFinCols) buf[q][t >> 5][t & 31] = s[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        s[q] = 0.0f;
        if (threadIdx.y == 0)
#pragma unroll
            for (int i = 0; i < 32; ++i) s[q] += buf[q][i][threadIdx.x];
    }
}

// Block (column block, gate group): the group's sums over its blocks'
// partials; dgate; with one group the other parameter gradients too, with
// several the group's terms of them go to its first slot for the next launch.
template <typename T>
__global__ void __launch_bounds__(1024) norm_fin_group_kernel(const __grid_constant__ NormFin p) {
    __shared__ float buf[4][32][kFinCols];
    const int c = blockIdx.x * kFinCols + threadIdx.x, C = p.C, nq = p.has_bias ? 4 : 2;
    for (long long g = blockIdx.y; g < p.groups; g += gridDim.y) {
        float s[4];
        fin_sums(p.part + g * p.blocks_per_group * C, p.slots, nq, p.blocks_per_group, 1, c, C, s,
                 buf);
        if (threadIdx.y != 0 || c >= C) continue;
        if (p.has_b) {
            const float w = get<T>(p.post_w, c, 1.0f), b = get<T>(p.post_bias, c, 0.0f);
            put<T>(p.dgate, g * C + c, p.scale * (w * s[1] + b * s[3]));
            const float gs = p.scale * get<T>(p.gate, g * C + c, 1.0f);
            s[1] *= gs;
            s[3] *= gs;
        }
        if (p.groups == 1) {
            put<T>(p.dpre_w, c, s[0]);
            put<T>(p.dpost_w, c, s[1]);
            put<T>(p.dpre_bias, c, s[2]);
            put<T>(p.dpost_bias, c, s[3]);
        } else {
            for (int q = 0; q < nq && index_ok(&g_block_status, g * p.blocks_per_group, p.slots); ++q)
                p.part_out[((long long)q * p.slots + g * p.blocks_per_group) * C + c] = s[q];
        }
    }
}

// Several gate groups: the sums of the groups' terms.
template <typename T>
__global__ void __launch_bounds__(1024) norm_fin_all_kernel(const __grid_constant__ NormFin p) {
    __shared__ float buf[4][32][kFinCols];
    const int c = blockIdx.x * kFinCols + threadIdx.x;
    float s[4];
    fin_sums(p.part, p.slots, p.has_bias ? 4 : 2, p.groups, p.blocks_per_group, c, p.C, s, buf);
    if (threadIdx.y != 0 || c >= p.C) return;
    put<T>(p.dpre_w, c, s[0]);
    put<T>(p.dpost_w, c, s[1]);
    if (!p.has_bias) return;
    put<T>(p.dpre_bias, c, s[2]);
    put<T>(p.dpost_bias, c, s[3]);
}

}  // namespace ccv3d
