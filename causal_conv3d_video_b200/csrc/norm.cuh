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
// HBM-bound (2 to 4 tensors moved forward, 4 to 6 backward, about 20 flops
// an element): a row is read once and stays in registers.  TPR threads share
// a row (a power of two within a warp, or the whole block for wide rows), so
// that the row statistics are a few shuffles and each thread keeps a fixed
// set of channels, whose weights it reads once per block and whose column
// sums it owns.
#pragma once
#include "elem.cuh"

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

// v = v * w + bias over a unit; a NULL w is ones, a NULL bias zeros.
template <typename T, bool V>
__device__ __forceinline__ void affine8(float (&v)[8], const T* w, const T* bias, int c0,
                                        int step, int C) {
    if (w != nullptr) {
        Raw8<T, V> r;
        float f[8];
        load8<T, V>(r, w, c0, step, C);
        unpack8<T, V>(r, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f[i];
    }
    if (bias != nullptr) {
        Raw8<T, V> r;
        float f[8];
        load8<T, V>(r, bias, c0, step, C);
        unpack8<T, V>(r, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
}

// Rows wider than a warp's share: at most 512 threads a row, so that a thread
// may hold 128 registers.
constexpr int norm_threads(int tpr) { return tpr == 0 ? 512 : 128; }

template <typename T, bool V, int TPR, int NU>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_fwd_kernel(const __grid_constant__ NormFwd p) {
    __shared__ float red[2][4][32];
    int turn = 0;
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int lane = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % tpr;
    const int rpb = (int)blockDim.x / tpr;
    const int C = p.C;
    const long long tensor = p.rows * C * (long long)sizeof(T);
    for (long long base = (long long)blockIdx.x * rpb; base < p.rows;
         base += (long long)gridDim.x * rpb) {
        const long long row = base + (int)threadIdx.x / tpr;
        const bool valid = row < p.rows;  // threads of a tail row still take part in the shuffles
        const long long at = (valid ? row : 0) * C;
        const T* h = static_cast<const T*>(p.h) + at;
        const bool ok = valid && in_bounds(&g_block_status, h, (long long)C * sizeof(T), p.h, tensor);
        Raw8<T, V> rh[NU], rb[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
            if (ok) load8<T, V>(rh[u], h, c0, tpr, C);
            else zero8<T, V>(rh[u]);
            if (p.b != nullptr) {
                if (ok) load8<T, V>(rb[u], static_cast<const T*>(p.b) + at, c0, tpr, C);
                else zero8<T, V>(rb[u]);
            }
        }
        float v[NU][8];
#pragma unroll
        for (int u = 0; u < NU; ++u) unpack8<T, V>(rh[u], v[u]);
        if (p.b != nullptr) {
            float m[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) unpack8<T, V>(rb[u], m[u]);
            if (p.post != kNormNone)
                normalise<V, TPR, NU>(m, p.post, lane, tpr, C, p.eps, p.inv_c, red, turn);
            const T* gate = p.gate == nullptr || !valid
                                ? static_cast<const T*>(p.gate)
                                : static_cast<const T*>(p.gate) + row / p.gate_rows * C;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c0 = unit_c0<V>(u, lane, tpr);
                affine8<T, V>(m[u], static_cast<const T*>(p.post_w),
                              static_cast<const T*>(p.post_bias), c0, tpr, C);
                affine8<T, V>(m[u], gate, nullptr, c0, tpr, C);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = fmaf(p.scale, m[u][i], v[u][i]);
                const Raw8<T, V> r = pack8<T, V>(v[u]);
                if (ok) store8<T, V>(r, static_cast<T*>(p.h_out) + at, c0, tpr, C);
                unpack8<T, V>(r, v[u]);  // the stored value is what the norm reads
            }
        }
        if (p.y != nullptr) {
            normalise<V, TPR, NU>(v, p.pre, lane, tpr, C, p.eps, p.inv_c, red, turn);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c0 = unit_c0<V>(u, lane, tpr);
                affine8<T, V>(v[u], static_cast<const T*>(p.pre_w),
                              static_cast<const T*>(p.pre_bias), c0, tpr, C);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = act_of<T>(v[u][i], p.act);
                if (ok) store8<T, V>(pack8<T, V>(v[u]), static_cast<T*>(p.y) + at, c0, tpr, C);
            }
        }
    }
}

// Gradients of the rows, and the column sums over this block's rows: block
// (group, j) takes every blocks_per_group-th step of the group's rows, from
// its j-th.  kBias: the sums of du and G are wanted too (a bias is there).
template <typename T, bool V, int TPR, int NU, bool kBias>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_bwd_kernel(const __grid_constant__ NormBwd p) {
    __shared__ float red[2][4][32];
    extern __shared__ float colbuf[];  // TPR > 0: [warps][C] for the block's column sums
    int turn = 0;
    constexpr int kQ = kBias ? 4 : 2;
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int lane = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % tpr;
    const int rpb = (int)blockDim.x / tpr;
    const int C = p.C;
    const long long tensor = p.rows * C * (long long)sizeof(T);
    float acc[kQ][NU][8];
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[q][u][i] = 0.0f;
    const long long group = blockIdx.x / p.blocks_per_group;
    const int part_of = (int)(blockIdx.x % p.blocks_per_group);
    const long long row0 = group * p.group_rows, row1 = row0 + p.group_rows;
    const T* gate = p.gate == nullptr ? nullptr : static_cast<const T*>(p.gate) + group * C;
    const T* pre_w = static_cast<const T*>(p.pre_w);
    const T* pre_bias = static_cast<const T*>(p.pre_bias);
    const T* post_w = static_cast<const T*>(p.post_w);
    for (long long base = row0 + (long long)part_of * rpb; base < row1;
         base += (long long)p.blocks_per_group * rpb) {
        const long long row = base + (int)threadIdx.x / tpr;
        const bool valid = row < row1;
        const long long at = (valid ? row : row0) * C;
        const T* h = static_cast<const T*>(p.h) + at;
        const bool ok = valid && in_bounds(&g_block_status, h, (long long)C * sizeof(T), p.h, tensor);
        // every load of the row is issued before the first of them is used
        Raw8<T, V> rh[NU], ry[NU], rg[NU], rb[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c0 = unit_c0<V>(u, lane, tpr);
            zero8<T, V>(rh[u]); zero8<T, V>(ry[u]); zero8<T, V>(rg[u]); zero8<T, V>(rb[u]);
            if (ok) {
                if (p.dy != nullptr) {
                    load8<T, V>(rh[u], h, c0, tpr, C);
                    load8<T, V>(ry[u], static_cast<const T*>(p.dy) + at, c0, tpr, C);
                }
                if (p.dh_out != nullptr)
                    load8<T, V>(rg[u], static_cast<const T*>(p.dh_out) + at, c0, tpr, C);
                if (p.b != nullptr)
                    load8<T, V>(rb[u], static_cast<const T*>(p.b) + at, c0, tpr, C);
            }
        }
        float G[NU][8];
#pragma unroll
        for (int u = 0; u < NU; ++u) unpack8<T, V>(rg[u], G[u]);
        if (p.dy != nullptr) {
            float n[NU][8], d[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) unpack8<T, V>(rh[u], n[u]);
            const float rstd =
                normalise<V, TPR, NU>(n, p.pre, lane, tpr, C, p.eps, p.inv_c, red, turn);
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c0 = unit_c0<V>(u, lane, tpr);
                unpack8<T, V>(ry[u], d[u]);
                if (p.act != kActNone) {
                    float a[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = n[u][i];
                    affine8<T, V>(a, pre_w, pre_bias, c0, tpr, C);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[u][i] *= act_grad_of<T>(a[i], p.act);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[0][u][i] = fmaf(d[u][i], n[u][i], acc[0][u][i]);
                    if constexpr (kBias) acc[2][u][i] += d[u][i];
                }
                affine8<T, V>(d[u], pre_w, nullptr, c0, tpr, C);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] = fmaf(d[u][i], n[u][i], s[0]);
                    s[1] += d[u][i];
                }
            }
            row_sum<TPR, 2>(s, red, turn);
            const float a = s[0] * p.inv_c, b = p.pre == kNormLayer ? s[1] * p.inv_c : 0.0f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[u][i] += rstd * (d[u][i] - b - n[u][i] * a);
        }
        if (p.dh != nullptr)
#pragma unroll
            for (int u = 0; u < NU; ++u)
                if (ok)
                    store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.dh) + at,
                                 unit_c0<V>(u, lane, tpr), tpr, C);
        if (p.b != nullptr) {
            float m[NU][8];
#pragma unroll
            for (int u = 0; u < NU; ++u) unpack8<T, V>(rb[u], m[u]);
            float rstd = 1.0f;
            if (p.post != kNormNone)
                rstd = normalise<V, TPR, NU>(m, p.post, lane, tpr, C, p.eps, p.inv_c, red, turn);
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c0 = unit_c0<V>(u, lane, tpr);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!ok || (V ? c0 : c0 + i * tpr) >= C) G[u][i] = 0.0f;
                    acc[1][u][i] = fmaf(G[u][i], m[u][i], acc[1][u][i]);
                    if constexpr (kBias) acc[3][u][i] += G[u][i];
                    G[u][i] *= p.scale;
                }
                affine8<T, V>(G[u], gate, nullptr, c0, tpr, C);
                affine8<T, V>(G[u], post_w, nullptr, c0, tpr, C);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] = fmaf(G[u][i], m[u][i], s[0]);
                    s[1] += G[u][i];
                }
            }
            if (p.db != nullptr) {
                if (p.post != kNormNone) {
                    row_sum<TPR, 2>(s, red, turn);
                    const float a = s[0] * p.inv_c;
                    const float b = p.post == kNormLayer ? s[1] * p.inv_c : 0.0f;
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            G[u][i] = rstd * (G[u][i] - b - m[u][i] * a);
                }
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    if (ok)
                        store8<T, V>(pack8<T, V>(G[u]), static_cast<T*>(p.db) + at,
                                     unit_c0<V>(u, lane, tpr), tpr, C);
            }
        }
    }
    // ---- this block's column sums -> its slot of the partials
    if (p.part == nullptr) return;
    const long long part_bytes = (long long)kQ * p.slots * C * 4;
    for (int q = 0; q < kQ; ++q) {
        float* out = p.part + ((long long)q * p.slots + blockIdx.x) * C;
        const bool fits = in_bounds(&g_block_status, out, (long long)C * 4, p.part, part_bytes);
        if constexpr (TPR == 0) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c0 = unit_c0<V>(u, lane, tpr), c = V ? c0 + i : c0 + i * tpr;
                    float a = 0.0f;
#pragma unroll
                    for (int k = 0; k < kQ; ++k) a = k == q ? acc[k][u][i] : a;
                    if (c < C && fits) out[c] = a;
                }
        } else {
            // rows of one warp by shuffles, then the warps through shared memory
            const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
            __syncthreads();
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a = 0.0f;
#pragma unroll
                    for (int k = 0; k < kQ; ++k) a = k == q ? acc[k][u][i] : a;
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

// Sum over `n` partial rows, `stride` rows apart, of column c, by the block's
// 32 rows of threads (threadIdx.y), in a fixed order.
__device__ __forceinline__ float fin_sum(const float* src, long long n, long long stride, int c,
                                         int C, float (*buf)[33]) {
    float a = 0.0f;
    if (c < C)
        for (long long i = threadIdx.y; i < n; i += 32) a += src[i * stride * C + c];
    __syncthreads();
    buf[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = 0.0f;
    if (threadIdx.y == 0)
        for (int i = 0; i < 32; ++i) a += buf[i][threadIdx.x];
    return a;
}

// Block (column block, gate group): the group's sums over its blocks'
// partials; dgate; with one group the other parameter gradients too, with
// several the group's terms of them go to its first slot for the next launch.
template <typename T>
__global__ void norm_fin_group_kernel(const __grid_constant__ NormFin p) {
    __shared__ float buf[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, C = p.C;
    for (long long g = blockIdx.y; g < p.groups; g += gridDim.y) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const int nq = p.has_bias ? 4 : 2;
        for (int q = 0; q < nq; ++q)
            s[q] = fin_sum(p.part + ((long long)q * p.slots + g * p.blocks_per_group) * C,
                           p.blocks_per_group, 1, c, C, buf);
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
            for (int q = 0; q < nq; ++q)
                p.part_out[((long long)q * p.slots + g * p.blocks_per_group) * C + c] = s[q];
        }
    }
}

// Several gate groups: the sums of the groups' terms.
template <typename T>
__global__ void norm_fin_all_kernel(const __grid_constant__ NormFin p) {
    __shared__ float buf[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, C = p.C;
    void* dst[4] = {p.dpre_w, p.dpost_w, p.dpre_bias, p.dpost_bias};
    for (int q = 0; q < (p.has_bias ? 4 : 2); ++q) {
        if (dst[q] == nullptr) continue;
        const float s = fin_sum(p.part + (long long)q * p.slots * C, p.groups, p.blocks_per_group,
                                c, C, buf);
        if (threadIdx.y == 0 && c < C) put<T>(dst[q], c, s);
    }
}

}  // namespace ccv3d
