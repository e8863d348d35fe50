// pointwise_simt.cuh -- the 1x1x1 convolution on FFMA: the fp32 contract (IEEE
// fp32, no TF32), single rows, and the passes around the product.
//
// The product of every direction is D(m, n) = sum_k A(m, k) B(n, k) with the
// operands read in place: forward A = x, B = w (both contiguous along k), dx
// A = dP (along k), B = w (along n), dw A = dP, B = x (both along m and n).
#pragma once
#include "elem.cuh"

namespace ccv3d {

// Epilogue of a forward product, or the fp32 partials of a split reduction.
struct PwOut {
    const void *bias, *residual;
    void *out, *pre;
    float* partial;   // not NULL: D goes to partial[split][M][N] and nothing else
    long long M;
    int N, act;
};

struct PwSimt {
    const void *A, *B;
    long long sam, sak, sbn, sbk;  // element strides; one of each pair is 1
    long long M, K;
    int N, splits, vec;  // vec: rows of both operands are 16-byte multiples
    long long k_per_split;
    PwOut o;
};

template <typename T>
__device__ __forceinline__ void pw_store(const PwOut& o, long long m, int n, float u) {
    const long long at = m * o.N + n;
    if (!in_bounds(&g_block_status, static_cast<T*>(o.out) + at, sizeof(T), o.out,
                   o.M * o.N * (long long)sizeof(T)))
        return;
    if (o.bias != nullptr) u += (float)static_cast<const T*>(o.bias)[n];
    if (o.pre != nullptr) static_cast<T*>(o.pre)[at] = (T)u;
    u = act_of<T>(u, o.act);
    if (o.residual != nullptr) u += (float)static_cast<const T*>(o.residual)[at];
    static_cast<T*>(o.out)[at] = (T)u;
}

constexpr int kPwK = 16, kPwPad = 4;

// kV operand values of a thread: along k (row r, k0 .. k0 + kV - 1) or along the
// row index (k, r0 .. ).  R: rows of the tile (256 threads fetch R x 16).
template <typename T, bool KMAJOR, int R>
__device__ __forceinline__ void pw_fetch(float (&v)[R / 16], const T* base, long long s_row,
                                         long long s_k, long long row0, long long rows,
                                         long long k0, long long k1, int tid, bool vec) {
    constexpr int kV = R / 16, kPer = 16 / kV;  // threads along a row's 16 k
    const long long r = KMAJOR ? row0 + tid / kPer : row0 + (tid & 15) * kV;
    const long long k = KMAJOR ? k0 + tid % kPer * kV : k0 + (tid >> 4);
    // (s_row = 1 or s_k = 1 along the contiguous direction)
    const T* p = base + (KMAJOR ? r * s_row + k : k * s_k + r);
    const bool whole = KMAJOR ? r < rows && k + kV <= k1 : k < k1 && r + kV <= rows;
    if (whole && vec) {
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + i);
            v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool in = KMAJOR ? r < rows && k + i < k1 : k < k1 && r + i < rows;
            v[i] = in ? (float)p[i] : 0.0f;
        }
    }
}

template <bool KMAJOR, int R>
__device__ __forceinline__ void pw_put(float (*s)[R + kPwPad], const float (&v)[R / 16], int tid) {
    constexpr int kV = R / 16, kPer = 16 / kV;
    if constexpr (KMAJOR) {
#pragma unroll
        for (int i = 0; i < kV; ++i) s[tid % kPer * kV + i][tid / kPer] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < kV; i += 4)
            *reinterpret_cast<float4*>(&s[tid >> 4][(tid & 15) * kV + i]) =
                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// S x S tile a block (S = 128 or 64), S/16 x S/16 values a thread, k in steps of
// 16 through two shared-memory buffers; the next step's operands wait in
// registers.  128 has the better ratio of FMAs to shared-memory reads; 64 is
// for products whose edges or few tiles would idle much of it.
template <typename T, bool AK, bool BK, int S>
__global__ void __launch_bounds__(256) pw_simt_kernel(const __grid_constant__ PwSimt p) {
    constexpr int kT = S / 16, kH = kT / 4;
    __shared__ float sa[2][kPwK][S + kPwPad], sb[2][kPwK][S + kPwPad];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int tiles_n = (p.N + S - 1) / S;
    const long long tile = blockIdx.x;
    const long long m0 = tile / tiles_n * S;
    const int n0 = (int)(tile % tiles_n) * S;
    const long long kb = (long long)blockIdx.z * p.k_per_split;
    const long long ke = kb + p.k_per_split < p.K ? kb + p.k_per_split : p.K;
    const T *A = static_cast<const T*>(p.A), *B = static_cast<const T*>(p.B);
    float acc[kT][kT] = {}, va[kT], vb[kT];
    pw_fetch<T, AK, S>(va, A, p.sam, p.sak, m0, p.M, kb, ke, tid, p.vec);
    pw_fetch<T, BK, S>(vb, B, p.sbn, p.sbk, n0, p.N, kb, ke, tid, p.vec);
    int cur = 0;
    for (long long k = kb; k < ke; k += kPwK, cur ^= 1) {
        pw_put<AK, S>(sa[cur], va, tid);
        pw_put<BK, S>(sb[cur], vb, tid);
        __syncthreads();
        if (k + kPwK < ke) {
            pw_fetch<T, AK, S>(va, A, p.sam, p.sak, m0, p.M, k + kPwK, ke, tid, p.vec);
            pw_fetch<T, BK, S>(vb, B, p.sbn, p.sbk, n0, p.N, k + kPwK, ke, tid, p.vec);
        }
#pragma unroll
        for (int kk = 0; kk < kPwK; ++kk) {
            float a[kT], b[kT];
#pragma unroll
            for (int h = 0; h < kH; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(&sa[cur][kk][h * 64 + ty * 4]);
                const float4 y = *reinterpret_cast<const float4*>(&sb[cur][kk][h * 64 + tx * 4]);
                a[h * 4] = x.x; a[h * 4 + 1] = x.y; a[h * 4 + 2] = x.z; a[h * 4 + 3] = x.w;
                b[h * 4] = y.x; b[h * 4 + 1] = y.y; b[h * 4 + 2] = y.z; b[h * 4 + 3] = y.w;
            }
#pragma unroll
            for (int i = 0; i < kT; ++i)
#pragma unroll
                for (int j = 0; j < kT; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        // (one barrier a step: the next step writes the other buffer, whose
        // readers passed this step's barrier)
    }
    // Epilogue: everything is read before the first store (out may be the
    // residual, so the compiler keeps a load after a store where it stands:
    // one by one, 64 residual loads waited out 64 memory latencies).
    const PwOut& o = p.o;
    auto row = [&](int i) { return m0 + (i >> 2) * 64 + ty * 4 + (i & 3); };
    auto col = [&](int j) { return n0 + (j >> 2) * 64 + tx * 4 + (j & 3); };
    if (o.partial != nullptr) {
#pragma unroll
        for (int i = 0; i < kT; ++i)
#pragma unroll
            for (int j = 0; j < kT; ++j)
                if (row(i) < p.M && col(j) < p.N)
                    o.partial[((long long)blockIdx.z * p.M + row(i)) * p.N + col(j)] = acc[i][j];
        return;
    }
    const T *bias = static_cast<const T*>(o.bias), *residual = static_cast<const T*>(o.residual);
    float res[kT][kT];
    if (residual != nullptr)
#pragma unroll
        for (int i = 0; i < kT; ++i)
#pragma unroll
            for (int j = 0; j < kT; ++j)
                res[i][j] = row(i) < p.M && col(j) < p.N ? (float)residual[row(i) * o.N + col(j)] : 0.0f;
    if (bias != nullptr)
#pragma unroll
        for (int j = 0; j < kT; ++j) {
            const float b = col(j) < p.N ? (float)bias[col(j)] : 0.0f;
#pragma unroll
            for (int i = 0; i < kT; ++i) acc[i][j] += b;
        }
    const long long bytes = o.M * o.N * (long long)sizeof(T);
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int j = 0; j < kT; ++j) {
            if (row(i) >= p.M || col(j) >= p.N) continue;
            T* out = static_cast<T*>(o.out) + row(i) * o.N + col(j);
            if (!in_bounds(&g_block_status, out, sizeof(T), o.out, bytes)) continue;
            if (o.pre != nullptr) static_cast<T*>(o.pre)[row(i) * o.N + col(j)] = (T)acc[i][j];
            float u = act_of<T>(acc[i][j], o.act);
            if (residual != nullptr) u += res[i][j];
            *out = (T)u;
        }
}

// The partials of a split reduction, added in order, through the epilogue.
template <typename T>
__global__ void __launch_bounds__(256) pw_join_kernel(const float* partial, int splits, int ldp,
                                                      const __grid_constant__ PwOut o) {
    const long long total = o.M * o.N, step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const long long m = i / o.N;
        const int n = (int)(i - m * o.N);
        float u = 0.0f;
        for (int s = 0; s < splits; ++s) u += partial[(s * o.M + m) * ldp + n];
        pw_store<T>(o, m, n, u);
    }
}

// Few rows (M <= kPwFewRows): bound by reading w once.  A warp takes CPW rows
// of w (output channels) and all rows of x; its lanes split k, eight values a
// load.  CPW = 1 for one row keeps the most warps loading; with several rows,
// four output channels share each load of x.
constexpr int kPwFewRows = 8;

template <typename T, int MR, int CPW, bool V>
__global__ void __launch_bounds__(128) pw_rows_kernel(const T* x, const T* w, int K,
                                                      const __grid_constant__ PwOut o) {
    const int lane = threadIdx.x & 31;
    const int n0 = (int)((blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * CPW);
    if (n0 >= o.N) return;
    float acc[CPW][MR] = {};
    const int M = (int)o.M;
    const int kstep = 32 * 8;
#pragma unroll 4
    for (int k = 0; k < K; k += kstep) {
        const int c0 = V ? k + lane * 8 : k + lane;
        Raw8<T, V> rw[CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            if (n0 + c < o.N) load8<T, V>(rw[c], w + (long long)(n0 + c) * K, c0, 32, K);
            else zero8<T, V>(rw[c]);
        }
        float f[CPW][8];
#pragma unroll
        for (int c = 0; c < CPW; ++c) unpack8<T, V>(rw[c], f[c]);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if (m >= M) break;
            Raw8<T, V> rx;
            float g[8];
            load8<T, V>(rx, x + (long long)m * K, c0, 32, K);
            unpack8<T, V>(rx, g);
#pragma unroll
            for (int c = 0; c < CPW; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][m] = fmaf(f[c][i], g[i], acc[c][m]);
        }
    }
#pragma unroll
    for (int c = 0; c < CPW; ++c)
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            float v = acc[c][m];
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
            // one lane per value
            if (lane == ((c * MR + m) & 31) && m < M && n0 + c < o.N)
                pw_store<T>(o, m, n0 + c, v);
        }
}

// dP = dout act'(pre) into dp (rows of ldp elements, those past N zeros), and
// the column sums of dP over this block's rows (blockIdx.y-th chunk) into
// colsum[chunk][N].  dp or colsum may be NULL.  tpr threads share a row.
template <typename T, bool V>
__global__ void __launch_bounds__(256) pw_dact_kernel(const T* pre, const T* dout, T* dp,
                                                      float* colsum, long long M, int N, int ldp,
                                                      int act, int tpr, long long chunk) {
    __shared__ float buf[256 * 8];
    const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rows = blockDim.x / tpr;
    const int cbase = blockIdx.x * tpr * 8;
    const int c0 = V ? cbase + lane * 8 : cbase + lane;
    const long long r0 = (long long)blockIdx.y * chunk;
    const long long r1 = r0 + chunk < M ? r0 + chunk : M;
    float acc[8] = {};
    // four rows at a time, all loads before the stores (dp could be any memory
    // to the compiler, which would not move a load before a store)
    constexpr int kU = 4;
    for (long long r = r0 + sub; r < r1; r += (long long)kU * rows) {
        Raw8<T, V> rd[kU], rp[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            const long long at = r + (long long)j * rows;
            zero8<T, V>(rd[j]);
            zero8<T, V>(rp[j]);
            if (at < r1) {
                load8<T, V>(rd[j], dout + at * N, c0, tpr, N);
                if (pre != nullptr) load8<T, V>(rp[j], pre + at * N, c0, tpr, N);
            }
        }
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            const long long at = r + (long long)j * rows;
            float d[8], u[8];
            unpack8<T, V>(rd[j], d);
            if (pre != nullptr) {
                unpack8<T, V>(rp[j], u);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] *= act_grad_of<T>(u[i], act);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += d[i];
            if (dp != nullptr && at < r1) store8<T, V>(pack8<T, V>(d), dp + at * ldp, c0, tpr, ldp);
        }
    }
    if (colsum == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[(sub * tpr + lane) * 8 + i] = acc[i];
    __syncthreads();
    for (int j = threadIdx.x; j < tpr * 8; j += blockDim.x) {
        float a = 0.0f;
        for (int s = 0; s < rows; ++s) a += buf[s * tpr * 8 + j];
        const int l = j >> 3, i = j & 7, c = V ? cbase + l * 8 + i : cbase + l + i * tpr;
        if (c < N) colsum[(long long)blockIdx.y * N + c] = a;
    }
}

// Columns' partial sums -> dst, in order.
template <typename T>
__global__ void __launch_bounds__(1024) pw_colsum_kernel(const float* part, int chunks, int N,
                                                         T* dst) {
    __shared__ float buf[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.0f;
    if (c < N)
        for (int i = threadIdx.y; i < chunks; i += 32) a += part[(long long)i * N + c];
    buf[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < N) {
        a = 0.0f;
        for (int i = 0; i < 32; ++i) a += buf[i][threadIdx.x];
        dst[c] = (T)a;
    }
}

}  // namespace ccv3d
