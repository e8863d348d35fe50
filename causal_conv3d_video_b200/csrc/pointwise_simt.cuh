// pointwise_simt.cuh -- the 1x1x1 convolution on FFMA: the fp32 contract (IEEE
// fp32, no TF32), single rows, and the passes around the product.
//
// The product of every direction is D(m, n) = sum_k A(m, k) B(n, k) with the
// operands read in place: forward A = x, B = w (both contiguous along k), dx
// A = dP (along k), B = w (along n), dw A = dP, B = x (both along m and n).
#pragma once
#include "bulk.cuh"
#include "elem.cuh"
#include "params.h"

namespace ccv3d {

// Epilogue of a forward product, or the fp32 partials of a split reduction.
struct PwOut {
    const void *bias, *residual;
    void *out, *pre;
    float* partial;   // not NULL: D goes to partial[split][M][ldp] and nothing else
    long long M;
    int N, act;
};

struct PwSimt {
    const void *A, *B;
    long long sam, sak, sbn, sbk;  // element strides; one of each pair is 1
    long long M, K;
    int N, ldp, splits, vec;  // vec: rows of both operands are 16-byte multiples
    long long k_per_split;
    long long a_elems, b_elems;  // extents of A and B (checked build)
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
// Terms of one chain of FMAs.  Roundings add up along a chain like a random walk
// of steps up to 2^-24 of the running sum, so its error grows as the root of its
// length (3515 terms: 1.1e-6 off in the 2-norm).  Chains of 1024 stay near 6e-7,
// and their sums, added up apart, near that for a hundred thousand terms.
constexpr int kPwChain = 1024;

// A thread's part of an operand tile of R rows x 16 k: with 16-byte rows kV
// values along the contiguous direction, otherwise kV single ones, 16 rows
// apart, neighbouring threads along the contiguous direction (so that a warp's
// load covers whole sectors).  The part moves on by 16 k a step.
template <typename T, bool KMAJOR, int R>
struct PwFetch {
    // kPer threads along a row's 16 k (parts of under four values go singly: vec is false)
    static constexpr int kV = R / 16, kPer = 16 / kV;
    const T* p;
    long long step, next_row;
    int rows, k;  // rows there are from the thread's on; its k in a step
    bool vec;
    const T* base_;
    long long elems_;
    __device__ __forceinline__ PwFetch(const T* base, long long elems, long long s_row,
                                       long long s_k, long long row0, long long n_rows,
                                       long long k0, int tid, bool v)
        : vec(v), base_(base), elems_(elems) {
        const int r = v ? (KMAJOR ? tid / kPer : (tid & 15) * kV) : (KMAJOR ? tid >> 4 : tid & 15);
        k = v && KMAJOR ? tid % kPer * kV : (KMAJOR ? tid & 15 : tid >> 4);
        // (s_row = 1 or s_k = 1 along the contiguous direction)
        const long long sr = KMAJOR ? s_row : 1, sk = KMAJOR ? 1 : s_k;
        p = base + (row0 + r) * sr + (k0 + k) * sk;
        step = kPwK * sk;
        next_row = 16 * sr;
        const long long left = n_rows - row0 - r;
        rows = (int)(left <= 0 ? 0 : (left < R ? left : R));
    }
    __device__ __forceinline__ bool there(const T* q, int n) const {
        return in_bounds(&g_block_status, q, n * (long long)sizeof(T), base_,
                         elems_ * (long long)sizeof(T));
    }
    // The values of the next step, of which `left` k remain from its first on.
    __device__ __forceinline__ void operator()(float (&v)[kV], int left) {
        if (!vec) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                v[i] = k < left && 16 * i < rows && there(p + i * next_row, 1)
                           ? (float)p[i * next_row] : 0.0f;
        } else if (kV % 4 == 0 && (KMAJOR ? rows > 0 && left >= k + kV : left > k && rows >= kV) &&
                   there(p, kV)) {
#pragma unroll
            for (int i = 0; i + 3 < kV; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(p + i);
                v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                v[i] = (KMAJOR ? rows > 0 && k + i < left : k < left && i < rows) && there(p + i, 1)
                           ? (float)p[i] : 0.0f;
        }
        p += step;
    }
    __device__ __forceinline__ void put(float (*s)[R + kPwPad], const float (&v)[kV], int tid) const {
        if (!vec) {
#pragma unroll
            for (int i = 0; i < kV; ++i) s[k][(KMAJOR ? tid >> 4 : tid & 15) + 16 * i] = v[i];
        } else if constexpr (KMAJOR) {
#pragma unroll
            for (int i = 0; i < kV; ++i) s[tid % kPer * kV + i][tid / kPer] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i + 3 < kV; i += 4)
                *reinterpret_cast<float4*>(&s[tid >> 4][(tid & 15) * kV + i]) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
};

// SM x SN tile a block (128 x 128, 64 x 64, 128 x 32 or 32 x 128), k in steps of 16
// through two shared-memory buffers; the next step's operands wait in
// registers.  A thread has 4 rows by 4 columns of each SM/GM x SN/GN part.  The
// largest has the best ratio of FMAs to shared-memory reads, the others are for
// products whose edges or few tiles would idle much of it.  kChains: a block sums
// more than kPwChain terms; the sums are kept in dynamic shared memory, SM * SN
// floats, a thread's own places, to which the accumulators are added after every
// chain.  (A form of its own: with the test in it the loop of the others takes up
// to 6 % longer.)
template <typename T, bool AK, bool BK, int SM, int SN, bool kChains>
__global__ void __launch_bounds__(256, SM * SN == 128 * 128 ? 2 : 4) pw_simt_kernel(
    const __grid_constant__ PwSimt p) {
    constexpr int kTx = SN == 32 ? 8 : (SM == 32 ? 32 : 16), kTy = 256 / kTx;  // threads across, down
    constexpr int kHm = SM / (kTy * 4), kHn = SN / (kTx * 4);
    constexpr int kA = 2 * kPwK * (SM + kPwPad), kB = 2 * kPwK * (SN + kPwPad);
    typedef float SlabA[2][kPwK][SM + kPwPad];
    typedef float SlabB[2][kPwK][SN + kPwPad];
    __shared__ __align__(16) float smem[kA + kB];
    extern __shared__ __align__(16) float pw_sums[];
    SlabA& sa = *reinterpret_cast<SlabA*>(smem);
    SlabB& sb = *reinterpret_cast<SlabB*>(smem + kA);
    constexpr int kGm = kTy * 4, kGn = kTx * 4;  // rows and columns of a part
    static_assert(kGm * SN <= kA + kB, "a row of parts fits the operands' buffers");
    const int tid = threadIdx.x, tx = tid % kTx, ty = tid / kTx;
    const int tiles_n = (p.N + SN - 1) / SN;
    const long long tile = blockIdx.x;
    const long long m0 = tile / tiles_n * SM;
    const int n0 = (int)(tile % tiles_n) * SN;
    const long long kb = (long long)blockIdx.z * p.k_per_split;
    const long long ke = kb + p.k_per_split < p.K ? kb + p.k_per_split : p.K;
    const T *A = static_cast<const T*>(p.A), *B = static_cast<const T*>(p.B);
    // accumulators and b values as pairs: one instruction, two FMAs
    f2 acc[kHm * 4][kHn * 2];
#pragma unroll
    for (int i = 0; i < kHm * 4; ++i)
#pragma unroll
        for (int j = 0; j < kHn * 2; ++j) acc[i][j] = f2_all(0.0f);
    float va[SM / 16], vb[SN / 16];
    PwFetch<T, AK, SM> fa(A, p.a_elems, p.sam, p.sak, m0, p.M, kb, tid, p.vec && SM >= 64);
    PwFetch<T, BK, SN> fb(B, p.b_elems, p.sbn, p.sbk, n0, p.N, kb, tid, p.vec && SN >= 64);
    int left = (int)(ke - kb);
    fa(va, left);
    fb(vb, left);
    int cur = 0;
    // (16 bytes of each thread side by side)
    [[maybe_unused]] ulonglong2* sums = reinterpret_cast<ulonglong2*>(pw_sums) + tid;
    [[maybe_unused]] auto chain_ends = [&](bool add, bool store) {
#pragma unroll
        for (int i = 0; i < kHm * 4; ++i)
#pragma unroll
            for (int j = 0; j < kHn; ++j) {
                ulonglong2& at = sums[(i * kHn + j) * 256];
                f2 &a = acc[i][2 * j], &b = acc[i][2 * j + 1];
                if (add) {
                    const ulonglong2 t = at;
                    a = f2_add(a, t.x);
                    b = f2_add(b, t.y);
                }
                if (store) {
                    at = make_ulonglong2(a, b);
                    a = b = f2_all(0.0f);
                }
            }
    };
    [[maybe_unused]] int whole = left;  // what was left at the end of the last whole chain
    for (; left > 0; left -= kPwK, cur ^= 1) {
        fa.put(sa[cur], va, tid);
        fb.put(sb[cur], vb, tid);
        __syncthreads();
        if (left > kPwK) {
            fa(va, left - kPwK);
            fb(vb, left - kPwK);
        }
#pragma unroll
        for (int kk = 0; kk < kPwK; ++kk) {
            float a[kHm * 4];
            f2 b[kHn * 2];
#pragma unroll
            for (int h = 0; h < kHm; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(&sa[cur][kk][h * kGm + ty * 4]);
                a[h * 4] = x.x; a[h * 4 + 1] = x.y; a[h * 4 + 2] = x.z; a[h * 4 + 3] = x.w;
            }
#pragma unroll
            for (int h = 0; h < kHn; ++h) {
                const ulonglong2 y =
                    *reinterpret_cast<const ulonglong2*>(&sb[cur][kk][h * kGn + tx * 4]);
                b[h * 2] = y.x;
                b[h * 2 + 1] = y.y;
            }
#pragma unroll
            for (int i = 0; i < kHm * 4; ++i) {
                const f2 a2 = f2_all(a[i]);
#pragma unroll
                for (int j = 0; j < kHn * 2; ++j) acc[i][j] = f2_fma(a2, b[j], acc[i][j]);
            }
        }
        // (one barrier a step: the next step writes the other buffer, whose
        // readers passed this step's barrier)
        if constexpr (kChains) {
            if (whole - left == kPwChain - kPwK && left > kPwK) {
                chain_ends(whole != (int)(ke - kb), true);
                whole = left - kPwK;
            }
        }
    }
    if constexpr (kChains)
        if (whole != (int)(ke - kb)) chain_ends(true, false);
    // Epilogue, a row of parts at a time through shared memory: the loop over
    // its values is then short (unrolled over the accumulators it outgrew the
    // instruction cache) and runs along the rows of out.  Four values' residuals
    // are read before their stores: out may be the residual, so the compiler
    // keeps a load after a store where it stands.
    const PwOut& o = p.o;
    const T *bias = static_cast<const T*>(o.bias), *residual = static_cast<const T*>(o.residual);
    const long long bytes = o.M * o.N * (long long)sizeof(T);
#pragma unroll
    for (int h = 0; h < kHm; ++h) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < kHn; ++g)
                *reinterpret_cast<ulonglong2*>(&smem[(ty * 4 + i) * SN + g * kGn + tx * 4]) =
                    make_ulonglong2(acc[h * 4 + i][g * 2], acc[h * 4 + i][g * 2 + 1]);
        __syncthreads();
        const long long mh = m0 + h * kGm;
        const int n = n0 + tid % SN;  // (256 is a multiple of SN: a thread's column)
        if (n >= p.N) continue;
        constexpr int kStep = 256 / SN;  // rows a pass
        if (o.partial != nullptr) {
            float* dst = o.partial + ((long long)blockIdx.z * p.M + mh) * p.ldp + n;
#pragma unroll 4
            for (int r = tid / SN; r < kGm; r += kStep)
                if (mh + r < p.M &&
                    in_bounds(&g_block_status, dst + (long long)r * p.ldp, 4, o.partial,
                              (long long)p.splits * p.M * p.ldp * 4))
                    dst[(long long)r * p.ldp] = smem[r * SN + tid % SN];
            continue;
        }
        const float b = bias != nullptr ? (float)bias[n] : 0.0f;
#pragma unroll 1
        for (int r = tid / SN; r < kGm; r += 4 * kStep) {
            float res[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long m = mh + r + j * kStep;
                res[j] = residual != nullptr && m < p.M &&
                                 in_bounds(&g_block_status, residual + m * o.N + n, sizeof(T), residual, bytes)
                             ? (float)residual[m * o.N + n] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long m = mh + r + j * kStep;
                T* out = static_cast<T*>(o.out) + m * o.N + n;
                if (m >= p.M || !in_bounds(&g_block_status, out, sizeof(T), o.out, bytes)) continue;
                const float u = smem[(r + j * kStep) * SN + tid % SN] + b;
                if (o.pre != nullptr) static_cast<T*>(o.pre)[m * o.N + n] = (T)u;
                *out = (T)(act_of<T>(u, o.act) + res[j]);
            }
        }
    }
}

// The partials of a split reduction, added in order, through the epilogue; four
// columns a thread (ldp, the partials' row, is a multiple of 4).
template <typename T>
__global__ void __launch_bounds__(256) pw_join_kernel(const float* partial, int splits, int ldp,
                                                      const __grid_constant__ PwOut o) {
    const int per = ldp / 4;
    const long long total = o.M * per, step = (long long)gridDim.x * blockDim.x;
    const T *bias = static_cast<const T*>(o.bias), *residual = static_cast<const T*>(o.residual);
    const long long bytes = o.M * o.N * (long long)sizeof(T);
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const long long m = i / per;
        const int n = (int)(i - m * per) * 4;
        float u[4] = {}, res[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = n + j < o.N;
            res[j] = in && residual != nullptr &&
                             in_bounds(&g_block_status, residual + m * o.N + n + j, sizeof(T), residual, bytes)
                         ? (float)residual[m * o.N + n + j] : 0.0f;
            b[j] = in && bias != nullptr ? (float)bias[n + j] : 0.0f;
        }
        const float* src = partial + m * ldp + n;
        if (!in_bounds(&g_block_status, src + (splits - 1) * o.M * ldp, 16, partial,
                       (long long)splits * o.M * ldp * 4))
            continue;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float4 x = *reinterpret_cast<const float4*>(src + s * o.M * ldp);
            u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            T* out = static_cast<T*>(o.out) + m * o.N + n + j;
            if (n + j >= o.N || !in_bounds(&g_block_status, out, sizeof(T), o.out, bytes)) continue;
            u[j] += b[j];
            if (o.pre != nullptr) static_cast<T*>(o.pre)[m * o.N + n + j] = (T)u[j];
            *out = (T)(act_of<T>(u[j], o.act) + res[j]);
        }
    }
}

// Few rows on FFMA (fp32, and bf16 whose rows are no multiple of 8): bound by
// reading w once.  A block of eight warps takes CPW rows of w (output channels)
// and all MR rows of x; its lanes split k, eight values a load, the warps'
// totals meet in shared memory.
constexpr int kPwFewRows = 8;

template <typename T, int MR, int CPW, bool V>
__global__ void __launch_bounds__(256) pw_rows_kernel(const T* x, const T* w, int K,
                                                      const __grid_constant__ PwOut o) {
    __shared__ float part[8][CPW * MR];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = (int)blockIdx.x * CPW;
    float acc[CPW][MR] = {};
    const int M = (int)o.M;
#pragma unroll 2
    for (int k = warp * 256; k < K; k += 8 * 256) {
        const int c0 = V ? k + lane * 8 : k + lane;
        Raw8<T, V> rw[CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const T* row = w + (long long)(n0 + c) * K;
            if (n0 + c < o.N && in_bounds(&g_block_status, row, (long long)K * sizeof(T), w,
                                          (long long)o.N * K * sizeof(T)))
                load8<T, V>(rw[c], row, c0, 32, K);
            else
                zero8<T, V>(rw[c]);
        }
        f2 f[CPW][4];
#pragma unroll
        for (int c = 0; c < CPW; ++c) unpack8<T, V>(rw[c], f[c]);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if (m >= M) break;
            Raw8<T, V> rx;
            f2 g[4];
            const T* row = x + (long long)m * K;
            if (in_bounds(&g_block_status, row, (long long)K * sizeof(T), x, M * (long long)K * sizeof(T)))
                load8<T, V>(rx, row, c0, 32, K);
            else
                zero8<T, V>(rx);
            unpack8<T, V>(rx, g);
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                f2 t = f2_mul(f[c][0], g[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) t = f2_fma(f[c][i], g[i], t);
                acc[c][m] += f2_sum(t);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CPW; ++c)
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            float v = acc[c][m];
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
            if (lane == ((c * MR + m) & 31)) part[warp][c * MR + m] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < CPW * MR; i += 256) {
        const int c = i / MR, m = i % MR;
        if (m >= M || n0 + c >= o.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s) v += part[s][i];
        pw_store<T>(o, m, n0 + c, v);
    }
}

// Few rows, bf16: still bound by reading w once, but FFMA would spend nine
// instructions on each weight for eight rows (64 us for 8 x 4096 x 4096).  So
// the warp-level matrix instruction (16 x 8 x 16), with the rows of x as its
// 16-row operand and eight output channels as its columns, fed straight from
// global memory: k may be taken in any order as long as both operands agree, so
// a thread loads 16 bytes, eight consecutive k, of its rows of w and x and they
// serve two instructions.  A block of eight warps takes 8 output channels (16
// would leave SMs with one block beside SMs with two at 4096 channels); the
// warps take turns along k and their totals meet in shared memory.  One thread
// has w copied to shared memory in bulk, kRwStages chunks of 512 k ahead (24 KB a
// block, seven blocks an SM, whatever the registers hold).  (tcgen05
// tiles of 256 rows would be all but empty here, and their start-up alone is as
// long as the whole read.)  MB: groups of 8 rows of x.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kRwStages = 3, kRwK = 512;
constexpr int kRwPitch = kRwK * 2 + 64;  // bytes of a row of a chunk: two rows' reads use all banks

template <int MB>
__global__ void __launch_bounds__(256) pw_rows_mma_kernel(const bf16_t* x, const bf16_t* w, int K,
                                                          const __grid_constant__ PwOut o) {
    constexpr int kTiles = (MB + 1) / 2;
    __shared__ __align__(16) uint8_t ring[kRwStages][8][kRwPitch];
    __shared__ float part[8][kTiles * 16][8 + 1];
    __shared__ __align__(8) uint64_t full[kRwStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n0 = (int)blockIdx.x * 8, M = (int)o.M;
    const int chunks = (K + kRwK - 1) / kRwK;
    auto issue = [&](int c) {
        const int k0 = c * kRwK;
        const uint32_t bytes = (uint32_t)min(kRwK, K - k0) * 2;  // (K is a multiple of 8)
        const uint32_t bar = smem_u32(&full[c % kRwStages]);
        mbar_arrive_expect_tx(bar, 8 * bytes);
        for (int r = 0; r < 8; ++r) {
            // channels past the end read as the last one (and are not stored)
            const bf16_t* from = w + (long long)min(n0 + r, o.N - 1) * K + k0;
            // checked build: a range outside w is recorded and read from its start
            if (!in_bounds(&g_block_status, from, bytes, w, (long long)o.N * K * 2)) from = w;
            bulk_g2s(smem_u32(ring[c % kRwStages][r]), from, bytes, bar);
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRwStages; ++s) mbar_init(smem_u32(&full[s]), 1);
        fence_mbar_init();
        for (int c = 0; c < kRwStages && c < chunks; ++c) issue(c);
    }
    __syncthreads();
    float acc[kTiles][4] = {};
    const bf16_t* xr[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) xr[m] = x + (long long)(m * 8 + g < M ? m * 8 + g : 0) * K;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // kRwStages until a wait runs out.  From then on nothing more is issued or
    // stored, and the waits left cover the chunks issued before: no copy lands in
    // shared memory that has become another block's.
    int waits = kRwStages;
    for (int c = 0; c < chunks; ++c) {
        // this thread's two 32-wide steps of the chunk; x is read before the wait
        uint4 rx[2][kTiles * 2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = c * kRwK + (u * 8 + warp) * 32 + t * 8;
#pragma unroll
            for (int m = 0; m < kTiles * 2; ++m)
                rx[u][m] = m < MB && k < K && in_bounds(&g_block_status, xr[m < MB ? m : 0] + k, 16,
                                                        x, o.M * K * 2)
                               ? *reinterpret_cast<const uint4*>(xr[m < MB ? m : 0] + k) : zero;
        }
        const int st = c % kRwStages;
        if (waits > 0 && !mbar_wait(smem_u32(&full[st]), (uint32_t)(c / kRwStages & 1),
                                    &g_block_status, kWaitLimitNs))
            --waits;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kk = (u * 8 + warp) * 32 + t * 8;
            const uint4 rw = c * kRwK + kk < K
                                 ? *reinterpret_cast<const uint4*>(ring[st][g] + kk * 2) : zero;
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                mma_16816(acc[m], rx[u][2 * m].x, rx[u][2 * m + 1].x, rx[u][2 * m].y,
                          rx[u][2 * m + 1].y, rw.x, rw.y);
                mma_16816(acc[m], rx[u][2 * m].z, rx[u][2 * m + 1].z, rx[u][2 * m].w,
                          rx[u][2 * m + 1].w, rw.z, rw.w);
            }
        }
        if (c + kRwStages < chunks) {
            __syncthreads();  // every warp is done with the chunk
            if (threadIdx.x == 0 && waits == kRwStages) issue(c + kRwStages);
        }
    }
    // d0, d1: row g, channels 2t and 2t + 1; d2, d3: row g + 8
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[warp][m * 16 + g + (i >> 1) * 8][2 * t + (i & 1)] = acc[m][i];
    if (!__syncthreads_and(waits == kRwStages)) return;  // a wait ran out
    for (int i = threadIdx.x; i < kTiles * 128; i += 256) {
        const int n = i & 7, m = i >> 3;  // channels side by side
        if (m >= M || n0 + n >= o.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s) v += part[s][m][n];
        pw_store<bf16_t>(o, m, n0 + n, v);
    }
}

// dP = dout act'(pre) into dp (rows of ldp elements, those past N zeros), and
// the column sums of dP over this block's rows (blockIdx.y-th chunk) into
// colsum[chunk][N].  dp or colsum may be NULL.  tpr threads share a row.
// In bf16 dP is rounded as it is stored: it is the tensor cores' operand, and x
// and w, which it meets there, have no more bits.  The rounding adds half a step
// of dP to each term, in the 2-norm as much as the gradients' own rounding: dx
// and dw are 2.35e-3 off, 1.66e-3 without it (16384 x 1024 -> 4096).  Kept in two
// bf16 parts it would cost each product twice its matrix instructions, 210 us of
// that call's 285.  The column sums take dP as it is before the rounding.
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
            if (at < r1 && in_bounds(&g_block_status, dout + at * N, (long long)N * sizeof(T), dout,
                                     M * N * (long long)sizeof(T))) {
                load8<T, V>(rd[j], dout + at * N, c0, tpr, N);
                // (pre has the extent of dout)
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
            if (dp != nullptr && at < r1 &&
                in_bounds(&g_block_status, dp + at * ldp, (long long)ldp * sizeof(T), dp,
                          M * ldp * (long long)sizeof(T)))
                store8<T, V>(pack8<T, V>(d), dp + at * ldp, c0, tpr, ldp);
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
        if (c < N && index_ok(&g_block_status, (long long)blockIdx.y * N + c, (long long)gridDim.y * N))
            colsum[(long long)blockIdx.y * N + c] = a;
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
        for (int i = threadIdx.y; i < chunks; i += 32)
            if (index_ok(&g_block_status, (long long)i * N + c, (long long)chunks * N))
                a += part[(long long)i * N + c];
    buf[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < N) {
        a = 0.0f;
        for (int i = 0; i < 32; ++i) a += buf[i][threadIdx.x];
        dst[c] = (T)a;
    }
}

}  // namespace ccv3d
