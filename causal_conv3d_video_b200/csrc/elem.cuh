// elem.cuh -- what the row kernels around the convolution share: loads and
// stores of eight channels, the activations and their derivatives, and the
// library-wide status word of those kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "checked.cuh"

namespace ccv3d {

typedef __nv_bfloat16 bf16_t;

// First error recorded on this device by a kernel of ccv3d_norm_*,
// ccv3d_pointwise_* or ccv3d_qcache_* (0: none): a bounded wait that ran out,
// or a bounds violation of the checked build.
static __device__ int g_block_status;

enum ActKind { kActNone = 0, kActSilu = 1, kActGelu = 2 };
enum NormKind { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

// 1 / (1 + exp(-v)).  For bf16 results the exponential and the reciprocal are
// the hardware's approximations (relative error near 2^-21, against 2^-9 of
// the result's own rounding); fp32 results use the accurate functions.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-v));
    else return 1.0f / (1.0f + expf(-v));
}

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(u); GELU in its tanh form, 0.5 u (1 + tanh z) = u * sigmoid(2 z).
// (-inf and values whose sigmoid underflows give -0 or 0, not NaN: the
// product is taken only where the sigmoid is not zero.)
template <typename T>
__device__ __forceinline__ float act_of(float u, int kind) {
    if (kind == kActNone) return u;
    const float s = sigmoid_of<T>(kind == kActSilu ? u : 2.0f * kGeluC * (u + kGeluA * u * u * u));
    return s == 0.0f ? 0.0f : u * s;
}

// act'(u): SiLU s (1 + u (1 - s)); GELU s + u s (1 - s) 2 z'(u).
template <typename T>
__device__ __forceinline__ float act_grad_of(float u, int kind) {
    if (kind == kActNone) return 1.0f;
    if (kind == kActSilu) {
        const float s = sigmoid_of<T>(u);
        const float t = 1.0f - s;
        return s == 0.0f ? 0.0f : (t == 0.0f ? s : s * (1.0f + u * t));
    }
    const float s = sigmoid_of<T>(2.0f * kGeluC * (u + kGeluA * u * u * u));
    const float t = s * (1.0f - s);
    return t == 0.0f ? s : s + 2.0f * u * t * kGeluC * (1.0f + 3.0f * kGeluA * u * u);
}

// ------------------------------------------------------------ eight channels
// A unit is eight channels of a row held by one thread: V, eight consecutive
// ones moved as 16-byte words (the row length is a multiple of 8); otherwise
// eight single ones `step` apart, so that neighbouring threads touch
// neighbouring channels.
template <typename T, bool V>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16, true> { uint4 a; };
template <>
struct Raw8<float, true> { float4 a, b; };
template <typename T>
struct Raw8<T, false> { T v[8]; };

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, bool V>
__device__ __forceinline__ void zero8(Raw8<T, V>& r) {
    if constexpr (!V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = T(0.0f);
    } else if constexpr (sizeof(T) == 2) {
        r.a = make_uint4(0, 0, 0, 0);
    } else {
        r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// Channels of unit base `c0` (stride `step` when single) of the row at `row`,
// C channels long; channels past C read as 0.
template <typename T, bool V>
__device__ __forceinline__ void load8(Raw8<T, V>& r, const T* row, int c0, int step, int C) {
    if constexpr (!V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * step;
            r.v[i] = c < C ? row[c] : T(0.0f);
        }
    } else if (c0 >= C) {
        zero8<T, V>(r);
    } else if constexpr (sizeof(T) == 2) {
        r.a = *reinterpret_cast<const uint4*>(row + c0);
    } else {
        r.a = *reinterpret_cast<const float4*>(row + c0);
        r.b = *reinterpret_cast<const float4*>(row + c0 + 4);
    }
}

template <typename T, bool V>
__device__ __forceinline__ void unpack8(const Raw8<T, V>& r, float (&f)[8]) {
    if constexpr (!V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)r.v[i];
    } else if constexpr (sizeof(T) == 2) {
        f[0] = lo_f(r.a.x); f[1] = hi_f(r.a.x); f[2] = lo_f(r.a.y); f[3] = hi_f(r.a.y);
        f[4] = lo_f(r.a.z); f[5] = hi_f(r.a.z); f[6] = lo_f(r.a.w); f[7] = hi_f(r.a.w);
    } else {
        f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
        f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
    }
}

template <typename T, bool V>
__device__ __forceinline__ Raw8<T, V> pack8(const float (&f)[8]) {
    Raw8<T, V> r;
    if constexpr (!V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) r.v[i] = __float2bfloat16_rn(f[i]);
            else r.v[i] = f[i];
        }
    } else if constexpr (sizeof(T) == 2) {
        r.a = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                         pack_bf16(f[6], f[7]));
    } else {
        r.a = make_float4(f[0], f[1], f[2], f[3]);
        r.b = make_float4(f[4], f[5], f[6], f[7]);
    }
    return r;
}

template <typename T, bool V>
__device__ __forceinline__ void store8(const Raw8<T, V>& r, T* row, int c0, int step, int C) {
    if constexpr (!V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * step;
            if (c < C) row[c] = r.v[i];
        }
    } else if (c0 < C) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(row + c0) = r.a;
        } else {
            *reinterpret_cast<float4*>(row + c0) = r.a;
            *reinterpret_cast<float4*>(row + c0 + 4) = r.b;
        }
    }
}

}  // namespace ccv3d
