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

// First error recorded on this device by a kernel of this translation unit (0:
// none): a bounded wait that ran out, or a bounds violation of the checked build.
// ccv3d_block_get_status reads that of each of ccv3d_norm_*, ccv3d_pointwise_* and
// ccv3d_qcache_*.
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
template <typename T>
__device__ __forceinline__ float act_of(float u, int kind) {
    if (kind == kActNone) return u;
    return u * sigmoid_of<T>(kind == kActSilu ? u : 2.0f * kGeluC * (u + kGeluA * u * u * u));
}

// act'(u): SiLU s (1 + u (1 - s)); GELU s + u s (1 - s) 2 z'(u), whose last
// factor may overflow where s (1 - s) is 0.
template <typename T>
__device__ __forceinline__ float act_grad_of(float u, int kind) {
    if (kind == kActNone) return 1.0f;
    if (kind == kActSilu) {
        const float s = sigmoid_of<T>(u);
        return s * fmaf(u, 1.0f - s, 1.0f);
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

// ------------------------------------------------------- pairs of fp32 values
// Two fp32 values in a 64-bit register: one instruction multiplies, adds or
// fuses both (each rounded as the single one would be), which halves the
// arithmetic of the row kernels.
typedef unsigned long long f2;

__device__ __forceinline__ f2 f2_make(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 f2_all(float a) { return f2_make(a, a); }
__device__ __forceinline__ void f2_get(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    float a, b;
    f2_get(v, a, b);
    return a + b;
}

// Eight channels as four pairs.
template <typename T, bool V>
__device__ __forceinline__ void unpack8(const Raw8<T, V>& r, f2 (&f)[4]) {
    float t[8];
    unpack8<T, V>(r, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_make(t[2 * i], t[2 * i + 1]);
}
template <typename T, bool V>
__device__ __forceinline__ Raw8<T, V> pack8(const f2 (&f)[4]) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_get(f[i], t[2 * i], t[2 * i + 1]);
    return pack8<T, V>(t);
}

// sigmoid of both, as sigmoid_of.
template <typename T>
__device__ __forceinline__ f2 f2_sigmoid(f2 v) {
    float a, b;
    if constexpr (sizeof(T) == 2) {
        f2_get(f2_mul(v, f2_all(-1.4426950408889634f)), a, b);  // exp(-v) = 2^(-v log2 e)
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
        f2_get(f2_add(f2_make(a, b), f2_all(1.0f)), a, b);
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
        return f2_make(a, b);
    } else {
        f2_get(v, a, b);
        return f2_make(sigmoid_of<T>(a), sigmoid_of<T>(b));
    }
}
// v act-transformed, as act_of.
template <typename T>
__device__ __forceinline__ f2 f2_act(f2 u, int kind) {
    if (kind == kActNone) return u;
    if (kind == kActSilu) return f2_mul(u, f2_sigmoid<T>(u));
    const f2 u3 = f2_mul(f2_mul(u, u), u);
    return f2_mul(u, f2_sigmoid<T>(f2_mul(f2_all(2.0f * kGeluC), f2_fma(u3, f2_all(kGeluA), u))));
}
// act', as act_grad_of.
template <typename T>
__device__ __forceinline__ f2 f2_act_grad(f2 u, int kind) {
    const f2 one = f2_all(1.0f);
    if (kind == kActNone) return one;
    if (kind == kActSilu) {
        const f2 s = f2_sigmoid<T>(u);
        return f2_mul(s, f2_fma(u, f2_fma(s, f2_all(-1.0f), one), one));
    }
    float a, b;
    f2_get(u, a, b);
    return f2_make(act_grad_of<T>(a, kActGelu), act_grad_of<T>(b, kActGelu));
}

}  // namespace ccv3d
