// qcache.cuh -- the ring cache held in 8 or 4 bits: frames quantised as they
// are written, and read back.
//
// 32 consecutive channels of a pixel form a group (the last group of a pixel
// may be shorter) and share a power-of-two scale 2^(c - 127), c one byte: the
// smallest for which the group's largest magnitude fits the format, so
// nothing saturates.  A code is the format's value nearest x 2^(127 - c), ties
// to even.  Scaling by a power of two is exact, so a code carries one
// rounding and a value read back (code times scale, at most 8 significant
// bits) is exact in bf16.  A group that holds a NaN or an infinity gets the
// scale byte 255 and reads back as NaN; a group of zeros gets scale byte 1.
//
// HBM-bound: e + 1 + 1/32 (8 bits) or e + 1/2 + 1/32 bytes a channel in each
// direction, e = 2 or 4.  A group is four threads of eight channels, its
// maximum two shuffles.  Frames are the grid's second axis, so a ring slot is
// found once per block.
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "elem.cuh"

namespace ccv3d {

enum QFormat { kQInt8 = 0, kQE4m3 = 1, kQE2m1 = 2 };
constexpr int kQGroup = 32;

struct QCacheJob {
    const void* src;       // write: x [N][T][pixels][C]; read: unused
    void* dst;             // read: [N][frames][pixels][C]
    uint8_t* codes;        // [N][slots][pixels][code bytes]
    uint8_t* scales;       // [N][slots][pixels][groups]
    long long pixels;      // H * W
    int N, C, groups, code_bytes, slots;
    int T, first;          // write: frames of x, and the first of them written
    int frames, slot;      // frames moved, and the slot of the first
};

// Scale byte of a group whose largest magnitude is `a` (finite, not NaN).
__device__ __forceinline__ int scale_byte(float a, int fmt) {
    const uint32_t bits = __float_as_uint(a);
    if (bits >= 0x7f800000u) return 255;  // infinity or NaN (the sign bit is clear)
    // largest value: 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8, 6 = 1.5 * 2^2
    const uint32_t top = fmt == kQInt8 ? 0x7e0000u : (fmt == kQE4m3 ? 0x600000u : 0x400000u);
    const int top_e = fmt == kQInt8 ? 6 : (fmt == kQE4m3 ? 8 : 2);
    // subnormal magnitudes have exponent field 0 and end below the clamp
    const int c = (int)(bits >> 23) - top_e + ((bits & 0x7fffffu) > top ? 1 : 0);
    return c < 1 ? 1 : c;
}

// Eight codes of the values x * 2^(127 - c): 8 bytes, or 4 for two codes a
// byte (the even channel in the low half).  c = 255 writes zeros.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], int c, int fmt) {
    // 2^(127 - c) has exponent field 254 - c (1 <= c <= 254; c = 254: 2^-127, subnormal)
    const float k = c >= 255 ? 0.0f
                             : (c == 254 ? __uint_as_float(0x400000u)
                                         : __uint_as_float((uint32_t)(254 - c) << 23));
    uint32_t w[2] = {0u, 0u};
    if (c >= 255) return make_uint2(0u, 0u);
    if (fmt == kQInt8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i >> 2] |= ((uint32_t)__float2int_rn(x[i] * k) & 255u) << (8 * (i & 3));
    } else if (fmt == kQE4m3) {
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            w[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[i] * k, x[i + 1] * k),
                                                            __NV_SATFINITE, __NV_E4M3)
                         << (8 * (i & 3));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            w[0] |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(x[i] * k, x[i + 1] * k),
                                                       __NV_E2M1, cudaRoundNearest)
                    << (4 * i);
    }
    return make_uint2(w[0], w[1]);
}

// The eight values that codes `w` and scale byte `c` stand for.
__device__ __forceinline__ void decode8(uint2 w, int c, int fmt, float (&x)[8]) {
    const float k = c >= 255 ? __uint_as_float(0x7fc00000u)
                             : (c == 0 ? __uint_as_float(0x400000u)
                                       : __uint_as_float((uint32_t)c << 23));
    if (fmt == kQInt8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    } else if (fmt == kQE4m3) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const __half2_raw h =
                __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w.x >> (4 * i)) & 255u), __NV_E2M1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= k;
}

// blockIdx.y = n * frames + i; V: the channel count is a multiple of 8.
template <typename T, bool V>
__global__ void __launch_bounds__(256) qcache_write_kernel(const __grid_constant__ QCacheJob p,
                                                           int fmt) {
    const int n = blockIdx.y / p.frames, i = blockIdx.y - n * p.frames;
    const long long slot = (long long)n * p.slots + (p.slot + i) % p.slots;
    const T* src = static_cast<const T*>(p.src) +
                   ((long long)n * p.T + p.first + i) * p.pixels * p.C;
    uint8_t* codes = p.codes + slot * p.pixels * p.code_bytes;
    uint8_t* scales = p.scales + slot * p.pixels * p.groups;
    const long long x_bytes = (long long)p.N * p.T * p.pixels * p.C * (long long)sizeof(T);
    const long long s_bytes = (long long)p.N * p.slots * p.pixels * p.groups;
    const int per = p.groups * 4;  // threads a pixel
    const long long units = p.pixels * per, step = (long long)gridDim.x * blockDim.x;
    // whole warps stay in the loop together: a group's four threads shuffle
    for (long long u0 = (long long)blockIdx.x * blockDim.x; u0 < units; u0 += step) {
        const long long u = u0 + threadIdx.x;
        const long long px = u / per;
        const int r = (int)(u - px * per), c0 = r * 8;
        const bool in = u < units;
        const T* row = src + px * p.C;
        Raw8<T, V> raw;
        float x[8];
        if (in && in_bounds(&g_block_status, row, (long long)p.C * sizeof(T), p.src, x_bytes))
            load8<T, V>(raw, row, c0, 1, p.C);
        else
            zero8<T, V>(raw);
        unpack8<T, V>(raw, x);
        // magnitudes as integers, whose order is the floats' and puts NaN on top
        uint32_t a = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = max(a, __float_as_uint(x[k]) & 0x7fffffffu);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int c = a == 0u ? 1 : scale_byte(__uint_as_float(a), fmt);
        if (!in) continue;
        if ((r & 3) == 0 &&
            in_bounds(&g_block_status, scales + px * p.groups + (r >> 2), 1, p.scales, s_bytes))
            scales[px * p.groups + (r >> 2)] = (uint8_t)c;
        const uint2 w = encode8(x, c, fmt);
        uint8_t* out = codes + px * p.code_bytes;
        if constexpr (V) {
            if (c0 < p.C) {
                if (fmt == kQE2m1) *reinterpret_cast<uint32_t*>(out + c0 / 2) = w.x;
                else *reinterpret_cast<uint2*>(out + c0) = w;
            }
        } else if (fmt == kQE2m1) {
            for (int k = 0; k < 4; ++k)
                if (c0 / 2 + k < p.code_bytes) out[c0 / 2 + k] = (uint8_t)(w.x >> (8 * k));
        } else {
            for (int k = 0; k < 8; ++k)
                if (c0 + k < p.C) out[c0 + k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
        }
    }
}

template <typename T, bool V>
__global__ void __launch_bounds__(256) qcache_read_kernel(const __grid_constant__ QCacheJob p,
                                                          int fmt) {
    const int n = blockIdx.y / p.frames, i = blockIdx.y - n * p.frames;
    const long long slot = (long long)n * p.slots + (p.slot + i) % p.slots;
    T* dst = static_cast<T*>(p.dst) + (long long)blockIdx.y * p.pixels * p.C;
    const uint8_t* codes = p.codes + slot * p.pixels * p.code_bytes;
    const uint8_t* scales = p.scales + slot * p.pixels * p.groups;
    const long long o_bytes = (long long)p.N * p.frames * p.pixels * p.C * (long long)sizeof(T);
    const long long s_bytes = (long long)p.N * p.slots * p.pixels * p.groups;
    const int per = (p.C + 7) / 8;  // threads a pixel
    const long long units = p.pixels * per, step = (long long)gridDim.x * blockDim.x;
    for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < units; u += step) {
        const long long px = u / per;
        const int r = (int)(u - px * per), c0 = r * 8;
        const uint8_t* in = codes + px * p.code_bytes;
        const uint8_t* sc = scales + px * p.groups + (r >> 2);
        if (!in_bounds(&g_block_status, sc, 1, p.scales, s_bytes)) continue;
        uint2 w = make_uint2(0u, 0u);
        if constexpr (V) {
            if (fmt == kQE2m1) w.x = *reinterpret_cast<const uint32_t*>(in + c0 / 2);
            else w = *reinterpret_cast<const uint2*>(in + c0);
        } else if (fmt == kQE2m1) {
            for (int k = 0; k < 4; ++k)
                if (c0 / 2 + k < p.code_bytes) w.x |= (uint32_t)in[c0 / 2 + k] << (8 * k);
        } else {
            for (int k = 0; k < 8; ++k)
                if (c0 + k < p.C) (k < 4 ? w.x : w.y) |= (uint32_t)in[c0 + k] << (8 * (k & 3));
        }
        float x[8];
        decode8(w, *sc, fmt, x);
        T* row = dst + px * p.C;
        if (in_bounds(&g_block_status, row, (long long)p.C * sizeof(T), p.dst, o_bytes))
            store8<T, V>(pack8<T, V>(x), row, c0, 1, p.C);
    }
}

}  // namespace ccv3d
