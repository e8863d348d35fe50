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
// found once per block.  Each thread moves kQUnits units of eight channels a
// block stride apart, all their loads before the first store.  Where C is a
// multiple of 32 (kFlat) a frame is one run of groups and a unit's places need
// no division by the channel count.
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

constexpr int kQUnits = 4;
constexpr int kQThreads = 256;

// Where unit u of a frame lies: its pixel, eight-channel unit of the pixel.
struct QPlace {
    long long px;
    int r;
};

// blockIdx.y = n * frames + i; V: the channel count is a multiple of 8, kFlat:
// of 32.
template <typename T, bool V, bool kFlat>
__global__ void __launch_bounds__(kQThreads) qcache_write_kernel(const __grid_constant__ QCacheJob p,
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
    const long long units = p.pixels * per;
    const long long u0 = (long long)blockIdx.x * (kQThreads * kQUnits) + threadIdx.x;
    Raw8<T, V> raw[kQUnits];
    QPlace at[kQUnits];
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const long long u = u0 + k * kQThreads;
        at[k].px = kFlat ? 0 : u / per;
        at[k].r = kFlat ? 0 : (int)(u - at[k].px * per);
        const T* row = kFlat ? src + u * 8 : src + at[k].px * p.C;
        const bool in = u < units;
        if (in && in_bounds(&g_block_status, row, (kFlat ? 8 : p.C) * (long long)sizeof(T), p.src, x_bytes))
            load8<T, V>(raw[k], row, at[k].r * 8, 1, kFlat ? 8 : p.C);
        else
            zero8<T, V>(raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const long long u = u0 + k * kQThreads;
        float x[8];
        unpack8<T, V>(raw[k], x);
        // magnitudes as integers, whose order is the floats' and puts NaN on top
        uint32_t a = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(x[j]) & 0x7fffffffu);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int c = a == 0u ? 1 : scale_byte(__uint_as_float(a), fmt);
        if (u >= units) continue;  // (whole groups of four threads)
        const int c0 = at[k].r * 8;
        uint8_t* sc = kFlat ? scales + (u >> 2) : scales + at[k].px * p.groups + (at[k].r >> 2);
        if ((threadIdx.x & 3) == 0 && in_bounds(&g_block_status, sc, 1, p.scales, s_bytes))
            *sc = (uint8_t)c;
        const uint2 w = encode8(x, c, fmt);
        if constexpr (kFlat) {
            if (fmt == kQE2m1) *reinterpret_cast<uint32_t*>(codes + u * 4) = w.x;
            else *reinterpret_cast<uint2*>(codes + u * 8) = w;
        } else {
            uint8_t* out = codes + at[k].px * p.code_bytes;
            if constexpr (V) {
                if (c0 < p.C) {
                    if (fmt == kQE2m1) *reinterpret_cast<uint32_t*>(out + c0 / 2) = w.x;
                    else *reinterpret_cast<uint2*>(out + c0) = w;
                }
            } else if (fmt == kQE2m1) {
                for (int j = 0; j < 4; ++j)
                    if (c0 / 2 + j < p.code_bytes) out[c0 / 2 + j] = (uint8_t)(w.x >> (8 * j));
            } else {
                for (int j = 0; j < 8; ++j)
                    if (c0 + j < p.C) out[c0 + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
            }
        }
    }
}

template <typename T, bool V, bool kFlat>
__global__ void __launch_bounds__(kQThreads) qcache_read_kernel(const __grid_constant__ QCacheJob p,
                                                                int fmt) {
    const int n = blockIdx.y / p.frames, i = blockIdx.y - n * p.frames;
    const long long slot = (long long)n * p.slots + (p.slot + i) % p.slots;
    T* dst = static_cast<T*>(p.dst) + (long long)blockIdx.y * p.pixels * p.C;
    const uint8_t* codes = p.codes + slot * p.pixels * p.code_bytes;
    const uint8_t* scales = p.scales + slot * p.pixels * p.groups;
    const long long o_bytes = (long long)p.N * p.frames * p.pixels * p.C * (long long)sizeof(T);
    const long long s_bytes = (long long)p.N * p.slots * p.pixels * p.groups;
    const int per = (p.C + 7) / 8;  // threads a pixel
    const long long units = p.pixels * per;
    const long long u0 = (long long)blockIdx.x * (kQThreads * kQUnits) + threadIdx.x;
    QPlace at[kQUnits];
    uint2 w[kQUnits];
    int c[kQUnits];
    bool ok[kQUnits];
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const long long u = u0 + k * kQThreads;
        at[k].px = kFlat ? 0 : u / per;
        at[k].r = kFlat ? 0 : (int)(u - at[k].px * per);
        const int c0 = at[k].r * 8;
        const uint8_t* in = codes + at[k].px * p.code_bytes;
        const uint8_t* sc = kFlat ? scales + (u >> 2) : scales + at[k].px * p.groups + (at[k].r >> 2);
        w[k] = make_uint2(0u, 0u);
        c[k] = 1;
        ok[k] = u < units && in_bounds(&g_block_status, sc, 1, p.scales, s_bytes);
        if (!ok[k]) continue;
        c[k] = *sc;
        if constexpr (kFlat) {
            if (fmt == kQE2m1) w[k].x = *reinterpret_cast<const uint32_t*>(codes + u * 4);
            else w[k] = *reinterpret_cast<const uint2*>(codes + u * 8);
        } else if constexpr (V) {
            if (fmt == kQE2m1) w[k].x = *reinterpret_cast<const uint32_t*>(in + c0 / 2);
            else w[k] = *reinterpret_cast<const uint2*>(in + c0);
        } else if (fmt == kQE2m1) {
            for (int j = 0; j < 4; ++j)
                if (c0 / 2 + j < p.code_bytes) w[k].x |= (uint32_t)in[c0 / 2 + j] << (8 * j);
        } else {
            for (int j = 0; j < 8; ++j)
                if (c0 + j < p.C) (j < 4 ? w[k].x : w[k].y) |= (uint32_t)in[c0 + j] << (8 * (j & 3));
        }
    }
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        if (!ok[k]) continue;
        float x[8];
        decode8(w[k], c[k], fmt, x);
        T* row = kFlat ? dst + (u0 + k * kQThreads) * 8 : dst + at[k].px * p.C;
        if (in_bounds(&g_block_status, row, (kFlat ? 8 : p.C) * (long long)sizeof(T), p.dst, o_bytes))
            store8<T, V>(pack8<T, V>(x), row, at[k].r * 8, 1, kFlat ? 8 : p.C);
    }
}

}  // namespace ccv3d
