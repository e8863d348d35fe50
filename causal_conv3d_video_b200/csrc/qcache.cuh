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

#include <type_traits>

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
// byte (the even channel in the low half).  c = 255 writes zeros.  An integer
// code is the low byte of x * 2^(127 - c) + 1.5 * 2^23, whose sum rounds to the
// nearest integer, ties to even: 10 instructions for eight codes, against about
// 36 with a conversion, a mask and a shift each (two 720 x 1280 x 96 frames
// written and read back: 182 -> 166 us).
__device__ __forceinline__ uint2 encode8(const f2 (&x)[4], int c, int fmt) {
    if (c >= 255) return make_uint2(0u, 0u);
    // 2^(127 - c) has exponent field 254 - c; scale_byte gives 1 to 253 (the largest
    // finite exponent field is 254, every format's top exponent at least 2)
    const f2 k = f2_all(__uint_as_float((uint32_t)(254 - c) << 23));
    uint32_t w[2] = {0u, 0u};
    if (fmt == kQInt8) {
        const f2 magic = f2_all(12582912.0f);
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_get(f2_fma(x[i], k, magic), lo, hi);
            v[2 * i] = __float_as_uint(lo);
            v[2 * i + 1] = __float_as_uint(hi);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(v[4 * i], v[4 * i + 1], 0x0040),
                               __byte_perm(v[4 * i + 2], v[4 * i + 3], 0x0040), 0x5410);
        return make_uint2(w[0], w[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v;
        f2_get(f2_mul(x[i], k), v.x, v.y);
        if (fmt == kQE4m3)
            w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)
                         << (16 * (i & 1));
        else
            w[0] |= (uint32_t)__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest) << (8 * i);
    }
    return make_uint2(w[0], w[1]);
}

// Largest magnitude of eight values, as the bits of a non-negative float, whose
// order is the floats' and puts NaN on top.  Eight bf16 values are compared two
// at a time as they are.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t magnitude8(const Raw8<bf16_t, true>& r) {
    constexpr uint32_t m = 0x7fff7fffu;
    const uint32_t a = max_u16x2(max_u16x2(r.a.x & m, r.a.y & m), max_u16x2(r.a.z & m, r.a.w & m));
    return max(a << 16, a & 0xffff0000u);
}
template <typename R>
__device__ __forceinline__ uint32_t magnitude8(const R& r) {
    float x[8];
    unpack8(r, x);
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
    return a;
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

// Eight consecutive values from p on, of which `n` (or more) are there, in
// loads of W values (the rows' and so p's alignment); the others are 0.
template <typename T, int W>
__device__ __forceinline__ void load_w(float (&x)[8], const T* p, int n) {
    if constexpr (W == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? (float)p[i] : 0.0f;
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 8; i += W) {
            uint32_t w[W / 2];
            if constexpr (W == 2) {
                w[0] = i < n ? *reinterpret_cast<const uint32_t*>(p + i) : 0u;
            } else {
                const uint2 t = i < n ? *reinterpret_cast<const uint2*>(p + i) : make_uint2(0u, 0u);
                w[0] = t.x;
                w[1] = t.y;
            }
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                x[i + 2 * j] = lo_f(w[j]);
                x[i + 2 * j + 1] = hi_f(w[j]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += W) {
            if constexpr (W == 2) {
                const float2 t = i < n ? *reinterpret_cast<const float2*>(p + i) : make_float2(0.f, 0.f);
                x[i] = t.x;
                x[i + 1] = t.y;
            } else {
                const float4 t = i < n ? *reinterpret_cast<const float4*>(p + i)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                x[i] = t.x; x[i + 1] = t.y; x[i + 2] = t.z; x[i + 3] = t.w;
            }
        }
    }
}
template <typename T, int W>
__device__ __forceinline__ void store_w(const float (&x)[8], T* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; i += W) {
        if (i >= n) continue;
        if constexpr (W == 1) {
            p[i] = (T)x[i];
        } else if constexpr (sizeof(T) == 2) {
            if constexpr (W == 2) *reinterpret_cast<uint32_t*>(p + i) = pack_bf16(x[i], x[i + 1]);
            else *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]));
        } else {
            if constexpr (W == 2) *reinterpret_cast<float2*>(p + i) = make_float2(x[i], x[i + 1]);
            else *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
    }
}
// The code bytes of eight values (`n` of them there) to or from a row of codes
// whose pieces of W values are aligned; one byte a value, or half of one.
template <int W>
__device__ __forceinline__ void put_codes(uint2 w, uint8_t* p, int n, bool half) {
    if (half) {
        const int m = (n + 1) / 2;  // bytes
        if constexpr (W == 4) {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (i < m) *reinterpret_cast<uint16_t*>(p + i) = (uint16_t)(w.x >> (8 * i));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < m) p[i] = (uint8_t)(w.x >> (8 * i));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i += W) {
        const uint32_t v = (i < 4 ? w.x : w.y) >> (8 * (i & 3));
        if (i >= n) continue;
        if constexpr (W == 4) *reinterpret_cast<uint32_t*>(p + i) = v;
        else if constexpr (W == 2) *reinterpret_cast<uint16_t*>(p + i) = (uint16_t)v;
        else p[i] = (uint8_t)v;
    }
}
template <int W>
__device__ __forceinline__ uint2 get_codes(const uint8_t* p, int n, bool half) {
    uint2 w = make_uint2(0u, 0u);
    if (half) {
        const int m = (n + 1) / 2;
        if constexpr (W == 4) {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (i < m) w.x |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + i) << (8 * i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < m) w.x |= (uint32_t)p[i] << (8 * i);
        }
        return w;
    }
#pragma unroll
    for (int i = 0; i < 8; i += W) {
        if (i >= n) continue;
        uint32_t v;
        if constexpr (W == 4) v = *reinterpret_cast<const uint32_t*>(p + i);
        else if constexpr (W == 2) v = *reinterpret_cast<const uint16_t*>(p + i);
        else v = p[i];
        (i < 4 ? w.x : w.y) |= v << (8 * (i & 3));
    }
    return w;
}

// Where unit u of a frame lies: its pixel, eight-channel unit of the pixel.
struct QPlace {
    long long px;
    int r;
};

// blockIdx.y = n * frames + i; W: values a load, 8, 4, 2 or 1, which divides the
// channel count; kFlat: 32 divides it.
template <typename T, int W, bool kFlat>
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
    const long long c_bytes = (long long)p.N * p.slots * p.pixels * p.code_bytes;
    const int per = p.groups * 4;  // threads a pixel
    const long long units = p.pixels * per;
    const long long u0 = (long long)blockIdx.x * (kQThreads * kQUnits) + threadIdx.x;
    // as loaded, or (pieces of rows that are no multiple of 16 bytes) as fp32
    typedef typename std::conditional<W == 8, Raw8<T, true>, Raw8<float, true>>::type Raw;
    Raw raw[kQUnits];
    QPlace at[kQUnits];
    auto fetch = [&](Raw& r, const T* q, int n) {  // (n <= 0: past the pixel's channels)
        if constexpr (W == 8) {
            load8<T, true>(r, q, 0, 1, n);
        } else {
            float v[8];
            load_w<T, W>(v, q, n);
            r = pack8<float, true>(v);
        }
    };
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const long long u = u0 + k * kQThreads;
        at[k].px = kFlat ? 0 : u / per;
        at[k].r = kFlat ? 0 : (int)(u - at[k].px * per);
        const T* row = kFlat ? src + u * 8 : src + at[k].px * p.C;
        const bool in = u < units;
        if (in && in_bounds(&g_block_status, row, (kFlat ? 8 : p.C) * (long long)sizeof(T), p.src, x_bytes))
            fetch(raw[k], row + at[k].r * 8, kFlat ? 8 : p.C - at[k].r * 8);
        else
            zero8(raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const long long u = u0 + k * kQThreads;
        uint32_t a = magnitude8(raw[k]);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int c = a == 0u ? 1 : scale_byte(__uint_as_float(a), fmt);
        if (u >= units) continue;  // (whole groups of four threads)
        const int c0 = at[k].r * 8;
        uint8_t* sc = kFlat ? scales + (u >> 2) : scales + at[k].px * p.groups + (at[k].r >> 2);
        if ((threadIdx.x & 3) == 0 && in_bounds(&g_block_status, sc, 1, p.scales, s_bytes))
            *sc = (uint8_t)c;
        f2 x[4];
        unpack8(raw[k], x);
        const uint2 w = encode8(x, c, fmt);
        if constexpr (W == 8) {
            uint8_t* out = kFlat ? codes : codes + at[k].px * p.code_bytes;
            const long long o = kFlat ? u * 8 : c0;
            if (kFlat || c0 < p.C) {
                if (fmt == kQE2m1) {
                    if (in_bounds(&g_block_status, out + o / 2, 4, p.codes, c_bytes))
                        *reinterpret_cast<uint32_t*>(out + o / 2) = w.x;
                } else if (in_bounds(&g_block_status, out + o, 8, p.codes, c_bytes)) {
                    *reinterpret_cast<uint2*>(out + o) = w;
                }
            }
        } else if (c0 < p.C) {
            uint8_t* row_codes = codes + at[k].px * p.code_bytes;
            if (in_bounds(&g_block_status, row_codes, p.code_bytes, p.codes, c_bytes))
                put_codes<W>(w, row_codes + (fmt == kQE2m1 ? c0 / 2 : c0), p.C - c0, fmt == kQE2m1);
        }
    }
}

template <typename T, int W, bool kFlat>
__global__ void __launch_bounds__(kQThreads) qcache_read_kernel(const __grid_constant__ QCacheJob p,
                                                                int fmt) {
    const int n = blockIdx.y / p.frames, i = blockIdx.y - n * p.frames;
    const long long slot = (long long)n * p.slots + (p.slot + i) % p.slots;
    T* dst = static_cast<T*>(p.dst) + (long long)blockIdx.y * p.pixels * p.C;
    const uint8_t* codes = p.codes + slot * p.pixels * p.code_bytes;
    const uint8_t* scales = p.scales + slot * p.pixels * p.groups;
    const long long o_bytes = (long long)p.N * p.frames * p.pixels * p.C * (long long)sizeof(T);
    const long long s_bytes = (long long)p.N * p.slots * p.pixels * p.groups;
    const long long c_bytes = (long long)p.N * p.slots * p.pixels * p.code_bytes;
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
        // (checked build) the unit's code bytes: its own in a flat frame, its pixel's otherwise
        const long long unit_bytes = fmt == kQE2m1 ? 4 : 8;
        const uint8_t* from = kFlat ? codes + u * unit_bytes : in;
        w[k] = make_uint2(0u, 0u);
        c[k] = 1;
        ok[k] = u < units && in_bounds(&g_block_status, sc, 1, p.scales, s_bytes) &&
                in_bounds(&g_block_status, from, kFlat ? unit_bytes : p.code_bytes, p.codes, c_bytes);
        if (!ok[k]) continue;
        c[k] = *sc;
        if constexpr (W == 8) {
            const long long o = kFlat ? u * 8 : c0;
            if (fmt == kQE2m1) w[k].x = *reinterpret_cast<const uint32_t*>((kFlat ? codes : in) + o / 2);
            else w[k] = *reinterpret_cast<const uint2*>((kFlat ? codes : in) + o);
        } else {
            w[k] = get_codes<W>(in + (fmt == kQE2m1 ? c0 / 2 : c0), p.C - c0, fmt == kQE2m1);
        }
    }
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        if (!ok[k]) continue;
        float x[8];
        decode8(w[k], c[k], fmt, x);
        T* row = kFlat ? dst + (u0 + k * kQThreads) * 8 : dst + at[k].px * p.C;
        if (!in_bounds(&g_block_status, row, (kFlat ? 8 : p.C) * (long long)sizeof(T), p.dst, o_bytes))
            continue;
        if constexpr (W == 8) store8<T, true>(pack8<T, true>(x), row, at[k].r * 8, 1, kFlat ? 8 : p.C);
        else store_w<T, W>(x, row + at[k].r * 8, p.C - at[k].r * 8);
    }
}

}  // namespace ccv3d
