// Rows in 8 bits, and the threads' columns of a row in eights.
//
// A row is cut into blocks of 128 columns (the last one shorter); a block holds e4m3
// codes and one fp32 scale, the smallest power of two, at least 2^-126, that brings its
// largest finite magnitude to at most 448.  e4m3 is a floating format, so a power of two
// loses no digits against amax / 448, and makes every product by the scale or its inverse
// exact: the only rounding is the one to 4 significant bits (half a step, 2^-4 relative,
// or 2^-10 of the scale below 2^-6 of it), and what is unpacked fits bf16 as it is (of scales
// below 2^-124 but for the last bits).
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "zero_ops.cuh"

namespace zf {

constexpr int kEightBlock = 128;

// The exponent field of a block's scale.  2^(e - 8) brings m 2^e with 1 <= m <= 1.75 to
// at most 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t eight_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(e < 1 ? 1 : e);
}
// Of the largest fp32 values, whose codes must not stand for 2^128.
constexpr uint32_t kEightTop = 247;

constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float finite_magnitude(float x) {
    const float m = fabsf(x);
    return m <= kLargest ? m : 0.0f;                 // 0 for infinities and NaN
}

// Code pairs of x / scale (low byte first); NaN becomes code 127.
__device__ __forceinline__ uint32_t eight_codes(float lo, float hi, float inverse) {
    const float2 v = unpair(mul2(pair(lo, hi), pair(inverse, inverse)));
    return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}
// The same where the block holds infinities, which become NaN (e4m3 has none, and a
// saturated one would pass for a value), or magnitudes next to 2^128 (240 instead of 256:
// half a step off at most).
__device__ __noinline__ uint32_t eight_codes_rare(float lo, float hi, float inverse, bool top) {
    lo = fabsf(lo) <= kLargest ? lo * inverse : __int_as_float(0x7FFFFFFF);
    hi = fabsf(hi) <= kLargest ? hi * inverse : __int_as_float(0x7FFFFFFF);
    if (top) {
        lo = lo > 240.0f ? 240.0f : lo < -240.0f ? -240.0f : lo;
        hi = hi > 240.0f ? 240.0f : hi < -240.0f ? -240.0f : hi;
    }
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 eight_values(uint32_t codes, float scale) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3));
    const float2 v = __half22float2(h);
    return make_float2(v.x * scale, v.y * scale);
}

template <class T>
struct alignas(16) Octet {
    T x[8];
};

__device__ __forceinline__ int off_16(const void* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16);
}

// Eight values from the aligned 16-byte words that hold them (one or two words more than
// eight values are, of which bytes beside the row are not used).
template <class T>
__device__ __forceinline__ Octet<T> shifted_octet(const char* words, int by) {
    constexpr int N = sizeof(Octet<T>) / 16;
    uint4 w[N + 1];
#pragma unroll
    for (int i = 0; i <= N; ++i) w[i] = reinterpret_cast<const uint4*>(words)[i];
    Octet<T> v;
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(&v)[i] = shifted<T>(w[i], w[i + 1], by);
    return v;
}

__device__ __forceinline__ uint2 shifted_codes(uint2 lo, uint2 hi, int bytes) {
    const uint64_t a = static_cast<uint64_t>(lo.y) << 32 | lo.x;
    const uint64_t b = static_cast<uint64_t>(hi.y) << 32 | hi.x;
    const uint64_t v = bytes == 0 ? a : a >> (8 * bytes) | b << (64 - 8 * bytes);
    return make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
}

// A thread's K octets of a row's columns.
//   WIDE   octet k holds columns 8 (k threads + t) ... + 7, reached by 16-byte words (8 of
//          codes); half a warp holds a block of 128
//   else   a warp holds 256 columns in turn, element e of lane l the 32 e + l'th, so that
//          single elements are reached side by side; elements 0 to 3 are one block
// All lanes of a warp call these together.
template <bool WIDE, int K>
struct Octets {
    int first, step, dim;
    __device__ Octets(int t, int threads, int d)
        : first(WIDE ? 8 * t : t / 32 * 256 + t % 32), step(8 * threads), dim(d) {}
    __device__ __forceinline__ int at(int k, int e) const {
        return first + k * step + (WIDE ? e : 32 * e);
    }
    __device__ __forceinline__ bool ok(int k, int e) const { return at(k, e) < dim; }

    // zeros where there are no columns
    template <class T>
    __device__ __forceinline__ Octet<T> load(const T* row, int k) const {
        Octet<T> v{};
        if (WIDE && at(k, 7) < dim) {
            constexpr int N = sizeof(v) / 16;
#pragma unroll
            for (int i = 0; i < N; ++i)
                reinterpret_cast<uint4*>(&v)[i] =
                    reinterpret_cast<const uint4*>(row + at(k, 0))[i];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (ok(k, e)) v.x[e] = row[at(k, e)];
            }
        }
        return v;
    }
    template <class T>
    __device__ __forceinline__ void store(T* row, int k, const float (&y)[8]) const {
        Octet<T> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.x[e] = narrow<T>(y[e]);
        if (WIDE && at(k, 7) < dim) {
            constexpr int N = sizeof(v) / 16;
#pragma unroll
            for (int i = 0; i < N; ++i)
                reinterpret_cast<uint4*>(row + at(k, 0))[i] = reinterpret_cast<uint4*>(&v)[i];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (ok(k, e)) row[at(k, e)] = v.x[e];
            }
        }
    }
    // parameters of an array that may start at any element; ones where there is none
    __device__ __forceinline__ void params(float (&w)[8], const void* p, bool f32, int k) const {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = p == nullptr || !ok(k, e) ? 1.0f : ld_param(p, f32, at(k, e));
    }

    // The same, and codes, of rows off the 16-byte grid (8-byte grid): aligned words are loaded
    // and shifted into place, and codes stored after lanes have handed the next one what lies
    // in its word.  (For the octets' mapping.)
    template <class T>
    __device__ __forceinline__ Octet<T> load_any(const T* row, int k) const {
        const T* const p = row + at(k, 0);
        const int mis = off_16(row);
        if (at(k, 7) >= dim || mis == 0) return load<T>(row, k);
        return shifted_octet<T>(reinterpret_cast<const char*>(p) - mis, mis);
    }
    __device__ __forceinline__ void store_eight_any(uint8_t* row, float* scales, int k,
                                                    const float (&y)[8]) const {
        uint32_t w[2];
        const uint32_t s = codes_of(w, y);
        const int c = at(k, 0), n = min(max(dim - c, 0), 8), rest = dim - c;
        if (c < dim && c % kEightBlock == 0) scales[c / kEightBlock] = __uint_as_float(s << 23);
        uint8_t* const p = row + c;
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 8), head = (8 - mis) % 8;
        const int lane = threadIdx.x % 32;
        const uint2 next = make_uint2(__shfl_down_sync(0xFFFFFFFFu, w[0], 1),
                                      __shfl_down_sync(0xFFFFFFFFu, w[1], 1));
        // no whole word (with the next lane), and the lane before left this one's first codes
        const bool last = rest < 8 + head || (mis != 0 && lane == 31);
        const bool alone = lane == 0 || rest < head;
        if (!last)
            *reinterpret_cast<uint2*>(p + head) = shifted_codes(make_uint2(w[0], w[1]), next, head);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < n && (e < head ? alone : last))
                p[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
        }
    }

    // An octet's codes in the block of half a warp's; the scale's exponent field.
    __device__ __forceinline__ static uint32_t codes_of(uint32_t (&w)[2], const float (&y)[8]) {
        // (the larger of a number and NaN is the number)
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        uint32_t s = eight_exponent(m);
        if (__any_sync(0xFFFFFFFFu, s >= kEightTop)) {
            m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_magnitude(y[e]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            s = eight_exponent(m);
            const float inverse = __uint_as_float((254 - s) << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = eight_codes_rare(y[4 * i], y[4 * i + 1], inverse, s == kEightTop) |
                       eight_codes_rare(y[4 * i + 2], y[4 * i + 3], inverse, s == kEightTop)
                           << 16;
        } else {
            const float inverse = __uint_as_float((254 - s) << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = eight_codes(y[4 * i], y[4 * i + 1], inverse) |
                       eight_codes(y[4 * i + 2], y[4 * i + 3], inverse) << 16;
        }
        return s;
    }

    __device__ __forceinline__ void store_eight(uint8_t* row, float* scales, int k,
                                                const float (&y)[8]) const {
        if constexpr (WIDE) {
            uint32_t w[2];
            const uint32_t s = codes_of(w, y);
            const int c = at(k, 0);
            if (c + 7 < dim) {
                *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c + e < dim) row[c + e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
                }
            }
            if (c < dim && c % kEightBlock == 0)
                scales[c / kEightBlock] = __uint_as_float(s << 23);
        } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float m = 0.0f;
#pragma unroll
                for (int e = 4 * b; e < 4 * b + 4; ++e) m = fmaxf(m, fabsf(y[e]));
                m = warp_max(m);
                uint32_t s = eight_exponent(m);
                const bool rare = s >= kEightTop;        // of the whole warp
                if (rare) {
                    m = 0.0f;
#pragma unroll
                    for (int e = 4 * b; e < 4 * b + 4; ++e) m = fmaxf(m, finite_magnitude(y[e]));
                    s = eight_exponent(warp_max(m));
                }
                const float inverse = __uint_as_float((254 - s) << 23);
#pragma unroll
                for (int e = 4 * b; e < 4 * b + 4; e += 2) {
                    const uint32_t w =
                        rare ? eight_codes_rare(y[e], y[e + 1], inverse, s == kEightTop)
                             : eight_codes(y[e], y[e + 1], inverse);
                    if (ok(k, e)) row[at(k, e)] = static_cast<uint8_t>(w);
                    if (ok(k, e + 1)) row[at(k, e + 1)] = static_cast<uint8_t>(w >> 8);
                }
                const int c = at(k, 4 * b);
                if (c < dim && c % kEightBlock == 0)
                    scales[c / kEightBlock] = __uint_as_float(s << 23);
            }
        }
    }
    __device__ __forceinline__ void load_eight(float (&y)[8], const uint8_t* row,
                                               const float* scales, int k) const {
        if constexpr (WIDE) {
            uint32_t w[2] = {0, 0};
            const int c = at(k, 0);
            if (c + 7 < dim) {
                const uint2 v = *reinterpret_cast<const uint2*>(row + c);
                w[0] = v.x;
                w[1] = v.y;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c + e < dim)
                        w[e / 4] |= static_cast<uint32_t>(row[c + e]) << (8 * (e % 4));
                }
            }
            const float s = c < dim ? scales[c / kEightBlock] : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 v = eight_values((w[e / 4] >> (8 * (e % 4))) & 0xFFFFu, s);
                y[e] = v.x;
                y[e + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = at(k, e);
                y[e] = 0.0f;
                if (c < dim) y[e] = eight_values(row[c], scales[c / kEightBlock]).x;
            }
        }
    }
};

__device__ __forceinline__ void values_of(float (&y)[8], uint2 codes, float scale) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint32_t w = e < 4 ? codes.x : codes.y;
        const float2 v = eight_values((w >> (8 * (e % 4))) & 0xFFFFu, scale);
        y[e] = v.x;
        y[e + 1] = v.y;
    }
}

}  // namespace zf
