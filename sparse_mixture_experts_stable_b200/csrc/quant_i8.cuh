// Rows quantised to 8 bits, one scale per row:
//
//   m = max |x|,   scale = m / 127 (fp32),   q = 127 x / m rounded to the nearest integer, ties to even
//
// q is the rounding of the exact quotient, so it does not depend on how it is computed.
// The fp32 product x (127 / m) is off by less than 2e-5 (|q| <= 127, two roundings of
// 2^-24 relative); where it lies nearer than 1e-4 to a tie, the quotient in fp64 decides.
// x and m have 24 bits each and x >= m / 254, so a quotient that is not a tie is at least
// 2^-34 from one, and fp64 rounds it by at most 2^-47.
// A row of zeros has scale 0.  A row with an infinity or a NaN has scale NaN and q = 0.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ int quantize_exact(float x, float m) {
    return __double2int_rn(127.0 * (double)x / (double)m);
}

struct RowQuant {
    float m, inv;  // inv = 127 / m, 0 where the row's q are all zero
    bool tiny;     // 127 / m does not fit fp32
    float scale;
};

// from the largest |x| of the row as its bits (a NaN's bits are above an infinity's, and that above the finite ones')
__device__ __forceinline__ RowQuant row_quant(uint32_t m_bits, int32_t* status, bool report) {
    RowQuant r;
    r.m = __uint_as_float(m_bits);
    r.tiny = false;
    if (m_bits >= 0x7f800000u) {
        if (report) set_status(status, MOE_ERR_NONFINITE);
        r.scale = __uint_as_float(0x7fffffffu);
        r.inv = 0.f;
        r.m = 0.f;
    } else if (m_bits == 0u) {
        r.scale = 0.f;
        r.inv = 0.f;
    } else {
        r.scale = r.m / 127.f;
        r.tiny = r.m < 1e-30f;
        r.inv = r.tiny ? 0.f : 127.f / r.m;
    }
    return r;
}

__device__ __forceinline__ int quantize(float x, const RowQuant& r) {
    if (r.inv == 0.f) return r.tiny ? quantize_exact(x, r.m) : 0;
    const float v = x * r.inv;
    const float f = rintf(v);
    if (fabsf(fabsf(v - f) - 0.5f) < 1e-4f) return quantize_exact(x, r.m);
    return (int)f;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t pack_i8x4(int a, int b, int c, int d) {
    return (uint32_t)(a & 0xff) | (uint32_t)(b & 0xff) << 8 | (uint32_t)(c & 0xff) << 16 | (uint32_t)d << 24;
}

// 8 consecutive elements of a 16-byte aligned row as fp32
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// One warp quantises the row src[0..D) into rows[0..n) of q (-1: none; row stride ldq) and returns the scale.
// vec: src rows start on 16 bytes and q rows on 8.  Elements past D of q are not written.
template <typename T>
__device__ __forceinline__ float quantize_row_warp(const T* __restrict__ src, int64_t D, const int* rows, int n,
                                                   int8_t* __restrict__ q, int64_t ldq, bool vec, int32_t* status) {
    const int lane = threadIdx.x & 31;
    const int64_t d8 = vec ? D / 8 * 8 : 0;
    uint32_t m = 0;
#pragma unroll 4
    for (int64_t c = lane * 8; c < d8; c += 256) {
        float v[8];
        load8(src + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    }
    for (int64_t c = d8 + lane; c < D; c += 32) m = max(m, abs_bits(to_f32(src[c])));
    m = __reduce_max_sync(0xffffffffu, m);
    const RowQuant r = row_quant(m, status, lane == 0);
#pragma unroll 4
    for (int64_t c = lane * 8; c < d8; c += 256) {
        float v[8];
        load8(src + c, v);
        int w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = quantize(v[i], r);
        const uint2 o = make_uint2(pack_i8x4(w[0], w[1], w[2], w[3]), pack_i8x4(w[4], w[5], w[6], w[7]));
        for (int j = 0; j < n; ++j)
            if (rows[j] >= 0) *reinterpret_cast<uint2*>(q + (int64_t)rows[j] * ldq + c) = o;
    }
    for (int64_t c = d8 + lane; c < D; c += 32) {
        const int8_t w = (int8_t)quantize(to_f32(src[c]), r);
        for (int j = 0; j < n; ++j)
            if (rows[j] >= 0) q[(int64_t)rows[j] * ldq + c] = w;
    }
    return r.scale;
}

}  // namespace moe
