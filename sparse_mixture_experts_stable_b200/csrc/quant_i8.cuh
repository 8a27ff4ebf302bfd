// Rows quantised to 8 bits, one scale per row:
//
//   m = max |x|,   scale = m / 127 (fp32),   q = 127 x / m rounded to the nearest integer, ties to even
//
// q is the rounding of the exact quotient, so it does not depend on how it is computed.
// fma(x, 127 / m, 1.5 2^23) rounds the product of x with the fp32 127 / m (off by 2^-24
// relative, 8e-6 as |q| <= 127) to an integer in its low bits, and the distance d of the
// product from it is exact to 2^-25.  Where |d| is above 0.49998 the sign of 254 x - h m
// decides, h / 2 the half-way point: both products are split by fma into their rounding and
// its error, the roundings' difference is exact because they are close, and the errors have
// less than 24 bits in common units, so the sign is exact too.
// With bf16 rows one value in a thousand is half-way (x = m / 2 is enough), and the detour
// was taken in every third step of a warp.  There 127 x is exact, and the quotient corrected
// by its residual, v = y + (127 x - y m) / m with y = x (127 / m) (Markstein's correction),
// is exact where it is half-way and otherwise at least 2^7 steps of fp32 away from that
// (x and m have 8 bits), so v rounds as the exact quotient does.
// Rows whose largest value is beyond 2^+-64 are first scaled by a power of two, which is
// exact where it matters.
// A row of zeros has scale 0.  A row with an infinity or a NaN has scale NaN and q = 0.
//
// Rows of up to four 16-byte steps of a team of warps are held in registers
// (quantize_team_kernel, scatter_i8_team_kernel).  Else a team takes a row twice: for the
// maximum with kBatch steps in flight, then for q, when the row still lies in the
// first-level cache.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

struct RowQuant {
    float m, inv;  // largest |x| after scaling, 127 / m; inv = 0 where the row's q are all zero
    float pre;     // the power of two that x is scaled by
    float scale;
};

// from the largest |x| of the row as its bits (a NaN's bits are above an infinity's, and that above the finite ones')
__device__ __forceinline__ RowQuant row_quant(uint32_t m_bits, int32_t* status, bool report) {
    RowQuant r;
    r.m = __uint_as_float(m_bits);
    r.pre = 1.f;
    r.inv = 0.f;
    if (m_bits >= 0x7f800000u) {
        if (report) set_status(status, MOE_ERR_NONFINITE);
        r.scale = __uint_as_float(0x7fffffffu);
        r.m = 0.f;
    } else if (m_bits == 0u) {
        r.scale = 0.f;
    } else {
        r.scale = r.m / 127.f;
        if (r.m < 0x1p-64f) r.pre = 0x1p100f;
        if (r.m > 0x1p64f) r.pre = 0x1p-64f;
        r.m *= r.pre;
        r.inv = 127.f / r.m;
    }
    return r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// values per lane and step: 16 bytes of the row
template <typename T>
constexpr int kChunk = 16 / (int)sizeof(T);

// kChunk consecutive values, as they lie in memory
template <typename T>
struct Raw {
    static constexpr int N = kChunk<T>;
    uint32_t w[4];
    __device__ __forceinline__ float get(int i) const {  // i: a constant
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(int i, T v) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v);
        else if (i & 1) w[i >> 1] |= (uint32_t)__bfloat16_as_ushort(v) << 16;
        else w[i >> 1] = __bfloat16_as_ushort(v);
    }
    // n values of p, zeros behind them.  vec: p lies on 16 bytes.
    __device__ __forceinline__ void load(const T* p, int64_t n, bool vec) {
        if (vec && n >= N) {
            const uint4 r = *reinterpret_cast<const uint4*>(p);
            w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        } else if (sizeof(T) == 2 && n >= N && (reinterpret_cast<uintptr_t>(p) & 3) == 0) {  // 16384 x 2050: 49 -> 36 us
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) set(i, i < n ? p[i] : from_f32<T>(0.f));
        }
    }
    // the largest |x| so far as bits: of fp32, or of two bf16 apart
    __device__ __forceinline__ uint32_t max_bits(uint32_t m) const {
        if constexpr (sizeof(T) == 4) {
            m = __vimax3_s32(m, w[0] & 0x7fffffffu, w[1] & 0x7fffffffu);
            return __vimax3_s32(m, w[2] & 0x7fffffffu, w[3] & 0x7fffffffu);
        } else {
            m = __vimax3_s16x2(m, w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu);
            return __vimax3_s16x2(m, w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu);
        }
    }
    // fp32 bits from max_bits'
    static __device__ __forceinline__ uint32_t join(uint32_t m) {
        return sizeof(T) == 4 ? m : max(m & 0xffff0000u, m << 16);
    }
};

// q where 127 x / m lies next to the half-way point between n and its neighbour on d's side
__device__ __forceinline__ int quantize_near(float x, float m, int n, float d) {
    const int h = 2 * n + (d > 0.f ? 1 : -1);
    const float a = 254.f * x, b = (float)h * m;
    const float rest = (a - b) + (fmaf(254.f, x, -a) - fmaf((float)h, m, -b));
    const int even = (h & 3) == 1 ? -1 : 1;  // the even neighbour of h / 2 is (h + even) / 2
    return (h + (rest > 0.f ? 1 : rest < 0.f ? -1 : even)) / 2;
}

// the chunk's q, four to a word
template <typename T>
__device__ __forceinline__ void quantize_chunk(const Raw<T>& x, const RowQuant& r, uint32_t (&w)[kChunk<T> / 4]) {
    constexpr float kMagic = 12582912.f;  // 1.5 2^23: a sum with it has the integer in its low bits
    [[maybe_unused]] constexpr float kNear = 0.49998f;
    constexpr int N = kChunk<T>;
    int q[N];
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x.get(i);
    if (r.pre != 1.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= r.pre;
    }
    if (r.inv == 0.f) {  // zeros, or not finite
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
    }
    if constexpr (sizeof(T) == 2) {
        const float inv_m = r.inv * (1.f / 127.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = v[i] * r.inv;
            q[i] = __float_as_int(fmaf(fmaf(-y, r.m, 127.f * v[i]), inv_m, y) + kMagic);
        }
    } else {
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaf(v[i], r.inv, kMagic);
            far = fmaxf(far, fabsf(fmaf(v[i], r.inv, kMagic - t)));
            q[i] = __float_as_int(t);
        }
        if (far > kNear) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = __int_as_float(q[i]) - kMagic, d = fmaf(v[i], r.inv, -n);
                if (fabsf(d) > kNear) q[i] = quantize_near(v[i], r.m, (int)n, d);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040),
                           0x5410);
}

// n of the chunk's q to p.  vec: p lies on the chunk's size.
template <int W>
__device__ __forceinline__ void store_chunk(int8_t* p, const uint32_t (&w)[W], int64_t n, bool vec) {
    if (vec && n >= 4 * W) {
        if constexpr (W == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4 * W; ++i)
            if (i < n) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// The largest |x| of a row as fp32 bits, over a team of WARPS warps.  WARPS > 1: all warps of the block, s_max their
// scratch; every thread calls it.  vecx: src lies on 16 bytes.
template <int WARPS, typename T>
__device__ __forceinline__ uint32_t row_max(const T* src, int64_t D, bool vecx, uint32_t* s_max) {
    constexpr int kStride = 32 * WARPS * kChunk<T>;
    constexpr int kBatch = WARPS == 8 ? 4 : 8;  // eight warps' blocks of 64 registers: 16384 x 8192 fp32 119 us, 130 with 8
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x;
    uint32_t m = 0;
    for (int64_t c = tid * kChunk<T>; c < D; c += kBatch * kStride) {
        Raw<T> x[kBatch];
#pragma unroll
        for (int s = 0; s < kBatch; ++s)
            if (c + s * kStride < D) x[s].load(src + c + s * kStride, D - c - s * kStride, vecx);
#pragma unroll
        for (int s = 0; s < kBatch; ++s)
            if (c + s * kStride < D) m = x[s].max_bits(m);
    }
    m = __reduce_max_sync(0xffffffffu, Raw<T>::join(m));
    if constexpr (WARPS > 1) {
        __syncthreads();  // s_max of the call before has been read
        if ((tid & 31) == 0) s_max[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m = max(m, s_max[w]);
    }
    return m;
}

// Whether a row that is not finite has a place to go to; one that has none (a padding token) may hold anything.
__device__ __forceinline__ bool reports(uint32_t m_bits, const int* rows, int n) {
    bool any = false;
    if (m_bits >= 0x7f800000u)
        for (int j = 0; j < n; ++j) any |= rows[j] >= 0;
    return any;
}

// The team quantises the row src[0..D) into rows[0..n) of q (-1: none; row stride ldq) and returns its scale.
// vecq: q rows start on 8 bytes.  Elements past D of q are not written.
template <int WARPS, typename T>
__device__ __forceinline__ float quantize_row(const T* src, int64_t D, const int* rows, int n, int8_t* q, int64_t ldq,
                                              bool vecx, bool vecq, uint32_t* s_max, int32_t* status) {
    constexpr int kStride = 32 * WARPS * kChunk<T>;
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const uint32_t m = row_max<WARPS>(src, D, vecx, s_max);
    const RowQuant r = row_quant(m, status, tid == 0 && reports(m, rows, n));
#pragma unroll 2
    for (int64_t c = tid * kChunk<T>; c < D; c += kStride) {
        Raw<T> x;
        x.load(src + c, D - c, vecx);
        uint32_t o[kChunk<T> / 4];
        quantize_chunk(x, r, o);
        for (int j = 0; j < n; ++j)
            if (rows[j] >= 0) store_chunk(q + (int64_t)rows[j] * ldq + c, o, D - c, vecq);
    }
    return r.scale;
}

}  // namespace moe
