// Grouped product of 8-bit integers on the tensor cores (see i8_gemm.cu) and the row quantisation before it.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moe {

enum I8Epilogue : int {
    I8_OUT = 0,    // out = acc xscale wscale (+ bias)
    I8_GELU = 1,   // out = gelu(acc xscale wscale (+ bias))
    I8_SWIGLU = 2  // two weights: out = silu(acc_gate ...) (acc_up ...)
};

struct I8Problem {
    const int8_t* x;       // (M, K), row stride ldx
    const float* xscale;   // (M)
    int64_t M, ldx;
    const int32_t* offsets;  // device (G + 1), or NULL: G = 1 and all M rows
    const int8_t* w;       // (G, N, K), row stride ldw
    const float* wscale;   // (G, N)
    const int8_t* w2;      // I8_SWIGLU: the up projection, laid out as w
    const float* wscale2;
    int64_t ldw;
    const float* bias;     // (G, N) or NULL; not with I8_SWIGLU
    int G;
    int64_t N, K;
    void* out;             // (M, N), row stride ldo
    int64_t ldo;
    moe_dtype out_dtype;
    int epilogue;
    uint32_t* tile_counter;  // one device word of scratch (zeroed by the call, in stream order)
    int32_t* status;
};

// Checks sizes and alignment and launches: the tensor-core kernel, or i8_skinny_run where i8_skinny_fits.
int i8_gemm_run(const I8Problem& p, cudaStream_t stream);

// Few rows per group: a kernel bound by the weights' bytes (i8_skinny.cu), on a problem that was checked.  f32x: p.x is
// (M, K) fp32 (row stride ldx in values, p.xscale unused) and is quantised on the way; epilogue I8_OUT only.
bool i8_skinny_fits(int64_t M, int G, int64_t N, int64_t K);
int i8_skinny_run(const I8Problem& p, bool f32x, cudaStream_t stream);

// silu(a) b by the fast exponential and quotient.  By CUDA's error tables __expf is off by 2 + 1.173 |a| steps of 2^-23 and
// __fdividef by 2, so with the sum and the product the result is off by less than (7 + 1.2 |a|) 2^-23 of itself; for a below
// -87.3, where the exponential passes 2^126, it is 0 instead of a value under 1.1e-36 |b|.  It is quantised to 8 bits next,
// by steps of 1 / 127 of the row's largest: an error e moves at most one value in 1 / (127 e) across a rounding border, 3400
// for |a| = 10 (16 with an error of 2^-11, tanh.approx's).
__device__ __forceinline__ float swiglu_f(float a, float b) { return __fdividef(a, 1.f + __expf(-a)) * b; }

// Rows of x in 8 bits: all M, or with offsets (G + 1, device) those in [offsets[0], offsets[G]).
int quantize_rows(const void* x, moe_dtype dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq,
                  float* scale, const int32_t* offsets, int G, int32_t* status, cudaStream_t stream);

}  // namespace moe
