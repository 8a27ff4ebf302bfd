// Exclusive prefix sums over a block.
#pragma once

#include "common.cuh"

namespace moe {

// Exclusive sums of v[0..E) in place (v[E] receives the total); every thread of the block takes part.
template <int THREADS>
__device__ __forceinline__ void block_scan(int* v, int E) {
    __shared__ int s_warp[THREADS / 32];
    const int per = (E + THREADS - 1) / THREADS;
    const int b = threadIdx.x * per;
    int sum = 0;
    for (int i = b; i < b + per && i < E; ++i) sum += v[i];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32 - 1; ++w)  // all at once
        if (w < warp) before += s_warp[w];
    int run = before + inc - sum;
    for (int i = b; i < b + per && i < E; ++i) {
        const int c = v[i];
        v[i] = run;
        run += c;
    }
    if (threadIdx.x == THREADS - 1) v[E] = before + inc;
    __syncthreads();
}

}  // namespace moe
