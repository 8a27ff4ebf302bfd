// moe_quantize_i8: rows in 8 bits, one scale per row, and the same for the experts' hidden rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "i8_gemm.cuh"
#include "quant_i8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t M, int64_t K, int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                    float* __restrict__ scale, bool vec, const int32_t* __restrict__ offsets, int G,
                    int32_t* status) {
    const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= M || (offsets && (r < offsets[0] || r >= offsets[G]))) return;
    const int zero = 0;
    const float s = quantize_row_warp(x + r * ldx, K, &zero, 1, q + r * ldq, 0, vec, status);
    if ((threadIdx.x & 31) == 0) scale[r] = s;
}

}  // namespace

int quantize_rows(const void* x, moe_dtype dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq,
                  float* scale, const int32_t* offsets, int G, int32_t* status, cudaStream_t stream) {
    if (M == 0) return MOE_OK;
    const bool vec = aligned16(x) && (ldx * dtype_size(dtype)) % 16 == 0 && (reinterpret_cast<uintptr_t>(q) & 7) == 0 &&
                     ldq % 8 == 0;
    const unsigned grid = (unsigned)((M + kWarps - 1) / kWarps);
    if (dtype == MOE_BF16)
        quantize_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), M, K, ldx,
                                                                      q, ldq, scale, vec, offsets, G, status);
    else
        quantize_kernel<float><<<grid, kThreads, 0, stream>>>(static_cast<const float*>(x), M, K, ldx, q, ldq, scale,
                                                              vec, offsets, G, status);
    return launch_status();
}

}  // namespace moe

using namespace moe;

extern "C" int moe_quantize_i8(const void* x, moe_dtype dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q,
                               int64_t ldq, float* scale, int32_t* dev_status, moe_stream_t stream) {
    MOE_REQUIRE(valid_dtype(dtype) && M >= 0 && K >= 1 && ldx >= K && ldq >= K, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M == 0 || (x && q && scale), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M < (int64_t(1) << 31), MOE_ERR_UNSUPPORTED);
    return quantize_rows(x, dtype, M, K, ldx, q, ldq, scale, nullptr, 0, dev_status,
                         reinterpret_cast<cudaStream_t>(stream));
}
