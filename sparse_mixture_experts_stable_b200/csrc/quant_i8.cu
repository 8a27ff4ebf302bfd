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

struct QuantParams {
    const void* x;
    int64_t M, K, ldx;
    int8_t* q;
    int64_t ldq;
    float* scale;
    bool vecx, vecq;         // x rows start on 16 bytes, q rows on 8
    const int32_t* offsets;  // the rows are [offsets[0], offsets[G]), or all M without
    int G;
    int32_t* status;
};

__device__ __forceinline__ void row_range(const QuantParams& p, int64_t& lo, int64_t& hi) {
    lo = 0, hi = p.M;
    if (p.offsets) {
        lo = max(p.offsets[0], 0);
        hi = min((int64_t)p.offsets[p.G], p.M);
    }
}

// One block per row.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) quantize_block_kernel(const QuantParams p) {
    __shared__ uint32_t s_max[kWarps];
    pdl_wait();
    pdl_next();
    int64_t lo, hi;
    row_range(p, lo, hi);
    const int64_t r = blockIdx.x;
    if (r < lo || r >= hi) return;
    const int zero = 0;
    const float s = quantize_row<kWarps>(static_cast<const T*>(p.x) + r * p.ldx, p.K, &zero, 1, p.q + r * p.ldq, 0, p.vecx,
                                         p.vecq, s_max, p.status);
    if (threadIdx.x == 0) p.scale[r] = s;
}

// One warp per row of up to STEPS steps, held in registers while the warp's next row is on its way: a row's loads
// otherwise wait for the arithmetic and the stores of the row before.  131072 x 512 fp32: 54 us, 5.0 TB/s of rows read
// (86 with a row per warp and block); 16384 x 2048 bf16: 21 us, 4.8 TB/s.
template <int STEPS, typename T>
__global__ void __launch_bounds__(kThreads, STEPS > 4 ? 2 : 3) quantize_warp_kernel(const QuantParams p) {
    constexpr int kStride = 32 * kChunk<T>;
    const int lane = threadIdx.x & 31, first = lane * kChunk<T>;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    pdl_wait();
    pdl_next();
    int64_t lo, hi;
    row_range(p, lo, hi);
    const T* x = static_cast<const T*>(p.x);
    int64_t r = lo + (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    Raw<T> next[STEPS];
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (s * kStride < p.K) next[s].load(x + row * p.ldx + first + s * kStride, p.K - first - s * kStride, p.vecx);
    };
    if (r < hi) load(r);
    for (; r < hi; r += step) {
        Raw<T> row[STEPS];
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) row[s] = next[s];
        if (r + step < hi) load(r + step);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (s * kStride < p.K) m = row[s].max_bits(m);
        const RowQuant rq = row_quant(__reduce_max_sync(0xffffffffu, Raw<T>::join(m)), p.status, lane == 0);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int c = first + s * kStride;
            if (c < p.K) {
                uint32_t o[kChunk<T> / 4];
                quantize_chunk(row[s], rq, o);
                store_chunk(p.q + r * p.ldq + c, o, p.K - c, p.vecq);
            }
        }
        if (lane == 0) p.scale[r] = rq.scale;
    }
}

template <typename T>
int launch(const QuantParams& p, cudaStream_t stream) {
    const int64_t sms = device_sm_count();
    const int64_t warp_rows = (p.M + kWarps - 1) / kWarps;
    const auto grid = [&](int resident) { return warp_rows < sms * resident ? warp_rows : sms * resident; };
    constexpr int kShort = 4, kLong = sizeof(T) == 2 ? 8 : 12;
    if (p.K <= 32 * kChunk<T> * kShort) return launch_pdl(quantize_warp_kernel<kShort, T>, grid(3), kThreads, 0, stream, p);
    // a warp each where the rows fill the card's warps and a warp's registers hold one; else a block each
    if (p.K <= 32 * kChunk<T> * kLong && p.M >= sms * 2 * kWarps)
        return launch_pdl(quantize_warp_kernel<kLong, T>, grid(2), kThreads, 0, stream, p);
    return launch_pdl(quantize_block_kernel<T>, p.M, kThreads, 0, stream, p);
}

}  // namespace

int quantize_rows(const void* x, moe_dtype dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq,
                  float* scale, const int32_t* offsets, int G, int32_t* status, cudaStream_t stream) {
    if (M == 0) return MOE_OK;
    QuantParams p{};
    p.x = x, p.M = M, p.K = K, p.ldx = ldx, p.q = q, p.ldq = ldq, p.scale = scale, p.offsets = offsets, p.G = G;
    p.status = status;
    p.vecx = aligned16(x) && (ldx * dtype_size(dtype)) % 16 == 0;
    p.vecq = (reinterpret_cast<uintptr_t>(q) & 7) == 0 && ldq % 8 == 0;
    return dtype == MOE_BF16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
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
