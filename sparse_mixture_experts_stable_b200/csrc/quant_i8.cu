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
constexpr int kResident = 3;  // blocks of teams per SM

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

// TEAM warps per row of up to four steps of the team, held in registers while the team's next row is on its way: a row's
// loads otherwise wait for the arithmetic and the stores of the row before.  131072 x 512 fp32: 54 us, 5.0 TB/s of rows read
// (86 with a row per warp and block); 16384 x 2048 bf16 20 us, 5.1 TB/s with what is written, fp32 29.5 us, 5.7 TB/s (44
// with a block per row); 16384 x 8192 bf16 67 us (78).  Eight steps of half as many warps: fp32 4096 60 us instead of 56.
template <int TEAM, typename T>
__global__ void __launch_bounds__(kThreads, kResident) quantize_team_kernel(const QuantParams p) {
    constexpr int STEPS = 4, kStride = 32 * TEAM * kChunk<T>;
    __shared__ uint32_t s_max[2][kWarps];  // rows take them in turn
    const int warp = threadIdx.x >> 5, team = warp / TEAM, tid = threadIdx.x % (32 * TEAM), first = tid * kChunk<T>;
    const int64_t step = (int64_t)gridDim.x * (kWarps / TEAM);
    pdl_wait();
    pdl_next();
    int64_t lo, hi;
    row_range(p, lo, hi);
    const T* x = static_cast<const T*>(p.x);
    int64_t r = lo + (int64_t)blockIdx.x * (kWarps / TEAM) + team;
    Raw<T> next[STEPS];
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (s * kStride < p.K) next[s].load(x + row * p.ldx + first + s * kStride, p.K - first - s * kStride, p.vecx);
    };
    if (r < hi) load(r);
    for (int turn = 0; r < hi; r += step, turn ^= 1) {
        Raw<T> row[STEPS];
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) row[s] = next[s];
        if (r + step < hi) load(r + step);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (s * kStride < p.K) m = row[s].max_bits(m);
        m = __reduce_max_sync(0xffffffffu, Raw<T>::join(m));
        if constexpr (TEAM > 1) {
            if ((threadIdx.x & 31) == 0) s_max[turn][warp] = m;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory");
#pragma unroll
            for (int w = 0; w < TEAM; ++w) m = max(m, s_max[turn][team * TEAM + w]);
        }
        const RowQuant rq = row_quant(m, p.status, tid == 0);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int c = first + s * kStride;
            if (c < p.K) {
                uint32_t o[kChunk<T> / 4];
                quantize_chunk(row[s], rq, o);
                store_chunk(p.q + r * p.ldq + c, o, p.K - c, p.vecq);
            }
        }
        if (tid == 0) p.scale[r] = rq.scale;
    }
}

template <int TEAM, typename T>
int launch_team(const QuantParams& p, cudaStream_t stream) {
    const int64_t most = device_sm_count() * kResident, need = (p.M + kWarps / TEAM - 1) / (kWarps / TEAM);
    return launch_pdl(quantize_team_kernel<TEAM, T>, need < most ? need : most, kThreads, 0, stream, p);
}

template <typename T>
int launch(const QuantParams& p, cudaStream_t stream) {
    constexpr int kStep = 32 * kChunk<T>;  // values of a warp's step
    if (p.K <= kStep * 4) return launch_team<1, T>(p, stream);
    // longer rows by the teams whose registers hold one, where they are enough for all of them; else a block each
    const int64_t warps = device_sm_count() * 2 * kWarps;
    if (p.K <= kStep * 8 && p.M >= warps / 2) return launch_team<2, T>(p, stream);
    if (p.K <= kStep * 16 && p.M >= warps / 4) return launch_team<4, T>(p, stream);
    if (p.K <= kStep * 32 && p.M >= warps / 8) return launch_team<8, T>(p, stream);
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
