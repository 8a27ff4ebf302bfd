// moe_sort, moe_sort_i8, moe_unsort, moe_unsort_backward: tokens sorted by
// expert into packed rows without a capacity, and back.
//
// Assignments i = t k + j are ordered by (expert, i): row = offsets[e] + #{earlier
// assignments to e}.  The order is a counting sort.  Up to kSmallCount assignments one
// launch does everything: every block counts all the keys itself, so no block waits
// for another.  Above, hist_kernel counts the keys of each super-block, base_kernel
// turns the counts into first rows, and every block of the row kernel adds the keys of
// its super-block that come before its own tokens.  Integer counts do not depend on
// the order of the shared-memory atomics that make them, so the rows are unique.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "quant_i8.cuh"

namespace moe {
namespace {

constexpr int kMaxE = 2048;
constexpr int kMaxK = 64;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kSmallCount = 4096;   // assignments that one launch handles by itself
constexpr int64_t kSuperCount = 4096;   // assignments per super-block (more when there are over kMaxSuper of them)
constexpr int64_t kMaxSuper = 256;
constexpr int kHistThreads = 512;

// What the row kernel does with each token's row of x.
enum RowOp : int { ROW_NONE = 0, ROW_COPY = 1, ROW_I8 = 2 };

struct SortParams {
    const int64_t* selected;
    int64_t T;
    int k, E;
    int64_t n;            // T * k
    int64_t super;        // assignments per super-block (a multiple of k), 0 in the one-launch form
    int64_t block_tokens; // tokens per block of the row kernel
    const int32_t* base;  // (super-blocks, E) first rows inside the expert, from base_kernel
    int32_t* offsets;
    int32_t* row;
    int32_t* source;
    const void* x;
    int64_t D, ldx;
    void* xs;
    int64_t ldxs;
    float* xscale;
    bool vec;             // ROW_I8: x rows start on 16 bytes, xs rows on 8
    int32_t* status;
};

// expert of an assignment, -1 for one that takes no part
__device__ __forceinline__ int key_of(int64_t e, int E, int32_t* status) {
    if (e >= 0 && e < E) return (int)e;
    if (e != -1) set_status(status, MOE_ERR_BAD_INDEX);
    return -1;
}

__global__ void __launch_bounds__(kHistThreads)
    hist_kernel(const int64_t* __restrict__ selected, int64_t n, int64_t super, int E, int32_t* __restrict__ hist,
                int32_t* status) {
    extern __shared__ int s_cnt[];
    for (int e = threadIdx.x; e < E; e += kHistThreads) s_cnt[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * super;
    const int64_t last = first + super < n ? first + super : n;
#pragma unroll 4
    for (int64_t i = first + threadIdx.x; i < last; i += kHistThreads) {
        const int key = key_of(selected[i], E, status);
        if (key >= 0) atomicAdd(&s_cnt[key], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kHistThreads) hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
}

constexpr int kBaseThreads = 1024;
constexpr int kBaseBatch = 16;

// hist (n_super, E) -> exclusive sums over the super-blocks in place, and offsets (E + 1).
__global__ void __launch_bounds__(kBaseThreads)
    base_kernel(int32_t* hist, int n_super, int E, int32_t* __restrict__ offsets) {
    __shared__ int s_total[kMaxE + 1];
    for (int e = threadIdx.x; e < E; e += kBaseThreads) {
        int run = 0;
        for (int a0 = 0; a0 < n_super; a0 += kBaseBatch) {
            int v[kBaseBatch];
#pragma unroll
            for (int u = 0; u < kBaseBatch; ++u) v[u] = a0 + u < n_super ? hist[(int64_t)(a0 + u) * E + e] : 0;
#pragma unroll
            for (int u = 0; u < kBaseBatch; ++u)
                if (a0 + u < n_super) {
                    hist[(int64_t)(a0 + u) * E + e] = run;
                    run += v[u];
                }
        }
        s_total[e] = run;
    }
    __syncthreads();
    block_scan<kBaseThreads>(s_total, E);
    for (int e = threadIdx.x; e <= E; e += kBaseThreads) offsets[e] = s_total[e];
}

// One warp copies a row to the rows dst[0..k) of the packed matrix (-1: none).
// V: the widest vector that every row start and the row length allow.
template <typename V>
__device__ __forceinline__ void copy_row(const SortParams& p, int64_t t, const int* rows, int lane) {
    constexpr int kBatch = 8;
    const int64_t nv = p.D, ldx = p.ldx, lds = p.ldxs;  // in units of V
    const V* src = static_cast<const V*>(p.x) + t * ldx;
    V* dst = static_cast<V*>(p.xs);
    for (int64_t v0 = lane; v0 < nv; v0 += 32 * kBatch) {
        V r[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (v0 + 32 * u < nv) r[u] = src[v0 + 32 * u];
        for (int j = 0; j < p.k; ++j) {
            const int rw = rows[j];
            if (rw < 0) continue;
            V* d = dst + (int64_t)rw * lds;
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (v0 + 32 * u < nv) d[v0 + 32 * u] = r[u];
        }
    }
}

// Shared memory: s_cnt[E + 1] (next row of each expert), s_row[block_tokens * k]; one-launch form: s_off[E + 1] too.
template <int OP, typename V>
__global__ void __launch_bounds__(kThreads) row_kernel(const SortParams p) {
    extern __shared__ int s_dyn[];
    int* s_cnt = s_dyn;
    int* s_row = s_cnt + p.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    const int ntok = (int)(p.T - t0 < p.block_tokens ? p.T - t0 : p.block_tokens);
    const int64_t first = t0 * p.k;  // this block's assignments: [first, first + n_own)
    const int n_own = ntok * p.k;

    int total;
    if (p.super == 0) {
        int* s_off = s_row + p.block_tokens * p.k;
        for (int e = threadIdx.x; e < p.E; e += kThreads) s_cnt[e] = s_off[e] = 0;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            const int key = key_of(p.selected[i], p.E, p.status);
            if (key >= 0) {
                atomicAdd(&s_off[key], 1);
                if (i < first) atomicAdd(&s_cnt[key], 1);
            }
        }
        __syncthreads();
        block_scan<kThreads>(s_off, p.E);
        for (int e = threadIdx.x; e < p.E; e += kThreads) s_cnt[e] += s_off[e];
        if (blockIdx.x == 0)
            for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = s_off[e];
        total = s_off[p.E];
    } else {
        const int64_t a = first / p.super;
        for (int e = threadIdx.x; e < p.E; e += kThreads) s_cnt[e] = p.base[a * p.E + e] + p.offsets[e];
        __syncthreads();
        for (int64_t i = a * p.super + threadIdx.x; i < first; i += kThreads) {
            const int key = key_of(p.selected[i], p.E, nullptr);
            if (key >= 0) atomicAdd(&s_cnt[key], 1);
        }
        total = p.offsets[p.E];
    }
    __syncthreads();

    // ranks of the own assignments, 32 at a time in order
    if (warp == 0) {
        for (int c = 0; c < n_own; c += 32) {
            const int li = c + lane;
            const int key = li < n_own ? key_of(p.selected[first + li], p.E, nullptr) : -1;
            const uint32_t match = __match_any_sync(0xffffffffu, key);
            int r = -1;
            if (key >= 0) r = s_cnt[key] + __popc(match & lanemask_lt());
            __syncwarp();
            if (key >= 0 && __ffs(match) - 1 == lane) s_cnt[key] += __popc(match);
            __syncwarp();
            if (li < n_own) {
                s_row[li] = r;
                p.row[first + li] = r;
                if (r >= 0) p.source[r] = (int32_t)(first + li);
                if (first + li >= total) p.source[first + li] = -1;  // behind the last row
            }
        }
    }
    if (OP == ROW_NONE) return;
    __syncthreads();
    for (int t = warp; t < ntok; t += kWarps) {
        const int* rows = s_row + t * p.k;
        if (OP == ROW_COPY) copy_row<V>(p, t0 + t, rows, lane);
        if (OP == ROW_I8) {
            int8_t* q = static_cast<int8_t*>(p.xs);
            const float scale = quantize_row_warp(static_cast<const V*>(p.x) + (t0 + t) * p.ldx, p.D, rows, p.k, q,
                                                  p.ldxs, p.vec, p.status);
            for (int j = lane; j < p.k; j += 32)
                if (rows[j] >= 0) p.xscale[rows[j]] = scale;
        }
    }
}

// super-block and row-block sizes for T tokens of k assignments
struct SortPlan {
    bool small;
    int64_t super, n_super, block_tokens;
};

SortPlan sort_plan(int64_t T, int32_t k) {
    SortPlan s{};
    const int64_t n = T * k;
    const int64_t sms = device_sm_count();
    s.small = n <= kSmallCount;
    if (s.small) {
        s.block_tokens = (T + 2 * sms - 1) / (2 * sms);
    } else {
        int64_t bt = 32;                          // T = 16384: 512 blocks
        while (bt > 1 && bt * k > 1024) bt >>= 1; // the rows of a block stay in shared memory
        s.block_tokens = bt;
        int64_t super = n / kMaxSuper > kSuperCount ? n / kMaxSuper : kSuperCount;
        const int64_t unit = bt * k;              // whole blocks per super-block
        s.super = (super + unit - 1) / unit * unit;
        s.n_super = (n + s.super - 1) / s.super;
    }
    if (s.block_tokens < 1) s.block_tokens = 1;
    return s;
}

template <int OP, typename V>
int launch_rows(const SortParams& p, int64_t blocks, size_t smem, cudaStream_t stream) {
    row_kernel<OP, V><<<(unsigned)blocks, kThreads, smem, stream>>>(p);
    return launch_status();
}

int sort_check(const int64_t* selected, int64_t T, int32_t k, int32_t E, const int32_t* offsets, const int32_t* row,
               const int32_t* source) {
    MOE_REQUIRE(T >= 0 && k >= 1 && E >= 1 && offsets, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T == 0 || (selected && row && source), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(k <= kMaxK && E <= kMaxE, MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(T < (int64_t(1) << 30) && T * k < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);
    return MOE_OK;
}

size_t sort_workspace(int64_t T, int32_t k, int32_t E) {
    const SortPlan s = sort_plan(T, k);
    return s.small ? 0 : align_up((size_t)s.n_super * E * sizeof(int32_t), 256);
}

// The order, then the rows of x (op).
int sort_run(SortParams p, int op, moe_dtype dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (p.T == 0) {
        MOE_CUDA_TRY(cudaMemsetAsync(p.offsets, 0, sizeof(int32_t) * ((size_t)p.E + 1), stream));
        return MOE_OK;
    }
    const SortPlan s = sort_plan(p.T, p.k);
    p.n = p.T * p.k;
    p.super = s.small ? 0 : s.super;
    p.block_tokens = s.block_tokens;
    if (!s.small) {
        MOE_REQUIRE(workspace && workspace_bytes >= sort_workspace(p.T, p.k, p.E), MOE_ERR_WORKSPACE);
        int32_t* hist = static_cast<int32_t*>(workspace);
        p.base = hist;
        hist_kernel<<<(unsigned)s.n_super, kHistThreads, sizeof(int) * p.E, stream>>>(p.selected, p.n, p.super, p.E,
                                                                                      hist, p.status);
        int rc = launch_status();
        if (rc != MOE_OK) return rc;
        base_kernel<<<1, kBaseThreads, 0, stream>>>(hist, (int)s.n_super, p.E, p.offsets);
        rc = launch_status();
        if (rc != MOE_OK) return rc;
    }
    const int64_t blocks = (p.T + s.block_tokens - 1) / s.block_tokens;
    const size_t smem = sizeof(int) * ((size_t)(s.small ? 2 : 1) * (p.E + 1) + (size_t)s.block_tokens * p.k);
    if (op == ROW_NONE) return launch_rows<ROW_NONE, float>(p, blocks, smem, stream);
    if (op == ROW_I8) {
        p.vec = aligned16(p.x) && (p.ldx * dtype_size(dtype)) % 16 == 0 &&
                (reinterpret_cast<uintptr_t>(p.xs) & 7) == 0 && p.ldxs % 8 == 0;
        return dtype == MOE_BF16 ? launch_rows<ROW_I8, __nv_bfloat16>(p, blocks, smem, stream)
                                 : launch_rows<ROW_I8, float>(p, blocks, smem, stream);
    }
    const size_t es = dtype_size(dtype);
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.xs) |
                          (uintptr_t)(p.D * es) | (uintptr_t)(p.ldx * es) | (uintptr_t)(p.ldxs * es);
    const int64_t per = (all & 15) == 0 ? 16 / es : (all & 3) == 0 ? 4 / es : 1;  // elements per vector
    p.D /= per;
    p.ldx /= per;
    p.ldxs /= per;
    if ((all & 15) == 0) return launch_rows<ROW_COPY, uint4>(p, blocks, smem, stream);
    if ((all & 3) == 0) return launch_rows<ROW_COPY, uint32_t>(p, blocks, smem, stream);
    return launch_rows<ROW_COPY, uint16_t>(p, blocks, smem, stream);
}

// ------------------------------- and back -----------------------------------

// V: 16 bytes, or one element, of a row of T; its values as fp32
template <typename T, typename V>
struct Vec {
    static constexpr int kN = sizeof(V) / sizeof(T);
    static __device__ __forceinline__ void unpack(const V& r, float (&v)[kN]) {
        const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = to_f32(e[i]);
    }
    static __device__ __forceinline__ V pack(const float (&v)[kN]) {
        V r;
        T* e = reinterpret_cast<T*>(&r);
#pragma unroll
        for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(v[i]);
        return r;
    }
};

struct UnsortParams {
    const void* ys;
    int64_t ldys, rows;
    const int32_t* row;
    const void* gates;  // (T, k) of the gate type, or NULL
    int64_t T;
    int k;
    int64_t N;
    const void* base;
    int64_t ldbase;
    void* y;            // moe_unsort: y (T, N); moe_unsort_backward: dys (rows, N)
    int64_t ldy;
    const void* dy;
    int64_t lddy;
    float* dgates;
    int split;          // moe_unsort: warps per token
    int32_t* status;
};

// the rows of token t that take part, in ascending j, and their gates, in shared memory; returns their count
template <typename G>
__device__ __forceinline__ int token_rows(const UnsortParams& p, int64_t t, int lane, int* s_row, float* s_gate) {
    int n = 0;
    for (int j0 = 0; j0 < p.k; j0 += 32) {
        const int j = j0 + lane;
        int r = -1;
        float g = 1.f;
        if (j < p.k) {
            r = p.row[t * p.k + j];
            if (r < -1 || r >= p.rows) {
                set_status(p.status, MOE_ERR_BAD_INDEX);
                r = -1;
            }
            if (r >= 0 && p.gates) g = to_f32(static_cast<const G*>(p.gates)[t * p.k + j]);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, r >= 0);
        if (r >= 0) {
            const int pos = n + __popc(m & lanemask_lt());
            s_row[pos] = r;
            s_gate[pos] = g;
        }
        n += __popc(m);
    }
    __syncwarp();
    return n;
}

// acc[u] += sum over the J rows from j on, in their order: J x U loads in flight
template <typename T, typename V, int J, int U>
__device__ __forceinline__ void add_rows(const T* ys, int64_t ldys, const int* s_row, const float* s_gate, int j,
                                         const int64_t (&col)[U], float (&acc)[U][Vec<T, V>::kN]) {
    V r[J][U];
#pragma unroll
    for (int i = 0; i < J; ++i) {
        const T* src = ys + (int64_t)s_row[j + i] * ldys;
#pragma unroll
        for (int u = 0; u < U; ++u) r[i][u] = *reinterpret_cast<const V*>(src + col[u]);
    }
#pragma unroll
    for (int i = 0; i < J; ++i) {
        const float g = s_gate[j + i];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[Vec<T, V>::kN];
            Vec<T, V>::unpack(r[i][u], v);
#pragma unroll
            for (int e = 0; e < Vec<T, V>::kN; ++e) acc[u][e] = fmaf(g, v[e], acc[u][e]);
        }
    }
}

// y[t] = base[t] + sum_j gate ys[row], j ascending, in fp32.  `split` warps share a token's columns; a warp takes U
// vectors per lane at a time and J rows, so that J x U loads are in flight: without that the rows come one latency
// after another.
template <typename T, typename G, typename V, int J, int U>
__global__ void __launch_bounds__(kThreads) unsort_kernel(const UnsortParams p) {
    constexpr int N = Vec<T, V>::kN;
    __shared__ int s_row[kWarps][kMaxK];
    __shared__ float s_gate[kWarps][kMaxK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t t = unit / p.split;
    if (t >= p.T) return;
    const int n = token_rows<G>(p, t, lane, s_row[warp], s_gate[warp]);
    const T* ys = static_cast<const T*>(p.ys);
    const T* base = p.base ? static_cast<const T*>(p.base) + t * p.ldbase : nullptr;
    T* y = static_cast<T*>(p.y) + t * p.ldy;
    for (int64_t c0 = (unit - t * p.split) * (32 * N * U); c0 < p.N; c0 += (int64_t)p.split * (32 * N * U)) {
        int64_t col[U];
        float acc[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + 32 * N * u + lane * N;
            col[u] = c < p.N ? c : p.N - N;  // past the end: the last vector again, not stored
#pragma unroll
            for (int e = 0; e < N; ++e) acc[u][e] = 0.f;
        }
        if (base) {
            V r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = *reinterpret_cast<const V*>(base + col[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) Vec<T, V>::unpack(r[u], acc[u]);
        }
        int j = 0;
        for (; n - j >= J; j += J) add_rows<T, V, J, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc);
        if (J > 4 && n - j >= 4) add_rows<T, V, 4, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc), j += 4;
        if (J > 2 && n - j >= 2) add_rows<T, V, 2, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc), j += 2;
        if (n - j >= 1) add_rows<T, V, 1, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * N * u + lane * N < p.N) *reinterpret_cast<V*>(y + col[u]) = Vec<T, V>::pack(acc[u]);
    }
}

// dys[row] = gate dy[t] and dgates[t, j] = dy[t] . ys[row], one warp per (t, j).  The warps of a token sit in one
// block, so that dy's row comes from memory once and from the first-level cache after that.
template <typename T, typename G, typename V, int U, bool DYS, bool DGATES>
__global__ void __launch_bounds__(kThreads) unsort_backward_kernel(const UnsortParams p) {
    constexpr int N = Vec<T, V>::kN;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= p.T * p.k) return;
    const int64_t t = unit / p.k;
    const int64_t r = p.row[unit];
    float dot = 0.f;
    if (r >= 0 && r < p.rows) {
        const float g = p.gates ? to_f32(static_cast<const G*>(p.gates)[unit]) : 1.f;
        const T* dy = static_cast<const T*>(p.dy) + t * p.lddy;
        const T* ys = static_cast<const T*>(p.ys) + r * p.ldys;
        T* dys = static_cast<T*>(p.y) + r * p.ldy;
        for (int64_t c0 = 0; c0 < p.N; c0 += 32 * N * U) {
            V a[U], b[U];
            int64_t col[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + 32 * N * u + lane * N;
                col[u] = c < p.N ? c : p.N - N;
                a[u] = *reinterpret_cast<const V*>(dy + col[u]);
                if (DGATES) b[u] = *reinterpret_cast<const V*>(ys + col[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float d[N];
                Vec<T, V>::unpack(a[u], d);
                const bool in = c0 + 32 * N * u + lane * N < p.N;
                if (DGATES) {
                    float v[N];
                    Vec<T, V>::unpack(b[u], v);
                    if (in) {
#pragma unroll
                        for (int e = 0; e < N; ++e) dot = fmaf(d[e], v[e], dot);
                    }
                }
                if (DYS && in) {
#pragma unroll
                    for (int e = 0; e < N; ++e) d[e] *= g;
                    *reinterpret_cast<V*>(dys + col[u]) = Vec<T, V>::pack(d);
                }
            }
        }
    } else if (r != -1 && lane == 0) {
        set_status(p.status, MOE_ERR_BAD_INDEX);
    }
    if (DGATES) {
        dot = warp_sum(dot);
        if (lane == 0) p.dgates[unit] = dot;
    }
}

constexpr int kFill = 16;  // warps per SM that a short batch is spread over

template <typename T, typename G, typename V, int J, int U>
int launch_unsort(UnsortParams p, cudaStream_t stream) {
    const int64_t groups = (p.N + 32 * Vec<T, V>::kN * U - 1) / (32 * Vec<T, V>::kN * U);
    const int64_t want = (int64_t)device_sm_count() * kFill / p.T;
    p.split = (int)(want < 1 ? 1 : want < groups ? want : groups);
    const int64_t grid = (p.T * p.split + kWarps - 1) / kWarps;
    unsort_kernel<T, G, V, J, U><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return launch_status();
}

template <typename T, typename G, typename V, int U>
int launch_backward(const UnsortParams& p, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.T * p.k + kWarps - 1) / kWarps);
    if (p.y && p.dgates) unsort_backward_kernel<T, G, V, U, true, true><<<grid, kThreads, 0, stream>>>(p);
    else if (p.y) unsort_backward_kernel<T, G, V, U, true, false><<<grid, kThreads, 0, stream>>>(p);
    else unsort_backward_kernel<T, G, V, U, false, true><<<grid, kThreads, 0, stream>>>(p);
    return launch_status();
}

// Rows that 16 bytes divide, or single elements (two loads for each of the 16-byte form's).
template <typename T, typename G>
int launch_back(const UnsortParams& p, bool backward, bool vec, cudaStream_t stream) {
    if (backward) return vec ? launch_backward<T, G, uint4, 4>(p, stream) : launch_backward<T, G, T, 8>(p, stream);
    if (p.k >= 6) return vec ? launch_unsort<T, G, uint4, 8, 1>(p, stream) : launch_unsort<T, G, T, 8, 2>(p, stream);
    if (p.k >= 3) return vec ? launch_unsort<T, G, uint4, 4, 2>(p, stream) : launch_unsort<T, G, T, 4, 4>(p, stream);
    return vec ? launch_unsort<T, G, uint4, 2, 4>(p, stream) : launch_unsort<T, G, T, 2, 8>(p, stream);
}

int unsort_run(const UnsortParams& p, bool backward, moe_dtype dtype, moe_dtype gate_dtype, cudaStream_t stream) {
    const size_t es = dtype_size(dtype);
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.ys) | reinterpret_cast<uintptr_t>(p.base) |
                          reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.dy) |
                          (uintptr_t)(p.N * es) | (uintptr_t)(p.ldys * es) | (uintptr_t)(p.ldy * es) |
                          (uintptr_t)(p.ldbase * es) | (uintptr_t)(p.lddy * es);
    const bool vec = (all & 15) == 0;
    const bool gb = gate_dtype == MOE_BF16;
    if (dtype == MOE_BF16)
        return gb ? launch_back<__nv_bfloat16, __nv_bfloat16>(p, backward, vec, stream)
                  : launch_back<__nv_bfloat16, float>(p, backward, vec, stream);
    return gb ? launch_back<float, __nv_bfloat16>(p, backward, vec, stream)
              : launch_back<float, float>(p, backward, vec, stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_sort_workspace_size(int64_t T, int32_t k, int32_t E) {
    if (T < 1 || k < 1 || E < 1 || k > kMaxK || E > kMaxE || T >= (int64_t(1) << 30) || T * k >= (int64_t(1) << 30))
        return 0;
    return sort_workspace(T, k, E);
}

extern "C" int moe_sort(const int64_t* selected, int64_t T, int32_t k, int32_t E, const void* x, moe_dtype dtype,
                        int64_t D, int64_t ldx, int32_t* offsets, int32_t* row, int32_t* source, void* xs,
                        int64_t ldxs, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                        moe_stream_t stream) {
    const int rc = sort_check(selected, T, k, E, offsets, row, source);
    if (rc != MOE_OK) return rc;
    SortParams p{};
    p.selected = selected, p.T = T, p.k = k, p.E = E;
    p.offsets = offsets, p.row = row, p.source = source, p.status = dev_status;
    int op = ROW_NONE;
    if (x) {
        MOE_REQUIRE(valid_dtype(dtype) && xs && D >= 1 && ldx >= D && ldxs >= D, MOE_ERR_INVALID_ARG);
        p.x = x, p.D = D, p.ldx = ldx, p.xs = xs, p.ldxs = ldxs;
        op = ROW_COPY;
    }
    return sort_run(p, op, dtype, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_sort_i8(const int64_t* selected, int64_t T, int32_t k, int32_t E, const void* x, moe_dtype dtype,
                           int64_t D, int64_t ldx, int32_t* offsets, int32_t* row, int32_t* source, int8_t* xq,
                           int64_t ldxq, float* xscale, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                           moe_stream_t stream) {
    const int rc = sort_check(selected, T, k, E, offsets, row, source);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(valid_dtype(dtype) && D >= 1 && ldx >= D && ldxq >= D, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T == 0 || (x && xq && xscale), MOE_ERR_INVALID_ARG);
    SortParams p{};
    p.selected = selected, p.T = T, p.k = k, p.E = E;
    p.offsets = offsets, p.row = row, p.source = source, p.status = dev_status;
    p.x = x, p.D = D, p.ldx = ldx, p.xs = xq, p.ldxs = ldxq, p.xscale = xscale;
    return sort_run(p, ROW_I8, dtype, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_unsort(const void* ys, int64_t ldys, int64_t rows, const int32_t* row, const void* gates,
                          moe_dtype gate_dtype, int64_t T, int32_t k, int64_t N, const void* base, int64_t ldbase,
                          void* y, int64_t ldy, moe_dtype dtype, int32_t* dev_status, moe_stream_t stream) {
    MOE_REQUIRE(valid_dtype(dtype) && valid_dtype(gate_dtype), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T >= 0 && k >= 1 && N >= 1 && rows >= 0 && ldys >= N && ldy >= N, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T == 0 || (row && y), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE((rows == 0 || ys) && (!base || ldbase >= N), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(k <= kMaxK && T < (int64_t(1) << 30) && T * k < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);
    if (T == 0) return MOE_OK;
    UnsortParams p{};
    p.ys = ys, p.ldys = ldys, p.rows = rows, p.row = row, p.gates = gates, p.T = T, p.k = k, p.N = N;
    p.base = base, p.ldbase = base ? ldbase : 0, p.y = y, p.ldy = ldy, p.status = dev_status;
    return unsort_run(p, false, dtype, gate_dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_unsort_backward(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows,
                                   const int32_t* row, const void* gates, moe_dtype gate_dtype, int64_t T, int32_t k,
                                   int64_t N, void* dys, int64_t lddys, float* dgates, moe_dtype dtype,
                                   int32_t* dev_status, moe_stream_t stream) {
    MOE_REQUIRE(valid_dtype(dtype) && valid_dtype(gate_dtype), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T >= 0 && k >= 1 && N >= 1 && rows >= 0 && lddy >= N, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T == 0 || (row && dy), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(!dgates || ((rows == 0 || ys) && ldys >= N), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(!dys || lddys >= N, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(k <= kMaxK && T < (int64_t(1) << 30) && T * k < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);
    if (T == 0 || (!dys && !dgates)) return MOE_OK;
    UnsortParams p{};
    p.ys = dgates ? ys : nullptr, p.ldys = dgates ? ldys : 0, p.rows = rows, p.row = row, p.gates = gates;
    p.T = T, p.k = k, p.N = N, p.y = dys, p.ldy = dys ? lddys : 0, p.dy = dy, p.lddy = lddy, p.dgates = dgates;
    p.status = dev_status;
    return unsort_run(p, true, dtype, gate_dtype, reinterpret_cast<cudaStream_t>(stream));
}
