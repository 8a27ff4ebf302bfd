// moe_sort, moe_sort_i8, moe_unsort, moe_unsort_backward: tokens sorted by
// expert into packed rows without a capacity, and back.
//
// Assignments i = t k + j are ordered by (expert, i): row = offsets[e] + #{earlier
// assignments to e}.  The order is a counting sort.  Up to kSmallCount assignments one
// launch does everything: every block counts all the keys itself, so no block waits
// for another, and copies (or quantises) its tokens' rows.  Above, hist_kernel counts the
// keys of each super-block, rank_kernel adds those of all the super-blocks (at most
// kMaxCounts counts, so each block does it for itself) and ranks the keys of its own by
// warp, and a last kernel writes the packed rows:
// one warp per assignment, so that a block's warps read the same token's row and write
// different ones (short blocks: the same rows written by 512 long-lived blocks took 117 us
// for T = 16384, k = 8, D = 2048 bf16).  Rows in 8 bits are quantised once per token, into
// shared memory.  Integer counts do not depend on the order of the shared-memory atomics
// that make them, so the rows are unique.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

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
// Assignments per super-block: a 64th of all, from 1024 to 4096, or more where the counts would pass kMaxCounts.
// Larger ones make rank_kernel's chain longer, smaller ones its reads of all the counts: the order of n = 131072,
// E = 256 takes 19.2 us with 1024, 10.9 with 2048 and 13.5 with 4096; n = 16382, E = 64 6.3, 7.7 and 11.9 us.
constexpr int64_t kMinSuper = 1024, kMaxSuper = 4096;
constexpr int64_t kMaxCounts = 65536;  // super-blocks * E that every block of rank_kernel reads
constexpr int kHistThreads = 512;
constexpr int kRankThreads = 512;
constexpr int kRankWarps = kRankThreads / 32;

// What the row kernel does with each token's row of x.
enum RowOp : int { ROW_NONE = 0, ROW_COPY = 1, ROW_I8 = 2 };

struct SortParams {
    const int64_t* selected;
    int64_t T;
    int k, E;
    int64_t n;            // T * k
    int64_t super;        // assignments per super-block
    int64_t block_tokens; // tokens per block of the one-launch form
    const int32_t* hist;  // (super-blocks, E) counts, from hist_kernel
    int n_super;
    int32_t* offsets;
    int32_t* row;
    int32_t* source;
    const void* x;
    int64_t D, ldx;
    void* xs;
    int64_t ldxs;
    float* xscale;
    bool vecx, vecq;      // ROW_I8: x rows start on 16 bytes, xs rows on 8
    int32_t* status;
};

// expert of an assignment, -1 for one that takes no part
__device__ __forceinline__ int key_of(int64_t e, int E, int32_t* status) {
    if (e >= 0 && e < E) return (int)e;
    if (e != -1) set_status(status, MOE_ERR_BAD_INDEX);
    return -1;
}

// hist[super-block][e]: its keys of expert e
__global__ void __launch_bounds__(kHistThreads) hist_kernel(const SortParams p, int32_t* __restrict__ hist) {
    extern __shared__ int s_cnt[];
    for (int e = threadIdx.x; e < p.E; e += kHistThreads) s_cnt[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * p.super;
    const int64_t last = first + p.super < p.n ? first + p.super : p.n;
    pdl_wait();
    pdl_next();
#pragma unroll 8
    for (int64_t i = first + threadIdx.x; i < last; i += kHistThreads) {
        const int key = key_of(p.selected[i], p.E, p.status);
        if (key >= 0) atomicAdd(&s_cnt[key], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kHistThreads) hist[(int64_t)blockIdx.x * p.E + e] = s_cnt[e];
}

// rows of the chunk's 32 assignments: next[key] + the lanes before with the same key; next moves on
__device__ __forceinline__ int rank_chunk(int key, int* next, int lane) {
    const uint32_t match = __match_any_sync(0xffffffffu, key);
    int r = -1;
    if (key >= 0) r = next[key] + __popc(match & lanemask_lt());
    __syncwarp();
    if (key >= 0 && __ffs(match) - 1 == lane) next[key] += __popc(match);
    __syncwarp();
    return r;
}

__device__ __forceinline__ void put_rank(const SortParams& p, int64_t i, int r, int total) {
    p.row[i] = r;
    if (r >= 0) p.source[r] = (int32_t)i;
    if (i >= total) p.source[i] = -1;  // behind the last row
}

// One block per super-block: its warps take consecutive pieces, count them, and rank them from where the warps before
// end.  Shared memory: counts (warps, E).
__global__ void __launch_bounds__(kRankThreads) rank_kernel(const SortParams p, int warps) {
    extern __shared__ int s_cnt[];
    __shared__ int s_total[kMaxE + 1];    // sums over all super-blocks, then over the experts before
    __shared__ int s_before[kMaxE];       // sums over the super-blocks before this one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < warps * p.E; i += kRankThreads) s_cnt[i] = 0;
    for (int e = threadIdx.x; e < p.E; e += kRankThreads) s_total[e] = s_before[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * p.super;
    const int64_t last = first + p.super < p.n ? first + p.super : p.n;
    const int64_t piece = (p.super + warps * 32 - 1) / (warps * 32) * 32;
    const int64_t w0 = first + warp * piece, w1 = w0 + piece < last ? w0 + piece : last;
    int* cnt = s_cnt + warp * p.E;
    pdl_wait();
    pdl_next();
    if (warp < warps) {
#pragma unroll 2
        for (int64_t i = w0 + lane; i < w1; i += 32) {
            const int key = key_of(p.selected[i], p.E, nullptr);
            if (key >= 0) atomicAdd(&cnt[key], 1);
        }
    }
    // the threads of an expert share the super-blocks
    const int segs = p.E < kRankThreads ? kRankThreads / p.E : 1;
    const int seg = p.E < kRankThreads ? threadIdx.x / p.E : 0;
    for (int e = threadIdx.x - seg * p.E; seg < segs && e < p.E; e += kRankThreads) {
        int total = 0, before = 0;
#pragma unroll 8
        for (int i = seg; i < p.n_super; i += segs) {
            // from the own super-block on, so that the blocks do not all ask for the same counts at once
            const int a = i + blockIdx.x < p.n_super ? i + blockIdx.x : i + blockIdx.x - p.n_super;
            const int c = p.hist[(int64_t)a * p.E + e];
            total += c;
            before += a < blockIdx.x ? c : 0;
        }
        atomicAdd(&s_total[e], total);
        atomicAdd(&s_before[e], before);
    }
    __syncthreads();
    block_scan<kRankThreads>(s_total, p.E);
    for (int e = threadIdx.x; e < p.E; e += kRankThreads) {
        int run = s_total[e] + s_before[e];
        for (int w = 0; w < warps; ++w) {
            const int c = s_cnt[w * p.E + e];
            s_cnt[w * p.E + e] = run;
            run += c;
        }
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += kRankThreads) p.offsets[e] = s_total[e];
    __syncthreads();
    if (warp >= warps) return;
    const int total = s_total[p.E];
#pragma unroll 2
    for (int64_t c = w0; c < w1; c += 32) {
        const int64_t i = c + lane;
        const int r = rank_chunk(i < w1 ? key_of(p.selected[i], p.E, nullptr) : -1, cnt, lane);
        if (i < w1) put_rank(p, i, r, total);
    }
}

// The TEAM threads from 0 on copy a row to the rows dst[0..k) of the packed matrix (-1: none).
// V: the widest vector that every row start and the row length allow.
template <int TEAM, typename V>
__device__ __forceinline__ void copy_row(const SortParams& p, int64_t t, const int* rows, int tid) {
    constexpr int kBatch = 8;
    const int64_t nv = p.D, ldx = p.ldx, lds = p.ldxs;  // in units of V
    const V* src = static_cast<const V*>(p.x) + t * ldx;
    V* dst = static_cast<V*>(p.xs);
    for (int64_t v0 = tid; v0 < nv; v0 += TEAM * kBatch) {
        V r[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (v0 + TEAM * u < nv) r[u] = src[v0 + TEAM * u];
        for (int j = 0; j < p.k; ++j) {
            const int rw = rows[j];
            if (rw < 0) continue;
            V* d = dst + (int64_t)rw * lds;
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (v0 + TEAM * u < nv) d[v0 + TEAM * u] = r[u];
        }
    }
}

// The one-launch form: the order, and the rows (OP).  WARPS: warps per token, one or the whole block.
// Shared memory: s_cnt[E + 1] (next row of each expert), s_off[E + 1], s_row[block_tokens * k].
template <int OP, int WARPS, typename V>
__global__ void __launch_bounds__(kThreads, OP == ROW_I8 ? 3 : 4) small_kernel(const SortParams p) {
    extern __shared__ int s_dyn[];
    __shared__ uint32_t s_max[kWarps];
    int* s_cnt = s_dyn;
    int* s_off = s_cnt + p.E + 1;
    int* s_row = s_off + p.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    const int ntok = (int)(p.T - t0 < p.block_tokens ? p.T - t0 : p.block_tokens);
    const int64_t first = t0 * p.k;  // this block's assignments: [first, first + n_own)
    const int n_own = ntok * p.k;
    for (int e = threadIdx.x; e < p.E; e += kThreads) s_cnt[e] = s_off[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_next();
#pragma unroll 4
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
    __syncthreads();

    // ranks of the own assignments, 32 at a time in order
    if (warp == 0) {
        const int total = s_off[p.E];
        for (int c = 0; c < n_own; c += 32) {
            const int li = c + lane;
            const int r = rank_chunk(li < n_own ? key_of(p.selected[first + li], p.E, nullptr) : -1, s_cnt, lane);
            if (li < n_own) {
                s_row[li] = r;
                put_rank(p, first + li, r, total);
            }
        }
    }
    if (OP == ROW_NONE) return;
    __syncthreads();
    const int tid = WARPS == 1 ? lane : threadIdx.x;
    for (int t = WARPS == 1 ? warp : 0; t < ntok; t += kWarps / WARPS) {
        const int* rows = s_row + t * p.k;
        if constexpr (OP == ROW_COPY) copy_row<32 * WARPS, V>(p, t0 + t, rows, tid);
        if constexpr (OP == ROW_I8) {
            int8_t* q = static_cast<int8_t*>(p.xs);
            const float scale = quantize_row<WARPS>(static_cast<const V*>(p.x) + (t0 + t) * p.ldx, p.D, rows, p.k, q,
                                                    p.ldxs, p.vecx, p.vecq, s_max, p.status);
            for (int j = tid; j < p.k; j += 32 * WARPS)
                if (rows[j] >= 0) p.xscale[rows[j]] = scale;
        }
    }
}

// xs[row[t, j]] = x[t] (both in units of V), one assignment per 2^shift lanes.
template <typename V>
__global__ void __launch_bounds__(kThreads) scatter_kernel(const SortParams p, int shift) {
    // 16 bytes: four at a time, so that more warps are resident (D = 2048 bf16: 109 us, 114 with eight)
    constexpr int kBatch = sizeof(V) == 16 ? 4 : 8;
    const int lane = threadIdx.x & 31, team = 1 << shift;
    const int64_t i = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 >> shift) + (lane >> shift);
    pdl_wait();
    pdl_next();
    if (i >= p.n) return;
    const int r = p.row[i];
    if (r < 0) return;
    const V* src = static_cast<const V*>(p.x) + (i / p.k) * p.ldx;
    V* dst = static_cast<V*>(p.xs) + r * p.ldxs;
    for (int64_t v0 = lane & (team - 1); v0 < p.D; v0 += team * kBatch) {
        V v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (v0 + team * u < p.D) v[u] = src[v0 + team * u];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (v0 + team * u < p.D) __stcs(dst + v0 + team * u, v[u]);
    }
}

constexpr int kI8Threads = 128;
constexpr int kI8Seg = 8192;  // values of a row in shared memory at a time

// The same in 8 bits, for rows too long for scatter_i8_team_kernel: a block per token quantises its row into shared memory,
// from where each warp writes every fourth of the token's rows.  Where the rows do not lie on 16 bytes a warp per token
// writes them as it goes.
template <typename T, bool SHARED>
__global__ void __launch_bounds__(kI8Threads) scatter_i8_kernel(const SortParams p) {
    __shared__ uint32_t s_max[kI8Threads / 32];
    __shared__ int s_row[SHARED ? 1 : kI8Threads / 32][kMaxK];
    extern __shared__ uint4 s_q[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = SHARED ? blockIdx.x : (int64_t)blockIdx.x * (kI8Threads / 32) + warp;
    pdl_wait();
    pdl_next();
    if (t >= p.T) return;
    int* rows = s_row[SHARED ? 0 : warp];
    for (int j = SHARED ? threadIdx.x : lane; j < p.k; j += SHARED ? kI8Threads : 32) rows[j] = p.row[t * p.k + j];
    const T* src = static_cast<const T*>(p.x) + t * p.ldx;
    int8_t* q = static_cast<int8_t*>(p.xs);
    float scale;
    if constexpr (SHARED) {
        const uint32_t m = row_max<kI8Threads / 32>(src, p.D, p.vecx, s_max);  // its barriers also bring `rows` to all threads
        const RowQuant r = row_quant(m, p.status, threadIdx.x == 0 && reports(m, rows, p.k));
        scale = r.scale;
        for (int64_t s0 = 0; s0 < p.D; s0 += kI8Seg) {
            const int len = (int)(p.D - s0 < kI8Seg ? p.D - s0 : kI8Seg);
            if (s0 > 0) __syncthreads();  // the segment before has been written
            for (int c = threadIdx.x * kChunk<T>; c < len; c += kI8Threads * kChunk<T>) {
                Raw<T> x;
                x.load(src + s0 + c, len - c, p.vecx);
                uint32_t o[kChunk<T> / 4];
                quantize_chunk(x, r, o);
                store_chunk(reinterpret_cast<int8_t*>(s_q) + c, o, kChunk<T>, true);
            }
            __syncthreads();
            for (int j = warp; j < p.k; j += kI8Threads / 32) {
                if (rows[j] < 0) continue;
                int8_t* dst = q + (int64_t)rows[j] * p.ldxs + s0;
                for (int c = lane; c < len / 16; c += 32) __stcs(reinterpret_cast<uint4*>(dst) + c, s_q[c]);
                for (int c = len / 16 * 16 + lane; c < len; c += 32) dst[c] = reinterpret_cast<const int8_t*>(s_q)[c];
            }
        }
    } else {
        __syncwarp();
        scale = quantize_row<1>(src, p.D, rows, p.k, q, p.ldxs, p.vecx, p.vecq, s_max, p.status);
    }
    for (int j = SHARED ? threadIdx.x : lane; j < p.k; j += SHARED ? kI8Threads : 32)
        if (rows[j] >= 0) p.xscale[rows[j]] = scale;
}

// The same for rows of up to four steps of a team of TEAM warps, which holds its token's row in registers and quantises it
// once.  T = 16384, rows alone: bf16 D = 2048 24 us with k = 1 and 56 with k = 8 (32 and 61 through shared memory), D = 1024
// 10.5 and 30 (23 and 38); fp32 D = 2048 32 and 65 (45 and 72).  Eight steps of four warps instead of shared memory gain at
// fp32 D = 4096 (130 -> 127 us, k = 8) and lose at bf16 D = 8192 (85 -> 98, k = 1).
template <typename T, int TEAM>
__global__ void __launch_bounds__(kI8Threads) scatter_i8_team_kernel(const SortParams p) {
    constexpr int STEPS = 4, kStride = 32 * TEAM * kChunk<T>;
    __shared__ uint32_t s_max[kI8Threads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x % (32 * TEAM), first = tid * kChunk<T>;
    const int64_t t = (int64_t)blockIdx.x * (kI8Threads / 32 / TEAM) + warp / TEAM;
    pdl_wait();
    pdl_next();
    if (t >= p.T) return;
    int rows[kMaxK / 32];
#pragma unroll
    for (int h = 0; h < kMaxK / 32; ++h) rows[h] = lane + 32 * h < p.k ? p.row[t * p.k + lane + 32 * h] : -1;
    const T* src = static_cast<const T*>(p.x) + t * p.ldx;
    Raw<T> x[STEPS];
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        if (s * kStride < p.D) x[s].load(src + first + s * kStride, p.D - first - s * kStride, p.vecx);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        if (s * kStride < p.D) m = x[s].max_bits(m);
    m = __reduce_max_sync(0xffffffffu, Raw<T>::join(m));
    if constexpr (TEAM > 1) {
        if (lane == 0) s_max[warp] = m;
        // constant barriers: with one in a register a block is given all 16, and fewer blocks are resident
        if (TEAM == 4 || warp < TEAM) asm volatile("bar.sync 1, %0;" ::"n"(32 * TEAM) : "memory");
        else asm volatile("bar.sync 2, %0;" ::"n"(32 * TEAM) : "memory");
#pragma unroll
        for (int w = 0; w < TEAM; ++w) m = max(m, s_max[warp / TEAM * TEAM + w]);
    }
    bool report = tid == 0;
    if (m >= 0x7f800000u) {  // a token without rows may hold anything; it is loaded before they are known, and written nowhere
        bool any = false;
#pragma unroll
        for (int h = 0; h < kMaxK / 32; ++h) any |= rows[h] >= 0;
        report &= __any_sync(0xffffffffu, any);
    }
    const RowQuant r = row_quant(m, p.status, report);
    uint32_t o[STEPS][kChunk<T> / 4];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        if (s * kStride < p.D) quantize_chunk(x[s], r, o[s]);
#pragma unroll
    for (int h = 0; h < kMaxK / 32; ++h) {
        for (int j = 0; j < 32 && j + 32 * h < p.k; ++j) {
            const int row = __shfl_sync(0xffffffffu, rows[h], j);
            if (row < 0) continue;
            int8_t* q = static_cast<int8_t*>(p.xs) + (int64_t)row * p.ldxs + first;
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                if (first + s * kStride < p.D) store_chunk(q + s * kStride, o[s], p.D - first - s * kStride, p.vecq);
        }
        if (tid < 32 && rows[h] >= 0) p.xscale[rows[h]] = r.scale;
    }
}

// super-blocks, or the one-launch form's blocks, for T tokens of k assignments
struct SortPlan {
    bool small;
    int64_t super, n_super, block_tokens;
};

SortPlan sort_plan(int64_t T, int32_t k, int32_t E) {
    SortPlan s{};
    const int64_t n = T * k;
    const int64_t sms = device_sm_count();
    s.small = n <= kSmallCount;
    s.block_tokens = (T + 2 * sms - 1) / (2 * sms);
    if (s.block_tokens < 1) s.block_tokens = 1;
    s.super = n / 64 < kMinSuper ? kMinSuper : n / 64 > kMaxSuper ? kMaxSuper : n / 64;
    const int64_t most = kMaxCounts / E;
    if (n > most * s.super) s.super = (n + most - 1) / most;
    s.n_super = (n + s.super - 1) / s.super;
    return s;
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
    const SortPlan s = sort_plan(T, k, E);
    return s.small ? 0 : align_up((size_t)s.n_super * E * sizeof(int32_t), 256);
}

// the widest vector that the rows' starts, strides and length allow: their units of 1 << result bytes
int row_vector(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t D, size_t es) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | (uintptr_t)(D * es) |
                          (uintptr_t)(lda * es) | (uintptr_t)(ldb * es);
    return (all & 15) == 0 ? 4 : (all & 3) == 0 ? 2 : 1;
}

int launch_scatter(SortParams p, size_t es, cudaStream_t stream) {
    const int bits = row_vector(p.x, p.ldx, p.xs, p.ldxs, p.D, es);
    p.D = p.D * es >> bits, p.ldx = p.ldx * es >> bits, p.ldxs = p.ldxs * es >> bits;
    int shift = 0;
    while (shift < 5 && (1 << shift) < p.D) ++shift;
    const int64_t per_block = kWarps * (32 >> shift);
    const int64_t grid = (p.n + per_block - 1) / per_block;
    if (bits == 4) return launch_pdl(scatter_kernel<uint4>, grid, kThreads, 0, stream, p, shift);
    if (bits == 2) return launch_pdl(scatter_kernel<uint32_t>, grid, kThreads, 0, stream, p, shift);
    return launch_pdl(scatter_kernel<uint16_t>, grid, kThreads, 0, stream, p, shift);
}

template <typename T>
int launch_scatter_i8(const SortParams& p, cudaStream_t stream) {
    constexpr int kPer = kI8Threads / 32;
    const int64_t warps = (p.T + kPer - 1) / kPer;
    constexpr int kStep = 32 * kChunk<T>;
    if (p.D <= kStep * 4) return launch_pdl(scatter_i8_team_kernel<T, 1>, warps, kI8Threads, 0, stream, p);
    if (p.D <= kStep * 8) return launch_pdl(scatter_i8_team_kernel<T, 2>, (p.T + 1) / 2, kI8Threads, 0, stream, p);
    if (p.D <= kStep * 16) return launch_pdl(scatter_i8_team_kernel<T, 4>, p.T, kI8Threads, 0, stream, p);
    if (!aligned16(p.xs) || p.ldxs % 16) return launch_pdl(scatter_i8_kernel<T, false>, warps, kI8Threads, 0, stream, p);
    const size_t smem = align_up((size_t)(p.D < kI8Seg ? p.D : kI8Seg), 16);
    return launch_pdl(scatter_i8_kernel<T, true>, p.T, kI8Threads, smem, stream, p);
}

// The order, and the rows by token (op), few blocks: every block counts all the keys.
int sort_small(SortParams p, int op, moe_dtype dtype, cudaStream_t stream) {
    const int64_t blocks = (p.T + p.block_tokens - 1) / p.block_tokens;
    const size_t smem = sizeof(int) * (2 * ((size_t)p.E + 1) + (size_t)p.block_tokens * p.k);
    const auto go = [&](auto kernel) { return launch_pdl(kernel, blocks, kThreads, smem, stream, p); };
    const bool share = p.block_tokens < kWarps;  // few tokens per block: its warps share each row
    if (op == ROW_NONE) return go(small_kernel<ROW_NONE, 1, float>);
    if (op == ROW_I8) {
        if (dtype == MOE_BF16)
            return share ? go(small_kernel<ROW_I8, kWarps, __nv_bfloat16>)
                         : go(small_kernel<ROW_I8, 1, __nv_bfloat16>);
        return share ? go(small_kernel<ROW_I8, kWarps, float>) : go(small_kernel<ROW_I8, 1, float>);
    }
    const size_t es = dtype_size(dtype);
    const int bits = row_vector(p.x, p.ldx, p.xs, p.ldxs, p.D, es);
    p.D = p.D * es >> bits, p.ldx = p.ldx * es >> bits, p.ldxs = p.ldxs * es >> bits;
    if (bits == 4) return share ? go(small_kernel<ROW_COPY, kWarps, uint4>) : go(small_kernel<ROW_COPY, 1, uint4>);
    if (bits == 2)
        return share ? go(small_kernel<ROW_COPY, kWarps, uint32_t>) : go(small_kernel<ROW_COPY, 1, uint32_t>);
    return share ? go(small_kernel<ROW_COPY, kWarps, uint16_t>) : go(small_kernel<ROW_COPY, 1, uint16_t>);
}

// The order, then the rows of x (op).
int sort_run(SortParams p, int op, moe_dtype dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (p.T == 0) {
        MOE_CUDA_TRY(cudaMemsetAsync(p.offsets, 0, sizeof(int32_t) * ((size_t)p.E + 1), stream));
        return MOE_OK;
    }
    const SortPlan s = sort_plan(p.T, p.k, p.E);
    p.n = p.T * p.k;
    p.super = s.super;
    p.block_tokens = s.block_tokens;
    if (op == ROW_I8) {
        p.vecx = aligned16(p.x) && (p.ldx * dtype_size(dtype)) % 16 == 0;
        p.vecq = (reinterpret_cast<uintptr_t>(p.xs) & 7) == 0 && p.ldxs % 8 == 0;
    }
    if (s.small) return sort_small(p, op, dtype, stream);

    MOE_REQUIRE(workspace && aligned16(workspace) && workspace_bytes >= sort_workspace(p.T, p.k, p.E), MOE_ERR_WORKSPACE);
    int32_t* hist = static_cast<int32_t*>(workspace);
    p.hist = hist, p.n_super = (int)s.n_super;
    int rc = launch_pdl(hist_kernel, s.n_super, kHistThreads, sizeof(int) * p.E, stream, p, hist);
    if (rc != MOE_OK) return rc;
    const int warps = 7168 / p.E < kRankWarps ? 7168 / p.E : kRankWarps;  // as many as 28 KB of counts allow
    rc = launch_pdl(rank_kernel, s.n_super, kRankThreads, sizeof(int) * p.E * warps, stream, p, warps);
    if (rc != MOE_OK || op == ROW_NONE) return rc;
    if (op == ROW_COPY) return launch_scatter(p, dtype_size(dtype), stream);
    return dtype == MOE_BF16 ? launch_scatter_i8<__nv_bfloat16>(p, stream) : launch_scatter_i8<float>(p, stream);
}

// ------------------------------- and back -----------------------------------

// V: 16 or 4 bytes, or one value, of a row of T (8 bytes of bf16 beside 16 of fp32); its values as fp32
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

// BYTES consecutive bytes
template <int BYTES>
using Bytes = std::conditional_t<BYTES == 16, uint4,
                                 std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, uint32_t, uint16_t>>>;

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
// after another.  Types: T of ys, TB of base, TY of y.  fp32 rows into bf16 tokens round each sum once; rows in bf16 halve
// the bytes and round every term first.  T = 16384, k = 8, D = 2048: 174 us and 104; T = 16: 2.4 both.
template <typename T, typename G, typename V, int J, int U, typename TB, typename TY>
__global__ void __launch_bounds__(kThreads) unsort_kernel(const UnsortParams p) {
    constexpr int N = Vec<T, V>::kN;
    using VB = Bytes<N * sizeof(TB)>;
    using VY = Bytes<N * sizeof(TY)>;
    __shared__ int s_row[kWarps][kMaxK];
    __shared__ float s_gate[kWarps][kMaxK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t t = unit / p.split;
    pdl_wait();
    pdl_next();
    if (t >= p.T) return;
    const int n = token_rows<G>(p, t, lane, s_row[warp], s_gate[warp]);
    const T* ys = static_cast<const T*>(p.ys);
    const TB* base = p.base ? static_cast<const TB*>(p.base) + t * p.ldbase : nullptr;
    TY* y = static_cast<TY*>(p.y) + t * p.ldy;
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
            VB r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = *reinterpret_cast<const VB*>(base + col[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) Vec<TB, VB>::unpack(r[u], acc[u]);
        }
        int j = 0;
        for (; n - j >= J; j += J) add_rows<T, V, J, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc);
        if (J > 4 && n - j >= 4) add_rows<T, V, 4, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc), j += 4;
        if (J > 2 && n - j >= 2) add_rows<T, V, 2, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc), j += 2;
        if (n - j >= 1) add_rows<T, V, 1, U>(ys, p.ldys, s_row[warp], s_gate[warp], j, col, acc);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * N * u + lane * N < p.N) *reinterpret_cast<VY*>(y + col[u]) = Vec<TY, VY>::pack(acc[u]);
    }
}

// dys[row] = gate dy[t] and dgates[t, j] = dy[t] . ys[row], one assignment (t, j) per TEAM lanes.  Those of a token
// sit in one block, so that dy's row comes from memory once and from the first-level cache after that.
template <typename T, typename G, typename V, int U, int TEAM, bool DYS, bool DGATES>
__global__ void __launch_bounds__(kThreads) unsort_backward_kernel(const UnsortParams p) {
    constexpr int N = Vec<T, V>::kN;
    const int at = threadIdx.x % TEAM;
    const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / TEAM;
    pdl_wait();
    pdl_next();
    const bool mine = unit < p.T * p.k;
    const int64_t r = mine ? p.row[unit] : -1;
    float dot = 0.f;
    if (r >= 0 && r < p.rows) {
        const float g = p.gates ? to_f32(static_cast<const G*>(p.gates)[unit]) : 1.f;
        const T* dy = static_cast<const T*>(p.dy) + unit / p.k * p.lddy;
        const T* ys = static_cast<const T*>(p.ys) + r * p.ldys;
        T* dys = static_cast<T*>(p.y) + r * p.ldy;
        for (int64_t c0 = 0; c0 < p.N; c0 += TEAM * N * U) {
            V a[U], b[U];
            int64_t col[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + (TEAM * u + at) * N;
                col[u] = c < p.N ? c : p.N - N;  // past the end: the last vector again, not used
                a[u] = *reinterpret_cast<const V*>(dy + col[u]);
                if (DGATES) b[u] = *reinterpret_cast<const V*>(ys + col[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float d[N];
                Vec<T, V>::unpack(a[u], d);
                const bool in = c0 + (TEAM * u + at) * N < p.N;
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
    } else if (mine && r != -1 && at == 0) {
        set_status(p.status, MOE_ERR_BAD_INDEX);
    }
    if (DGATES) {
#pragma unroll
        for (int o = TEAM / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (mine && at == 0) p.dgates[unit] = dot;
    }
}

constexpr int kFill = 16;  // warps per SM that a short batch is spread over

template <typename T, typename G, typename V, int J, int U, typename TB, typename TY>
int launch_unsort(UnsortParams p, cudaStream_t stream) {
    const int64_t groups = (p.N + 32 * Vec<T, V>::kN * U - 1) / (32 * Vec<T, V>::kN * U);
    // two warps per token at least, of wide rows: T = 16384, k = 8, D = 2048 bf16 118 us with one, 115 with two, 120 with
    // four; D = 2047 296, 254 and 250
    const int64_t least = groups >= 4 ? 2 : 1, fill = (int64_t)device_sm_count() * kFill / p.T;
    const int64_t want = fill < least ? least : fill;
    p.split = (int)(want < groups ? want : groups);
    const int64_t grid = (p.T * p.split + kWarps - 1) / kWarps;
    return launch_pdl(unsort_kernel<T, G, V, J, U, TB, TY>, grid, kThreads, 0, stream, p);
}

template <typename T, typename G, typename V, int U, int TEAM>
int launch_backward(const UnsortParams& p, cudaStream_t stream) {
    const int64_t grid = (p.T * p.k * TEAM + kThreads - 1) / kThreads;
    const auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kThreads, 0, stream, p); };
    if (p.y && p.dgates) return go(unsort_backward_kernel<T, G, V, U, TEAM, true, true>);
    return p.y ? go(unsort_backward_kernel<T, G, V, U, TEAM, true, false>)
               : go(unsort_backward_kernel<T, G, V, U, TEAM, false, true>);
}

// V: the widest of 16 bytes, 4 and one value that the rows' starts and length allow.  T = 16384, k = 8 bf16: the way back
// and its gradient take 118 and 179 us at D = 2048, 146 and 228 at 2046, 296 and 297 at 2047.  (Whole 16-byte loads shifted
// to an odd row's start took 228 and 449.)  Loads at a time: 8 vectors, for narrower ones 16 on the way back; the gradient
// 4 of each operand, for fp32 values 8 (D = 1001: 221 us, 263 with 4; bf16 D = 2046: 284 us with 8).
// The gradient of rows of up to eight vectors: eight lanes each (D = 64: 9 us, 44 with a warp each).
template <typename T, typename G, typename V, int X, typename TB, typename TY>
int launch_back(const UnsortParams& p, bool backward, cudaStream_t stream) {
    if constexpr (std::is_same_v<T, TB> && std::is_same_v<T, TY>)  // the gradient's tensors have one type
        if (backward)
            return p.N <= 8 * Vec<T, V>::kN ? launch_backward<T, G, V, 1, 8>(p, stream)
                                            : launch_backward<T, G, V, sizeof(T) == 2 ? 4 : 4 * X, 32>(p, stream);
    if (p.k >= 6) return launch_unsort<T, G, V, 8, X, TB, TY>(p, stream);
    if (p.k >= 3) return launch_unsort<T, G, V, 4, 2 * X, TB, TY>(p, stream);
    return launch_unsort<T, G, V, 2, 4 * X, TB, TY>(p, stream);
}

template <typename T, typename G, typename TB = T, typename TY = T>
int launch_back(const UnsortParams& p, bool backward, int bytes, cudaStream_t stream) {
    if (bytes == 16) return launch_back<T, G, uint4, 1, TB, TY>(p, backward, stream);
    if constexpr (sizeof(T) == 2)
        if (bytes < 4) return launch_back<T, G, uint16_t, 2, TB, TY>(p, backward, stream);
    return launch_back<T, G, uint32_t, 2, TB, TY>(p, backward, stream);
}

// dtype: of ys and the gradient's tensors
int unsort_run(const UnsortParams& p, bool backward, moe_dtype dtype, moe_dtype gate_dtype, moe_dtype base_dtype,
               moe_dtype y_dtype, cudaStream_t stream) {
    const size_t es = dtype_size(dtype);
    // a vector of ys is as many values of the others: their addresses and strides in bytes of ys' type
    const auto at = [&](const void* a, int64_t ld, moe_dtype t) {
        return (uintptr_t)(reinterpret_cast<uintptr_t>(a) * (es / dtype_size(t))) | (uintptr_t)(ld * es);
    };
    const uintptr_t all = at(p.ys, p.ldys, dtype) | at(p.base, p.ldbase, base_dtype) | at(p.y, p.ldy, y_dtype) |
                          at(p.dy, p.lddy, dtype) | (uintptr_t)(p.N * es);
    const int bytes = (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 2;
    const bool gb = gate_dtype == MOE_BF16;
    using bf16 = __nv_bfloat16;
    if (dtype == MOE_BF16)
        return gb ? launch_back<bf16, bf16>(p, backward, bytes, stream) : launch_back<bf16, float>(p, backward, bytes, stream);
    if (y_dtype == MOE_F32)
        return gb ? launch_back<float, bf16>(p, backward, bytes, stream) : launch_back<float, float>(p, backward, bytes, stream);
    if (base_dtype == MOE_F32)
        return gb ? launch_back<float, bf16, float, bf16>(p, false, bytes, stream)
                  : launch_back<float, float, float, bf16>(p, false, bytes, stream);
    return gb ? launch_back<float, bf16, bf16, bf16>(p, false, bytes, stream)
              : launch_back<float, float, bf16, bf16>(p, false, bytes, stream);
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

extern "C" int moe_unsort_ex(const void* ys, int64_t ldys, int64_t rows, moe_dtype dtype, const int32_t* row,
                             const void* gates, moe_dtype gate_dtype, int64_t T, int32_t k, int64_t N, const void* base,
                             int64_t ldbase, moe_dtype base_dtype, void* y, int64_t ldy, moe_dtype y_dtype,
                             int32_t* dev_status, moe_stream_t stream) {
    MOE_REQUIRE(valid_dtype(dtype) && valid_dtype(gate_dtype) && valid_dtype(base_dtype) && valid_dtype(y_dtype),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T >= 0 && k >= 1 && N >= 1 && rows >= 0 && ldys >= N && ldy >= N, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(T == 0 || (row && y), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE((rows == 0 || ys) && (!base || ldbase >= N), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(k <= kMaxK && T < (int64_t(1) << 30) && T * k < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(y_dtype == dtype || dtype == MOE_F32, MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(!base || base_dtype == dtype || base_dtype == y_dtype, MOE_ERR_UNSUPPORTED);
    if (T == 0) return MOE_OK;
    UnsortParams p{};
    p.ys = ys, p.ldys = ldys, p.rows = rows, p.row = row, p.gates = gates, p.T = T, p.k = k, p.N = N;
    p.base = base, p.ldbase = base ? ldbase : 0, p.y = y, p.ldy = ldy, p.status = dev_status;
    return unsort_run(p, false, dtype, gate_dtype, base ? base_dtype : dtype, y_dtype,
                      reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_unsort(const void* ys, int64_t ldys, int64_t rows, const int32_t* row, const void* gates,
                          moe_dtype gate_dtype, int64_t T, int32_t k, int64_t N, const void* base, int64_t ldbase,
                          void* y, int64_t ldy, moe_dtype dtype, int32_t* dev_status, moe_stream_t stream) {
    return moe_unsort_ex(ys, ldys, rows, dtype, row, gates, gate_dtype, T, k, N, base, ldbase, dtype, y, ldy, dtype,
                         dev_status, stream);
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
    return unsort_run(p, true, dtype, gate_dtype, dtype, dtype, reinterpret_cast<cudaStream_t>(stream));
}
