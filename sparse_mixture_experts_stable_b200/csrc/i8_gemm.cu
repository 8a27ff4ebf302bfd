// Grouped product of 8-bit integers with one scale per token and one per output
// channel, on the tensor cores (tcgen05 kind::i8, exact int32 sums in tensor memory):
//
//   out[m, n] = epilogue( (sum_k X[m, k] W[g, n, k]) * xscale[m] * wscale[g, n] ),   offsets[g] <= m < offsets[g + 1]
//
// The weights are on the MMA's M side, so that a group's row count sets the MMA's N and
// a ragged expert wastes at most 31 token rows.  Two CTAs on two SMs share each MMA of
// 256 weight rows x up to 256 tokens, and a tile has two accumulators on the same
// tokens: 512 output features of one weight, or 256 features of gate and up (SwiGLU).
// Per 128-deep K block that is 48 KB of shared memory per SM (two weight tiles of
// 16 KB, half of the tokens) for 2 x 128 x 256 x 128 products, and four stages fit.
// The accumulators fill all 512 TMEM columns.
//
// Warp roles (576 threads per CTA, one persistent CTA per SM):
//   warp 0      TMA producer; the even CTA's draws tiles from a global counter and hands
//               each index to both CTAs through a small queue
//   warp 1      TMEM owner and MMA issuer (one lane of the even CTA)
//   warps 2-17  epilogue: warp w drains TMEM lanes 32 (w % 4).. (32 features of each
//               accumulator) for the 64 tokens [64 r, 64 r + 64), r = (w - 2) / 4
// Every wait is bounded (kWaitLimitNs); after a timeout nothing more is written.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "i8_gemm.cuh"
#include "tc_gemm.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kM = 128;        // features per CTA and accumulator (half of the pair's M = 256)
constexpr int kBK = 128;       // K per stage: one 128-byte swizzle row
constexpr int kNT = 256;       // most tokens per tile (MMA N)
constexpr int kBox = 32;       // token rows per TMA box
constexpr int kStages = 4;
constexpr int kEpiWarps = 16;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kMaxGroups = 2048;
constexpr int kQueue = 4;      // tile indices in flight between the producer and the consumers
constexpr int kWBytes = kM * kBK;
constexpr int kXBytes = (kNT / 2) * kBK;
constexpr int kStageBytes = 2 * kWBytes + kXBytes;
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + 256;
// consumers of a queue slot, all counted on the even CTA: its MMA issuer and
// epilogue warps, the odd CTA's producer and epilogue warps
constexpr int kQueueConsumers = 1 + kEpiWarps + 1 + kEpiWarps;

struct Params {
    int G;
    int64_t M, N;
    const int32_t* offsets;
    const float* xscale;
    const float* wscale;
    const float* wscale2;
    const float* bias;
    int tile_f;   // output features per tile: 512, or 256 for SwiGLU
    int f_tiles;
    int k_blocks;
    void* out;
    int64_t ldo;
    uint32_t* tile_counter;  // zero at launch: the next tile to hand out
    int32_t* status;
};

__device__ __forceinline__ int row_offset(const Params& p, int g) {
    if (!p.offsets) return g == 0 ? 0 : (int)p.M;
    const int o = p.offsets[g];
    return o < 0 ? 0 : (o > p.M ? (int)p.M : o);
}

// A group's rows split into ceil(rows / 256) tiles of equal size (a multiple of the TMA box).
__device__ __forceinline__ int token_span(int rows) {
    const int n_tt = (rows + kNT - 1) / kNT;
    if (n_tt <= 0) return kNT;
    const int span = (rows + n_tt - 1) / n_tt;
    return (span + kBox - 1) / kBox * kBox;
}

// the tokens of one CTA: a tile's n tokens in two halves of a multiple of 16
__device__ __forceinline__ int token_half(int n) { return ((n + 1) / 2 + 15) / 16 * 16; }

struct Tile {
    int g, ft, row0, n;  // group, feature tile, first row of X, rows
};

// Feature tiles fastest, so that tiles which run together share the group's tokens.
__device__ __forceinline__ Tile decode(int tile, const int* prefix, const int* off, const Params& p) {
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    Tile t;
    t.g = lo;
    const int local = tile - prefix[lo];
    const int tt = local / p.f_tiles;
    t.ft = local - tt * p.f_tiles;
    const int rows = off[lo + 1] - off[lo];
    const int span = token_span(rows);
    t.row0 = off[lo] + tt * span;
    t.n = rows - tt * span < span ? rows - tt * span : span;
    return t;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int EPI, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    i8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
              const __grid_constant__ CUtensorMap tmX, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_prefix[kMaxGroups + 1];
    __shared__ int s_off[kMaxGroups + 1];
    __shared__ int s_tile[kQueue];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
    uint64_t* full = bars;                // even CTA: a stage's loads of both CTAs have landed
    uint64_t* empty = bars + kStages;     // both CTAs: the stage's MMAs are done
    uint64_t* tfull = bars + 2 * kStages; // both CTAs: the accumulators hold a finished tile
    uint64_t* tempty = tfull + 1;         // even CTA: both epilogues drained the accumulators
    uint64_t* qfull = tempty + 1;         // both CTAs: s_tile[q] holds the next tile
    uint64_t* qempty = qfull + kQueue;    // even CTA: every consumer has read s_tile[q]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * kEpiWarps);
        for (int q = 0; q < kQueue; ++q) {
            mbar_init(&qfull[q], 1);
            mbar_init(&qempty[q], kQueueConsumers);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW2)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // tiles before each group; offsets that run backwards leave the group empty
    for (int g = threadIdx.x; g <= p.G; g += kThreads) s_off[g] = row_offset(p, g);
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
        const int r = s_off[g + 1] - s_off[g];
        if (r < 0) set_status(p.status, MOE_ERR_BAD_INDEX);
        s_prefix[g] = r > 0 ? (r + token_span(r) - 1) / token_span(r) * p.f_tiles : 0;
    }
    __syncthreads();
    block_scan<kThreads>(s_prefix, p.G);
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    const int total = s_prefix[p.G];
    const uint32_t tmem_base = s_tmem;
    // the even CTA's barriers as shared::cluster addresses
    const uint32_t full_l = mapa_shared(smem_u32(full), 0);
    const uint32_t tempty_l = mapa_shared(smem_u32(tempty), 0);
    const uint32_t qempty_l = mapa_shared(smem_u32(qempty), 0);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int i = 0;; ++i) {
                const int q = i % kQueue;
                const uint32_t qph = (uint32_t)(i / kQueue) & 1u;
                int tile;
                if (leader) {
                    if (!mbar_wait_cluster(&qempty[q], qph ^ 1u, p.status)) {
                        s_abort = 1;
                        tile = -1;
                    } else {
                        tile = s_abort ? -1 : (int)atomicAdd(p.tile_counter, 1u);
                        if (tile >= total) tile = -1;
                    }
                    s_tile[q] = tile;
                    st_cluster_u32(mapa_shared(smem_u32(&s_tile[q]), 1), tile);
                    mbar_arrive(&qfull[q]);
                    mbar_arrive_cluster(mapa_shared(smem_u32(&qfull[q]), 1));  // release: orders the store
                } else {
                    tile = -1;
                    if (mbar_wait_cluster(&qfull[q], qph, p.status)) tile = s_tile[q];
                    else s_abort = 1;
                    mbar_arrive_cluster(qempty_l + 8u * (uint32_t)q);
                }
                if (tile < 0) break;
                const Tile t = decode(tile, s_prefix, s_off, p);
                const int half = token_half(t.n);
                const int nbox = (half + kBox - 1) / kBox;
                const int64_t f0 = (int64_t)t.ft * p.tile_f + (int64_t)rank * kM;
                const int32_t w_y = (int32_t)(t.g * p.N + f0);
                const bool two = EPI == I8_SWIGLU || (int64_t)t.ft * p.tile_f + 2 * kM < p.N;
                const int32_t w_y2 = EPI == I8_SWIGLU ? w_y : w_y + 2 * kM;
                const int32_t x_y = t.row0 + (int32_t)rank * half;
                const uint32_t tx_pair = 2u * (uint32_t)((two ? 2 : 1) * kWBytes + nbox * kBox * kBK);
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.status)) {
                        s_abort = 1;
                        break;
                    }
                    if (leader) mbar_expect_tx(&full[stage], tx_pair);
                    const uint32_t fb = full_l + 8u * (uint32_t)stage;
                    uint8_t* st = smem + stage * kStageBytes;
                    tma_load_2d_pair(st, &tmW, kb * kBK, w_y, fb);
                    if (two) tma_load_2d_pair(st + kWBytes, &tmW2, kb * kBK, w_y2, fb);
                    for (int b = 0; b < nbox; ++b)
                        tma_load_2d_pair(st + 2 * kWBytes + b * (kBox * kBK), &tmX, kb * kBK, x_y + b * kBox, fb);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------
        if (lane == 0 && leader) {
            int stage = 0;
            uint32_t phase = 0;
            bool ready = false;  // full[stage] was seen complete by an early test
            for (uint32_t it = 0;; ++it) {
                const int q = (int)(it % kQueue);
                if (!mbar_wait(&qfull[q], (it / kQueue) & 1u, p.status)) {
                    s_abort = 1;
                    break;
                }
                const int tile = s_tile[q];
                mbar_arrive(&qempty[q]);
                if (tile < 0) break;
                const Tile t = decode(tile, s_prefix, s_off, p);
                const uint32_t idesc = make_idesc_i8(2 * kM, 2 * token_half(t.n));
                const bool two = EPI == I8_SWIGLU || (int64_t)t.ft * p.tile_f + 2 * kM < p.N;
                if (!mbar_wait_cluster(tempty, (it & 1u) ^ 1u, p.status)) {
                    s_abort = 1;
                    break;
                }
                tc_fence_after();
                bool ok = true;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!ready && !mbar_wait(&full[stage], phase, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + stage * kStageBytes);
                    const uint64_t wd = sw128_desc(st), wd2 = sw128_desc(st + kWBytes);
                    const uint64_t xd = sw128_desc(st + 2 * kWBytes);
                    const int ns = stage + 1 == kStages ? 0 : stage + 1;
                    const uint32_t np = stage + 1 == kStages ? phase ^ 1u : phase;
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk) {
                        const uint32_t accum = (kb > 0 || kk > 0) ? 1u : 0u;
                        tc_mma_i8_pair(tmem_base, wd + 2 * kk, xd + 2 * kk, idesc, accum);
                        if (two) tc_mma_i8_pair(tmem_base + 256, wd2 + 2 * kk, xd + 2 * kk, idesc, accum);
                        // the tensor core takes new MMAs only as it finishes old ones: look at the
                        // next stage while this one's MMAs are being accepted
                        if (kk == 1) ready = mbar_test(smem_u32(&full[ns]), np);
                    }
                    tc_commit_pair(&empty[stage]);
                    stage = ns;
                    phase = np;
                }
                if (!ok) {
                    s_abort = 1;
                    break;
                }
                tc_commit_pair(tfull);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------- epilogue --------------------------------
        const int q = warp & 3;          // TMEM lane quarter: features 32q .. 32q+31 of this CTA's 128
        const int r = (warp - 2) >> 2;   // token quarter: tokens 64r .. 64r+63 of the tile
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        for (uint32_t it = 0;; ++it) {
            const int q_slot = (int)(it % kQueue);
            int tile = -1;
            if (lane == 0) {
                if (mbar_wait_cluster(&qfull[q_slot], (it / kQueue) & 1u, p.status)) tile = s_tile[q_slot];
                else s_abort = 1;
                mbar_arrive_cluster(qempty_l + 8u * (uint32_t)q_slot);
            }
            tile = __shfl_sync(0xffffffffu, tile, 0);
            if (tile < 0) break;
            const Tile t = decode(tile, s_prefix, s_off, p);
            // this thread's features, their scales, and the scales of this warp's tokens
            const int64_t f = (int64_t)t.ft * p.tile_f + (int64_t)rank * kM + q * 32 + lane;
            const int64_t f2 = EPI == I8_SWIGLU ? f : f + 2 * kM;
            float ws = 0.f, ws2 = 0.f, bs = 0.f, bs2 = 0.f;
            if (f < p.N) ws = p.wscale[t.g * p.N + f];
            if (f2 < p.N) ws2 = (EPI == I8_SWIGLU ? p.wscale2 : p.wscale)[t.g * p.N + f2];
            if (EPI != I8_SWIGLU && p.bias) {
                if (f < p.N) bs = p.bias[t.g * p.N + f];
                if (f2 < p.N) bs2 = p.bias[t.g * p.N + f2];
            }
            float xs[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = 64 * r + 32 * h + lane;
                xs[h] = tok < t.n ? p.xscale[t.row0 + tok] : 0.f;
            }
            int ok = 1;
            if (lane == 0) ok = mbar_wait(tfull, it & 1u, p.status) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) s_abort = 1;
            tc_fence_after();
            const bool live = !s_abort;
            TO* out = static_cast<TO*>(p.out) + (int64_t)(t.row0 + 64 * r) * p.ldo;
            constexpr bool kPacked = sizeof(TO) == 2;  // bf16 results wait in registers until TMEM is released
            uint32_t h1[4][8], h2[4][8];

#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                const int tok0 = 64 * r + 16 * ch;
                if (tok0 < t.n) {
                    uint32_t a[16], b[16];
                    tmem_ld16(tmem_base + lane_off + (uint32_t)tok0, a);
                    tmem_ld16(tmem_base + 256 + lane_off + (uint32_t)tok0, b);
                    tmem_ld_wait(a, b);
                    float u[16], v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = __shfl_sync(0xffffffffu, xs[ch >> 1], (16 * ch + i) & 31);
                        u[i] = (float)(int)a[i] * (ws * x);
                        v[i] = (float)(int)b[i] * (ws2 * x);
                        if (EPI == I8_SWIGLU) {
                            u[i] = swiglu_f(u[i], v[i]);
                        } else {
                            u[i] += bs;
                            v[i] += bs2;
                        }
                        if (EPI == I8_GELU) {
                            u[i] = gelu_f(u[i]);
                            v[i] = gelu_f(v[i]);
                        }
                    }
                    if (kPacked) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            h1[ch][i] = pack_bf16x2(u[2 * i], u[2 * i + 1]);
                            if (EPI != I8_SWIGLU) h2[ch][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                        }
                    } else if (live) {
                        TO* dst = out + (int64_t)16 * ch * p.ldo;
                        const int n = t.n - tok0 < 16 ? t.n - tok0 : 16;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < n) {
                                if (f < p.N) dst[i * p.ldo + f] = from_f32<TO>(u[i]);
                                if (EPI != I8_SWIGLU && f2 < p.N) dst[i * p.ldo + f2] = from_f32<TO>(v[i]);
                            }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_l);  // TMEM drained: the next tile's MMAs may start
            if (kPacked && live) {
                // for each token the warp writes 32 consecutive features of each accumulator
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    const int n = t.n - 64 * r - 16 * ch;
                    TO* dst = out + (int64_t)16 * ch * p.ldo;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < n) {
                            const int sh = (i & 1) * 16;
                            if (f < p.N) reinterpret_cast<uint16_t*>(dst)[i * p.ldo + f] = (uint16_t)(h1[ch][i >> 1] >> sh);
                            if (EPI != I8_SWIGLU && f2 < p.N)
                                reinterpret_cast<uint16_t*>(dst)[i * p.ldo + f2] = (uint16_t)(h2[ch][i >> 1] >> sh);
                        }
                }
            }
        }
    }

    tc_fence_before();
    cluster_sync();  // neither CTA leaves while the other may still signal its barriers or read its stages
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
    }
}

template <int EPI, typename TO>
int launch(const CUtensorMap& mw, const CUtensorMap& mw2, const CUtensorMap& mx, const Params& kp, int grid,
           cudaStream_t stream) {
    static bool attr_set[64] = {false};
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !attr_set[dev]) {
        MOE_CUDA_TRY(cudaFuncSetAttribute(i8_kernel<EPI, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)kSmemBytes));
        if (dev < 64) attr_set[dev] = true;
    }
    i8_kernel<EPI, TO><<<grid, kThreads, kSmemBytes, stream>>>(mw, mw2, mx, kp);
    return launch_status();
}

}  // namespace

int i8_gemm_run(const I8Problem& p, cudaStream_t stream) {
    const bool dual = p.epilogue == I8_SWIGLU;
    MOE_REQUIRE(p.G >= 1 && p.N >= 1 && p.K >= 1 && p.M >= 0 && (p.offsets || p.G == 1), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(p.ldx >= p.K && p.ldw >= p.K && p.ldo >= p.N && valid_dtype(p.out_dtype), MOE_ERR_INVALID_ARG);
    if (p.M == 0) return MOE_OK;
    MOE_REQUIRE(p.x && p.xscale && p.w && p.wscale && p.out && (!dual || (p.w2 && p.wscale2 && !p.bias)),
                MOE_ERR_INVALID_ARG);
    // K: the int32 sums of 128 x 128 products; the rest: 32-bit tile and row indices, tensor-map limits
    MOE_REQUIRE(p.G <= kMaxGroups && p.K <= 131071, MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(p.M < (int64_t(1) << 30) && p.N < (int64_t(1) << 30) && p.G * p.N < (int64_t(1) << 30),
                MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(aligned16(p.x) && aligned16(p.w) && p.ldx % 16 == 0 && p.ldw % 16 == 0 && p.ldx < (int64_t(1) << 38) &&
                    p.ldw < (int64_t(1) << 38),
                MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(!dual || aligned16(p.w2), MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE((reinterpret_cast<uintptr_t>(p.out) % dtype_size(p.out_dtype)) == 0, MOE_ERR_INVALID_ARG);
    if (i8_skinny_fits(p.M, p.G, p.N, p.K)) return i8_skinny_run(p, false, stream);
    MOE_REQUIRE(p.tile_counter, MOE_ERR_WORKSPACE);

    Params kp{};
    kp.G = p.G, kp.M = p.M, kp.N = p.N, kp.offsets = p.offsets;
    kp.xscale = p.xscale, kp.wscale = p.wscale, kp.wscale2 = p.wscale2, kp.bias = p.bias;
    kp.tile_f = dual ? 2 * kM : 4 * kM;
    kp.f_tiles = (int)((p.N + kp.tile_f - 1) / kp.tile_f);
    kp.k_blocks = (int)((p.K + kBK - 1) / kBK);
    kp.out = p.out, kp.ldo = p.ldo, kp.tile_counter = p.tile_counter, kp.status = p.status;
    const int64_t max_tiles = kp.f_tiles * ((p.M + kNT - 1) / kNT + p.G - 1);  // every group may end a tile early
    MOE_REQUIRE(max_tiles < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);

    CUtensorMap mw, mw2, mx;
    MOE_REQUIRE(make_map_i8(&mw, p.w, p.K, p.G * p.N, p.ldw, kM), MOE_ERR_CUDA);
    MOE_REQUIRE(make_map_i8(&mw2, dual ? p.w2 : p.w, p.K, p.G * p.N, p.ldw, kM), MOE_ERR_CUDA);
    MOE_REQUIRE(make_map_i8(&mx, p.x, p.K, p.M, p.ldx, kBox), MOE_ERR_CUDA);
    MOE_CUDA_TRY(cudaMemsetAsync(p.tile_counter, 0, sizeof(uint32_t), stream));
    int64_t pairs = device_sm_count() / 2;
    if (max_tiles < pairs) pairs = max_tiles;
    if (pairs < 1) pairs = 1;
    const int grid = (int)(2 * pairs);
    const bool bf = p.out_dtype == MOE_BF16;
    switch (p.epilogue) {
        case I8_OUT: return bf ? launch<I8_OUT, __nv_bfloat16>(mw, mw2, mx, kp, grid, stream)
                               : launch<I8_OUT, float>(mw, mw2, mx, kp, grid, stream);
        case I8_GELU: return bf ? MOE_ERR_UNSUPPORTED : launch<I8_GELU, float>(mw, mw2, mx, kp, grid, stream);
        case I8_SWIGLU: return bf ? MOE_ERR_UNSUPPORTED : launch<I8_SWIGLU, float>(mw, mw2, mx, kp, grid, stream);
        default: return MOE_ERR_INVALID_ARG;
    }
}

}  // namespace moe

using namespace moe;

namespace {

constexpr size_t kCounterBytes = 256;

bool ffn_sizes_ok(moe_ffn_kind kind, int32_t G, int64_t M, int64_t D, int64_t F, int64_t Dout) {
    return G >= 1 && M >= 0 && D >= 1 && Dout >= 1 && (kind == MOE_FFN_LINEAR || F >= 1) &&
           M < (int64_t(1) << 30) && F < (int64_t(1) << 30);
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

extern "C" size_t moe_matmul_i8_workspace_size(int64_t M, int32_t G, int64_t N, int64_t K) {
    return M < 1 || G < 1 || N < 1 || K < 1 || i8_skinny_fits(M, G, N, K) ? 0 : kCounterBytes;
}

extern "C" int moe_matmul_i8(const int8_t* xq, const float* xscale, int64_t M, int64_t ldx, const int32_t* offsets,
                             const int8_t* wq, const float* wscale, int64_t ldw, const float* bias, int32_t G,
                             int64_t N, int64_t K, void* out, int64_t ldo, moe_dtype out_dtype, int32_t* dev_status,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    const size_t need = moe_matmul_i8_workspace_size(M, G, N, K);
    MOE_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), MOE_ERR_WORKSPACE);
    I8Problem p{};
    p.x = xq, p.xscale = xscale, p.M = M, p.ldx = ldx, p.offsets = offsets, p.w = wq, p.wscale = wscale;
    p.ldw = ldw, p.bias = bias, p.G = G, p.N = N, p.K = K, p.out = out, p.ldo = ldo, p.out_dtype = out_dtype;
    p.epilogue = I8_OUT, p.tile_counter = static_cast<uint32_t*>(workspace), p.status = dev_status;
    return i8_gemm_run(p, reinterpret_cast<cudaStream_t>(stream));
}

// workspace: [counters | hscale (M) | hq (M, round16(F)) | h (M, F) fp32]
extern "C" size_t moe_expert_ffn_i8_workspace_size(moe_ffn_kind kind, int32_t G, int64_t M, int64_t D, int64_t F,
                                                   int64_t Dout) {
    if (!ffn_sizes_ok(kind, G, M, D, F, Dout) || M == 0) return 0;
    if (kind == MOE_FFN_LINEAR) return kCounterBytes;
    return kCounterBytes + align_up((size_t)M * sizeof(float), 256) + align_up((size_t)M * round16(F), 256) +
           (size_t)M * F * sizeof(float);
}

extern "C" int moe_expert_ffn_i8(moe_ffn_kind kind, const int8_t* xq, const float* xscale, int64_t M, int64_t ldx,
                                 const int32_t* offsets, int32_t G, int64_t D, int64_t F, int64_t Dout,
                                 const int8_t* w1, const float* s1, int64_t ldw1, const float* b1, const int8_t* w2,
                                 const float* s2, int64_t ldw2, const float* b2, const int8_t* w3, const float* s3,
                                 void* ys, int64_t ldys, moe_dtype out_dtype, int32_t* dev_status, void* workspace,
                                 size_t workspace_bytes, moe_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    MOE_REQUIRE(kind == MOE_FFN_LINEAR || kind == MOE_FFN_GELU_MLP || kind == MOE_FFN_SWIGLU, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(ffn_sizes_ok(kind, G, M, D, F, Dout), MOE_ERR_INVALID_ARG);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(workspace && workspace_bytes >= moe_expert_ffn_i8_workspace_size(kind, G, M, D, F, Dout),
                MOE_ERR_WORKSPACE);
    I8Problem p{};
    p.x = xq, p.xscale = xscale, p.M = M, p.ldx = ldx, p.offsets = offsets, p.w = w1, p.wscale = s1, p.ldw = ldw1;
    p.G = G, p.K = D, p.tile_counter = static_cast<uint32_t*>(workspace), p.status = dev_status;
    if (kind == MOE_FFN_LINEAR) {
        p.bias = b1, p.N = Dout, p.out = ys, p.ldo = ldys, p.out_dtype = out_dtype, p.epilogue = I8_OUT;
        return i8_gemm_run(p, stream);
    }
    // the second product's arguments are checked before the first is enqueued
    MOE_REQUIRE(w2 && s2 && ys && ldw2 >= F && ldys >= Dout && valid_dtype(out_dtype), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(aligned16(w2) && ldw2 % 16 == 0 && F <= 131071 && G * Dout < (int64_t(1) << 30) &&
                    reinterpret_cast<uintptr_t>(ys) % dtype_size(out_dtype) == 0,
                MOE_ERR_UNSUPPORTED);
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kCounterBytes;
    float* hscale = reinterpret_cast<float*>(ws);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + align_up((size_t)M * sizeof(float), 256));
    float* h = reinterpret_cast<float*>(hq + align_up((size_t)M * round16(F), 256));
    MOE_REQUIRE(aligned16(ws), MOE_ERR_INVALID_ARG);
    p.N = F, p.out = h, p.ldo = F, p.out_dtype = MOE_F32;
    if (kind == MOE_FFN_SWIGLU) p.w2 = w3, p.wscale2 = s3, p.epilogue = I8_SWIGLU;
    else p.bias = b1, p.epilogue = I8_GELU;
    int rc = i8_gemm_run(p, stream);
    if (rc != MOE_OK) return rc;
    I8Problem d{};
    d.x = hq, d.xscale = hscale, d.M = M, d.ldx = round16(F), d.offsets = offsets, d.w = w2, d.wscale = s2;
    d.ldw = ldw2, d.bias = kind == MOE_FFN_GELU_MLP ? b2 : nullptr, d.G = G, d.N = Dout, d.K = F, d.out = ys;
    d.ldo = ldys, d.out_dtype = out_dtype, d.epilogue = I8_OUT;
    d.tile_counter = static_cast<uint32_t*>(workspace) + 16, d.status = dev_status;
    if (i8_skinny_fits(M, G, Dout, F)) {  // which quantises the hidden rows itself
        d.x = reinterpret_cast<const int8_t*>(h), d.ldx = F;
        return i8_skinny_run(d, true, stream);
    }
    rc = quantize_rows(h, MOE_F32, M, F, F, hq, round16(F), hscale, offsets, G, dev_status, stream);
    if (rc != MOE_OK) return rc;
    return i8_gemm_run(d, stream);
}
