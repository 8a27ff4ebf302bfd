// Grouped product of 8-bit integers with one scale per token and one per output
// channel, on the tensor cores (tcgen05 kind::i8, exact int32 sums in tensor memory):
//
//   out[m, n] = epilogue( (sum_k X[m, k] W[g, n, k]) * xscale[m] * wscale[g, n] ),   offsets[g] <= m < offsets[g + 1]
//
// The weights are on the MMA's M side, so that a group's row count sets the MMA's N and
// a ragged expert wastes at most 31 token rows.  Two CTAs on two SMs share each MMA of
// 256 weight rows x up to 256 tokens: 256 output features, or 128 of gate and up (SwiGLU;
// 64 rows of each per CTA, so that one warp has a feature's gate and another one its up, and
// they exchange them through shared memory.  16 rows of each in turn would put both into
// one warp's TMEM lanes, but the TMA copy of so many small boxes takes longer than the
// MMAs, at 70 cycles each).  Per 128-deep K block that is 32 KB of shared memory per SM,
// and five stages fit.  The two
// halves of TMEM hold two tiles' accumulators, so a tile's epilogue runs under the next
// one's MMAs.  (Two accumulators on the same tokens would need 24 KB a block and MMA, but
// the epilogue then stands alone: 2.2 us of MMAs and 8 us of epilogue per tile at K = 512.)
//
// Warp roles (576 threads per CTA, one persistent CTA per SM):
//   warp 0      TMA producer
//   warp 1      TMEM owner; in the even CTA one lane issues the MMAs, in the odd one it hands
//               out tiles to both CTAs through a small queue, in turn or, where groups make
//               them uneven, from a global counter (finding a tile's group takes as long as
//               one of its K blocks, so no other role does it)
//   warps 2-17  epilogue: warp w drains TMEM lanes 32 (w % 4).. for the 64 tokens
//               [64 r, 64 r + 64), r = (w - 2) / 4.  16-bit results are transposed through
//               shared memory (stmatrix) and written 64 bytes per token.  The next tile's
//               scales are on their way while one is worked on.
// What bounds it: an MMA of 32 in depth is accepted every 180 to 190 cycles whatever its N
// (K block 715 cycles at N = 128, 757 at 256), so a group's rows are cut into as few tiles
// as 256 tokens allow.  16384 x 2048 x 2048 bf16: 60 us, 2300 TOPS (torch._int_mm without
// scales 57); SwiGLU of 131072 rows in 256 groups, 2048 x 512: 300 us; the product back,
// 512 x 2048: 209 us, half of it the rows' bytes; 263 with fp32 rows.
// Every wait on an mbarrier is bounded (kWaitLimitNs); after a timeout nothing more is written, and the barriers that warps
// share are still met by all of them.
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
constexpr int kStages = 5;
constexpr int kEpiWarps = 16;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kMaxGroups = 2048;
constexpr int kQueue = 4;      // tile indices in flight between the producer and the consumers
constexpr int kWBytes = kM * kBK;
constexpr int kXBytes = (kNT / 2) * kBK;
constexpr int kStageBytes = kWBytes + kXBytes;
constexpr int kStoreBytes = 32 * 32 * 2;  // per epilogue warp: 32 tokens x 32 features of 16 bits, or 16 x 32 of 32
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kStoreBytes + 256;
// consumers of a queue slot, all counted on the odd CTA: both producers, the MMA issuer and both CTAs' epilogue warps
constexpr int kQueueConsumers = 2 + 1 + 2 * kEpiWarps;

struct Params {
    int G;
    int64_t M, N;
    const int32_t* offsets;
    const float* xscale;
    const float* wscale;
    const float* wscale2;
    const float* bias;
    int tile_f;   // output features per tile: 256, or 128 for SwiGLU
    int f_tiles;
    int k_blocks;
    int max_span; // most tokens per tile
    bool vec_out; // rows of out start on 16 bytes
    void* out;
    int64_t ldo;
    uint32_t* tile_counter;  // zero at launch: the next tile to hand out; NULL: every pair's in turn
    int32_t* status;
};

__device__ __forceinline__ int row_offset(const Params& p, int g) {
    if (!p.offsets) return g == 0 ? 0 : (int)p.M;
    const int o = p.offsets[g];
    return o < 0 ? 0 : (o > p.M ? (int)p.M : o);
}

// A group's rows split into ceil(rows / max_span) tiles of equal size (a multiple of the TMA box).
__device__ __forceinline__ int token_span(int rows, int max_span) {
    const int n_tt = (rows + max_span - 1) / max_span;
    if (n_tt <= 0) return max_span;
    const int span = (rows + n_tt - 1) / n_tt;
    return (span + kBox - 1) / kBox * kBox;
}

// the tokens of one CTA: a tile's n tokens in two halves of a multiple of 16
__device__ __forceinline__ int token_half(int n) { return ((n + 1) / 2 + 15) / 16 * 16; }

struct __align__(16) Tile {
    int g, ft, row0, n;  // group (-1: no more tiles), feature tile, first row of X, rows
};

// The tile's place, found by the 32 lanes of a warp together.  Feature tiles fastest, so that tiles which run together
// share the group's tokens.
__device__ __forceinline__ Tile decode(int tile, const int* prefix, const int* off, const Params& p, int lane) {
    // the last group whose first tile is not behind this one: a 32nd of the groups, then the group
    const int stride = (p.G + 31) / 32;
    const int probe = lane * stride;
    const int part = __popc(__ballot_sync(0xffffffffu, probe < p.G && prefix[probe] <= tile)) - 1;
    int g = part * stride - 1;
    for (int i = 0; i < stride; i += 32) {
        const int at = part * stride + i + lane;
        g += __popc(__ballot_sync(0xffffffffu, i + lane < stride && at < p.G && prefix[at] <= tile));
    }
    Tile t;
    t.g = g;
    const int local = tile - prefix[g];
    const int tt = local / p.f_tiles;
    t.ft = local - tt * p.f_tiles;
    const int rows = off[g + 1] - off[g];
    const int span = token_span(rows, p.max_span);
    t.row0 = off[g] + tt * span;
    t.n = rows - tt * span < span ? rows - tt * span : span;
    return t;
}

__device__ __forceinline__ void st_cluster_tile(uint32_t addr, const Tile& t) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(t.g), "r"(t.ft), "r"(t.row0), "r"(t.n)
                 : "memory");
}

// Takes a tile from this CTA's copy of a queue slot; one thread per consumer.  It arrives without release, but not before the
// slot has been read (each of a tile's four words is below 2^30 or -1, so bits 30 and 31 of their xor are equal: it is never
// 0x7fffffff).  A release in the producers and the issuer alone, which have no global stores in flight, costs 16384 x 2048 x
// 2048 62.4 us instead of 59.7.
__device__ __forceinline__ Tile take_tile(uint64_t* qfull, const Tile* slots, uint32_t qempty_l, uint32_t it, int32_t* status,
                                          volatile int* abort) {
    const uint32_t slot = it % kQueue;
    Tile t;
    t.g = t.ft = t.row0 = t.n = -1;
    if (mbar_wait_cluster(&qfull[slot], (it / kQueue) & 1u, status)) t = slots[slot];
    else *abort = 1;
    mbar_arrive_cluster_relaxed(qempty_l + 8u * slot, (uint32_t)(t.g ^ t.ft ^ t.row0 ^ t.n));
    return t;
}

template <int EPI, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    i8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
              const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmX128, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_prefix[kMaxGroups + 1];
    __shared__ int s_off[kMaxGroups + 1];
    __shared__ Tile s_tile[kQueue];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* store = smem + kStages * kStageBytes;  // the epilogue warps' transposed chunks
    uint64_t* bars = reinterpret_cast<uint64_t*>(store + kEpiWarps * kStoreBytes);
    uint64_t* full = bars;                // even CTA: a stage's loads of both CTAs have landed
    uint64_t* empty = bars + kStages;     // both CTAs: the stage's MMAs are done
    uint64_t* tfull = bars + 2 * kStages; // both CTAs: an accumulator holds a finished tile
    uint64_t* tempty = tfull + 2;         // even CTA: both epilogues drained the accumulator
    uint64_t* qfull = tempty + 2;         // both CTAs: s_tile[q] holds the next tile
    uint64_t* qempty = qfull + kQueue;    // odd CTA: every consumer has read s_tile[q]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kEpiWarps);
        }
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
    pdl_wait();
    pdl_next();
    for (int g = threadIdx.x; g <= p.G; g += kThreads) s_off[g] = row_offset(p, g);
    __syncthreads();
    // Offsets that run backwards become their running maximum: no row has two groups, and the tiles fit in an int.
    bool back = false;
    for (int g = threadIdx.x; g < p.G; g += kThreads) back |= s_off[g + 1] < s_off[g];
    if (__syncthreads_or(back)) {
        if (threadIdx.x == 0) {
            set_status(p.status, MOE_ERR_BAD_INDEX);
            for (int g = 0; g < p.G; ++g) s_off[g + 1] = max(s_off[g + 1], s_off[g]);
        }
        __syncthreads();
    }
    // tiles before each group
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
        const int r = s_off[g + 1] - s_off[g];
        const int span = token_span(r, p.max_span);
        s_prefix[g] = r > 0 ? (r + span - 1) / span * p.f_tiles : 0;
    }
    __syncthreads();
    block_scan<kThreads>(s_prefix, p.G);
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    const int total = s_prefix[p.G];
    const uint32_t tmem_base = s_tmem;
    // barriers of the even, and the odd CTA as shared::cluster addresses
    const uint32_t full_l = mapa_shared(smem_u32(full), 0);
    const uint32_t tempty_l = mapa_shared(smem_u32(tempty), 0);
    const uint32_t qempty_l = mapa_shared(smem_u32(qempty), 1);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                const Tile t = take_tile(qfull, s_tile, qempty_l, it, p.status, &s_abort);
                if (t.g < 0) break;
                const int half = token_half(t.n);
                const int nbox = (half + kBox - 1) / kBox;
                const int32_t w_y = (int32_t)(t.g * p.N + (int64_t)t.ft * p.tile_f + (int64_t)rank * (p.tile_f / 2));
                const int32_t x_y = t.row0 + (int32_t)rank * half;
                const uint32_t tx_pair = 2u * (uint32_t)(kWBytes + nbox * kBox * kBK);
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.status)) {
                        s_abort = 1;
                        ok = false;
                        break;
                    }
                    if (leader) mbar_expect_tx(&full[stage], tx_pair);
                    const uint32_t fb = full_l + 8u * (uint32_t)stage;
                    uint8_t* st = smem + stage * kStageBytes;
                    tma_load_2d_pair(st, &tmW, kb * kBK, w_y, fb);
                    if (EPI == I8_SWIGLU) tma_load_2d_pair(st + kWBytes / 2, &tmW2, kb * kBK, w_y, fb);
                    if (nbox == 4)  // most often, and only if max_span is kNT: one copy is issued faster than four
                        tma_load_2d_pair(st + kWBytes, &tmX128, kb * kBK, x_y, fb);
                    else
                        for (int b = 0; b < nbox; ++b)
                            tma_load_2d_pair(st + kWBytes + b * (kBox * kBK), &tmX, kb * kBK, x_y + b * kBox, fb);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The CTA does not end before its copies have landed and the MMAs that read them are done; after a timeout not
            // before one more wait, much longer than either takes.
            for (int s = 0; s < kStages && mbar_wait(&empty[stage], phase ^ 1u, p.status); ++s) {
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
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
                const Tile t = take_tile(qfull, s_tile, qempty_l, it, p.status, &s_abort);
                if (t.g < 0) break;
                const uint32_t idesc = make_idesc_i8(2 * kM, 2 * token_half(t.n));
                const uint32_t acc = it & 1u, aph = (it >> 1) & 1u;
                if (!mbar_wait_cluster(&tempty[acc], aph ^ 1u, p.status)) {
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
                    const uint64_t wd = sw128_desc(st), xd = sw128_desc(st + kWBytes);
                    const int ns = stage + 1 == kStages ? 0 : stage + 1;
                    const uint32_t np = stage + 1 == kStages ? phase ^ 1u : phase;
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk) {
                        const uint32_t accum = (kb > 0 || kk > 0) ? 1u : 0u;
                        tc_mma_i8_pair(tmem_base + acc * kNT, wd + 2 * kk, xd + 2 * kk, idesc, accum);
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
                tc_commit_pair(&tfull[acc]);
            }
        } else if (!leader) {
            // ------------------------------ tile scheduler ----------------------------
            const int step = p.tile_counter ? 0 : (int)(gridDim.x / 2);
            int ahead = (int)(blockIdx.x / 2);  // the next tile; from the counter it is asked for one tile early
            if (!step && lane == 0) ahead = (int)atomicAdd(p.tile_counter, 1u);
            for (int i = 0;; ++i) {
                const int q = i % kQueue;
                int tile = __shfl_sync(0xffffffffu, ahead, 0);
                if (step) ahead += step;
                else if (lane == 0 && tile < total) ahead = (int)atomicAdd(p.tile_counter, 1u);
                Tile t;
                t.g = t.ft = t.row0 = t.n = -1;
                if (tile < total) t = decode(tile, s_prefix, s_off, p, lane);
                if (lane == 0) {
                    if (!mbar_wait_cluster(&qempty[q], ((uint32_t)(i / kQueue) & 1u) ^ 1u, p.status)) s_abort = 1;
                    if (s_abort) t.g = -1;
                    s_tile[q] = t;
                    st_cluster_tile(mapa_shared(smem_u32(&s_tile[q]), 0), t);
                    mbar_arrive(&qfull[q]);
                    mbar_arrive_cluster(mapa_shared(smem_u32(&qfull[q]), 0));  // release: orders the store
                }
                if (__shfl_sync(0xffffffffu, t.g, 0) < 0) break;
            }
        }
        __syncwarp();
    } else {
        // -------------------------------- epilogue --------------------------------
        const int q = warp & 3;          // TMEM lane quarter: weight rows 32q .. 32q+31 of this CTA's 128
        const int r = (warp - 2) >> 2;   // token quarter: tokens 64r .. 64r+63 of the tile
        const int gl = lane >> 2, c2 = 2 * (lane & 3);  // row and first column of this lane in an 8 x 8 block
        const bool up = EPI == I8_SWIGLU && q >= 2;
        uint8_t* stage_out = store + (warp - 2) * kStoreBytes;
        // What a tile's epilogue needs besides the sums.
        struct Work {
            Tile t;
            int64_t f0;          // the features of this warp's weight rows: 32 from here
            float ws[4], bs[4];  // scales and biases of rows gl, gl + 8, gl + 16, gl + 24
            float xs[2];         // scales of tokens 64 r + lane, 64 r + 32 + lane
        };
        const auto take = [&](uint32_t it) {
            Work w;
            if (lane == 0) w.t = take_tile(qfull, s_tile, qempty_l, it, p.status, &s_abort);
            w.t.g = __shfl_sync(0xffffffffu, w.t.g, 0);
            if (w.t.g < 0) return w;
            w.t.ft = __shfl_sync(0xffffffffu, w.t.ft, 0);
            w.t.row0 = __shfl_sync(0xffffffffu, w.t.row0, 0);
            w.t.n = __shfl_sync(0xffffffffu, w.t.n, 0);
            w.f0 = (int64_t)w.t.ft * p.tile_f + (int64_t)rank * (p.tile_f / 2) + (EPI == I8_SWIGLU ? q & 1 : q) * 32;
            const float* scales = up ? p.wscale2 : p.wscale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t f = w.f0 + gl + 8 * i;
                w.ws[i] = f < p.N ? scales[w.t.g * p.N + f] : 0.f;
                w.bs[i] = EPI != I8_SWIGLU && p.bias && f < p.N ? p.bias[w.t.g * p.N + f] : 0.f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = 64 * r + 32 * h + lane;
                w.xs[h] = tok < w.t.n ? p.xscale[w.t.row0 + tok] : 0.f;
            }
            return w;
        };
        // Whether this warp has a tile.  SwiGLU: and its partner, so that neither waits for one that has given up.
        const int bar = 1 + 2 * r + (q & 1);
        const auto going = [&](bool mine) {
            if (EPI != I8_SWIGLU) return mine;
            uint32_t both;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 q, %2, 0;\n\t"
                "bar.red.and.pred p, %1, 64, q;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}\n"
                : "=r"(both)
                : "r"(bar), "r"((uint32_t)mine)
                : "memory");
            return both != 0;
        };
        Work cur = take(0);
        for (uint32_t it = 0; going(cur.t.g >= 0); ++it) {
            const Work next = take(it + 1);
            const Tile& t = cur.t;
            const uint32_t acc = it & 1u;
            int ok = 1;
            if (lane == 0) ok = mbar_wait(&tfull[acc], (it >> 1) & 1u, p.status) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) s_abort = 1;
            tc_fence_after();
            const bool live = !s_abort;
            const int left = t.n - 64 * r;  // tokens from this warp's first on
            const uint32_t tmem = tmem_base + acc * kNT + ((uint32_t)(q * 32) << 16) + (uint32_t)(64 * r);
            // The warp's columns are in registers (tcgen05.wait::ld has returned in all lanes): hand the accumulator back.
            const auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(tempty_l + 8u * acc, 0);
            };
            // v[i][j][e]: row gl + 8 i, token 16 c + 8 j + c2 + e of this warp's 64.  The weight's scale first: tokens
            // may be very large or small, and the scales' product could leave fp32's range where the result does not.
            const auto sums = [&](int c, float (&v)[4][2][2]) {
                uint32_t raw[16];
                tmem_ld_32x16(tmem + 16u * (uint32_t)c, raw);
                tmem_ld_wait(raw);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = __shfl_sync(0xffffffffu, c < 2 ? cur.xs[0] : cur.xs[1], (16 * c + 8 * j + c2 + e) & 31);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i][j][e] = (float)(int)raw[8 * (i >> 1) + 4 * j + 2 * (i & 1) + e] * cur.ws[i] * x;
                    }
            };
            // eight lanes of consecutive features: a whole sector
            const auto put = [&](int c, const float (&v)[4][2][2]) {
                if (!live) return;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = 16 * c + 8 * j + c2 + e;
                        if (tok >= left) continue;
                        TO* dst = static_cast<TO*>(p.out) + (int64_t)(t.row0 + 64 * r + tok) * p.ldo + cur.f0 + gl;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (cur.f0 + gl + 8 * i < p.N) dst[8 * i] = from_f32<TO>(v[i][j][e]);
                    }
            };
            if (left <= 0) {
                release();
            } else if constexpr (EPI == I8_SWIGLU) {
                // The gate's warp finishes the first 32 tokens, the up's the other 32: each gives the other one 16 tokens'
                // products at a time, lane to lane.
                const int mine = up ? 2 : 0, other = 2 - mine;
                uint4* give = reinterpret_cast<uint4*>(stage_out) + lane;
                const uint4* get = reinterpret_cast<const uint4*>(store + (warp - 2 + (up ? 2 : -2)) * kStoreBytes) + lane;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float v[4][2][2], w[4][2][2];
                    if (16 * (other + s) < left) {
                        sums(other + s, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            give[32 * i] = make_uint4(__float_as_uint(v[i][0][0]), __float_as_uint(v[i][0][1]),
                                                      __float_as_uint(v[i][1][0]), __float_as_uint(v[i][1][1]));
                    }
                    const bool own = 16 * (mine + s) < left;
                    if (own) sums(mine + s, v);
                    if (s == 1) release();
                    asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
                    if (own) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 u = get[32 * i];
                            w[i][0][0] = __uint_as_float(u.x), w[i][0][1] = __uint_as_float(u.y);
                            w[i][1][0] = __uint_as_float(u.z), w[i][1][1] = __uint_as_float(u.w);
                        }
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");  // the partner's buffer is read
                    if (own) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    v[i][j][e] = up ? swiglu_f(w[i][j][e], v[i][j][e]) : swiglu_f(v[i][j][e], w[i][j][e]);
                        put(mine + s, v);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (16 * c >= left) continue;
                    float v[4][2][2];
                    sums(c, v);
                    if (c == 3 || left <= 16 * (c + 1)) release();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                v[i][j][e] += cur.bs[i];
                                if (EPI == I8_GELU) v[i][j][e] = gelu_f(v[i][j][e]);
                            }
                    if constexpr (sizeof(TO) == 4) {
                        put(c, v);
                    } else {
                        // 32 tokens at a time: lane 8 m + k addresses token 8 j + k, features 8 m ..; the 16-byte pieces are
                        // swizzled by token pairs
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int tok = 16 * (c & 1) + 8 * j + (lane & 7), m = (lane >> 3) ^ ((tok >> 1) & 3);
                            stmatrix_x4_trans(smem_u32(stage_out + tok * 64 + m * 16), pack_bf16x2(v[0][j][0], v[0][j][1]),
                                              pack_bf16x2(v[1][j][0], v[1][j][1]), pack_bf16x2(v[2][j][0], v[2][j][1]),
                                              pack_bf16x2(v[3][j][0], v[3][j][1]));
                        }
                        if ((c & 1) == 0 && left > 16 * (c + 1)) continue;
                        const int n = left - 32 * (c >> 1) < 32 ? left - 32 * (c >> 1) : 32;
                        TO* out = static_cast<TO*>(p.out) + (int64_t)(t.row0 + 64 * r + 32 * (c >> 1)) * p.ldo + cur.f0;
                        __syncwarp();
                        if (live && p.vec_out && cur.f0 + 32 <= p.N) {
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                const int tok = 8 * s + gl, m = (lane & 3) ^ ((tok >> 1) & 3);
                                const uint4 w = *reinterpret_cast<const uint4*>(stage_out + tok * 64 + m * 16);
                                if (tok < n) *reinterpret_cast<uint4*>(out + (int64_t)tok * p.ldo + 8 * (lane & 3)) = w;
                            }
                        } else if (live) {
                            for (int tok = 0; tok < n; ++tok) {
                                const int m = (lane >> 3) ^ ((tok >> 1) & 3);
                                const uint16_t w = *reinterpret_cast<const uint16_t*>(stage_out + tok * 64 + m * 16 + 2 * (lane & 7));
                                if (cur.f0 + lane < p.N) reinterpret_cast<uint16_t*>(out)[(int64_t)tok * p.ldo + lane] = w;
                            }
                        }
                        __syncwarp();  // the chunk is read
                    }
                }
            }
            cur = next;
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
int launch(const CUtensorMap& mw, const CUtensorMap& mw2, const CUtensorMap& mx, const CUtensorMap& mx128, const Params& kp, int grid,
           cudaStream_t stream) {
    static bool attr_set[64] = {false};
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !attr_set[dev]) {
        MOE_CUDA_TRY(cudaFuncSetAttribute(i8_kernel<EPI, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)kSmemBytes));
        if (dev < 64) attr_set[dev] = true;
    }
    return launch_pdl(i8_kernel<EPI, TO>, grid, kThreads, kSmemBytes, stream, mw, mw2, mx, mx128, kp);
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
    MOE_REQUIRE(p.G == 1 || p.tile_counter, MOE_ERR_WORKSPACE);

    Params kp{};
    kp.G = p.G, kp.M = p.M, kp.N = p.N, kp.offsets = p.offsets;
    kp.xscale = p.xscale, kp.wscale = p.wscale, kp.wscale2 = p.wscale2, kp.bias = p.bias;
    kp.tile_f = dual ? kM : 2 * kM;
    kp.f_tiles = (int)((p.N + kp.tile_f - 1) / kp.tile_f);
    kp.k_blocks = (int)((p.K + kBK - 1) / kBK);
    kp.out = p.out, kp.ldo = p.ldo, kp.status = p.status;
    kp.vec_out = aligned16(p.out) && (p.ldo * dtype_size(p.out_dtype)) % 16 == 0;
    // One group: smaller tiles while they leave pairs idle, all of a size, so the pairs take them in turn.  Several:
    // tiles of up to 256 tokens, drawn from the counter.
    int64_t pairs = device_sm_count() / 2;
    kp.max_span = kNT;
    if (p.G == 1)
        while (kp.max_span > 2 * kBox && 2 * kp.f_tiles * ((p.M + kp.max_span - 1) / kp.max_span) <= pairs) kp.max_span /= 2;
    const int64_t max_tiles = kp.f_tiles * ((p.M + kp.max_span - 1) / kp.max_span + p.G - 1);  // every group may end one early
    MOE_REQUIRE(max_tiles < (int64_t(1) << 30), MOE_ERR_UNSUPPORTED);

    CUtensorMap mw, mw2, mx, mx128;
    MOE_REQUIRE(make_map_i8(&mw, p.w, p.K, p.G * p.N, p.ldw, dual ? kM / 2 : kM), MOE_ERR_CUDA);
    if (dual) MOE_REQUIRE(make_map_i8(&mw2, p.w2, p.K, p.G * p.N, p.ldw, kM / 2), MOE_ERR_CUDA);
    else mw2 = mw;
    MOE_REQUIRE(make_map_i8(&mx, p.x, p.K, p.M, p.ldx, kBox), MOE_ERR_CUDA);
    if (kp.max_span == kNT) MOE_REQUIRE(make_map_i8(&mx128, p.x, p.K, p.M, p.ldx, kNT / 2), MOE_ERR_CUDA);
    else mx128 = mx;
    if (p.G > 1 && max_tiles > pairs) {
        kp.tile_counter = p.tile_counter;
        MOE_CUDA_TRY(cudaMemsetAsync(p.tile_counter, 0, sizeof(uint32_t), stream));
    }
    if (max_tiles < pairs) pairs = max_tiles;
    if (pairs < 1) pairs = 1;
    const int grid = (int)(2 * pairs);
    const bool bf = p.out_dtype == MOE_BF16;
    switch (p.epilogue) {
        case I8_OUT: return bf ? launch<I8_OUT, __nv_bfloat16>(mw, mw2, mx, mx128, kp, grid, stream)
                               : launch<I8_OUT, float>(mw, mw2, mx, mx128, kp, grid, stream);
        case I8_GELU: return bf ? MOE_ERR_UNSUPPORTED : launch<I8_GELU, float>(mw, mw2, mx, mx128, kp, grid, stream);
        case I8_SWIGLU: return bf ? MOE_ERR_UNSUPPORTED : launch<I8_SWIGLU, float>(mw, mw2, mx, mx128, kp, grid, stream);
        default: return MOE_ERR_INVALID_ARG;
    }
}

}  // namespace moe

using namespace moe;

namespace {

constexpr size_t kCounterBytes = 256;

bool ffn_sizes_ok(moe_ffn_kind kind, int32_t G, int64_t M, int64_t D, int64_t F, int64_t Dout) {
    return G >= 1 && M >= 0 && D >= 1 && Dout >= 1 && (kind == MOE_FFN_LINEAR || F >= 1);
}

// in 32 bits, and so that no product of two of them passes 64
bool ffn_limits_ok(moe_ffn_kind kind, int64_t M, int64_t F, int64_t Dout) {
    return M < (int64_t(1) << 30) && Dout < (int64_t(1) << 30) && (kind == MOE_FFN_LINEAR || F < (int64_t(1) << 30));
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

extern "C" size_t moe_matmul_i8_workspace_size(int64_t M, int32_t G, int64_t N, int64_t K) {
    return M < 1 || G <= 1 || N < 1 || K < 1 || i8_skinny_fits(M, G, N, K) ? 0 : kCounterBytes;
}

extern "C" int moe_matmul_i8(const int8_t* xq, const float* xscale, int64_t M, int64_t ldx, const int32_t* offsets,
                             const int8_t* wq, const float* wscale, int64_t ldw, const float* bias, int32_t G,
                             int64_t N, int64_t K, void* out, int64_t ldo, moe_dtype out_dtype, int32_t* dev_status,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    const size_t need = moe_matmul_i8_workspace_size(M, G, N, K);
    MOE_REQUIRE(need == 0 || (workspace && aligned16(workspace) && workspace_bytes >= need), MOE_ERR_WORKSPACE);
    I8Problem p{};
    p.x = xq, p.xscale = xscale, p.M = M, p.ldx = ldx, p.offsets = offsets, p.w = wq, p.wscale = wscale;
    p.ldw = ldw, p.bias = bias, p.G = G, p.N = N, p.K = K, p.out = out, p.ldo = ldo, p.out_dtype = out_dtype;
    p.epilogue = I8_OUT, p.tile_counter = static_cast<uint32_t*>(workspace), p.status = dev_status;
    return i8_gemm_run(p, reinterpret_cast<cudaStream_t>(stream));
}

// workspace: [counters | hscale (M) | hq (M, round16(F)) | h (M, F) fp32]
extern "C" size_t moe_expert_ffn_i8_workspace_size(moe_ffn_kind kind, int32_t G, int64_t M, int64_t D, int64_t F,
                                                   int64_t Dout) {
    if (!ffn_sizes_ok(kind, G, M, D, F, Dout) || !ffn_limits_ok(kind, M, F, Dout) || M == 0) return 0;
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
    MOE_REQUIRE(ffn_limits_ok(kind, M, F, Dout), MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(kind != MOE_FFN_SWIGLU || (!b1 && !b2), MOE_ERR_INVALID_ARG);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(workspace && aligned16(workspace) &&
                    workspace_bytes >= moe_expert_ffn_i8_workspace_size(kind, G, M, D, F, Dout),
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
    MOE_REQUIRE(aligned16(w2) && ldw2 % 16 == 0 && ldw2 < (int64_t(1) << 38) && F <= 131071 && G * Dout < (int64_t(1) << 30) &&
                    reinterpret_cast<uintptr_t>(ys) % dtype_size(out_dtype) == 0,
                MOE_ERR_UNSUPPORTED);
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kCounterBytes;
    float* hscale = reinterpret_cast<float*>(ws);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + align_up((size_t)M * sizeof(float), 256));
    float* h = reinterpret_cast<float*>(hq + align_up((size_t)M * round16(F), 256));
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
