// The product of i8_gemm.cu where a group has few rows: the weights' bytes, read once, are
// what it costs, and the tensor memory, barriers and maps of that kernel take longer to set
// up than a short product takes.  A tile of 128 or 256 features would also leave most SMs
// without one.
//
// A block takes a contiguous run of units; a unit is up to kTok tokens of a group (they lie
// in shared memory) and a block of features, 16 weight rows per warp (8 of gate and 8 of up
// for SwiGLU) or, where units are few, per `ksplit` warps that share the depth.  Every warp
// streams its rows through a ring of its own, kStages stages of 16 x 256 bytes filled by TMA:
// 128 KB are in flight per SM whatever the arithmetic takes, at two instructions per stage
// (a bulk copy per row took longer to issue than to arrive), and no warp waits for another
// one's loads.  Products are m16n8k32 of the warp-level tensor instructions on 8-bit
// integers: with dp4a the arithmetic of 8 tokens took twice as long as the weights' way from
// memory, with these it is a tenth of it, so tcgen05 has nothing to win here.  The order of
// k is free as long as both operands share it, so a lane's four bytes of each fragment are
// neighbours and come in 16-byte reads.  With fp32 rows (the experts' hidden rows) every
// block quantises the rows that it stages: a few KB, against a launch and a round trip
// through memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "i8_gemm.cuh"
#include "quant_i8.cuh"
#include "tc_gemm.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;    // weight rows of a stage
constexpr int kSeg = 256;    // bytes of each: two TMA boxes side by side
constexpr int kStageBytes = kRows * kSeg;
constexpr int kStages = 5;
constexpr int kTok = 16;                 // tokens in shared memory at a time, at most
constexpr int kMaxG = 1024;
constexpr int64_t kMaxK = 4096;
constexpr size_t kRingBytes = (size_t)kWarps * kStages * kStageBytes;
constexpr size_t kTokBytes = (size_t)kTok * (2048 + 64);

struct SkinnyParams {
    I8Problem p;
    int K16;      // 16-byte pieces of a row
    int segs;     // kSeg-byte pieces of a row
    int xpitch;   // bytes between tokens in shared memory, 64 modulo 128
    int tok;      // tokens in shared memory at a time: 8 or 16
    int ksplit;   // warps that share a row's depth: 1, 2, 4 or 8
    int fblocks;  // units of a group's tokens
    bool vecx;    // fp32 rows start on 16 bytes
};

// the first n bytes of a 16-byte piece, zeros behind them
static __device__ __noinline__ uint4 load_part(const int8_t* s, int n) {
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) v[i >> 2] |= (uint32_t)(uint8_t)s[i] << (8 * (i & 3));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// d += a b: 16 weight rows x 32 values, 8 tokens
__device__ __forceinline__ void mma_i8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the threads of one team of warps
__device__ __forceinline__ void team_sync(int team, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// A place in the sequence of units: item (tokens of a group) and feature block.
struct Cursor {
    int item, fb, g;
    // prefix[g]: the items before group g
    __device__ __forceinline__ void seek(int unit, int fblocks, const int* prefix, int G) {
        item = unit / fblocks;
        fb = unit - item * fblocks;
        g = 0;
        find(prefix, G);
    }
    __device__ __forceinline__ void next(int fblocks, const int* prefix, int G) {
        if (++fb < fblocks) return;
        fb = 0;
        ++item;
        if (prefix[g + 1] <= item) find(prefix, G);
    }
    // the group of the item, from g on (the groups without rows between two with rows may be hundreds)
    __device__ __forceinline__ void find(const int* prefix, int G) {
        int lo = g, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= item) lo = mid;
            else hi = mid - 1;
        }
        g = lo;
    }
};

template <int EPI, typename TO, bool F32X>
__global__ void __launch_bounds__(kThreads, 1)
    skinny_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_w2,
                  const SkinnyParams sp) {
    constexpr int FROWS = EPI == I8_SWIGLU ? kRows / 2 : kRows;  // output features of 16 weight rows
    extern __shared__ uint8_t s_raw[];                           // rings of the warps, then the tokens (tok, xpitch)
    __shared__ uint64_t s_bar[kWarps][kStages];
    __shared__ int s_prefix[kMaxG + 1], s_off[kMaxG + 1];
    __shared__ float s_scale[kTok];
    __shared__ int s_red[2][kWarps][8][32];
    uint8_t* s_dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
    const I8Problem& p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kpart = warp % sp.ksplit, team = warp / sp.ksplit, teams = kWarps / sp.ksplit;
    uint8_t* ring = s_dyn + (size_t)warp * kStages * kStageBytes;
    uint8_t* s_x = s_dyn + kRingBytes;
    if (lane < kStages) tc::mbar_init(&s_bar[warp][lane], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_next();
    for (int g = threadIdx.x; g <= p.G; g += kThreads)
        s_off[g] = p.offsets ? min(max(p.offsets[g], 0), (int)p.M) : g == 0 ? 0 : (int)p.M;
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
        const int n = s_off[g + 1] - s_off[g];
        if (n < 0) set_status(p.status, MOE_ERR_BAD_INDEX);
        s_prefix[g] = n > 0 ? (n + sp.tok - 1) / sp.tok : 0;
    }
    __syncthreads();
    block_scan<kThreads>(s_prefix, p.G);
    const int64_t units = (int64_t)s_prefix[p.G] * sp.fblocks;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    if (u0 >= u1) return;

    Cursor load, use;
    load.seek(u0, sp.fblocks, s_prefix, p.G);
    use = load;
    int load_unit = u0, load_seg = kpart, ahead = 0;  // ahead: stages on their way
    // where this warp's features of a unit begin; it takes part if they exist
    const auto feature = [&](const Cursor& c) { return ((int64_t)c.fb * teams + team) * FROWS; };
    // Fills the stage with the next piece of this warp's sequence, if there is one.
    const auto fetch = [&](int stage) {
        while (load_unit < u1 && (feature(load) >= p.N || load_seg >= sp.segs)) {
            ++load_unit;
            load_seg = kpart;
            load.next(sp.fblocks, s_prefix, p.G);
        }
        if (load_unit >= u1) return;
        if (lane == 0) {
            uint64_t* bar = &s_bar[warp][stage];
            uint8_t* dst = ring + stage * kStageBytes;
            const int row = (int)(load.g * p.N + feature(load));
            tc::mbar_expect_tx(bar, kStageBytes);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int k = load_seg * kSeg + b * 128;
                tc::tma_load_2d(dst + b * kRows * 128, &tm_w, k, row, bar);
                if (EPI == I8_SWIGLU) tc::tma_load_2d(dst + b * kRows * 128 + FROWS * 128, &tm_w2, k, row, bar);
            }
        }
        load_seg += sp.ksplit;
        ++ahead;
    };
    for (int s = 0; s < kStages - 1; ++s) fetch(s);

    // Fragment row (weight row, token) and 16-byte column of this lane.  Weight row gl of the fragment is row wr of the
    // stage, so that the eight lanes of a read see rows 4 apart: the swizzle then gives them different banks.
    const int gl = lane >> 2, q = lane & 3, wr = gl >> 1 | (gl & 1) << 2;
    uint32_t phase = 0;                      // a bit per stage
    int stage = 0, item = -1, t0 = 0, nt = 0;
    for (int unit = u0; unit < u1; ++unit) {
        if (use.item != item) {  // other tokens (the same for all warps)
            item = use.item;
            t0 = s_off[use.g] + (item - s_prefix[use.g]) * sp.tok;
            nt = min(s_off[use.g + 1] - t0, sp.tok);
            __syncthreads();  // the tokens before have been read
            if constexpr (F32X) {
                for (int t = warp; t < nt; t += kWarps) {
                    const float* src = reinterpret_cast<const float*>(p.x) + (int64_t)(t0 + t) * p.ldx;
                    const RowQuant r = row_quant(row_max<1>(src, p.K, sp.vecx, nullptr), p.status, lane == 0);
                    for (int c = lane * 4; c < sp.xpitch - 64; c += 128) {
                        Raw<float> x;
                        uint32_t o[1] = {0};
                        if (c < p.K) {
                            x.load(src + c, p.K - c, sp.vecx);
                            quantize_chunk(x, r, o);
                        }
                        *reinterpret_cast<uint32_t*>(s_x + t * sp.xpitch + c) = o[0];
                    }
                    if (lane == 0) s_scale[t] = r.scale;
                }
            } else {
                for (int t = warp; t < nt; t += kWarps) {
                    const int8_t* src = p.x + (int64_t)(t0 + t) * p.ldx;
                    for (int c = lane * 16; c < sp.xpitch - 64; c += 512) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (c + 16 <= p.K) v = *reinterpret_cast<const uint4*>(src + c);
                        else if (c < p.K) v = load_part(src + c, (int)p.K - c);
                        *reinterpret_cast<uint4*>(s_x + t * sp.xpitch + c) = v;
                    }
                }
                if (threadIdx.x < nt) s_scale[threadIdx.x] = p.xscale[t0 + threadIdx.x];
            }
            __syncthreads();
        }
        const int64_t f0 = feature(use);
        const bool live = f0 < p.N;
        // features of this lane's sums: weight rows wr and wr + 8
        const int64_t fa = f0 + wr, fc = EPI == I8_SWIGLU ? fa : fa + 8;
        float wsa = 0.f, wsc = 0.f, ba = 0.f, bc = 0.f;
        if (fa < p.N) wsa = p.wscale[use.g * p.N + fa];
        if (fc < p.N) wsc = (EPI == I8_SWIGLU ? p.wscale2 : p.wscale)[use.g * p.N + fc];
        if (EPI != I8_SWIGLU && p.bias) {
            if (fa < p.N) ba = p.bias[use.g * p.N + fa];
            if (fc < p.N) bc = p.bias[use.g * p.N + fc];
        }
        int acc[2][4] = {}, part[2][4] = {};  // two chains of products each
        if (live) {
            for (int seg = kpart; seg < sp.segs; seg += sp.ksplit) {
                fetch(stage == 0 ? kStages - 1 : stage - 1);
                const bool landed = __all_sync(0xffffffffu, tc::mbar_wait(&s_bar[warp][stage], phase >> stage & 1, p.status));
                phase ^= 1u << stage;
                --ahead;
                if (!landed) {  // timed out (status set): the copies in flight are waited for, nothing more is written
                    for (int i = 0; i < ahead; ++i) {
                        stage = stage + 1 == kStages ? 0 : stage + 1;
                        tc::mbar_wait(&s_bar[warp][stage], phase >> stage & 1, p.status);
                    }
                    return;
                }
                const uint8_t* st = ring + stage * kStageBytes + wr * 128;
                const uint8_t* xr = s_x + gl * sp.xpitch + seg * kSeg + q * 16;
                const int windows = min(kSeg, (int)p.K - seg * kSeg + 63) / 64;
#pragma unroll
                for (int i = 0; i < kSeg / 64; ++i) {
                    if (i >= windows) break;
                    const uint8_t* w = st + (i >> 1) * (kRows * 128) + ((4 * (i & 1) + q) ^ wr) * 16;
                    const uint4 a = *reinterpret_cast<const uint4*>(w);
                    const uint4 c = *reinterpret_cast<const uint4*>(w + 8 * 128);
                    const uint4 b = *reinterpret_cast<const uint4*>(xr + 64 * i);
                    mma_i8(acc[0], a.x, c.x, a.y, c.y, b.x, b.y);
                    mma_i8(part[0], a.z, c.z, a.w, c.w, b.z, b.w);
                    if (nt > 8) {
                        const uint4 d = *reinterpret_cast<const uint4*>(xr + 8 * sp.xpitch + 64 * i);
                        mma_i8(acc[1], a.x, c.x, a.y, c.y, d.x, d.y);
                        mma_i8(part[1], a.z, c.z, a.w, c.w, d.z, d.w);
                    }
                }
                __syncwarp();  // the stage may be filled again
                if (++stage == kStages) stage = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += part[i >> 2][i & 3];
        int(*red)[8][32] = s_red[unit & 1];  // the unit before may still be read
        if (sp.ksplit > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) red[warp][i][lane] = acc[i >> 2][i & 3];
            team_sync(team, 32 * sp.ksplit);
        }
        // tokens 2q, 2q + 1, 8 + 2q, 9 + 2q; the warps that share the depth share them
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (i >> 1) * 8 + 2 * q + (i & 1);
            if (!live || i % sp.ksplit != kpart || (i >> 1) * 8 >= nt) continue;
            int sa = acc[i >> 1][i & 1], sc = acc[i >> 1][2 + (i & 1)];
            if (sp.ksplit > 1) {
                sa = sc = 0;
                for (int w = 0; w < sp.ksplit; ++w) {
                    sa += red[warp - kpart + w][(i >> 1) * 4 + (i & 1)][lane];
                    sc += red[warp - kpart + w][(i >> 1) * 4 + 2 + (i & 1)][lane];
                }
            }
            if (t >= nt) continue;
            const float x = s_scale[t];
            float u = (float)sa * (wsa * x), v = (float)sc * (wsc * x);
            TO* out = static_cast<TO*>(p.out) + (int64_t)(t0 + t) * p.ldo;
            if (EPI == I8_SWIGLU) {
                if (fa < p.N) out[fa] = from_f32<TO>(swiglu_f(u, v));
            } else {
                u += ba, v += bc;
                if (EPI == I8_GELU) u = tc::gelu_f(u), v = tc::gelu_f(v);
                if (fa < p.N) out[fa] = from_f32<TO>(u);
                if (fc < p.N) out[fc] = from_f32<TO>(v);
            }
        }
        use.next(sp.fblocks, s_prefix, p.G);
    }
}

template <int EPI, typename TO, bool F32X>
int launch(const I8Problem& p, cudaStream_t stream) {
    const auto kernel = skinny_kernel<EPI, TO, F32X>;
    static bool attr_set[64] = {false};
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !attr_set[dev]) {
        MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)(1024 + kRingBytes + kTokBytes)));
        if (dev < 64) attr_set[dev] = true;
    }
    SkinnyParams sp{};
    sp.p = p;
    sp.K16 = (int)((p.K + 15) / 16);
    sp.segs = (int)((p.K + kSeg - 1) / kSeg);
    sp.xpitch = (int)((p.K + 127) / 128 * 128 + 64);
    sp.tok = p.K <= 2048 ? kTok : kTok / 2;
    sp.vecx = aligned16(p.x) && p.ldx % 4 == 0;
    // warps share a row's depth until the blocks have some four units each (more warps on a depth mean more waiting for one another)
    const int64_t items = (p.M + sp.tok - 1) / sp.tok + (p.M < p.G ? p.M : p.G) - 1;  // at most
    const int64_t sms = device_sm_count();
    int64_t units = 0;
    for (sp.ksplit = 1;; sp.ksplit *= 2) {
        const int64_t per = kWarps / sp.ksplit * (EPI == I8_SWIGLU ? kRows / 2 : kRows);
        sp.fblocks = (int)((p.N + per - 1) / per);
        units = items * sp.fblocks;
        if (sp.ksplit == kWarps || 2 * sp.ksplit > sp.segs || units >= 4 * sms) break;
    }
    CUtensorMap mw, mw2;
    constexpr bool dual = EPI == I8_SWIGLU;
    MOE_REQUIRE(make_map_i8(&mw, p.w, p.K, p.G * p.N, p.ldw, dual ? kRows / 2 : kRows), MOE_ERR_CUDA);
    if (dual) MOE_REQUIRE(make_map_i8(&mw2, p.w2, p.K, p.G * p.N, p.ldw, kRows / 2), MOE_ERR_CUDA);
    return launch_pdl(kernel, units < sms ? units : sms, kThreads, 1024 + kRingBytes + (size_t)sp.tok * sp.xpitch, stream,
                      mw, dual ? mw2 : mw, sp);
}

}  // namespace

bool i8_skinny_fits(int64_t M, int G, int64_t N, int64_t K) {
    if (K > kMaxK || G > kMaxG) return false;
    if (G == 1) return M <= 2048 && M * N * K <= 600000000;
    return M <= 4 * (int64_t)G;
}

int i8_skinny_run(const I8Problem& p, bool f32x, cudaStream_t stream) {
    const bool bf = p.out_dtype == MOE_BF16;
    if (p.epilogue == I8_OUT) {
        if (f32x) return bf ? launch<I8_OUT, __nv_bfloat16, true>(p, stream) : launch<I8_OUT, float, true>(p, stream);
        return bf ? launch<I8_OUT, __nv_bfloat16, false>(p, stream) : launch<I8_OUT, float, false>(p, stream);
    }
    if (f32x || bf) return MOE_ERR_UNSUPPORTED;
    return p.epilogue == I8_GELU ? launch<I8_GELU, float, false>(p, stream) : launch<I8_SWIGLU, float, false>(p, stream);
}

}  // namespace moe
