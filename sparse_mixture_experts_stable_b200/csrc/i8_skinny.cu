// The product of i8_gemm.cu where a group has few rows: the weights' bytes, read once, are
// what it costs, and the tensor memory, barriers and maps of that kernel take longer to set
// up than a short product takes.  A tile of 128 or 256 features would also leave most SMs
// without one.
//
// A block takes a contiguous run of units; a unit is up to kTok tokens of a group (they lie
// in shared memory) and a block of 128 weight rows (64 of gate and 64 of up for SwiGLU), 16
// per warp; where units are few, `ksplit` warps share 16 rows' depth and a unit has fewer
// rows.  One thread fills a ring of kStages stages of 32 KB, 256 bytes of each row, by TMA:
// up to 160 KB are in flight per SM whatever the arithmetic takes.  (Rings of the warps' own
// took 8 to 16 copies for the same 32 KB; the SM issues one in some 70 cycles, and that was
// as long as the memory needs.)  A row's 256 bytes lie in two swizzled halves, and the rows
// that a warp reads together are chosen so that they meet no bank conflict: with unswizzled
// rows of 256 bytes a stage took 900 cycles of shared memory, and the memory brings one in
// 1400 (103 experts of 2048 x 512 26.4 us, now 24.2; of 1024 x 2048 40.1, now 38.4).
// Products are m16n8k32 of the warp-level tensor instructions on 8-bit integers: a tenth of
// the weights' time, so tcgen05 has nothing to win here.  The order of k is free as long as
// both operands share it, so a lane's four bytes of each fragment are neighbours and come in
// 16-byte reads.  With fp32 rows (the experts' hidden rows) every block quantises the rows
// that it stages: a few KB, against a launch and a round trip through memory.
// What bounds it: the weights stream at 6.7 TB/s (one row times 131072 x 2048: 46 us); a
// launch costs 7 us besides: 1.7 us until the first copy is asked for (offsets, their scan),
// 2 until it is there and the tokens are staged, the last unit and the launch itself.  Two
// sets of eight warps that take the stages in turn gained nothing (26.2 us and 40.9).
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

constexpr int kWarps = 8;                      // that multiply; one more loads
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRows = 16;                      // weight rows of a warp
constexpr int kSeg = 256;                      // bytes of each in a stage,
constexpr int kHalf = 128;                     // in two swizzled halves
constexpr int kStageBytes = kWarps * kRows * kSeg;
constexpr int kStages = 5;
constexpr int kTok = 16;                 // tokens in shared memory at a time, at most
constexpr int kMaxG = 1024;
constexpr int64_t kMaxK = 4096;
constexpr size_t kRingBytes = (size_t)kStages * kStageBytes;
constexpr size_t kTokBytes = (size_t)kTok * (2048 + 64) + kSeg;  // the last piece is read whole

struct SkinnyParams {
    I8Problem p;
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
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// `threads` of the block; barrier 0 is __syncthreads'
__device__ __forceinline__ void part_sync(int barrier, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}

// A place in the sequence of units: item (tokens of a group) and feature block.
struct Cursor {
    int item, fb, g;
    // prefix[g]: the items before group g.  By the 32 lanes of a warp together: the last group whose items do not begin
    // behind this one, in a 32nd of the groups, then in that.
    __device__ __forceinline__ void seek(int unit, int fblocks, const int* prefix, int G, int lane) {
        item = unit / fblocks;
        fb = unit - item * fblocks;
        const int stride = (G + 31) / 32;  // up to 32, as G is up to kMaxG
        const int part = __popc(__ballot_sync(0xffffffffu, lane * stride < G && prefix[lane * stride] <= item)) - 1;
        const int at = part * stride + lane;
        g = part * stride - 1 + __popc(__ballot_sync(0xffffffffu, lane < stride && at < G && prefix[at] <= item));
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
    extern __shared__ uint8_t s_raw[];                           // the ring, then the tokens (tok, xpitch)
    __shared__ uint64_t s_full[kStages], s_empty[kStages];
    __shared__ int s_prefix[kMaxG + 1], s_off[kMaxG], s_end[kMaxG];
    __shared__ float s_scale[kTok];
    __shared__ int s_red[2][kWarps][8][32];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_x = ring + kRingBytes;
    const I8Problem& p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int teams = kWarps / sp.ksplit;
    if (threadIdx.x < kStages) {
        tc::mbar_init(&s_full[threadIdx.x], 1);
        tc::mbar_init(&s_empty[threadIdx.x], kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_next();
    bool back = false;
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
        int lo = 0, hi = (int)p.M;
        if (p.offsets) lo = min(max(p.offsets[g], 0), hi), hi = min(max(p.offsets[g + 1], 0), hi);
        back |= hi < lo;
        s_off[g] = lo;
        s_end[g] = hi;
        s_prefix[g] = hi > lo ? (hi - lo + sp.tok - 1) / sp.tok : 0;
    }
    if (__syncthreads_or(back)) {  // offsets that run backwards become their running maximum: no row has two groups
        if (threadIdx.x == 0) {
            set_status(p.status, MOE_ERR_BAD_INDEX);
            for (int g = 0, run = 0; g < p.G; ++g) {
                s_off[g] = max(s_off[g], run);
                run = s_end[g] = max(s_end[g], s_off[g]);
                s_prefix[g] = (s_end[g] - s_off[g] + sp.tok - 1) / sp.tok;
            }
        }
        __syncthreads();
    }
    block_scan<kThreads>(s_prefix, p.G);
    // in 32 bits: 64-bit divisions take 800 cycles here
    const uint32_t units = (uint32_t)s_prefix[p.G] * (uint32_t)sp.fblocks;
    const uint32_t share = units / gridDim.x, more = units - share * gridDim.x;
    const int u0 = (int)(share * blockIdx.x + min(blockIdx.x, more)), u1 = u0 + (int)(share + (blockIdx.x < more ? 1 : 0));
    if (u0 >= u1) return;

    Cursor use;
    use.seek(u0, sp.fblocks, s_prefix, p.G, lane);
    if (warp == kWarps) {
        // -------------------------------- loads --------------------------------
        if (lane == 0) {
            const int rows = teams * kRows, half = teams * FROWS;  // of a piece of the depth; of gate, for SwiGLU
            int stage = 0;
            uint32_t phase = 0, used = 0, last = 0;  // used, last: a bit per stage
            bool ok = true;
            for (int unit = u0; unit < u1 && ok; ++unit, use.next(sp.fblocks, s_prefix, p.G)) {
                const int row = (int)(use.g * p.N + (int64_t)use.fb * half);
                for (int seg = 0; seg < sp.segs; seg += sp.ksplit) {
                    if (!tc::mbar_wait(&s_empty[stage], phase ^ 1u, p.status)) {
                        ok = false;
                        break;
                    }
                    const int parts = min(sp.ksplit, sp.segs - seg);
                    uint8_t* dst = ring + stage * kStageBytes;
                    tc::mbar_expect_tx(&s_full[stage], (uint32_t)(parts * rows * kSeg));
                    for (int k = 0; k < 2 * parts; ++k, dst += rows * kHalf) {
                        tc::tma_load_2d(dst, &tm_w, seg * kSeg + k * kHalf, row, &s_full[stage]);
                        if (EPI == I8_SWIGLU) tc::tma_load_2d(dst + half * kHalf, &tm_w2, seg * kSeg + k * kHalf, row, &s_full[stage]);
                    }
                    used |= 1u << stage;
                    last = (last & ~(1u << stage)) | phase << stage;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < kStages; ++s)  // whatever happens, the block does not end before its copies have landed
                if (used >> s & 1) tc::mbar_wait(&s_full[s], last >> s & 1, p.status);
        }
        return;
    }

    // -------------------------------- products --------------------------------
    const int kpart = warp % sp.ksplit, team = warp / sp.ksplit;
    // this warp's place in a stage: its piece of the depth, its rows (for SwiGLU those of gate; up's follow all of gate's)
    const int w_half = teams * kRows * kHalf;  // from the first 128 bytes of the piece's rows to the second
    const int w_at = kpart * 2 * w_half + team * FROWS * kHalf, w_second = (EPI == I8_SWIGLU ? teams * FROWS : 8) * kHalf;
    bool dead = false;  // a wait timed out (status set): nothing more is written, the barriers are kept
    const int gl = lane >> 2, q = lane & 3;  // fragment row (token) and 16-byte column of this lane
    // Weight row of the fragment row: those that are read together, an even and the next one, are four apart, so the
    // swizzle (16-byte column ^ row) puts them in different banks.
    const int wl = gl >> 1 | (gl & 1) << 2;
    uint32_t phase = 0;
    int stage = 0, item = -1, t0 = 0, nt = 0;
    for (int unit = u0; unit < u1; ++unit) {
        if (use.item != item) {  // other tokens (the same for all warps)
            item = use.item;
            t0 = s_off[use.g] + (item - s_prefix[use.g]) * sp.tok;
            nt = min(s_end[use.g] - t0, sp.tok);
            part_sync(kWarps + 1, kWarps * 32);  // the tokens before have been read
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
                float scale = 0.f;
                if (threadIdx.x < nt) scale = p.xscale[t0 + threadIdx.x];
                // pieces of all tokens, four per thread on their way
                const int per = (sp.xpitch - 64) / 16;
                for (int i0 = threadIdx.x; i0 < nt * per; i0 += 4 * kWarps * 32) {
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int i = i0 + u * kWarps * 32, t = i / per, c = (i - t * per) * 16;
                        v[u] = make_uint4(0, 0, 0, 0);
                        if (i >= nt * per) continue;
                        const int8_t* src = p.x + (int64_t)(t0 + t) * p.ldx + c;
                        if (c + 16 <= p.K) v[u] = *reinterpret_cast<const uint4*>(src);
                        else if (c < p.K) v[u] = load_part(src, (int)p.K - c);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int i = i0 + u * kWarps * 32, t = i / per, c = (i - t * per) * 16;
                        if (i < nt * per) *reinterpret_cast<uint4*>(s_x + t * sp.xpitch + c) = v[u];
                    }
                }
                if (threadIdx.x < nt) s_scale[threadIdx.x] = scale;
            }
            part_sync(kWarps + 1, kWarps * 32);
        }
        const int64_t f0 = ((int64_t)use.fb * teams + team) * FROWS;
        // features of this lane's sums: weight rows wl and wl + 8
        const int64_t fa = f0 + wl, fc = EPI == I8_SWIGLU ? fa : fa + 8;
        float wsa = 0.f, wsc = 0.f, ba = 0.f, bc = 0.f;
        if (fa < p.N) wsa = p.wscale[use.g * p.N + fa];
        if (fc < p.N) wsc = (EPI == I8_SWIGLU ? p.wscale2 : p.wscale)[use.g * p.N + fc];
        if (EPI != I8_SWIGLU && p.bias) {
            if (fa < p.N) ba = p.bias[use.g * p.N + fa];
            if (fc < p.N) bc = p.bias[use.g * p.N + fc];
        }
        int acc[2][4] = {}, part[2][4] = {};  // two chains of products each
        for (int seg = kpart; seg - kpart < sp.segs; seg += sp.ksplit) {
            if (!dead) dead = !__all_sync(0xffffffffu, tc::mbar_wait(&s_full[stage], phase, p.status));
            if (seg < sp.segs) {
                const uint8_t* wr = ring + stage * kStageBytes + w_at + wl * kHalf;
                const uint8_t* xr = s_x + gl * sp.xpitch + seg * kSeg + q * 16;
                // beyond K the weights' pieces hold zeros
                uint4 a[kSeg / 64], c[kSeg / 64], b[kSeg / 64];
#pragma unroll
                for (int i = 0; i < kSeg / 64; ++i) {
                    const uint8_t* w = wr + (i >> 1) * w_half + ((q + 4 * (i & 1)) ^ wl) * 16;
                    a[i] = *reinterpret_cast<const uint4*>(w);
                    c[i] = *reinterpret_cast<const uint4*>(w + w_second);
                    b[i] = *reinterpret_cast<const uint4*>(xr + 64 * i);
                }
#pragma unroll
                for (int i = 0; i < kSeg / 64; ++i) {
                    mma_i8(acc[0], a[i].x, c[i].x, a[i].y, c[i].y, b[i].x, b[i].y);
                    mma_i8(part[0], a[i].z, c[i].z, a[i].w, c[i].w, b[i].z, b[i].w);
                }
                if (nt > 8) {
#pragma unroll
                    for (int i = 0; i < kSeg / 64; ++i) b[i] = *reinterpret_cast<const uint4*>(xr + 8 * sp.xpitch + 64 * i);
#pragma unroll
                    for (int i = 0; i < kSeg / 64; ++i) {
                        mma_i8(acc[1], a[i].x, c[i].x, a[i].y, c[i].y, b[i].x, b[i].y);
                        mma_i8(part[1], a[i].z, c[i].z, a[i].w, c[i].w, b[i].z, b[i].w);
                    }
                }
            }
            __syncwarp();  // the stage is read
            if (lane == 0) tc::mbar_arrive(&s_empty[stage]);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += part[i >> 2][i & 3];
        int(*red)[8][32] = s_red[unit & 1];  // the unit before may still be read
        if (sp.ksplit > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) red[warp][i][lane] = acc[i >> 2][i & 3];
            part_sync(1 + team, 32 * sp.ksplit);
        }
        // tokens 2q, 2q + 1, 8 + 2q, 9 + 2q; the warps that share the depth share them
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (i >> 1) * 8 + 2 * q + (i & 1);
            if (dead || f0 >= p.N || i % sp.ksplit != kpart || (i >> 1) * 8 >= nt) continue;
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
            float u = (float)sa * wsa * x, v = (float)sc * wsc * x;  // in this order: the scales' product could leave fp32
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
    sp.segs = (int)((p.K + kSeg - 1) / kSeg);
    sp.xpitch = (int)((p.K + 127) / 128 * 128 + 64);
    sp.tok = p.K <= 2048 ? kTok : kTok / 2;
    sp.vecx = aligned16(p.x) && p.ldx % 4 == 0;
    // warps share a row's depth until the blocks have some two units each; more warps on a depth mean more waiting for one
    // another and more copies per stage
    const int64_t items = (p.M + sp.tok - 1) / sp.tok + (p.M < p.G ? p.M : p.G) - 1;  // at most
    const int64_t sms = device_sm_count();
    int64_t units = 0;
    for (sp.ksplit = 1;; sp.ksplit *= 2) {
        const int64_t per = kWarps / sp.ksplit * (EPI == I8_SWIGLU ? kRows / 2 : kRows);
        sp.fblocks = (int)((p.N + per - 1) / per);
        units = items * sp.fblocks;
        if (sp.ksplit == kWarps || 2 * sp.ksplit > sp.segs || units >= 2 * sms) break;
    }
    CUtensorMap mw, mw2;
    constexpr bool dual = EPI == I8_SWIGLU;
    const int box = kWarps / sp.ksplit * (dual ? kRows / 2 : kRows);
    MOE_REQUIRE(make_map_i8(&mw, p.w, p.K, p.G * p.N, p.ldw, box), MOE_ERR_CUDA);
    if (dual) MOE_REQUIRE(make_map_i8(&mw2, p.w2, p.K, p.G * p.N, p.ldw, box), MOE_ERR_CUDA);
    return launch_pdl(kernel, units < sms ? units : sms, kThreads, 1024 + kRingBytes + (size_t)sp.tok * sp.xpitch + kSeg, stream,
                      mw, dual ? mw2 : mw, sp);
}

}  // namespace

// Where this kernel is the faster one.  One group: N = K = 2048 13.1 us at 128 rows, as the tiles, 9.7 at 64 (tiles 20).
// Groups: SwiGLU experts (E = 256, 2048 x 512, weights in memory) 108 us with 2 rows a group on average (tiles 140), 162 with
// 8 (175), 198 with 12 (179); (E = 64, 1000 x 200) 27 us with 8 (39), 33 with 16 (42).
// The rule knows the mean only, and a full group has its weights read once per kTok rows: G + M / kTok blocks of weights in
// all at most, half as many again as a balanced call's (K > 2048: twice as many), and fewer groups' from memory.  All rows in one of 256 groups of 2048 x 512: 256 rows 8 us (tiles 15), 1024 17 (15), 2048 28
// (17); balanced 55 (66); half of 2048 in one 65 (69).  1024 groups of 2048 x 2048, 8192 rows: in one 305 us (45), balanced
// 635 (748), half in one 728 (752).
// kMaxK: the tokens' rows lie whole in shared memory beside the ring (33 KB for 8 of 4096).  One row times 2048 x 4096 6 us,
// 2048 x 4112 (tiles, of which 8 pairs have one) 19, 2048 x 8192 31, 4096 x 14336 49.  kMaxG: the groups' tables; 8 rows each
// of 1024 groups of 512 x 512 61 us, of 1025 (tiles) 69.
bool i8_skinny_fits(int64_t M, int G, int64_t N, int64_t K) {
    if (K > kMaxK || G > kMaxG || N >= (int64_t(1) << 30)) return false;  // N: the product below stays in 64 bits
    return G == 1 ? M <= 2048 && M * N * K <= 600000000 : M <= 8 * (int64_t)G;
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
