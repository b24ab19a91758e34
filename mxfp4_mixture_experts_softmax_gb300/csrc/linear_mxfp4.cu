// linear_mxfp4.cu -- a dense projection with MXFP4 weights and activations
// quantised to MXFP4 inside the call:
//   xq = decode(quantise(x))  per token, blocks of 32 along K
//   out[t, n] = residual[t, n] + sum_k decode(W)[n, k] * xq[t, k]
// with fp32 sums and one rounding to the output type.
//
// quantize_rows_kernel encodes x; linear_stream_kernel (up to 64 tokens) or
// linear_pair_kernel multiplies, on the block-scaled tensor cores (tcgen05.mma
// kind::mxf4, both scales applied by the MMA, K = 64 an instruction).
//
// linear_stream_kernel: the weights are the MMA's M side (128 rows a CTA) and the tokens
// its N side (NT = 16 .. 128 columns), so one token costs no more tensor work than
// sixteen and the weight stream, which bounds small batches, is read once per
// token tile.  A stage is 256 k: one 128-byte row of packed codes per weight row and
// token, two TMA boxes in the 128-byte swizzle.  Few weight tiles do not fill the
// GPU, so a cluster of S CTAs splits K: each multiplies its range of stages,
// leaves its fp32 partial tile in shared memory, and the CTAs of the cluster
// each add a share of the tile over the S partials (distributed shared
// memory, in rank order: the result does not depend on timing).
// 192 threads, two to four CTAs per SM, so that one CTA's start and end overlap the
// others' stream:
//   * producer warp: the TMA loads.  The weights of the first stages are asked for
//     before the quantisation kernel has finished (programmatic launch);
//   * MMA warp: one thread;
//   * 4 warps, one per tensor-memory lane quadrant: write each stage's scale
//     factors into tensor memory (layout as in ffn_mxfp4act.cu), then drain the
//     accumulator.  For up to 16 tokens whose CTAs all run at once they also encode
//     the stage's part of x themselves (FUSED): one launch, 3 us less than two.
// Bound by HBM for wide outputs (16 x 100003 x 4096: 42 us with the encoding, 224 MB, 5.3
// TB/s), by its chain of latencies below (16 x 4096 x 4096: 8.4 us; 64 x 4096 x 4096: 10.8
// with the encoding).
// Every wait is bounded (see mbar_wait).
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "mxf4.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kBK = 256;  // k per stage: one 128-byte row of packed codes
constexpr int kRowBytes = kBK / 2;
constexpr int kMRows = 128;
constexpr int kABytes = kMRows * kRowBytes;

// ------------------------------------------------------------ quantisation

// Eight values of a row from `p`: one or two 16-byte loads, or element by
// element where the row's start is not 16-byte aligned.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* p, float* v) {
    if (F32) {
        const float* f = reinterpret_cast<const float*>(p);
        if (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(f));
            const float4 b = __ldg(reinterpret_cast<const float4*>(f) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldg(f + i);
        }
    } else if (VEC) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)__ldg(h + i) << 16);
    }
}

// The MXFP4 encoding of a 32-value block held by four neighbouring lanes, eight
// values each: this lane's four code bytes, and the block's scale byte in all
// four.  The rule of moe_quantize_mxfp4, except that a block that holds an
// infinity or a NaN gets scale byte 255 (E8M0's NaN) and codes 0, so that it
// decodes to NaN and the MMA carries it into every output of its token.
__device__ __forceinline__ uint32_t quantize8(const float v[8], uint32_t& sbyte) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    if (mx >= 0x7F800000u) {
        sbyte = 255u;
        return 0u;
    }
    sbyte = mx_scale_byte(__uint_as_float(mx));
    return e2m1x8(v, mx_inv_scale(sbyte));
}

// The same for eight bf16 values (two a word, the first in the low half): the largest magnitude
// from the bit patterns, two at a time, a fifth of the instructions less.
__device__ __forceinline__ uint32_t quantize8(const uint4& w, uint32_t& sbyte) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t m = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu), __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t mx = max(m << 16, m & 0xFFFF0000u);  // fp32 bits
    if (mx >= 0x7F800000u) {
        sbyte = 255u;
        return 0u;
    }
    sbyte = mx_scale_byte(__uint_as_float(mx));
    const float v[8] = {bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1]),
                        bf16_lo(u[2]), bf16_hi(u[2]), bf16_lo(u[3]), bf16_hi(u[3])};
    return e2m1x8(v, mx_inv_scale(sbyte));
}

// Where the eight scale bytes of row r, stage st (256 k) lie for the pair kernel:
// blocks of (128 rows, one stage), a kilobyte each.
__device__ __forceinline__ size_t sf_block(int r, int st, int nk) {
    return ((size_t)(r >> 7) * nk + st) * 1024 + (size_t)(r & 127) * 8;
}

struct QuantArgs {
    const void* x;       // [T] rows of K values, ldx elements apart
    long long ldx;
    int T, K;
    uint8_t* codes;      // [T][K/2]
    uint8_t* scales;     // [T][pitch] (K/32 bytes, zeros up to the next multiple of 8), or
    int pitch;           // 0: in sf_block's layout, and
    const uint8_t* ws;   // the weights' scale bytes [N][K/32] in it too
    uint8_t* wsb;
    int N;
    int xblocks;         // thread blocks that encode x; the others lay ws out
    int parts;           // warps that share a row of x
};

// One warp takes up to kQuantAhead times 256 values of a row, eight per lane: every load
// and store is coalesced, all loads are in flight before the first value is used.  For long
// prompts it reads 2 bytes and writes 17/32 a value: 8192 x 4096 in 14.4 us, 5.9 TB/s (20 us
// when the magnitudes were taken value by value: the instructions bound it); for short
// ones the launch is its time.  The weights' scales (1/16 of their codes' bytes) are laid
// out for linear_pair_kernel by further blocks of the same launch: two stages of a row per
// thread, neighbouring rows in neighbouring threads.
constexpr int kQuantAhead = 4;

template <bool F32, bool VEC>
__global__ void __launch_bounds__(256, F32 || !VEC ? 5 : 8) quantize_rows_kernel(const QuantArgs a) {
    pdl_begin();
    if ((int)blockIdx.x >= a.xblocks) {
        const int KG = a.K / 32, nk = (a.K + kBK - 1) / kBK, pairs = (nk + 1) / 2;
        const bool vec = KG % 16 == 0 && ((uintptr_t)a.ws & 15) == 0;
        const uint32_t items = (uint32_t)a.N * (uint32_t)pairs;  // (at most 2^24 x 2^7)
        for (uint32_t it = ((uint32_t)blockIdx.x - (uint32_t)a.xblocks) * blockDim.x + threadIdx.x; it < items;
             it += (gridDim.x - (uint32_t)a.xblocks) * blockDim.x) {
            const int p2 = (int)(it / (uint32_t)a.N), r = (int)(it - (uint32_t)p2 * (uint32_t)a.N);
            const uint8_t* p = a.ws + (size_t)r * KG + 16 * p2;
            uint32_t w[4] = {0, 0, 0, 0};
            if (vec) {  // K is a multiple of 512: whole pairs
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (16 * p2 + j < KG) w[j >> 2] |= (uint32_t)__ldg(p + j) << (8 * (j & 3));
            }
            *reinterpret_cast<uint2*>(a.wsb + sf_block(r, 2 * p2, nk)) = make_uint2(w[0], w[1]);
            if (2 * p2 + 1 < nk) *reinterpret_cast<uint2*>(a.wsb + sf_block(r, 2 * p2 + 1, nk)) = make_uint2(w[2], w[3]);
        }
        pdl_end();
        return;
    }
    const int lane = threadIdx.x & 31;
    const int segs = (a.K + kBK - 1) / kBK, chunk = (segs + a.parts - 1) / a.parts;
    const uint32_t it = blockIdx.x * 8u + (threadIdx.x >> 5);  // (rows x parts is below 2^31: x fits in memory)
    const int t = (int)(it / (uint32_t)a.parts), s0 = (int)(it - (uint32_t)t * (uint32_t)a.parts) * chunk;
    if (t < a.T && s0 < segs) {
        constexpr int kSize = F32 ? 4 : 2;
        const int k0 = s0 * kBK + lane * 8, n = min(chunk, segs - s0);
        const char* src = reinterpret_cast<const char*>(a.x) + ((size_t)t * a.ldx + k0) * kSize;
        uint8_t* codes = a.codes + (size_t)t * (a.K / 2) + k0 / 2;
        uint8_t* scales = a.scales + (a.pitch ? (size_t)t * a.pitch + s0 * 8 : sf_block(t, s0, segs)) + (lane >> 2);
        const int next = a.pitch ? 8 : 1024;
        using Values = std::conditional_t<F32 || !VEC, float[8], uint4>;
        Values v[kQuantAhead];
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            const bool in = u < n && k0 + u * kBK < a.K;
            if constexpr (!F32 && VEC) {
                v[u] = in ? __ldg(reinterpret_cast<const uint4*>(src + u * kBK * kSize)) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
                if (in) load8<F32, VEC>(src + u * kBK * kSize, v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            if (u >= n) break;
            uint32_t sb;
            const uint32_t c = quantize8(v[u], sb);
            if (k0 + u * kBK < a.K) *reinterpret_cast<uint32_t*>(codes + u * (kBK / 2)) = c;
            if ((lane & 3) == 0) scales[u * next] = (uint8_t)sb;  // (0 past K)
        }
    }
    pdl_end();
}

// ----------------------------------------------------------------- product

struct StreamArgs {
    const void* x;           // FUSED: [T] rows, ldx elements apart
    long long ldx;
    int x_f32, x_vec;
    const uint8_t* scales;   // [N][K/32]
    const uint8_t* xscales;  // [T][xpitch]
    int xpitch;
    const void* residual;    // [T] rows, ldr elements apart, of the output's type; or null
    void* out;               // [T] rows, ldo elements apart
    long long ldr, ldo;
    int T, N, K;
    int out_f32;
};

// out[t][n] = residual + v, rounded once
__device__ __forceinline__ void store_out(const StreamArgs& a, int t, int n, float v) {
    if (a.out_f32) {
        if (a.residual) v += reinterpret_cast<const float*>(a.residual)[(size_t)t * a.ldr + n];
        reinterpret_cast<float*>(a.out)[(size_t)t * a.ldo + n] = v;
    } else {
        if (a.residual)
            v += __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(a.residual)[(size_t)t * a.ldr + n] << 16);
        reinterpret_cast<uint16_t*>(a.out)[(size_t)t * a.ldo + n] = f32_to_bf16_bits(v);
    }
}

StreamArgs stream_args(const LinearMxfp4& p) {
    StreamArgs a = {};
    a.scales = p.scales;
    a.residual = p.residual;
    a.out = p.out;
    a.ldr = p.ldr;
    a.ldo = p.ldo;
    a.T = p.T;
    a.N = p.N;
    a.K = p.K;
    a.out_f32 = p.out_f32;
    return a;
}

constexpr int kStreamThreads = 192;

template <int NT, bool FUSED>
struct StreamLayout {
    static constexpr int kBBytes = NT * kRowBytes;
    static constexpr int kStage = kABytes + kBBytes;  // a multiple of 1024
    // CTAs per SM: four short ones for the fewest tokens, whose CTAs only pass weights on
    // (16 x 100003 x 4096: 42 us against 46 with two)
    static constexpr int kPerSm = NT == 16 && !FUSED ? 4 : 2;
    static constexpr int kFit = (kPerSm == 4 ? 54 : 110) * 1024 / kStage;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kBar = kStages * kStage;
    static constexpr int kXsf = kBar + 256;           // FUSED: a stage's scale bytes of 16 tokens, two stages
    static constexpr int kTotal = kXsf + 256 + 1024;  // + barriers, alignment slack
    static_assert(kStages >= 3, "ring depth");
    static_assert(NT * kMRows * 4 <= kBar, "the partial tile takes the ring's place");
    static constexpr int kNJ = (NT + 31) / 32;        // scale columns of the tokens
    // tensor memory: the accumulator, then per stage 32 columns of scale
    // factors, each 128-k chunk's block on a multiple of 8 columns (weights at
    // +0 and +8, tokens at +16 and +24)
    static constexpr int kSfCols = 32;
    static constexpr int kSfCol0 = NT < 32 ? 32 : NT;
    static constexpr int kCols = 512 / kPerSm;
    static_assert(kSfCol0 + kStages * kSfCols <= kCols, "tensor memory, a CTA's share");
};

template <int NT, bool FUSED>
__global__ void __launch_bounds__(kStreamThreads, (StreamLayout<NT, FUSED>::kPerSm))
    linear_stream_kernel(const StreamArgs a, const int splits,
                         const __grid_constant__ CUtensorMap w_map,
                         const __grid_constant__ CUtensorMap x_map) {
    using L = StreamLayout<NT, FUSED>;
    constexpr int kStages = L::kStages, kNJ = L::kNJ;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* tma_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* sf_full = tma_full + kStages;
    uint64_t* stage_free = sf_full + kStages;
    uint64_t* acc_full = stage_free + kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)blockIdx.x % splits;  // the cluster is `splits` neighbours in x
    const int n0 = (int)blockIdx.x / splits * kMRows, t0 = (int)blockIdx.y * NT;
    const int KG = a.K / 32;
    const int nk = (a.K + kBK - 1) / kBK;
    const int st0 = (int)((long long)nk * rank / splits), st1 = (int)((long long)nk * (rank + 1) / splits);

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&tma_full[s], 1);
            mbar_init(&sf_full[s], 4);
            mbar_init(&stage_free[s], 1);
        }
        mbar_init(acc_full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<false>(tmem_slot, L::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (FUSED: the kernel before this one may have written anything that is read here)
    if (FUSED) pdl_begin();

    if (warp == 0) {
        // ------------------------------------------------------- producer
        if (lane == 0) {
            auto load_w = [&](int i) {
                const int s = i % kStages;
                mbar_arrive_expect_tx(&tma_full[s], (uint32_t)(FUSED ? kABytes : L::kStage));
                tma_load_2d(smem_u32(smem + s * L::kStage), &w_map, (st0 + i) * kRowBytes, n0, &tma_full[s]);
            };
            auto load_x = [&](int i) {
                const int s = i % kStages;
                tma_load_2d(smem_u32(smem + s * L::kStage + kABytes), &x_map, (st0 + i) * kRowBytes, t0,
                            &tma_full[s]);
            };
            const int n = st1 - st0, first = min(n, kStages);
            for (int i = 0; i < first; ++i) load_w(i);
            if (!FUSED) {
                pdl_begin();
                for (int i = 0; i < first; ++i) load_x(i);
            }
            int i = first;
            for (; i < n; ++i) {
                if (!mbar_wait(&stage_free[i % kStages], ((i / kStages) - 1) & 1)) break;
                load_w(i);
                if (!FUSED) load_x(i);
            }
            // wait (bounded) until the last loads landed before the CTA can exit
            for (int d = 0; d < kStages && d < i; ++d) {
                const int u = i - 1 - d;
                if (!mbar_wait(&tma_full[u % kStages], (u / kStages) & 1)) break;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id0 = idesc_mxf4(kMRows, NT, 0), id2 = idesc_mxf4(kMRows, NT, 2);
            for (int i = 0; i < st1 - st0; ++i) {
                const int s = i % kStages;
                const uint32_t par = (i / kStages) & 1;
                if (!mbar_wait(&tma_full[s], par) || !mbar_wait(&sf_full[s], par)) break;
                tc_fence_after();
                const uint64_t ad = sdesc_sw128(smem_u32(smem + s * L::kStage));
                const uint64_t bd = sdesc_sw128(smem_u32(smem + s * L::kStage + kABytes));
                const uint32_t sf = tmem + (uint32_t)(L::kSfCol0 + s * L::kSfCols);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // K = 64 each: +32 bytes in the swizzle atom
                    mma_mxf4(tmem, ad + 2u * kk, bd + 2u * kk, (kk & 1) ? id2 : id0, sf + 8u * (kk >> 1),
                             sf + 16u + 8u * (kk >> 1), (i | kk) != 0 ? 1u : 0u);
                mma_commit(&stage_free[s]);
            }
            mma_commit(acc_full);  // every MMA issued has completed when this arrives
            mbar_wait(acc_full, 0);
        }
    } else {
        // ------------------------------------- scale factors, then the drain
        const int quad = warp & 3;
        const int wrow = n0 + 32 * quad + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
        const uint8_t* sa = wrow < a.N ? a.scales + (size_t)wrow * KG : nullptr;
        const bool vec = KG % 8 == 0 && ((uintptr_t)a.scales & 7) == 0;
        if (sa)  // this row's scale bytes of the CTA's range, on their way into L2
            for (int g = 8 * st0; g < min(8 * st1, KG); g += 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(sa + g));
        auto load_sa = [&](int st) {
            uint2 r = make_uint2(0, 0);
            if (!sa) return r;
            if (vec) return __ldg(reinterpret_cast<const uint2*>(sa + 8 * st));
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * st + j < KG) w[j >> 2] |= (uint32_t)__ldg(sa + 8 * st + j) << (8 * (j & 3));
            return make_uint2(w[0], w[1]);
        };
        uint2 an = load_sa(st0);
        if (!FUSED) pdl_begin();
        const uint8_t* sb[kNJ];
#pragma unroll
        for (int j = 0; j < kNJ; ++j) {
            const int t = t0 + 32 * j + lane;
            sb[j] = (!FUSED && 32 * j + lane < NT && t < a.T) ? a.xscales + (size_t)t * a.xpitch : nullptr;
        }
        uint2 bn[kNJ];
        auto load_sb = [&](int st) {
#pragma unroll
            for (int j = 0; j < kNJ; ++j)
                bn[j] = sb[j] ? *reinterpret_cast<const uint2*>(sb[j] + 8 * st) : make_uint2(0, 0);
        };
        load_sb(st0);
        // FUSED: this lane's eight values of tokens quad, quad + 4, ... of stage st, the
        // four loads together
        float xv[FUSED ? 4 : 1][8];
        auto load_xv = [&](int st) {
            const int k = st * kBK + 8 * lane, esize = a.x_f32 ? 4 : 2;
            auto each = [&](auto load) {
#pragma unroll
                for (int u = 0; u < (FUSED ? 4 : 0); ++u) {
                    const int t = quad + 4 * u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) xv[u][i] = 0.0f;
                    if (t < a.T && k < a.K) load(reinterpret_cast<const char*>(a.x) + ((size_t)t * a.ldx + k) * esize, xv[u]);
                }
            };
            if (a.x_f32) {
                if (a.x_vec)
                    each([](const void* p, float* v) { load8<true, true>(p, v); });
                else
                    each([](const void* p, float* v) { load8<true, false>(p, v); });
            } else if (a.x_vec) {
                each([](const void* p, float* v) { load8<false, true>(p, v); });
            } else {
                each([](const void* p, float* v) { load8<false, false>(p, v); });
            }
        };
        if (FUSED) load_xv(st0);
        bool ok = true;
        for (int i = 0; i < st1 - st0 && ok; ++i) {
            const int s = i % kStages;
            const uint32_t av[2] = {an.x, an.y};
            uint32_t bv[2][kNJ];
#pragma unroll
            for (int j = 0; j < kNJ; ++j) bv[0][j] = bn[j].x, bv[1][j] = bn[j].y;
            if (i + 1 < st1 - st0) {
                an = load_sa(st0 + i + 1);
                load_sb(st0 + i + 1);
            }
            bool free = i < kStages || mbar_wait_warp(&stage_free[s], ((i / kStages) - 1) & 1);
            if (FUSED) {
                // encode into the stage's rows (128-byte swizzle); the four warps meet
                // before the scale bytes are read back
                if (free) {
                    uint8_t* rows = smem + s * L::kStage + kABytes;
                    uint8_t* xsf = smem + L::kXsf + (i & 1) * 128;
#pragma unroll
                    for (int u = 0; u < (FUSED ? 4 : 0); ++u) {
                        const int t = quad + 4 * u;
                        uint32_t sbyte;
                        const uint32_t c = quantize8(xv[u], sbyte);
                        *reinterpret_cast<uint32_t*>(rows + t * kRowBytes + (((lane >> 2) ^ (t & 7)) << 4) + (lane & 3) * 4) = c;
                        if ((lane & 3) == 0) xsf[t * 8 + (lane >> 2)] = (uint8_t)sbyte;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                free = all_at_barrier(free, 1, 128);
                if (free) {
                    const uint2 v = lane < 16 ? *reinterpret_cast<const uint2*>(smem + L::kXsf + (i & 1) * 128 + lane * 8)
                                              : make_uint2(0, 0);
                    bv[0][0] = v.x, bv[1][0] = v.y;
                    if (i + 1 < st1 - st0) load_xv(st0 + i + 1);
                }
            }
            if (!free) {
                ok = false;
                break;
            }
            tc_fence_after();  // after the MMAs that last read these columns
            const uint32_t col = lane_base + (uint32_t)(L::kSfCol0 + s * L::kSfCols);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tmem_st_cols<1>(col + 8u * c + (uint32_t)quad, &av[c]);
                tmem_st_cols<kNJ>(col + 16u + 8u * c, bv[c]);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sf_full[s]);
        }
        if (ok && mbar_wait_warp(acc_full, 0)) {
            tc_fence_after();
            float* part = reinterpret_cast<float*>(smem);  // [NT][128], over the ring: its loads are used
            const int ncol = min(NT, a.T - t0);
#pragma unroll 1
            for (int c0 = 0; c0 < ncol; c0 += 16) {
                uint32_t v[16];
                tmem_ld16_nowait(lane_base + (uint32_t)c0, v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (c0 + i >= ncol) break;
                    if (splits > 1)
                        part[(c0 + i) * kMRows + 32 * quad + lane] = __uint_as_float(v[i]);
                    else if (wrow < a.N)
                        store_out(a, t0 + c0 + i, wrow, __uint_as_float(v[i]));
                }
            }
            tc_fence_before();
        }
    }

    __syncwarp();
    if (splits > 1) {
        // the partial tiles of the cluster's CTAs, each element added in rank
        // order by one thread
        cluster_sync_all();
        const int total = min(NT, a.T - t0) * kMRows;
        const uint32_t base = smem_u32(smem);
        uint32_t peer[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer[r]) : "r"(base), "r"(r < splits ? r : 0));
        for (int i = rank * kStreamThreads + tid; i < total; i += splits * kStreamThreads) {
            float p[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < splits)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[r]) : "r"(peer[r] + 4u * (uint32_t)i));
            float v = p[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < splits) v += p[r];
            const int n = n0 + (i & (kMRows - 1));
            if (n < a.N) store_out(a, t0 + i / kMRows, n, v);
        }
        cluster_sync_all();  // no CTA leaves while another reads its partial tile
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<false>(tmem, L::kCols);
    }
    pdl_end();
}

// ------------------------------------------------------ product, large batches

// Long prompts are bound by the tensor cores and by the shared memory that feeds them,
// so tokens are the MMA's M side in pairs of CTAs (cta_group::2: 256 tokens x TN weight
// rows, each CTA loading its 128 tokens and half of the weight rows), persistent, in an
// order that keeps a weight tile on neighbouring pairs (squarer groups of tiles took the
// same time).  A stage (256 k) also brings the scale bytes of its rows (sf_block), which
// four warps, one per tensor-memory lane quadrant, write into tensor memory; letting the
// MMA thread copy them there (tcgen05.cp, six copies a stage) held the products up by a
// third, also when issued a stage ahead; eight such warps changed nothing.
// Eight epilogue warps read the accumulator into registers, free it, and store through
// shared memory in full lines.
//
// An MMA of K = 64 takes about 122 clocks for TN = 256 and hardly fewer for 128 or 192,
// so TN = 256 does most per clock, although tensor memory then has room for one
// accumulator only and a tile waits about 800 clocks while the last one is read (192 with
// two accumulators: 144 us where 256 took 118).  8192 x 8192 x 4096: 88 us, 6.2 PFLOP/s;
// 9700 clocks for a tile's 64 MMAs (8000 without the loads into shared memory), 800 between
// tiles, 14 tiles for most pairs and 13 for the others.  Shared memory is what bounds it: each
// of a tile's 16 stages writes 36 KB there and its MMAs read 32 KB, at 128 bytes a clock
// 8700 of the 9700 clocks.  Fewer stages (3 or 4 for 5) or
// half of the loads changed little; output by TMA instead of stores cost 8%: its reads
// come in a burst that the operands' loads wait for.
struct PairArgs {
    const uint8_t* sfa;   // x's scale bytes: ceil(T / 256) * 2 rows of blocks
    const uint8_t* sfb;   // the weights': ceil(N / 256) * 2
    StreamArgs o;         // output, residual, sizes
};

// Four warpgroups: the scale warps; the producer, the MMA and two idle warps; two of epilogue
// warps, which take registers from the others so that a warp holds its 128 columns.
constexpr int kPairThreads = 512;
constexpr int kPairProducer = 4, kPairMma = 5, kPairEpiWarp0 = 8;
constexpr int kPairRegs = 56, kPairEpiRegs = 192;
static_assert(256 * (kPairRegs + kPairEpiRegs) <= kPairThreads * 128, "registers of the launch");

template <int TN>
struct PairLayout {
    static constexpr int kBRows = TN / 2;                     // weight rows per CTA
    static constexpr int kBBytes = kBRows * kRowBytes;
    static constexpr int kSfaBytes = 1024;                    // 128 tokens x 256 k
    static constexpr int kSfbBytes = TN / 128 * 1024;         // all TN weight rows
    static constexpr int kSf = kABytes + kBBytes;
    static constexpr int kStage = kSf + kSfaBytes + kSfbBytes;
    static_assert(kStage % 1024 == 0, "alignment");
    // per epilogue warp: 32 rows x 128 bytes, 16-byte part q of row r at q ^ (r & 7)
    static constexpr int kStgWarp = 32 * 128;
    static constexpr int kFit = (232448 - 1024 - 256 - 8 * kStgWarp) / kStage;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kStg = kStages * kStage;
    static constexpr int kBar = kStg + 8 * kStgWarp;
    static constexpr int kTotal = kBar + 256 + 1024;
    static_assert(kStages >= 4 && kTotal <= 232448, "shared memory");
    // tensor memory: accumulators, then 32 columns of scale factors per stage (tokens at
    // +0 and +8 for the two 128-k chunks, weights at +16 and +24)
    static constexpr int kAccBufs = TN == 128 ? 2 : 1;
    static constexpr int kSfCol0 = kAccBufs * TN;
    static_assert(kSfCol0 + kStages * 32 <= 512, "tensor memory");
};

// ES: bytes of an output value; RES: a residual; VEC: the output's and the residual's rows
// start on 16 bytes.  (One kernel with all the forms spilled the accumulator: 111 us where
// these take 102.  Of these only the 256-wide ones with a residual spill, up to 52 bytes.)
template <int TN, int ES, bool RES, bool VEC>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const PairArgs a, const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap w_map) {
    using L = PairLayout<TN>;
    constexpr int kStages = L::kStages, kAccBufs = L::kAccBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* tma_full = reinterpret_cast<uint64_t*>(smem + L::kBar);  // this CTA's loads
    uint64_t* sf_full = tma_full + kStages;     // even CTA: loads and scale factors of both
    uint64_t* stage_free = sf_full + kStages;
    uint64_t* acc_full = stage_free + kStages;  // [2]
    uint64_t* acc_free = acc_full + 2;          // [2], even CTA: drained by both
    uint64_t* drain = acc_free + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x & 1u), pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int T = a.o.T, N = a.o.N;
    const int mts = (T + 255) / 256, nts = (N + TN - 1) / TN, tiles = mts * nts;
    const int nk = (a.o.K + kBK - 1) / kBK;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&tma_full[s], 1);
            mbar_init(&sf_full[s], 8);
            mbar_init(&stage_free[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 16);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPairMma) tmem_alloc<true>(tmem_slot, 512);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_begin();

    if (warp >= kPairEpiWarp0) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairEpiRegs));
        // -------------------------------------------------------- epilogue
        constexpr int kCols = TN / 2;  // columns per warp
        const int quad = warp & 3, half = (warp - kPairEpiWarp0) >> 2;
        uint8_t* stg = smem + L::kStg + (warp - kPairEpiWarp0) * L::kStgWarp;
        auto part = [&](int r, int q) { return stg + r * 128 + ((q ^ (r & 7)) << 4); };
        // The columns go through shared memory 128 bytes a row at a time (so many passes a
        // tile), out in full lines; bf16 is rounded before it is staged (half the traffic in
        // shared memory, which the MMA's operands share).  The residual (RES) comes in the
        // same way, its loads one pass ahead, asked for while the tile before is multiplied:
        // 8192 x 8192 x 4096 with one takes 121 us in bf16 and 161 in fp32 (102 and 120
        // without; 174 and 335 when its loads stood between the accumulator and the stores).
        // Without VEC the output is written element by element, from fp32 (and store_out
        // adds the residual): 173 us in both types, 718 and 869 with a residual, whose
        // elements come one by one between the accumulator and the stores; 128 x 100003 x 4096
        // in fp32 86 us, where 100000 columns take 67.
        constexpr int kBox = 128 / ES;  // columns a pass
        const int lr = lane >> 3, lc = (lane & 7) * (16 / ES);  // coalesced: rows lr + 4 i, columns lc ..
        uint4 rr[RES ? 8 : 1];
        auto load = [&](int t, int n) {
#pragma unroll
            for (int i = 0; i < (RES ? 8 : 0); ++i) {
                rr[i] = make_uint4(0, 0, 0, 0);
                const int row = t + lr + 4 * i, col = n + lc;
                if (row >= T || col >= N) continue;
                const char* src = reinterpret_cast<const char*>(a.o.residual) + ((size_t)row * a.o.ldr + col) * ES;
                if (col + 16 / ES <= N) {
                    rr[i] = *reinterpret_cast<const uint4*>(src);
                } else {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 16 / ES; ++k)
                        if (col + k < N) {
                            if (ES == 4)
                                w[k & 3] = reinterpret_cast<const uint32_t*>(src)[k];
                            else
                                w[k >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(src)[k] << (16 * (k & 1));
                        }
                    rr[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        };
        auto t_of = [&](int tile) { return tile % mts * 256 + rank * 128 + quad * 32; };
        auto n_of = [&](int tile) { return tile / mts * TN + half * kCols; };
        if (pair < tiles) load(t_of(pair), n_of(pair));
        uint32_t it = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++it) {
            const int t = t_of(tile), n = n_of(tile);
            const uint32_t b = it % kAccBufs;
            if (!mbar_wait_warp(&acc_full[b], (it / kAccBufs) & 1)) break;
            tc_fence_after();
            uint32_t v[kCols];
            const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + b * TN + (uint32_t)(half * kCols);
#pragma unroll
            for (int c = 0; c < kCols; c += 16) tmem_ld16_nowait(taddr + c, v + c);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {  // drained: the next tile may use it
                if (rank == 0)
                    mbar_arrive(&acc_free[b]);
                else
                    mbar_arrive_remote(&acc_free[b], 0);
            }
#pragma unroll
            for (int c0 = 0; c0 < kCols; c0 += kBox) {
                if (t >= T || n + c0 >= N) break;
                if (RES) {
#pragma unroll
                    for (int i = 0; i < (RES ? 8 : 0); ++i) *reinterpret_cast<uint4*>(part(lr + 4 * i, lane & 7)) = rr[i];
                    __syncwarp();
                    if (c0 + kBox < kCols) load(t, n + c0 + kBox);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint4* d = reinterpret_cast<uint4*>(part(lane, q));
                    uint32_t o[4], p[4] = {0, 0, 0, 0};
                    if (RES) {
                        const uint4 x = *d;
                        p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (ES == 4) {
                            const float x = __uint_as_float(v[c0 + 4 * q + i]);
                            o[i] = __float_as_uint(RES ? x + __uint_as_float(p[i]) : x);
                        } else {
                            float lo = __uint_as_float(v[c0 + 8 * q + 2 * i]), hi = __uint_as_float(v[c0 + 8 * q + 2 * i + 1]);
                            if (RES) lo += bf16_lo(p[i]), hi += bf16_hi(p[i]);
                            o[i] = f32x2_to_bf16x2_bits(lo, hi);
                        }
                    }
                    *d = make_uint4(o[0], o[1], o[2], o[3]);
                }
                __syncwarp();
                if (VEC) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = t + lr + 4 * i, col = n + c0 + lc;
                        if (row >= T) break;
                        const uint8_t* src = part(lr + 4 * i, lane & 7);
                        char* dst = reinterpret_cast<char*>(a.o.out) + ((size_t)row * a.o.ldo + col) * ES;
                        if (col + 16 / ES <= N)
                            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
                        else
                            for (int k = 0; k < (N - col) * ES; k += 2)
                                *reinterpret_cast<uint16_t*>(dst + k) = *reinterpret_cast<const uint16_t*>(src + k);
                    }
                } else {
                    for (int r = 0; r < 32 && t + r < T; ++r)
                        if (n + c0 + lane < N)
                            store_out(a.o, t + r, n + c0 + lane,
                                      reinterpret_cast<const float*>(part(r, lane >> 2))[lane & 3]);
                }
                __syncwarp();
            }
            if (tile + pairs < tiles) load(t_of(tile + pairs), n_of(tile + pairs));
        }
        // The kernel's end, as below, but apart from the other roles': where they met at one
        // barrier, values that only those need stayed in these warps' registers over the loop
        // (36 bytes of spills; 8192 x 8192 x 4096: 112 us for 102).
        tc_fence_before();
        cluster_sync_all();
        pdl_end();
        return;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegs));
        if (warp == kPairProducer) {
            // ------------------------------------------------------- producer
            if (lane == 0) {
                uint32_t gs = 0;
                bool ok = true;
                for (int tile = pair; tile < tiles && ok; tile += pairs) {
                    const int nt = tile / mts, mt = tile - nt * mts;
                    const int arow = mt * 256 + rank * 128, brow = nt * TN + rank * L::kBRows;
                    const uint8_t* sfa = a.sfa + (size_t)(mt * 2 + rank) * nk * 1024;
                    const uint8_t* sfb = a.sfb + (size_t)nt * (TN / 128) * nk * 1024;
                    for (int st = 0; st < nk; ++st, ++gs) {
                        const int s = gs % kStages;
                        if (gs >= (uint32_t)kStages && !mbar_wait(&stage_free[s], ((gs / kStages) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        const uint32_t base = smem_u32(smem + s * L::kStage);
                        mbar_arrive_expect_tx(&tma_full[s], (uint32_t)L::kStage);
                        tma_load_2d(base, &x_map, st * kRowBytes, arow, &tma_full[s]);
                        tma_load_2d(base + kABytes, &w_map, st * kRowBytes, brow, &tma_full[s]);
                        bulk_copy_g2s(base + L::kSf, sfa + (size_t)st * 1024, 1024, &tma_full[s]);
#pragma unroll
                        for (int j = 0; j < TN / 128; ++j)
                            bulk_copy_g2s(base + L::kSf + L::kSfaBytes + j * 1024,
                                          sfb + ((size_t)j * nk + st) * 1024, 1024, &tma_full[s]);
                    }
                }
                // wait (bounded) until the last loads landed before the CTA can exit
                for (int d = 0; d < kStages && d < (int)gs; ++d) {
                    const uint32_t u = gs - 1 - d;
                    if (!mbar_wait(&tma_full[u % kStages], (u / kStages) & 1)) break;
                }
            }
        } else if (warp == kPairMma) {
            if (lane == 0 && rank == 0) {
                // -------------------------------------------------------- MMA
                constexpr uint32_t id0 = idesc_mxf4(256, TN, 0), id2 = idesc_mxf4(256, TN, 2);
                uint32_t gs = 0, it = 0;
                bool ok = true;
                for (int tile = pair; tile < tiles && ok; tile += pairs, ++it) {
                    const uint32_t b = it % kAccBufs;
                    if (it >= (uint32_t)kAccBufs && !mbar_wait(&acc_free[b], ((it / kAccBufs) - 1) & 1)) break;
                    tc_fence_after();
                    const uint32_t d_tmem = tmem + b * TN;
                    for (int st = 0; st < nk; ++st, ++gs) {
                        const int s = gs % kStages;
                        // (arrived at once the stage's loads and scale factors are there, by both CTAs)
                        if (!mbar_wait(&sf_full[s], (gs / kStages) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t base = smem_u32(smem + s * L::kStage);
                        const uint32_t sf = tmem + (uint32_t)(L::kSfCol0 + s * 32);
                        const uint64_t ad = sdesc_sw128(base), bd = sdesc_sw128(base + kABytes);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // K = 64 each: +32 bytes in the swizzle atom
                            mma_mxf4_pair(d_tmem, ad + 2u * kk, bd + 2u * kk, (kk & 1) ? id2 : id0, sf + 8u * (kk >> 1),
                                          sf + 16u + 8u * (kk >> 1), (st | kk) != 0 ? 1u : 0u);
                        mma_commit_pair(&stage_free[s]);
                    }
                    if (ok) mma_commit_pair(&acc_full[b]);
                }
                mma_commit_pair(drain);  // every MMA issued has completed when this arrives
                mbar_wait(drain, 0);
            } else if (lane == 0) {
                mbar_wait(drain, 0);  // odd CTA: the pair's MMAs and their commits to it are done
            }
        } else if (warp < 4) {
            // -------------------------------------------------- scale factors
            // token r's at lane r, column base + r / 32; weight row n's at lane 32 q + n % 32,
            // column base + n / 32, in every quadrant q
            constexpr int NJ = TN / 32;
            const int quad = warp & 3;
            const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)L::kSfCol0;
            uint32_t gs = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                for (int st = 0; st < nk; ++st, ++gs) {
                    const int s = gs % kStages;
                    // the stage is filled again only after the MMAs that read these columns
                    if (!mbar_wait_warp(&tma_full[s], (gs / kStages) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sf = smem_u32(smem + s * L::kStage + L::kSf) + 8 * lane;
                    const uint2 av = lds64(sf + 256 * quad);
                    uint32_t b0[NJ], b1[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const uint2 v = lds64(sf + L::kSfaBytes + 256 * j);
                        b0[j] = v.x, b1[j] = v.y;
                    }
                    tc_fence_after();
                    const uint32_t col = lane_base + (uint32_t)(s * 32);
                    tmem_st_cols<1>(col + (uint32_t)quad, &av.x);
                    tmem_st_cols<1>(col + 8u + (uint32_t)quad, &av.y);
                    tmem_st_cols<NJ>(col + 16u, b0);
                    tmem_st_cols<NJ>(col + 24u, b1);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(&sf_full[s]);
                        else
                            mbar_arrive_remote(&sf_full[s], 0);
                    }
                }
            }
        }
    }

    tc_fence_before();
    // neither CTA releases its memory while the other may still arrive there or the
    // pair's MMAs may still run
    cluster_sync_all();
    if (warp == kPairMma) {
        tc_fence_after();
        tmem_dealloc<true>(tmem, 512);
    }
    pdl_end();
}

template <int TN, int ES, bool RES, bool VEC>
cudaError_t launch_pair_as(const LinearMxfp4& p, const uint8_t* xcodes, const uint8_t* sfa, const uint8_t* sfb,
                           cudaStream_t s) {
    const auto kernel = linear_pair_kernel<TN, ES, RES, VEC>;
    const size_t smem = PairLayout<TN>::kTotal;
    cudaError_t err = ensure_dynamic_smem((const void*)kernel, smem);
    if (err != cudaSuccess) return err;
    CUtensorMap w_map, x_map;
    err = encode_codes_map(&w_map, p.codes, p.K / 2, (uint64_t)p.N, kRowBytes, TN / 2);
    if (err != cudaSuccess) return err;
    err = encode_codes_map(&x_map, xcodes, p.K / 2, (uint64_t)p.T, kRowBytes, kMRows);
    if (err != cudaSuccess) return err;
    int pairs = 0;
    err = max_active_pairs((const void*)kernel, kPairThreads, smem, &pairs);
    if (err != cudaSuccess) return err;
    if (pairs < 1) return cudaErrorNotSupported;
    PairArgs a;
    a.sfa = sfa;
    a.sfb = sfb;
    a.o = stream_args(p);
    const long long tiles = (long long)((p.T + 255) / 256) * ((p.N + TN - 1) / TN);
    const int grid = 2 * (int)std::min<long long>(tiles, pairs);
    return launch_pdl_cluster(kernel, dim3((unsigned)grid), dim3(kPairThreads), smem, s, 2u, a, x_map, w_map);
}

template <int TN>
cudaError_t launch_pair(const LinearMxfp4& p, const uint8_t* xcodes, const uint8_t* sfa, const uint8_t* sfb,
                        cudaStream_t s) {
    const long long es = p.out_f32 ? 4 : 2;
    const bool vec = (uintptr_t)p.out % 16 == 0 && p.ldo * es % 16 == 0 &&
                     (!p.residual || ((uintptr_t)p.residual % 16 == 0 && p.ldr * es % 16 == 0));
    if (!vec) return launch_pair_as<TN, 4, false, false>(p, xcodes, sfa, sfb, s);
    if (p.out_f32)
        return p.residual ? launch_pair_as<TN, 4, true, true>(p, xcodes, sfa, sfb, s)
                          : launch_pair_as<TN, 4, false, true>(p, xcodes, sfa, sfb, s);
    return p.residual ? launch_pair_as<TN, 2, true, true>(p, xcodes, sfa, sfb, s)
                      : launch_pair_as<TN, 2, false, true>(p, xcodes, sfa, sfb, s);
}

int row_tiles(int N) { return (N + kMRows - 1) / kMRows; }

// Split K while the CTAs do not fill two per SM and every split has a stage.
int stream_splits(const LinearMxfp4& p, int NT) {
    const long long tiles = (long long)row_tiles(p.N) * ((p.T + NT - 1) / NT);
    const int nk = (p.K + kBK - 1) / kBK;
    int splits = 1;
    while (splits < 8 && 2 * splits <= nk && tiles * 2 * splits <= 2LL * num_sms()) splits *= 2;
    return splits;
}

template <int NT, bool FUSED>
cudaError_t launch_stream(const LinearMxfp4& p, const uint8_t* xcodes, const uint8_t* xscales, int xpitch,
                          cudaStream_t s) {
    const size_t smem = StreamLayout<NT, FUSED>::kTotal;
    cudaError_t err = ensure_dynamic_smem((const void*)linear_stream_kernel<NT, FUSED>, smem);
    if (err != cudaSuccess) return err;
    CUtensorMap w_map, x_map;
    err = encode_codes_map(&w_map, p.codes, p.K / 2, (uint64_t)p.N, kRowBytes, kMRows);
    if (err != cudaSuccess) return err;
    if (FUSED) {
        x_map = w_map;  // not read
    } else {
        err = encode_codes_map(&x_map, xcodes, p.K / 2, (uint64_t)p.T, kRowBytes, NT);
        if (err != cudaSuccess) return err;
    }
    StreamArgs a = stream_args(p);
    a.xscales = xscales;
    a.xpitch = xpitch;
    a.x = p.x;
    a.ldx = p.ldx;
    a.x_f32 = p.x_f32;
    a.x_vec = (uintptr_t)p.x % 16 == 0 && p.ldx * (p.x_f32 ? 4 : 2) % 16 == 0;
    const int tok_tiles = (p.T + NT - 1) / NT, splits = stream_splits(p, NT);
    return launch_pdl_cluster(linear_stream_kernel<NT, FUSED>, dim3((unsigned)row_tiles(p.N) * splits, (unsigned)tok_tiles),
                              dim3(kStreamThreads), smem, s, (unsigned)splits, a, splits, w_map, x_map);
}

template <bool F32>
cudaError_t launch_quantize_rows(QuantArgs a, cudaStream_t s) {
    // a warp takes kQuantAhead stages of a row, or fewer while the GPU has idle warps
    const int warps = num_sms() * 4 * 8, segs = (a.K + kBK - 1) / kBK;
    a.parts = std::max(std::min(segs, warps / std::max(a.T, 1)), (segs + kQuantAhead - 1) / kQuantAhead);
    a.xblocks = (int)(((long long)a.T * a.parts + 7) / 8);
    const long long witems = (long long)a.N * (((a.K + kBK - 1) / kBK + 1) / 2);
    const int wblocks = a.wsb ? (int)std::min<long long>((witems + 255) / 256, (long long)num_sms()) : 0;
    // 16-byte loads where every row starts on a 16-byte boundary
    const bool vec = ((uintptr_t)a.x % 16) == 0 && (a.ldx * (F32 ? 4 : 2)) % 16 == 0;
    return launch_pdl(vec ? quantize_rows_kernel<F32, true> : quantize_rows_kernel<F32, false>, dim3(a.xblocks + wblocks),
                      dim3(256), 0, s, a);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// bytes of a token's scale row: whole stages
int xscale_pitch(int K) { return (K + kBK - 1) / kBK * 8; }
// bytes of `rows` rows' scale blocks, whole tiles of 256 rows
size_t sf_bytes(int rows, int K) { return (size_t)((rows + 255) / 256) * 2 * (size_t)((K + kBK - 1) / kBK) * 1024; }

// Most stages of a CTA that encodes x itself: a stage's encoding takes about 1 us, which only
// the first loads hide (16 x 4096 x 4096, 2 stages: 8.4 us against 9.1 in two launches; 16 x
// 8192 x 4096, 4 stages: 12.8 against 10.6; 16 x 32000 x 4096, 16 stages: 39 against 17).
constexpr int kFusedStages = 2;

// Batches from here on go to the CTA pairs.
bool use_pairs(int T, int N) { return T > 64 && N >= 128; }

}  // namespace

size_t linear_mxfp4_workspace(int T, int N, int K) {
    const size_t codes = align256((size_t)T * (K / 2));
    return use_pairs(T, N) ? codes + sf_bytes(T, K) + sf_bytes(N, K) : codes + align256((size_t)T * xscale_pitch(K));
}

cudaError_t launch_linear_mxfp4(const LinearMxfp4& p, void* workspace, cudaStream_t s) {
    // few tokens, one wave of CTAs and a few stages each: they encode x themselves
    if (p.T <= 16) {
        const int splits = stream_splits(p, 16), nk = (p.K + kBK - 1) / kBK;
        if ((long long)row_tiles(p.N) * splits <= 2LL * num_sms() && (nk + splits - 1) / splits <= kFusedStages)
            return launch_stream<16, true>(p, nullptr, nullptr, 0, s);
    }
    QuantArgs q = {};
    q.x = p.x;
    q.ldx = p.ldx;
    q.T = p.T;
    q.K = p.K;
    q.codes = reinterpret_cast<uint8_t*>(workspace);
    q.scales = q.codes + align256((size_t)p.T * (p.K / 2));
    const bool pairs = use_pairs(p.T, p.N);
    if (pairs) {
        q.ws = p.scales;
        q.wsb = q.scales + sf_bytes(p.T, p.K);
        q.N = p.N;
    } else {
        q.pitch = xscale_pitch(p.K);
    }
    cudaError_t err = p.x_f32 ? launch_quantize_rows<true>(q, s) : launch_quantize_rows<false>(q, s);
    if (err != cudaSuccess) return err;
    if (pairs) {
        // half-width tiles where full ones would leave pairs idle: they take three quarters of
        // the time (turns of the pairs, half and full width, and us with the encoding: 512 x
        // 4096 x 4096 1 and 1, 11.9 and 13.4; 1536 x 4096 x 4096 3 and 2, 23.2 and 22.2;
        // 1024 x 16384 x 4096 7 and 4, 42.4 and 35.8)
        const long long mts = (p.T + 255) / 256, most = num_sms() / 2;
        const long long w256 = (mts * ((p.N + 255) / 256) + most - 1) / most, w128 = (mts * ((p.N + 127) / 128) + most - 1) / most;
        return 4 * w128 <= 5 * w256 ? launch_pair<128>(p, q.codes, q.scales, q.wsb, s)
                                    : launch_pair<256>(p, q.codes, q.scales, q.wsb, s);
    }
    // the narrowest token tile that holds the batch
    if (p.T <= 16) return launch_stream<16, false>(p, q.codes, q.scales, q.pitch, s);
    if (p.T <= 32) return launch_stream<32, false>(p, q.codes, q.scales, q.pitch, s);
    if (p.T <= 64) return launch_stream<64, false>(p, q.codes, q.scales, q.pitch, s);
    return launch_stream<128, false>(p, q.codes, q.scales, q.pitch, s);
}

cudaError_t read_device_error_linear(int* flag, int clear) {
    int wait = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&wait, g_device_error, sizeof(int));
    if (err != cudaSuccess) return err;
    *flag = wait ? 1 : 0;
    if (!clear) return cudaSuccess;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace moe
