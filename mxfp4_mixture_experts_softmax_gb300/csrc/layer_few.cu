// layer_few.cu -- the whole mixture-of-experts layer for up to 16 tokens in one
// cooperative launch: router product, softmax top-K, gate_up, SwiGLU, down and
// the weighted sum.
//
//   l = Wr x (fp32), ids = the K largest (ties to the lower id),
//   w = softmax(l)[ids], renormalised over the K if asked; the shared expert
//       (if any) with weight 1 or sigmoid(gate . x);
//   out = bf16(sum over e of w_e W2_e (silu(Wg_e x) * (Wu_e x)))
//
// What bounds it: the weights of the touched experts are read once (11 x 6.7
// MB for one token of a 4096/1024 layer with top-10 of 512 and a shared
// expert) and everything else is latency, so one grid of one CTA per SM keeps
// one TMA ring running through all phases and only two grid-wide barriers
// stand between them (logits complete; h complete).  While the CTAs meet at a
// barrier the ring fills with the next phase's weights: the shared expert's
// before the routing is known, W2's before h is.
//
// Weights are the M side of m16n8k16 MMAs, tokens the N side (8 per n-tile):
// all tokens are multiplied with every touched expert, which costs nothing at
// N = 8, and an n-tile none of whose tokens chose the expert is skipped.  A
// slot is 16 weight rows x 256 k (2 KB of codes in the 128-byte TMA swizzle),
// a stage 16 slots, one per consumer warp:
//   gate_up  a unit is 8 gate and the 8 matching up rows of one expert over
//            all of H, one slot per 256 k: warp w always multiplies the same
//            256 k, so its x fragment stays in registers for the whole phase
//            (f16 rows scaled by a power of two, as in ffn_decode.cu, exact for
//            elements within 2^29 of the row's largest).  Units go round the CTAs.
//   down     16 output rows x the slots (expert, 256 of I), in one sequence that
//            is cut into equal ranges, one per CTA.  A warp adds its slots'
//            products, times routing weight, into registers until the output
//            rows change.  Rows that a cut divides are joined by the CTA that
//            finishes last, adding the CTAs' partial sums in their order: the
//            result does not depend on timing.
// h stays in fp32 between the phases; the down product reads it as f16 scaled by
// a power of two per (token, expert) row (11 significant bits for elements
// within 2^14 of the row's largest, 2^-25 of that largest below).
// Warps: 16 consumers, one producer (TMA), one epilogue (adds the consumers'
// partial sums over k, SwiGLU, stores).  Every wait is bounded (mbar_wait,
// grid_wait).
#include <algorithm>

#include "moe_internal.h"
#include "route_device.cuh"

namespace moe {

namespace {

constexpr int kConsumerWarps = 16;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kProducerWarp = kConsumerWarps;
constexpr int kThreads = kConsumers + 64;  // the last warp is the epilogue
constexpr int kSlotBytes = 16 * 128;
constexpr int kStageBytes = kConsumerWarps * kSlotBytes;
constexpr int kSmemLimit = 232448;
constexpr int kMaxList = 528;   // touched experts, and (token, slot) pairs: 16 * 33
constexpr int kMaxGrid = 256;   // CTAs that the workspace holds partial sums of
constexpr int kMaxTasks = 64;   // router dot products (row x k range) of one CTA

struct FewArgs {
    const uint16_t* x;       // [T][H] bf16
    const uint16_t* wr;      // [E][H] bf16
    const uint16_t* gate;    // [H] bf16 or null
    const uint8_t* s13;      // [Et][2I][H/32]
    const uint8_t* s2;       // [Et][H][I/32]
    uint16_t* out;           // [T][H] bf16
    int32_t* ids;            // [T][Kt] or null
    float* w;                // [T][Kt] or null
    uint32_t* sync;          // [3] barrier counters, zero between calls
    float* logits;           // [T][E + 1]: the last one the shared expert's gate
    uint32_t* hmax;          // [T * Kt] largest |h| of a pair, as bits
    uint32_t* joined;        // [H / 16] CTAs that left a partial sum of these output rows
    float* h;                // [T * Kt][I]
    float4* partial;         // [grid][2][NT * 32] partial sums of cut output rows
    int T, H, I, E, K, shared, renorm;
    // decode group factor 2^(s-126) as fp32 bits s * exp_one + exp_bias, runtime
    // values so that the multiply-add stays one instruction
    uint32_t exp_one, exp_bias;
};

template <int NT>
struct FewLayout {
    static constexpr int kPartBytes = NT * kConsumerWarps * 32 * 16;  // one partial-sum buffer
    static constexpr int kListBytes = kMaxList * (4 + 4 + 4) + 16 * 4 + 64;
    static constexpr int kFixed = 2 * kPartBytes + kListBytes + 256 + 1024;
    static constexpr int kStages = (kSmemLimit - kFixed) / kStageBytes;
    static_assert(kStages >= 4, "ring depth");
    static constexpr int kPart = kStages * kStageBytes;
    static constexpr int kList = kPart + 2 * kPartBytes;
    static constexpr int kBar = (kList + kListBytes + 7) / 8 * 8;
    static constexpr int kTotal = kBar + 256 + 1024;
    static_assert(kTotal <= kSmemLimit, "shared memory");
    // scratch of the routing phase, over the partial-sum buffers
    static constexpr int kMask = kPart;                 // [1025] token masks by expert
    static constexpr int kFirst = kMask + 1028 * 4;     // [1025] first pair by expert (16 bits)
    static constexpr int kIds = kFirst + 1028 * 2;      // [16][33]
    static constexpr int kW = kIds + 16 * 33 * 4;
    static constexpr int kRed = kW + 16 * 33 * 4;       // [kMaxTasks][16]
    static_assert(kRed + kMaxTasks * 16 * 4 + 256 <= kList, "routing scratch");
};

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Adds one to a grid-wide counter; the caller's earlier writes (and those of
// threads it has synchronised with) are visible to whoever reads the sum.
__device__ __forceinline__ uint32_t add_release(uint32_t* p) {
    uint32_t v;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Bounded wait (see kWaitLimitNs) until `n` CTAs have added to the counter.
__device__ __forceinline__ bool grid_wait(const uint32_t* p, uint32_t n) {
    if (ld_acquire(p) == n) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (ld_acquire(p) == n) return true;
        if ((i & 63) == 0) {
            if (*(volatile int*)&g_device_error) return false;
            if (global_ns() - t0 > kWaitLimitNs) {
                atomicExch(&g_device_error, 1);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

__device__ __forceinline__ float bf16f(uint32_t bits) { return __uint_as_float(bits << 16); }

// Eight codes (two per byte, the even k in the low nibble) -> four f16x2.
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t out[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}

// acc[n] += one slot (16 rows x 256 k) times the token fragments b[n]: per 32-k
// scale group two MMAs into a fresh partial sum, added times 2^(s - 126).
// lm: this lane's four ldmatrix offsets within a slot.
template <int NT>
__device__ __forceinline__ void slot_mma(uint32_t slot, const uint32_t lm[4], uint2 sc0, uint2 sc1,
                                         const uint4 (&b)[NT][8], uint32_t need, const FewArgs& a,
                                         float (&acc)[NT][4]) {
#pragma unroll
    for (int gp = 0; gp < 4; ++gp) {
        uint32_t w[4];
        ldmatrix_x4(slot + lm[gp], w);
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
            const int gl = 2 * gp + gi;
            const uint32_t b0 = __byte_perm(gl < 4 ? sc0.x : sc0.y, 0, 0x4440 + (gl & 3));
            const uint32_t b1 = __byte_perm(gl < 4 ? sc1.x : sc1.y, 0, 0x4440 + (gl & 3));
            const float f0 = __uint_as_float(b0 * a.exp_one + a.exp_bias);
            const float f1 = __uint_as_float(b1 * a.exp_one + a.exp_bias);
            uint32_t ta[4], tb[4];
            codes_to_f16x2(w[gi ? 2 : 0], ta);
            codes_to_f16x2(w[gi ? 3 : 1], tb);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (NT > 1 && !((need >> n) & 1u)) continue;  // warp-uniform
                float t4[4];
                mma_f16_16816_z(t4, ta[0], tb[0], ta[1], tb[1], b[n][gl].x, b[n][gl].y);
                mma_f16_16816_acc(t4, ta[2], tb[2], ta[3], tb[3], b[n][gl].z, b[n][gl].w);
                acc[n][0] = fmaf(t4[0], f0, acc[n][0]);
                acc[n][1] = fmaf(t4[1], f0, acc[n][1]);
                acc[n][2] = fmaf(t4[2], f1, acc[n][2]);
                acc[n][3] = fmaf(t4[3], f1, acc[n][3]);
            }
        }
    }
}

// Eight scale bytes of a row from group 8 * slice on (zeros past its end).
__device__ __forceinline__ uint2 load_scales(const uint8_t* row, int slice, int groups, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint2*>(row + 8 * slice));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (8 * slice + j < groups) w[j >> 2] |= (uint32_t)__ldg(row + 8 * slice + j) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The range of the down phase's slots that CTA b of G multiplies.
__device__ __forceinline__ long long cut(long long slots, int b, int G) { return slots * b / G; }

// NT: n-tiles of 8 tokens; NC: 256-k slices of H per consumer warp.
template <int NT, int NC>
__global__ void __launch_bounds__(kThreads, 1)
    layer_few_kernel(const FewArgs a, const __grid_constant__ CUtensorMap w13_map,
                     const __grid_constant__ CUtensorMap w2_map) {
    pdl_begin();
    using L = FewLayout<NT>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float4* part = reinterpret_cast<float4*>(smem + L::kPart);        // [2][NT][16 warps][32]
    int32_t* list_e = reinterpret_cast<int32_t*>(smem + L::kList);    // touched experts
    uint32_t* list_m = reinterpret_cast<uint32_t*>(list_e + kMaxList);  // first pair << 16 | token mask
    float* pair_w = reinterpret_cast<float*>(list_m + kMaxList);      // routing weight of a pair
    float* rscale = pair_w + kMaxList;                                // [16] factor undoing x's scaling
    int32_t* info = reinterpret_cast<int32_t*>(rscale + 16);          // [0] list length, [1] barrier outcome,
                                                                      // [2] outcome of the second one
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + kStages;
    uint64_t* part_full = empty + kStages;  // [2]
    uint64_t* part_free = part_full + 2;    // [2]
    uint64_t* h_ready = part_free + 2;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = (int)blockIdx.x, G = (int)gridDim.x;
    const int T = a.T, H = a.H, I = a.I;
    const int Kt = a.K + a.shared, Et = a.E + a.shared;
    // gate_up: slots per unit, units per stage (NC == 1), units per expert
    const int sg = (H + 255) / 256;
    const int ups = NC == 1 ? kConsumerWarps / sg : 1;
    const int upe = I / 8;
    const int KGH = H / 32, KGI = I / 32;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumerWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&part_full[i], kConsumerWarps);
            mbar_init(&part_free[i], 1);
        }
        mbar_init(h_ready, 1);
        info[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    // gate_up stage `st` of this CTA: unit k (k-th of the CTA: b + k G) and slice of slot w
    auto gate_up_slot = [&](int st, int w, int& k, int& slice) {
        if (NC == 1) {
            k = st * ups + w / sg;
            slice = w % sg;
            return w / sg < ups;
        }
        k = st / NC;
        slice = (st % NC) * kConsumerWarps + w;
        return slice < sg;
    };
    auto my_units = [&](int units) { return units > b ? (units - b + G - 1) / G : 0; };
    auto gate_up_stages = [&](int n) { return NC == 1 ? (n + ups - 1) / ups : n * NC; };

    // producer: one gate_up stage; lane w loads slot w (8 gate rows, 8 up rows)
    auto issue_gate_up = [&](uint32_t gs, int st, int nunits, bool routed) {
        const int s = gs % kStages;
        int k, slice;
        const bool on = gate_up_slot(st, lane & 15, k, slice) && lane < kConsumerWarps && k < nunits;
        const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, on));
        if (lane == 0) mbar_arrive_expect_tx(&full[s], n * kSlotBytes);
        __syncwarp();
        if (on) {
            const int u = b + k * G, i = u / upe, blk = u - i * upe;
            const int e = routed ? list_e[i] : a.E;  // the shared expert is first in the list
            const int row = e * 2 * I + blk * 8;
            const uint32_t dst = smem_u32(smem + s * kStageBytes + lane * kSlotBytes);
            tma_load_2d(dst, &w13_map, slice * 128, row, &full[s]);
            tma_load_2d(dst + 1024, &w13_map, slice * 128, row + I, &full[s]);
            // the scale bytes of this slot's rows, shared by the unit's slots
            for (int r = slice; r < 16; r += sg) {
                const uint8_t* p = a.s13 + (size_t)(row + (r < 8 ? r : I + r - 8)) * KGH;
                for (int o = 0; o < KGH; o += 128) prefetch_l2(p + o);
            }
        }
        __syncwarp();
    };

    uint32_t gs = 0;  // stages issued (producer) or consumed so far

    if (warp == kProducerWarp) {
        // the shared expert's units need no routing: fill the ring with them
        if (a.shared) {
            const int n = my_units(upe);
            const int stages = NC == 1 ? n / ups : n * NC;  // whole stages only
            for (; (int)gs < min(stages, kStages); ++gs) issue_gate_up(gs, (int)gs, n, false);
        }
    } else if (warp < kConsumerWarps) {
        // ------------------------------------------------------- router
        // rows b, b + G, ... of [Wr; gate], each split over k so that all warps work; the
        // same split in every CTA, so that equal rows give equal logits
        const int rows = a.E + (a.gate ? 1 : 0);
        const int nrows = rows > b ? (rows - b + G - 1) / G : 0;
        const int Q = max(1, kConsumerWarps / ((rows + G - 1) / G));
        float* red = reinterpret_cast<float*>(smem + L::kRed);
        const int units = H / 8;
        for (int task = warp; task < nrows * Q; task += kConsumerWarps) {
            const int e = b + (task / Q) * G, q = task % Q;
            const uint4* w4 = reinterpret_cast<const uint4*>(e < a.E ? a.wr + (size_t)e * H : a.gate);
            float acc[8 * NT];
#pragma unroll
            for (int t = 0; t < 8 * NT; ++t) acc[t] = 0.0f;
            const int u1 = units * (q + 1) / Q;
            for (int u = units * q / Q + lane; u < u1; u += 32) {
                const uint4 wv = __ldg(w4 + u);
                const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                for (int t = 0; t < 8 * NT; ++t) {
                    if (t < T) {
                        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)t * H) + u);
                        const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[t] = fmaf(bf16f(ww[i] & 0xFFFFu), bf16f(xx[i] & 0xFFFFu), acc[t]);
                            acc[t] = fmaf(__uint_as_float(ww[i] & 0xFFFF0000u),
                                          __uint_as_float(xx[i] & 0xFFFF0000u), acc[t]);
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 8 * NT; ++t) {
                if (t >= T) break;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
                if (lane == t) red[task * 16 + t] = acc[t];
            }
        }
        consumers_sync();
        for (int i = tid; i < nrows * T; i += kConsumers) {
            const int r = i / T, t = i - r * T;
            float v = 0.0f;
            for (int q = 0; q < Q; ++q) v += red[(r * Q + q) * 16 + t];
            a.logits[(size_t)t * (a.E + 1) + b + r * G] = v;
        }
        // what later phases add to starts at zero
        for (int i = b * kConsumers + tid; i < T * Kt; i += G * kConsumers) a.hmax[i] = 0u;
        for (int i = b * kConsumers + tid; i < H / 16; i += G * kConsumers) a.joined[i] = 0u;
        __threadfence();
        consumers_sync();
        if (tid == 0) add_release(&a.sync[0]);

        // while the others finish: the rows' powers of two, the masks' zeros
        if (warp < T) {
            uint32_t mx = 0;
            const uint4* xr = reinterpret_cast<const uint4*>(a.x + (size_t)warp * H);
            for (int u = lane; u < units; u += 32) {
                const uint4 v = __ldg(xr + u);
                const uint32_t xx[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) mx = max(mx, max(xx[i] & 0x7FFFu, (xx[i] >> 16) & 0x7FFFu));
            }
            mx = __reduce_max_sync(0xFFFFFFFFu, mx);
            // (the MMA's group factor is 2^(s-126): the rest of it goes in here)
            if (lane == 0) rscale[warp] = __uint_as_float((uint32_t)(127 - row_f16_shift(mx)) << 23) * 0.5f;
        }
        uint32_t* mask = reinterpret_cast<uint32_t*>(smem + L::kMask);
        uint16_t* first = reinterpret_cast<uint16_t*>(smem + L::kFirst);
        int32_t* ids_s = reinterpret_cast<int32_t*>(smem + L::kIds);
        float* w_s = reinterpret_cast<float*>(smem + L::kW);
        for (int e = tid; e < Et; e += kConsumers) mask[e] = 0u;
        if (tid == 0) info[1] = grid_wait(&a.sync[0], (uint32_t)G) ? 1 : 0;
        consumers_sync();

        // ------------------------------------------------------ routing
        // every CTA routes all tokens, one warp each, and builds the same list
        if (info[1]) {
            if (warp < T) {
                const float* l = a.logits + (size_t)warp * (a.E + 1);
                const float sw = a.gate ? 1.0f / (1.0f + expf(-__ldcg(l + a.E))) : 1.0f;
                int32_t* wi = ids_s + warp * 33;
                float* ww = w_s + warp * 33;
                if (a.E <= 128)
                    route_token<4, true>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
                else if (a.E <= 512)
                    route_token<16, true>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
                else
                    route_token<32, true>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
                __syncwarp();
                for (int j = lane; j < Kt; j += 32) {
                    // a slot without an expert (only where every logit left is a NaN of the
                    // lowest order; its weight is NaN) goes to expert 0
                    if (wi[j] < 0) wi[j] = 0;
                    atomicOr(&mask[wi[j]], 1u << warp);
                    if (b == 0 && a.ids) a.ids[warp * Kt + j] = wi[j];
                    if (b == 0 && a.w) a.w[warp * Kt + j] = ww[j];
                }
            }
            consumers_sync();
            // list: the shared expert first, then the touched routed ones by id;
            // warp w orders experts 64 w .. 64 w + 63
            int32_t* sums = reinterpret_cast<int32_t*>(smem + L::kRed);  // [16][2] experts, pairs
            int ne[2], np[2];
            uint32_t mk[2];
            int ce = 0, cp = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 64 * warp + 32 * i + lane;
                mk[i] = e < a.E ? mask[e] : 0u;
                const uint32_t hot = __ballot_sync(0xFFFFFFFFu, mk[i] != 0);
                int c = __popc(mk[i]);
                const int own = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, c, o);
                    if (lane >= o) c += v;
                }
                ne[i] = ce + __popc(hot & lanemask_lt());
                np[i] = cp + c - own;
                ce += __popc(hot);
                cp += __shfl_sync(0xFFFFFFFFu, c, 31);
            }
            if (lane == 0) {
                sums[2 * warp] = ce;
                sums[2 * warp + 1] = cp;
            }
            consumers_sync();
            int be = a.shared, bp = a.shared ? T : 0;
            int te = be;
            for (int i = 0; i < kConsumerWarps; ++i) {
                if (i < warp) {
                    be += sums[2 * i];
                    bp += sums[2 * i + 1];
                }
                te += sums[2 * i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!mk[i]) continue;
                const int e = 64 * warp + 32 * i + lane;
                list_e[be + ne[i]] = e;
                list_m[be + ne[i]] = (uint32_t)(bp + np[i]) << 16 | mk[i];
                first[e] = (uint16_t)(bp + np[i]);
            }
            if (tid == 0) {
                info[0] = te;
                if (a.shared) {
                    list_e[0] = a.E;
                    list_m[0] = (1u << T) - 1u;
                    first[a.E] = 0;
                }
            }
            consumers_sync();
            for (int i = tid; i < T * Kt; i += kConsumers) {
                const int t = i / Kt, e = ids_s[t * 33 + i - t * Kt];
                pair_w[first[e] + __popc(mask[e] & ((1u << t) - 1u))] = w_s[t * 33 + i - t * Kt];
            }
        }
    }
    __syncthreads();  // the list is there (or the barrier gave up)

    const bool routed = info[1] != 0;
    const int nlist = routed ? info[0] : 0;
    const int nunits = my_units(nlist * upe);
    const int gstages = gate_up_stages(nunits);
    const int sd = (I + 255) / 256;
    const int Q = nlist * sd;                        // down: slots per 16 output rows
    const long long slots = (long long)(H / 16) * Q;
    const long long lo = cut(slots, b, G), hi = cut(slots, b + 1, G);
    const int dstages = (int)((hi - lo + kConsumerWarps - 1) / kConsumerWarps);
    const int ru0 = Q > 0 ? (int)(lo / Q) : 0;                       // first rows of this CTA
    const int pieces = hi > lo ? (int)((hi - 1) / Q) - ru0 + 1 : 0;  // groups of 16 output rows

    if (warp == kProducerWarp) {
        // ------------------------------------------------------- producer
        bool ok = routed;
        for (; (int)gs < gstages && ok; ++gs) {
            if (gs >= (uint32_t)kStages && !mbar_wait_warp(&empty[gs % kStages], ((gs / kStages) - 1) & 1)) {
                ok = false;
                break;
            }
            issue_gate_up(gs, (int)gs, nunits, true);
        }
        for (int st = 0; st < dstages && ok; ++st, ++gs) {
            const int s = gs % kStages;
            if (gs >= (uint32_t)kStages && !mbar_wait_warp(&empty[s], ((gs / kStages) - 1) & 1)) {
                ok = false;
                break;
            }
            const long long slot = lo + (long long)st * kConsumerWarps + lane;
            const bool on = lane < kConsumerWarps && slot < hi;
            const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, on));
            if (lane == 0) mbar_arrive_expect_tx(&full[s], n * kSlotBytes);
            __syncwarp();
            if (on) {
                const int ru = (int)(slot / Q), q = (int)(slot - (long long)ru * Q);
                const int i = q / sd, slice = q - i * sd;
                const int row = list_e[i] * H + ru * 16;
                tma_load_2d(smem_u32(smem + s * kStageBytes + lane * kSlotBytes), &w2_map, slice * 128, row,
                            &full[s]);
                for (int r = slice; r < 16; r += sd) {
                    const uint8_t* p = a.s2 + (size_t)(row + r) * KGI;
                    for (int o = 0; o < KGI; o += 128) prefetch_l2(p + o);
                }
            }
            __syncwarp();
        }
        // wait (bounded) until the last loads landed before the CTA can exit
        for (int d = 0; d < kStages && d < (int)gs; ++d) {
            const uint32_t u = gs - 1 - d;
            if (!mbar_wait_warp(&full[u % kStages], (u / kStages) & 1)) break;
        }
    } else if (warp < kConsumerWarps) {
        // ------------------------------------------------------ consumers
        const int r = lane >> 2, c = lane & 3, mj = lane >> 3, mi = lane & 7;
        uint32_t lm[4];
#pragma unroll
        for (int gp = 0; gp < 4; ++gp)
            lm[gp] = (uint32_t)((mj & 1) * 1024 + mi * 128 + (((2 * gp + (mj >> 1)) ^ mi) << 4));
        const uint32_t slot_base = smem_u32(smem) + warp * kSlotBytes;
        bool failed = !routed;
        uint32_t pc = 0;  // partial-sum buffers handed to the epilogue

        auto hand_over = [&](const float (&acc)[NT][4]) {
            const int buf = pc & 1;
            if (!failed && pc >= 2 && !mbar_wait_warp(&part_free[buf], ((pc >> 1) - 1) & 1)) failed = true;
            if (!failed) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    part[((buf * NT + n) * kConsumerWarps + warp) * 32 + lane] =
                        make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_full[buf]);
            ++pc;
        };

        // -------------------------------------------------------- gate_up
        {
            uint4 xb[NC][NT][8];
            const int sl0 = NC == 1 ? warp % sg : warp;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int t = 8 * n + r;
                    // 2^sigma from the factor 2^-sigma / 2
                    const float up = t < T ? 0.5f / rscale[t] : 0.0f;
#pragma unroll
                    for (int gl = 0; gl < 8; ++gl) {
                        const int k = (sl0 + ch * kConsumerWarps) * 256 + 32 * gl + 8 * c;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (t < T && k < H) {
                            const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)t * H + k));
                            v = make_uint4(bf16x2_to_f16x2_scaled(q.x, up), bf16x2_to_f16x2_scaled(q.y, up),
                                           bf16x2_to_f16x2_scaled(q.z, up), bf16x2_to_f16x2_scaled(q.w, up));
                        }
                        xb[ch][n][gl] = v;
                    }
                }
            const bool vec = KGH % 8 == 0 && ((uintptr_t)a.s13 & 7) == 0;
            auto scales_of = [&](int st, uint2& s0, uint2& s1) {
                int k, slice;
                s0 = s1 = make_uint2(0, 0);
                if (!gate_up_slot(st, warp, k, slice) || k >= nunits) return;
                const int u = b + k * G, i = u / upe;
                const uint8_t* p = a.s13 + ((size_t)list_e[i] * 2 * I + (u - i * upe) * 8 + r) * KGH;
                s0 = load_scales(p, slice, KGH, vec);
                s1 = load_scales(p + (size_t)I * KGH, slice, KGH, vec);
            };
            uint2 n0 = make_uint2(0, 0), n1 = n0;
            if (gstages > 0) scales_of(0, n0, n1);
            for (int st = 0; st < gstages; st += NC) {
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
#pragma unroll
                for (int ch = 0; ch < NC; ++ch, ++gs) {
                    const int s = gs % kStages;
                    const uint2 s0 = n0, s1 = n1;
                    if (st + ch + 1 < gstages) scales_of(st + ch + 1, n0, n1);
                    if (!failed && !mbar_wait_warp(&full[s], (gs / kStages) & 1)) failed = true;
                    int k, slice;
                    if (!failed && gate_up_slot(st + ch, warp, k, slice) && k < nunits) {
                        const uint32_t m = list_m[(b + k * G) / upe];
                        slot_mma<NT>(slot_base + s * kStageBytes, lm, s0, s1, xb[ch],
                                     ((m & 0xFFu) ? 1u : 0u) | ((m & 0xFF00u) ? 2u : 0u), a, acc);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                }
                hand_over(acc);
            }
        }
        // ----------------------------------------------------------- down
        {
            if (!failed && !mbar_wait_warp(h_ready, 0)) failed = true;
            if (!failed && !info[2]) failed = true;
            const bool vec = KGI % 8 == 0 && ((uintptr_t)a.s2 & 7) == 0;
            float acc[NT][4];
            int piece = 0;
            auto clear = [&]() {
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
            };
            clear();
            auto place = [&](long long slot, int& ru, int& i, int& slice) {
                ru = (int)(slot / Q);
                const int q = (int)(slot - (long long)ru * Q);
                i = q / sd;
                slice = q - i * sd;
            };
            auto scales_of = [&](long long slot, uint2& s0, uint2& s1) {
                s0 = s1 = make_uint2(0, 0);
                if (slot >= hi) return;
                int ru, i, slice;
                place(slot, ru, i, slice);
                const uint8_t* p = a.s2 + ((size_t)list_e[i] * H + ru * 16 + r) * KGI;
                s0 = load_scales(p, slice, KGI, vec);
                s1 = load_scales(p + (size_t)8 * KGI, slice, KGI, vec);
            };
            uint2 n0, n1;
            scales_of(lo + warp, n0, n1);
            for (int st = 0; st < dstages; ++st, ++gs) {
                const int s = gs % kStages;
                const long long slot = lo + (long long)st * kConsumerWarps + warp;
                const uint2 s0 = n0, s1 = n1;
                scales_of(slot + kConsumerWarps, n0, n1);
                int ru = 0, i = 0, slice = 0;
                if (slot < hi) {
                    place(slot, ru, i, slice);
                    while (piece < ru - ru0) {  // this warp's part of the earlier rows is complete
                        hand_over(acc);
                        clear();
                        ++piece;
                    }
                }
                uint4 hb[NT][8];
                float f[NT];  // routing weight and 2^-sigma of this lane's token
                uint32_t need = 0;
                if (slot < hi && !failed) {
                    const uint32_t m = list_m[i];
                    need = ((m & 0xFFu) ? 1u : 0u) | ((m & 0xFF00u) ? 2u : 0u);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int t = 8 * n + r;
                        f[n] = 0.0f;
#pragma unroll
                        for (int gl = 0; gl < 8; ++gl) hb[n][gl] = make_uint4(0, 0, 0, 0);
                        if ((m >> t) & 1u) {
                            const int p = (int)(m >> 16) + __popc(m & ((1u << t) - 1u));
                            const int sh = f32_f16_shift(__ldcg(a.hmax + p));
                            const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
                            f[n] = pair_w[p] * __uint_as_float((uint32_t)(127 - sh) << 23) * 0.5f;
                            const float* hp = a.h + (size_t)p * I + 256 * slice + 8 * c;
#pragma unroll
                            for (int gl = 0; gl < 8; ++gl) {
                                if (256 * slice + 32 * gl < I) {
                                    const float4 u = __ldcg(reinterpret_cast<const float4*>(hp + 32 * gl));
                                    const float4 v = __ldcg(reinterpret_cast<const float4*>(hp + 32 * gl) + 1);
                                    const __half2 h0 = __floats2half2_rn(u.x * up, u.y * up);
                                    const __half2 h1 = __floats2half2_rn(u.z * up, u.w * up);
                                    const __half2 h2 = __floats2half2_rn(v.x * up, v.y * up);
                                    const __half2 h3 = __floats2half2_rn(v.z * up, v.w * up);
                                    hb[n][gl] = make_uint4(*reinterpret_cast<const uint32_t*>(&h0),
                                                           *reinterpret_cast<const uint32_t*>(&h1),
                                                           *reinterpret_cast<const uint32_t*>(&h2),
                                                           *reinterpret_cast<const uint32_t*>(&h3));
                                }
                            }
                        }
                    }
                }
                if (!failed && !mbar_wait_warp(&full[s], (gs / kStages) & 1)) failed = true;
                if (!failed && slot < hi) {
                    float d[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.0f;
                    slot_mma<NT>(slot_base + s * kStageBytes, lm, s0, s1, hb, need, a, d);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        // columns 2c and 2c + 1: the factors of lanes with that r.  A token
                        // that did not choose the expert adds nothing, whatever its column is
                        const float g0 = __shfl_sync(0xFFFFFFFFu, f[n], 8 * c);
                        const float g1 = __shfl_sync(0xFFFFFFFFu, f[n], 8 * c + 4);
                        const uint32_t m2 = list_m[i] >> (8 * n + 2 * c);
                        if (m2 & 1u) {
                            acc[n][0] = fmaf(d[n][0], g0, acc[n][0]);
                            acc[n][2] = fmaf(d[n][2], g0, acc[n][2]);
                        }
                        if (m2 & 2u) {
                            acc[n][1] = fmaf(d[n][1], g1, acc[n][1]);
                            acc[n][3] = fmaf(d[n][3], g1, acc[n][3]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
            }
            for (; piece < pieces; ++piece) {
                hand_over(acc);
                clear();
            }
        }
    } else {
        // ------------------------------------------------------- epilogue
        const int r = lane >> 2, c = lane & 3;
        uint32_t pc = 0;
        bool ok = routed;
        // the sum of one n-tile's partial sums over warps w0 .. w0 + n - 1
        auto sum_of = [&](int buf, int nt, int w0, int n) {
            float4 v = make_float4(0, 0, 0, 0);
            const float4* p = part + ((buf * NT + nt) * kConsumerWarps + w0) * 32 + lane;
#pragma unroll 4
            for (int w = 0; w < n; ++w) {
                const float4 q = p[w * 32];
                v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
            }
            return v;
        };
        for (int st = 0; st < gstages && ok; st += NC, ++pc) {
            const int buf = pc & 1;
            if (!mbar_wait_warp(&part_full[buf], (pc >> 1) & 1)) {
                ok = false;
                break;
            }
            for (int j = 0; j < ups; ++j) {
                const int k = NC == 1 ? st * ups + j : st / NC;
                if (k >= nunits) break;
                const int u = b + k * G, i = u / upe;
                const uint32_t m = list_m[i];
                const int col = (u - i * upe) * 8 + r;  // of I
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 v = sum_of(buf, nt, NC == 1 ? j * sg : 0, NC == 1 ? sg : kConsumerWarps);
                    const float g[2] = {v.x, v.y}, up[2] = {v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int t = 8 * nt + 2 * c + q;
                        const bool on = (m >> t) & 1u;
                        float hv = 0.0f;
                        const int p = (int)(m >> 16) + __popc(m & ((1u << t) - 1u));
                        if (on) {
                            const float rs = rscale[t];
                            hv = silu(g[q] * rs) * (up[q] * rs);
                            a.h[(size_t)p * I + col] = hv;
                        }
                        uint32_t mx = __float_as_uint(hv) & 0x7FFFFFFFu;
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                        if (on && r == 0) atomicMax(a.hmax + p, mx);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_free[buf]);
        }
        // h of this CTA is complete; wait for everybody's
        __threadfence();
        __syncwarp();
        if (lane == 0 && ok) {
            add_release(&a.sync[1]);
            ok = grid_wait(&a.sync[1], (uint32_t)G);
            if (ok) {
                info[2] = 1;
                // the last CTA past the second barrier leaves the counters at zero
                if (add_release(&a.sync[2]) == (uint32_t)G - 1) {
                    a.sync[0] = 0u;
                    a.sync[1] = 0u;
                    a.sync[2] = 0u;
                }
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        if (lane == 0) mbar_arrive(h_ready);

        for (int piece = 0; piece < pieces && ok; ++piece, ++pc) {
            const int buf = pc & 1;
            if (!mbar_wait_warp(&part_full[buf], (pc >> 1) & 1)) {
                ok = false;
                break;
            }
            const int ru = ru0 + piece;
            float4 v[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) v[nt] = sum_of(buf, nt, 0, kConsumerWarps);
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_free[buf]);
            const long long s0 = (long long)ru * Q, s1 = s0 + Q;
            bool write = true;
            if (s0 < lo || s1 > hi) {
                // rows cut between CTAs: the one that comes last adds the partial
                // sums in CTA order
                float4* mine = a.partial + ((size_t)b * 2 + (piece ? 1 : 0)) * NT * 32;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) __stcg(mine + nt * 32 + lane, v[nt]);
                const int b0 = (int)(((s0 + 1) * G - 1) / slots), b1 = (int)((s1 * G - 1) / slots);
                // (fewer slots than CTAs: some CTAs have none)
                const uint32_t parts = slots >= G ? (uint32_t)(b1 - b0 + 1) : (uint32_t)Q;
                __threadfence();
                __syncwarp();
                uint32_t old = 0;
                if (lane == 0) old = add_release(&a.joined[ru]);
                old = __shfl_sync(0xFFFFFFFFu, old, 0);
                write = old == parts - 1;
                if (write) {
                    __threadfence();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) v[nt] = make_float4(0, 0, 0, 0);
                    for (int bb = b0; bb <= b1; ++bb) {
                        const long long l0 = cut(slots, bb, G);
                        if (l0 == cut(slots, bb + 1, G)) continue;
                        const float4* p = a.partial + ((size_t)bb * 2 + (l0 / Q == ru ? 0 : 1)) * NT * 32 + lane;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float4 q = __ldcg(p + nt * 32);
                            v[nt].x += q.x, v[nt].y += q.y, v[nt].z += q.z, v[nt].w += q.w;
                        }
                    }
                }
            }
            if (write) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int t = 8 * nt + 2 * c;
                    uint16_t* o = a.out + (size_t)t * H + ru * 16 + r;
                    if (t < T) {
                        o[0] = f32_to_bf16_bits(v[nt].x);
                        o[8] = f32_to_bf16_bits(v[nt].z);
                    }
                    if (t + 1 < T) {
                        o[H] = f32_to_bf16_bits(v[nt].y);
                        o[H + 8] = f32_to_bf16_bits(v[nt].w);
                    }
                }
            }
        }
    }
    pdl_end();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct FewWorkspace {
    size_t sync, logits, hmax, joined, h, partial, total;
};

FewWorkspace few_workspace(int T, int H, int I, int E, int Kt) {
    FewWorkspace w;
    w.sync = 0;
    w.logits = 256;
    w.hmax = w.logits + align256((size_t)T * (E + 1) * 4);
    w.joined = w.hmax + align256((size_t)T * Kt * 4);
    w.h = w.joined + align256((size_t)(H / 16) * 4);
    w.partial = w.h + align256((size_t)T * Kt * I * 4);
    w.total = w.partial + (size_t)kMaxGrid * 2 * 2 * 512;
    return w;
}

template <int NT, int NC>
cudaError_t launch_few(const FewArgs& a, const CUtensorMap& w13, const CUtensorMap& w2, int grid,
                       cudaStream_t s) {
    const size_t smem = FewLayout<NT>::kTotal;
    cudaError_t err = ensure_dynamic_smem((const void*)layer_few_kernel<NT, NC>, smem);
    if (err != cudaSuccess) return err;
    // cooperative: the grid's CTAs wait for one another, so all must be resident
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_few_kernel<NT, NC>, a, w13, w2);
}

}  // namespace

size_t layer_few_workspace(int T, int H, int I, int E, int Kt) { return few_workspace(T, H, I, E, Kt).total; }

cudaError_t launch_layer_few(const LayerFew& p, void* workspace, cudaStream_t s) {
    const int Kt = p.K + p.shared, Et = p.E + p.shared;
    const FewWorkspace L = few_workspace(p.T, p.H, p.I, p.E, Kt);
    char* ws = reinterpret_cast<char*>(workspace);
    FewArgs a;
    a.x = p.x;
    a.wr = p.w_router;
    a.gate = p.w_shared_gate;
    a.s13 = p.s13;
    a.s2 = p.s2;
    a.out = p.out;
    a.ids = p.topk_ids;
    a.w = p.topk_w;
    a.sync = reinterpret_cast<uint32_t*>(ws + L.sync);
    a.logits = reinterpret_cast<float*>(ws + L.logits);
    a.hmax = reinterpret_cast<uint32_t*>(ws + L.hmax);
    a.joined = reinterpret_cast<uint32_t*>(ws + L.joined);
    a.h = reinterpret_cast<float*>(ws + L.h);
    a.partial = reinterpret_cast<float4*>(ws + L.partial);
    a.T = p.T;
    a.H = p.H;
    a.I = p.I;
    a.E = p.E;
    a.K = p.K;
    a.shared = p.shared;
    a.renorm = p.renormalize;
    a.exp_one = a.exp_bias = 1u << 23;
    CUtensorMap w13, w2;
    cudaError_t err = encode_codes_map(&w13, p.w13, p.H / 2, (uint64_t)Et * 2 * p.I, 128, 8);
    if (err != cudaSuccess) return err;
    err = encode_codes_map(&w2, p.w2, p.I / 2, (uint64_t)Et * p.H, 128, 16);
    if (err != cudaSuccess) return err;
    // no more CTAs than the widest phase has pieces of work for (a barrier of
    // fewer CTAs is shorter)
    const long long touched = std::min<long long>((long long)p.T * p.K, p.E) + p.shared;
    const long long work = std::max({(long long)p.E + 1, touched * (p.I / 8),
                                     (long long)(p.H / 16) * touched * ((p.I + 255) / 256)});
    const int grid = (int)std::min<long long>({work, (long long)num_sms(), (long long)kMaxGrid});
    if ((p.E + 1 + grid - 1) / grid > kMaxTasks) return cudaErrorNotSupported;
    if (p.T > 8) return launch_few<2, 1>(a, w13, w2, grid, s);
    if (p.H > 4096) return launch_few<1, 2>(a, w13, w2, grid, s);
    return launch_few<1, 1>(a, w13, w2, grid, s);
}

cudaError_t read_device_error_few(int* flag, int clear) {
    int wait = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&wait, g_device_error, sizeof(int));
    if (err != cudaSuccess) return err;
    *flag = wait ? 1 : 0;
    if (!clear) return cudaSuccess;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace moe
