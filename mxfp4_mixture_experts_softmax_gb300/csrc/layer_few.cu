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
// one TMA ring running through all phases and three grid-wide barriers stand
// between them (logits complete; h complete; y complete).  While the CTAs meet at a
// barrier the ring fills with the next phase's weights: the shared expert's
// before the routing is known, W2's before h is.
//
// Weights are the M side of m16n8k16 MMAs, tokens the N side.  The work list holds
// an entry per touched expert and 8 of its tokens (an expert with 9 to 16 tokens has two
// entries and is streamed twice, the second time from L2).  A slot is 16
// weight rows x 256 k (2 KB of codes in the 128-byte TMA swizzle), a stage
// up to 16 slots, one per consumer warp, and their scale bytes:
//   gate_up  a unit is 8 gate and the 8 matching up rows of one entry over all
//            of H, one slot per 256 k.  Each CTA takes an equal share of the
//            shared expert's units and a contiguous range of the others, so that a
//            warp keeps its x fragment (its 256 k of the entry's tokens) in
//            registers until the entry changes, once or twice in a call.  x
//            enters as f16 rows scaled by a power of two, as in ffn_decode.cu
//            (exact for elements within 2^29 of the row's largest).
//   down     its own list has an entry per touched expert and 4 of its tokens: h takes
//            part as two f16 terms, the high ones in columns 0 .. 3, what they leave in
//            columns 4 .. 7.  An item is 16 output rows of one entry, one slot per 256
//            of I; each CTA takes a contiguous range of the items, an entry's rows next to
//            each other, so the h fragment too stays in registers.  y goes to the
//            workspace in fp32 by (token, expert) pair; after a third barrier
//            each CTA adds up its share of the outputs, a token's pairs in slot
//            order, times routing weight.
// Measured (cold weights, call after call in one graph; 4096/1024, top-10 of 512 and a shared
// expert): 36.7 us for one token (74 MB of weights), 84 for 5, 189 for 16 (about 140 touched
// experts, 940 MB of weights, 5.0 TB/s).  By clock stamps in a build with them, one token:
// router and first barrier 5.2, top-K and lists 4.3, gate_up 13, second barrier 3, down 6,
// third barrier and sum 4.6.  16 tokens, 206 with the stamps: 16 until the lists are there,
// gate_up 112, second barrier 10 (the slowest CTA ends 6 after the mean), down 62, third
// barrier and sum 6 -- there the consumers, not HBM, set the pace: HBM would bring a stage
// every 0.8 us, and one takes them 0.95 in gate_up and 1.04 in down (issue slots half used,
// the conversion and its scaling most of them, waits for a stage a tenth).
// What a warp does for a stage beside its products (waits, arrivals, handing its sums
// over) takes longer than one slot's products, so the consumers take the stages two
// at a time.  A warp turns its slot's scale bytes into fp32 factors once, through shared
// memory (each of the four lanes that share a row would otherwise do it again: 130
// of the 330 cycles that 16 warps take per slot and scheduler).
// h passes between the phases as the sum of two f16 terms, the nearest and the nearest of
// what that leaves, with a power of two per 8 values (22 significant bits; one term would err
// by 2.5e-4 of the result); the down product brings a pair's row to one power of two
// (elements below 2^-15 of the row's largest keep fewer bits, down to 2^-38 of it).
// The terms share the columns that 4 tokens leave free, so the products cost what they
// did with one term; an expert with 5 to 8 tokens is multiplied twice instead (its weights
// come from L2 the second time).  No result depends on timing.
// Warps: 16 consumers, one producer (TMA), two epilogue warps, one per stage of a pair
// (adding the consumers' partial sums over k, SwiGLU, stores).  Every wait
// is bounded (mbar_wait, grid_wait).
#include <string.h>

#include <algorithm>

#include "moe_internal.h"
#include "route_device.cuh"

namespace moe {

namespace {

constexpr int kConsumerWarps = 16;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kProducerWarp = kConsumerWarps;
constexpr int kEpiWarp0 = kConsumerWarps + 1;
constexpr int kThreads = kConsumers + 3 * 32;
constexpr int kSlotBytes = 16 * 128;
constexpr int kCodeBytes = kConsumerWarps * kSlotBytes;    // a stage's codes
constexpr int kScaleBytes = kConsumerWarps * 16 * 8;       // and scale bytes
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kSmemLimit = 232448;
constexpr int kMaxPairs = 528;  // (token, slot) pairs: 16 * 33
constexpr int kMaxEntries = 516;  // of either list: at most one per routed pair, 512, and the shared expert's 4
constexpr int kMaxGrid = 256;

struct FewArgs {
    const uint16_t* x;       // [T][H] bf16
    const uint16_t* wr;      // [E][H] bf16
    const uint16_t* gate;    // [H] bf16 or null
    const uint8_t* s13;      // [Et][2I][H/32]
    const uint8_t* s2;       // [Et][H][I/32]
    uint16_t* out;           // [T][H] bf16
    int32_t* ids;            // [T][Kt] or null
    float* w;                // [T][Kt] or null
    uint32_t* sync;          // [4] barrier counters, zero between calls
    float* logits;           // [T][E + 1]: column E the shared expert's gate
    uint32_t* hmax;          // [T * Kt] largest |h| of a pair, as bits
    uint16_t* h;             // [T * Kt][2 terms][I] f16, times 2^shift of their 8 values
    int8_t* hshift;          // [T * Kt][shift_pitch(I)], see shift_at
    float* y;                // [T * Kt][H] expert outputs by pair
    int T, H, I, E, K, shared, renorm;
    int router_rows;         // rows of [Wr; gate] per CTA, at most 16
    int router_k;            // k of them and of x that fit shared memory at once
    // units of a stage, items of a stage; division by I / 8, H / 16 and E (div_by)
    int ups, ips;
    uint32_t upe_m, ru_m, e_m;
};

// The weights as the TMA reads them: whole 256-k slices (w13 [slice][gate, up][row],
// w2 [slice][row]), the first 16 in one box, the rest of a row of more than 16 in
// another, and what is left of a row past its last whole slice; and the scale bytes.
struct FewMaps {
    CUtensorMap w13, w13_rest, w13_tail, w2, w2_rest, w2_tail, s13, s2;
};

// shared memory
constexpr int kPartBytes = 2 * kConsumerWarps * 32 * 16;  // one buffer: the sums of a pair of stages
constexpr int kFactorBytes = 2 * kConsumerWarps * 16 * 32;  // a slot's 16 x 8 factors per warp, two stages
constexpr int kListBytes = kMaxPairs * (4 + 2 + 1) + kMaxEntries * (2 + 2 + 2 + 2) + 64 + 32;
constexpr int kBarBytes = 192;
constexpr int kStages = (kSmemLimit - 1024 - kBarBytes - kListBytes - 2 * kPartBytes - kFactorBytes) / kStageBytes;
static_assert(kStages >= 5, "ring depth");
constexpr int kPart = kStages * kStageBytes;
constexpr int kFactors = kPart + 2 * kPartBytes;
constexpr int kList = kFactors + kFactorBytes;
constexpr int kBar = (kList + kListBytes + 7) / 8 * 8;
constexpr int kSmemBytes = kBar + kBarBytes + 1024;  // + alignment slack
static_assert(kSmemBytes <= kSmemLimit, "shared memory");
static_assert((2 * kStages + 6) * 8 <= kBarBytes, "barriers");
// scratch of the routing phase: over the partial sums, and the logits over the last stages
constexpr int kMask = kPart;                 // [1025] token masks by expert
constexpr int kFirst = kMask + 1028 * 4;     // [1025] first pair by expert (16 bits)
constexpr int kIds = kFirst + 1028 * 2;      // [16][33]
constexpr int kSums = kIds + 16 * 33 * 4;    // [16]
static_assert(kSums + 16 * 4 <= kFactors, "routing scratch");
constexpr int kLogitStages = 2;              // 64 KB: 16 tokens x 1024 experts
constexpr int kEarlyStages = kStages - kLogitStages;  // loads before the routing is known

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Adds one to a grid-wide counter; the caller's earlier writes, and those of
// threads it has synchronised with, are visible to whoever reads the sum.
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

__device__ __forceinline__ void consumers_sync() { barrier_sync(1, kConsumers); }

// v / d for v < 2^20 and d < 2^12, m = div_magic(d)
__host__ __device__ __forceinline__ uint32_t div_magic(uint32_t d) { return d > 1 ? 0xFFFFFFFFu / d + 1u : 0u; }
__device__ __forceinline__ uint32_t div_by(uint32_t v, uint32_t m) { return m ? __umulhi(v, m) : v; }

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

// d = a b (+ d): m16n8k16, fp32 sums.  Not volatile, so that independent products are
// interleaved (the helpers of moe_device.cuh keep their order).
__device__ __forceinline__ void mma_first(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_next(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The router's products: bf16, 32 k of rows r and r + 8 (wa, wb) by 32 k of token r (x)
__device__ __forceinline__ void mma_bf16_32(float d[4], uint4 wa, uint4 wb, uint4 x) {
    asm("{\n\t"
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%6,%5,%7}, {%12,%13}, "
        "{%16,%16,%16,%16};\n\t"
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%8,%10,%9,%11}, {%14,%15}, "
        "{%0,%1,%2,%3};\n\t}"
        : "=&f"(d[0]), "=&f"(d[1]), "=&f"(d[2]), "=&f"(d[3])
        : "r"(wa.x), "r"(wa.y), "r"(wb.x), "r"(wb.y), "r"(wa.z), "r"(wa.w), "r"(wb.z), "r"(wb.w), "r"(x.x),
          "r"(x.y), "r"(x.z), "r"(x.w), "f"(0.0f));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts_f4(uint32_t addr, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// acc += one slot (16 rows x 256 k) times the token fragment b: per 32-k scale
// group two MMAs into a fresh partial sum, added times the group's factor.  lm:
// this lane's four ldmatrix offsets within a slot; fr: the factors of its row r (8
// floats; row r + 8 lies 256 bytes on).
__device__ __forceinline__ void slot_mma(uint32_t slot, const uint32_t lm[4], uint32_t fr, const uint4 (&b)[8],
                                         float (&acc)[4]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const float4 fa = lds_f4(fr + 16 * half), fb = lds_f4(fr + 256 + 16 * half);
        const float f0[4] = {fa.x, fa.y, fa.z, fa.w}, f1[4] = {fb.x, fb.y, fb.z, fb.w};
        uint32_t w[2][4];
        ldmatrix_x4(slot + lm[2 * half], w[0]);
        ldmatrix_x4(slot + lm[2 * half + 1], w[1]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int gl = 4 * half + q;
            uint32_t ta[4], tb[4];
            codes_to_f16x2(w[q >> 1][q & 1 ? 2 : 0], ta);
            codes_to_f16x2(w[q >> 1][q & 1 ? 3 : 1], tb);
            float t4[4];
            mma_first(t4, ta[0], tb[0], ta[1], tb[1], b[gl].x, b[gl].y);
            mma_next(t4, ta[2], tb[2], ta[3], tb[3], b[gl].z, b[gl].w);
            acc[0] = fmaf(t4[0], f0[q], acc[0]);
            acc[1] = fmaf(t4[1], f0[q], acc[1]);
            acc[2] = fmaf(t4[2], f1[q], acc[2]);
            acc[3] = fmaf(t4[3], f1[q], acc[3]);
        }
    }
}

// Four bytes from byte `at` of a matrix of `words` 32-bit words on, of which the
// first n count (zeros for the others): two aligned words and a shift, whatever the
// row's alignment, and no word past the matrix.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* base, size_t at, int n, size_t words) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(base);
    const size_t w = at >> 2;
    const uint32_t v = __funnelshift_r(__ldg(p + w), __ldg(p + min(w + 1, words - 1)), (uint32_t)(at & 3) * 8u);
    return n >= 4 ? v : (n > 0 ? v & ((1u << (8 * n)) - 1u) : 0u);
}

// Softmax top-K routing of one token by one warp, with route_token's results, written
// for a warp that has its scheduler to itself: what counts is the length of a round's
// chain of dependent steps (two warp-wide integer reductions a round).  2.8 us for the 10
// largest of 512 (every expert's rank at once, without rounds, took longer).  A call of one
// token takes 36.7 us with it and 38.2 with route_token in its place (top-10 of 512), 31.7
// and 39.9 (512/256, top-32 of 1024); of 16 tokens 189 and 197, as route_token leaves the
// consumers fewer registers.
template <int VPL>
__device__ __forceinline__ void route_few(const float* l, int E, int K, int with_shared, int renormalize,
                                          float shared_weight, int32_t* ids, float* w, int lane) {
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane + 32 * i < E ? order_key(l[lane + 32 * i]) : 0u;
    int my_id = 0;
    uint32_t my_key = 0u, top = 0u;
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        uint32_t t[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) t[i] = key[i];
#pragma unroll
        for (int o = VPL / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) t[i] = max(t[i], t[i + o]);
        const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, t[0]);
        // the lowest expert that holds it
#pragma unroll
        for (int i = 0; i < VPL; ++i) t[i] = key[i] == best ? 1u << i : 0u;
#pragma unroll
        for (int o = VPL / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) t[i] |= t[i + o];
        const uint32_t le = t[0] && best ? (uint32_t)(lane + 32 * (__ffs((int)t[0]) - 1)) : 0xFFFFFFFFu;
        const int e = (int)__reduce_min_sync(0xFFFFFFFFu, le);  // -1 if none is left
        const int own = e >= 0 && (e & 31) == lane ? e >> 5 : -1;
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = i == own ? 0u : key[i];
        if (lane == k) {
            my_id = e;
            my_key = best;
        }
        if (k == 0) top = best;
    }
    const float m = key_to_float(top);
    float z = 0.0f;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) z += expf(l[e] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    const float p = lane < K ? expf(key_to_float(my_key) - m) / z : 0.0f;
    float s = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane < K) {
        ids[lane] = my_id;
        w[lane] = renormalize ? p / s : p;
    }
    if (with_shared && lane == 0) {
        ids[K] = E;
        w[K] = shared_weight;
    }
}

// 2^(s - 127) of four scale bytes (0 for byte 0)
__device__ __forceinline__ float4 factors(uint32_t w) {
    return make_float4(__uint_as_float((w << 23) & 0x7F800000u), __uint_as_float((w << 15) & 0x7F800000u),
                       __uint_as_float((w << 7) & 0x7F800000u), __uint_as_float((w >> 1) & 0x7F800000u));
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// h's shifts: one byte per 8 values, those of 256 values (32 bytes) ordered so
// that the lane that multiplies values 32 g + 8 c .. 32 g + 8 c + 7, g = 0..7, finds
// its eight in one 8-byte word.
__host__ __device__ __forceinline__ int shift_pitch(int I) { return (I + 255) / 256 * 32; }
__device__ __forceinline__ int shift_at(int blk) { return (blk & ~31) | ((blk & 3) << 3) | ((blk >> 2) & 7); }

// The first of n things that CTA b of G takes (n * G < 2^32).
__device__ __forceinline__ int cut(int n, int b, int G) { return (int)((uint32_t)n * (uint32_t)b / (uint32_t)G); }

// NC: stages of a gate_up unit (H <= NC * 4096).  SF: the scale bytes come with the
// codes (rows of whole 16-byte units, which the TMA can read); else each warp loads
// its own, a pair of stages ahead.
template <int NC, bool SF>
__global__ void __launch_bounds__(kThreads, 1)
    layer_few_kernel(const FewArgs a, const __grid_constant__ FewMaps maps) {
    pdl_begin();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float4* part = reinterpret_cast<float4*>(smem + kPart);             // [2 buffers][2 stages][16 warps][32]
    float* w_s = reinterpret_cast<float*>(smem + kList);                // [T][Kt] routing weights
    float* rscale = w_s + kMaxPairs;                                    // [16] factor undoing x's scaling
    int32_t* info = reinterpret_cast<int32_t*>(rscale + 16);            // [0] entries, [1] outcome of the first
                                                                        // barrier, [2] of the second, [3] of the
                                                                        // third, [4] down's entries
    uint16_t* list_e = reinterpret_cast<uint16_t*>(info + 8);           // an entry's expert
    uint16_t* list_p = list_e + kMaxEntries;                            // its first pair << 4 | its tokens
    uint16_t* down_e = list_p + kMaxEntries;                            // the same for down's entries
    uint16_t* down_p = down_e + kMaxEntries;
    uint16_t* pair_of = down_p + kMaxEntries;                           // [T][Kt] pair of a token's slot
    uint8_t* pair_t = reinterpret_cast<uint8_t*>(pair_of + kMaxPairs);  // a pair's token
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBar);
    uint64_t* empty = full + kStages;
    uint64_t* part_full = empty + kStages;    // [2]
    uint64_t* part_free = part_full + 2;      // [2]
    uint64_t* h_ready = part_free + 2;
    uint64_t* router_full = h_ready + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = (int)blockIdx.x, G = (int)gridDim.x;
    const int T = a.T, H = a.H, I = a.I;
    const int Kt = a.K + a.shared, Et = a.E + a.shared;
    const int KGH = H / 32, KGI = I / 32;
    // gate_up: slots per unit, units per stage (NC == 1), units per entry
    const int sg = (H + 255) / 256, sg_whole = H / 256;
    const int ups = a.ups, upe = I / 8;
    const uint32_t upe_m = a.upe_m;
    const int sfp = NC == 1 ? KGH : 128;  // bytes between a unit's scale rows in a stage
    // down: items per entry, slots per item, items per stage or stages per item
    const int RU = H / 16;
    const uint32_t ru_m = a.ru_m;
    const int sd = (I + 255) / 256, sd_whole = I / 256;
    const int spi = (sd + kConsumerWarps - 1) / kConsumerWarps;
    const int ips = a.ips;
    const int sfp2 = spi == 1 ? KGI : 128;

    // router rows of this CTA, and what of them and of x lies in the ring: `rows` rows of
    // Wr (the gate last), then x's T, each 64 bytes past a multiple of 128 from the next
    const int row0 = b * a.router_rows, rows = max(min(a.router_rows, a.E + (a.gate ? 1 : 0) - row0), 0);
    const int rpitch = a.router_k * 2 + 64;
    auto load_router = [&](int k0) {  // the producer: rows' and tokens' k0 .. k0 + router_k
        const uint32_t bytes = (uint32_t)min(a.router_k, H - k0) * 2u;
        if (lane == 0) mbar_arrive_expect_tx(router_full, (uint32_t)(rows + T) * bytes);
        __syncwarp();
        if (lane < rows + T) {
            const uint16_t* src = lane >= rows ? a.x + (size_t)(lane - rows) * H
                                               : (row0 + lane < a.E ? a.wr + (size_t)(row0 + lane) * H : a.gate);
            bulk_copy_g2s(smem_u32(smem) + lane * rpitch, src + k0, bytes, router_full);
        }
    };
    if (warp == kProducerWarp) {
        if (lane == 0) {
            mbar_init(router_full, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        load_router(0);  // ahead of everything else
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], kConsumerWarps);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&part_full[i], kConsumerWarps);
                mbar_init(&part_free[i], 2);
            }
            mbar_init(h_ready, 1);
            info[2] = info[3] = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    __syncthreads();

    // The shared expert's entries come first: its units are dealt out before the routing is
    // known (from the last CTA on, as the others' are from the first: a CTA that gets one
    // more of these tends to get one less of those).
    const int shared_units = a.shared ? (T + 7) / 8 * upe : 0;
    const int sh0 = cut(shared_units, G - 1 - b, G), nsh = cut(shared_units, G - b, G) - sh0;
    int other0 = 0, nunits = nsh;  // first of the others, units in all
    // entry and 8-row block of this CTA's k-th unit
    auto unit_at = [&](int k, int& i, int& blk) {
        const int u = k < nsh ? sh0 + k : shared_units + other0 + k - nsh;
        i = (int)div_by((uint32_t)u, upe_m);
        blk = u - i * upe;
    };

    // producer: gate_up stage `st`.  Lane j loads the stage's j-th unit: 8 gate and 8
    // up rows, as many 256-k slices as the stage takes
    auto issue_gate_up = [&](uint32_t gs, int st, bool routed) {
        const int s = gs % kStages;
        const int k0 = NC == 1 ? st * ups : st / NC;
        const int sl0 = NC == 1 ? 0 : (st % NC) * kConsumerWarps;  // the stage's first slice
        const int n = min(ups, nunits - k0);
        const int whole = min(max(sg_whole - sl0, 0), kConsumerWarps);  // slices in the box
        const bool tail = sg_whole < sg && sg_whole - sl0 < kConsumerWarps;
        const uint32_t bytes =
            (uint32_t)(whole + (tail ? 1 : 0)) * kSlotBytes + (SF ? 16u * (uint32_t)sfp : 0u);
        if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)n * bytes);
        __syncwarp();
        if (lane < n) {
            int i, blk;
            unit_at(k0 + lane, i, blk);
            const int row = (routed ? (int)list_e[i] : a.E) * 2 * I + blk * 8;
            const uint32_t base = smem_u32(smem + s * kStageBytes);
            const uint32_t dst = base + (NC == 1 ? lane * sg : 0) * kSlotBytes;
            if (whole)
                tma_load_4d(dst, NC > 1 && sl0 > 0 ? &maps.w13_rest : &maps.w13, 0, row, 0, sl0, &full[s]);
            if (tail)
                tma_load_3d(dst + whole * kSlotBytes, &maps.w13_tail, sg_whole * 128, row, 0, &full[s]);
            if (SF)
                tma_load_3d(base + kCodeBytes + lane * 16 * sfp, &maps.s13, sl0 * 8, row, 0, &full[s]);
        }
        if (!SF && (NC == 1 || sl0 == 0)) {  // the units' scale rows, on their way into L2
            for (int q = lane; q < n * 16; q += 32) {
                int i, blk;
                unit_at(k0 + q / 16, i, blk);
                const int r = q % 16, row = blk * 8 + (r < 8 ? r : I + r - 8);
                const uint8_t* p = a.s13 + ((size_t)(routed ? (int)list_e[i] : a.E) * 2 * I + row) * KGH;
                for (int o = 0; o < KGH; o += 128) prefetch_l2(p + o);
            }
        }
        __syncwarp();
    };

    uint32_t gs = 0;  // stages issued (producer) or consumed so far

    if (warp == kProducerWarp) {
        // the router's further k, where all of it does not fit at once
        for (int k0 = a.router_k; k0 < H; k0 += a.router_k) {
            barrier_sync(3, kConsumers + 32);
            load_router(k0);
        }
        // whole stages of the shared expert's units need no routing (the ring is free once
        // the router has read it)
        barrier_sync(3, kConsumers + 32);
        const int stages = NC == 1 ? nsh / ups : nsh * NC;
        for (; (int)gs < min(stages, kEarlyStages); ++gs) issue_gate_up(gs, (int)gs, false);
    } else if (warp < kConsumerWarps) {
        // ------------------------------------------------------- router
        // each CTA multiplies a few rows of [Wr; gate], spread over the warps 32 k at a
        // time.  Equal rows give equal logits: every row's sums have one order.
        const int r = lane >> 2, c = lane & 3;
        float racc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        uint32_t xmax = 0;  // the largest |x| of token `warp`
        bool router_ok = true;
        for (int k0 = 0, u = 0; k0 < H; k0 += a.router_k, ++u) {
            const int kg = min(a.router_k, H - k0) / 32;
            if (u) {  // the last piece has been read: the next may take its place
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                barrier_arrive(3, kConsumers + 32);
            }
            router_ok = router_ok && mbar_wait_warp(router_full, u & 1);
            if (!router_ok) continue;
            const uint32_t base = smem_u32(smem) + 16 * c, xs = base + rows * rpitch;
            // (rows and tokens that do not exist: the first one, not used)
            const uint32_t wa = base + (r < rows ? r : 0) * rpitch, wb = base + (r + 8 < rows ? r + 8 : 0) * rpitch;
            const uint32_t xa = xs + (r < T ? r : 0) * rpitch, xb = xs + (8 + r < T ? 8 + r : 0) * rpitch;
            if (rows > 0) {
#pragma unroll 2
                for (int g = warp; g < kg; g += kConsumerWarps) {
                    const uint4 va = lds128(wa + 64 * g), vb = lds128(wb + 64 * g);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (n && T <= 8) break;
                        float t4[4];
                        mma_bf16_32(t4, va, vb, lds128((n ? xb : xa) + 64 * g));
#pragma unroll
                        for (int i = 0; i < 4; ++i) racc[n][i] += t4[i];
                    }
                }
            }
            if (warp < T) {
                const uint32_t xr = smem_u32(smem) + (rows + warp) * rpitch;
#pragma unroll 4
                for (int q = lane; q < kg * 4; q += 32) {
                    const uint4 v = lds128(xr + 16 * q);
                    const uint32_t xx[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) xmax = max(xmax, max(xx[i] & 0x7FFFu, (xx[i] >> 16) & 0x7FFFu));
                }
            }
        }
        xmax = __reduce_max_sync(0xFFFFFFFFu, xmax);
        // the power of two that scales token `warp`
        if (warp < T && lane == 0) rscale[warp] = __uint_as_float((uint32_t)(127 - row_f16_shift(xmax)) << 23);
#pragma unroll
        for (int n = 0; n < 2; ++n)
            part[(n * kConsumerWarps + warp) * 32 + lane] = make_float4(racc[n][0], racc[n][1], racc[n][2], racc[n][3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring goes back to the TMA
        consumers_sync();
        if (tid < 256) {  // one (row, token) each
            const float* p = reinterpret_cast<const float*>(part) + (tid >> 7) * kConsumerWarps * 128 + (tid & 127);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kConsumerWarps; ++w) v += p[w * 128];
            const int l = (tid & 127) >> 2, q = tid & 3;
            const int row = (l >> 2) + (q & 2 ? 8 : 0), t = 8 * (tid >> 7) + 2 * (l & 3) + (q & 1);
            if (row < rows && t < T) a.logits[(size_t)t * (a.E + 1) + row0 + row] = v;
        }
        barrier_arrive(3, kConsumers + 32);
        // what gate_up raises starts at zero
        for (int i = b * kConsumers + tid; i < T * Kt; i += G * kConsumers) a.hmax[i] = 0u;
        consumers_sync();
        if (tid == 0) add_release(&a.sync[0]);

        // while the others finish: the masks' zeros
        uint32_t* mask = reinterpret_cast<uint32_t*>(smem + kMask);
        uint16_t* first = reinterpret_cast<uint16_t*>(smem + kFirst);
        int32_t* ids_s = reinterpret_cast<int32_t*>(smem + kIds);
        float* logit_s = reinterpret_cast<float*>(smem + kEarlyStages * kStageBytes);  // [T][E]
        for (int e = tid; e < Et; e += kConsumers) mask[e] = 0u;
        if (tid == 0) info[1] = router_ok && grid_wait(&a.sync[0], (uint32_t)G) ? 1 : 0;
        consumers_sync();

        // ------------------------------------------------------ routing
        // every CTA routes all tokens, one warp each, and builds the same list
        if (info[1]) {
            // (loads are kept few in the code: a call runs every line of it once or twice,
            // and fetching straight-line code costs more than running it)
#pragma unroll 4
            for (int q = tid; q < T * a.E; q += kConsumers) {
                const int t = (int)div_by((uint32_t)q, a.e_m);
                logit_s[q] = __ldcg(a.logits + q + t);  // written by this kernel: read from L2
            }
            consumers_sync();
            if (warp < T) {
                const float* l = logit_s + warp * a.E;
                const float sw = a.gate ? 1.0f / (1.0f + expf(-__ldcg(a.logits + (size_t)warp * (a.E + 1) + a.E))) : 1.0f;
                int32_t* wi = ids_s + warp * 33;
                float* ww = w_s + warp * Kt;
                if (a.E <= 128)
                    route_few<4>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
                else if (a.E <= 512)
                    route_few<16>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
                else
                    route_few<32>(l, a.E, a.K, a.shared, a.renorm, sw, wi, ww, lane);
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
            // lists: the shared expert first, then the touched routed ones by id;
            // warp w orders experts 64 w .. 64 w + 63.  An expert's pairs, its entries of down
            // and of gate_up are counted together, in 12, 10 and 10 bits (at most 528, 516, 516)
            uint32_t* sums = reinterpret_cast<uint32_t*>(smem + kSums);  // by warp
            auto counts = [](int n) { return (uint32_t)n | (uint32_t)((n + 3) / 4) << 12 | (uint32_t)((n + 7) / 8) << 22; };
            uint32_t at[2], mk[2], run = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 64 * warp + 32 * i + lane;
                mk[i] = e < a.E ? mask[e] : 0u;
                const uint32_t own = counts(__popc(mk[i]));
                uint32_t v = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                    if (lane >= o) v += u;
                }
                at[i] = run + v - own;
                run += __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (lane == 0) sums[warp] = run;
            consumers_sync();
            uint32_t before = a.shared ? counts(T) : 0u, total = before;
            for (int i = 0; i < kConsumerWarps; ++i) {
                if (i < warp) before += sums[i];
                total += sums[i];
            }
            // expert e with n tokens, `c` counted before it (unrolled, these loops cost a call of one
            // token 0.8 us in instruction fetches)
            auto enter = [&](int e, uint32_t c, int n) {
                const int p = c & 4095u, d = (c >> 12) & 1023u, g = c >> 22;
#pragma unroll 1
                for (int j = 0; j < n; j += 8) {
                    list_e[g + j / 8] = (uint16_t)e;
                    list_p[g + j / 8] = (uint16_t)((p + j) << 4 | min(n - j, 8));
                }
#pragma unroll 1
                for (int j = 0; j < n; j += 4) {
                    down_e[d + j / 4] = (uint16_t)e;
                    down_p[d + j / 4] = (uint16_t)((p + j) << 4 | min(n - j, 4));
                }
                first[e] = (uint16_t)p;
            };
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (mk[i]) enter(64 * warp + 32 * i + lane, before + at[i], __popc(mk[i]));
            if (tid == 0) {
                info[0] = (int)(total >> 22);
                info[4] = (int)((total >> 12) & 1023u);
                if (a.shared) enter(a.E, 0, T);
            }
            consumers_sync();
            for (int i = tid; i < T * Kt; i += kConsumers) {
                const int t = i / Kt, e = ids_s[t * 33 + i - t * Kt];
                const int p = first[e] + __popc(mask[e] & ((1u << t) - 1u));
                pair_of[i] = (uint16_t)p;
                pair_t[p] = (uint8_t)t;
            }
            // the logits' place in shared memory goes back to the TMA
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
    }
    __syncthreads();  // the list is there (or the barrier gave up)

    const bool routed = info[1] != 0;
    const int nent = routed ? info[0] : 0, ndown = routed ? info[4] : 0;
    const int others = max(nent * upe - shared_units, 0);
    other0 = cut(others, b, G);
    nunits = routed ? nsh + cut(others, b + 1, G) - other0 : 0;
    const int gstages = NC == 1 ? (nunits + ups - 1) / ups : nunits * NC;
    // down: items (entry, 16 output rows) in that order, cut into one range per CTA
    const int items = RU * ndown;
    const int lo = cut(items, b, G), hi = cut(items, b + 1, G);
    const int dstages = (hi - lo + ips - 1) / ips * spi;
    // the stages of a phase are consumed in pairs (a unit's or item's two stages, or two
    // independent ones), each handing one buffer of sums over to the epilogue
    const int ghands = (gstages + 1) / 2, dhands = (dstages + 1) / 2;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------- producer
        bool ok = routed;
        for (; (int)gs < gstages && ok; ++gs) {
            if (gs >= (uint32_t)kStages && !mbar_wait_warp(&empty[gs % kStages], ((gs / kStages) - 1) & 1)) {
                ok = false;
                break;
            }
            issue_gate_up(gs, (int)gs, true);
        }
        for (int st = 0; st < dstages && ok; ++st, ++gs) {
            const int s = gs % kStages;
            if (gs >= (uint32_t)kStages && !mbar_wait_warp(&empty[s], ((gs / kStages) - 1) & 1)) {
                ok = false;
                break;
            }
            const int it0 = lo + (spi > 1 ? st / spi : st * ips), sl0 = (st % spi) * kConsumerWarps;
            const int n = min(ips, hi - it0);
            const int whole = min(max(sd_whole - sl0, 0), kConsumerWarps);
            const bool tail = sd_whole < sd && sd_whole - sl0 < kConsumerWarps;
            const uint32_t bytes =
                (uint32_t)(whole + (tail ? 1 : 0)) * kSlotBytes + (SF ? 16u * (uint32_t)sfp2 : 0u);
            if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)n * bytes);
            __syncwarp();
            if (lane < n) {
                const int i = (int)div_by((uint32_t)(it0 + lane), ru_m);
                const int row = (int)down_e[i] * H + (it0 + lane - i * RU) * 16;
                const uint32_t base = smem_u32(smem + s * kStageBytes);
                const uint32_t dst = base + (spi > 1 ? 0 : lane * sd) * kSlotBytes;
                if (whole) tma_load_3d(dst, sl0 > 0 ? &maps.w2_rest : &maps.w2, 0, row, sl0, &full[s]);
                if (tail) tma_load_2d(dst + whole * kSlotBytes, &maps.w2_tail, sd_whole * 128, row, &full[s]);
                if (SF) tma_load_2d(base + kCodeBytes + lane * 16 * sfp2, &maps.s2, sl0 * 8, row, &full[s]);
            }
            if (!SF && sl0 == 0) {
                for (int q = lane; q < n * 16; q += 32) {
                    const int it = it0 + q / 16, i = (int)div_by((uint32_t)it, ru_m);
                    const uint8_t* p = a.s2 + ((size_t)down_e[i] * H + (it - i * RU) * 16 + q % 16) * KGI;
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
        const uint32_t ring = smem_u32(smem);
        bool failed = !routed;

        // the pair's sums to the epilogue: hand-over h, acc[i] of its i-th stage (or, if
        // `one`, acc[0] of both)
        auto hand_over = [&](int h, const float (&acc)[2][4], bool one) {
            const int buf = h & 1;
            if (!failed && h >= 2 && !mbar_wait_warp(&part_free[buf], ((h >> 1) - 1) & 1)) failed = true;
            if (!failed) {
                float4* p = part + (buf * 2 * kConsumerWarps + warp) * 32 + lane;
                p[0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
                if (!one)
                    p[kConsumerWarps * 32] = make_float4(acc[1][0], acc[1][1], acc[1][2], acc[1][3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_full[buf]);
        };
        // stage st's slot of this warp times b.  Lane 2 q + z turns the scale bytes 4 z .. of
        // the slot's row q into factors: from the stage (byte raw on), or from word w
        const uint32_t fac = smem_u32(smem + kFactors) + warp * 1024;  // two slots' factors
        auto multiply = [&](int st, bool on, uint32_t raw, uint32_t w, const uint4 (&b)[8], float (&acc)[4]) {
            const uint32_t stage = ring + (st % kStages) * kStageBytes;
            if (!failed && !mbar_wait_warp(&full[st % kStages], (st / kStages) & 1)) failed = true;
            if (!failed && on) {
                const uint32_t f = fac + (st & 1) * 512;
                sts_f4(f + 16 * lane, factors(SF ? lds32(stage + kCodeBytes + raw) : w));
                __syncwarp();
                slot_mma(stage + warp * kSlotBytes, lm, f + 32 * r, b, acc);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st % kStages]);
        };

        // -------------------------------------------------------- gate_up
        {
            const int j = NC == 1 ? warp / sg : 0;          // this warp's unit within a stage
            const int q0 = NC == 1 ? warp - j * sg : warp;  // and its (first) slice
            uint4 xb[NC][8];
            int have = -1;  // the entry whose x fragment is in xb
            auto load_x = [&](int i) {
                const int n = list_p[i] & 15, p = list_p[i] >> 4;
                const int t = r < n ? (int)pair_t[p + r] : 0;
                const float up = 1.0f / rscale[t];  // 2^sigma, exact
                const uint16_t* xr = a.x + (size_t)t * H;
#pragma unroll
                for (int f = 0; f < NC; ++f)
#pragma unroll
                    for (int gl = 0; gl < 8; ++gl) {
                        const int k = (q0 + f * kConsumerWarps) * 256 + 32 * gl + 8 * c;
                        xb[f][gl] = r < n && k < H ? __ldg(reinterpret_cast<const uint4*>(xr + k)) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                for (int f = 0; f < NC; ++f)
#pragma unroll
                    for (int gl = 0; gl < 8; ++gl) {
                        const uint4 q = xb[f][gl];
                        xb[f][gl] = make_uint4(bf16x2_to_f16x2_scaled(q.x, up), bf16x2_to_f16x2_scaled(q.y, up),
                                               bf16x2_to_f16x2_scaled(q.z, up), bf16x2_to_f16x2_scaled(q.w, up));
                    }
                have = i;
            };
            // where this lane's scale word lies: row lane / 2 of the slot, groups 4 (lane % 2) ..
            const int srow = lane >> 1, sgrp = 4 * (lane & 1);
            const uint32_t raw = (uint32_t)((j * 16 + srow) * sfp + q0 * 8 + sgrp);
            const size_t words = (size_t)Et * 2 * I * KGH / 4;
            uint32_t sw[2] = {0, 0};
            auto load_sw = [&](int h) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = NC == 1 ? (2 * h + i) * ups + j : h, grp = (q0 + (NC == 1 ? 0 : i * kConsumerWarps)) * 8 + sgrp;
                    sw[i] = 0;
                    if (SF || j >= ups || k >= nunits || grp >= KGH) continue;
                    int e, blk;
                    unit_at(k, e, blk);
                    const int row = blk * 8 + (srow < 8 ? srow : I + srow - 8);
                    sw[i] = load_scales(a.s13, ((size_t)list_e[e] * 2 * I + row) * KGH + grp, KGH - grp, words);
                }
            };
            load_sw(0);
            for (int h = 0; h < ghands; ++h) {
                float acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                const uint32_t w[2] = {sw[0], sw[1]};
                load_sw(h + 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int st = 2 * h + i, k = NC == 1 ? st * ups + j : h;
                    if (st >= gstages) break;
                    const bool on = j < ups && k < nunits && q0 + (NC == 1 ? 0 : i * kConsumerWarps) < sg;
                    if (on && !failed) {
                        int e, blk;
                        unit_at(k, e, blk);
                        if (e != have) load_x(e);
                    }
                    multiply(st, on, raw, w[i], xb[NC == 1 ? 0 : i], acc[NC == 1 ? i : 0]);
                }
                hand_over(h, acc, NC > 1);
            }
        }
        // ----------------------------------------------------------- down
        {
            const int j = spi > 1 ? 0 : warp / sd;          // this warp's item within a stage
            const int q0 = spi > 1 ? warp : warp - j * sd;  // and its (first) slice
            const int hpitch = shift_pitch(I);
            uint4 hb[8];
            int have = -1;  // entry (times stages per item, plus the chunk) whose h fragment is in hb
            // column r: term r / 4 of h of the entry's token r % 4, with one power of two for
            // the row: each 8 values' own shift comes down to the row's
            auto load_h = [&](int i, int slice, int key) {
                const int n = down_p[i] & 15, p = (down_p[i] >> 4) + (r & 3);
                have = key;
#pragma unroll
                for (int gl = 0; gl < 8; ++gl) hb[gl] = make_uint4(0, 0, 0, 0);
                if ((r & 3) >= n) return;
                const uint16_t* hp = a.h + (size_t)(2 * p + (r >> 2)) * I + 256 * slice + 8 * c;
#pragma unroll
                for (int gl = 0; gl < 8; ++gl)
                    if (256 * slice + 32 * gl < I) hb[gl] = __ldcg(reinterpret_cast<const uint4*>(hp + 32 * gl));
                const uint2 us = __ldcg(reinterpret_cast<const uint2*>(a.hshift + (size_t)p * hpitch + 32 * slice + 8 * c));
                const int sh = f32_f16_shift(__ldcg(a.hmax + p));
#pragma unroll
                for (int gl = 0; gl < 8; ++gl) {
                    if (256 * slice + 32 * gl >= I) break;
                    const int u = (int)(int8_t)((gl < 4 ? us.x : us.y) >> (8 * (gl & 3)));
                    const __half2 g = __float2half2_rn(__uint_as_float((uint32_t)max(127 + sh - u, 0) << 23));
                    __half2* w = reinterpret_cast<__half2*>(&hb[gl]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q] = __hmul2(w[q], g);
                }
            };
            const int srow = lane >> 1, sgrp = 4 * (lane & 1);
            const uint32_t raw = (uint32_t)((j * 16 + srow) * sfp2 + q0 * 8 + sgrp);
            const size_t words = (size_t)Et * H * KGI / 4;
            uint32_t sw[2] = {0, 0};
            auto load_sw = [&](int h) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int item = lo + (spi > 1 ? h : (2 * h + i) * ips + j), grp = (q0 + (spi > 1 ? i * kConsumerWarps : 0)) * 8 + sgrp;
                    sw[i] = 0;
                    if (SF || j >= ips || item >= hi || grp >= KGI) continue;
                    const int e = (int)div_by((uint32_t)item, ru_m);
                    sw[i] = load_scales(a.s2, ((size_t)down_e[e] * H + (item - e * RU) * 16 + srow) * KGI + grp, KGI - grp, words);
                }
            };
            load_sw(0);
            if (!failed && !mbar_wait_warp(h_ready, 0)) failed = true;
            if (!failed && !info[2]) failed = true;
            for (int h = 0; h < dhands; ++h) {
                float acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                const uint32_t w[2] = {sw[0], sw[1]};
                load_sw(h + 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int st = 2 * h + i;
                    if (st >= dstages) break;
                    const int slice = q0 + (spi > 1 ? i * kConsumerWarps : 0);
                    const int item = lo + (spi > 1 ? h : st * ips + j);
                    const bool on = j < ips && item < hi && slice < sd;
                    if (on && !failed) {
                        const int e = (int)div_by((uint32_t)item, ru_m), key = e * spi + (spi > 1 ? i : 0);
                        if (key != have) load_h(e, slice, key);
                    }
                    if (spi == 1)
                        multiply(gstages + st, on, raw, w[i], hb, acc[i]);
                    else
                        multiply(gstages + st, on, raw, w[i], hb, acc[0]);
                }
                hand_over(ghands + h, acc, spi > 1);
            }
        }
    } else {
        // ------------------------------------------------------- epilogue
        // warp `me` takes the sums of a pair's stage `me` (the first one has those of
        // units and items of two stages)
        const int me = warp - kEpiWarp0, r = lane >> 2, c = lane & 3;
        const int hpitch = shift_pitch(I);
        bool ok = routed;
        // the sum of warps w0 .. w0 + n - 1: this lane's rows r and r + 8 (x, z for column
        // 2c, y, w for 2c + 1)
        auto sum_of = [&](int buf, int w0, int n) {
            float4 v = make_float4(0, 0, 0, 0);
            const float4* p = part + ((buf * 2 + me) * kConsumerWarps + w0) * 32 + lane;
#pragma unroll 4
            for (int w = 0; w < n; ++w) {
                const float4 q = p[w * 32];
                v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
            }
            return v;
        };
        for (int h = 0; h < ghands; ++h) {
            const int buf = h & 1;
            if (ok && !mbar_wait_warp(&part_full[buf], (h >> 1) & 1)) ok = false;
            if (!ok) break;
            for (int j = 0; j < ups; ++j) {
                const int k = NC == 1 ? (2 * h + me) * ups + j : (me ? nunits : h);
                if (k >= nunits) break;
                int i, blk;
                unit_at(k, i, blk);
                const int n = list_p[i] & 15, p0 = list_p[i] >> 4;
                const float4 v = NC == 1 ? sum_of(buf, j * sg, sg) : sum_of(buf, 0, kConsumerWarps);
                const float g[2] = {v.x, v.y}, up[2] = {v.z, v.w};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // this lane: row r of the unit's 8, pair p0 + 2c + q
                    const int p = p0 + 2 * c + q;
                    const bool on = 2 * c + q < n;
                    const float rs = on ? rscale[pair_t[p]] : 0.0f;
                    const float hv = on ? silu(g[q] * rs) * (up[q] * rs) : 0.0f;
                    uint32_t mx = __float_as_uint(hv) & 0x7FFFFFFFu;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                    if (on) {
                        const int sh = f32_f16_shift(mx);
                        const float s = hv * __uint_as_float((uint32_t)(127 + sh) << 23);
                        const __half hi = __float2half_rn(s);
                        // (nothing is left next to an infinity)
                        const __half lo = __float2half_rn(fabsf(s) < 65504.0f ? s - __half2float(hi) : 0.0f);
                        uint16_t* h = a.h + (size_t)(2 * p) * I + blk * 8 + r;
                        h[0] = __half_as_ushort(hi);
                        h[I] = __half_as_ushort(lo);
                        if (r == 0) {
                            // (eight zeros: a shift so high that they come down to zero)
                            a.hshift[(size_t)p * hpitch + shift_at(blk)] = (int8_t)(mx ? sh : 127);
                            atomicMax(a.hmax + p, mx);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_free[buf]);
        }
        // h of this CTA is complete; wait for everybody's
        ok = all_at_barrier(ok, 2, 64);
        if (me == 0 && lane == 0) {
            if (ok) {
                add_release(&a.sync[1]);
                if (grid_wait(&a.sync[1], (uint32_t)G)) info[2] = 1;
            }
            mbar_arrive(h_ready);
        }
        if (ok && !mbar_wait_warp(h_ready, 0)) ok = false;
        ok = ok && info[2];

        int have = -1;
        float f[2] = {0, 0};  // 2^-sigma of the pairs in columns 2c and 2c + 1
        for (int h = 0; h < dhands; ++h) {
            const int buf = (ghands + h) & 1;
            if (ok && !mbar_wait_warp(&part_full[buf], ((ghands + h) >> 1) & 1)) ok = false;
            if (!ok) break;
            for (int j = 0; j < ips; ++j) {
                const int item = spi == 1 ? lo + (2 * h + me) * ips + j : (me ? hi : lo + h);
                if (item >= hi) break;
                const int i = (int)div_by((uint32_t)item, ru_m);
                // this lane's columns 2c and 2c + 1: tokens (c < 2), or the rest terms of lane
                // c - 2's, which are added to those
                const int n = down_p[i] & 15, p = (down_p[i] >> 4) + 2 * c;
                if (i != have) {
                    have = i;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (2 * c + q < n)
                            f[q] = __uint_as_float((uint32_t)(127 - f32_f16_shift(__ldcg(a.hmax + p + q))) << 23);
                }
                float4 v = spi == 1 ? sum_of(buf, j * sd, sd) : sum_of(buf, 0, kConsumerWarps);
                v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, 2), v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, 2);
                v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, 2), v.w += __shfl_xor_sync(0xFFFFFFFFu, v.w, 2);
                float* y = a.y + (size_t)p * H + (item - i * RU) * 16 + r;
                if (2 * c < n) {
                    __stcg(y, v.x * f[0]);
                    __stcg(y + 8, v.z * f[0]);
                }
                if (2 * c + 1 < n) {
                    __stcg(y + H, v.y * f[1]);
                    __stcg(y + H + 8, v.w * f[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_free[buf]);
        }
        if (!ok && lane == 0) info[2] = 0;
    }

    // ------------------------------------------------------------ weighted sum
    // once every CTA's y is there, each CTA adds up its share of the outputs
    __syncthreads();
    if (tid == 0 && info[2]) {
        add_release(&a.sync[2]);
        info[3] = grid_wait(&a.sync[2], (uint32_t)G) ? 1 : 0;
        // the last CTA past this barrier leaves the counters at zero
        if (info[3] && add_release(&a.sync[3]) == (uint32_t)G - 1)
            a.sync[0] = a.sync[1] = a.sync[2] = a.sync[3] = 0u;
    }
    __syncthreads();
    if (info[3]) {
        const int n = T * H, q1 = cut(n, b + 1, G);
        for (int q = cut(n, b, G) + tid; q < q1; q += kThreads) {
            const int t = q / H, row = q - t * H;
            float v = 0.0f;
            for (int j0 = 0; j0 < Kt; j0 += 12) {  // (the loads of twelve slots together)
                float y[12];
#pragma unroll
                for (int j = 0; j < 12; ++j)
                    y[j] = __ldcg(a.y + (size_t)pair_of[t * Kt + min(j0 + j, Kt - 1)] * H + row);
#pragma unroll
                for (int j = 0; j < 12; ++j)
                    if (j0 + j < Kt) v = fmaf(w_s[t * Kt + j0 + j], y[j], v);
            }
            a.out[q] = f32_to_bf16_bits(v);
        }
    }
    pdl_end();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct FewWorkspace {
    size_t sync, logits, hmax, h, hshift, y, total;
};

FewWorkspace few_workspace(int T, int H, int I, int E, int Kt) {
    const size_t pairs = (size_t)T * Kt;
    FewWorkspace w;
    w.sync = 0;
    w.logits = 256;
    w.hmax = w.logits + align256((size_t)T * (E + 1) * 4);
    w.h = w.hmax + align256(pairs * 4);
    w.hshift = w.h + align256(pairs * I * 2 * 2);
    w.y = w.hshift + align256(pairs * shift_pitch(I));
    w.total = w.y + align256(pairs * H * 4);
    return w;
}

// The maps of FewMaps; those that no load uses stay empty.
cudaError_t few_maps(const LayerFew& p, bool scales, FewMaps* m) {
    const uint64_t Et = (uint64_t)p.E + p.shared, H = p.H, I = p.I;
    const uint32_t sg = (uint32_t)p.H / 256, sd = (uint32_t)p.I / 256, most = kConsumerWarps;
    cudaError_t err = cudaSuccess;
    memset(m, 0, sizeof(*m));
    {  // {128 bytes, row, gate or up, slice}
        const uint64_t dims[4] = {128, Et * 2 * I - I, 2, sg}, strides[3] = {H / 2, I * (H / 2), 128};
        const uint32_t box[4] = {128, 8, 2, std::min(sg, most)}, rest[4] = {128, 8, 2, sg - most};
        if (sg > 0) err = encode_nd_map(&m->w13, p.w13, 4, dims, strides, box, true);
        if (err == cudaSuccess && sg > most) err = encode_nd_map(&m->w13_rest, p.w13, 4, dims, strides, rest, true);
    }
    if (err == cudaSuccess && p.H % 256) {  // {byte of the row, row, gate or up}
        const uint64_t dims[3] = {H / 2, Et * 2 * I - I, 2}, strides[2] = {H / 2, I * (H / 2)};
        const uint32_t box[3] = {128, 8, 2};
        err = encode_nd_map(&m->w13_tail, p.w13, 3, dims, strides, box, true);
    }
    if (err == cudaSuccess && scales) {  // {scale byte, row, gate or up}
        const uint64_t dims[3] = {H / 32, Et * 2 * I - I, 2}, strides[2] = {H / 32, I * (H / 32)};
        const uint32_t box[3] = {(uint32_t)std::min<uint64_t>(H / 32, 128), 8, 2};
        err = encode_nd_map(&m->s13, p.s13, 3, dims, strides, box, false);
    }
    {  // {128 bytes, row, slice}
        const uint64_t dims[3] = {128, Et * H, sd}, strides[2] = {I / 2, 128};
        const uint32_t box[3] = {128, 16, std::min(sd, most)}, rest[3] = {128, 16, sd - most};
        if (err == cudaSuccess && sd > 0) err = encode_nd_map(&m->w2, p.w2, 3, dims, strides, box, true);
        if (err == cudaSuccess && sd > most) err = encode_nd_map(&m->w2_rest, p.w2, 3, dims, strides, rest, true);
    }
    if (err == cudaSuccess && p.I % 256) err = encode_codes_map(&m->w2_tail, p.w2, p.I / 2, Et * H, 128, 16);
    if (err == cudaSuccess && scales) {
        const uint64_t dims[2] = {I / 32, Et * H}, strides[1] = {I / 32};
        const uint32_t box[2] = {(uint32_t)std::min<uint64_t>(I / 32, 128), 16};
        err = encode_nd_map(&m->s2, p.s2, 2, dims, strides, box, false);
    }
    return err;
}

template <int NC, bool SF>
cudaError_t launch_few(const FewArgs& a, const FewMaps& maps, int grid, cudaStream_t s) {
    cudaError_t err = ensure_dynamic_smem((const void*)layer_few_kernel<NC, SF>, kSmemBytes);
    if (err != cudaSuccess) return err;
    // cooperative: the grid's CTAs wait for one another, so all must be resident
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_few_kernel<NC, SF>, a, maps);
}

}  // namespace

size_t layer_few_workspace(int T, int H, int I, int E, int Kt) { return few_workspace(T, H, I, E, Kt).total; }

cudaError_t launch_layer_few(const LayerFew& p, void* workspace, cudaStream_t s) {
    const int Kt = p.K + p.shared;
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
    a.h = reinterpret_cast<uint16_t*>(ws + L.h);
    a.hshift = reinterpret_cast<int8_t*>(ws + L.hshift);
    a.y = reinterpret_cast<float*>(ws + L.y);
    a.T = p.T;
    a.H = p.H;
    a.I = p.I;
    a.E = p.E;
    a.K = p.K;
    a.shared = p.shared;
    a.renorm = p.renormalize;
    // scale rows that the TMA can read: whole 16-byte units
    const bool sf = p.H % 512 == 0 && p.I % 512 == 0 && ((uintptr_t)p.s13 | (uintptr_t)p.s2) % 16 == 0;
    const int sg = (p.H + 255) / 256, sd = (p.I + 255) / 256;
    a.ups = sg <= kConsumerWarps ? kConsumerWarps / sg : 1;
    a.ips = sd <= kConsumerWarps ? kConsumerWarps / sd : 1;
    a.upe_m = div_magic((uint32_t)p.I / 8);
    a.ru_m = div_magic((uint32_t)p.H / 16);
    a.e_m = div_magic((uint32_t)p.E);
    FewMaps maps;
    cudaError_t err = few_maps(p, sf, &maps);
    if (err != cudaSuccess) return err;
    // no more CTAs than the widest phase has pieces of work for (a barrier of
    // fewer CTAs is shorter)
    const long long touched = std::min<long long>((long long)p.T * p.K, p.E) + p.shared;
    const int rows = p.E + (p.w_shared_gate ? 1 : 0);
    const long long work = std::max({(long long)rows, touched * (p.I / 8), (long long)(p.H / 16) * touched});
    const int grid = (int)std::min<long long>({work, (long long)num_sms(), (long long)kMaxGrid});
    a.router_rows = (rows + grid - 1) / grid;
    if (a.router_rows > 16) return cudaErrorNotSupported;  // fewer than 65 SMs
    // as many k as the ring holds of the rows and the tokens (whole groups of 32)
    a.router_k = std::min(p.H, ((kStages * kStageBytes / (a.router_rows + p.T) - 64) / 2) & ~31);
    if (p.H > 4096) return sf ? launch_few<2, true>(a, maps, grid, s) : launch_few<2, false>(a, maps, grid, s);
    return sf ? launch_few<1, true>(a, maps, grid, s) : launch_few<1, false>(a, maps, grid, s);
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
