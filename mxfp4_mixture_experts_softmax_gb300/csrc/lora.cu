// lora.cu -- low-rank adapters of many requests beside a shared projection:
//
//   out[t] = residual[t] + scale[a] * B[a] (A[a] x_t)      a = the adapter of token t
//   out[t] = residual[t]                                   for a token without one
//
// One launch, no workspace.  A cluster of CTAs takes 16 tokens of one adapter (moe_permute's grouping).  Its
// CTAs split the sum over K (v = A x), join their parts through distributed shared memory in rank order, and
// split the N outputs.  x and the residual are read once, out is written once, and v never leaves the chip; A
// and B are read once per 16 tokens, from L2 after the first.  It is bound by latency for few tokens and by the
// weights of all their adapters for more: 64 tokens with 64 adapters of rank 16 at 4096 x 8192 take 10.0 us in a graph
// with the weights in L2 and 12.0 with weights from HBM (26 MB: 2.2 TB/s).  Long prompts of one adapter go to lora_prompt.cu where they can.
//
// The products run as warp MMAs (bf16, m16n8k16) straight from global memory into registers.  Both operands
// of an MMA may permute their k alike, so a lane takes 8 neighbouring k of a row (16 bytes) as its four k of
// two MMAs, and neighbouring output columns likewise.  What bounds such code is how many loads a warp has on their
// way, so none of them stands behind a choice (loads inside branches, each waited for there: 14.9 us for
// the 64 tokens above), and two blocks fit an SM (128 registers a thread; with one: 18.6 -> 31 us at rank 64).
//
// Products are exact: bf16 times bf16, an fp32 x as three bf16 terms.  Sums are fp32.
// v, an fp32 sum, enters the second product as bf16 terms: two for a bf16 output (2^-16 of
// v, a hundredth of the output's own rounding), three for fp32 (2^-24).
#include <algorithm>

#include "lora_device.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTokens = 16;  // that a cluster takes at a time: one MMA's rows

__device__ __forceinline__ void mma_bf16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

// Eight fp32 values as three words-of-two-bf16 terms each: v = t[0] + t[1] + t[2] exactly.
__device__ __forceinline__ void split8(const float* v, uint32_t t[3][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[2][3];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float r = split_bf16(v[2 * i + k], w[k][0]);
            const float r2 = split_bf16(r, w[k][1]);
            w[k][2] = __float_as_uint(r2) >> 16;
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) t[j][i] = w[0][j] | (w[1][j] << 16);
    }
}

// Eight values of a row of x from element k on, as bf16 words (bf16 rows) or as they are.
template <bool F32>
struct Chunk {
    uint32_t w[F32 ? 8 : 4];
};

template <bool F32>
__device__ __forceinline__ void load_x(Chunk<F32>& c, const void* row, int k, bool wide) {
    constexpr int W = F32 ? 8 : 4;
    if (wide) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)k * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 v = __ldg(q + i);
            c.w[4 * i] = v.x, c.w[4 * i + 1] = v.y, c.w[4 * i + 2] = v.z, c.w[4 * i + 3] = v.w;
        }
    } else if (F32) {
        const uint32_t* q = static_cast<const uint32_t*>(row) + k;
#pragma unroll
        for (int i = 0; i < 8; ++i) c.w[i & (W - 1)] = __ldg(q + i);
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(row) + k;
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __ldg(q + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) c.w[i] = h[2 * i] | (h[2 * i + 1] << 16);
    }
}

// The first n of the bf16 in W words, zeros behind them.
template <int W>
__device__ __forceinline__ void keep_first(uint32_t* w, int n) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = n >= 2 * i + 2 ? w[i] : n == 2 * i + 1 ? w[i] & 0xFFFFu : 0u;
}

template <int RT>
struct Shape {
    static constexpr int kRanks = 8 * RT;
    // fp32 rows of v: 8 floats of padding put the four rows of a half-warp's stores in separate banks
    static constexpr int kPart = kRanks + 8;
    // bf16 rows of v's terms: the two rows of eight lanes' 16-byte reads fall in separate halves of the banks
    static constexpr int kTerm = kRanks <= 32 ? kRanks : kRanks + 32;
    static constexpr int kPartFloats = kWarps * kTokens * kPart;
    static constexpr int kTermHalves = kTokens * kTerm;
    // v's terms take the place of its parts, which are done with by then
    static constexpr size_t kBytes = (size_t)kPartFloats * 4 + (size_t)kTokens * kPart * 4;
    static_assert(3 * kTermHalves * 2 <= kPartFloats * 4, "v's terms do not fit over its parts");
};

// v's parts: the 16 tokens times all ranks over this warp's units of 32 k.
template <int RT, bool XF32>
__device__ __forceinline__ void shrink(const Lora& p, const uint16_t* a, const int* tok, int cta, int ctas,
                                       float* part) {
    using S = Shape<RT>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int units = (p.K + 31) / 32;
    const int u0 = (int)((long long)units * cta / ctas), u1 = (int)((long long)units * (cta + 1) / ctas);
    // All loads are made, so that they are on their way together: a row without a token reads another's (its
    // outputs go nowhere), a k behind the last reads before it and counts as 0, and so do a rank's
    // sums behind the adapter's.
    const void* row[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        row[i] = static_cast<const uint8_t*>(p.x) + (size_t)max(tok[i * 8 + g], 0) * p.ldx * (XF32 ? 4 : 2);
    float acc[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = 0.0f;

    constexpr int kAhead = RT <= 4 ? 4 : 2;
#pragma unroll kAhead
    for (int u = u0 + warp; u < u1; u += kWarps) {
        const bool in = u * 32 + 8 * tq < p.K;
        const int k = in ? u * 32 + 8 * tq : p.K - 8;
        Chunk<XF32> x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) load_x<XF32>(x[i], row[i], k, p.x_wide);
        uint4 w[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            w[r] = __ldg(reinterpret_cast<const uint4*>(a + (size_t)min(r * 8 + g, p.R - 1) * p.K + k));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < (XF32 ? 8 : 4); ++j) x[i].w[j] = in ? x[i].w[j] : 0u;
        if constexpr (XF32) {
            uint32_t lo[3][4], hi[3][4];  // rows g and g + 8
            split8(reinterpret_cast<const float*>(x[0].w), lo);
            split8(reinterpret_cast<const float*>(x[1].w), hi);
#pragma unroll
            for (int j = 2; j >= 0; --j)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    mma_bf16(acc[r], lo[j][0], hi[j][0], lo[j][1], hi[j][1], w[r].x, w[r].y);
                    mma_bf16(acc[r], lo[j][2], hi[j][2], lo[j][3], hi[j][3], w[r].z, w[r].w);
                }
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t *lo = x[0].w, *hi = x[1].w;
                mma_bf16(acc[r], lo[0], hi[0], lo[1], hi[1], w[r].x, w[r].y);
                mma_bf16(acc[r], lo[2], hi[2], lo[3], hi[3], w[r].z, w[r].w);
            }
        }
    }
    float* mine = part + (size_t)warp * kTokens * S::kPart + g * S::kPart + 2 * tq;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        *reinterpret_cast<float2*>(mine + r * 8) = make_float2(acc[r][0], acc[r][1]);
        *reinterpret_cast<float2*>(mine + r * 8 + 8 * S::kPart) = make_float2(acc[r][2], acc[r][3]);
    }
}

// The residual of a unit of 32 columns and 16 rows, as it lies in memory (what is made of it would wait for it).
// Wide rows: eight neighbouring columns of rows g and g + 8 a lane.  Others pass in turns of Q rows, Q = 4, 2 or 1
// neighbouring columns of a row a lane (p.vec: as many as rows' addresses allow; fp32: 1).
// What there is no token or no column for is read elsewhere in the residual, and goes nowhere.
constexpr int kStagePitch = 36;
struct Residual {
    uint32_t w[16];
    template <int Q>
    __device__ __forceinline__ void load_turns(const Lora& p, const int* tok, int at) {
        const int lane = threadIdx.x & 31, sub = lane / (32 / Q), n = min(at + Q * (lane % (32 / Q)), p.N - Q);
        const uint16_t* base = static_cast<const uint16_t*>(p.residual) + n;
#pragma unroll
        for (int i = 0; i < 16 / Q; ++i) {
            const uint16_t* from = base + (long long)max(tok[Q * i + sub], 0) * p.ldr;
            if constexpr (Q == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                w[2 * i] = v.x, w[2 * i + 1] = v.y;
            } else if constexpr (Q == 2) {
                w[i] = *reinterpret_cast<const uint32_t*>(from);
            } else {
                w[i] = *from;
            }
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void load(const Lora& p, const int* tok, int at) {
        const int lane = threadIdx.x & 31;
        if (!p.residual) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = 0u;
        } else if (WHOLE) {
            const int n = min(at + 8 * (lane & 3), p.N - 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long from = (long long)max(tok[8 * i + (lane >> 2)], 0) * p.ldr + n;
                if (p.out_f32) {
                    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p.residual) + from);
                    const uint4 a = q[0], b = q[1];
                    w[8 * i] = a.x, w[8 * i + 1] = a.y, w[8 * i + 2] = a.z, w[8 * i + 3] = a.w;
                    w[8 * i + 4] = b.x, w[8 * i + 5] = b.y, w[8 * i + 6] = b.z, w[8 * i + 7] = b.w;
                } else {
                    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + from);
                    w[8 * i] = a.x, w[8 * i + 1] = a.y, w[8 * i + 2] = a.z, w[8 * i + 3] = a.w;
                }
            }
        } else if (p.out_f32) {
            const int n = min(at + lane, p.N - 1);
#pragma unroll
            for (int r = 0; r < 16; ++r) w[r] = static_cast<const uint32_t*>(p.residual)[(long long)max(tok[r], 0) * p.ldr + n];
        } else if (p.vec == 4) {
            load_turns<4>(p, tok, at);
        } else if (p.vec == 2) {
            load_turns<2>(p, tok, at);
        } else {
            load_turns<1>(p, tok, at);
        }
    }
    // Wide rows: column k of row g (i = 0) or g + 8 (i = 1).
    __device__ __forceinline__ float wide_value(const Lora& p, int i, int k) const {
        return p.out_f32 ? __uint_as_float(w[8 * i + k])
                         : __uint_as_float((k & 1) ? w[8 * i + k / 2] & 0xFFFF0000u : w[8 * i + k / 2] << 16);
    }
    // Others: the staged sums of the unit that starts at column `at`, plus this, to out.
    template <int Q>
    __device__ __forceinline__ void store_turns(const Lora& p, const int* tok, const float* stage, int at) const {
        const int lane = threadIdx.x & 31, sub = lane / (32 / Q), c = Q * (lane % (32 / Q));
        if (at + c >= p.N) return;
        uint32_t o[16];
#pragma unroll
        for (int i = 0; i < 16 / Q; ++i) {
            const float* v = stage + (Q * i + sub) * kStagePitch + c;
            if constexpr (Q == 4) {
                const float4 u = *reinterpret_cast<const float4*>(v);
                o[2 * i] = f32x2_to_bf16x2_bits(u.x + __uint_as_float(w[2 * i] << 16), u.y + __uint_as_float(w[2 * i] & 0xFFFF0000u));
                o[2 * i + 1] = f32x2_to_bf16x2_bits(u.z + __uint_as_float(w[2 * i + 1] << 16),
                                                    u.w + __uint_as_float(w[2 * i + 1] & 0xFFFF0000u));
            } else if constexpr (Q == 2) {
                const float2 u = *reinterpret_cast<const float2*>(v);
                o[i] = f32x2_to_bf16x2_bits(u.x + __uint_as_float(w[i] << 16), u.y + __uint_as_float(w[i] & 0xFFFF0000u));
            } else {
                o[i] = f32_to_bf16_bits(v[0] + __uint_as_float(w[i] << 16));
            }
        }
#pragma unroll
        for (int i = 0; i < 16 / Q; ++i) {
            const int t = tok[Q * i + sub];
            if (t < 0) continue;
            uint16_t* to = static_cast<uint16_t*>(p.out) + (long long)t * p.ldo + at + c;
            if constexpr (Q == 4)
                *reinterpret_cast<uint2*>(to) = make_uint2(o[2 * i], o[2 * i + 1]);
            else if constexpr (Q == 2)
                *reinterpret_cast<uint32_t*>(to) = o[i];
            else
                *to = (uint16_t)o[i];
        }
    }
    __device__ __forceinline__ void store(const Lora& p, const int* tok, const float* stage, int at) const {
        const int lane = threadIdx.x & 31;
        if (p.out_f32) {
            if (at + lane >= p.N) return;
            float o[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = stage[r * kStagePitch + lane] + __uint_as_float(w[r]);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (tok[r] >= 0) static_cast<float*>(p.out)[(long long)tok[r] * p.ldo + at + lane] = o[r];
        } else if (p.vec == 4) {
            store_turns<4>(p, tok, stage, at);
        } else if (p.vec == 2) {
            store_turns<2>(p, tok, stage, at);
        } else {
            store_turns<1>(p, tok, stage, at);
        }
    }
};

// B's columns of the warp's next UN units of 32, as the MMAs take them.  (Asking for them a turn
// ahead, the first ones before v is made, costs registers and was slower: 15.7 us for 14.9, 64 tokens of 64 adapters.)
template <int RT>
struct Columns {
    static constexpr bool kShort = RT <= 2;         // at most 16 ranks: one MMA, 4 k a lane
    static constexpr int KU = kShort ? 1 : RT / 4;  // else units of 32 k, two MMAs, 8 k a lane
    static constexpr int W = kShort ? 2 : 4;        // words a lane and unit
    static constexpr int UN = RT <= 4 ? 2 : 1;
    uint32_t w[UN][4][KU][W];
    __device__ __forceinline__ void load(const Lora& p, const uint16_t* b, int u) {
        const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int v = 0; v < UN; ++v) {
            const int n0 = (u + v * kWarps) * 32 + (g >> 1) * 8 + (g & 1);
            const uint16_t* at = b + (size_t)min(n0, p.N - 1) * p.R;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (columns behind the last are read as the last of these, and not used)
                const int step = min(2 * j, max(p.N - 1 - n0, 0)) * p.R;
#pragma unroll
                for (int q = 0; q < KU; ++q) {
                    const uint16_t* from = at + step + min(q * 32 + 2 * W * tq, p.R - 2 * W);
                    if constexpr (kShort) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2*>(from));
                        w[v][j][q][0] = x.x, w[v][j][q][1] = x.y;
                    } else {
                        const uint4 x = __ldg(reinterpret_cast<const uint4*>(from));
                        w[v][j][q][0] = x.x, w[v][j][q][1] = x.y, w[v][j][q][W - 2] = x.z, w[v][j][q][W - 1] = x.w;
                    }
                }
            }
        }
    }
};

// out for this CTA's columns, UN times 32 a warp at a time, all tokens of the tile.
template <int RT, bool WHOLE>
__device__ __forceinline__ void expand(const Lora& p, const uint16_t* b, int rank, const int* tok, int cta, int ctas,
                                       const uint16_t* terms, float* staging) {
    using S = Shape<RT>;
    using B = Columns<RT>;
    constexpr bool kShort = B::kShort;
    constexpr int KU = B::KU, W = B::W, UN = B::UN;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int units = (p.N + 31) / 32;
    const int u0 = (int)((long long)units * cta / ctas), u1 = (int)((long long)units * (cta + 1) / ctas);
    const int nterms = p.out_f32 ? 3 : 2;
    // Rows that do not lie on 16 bytes pass through shared memory, p.vec neighbouring columns a lane (a lane's eight
    // columns one by one took 190 us for 8192 rows of 4095; through shared memory 4095 take 81 and 4092 take 63).
    float* stage = staging + warp * 16 * kStagePitch;
    const int t0 = tok[g], t1 = tok[8 + g];
    for (int u = u0 + warp; u < u1; u += UN * kWarps) {
        Columns<RT> columns;
        columns.load(p, b, u);
        auto& bw = columns.w;
        Residual res[UN];
#pragma unroll
        for (int v = 0; v < UN; ++v) res[v].template load<WHOLE>(p, tok, (u + v * kWarps) * 32);
        // what lies behind an adapter's rank is not its own, and may be NaN
#pragma unroll
        for (int q = 0; q < KU; ++q) {
            const int left = rank - (q * 32 + 2 * W * tq);
            if (left < 2 * W) {
#pragma unroll
                for (int v = 0; v < UN; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j) keep_first<W>(bw[v][j][q], left);
            }
        }
        float acc[UN][4][4];
#pragma unroll
        for (int v = 0; v < UN; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[v][j][i] = 0.0f;
#pragma unroll 1
        for (int e = nterms - 1; e >= 0; --e) {
            const uint16_t* at = terms + (size_t)e * S::kTermHalves + g * S::kTerm + 2 * W * tq;
#pragma unroll
            for (int q = 0; q < KU; ++q) {
                uint32_t lo[4], hi[4];
                if constexpr (kShort) {
                    const uint2 a = *reinterpret_cast<const uint2*>(at), c = *reinterpret_cast<const uint2*>(at + 8 * S::kTerm);
                    lo[0] = a.x, lo[1] = a.y, hi[0] = c.x, hi[1] = c.y;
                } else {
                    const uint4 a = *reinterpret_cast<const uint4*>(at + q * 32),
                                c = *reinterpret_cast<const uint4*>(at + 8 * S::kTerm + q * 32);
                    lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w, hi[0] = c.x, hi[1] = c.y, hi[2] = c.z, hi[3] = c.w;
                }
#pragma unroll
                for (int v = 0; v < UN; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int h = 0; h < W / 2; ++h)
                            mma_bf16(acc[v][j], lo[2 * h], hi[2 * h], lo[2 * h + 1], hi[2 * h + 1], bw[v][j][q][2 * h],
                                     bw[v][j][q][2 * h + 1]);
            }
        }
#pragma unroll
        for (int v = 0; v < UN; ++v) {
            const int at = (u + v * kWarps) * 32, n0 = at + 8 * tq, count = u + v * kWarps < u1 ? p.N - n0 : 0;
            if (WHOLE) {
                float r[2][8];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[i][k] = res[v].wide_value(p, i, k) + acc[v][k >> 1][2 * i + (k & 1)];
                if (t0 >= 0) store_out(p.out, p.out_f32, (long long)t0 * p.ldo + n0, count, true, r[0]);
                if (t1 >= 0) store_out(p.out, p.out_f32, (long long)t1 * p.ldo + n0, count, true, r[1]);
            } else if (u + v * kWarps < u1) {
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    float* to = stage + g * kStagePitch + 8 * tq + 2 * j;
                    *reinterpret_cast<float4*>(to) = make_float4(acc[v][j][0], acc[v][j][1], acc[v][j + 1][0], acc[v][j + 1][1]);
                    *reinterpret_cast<float4*>(to + 8 * kStagePitch) =
                        make_float4(acc[v][j][2], acc[v][j][3], acc[v][j + 1][2], acc[v][j + 1][3]);
                }
                __syncwarp();
                res[v].store(p, tok, stage, at);
                __syncwarp();
            }
        }
    }
}

// WHOLE: p.whole, known to the compiler.  Asked at run time both forms cost registers, which spilled: 64 tokens of 64
// adapters in a graph, weights from HBM, 12.4 us against 11.8, 1024 tokens 9.9 against 9.4 (fp32 x and output alone took 151 against 154).
template <int RT, bool XF32, bool WHOLE>
__global__ void __launch_bounds__(kThreads, RT <= 8 ? 2 : 1) lora_kernel(const __grid_constant__ Lora p) {
    using S = Shape<RT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int tok[kTokens];
    pdl_begin();
    const int ctas = p.ctas, item = blockIdx.x / ctas, cta = blockIdx.x % ctas;
    if (item >= p.tiles) {
        copy_rows<kThreads>(p, (item - p.tiles) * kThreads, cta, ctas);
        pdl_end_block();
        return;
    }
    // higher tiles are taken in pieces
    const int pieces = p.tile_m / kTokens, tile = item / pieces;
    int used = __ldg(p.num_tiles);
    const int adapter = __ldg(p.tile_expert + tile);
    // (positions follow one another from tile to tile)
    int q = threadIdx.x < kTokens ? __ldg(p.sorted_pairs + (size_t)item * kTokens + threadIdx.x) : -1;
    if (used < 0 || used > p.tiles / pieces) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_index_error();
        used = 0;
    }
    if (tile >= used) return;
    if ((unsigned)adapter >= (unsigned)p.adapters) {
        if (threadIdx.x == 0) flag_index_error();
        return;
    }
    // (uniform over the cluster: its CTAs read the same words)
    const int rank = p.ranks ? min(max(__ldg(p.ranks + adapter), 0), p.R) : p.R;
    const float scale = p.scale ? __ldg(p.scale + adapter) : 1.0f;
    const uint16_t* b = p.b + (size_t)adapter * p.N * p.R;
    float* part = reinterpret_cast<float*>(smem);
    float* sum = part + S::kPartFloats;
    uint16_t* terms = reinterpret_cast<uint16_t*>(part);
    if (threadIdx.x < kTokens) {
        if (q >= p.T) {
            flag_index_error();
            q = -1;
        }
        tok[threadIdx.x] = q;
    }
    __syncthreads();
    if (tok[0] < 0) return;  // the empty end of a tile

    shrink<RT, XF32>(p, p.a + (size_t)adapter * p.R * p.K, tok, cta, ctas, part);
    __syncthreads();
    for (int i = threadIdx.x; i < kTokens * S::kRanks; i += kThreads) {
        const int at = (i / S::kRanks) * S::kPart + i % S::kRanks;
        float v = part[at];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += part[at + w * kTokens * S::kPart];
        sum[at] = v;
    }
    if (ctas > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const int nterms = p.out_f32 ? 3 : 2;
    for (int i = threadIdx.x; i < kTokens * S::kRanks; i += kThreads) {
        const int t = i / S::kRanks, r = i % S::kRanks;
        const float* at = sum + t * S::kPart + r;
        float v = *at;
        if (ctas > 1) {
            float part_of[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) part_of[c] = c < ctas ? ld_cluster(at, c) : 0.0f;
            v = part_of[0];
#pragma unroll
            for (int c = 1; c < 8; ++c) v += part_of[c];
        }
        v = r < rank ? v * scale : 0.0f;
        uint32_t hi, mid;
        const float rest = split_bf16(v, hi);
        uint16_t* to = terms + t * S::kTerm + r;
        to[0] = (uint16_t)hi;
        if (nterms == 2) {
            to[S::kTermHalves] = f32_to_bf16_bits(rest);
        } else {
            const float last = split_bf16(rest, mid);
            to[S::kTermHalves] = (uint16_t)mid;
            to[2 * S::kTermHalves] = f32_to_bf16_bits(last);
        }
    }
    // this CTA has read the others' sums
    if (ctas > 1) cluster_arrive();
    __syncthreads();
    expand<RT, WHOLE>(p, b, rank, tok, cta, ctas, terms, sum + kTokens * S::kPart);
    pdl_end_block();
    // a CTA's shared memory has to live until the others have read it
    if (ctas > 1) cluster_wait();
}

template <int RT, bool XF32, bool WHOLE>
cudaError_t launch_one(const Lora& p, int items, cudaStream_t s) {
    const auto kernel = lora_kernel<RT, XF32, WHOLE>;
    const size_t smem = Shape<RT>::kBytes + (WHOLE ? 0 : kWarps * 16 * kStagePitch * 4);
    // (the limit without it is on static and dynamic shared memory together)
    const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem + 1024);
    if (err != cudaSuccess) return err;
    if (p.ctas == 1) return launch_pdl(kernel, dim3(items), dim3(kThreads), smem, s, p);
    return launch_pdl_cluster(kernel, dim3((unsigned)(items * p.ctas)), dim3(kThreads), smem, s, p.ctas, p);
}

template <bool XF32, bool WHOLE>
cudaError_t launch_ranks(const Lora& p, int items, cudaStream_t s) {
    if (p.R <= 16) return launch_one<2, XF32, WHOLE>(p, items, s);
    if (p.R <= 32) return launch_one<4, XF32, WHOLE>(p, items, s);
    if (p.R <= 64) return launch_one<8, XF32, WHOLE>(p, items, s);
    return launch_one<16, XF32, WHOLE>(p, items, s);
}

bool wide_rows(const void* p, int f32, long long ld) {
    return (uintptr_t)p % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

}  // namespace

bool lora_tile_supported(int tile_m) { return tile_m == 16 || tile_m == 32 || tile_m == 64 || tile_m == 128; }

// Tile height: 128 where prompts fill such tiles and there are enough of them for the SMs (4096 tokens of 4
// adapters at 4096 x 4096, rank 64: 32.8 us in tiles of 128, 52.6 in tiles of 16; rank 16: 30.1 and 31.0;
// 2048 tokens at rank 16: 27 and 18.5), else 16.  (`adapters` may be a pool of which few are used: then 16, where 8192
// tokens of four prompts of a pool of 128 take 101 us at rank 64, and 70 in tiles of 128.)
int lora_tile_rule(int T, int adapters) {
    const int each = T / std::max(1, std::min(T, adapters));
    return each >= 96 && T >= 2560 ? 128 : 16;
}

cudaError_t launch_lora(const Lora& given, cudaStream_t s) {
    Lora p = given;
    // a used tile holds a token, and only an adapter's last one is not full
    p.tiles = (int)std::min<long long>({(long long)p.max_tiles, (long long)p.T,
                                        (long long)p.T / p.tile_m + std::min(p.adapters, p.T)});
    p.x_wide = wide_rows(p.x, p.x_f32, p.ldx);
    p.res_wide = p.residual && wide_rows(p.residual, p.out_f32, p.ldr);
    p.out_wide = wide_rows(p.out, p.out_f32, p.ldo);
    p.whole = p.out_wide && (!p.residual || p.res_wide) && p.N % 8 == 0;
    p.vec = p.out_f32 ? 1 : 4;
    while (p.vec > 1 && (p.N % p.vec || p.ldo % p.vec || (uintptr_t)p.out % (2 * p.vec) ||
                         (p.residual && (p.ldr % p.vec || (uintptr_t)p.residual % (2 * p.vec)))))
        p.vec /= 2;
    if (lora_prompt_supported(p)) return launch_lora_prompt(p, s);
    p.tiles *= p.tile_m / kTokens;
    // CTAs a piece: two for each SM in all, which run at once (four: 64 tokens of 64 adapters in 18.3 us
    // instead of 14.9), for the pieces that these tokens can fill
    const int widest = std::max(p.K, p.N);
    const long long likely = std::min<long long>(p.tiles, (long long)p.T / kTokens + std::min(p.adapters, p.T));
    p.ctas = 8;
    while (p.ctas > 1 && (likely * p.ctas > 2LL * num_sms() || p.ctas * 64 > widest)) p.ctas /= 2;
    const bool in_place = p.residual == p.out && p.ldr == p.ldo;
    const int items = p.tiles + (in_place ? 0 : (p.T + kThreads - 1) / kThreads);
    if (p.whole) return p.x_f32 ? launch_ranks<true, true>(p, items, s) : launch_ranks<false, true>(p, items, s);
    return p.x_f32 ? launch_ranks<true, false>(p, items, s) : launch_ranks<false, false>(p, items, s);
}

cudaError_t read_device_error_lora(int* flag, int clear) {
    int index = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&index, g_index_error, sizeof(int));
    if (err != cudaSuccess) return err;
    *flag = index ? 2 : 0;
    if (!clear) return cudaSuccess;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_index_error, &zero, sizeof(int));
}

}  // namespace moe
