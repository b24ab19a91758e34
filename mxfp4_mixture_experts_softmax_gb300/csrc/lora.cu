// lora.cu -- low-rank adapters of many requests beside a shared projection:
//
//   out[t] = residual[t] + scale[a] * B[a] (A[a] x_t)      a = the adapter of token t
//   out[t] = residual[t]                                   for a token without one
//
// One launch, no workspace.  A cluster of CTAs takes a tile of up to 16, 32 or 64
// tokens of one adapter (moe_permute's grouping).  Its CTAs split the sum over K
// (v = A x), join their parts through distributed shared memory in rank order, and
// split the N outputs.  x and the residual are read once, out is written once, and
// v never leaves the chip; A and B are read once per tile, from L2 after the first.
// At ranks up to 128 this is far below the ridge, so what bounds it is HBM for long
// prompts and latency for few tokens; the products run as warp MMAs (bf16,
// m16n8k16) straight from global memory into registers.  Both operands of an MMA
// may permute their k alike, so a lane takes 8 neighbouring k of a row (16 bytes)
// as its four k of two MMAs, and neighbouring output columns likewise.
//
// Products are exact: bf16 times bf16, an fp32 x as three bf16 terms.  Sums are fp32.
// v, an fp32 sum, enters the second product as bf16 terms: two for a bf16 output (2^-16 of
// v, a hundredth of the output's own rounding), three for fp32 (2^-24).
#include <algorithm>

#include "lora_device.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

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
__device__ __forceinline__ void load_x(Chunk<F32>& c, const void* row, int k, bool ok, bool wide) {
    constexpr int W = F32 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < W; ++i) c.w[i] = 0u;
    if (!ok) return;
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
#pragma unroll
        for (int i = 0; i < 4; ++i) c.w[i] = (uint32_t)__ldg(q + 2 * i) | ((uint32_t)__ldg(q + 2 * i + 1) << 16);
    }
}

// The first n of the eight bf16 in four words, zeros behind them.
__device__ __forceinline__ void keep_first(uint32_t* w, int words, int n) {
    for (int i = 0; i < words; ++i) w[i] = n >= 2 * i + 2 ? w[i] : n == 2 * i + 1 ? w[i] & 0xFFFFu : 0u;
}

template <int MT, int RT, int TW>
struct Shape {
    static constexpr int kTokens = 16 * MT * TW;  // of a tile
    static constexpr int kKWarps = kWarps / TW;   // warps that split K
    static constexpr int kRanks = 8 * RT;
    // fp32 rows of v: 8 floats of padding put the four rows of a half-warp's stores in separate banks
    static constexpr int kPart = kRanks + 8;
    // bf16 rows of v's terms: the two rows of eight lanes' 16-byte reads fall in separate halves of the banks
    static constexpr int kTerm = kRanks <= 32 ? kRanks : kRanks + 32;
    static constexpr int kPartFloats = kKWarps * kTokens * kPart;
    static constexpr int kTermHalves = kTokens * kTerm;
    // v's terms take the place of its parts, which are done with by then
    static constexpr size_t kBytes = (size_t)kPartFloats * 4 + (size_t)kTokens * kPart * 4;
    static_assert(3 * kTermHalves * 2 <= kPartFloats * 4, "v's terms do not fit over its parts");
};

// v's parts: this warp's MT x 16 tokens times all ranks over its units of 32 k.
template <int MT, int RT, int TW, bool XF32>
__device__ __forceinline__ void shrink(const Lora& p, const uint16_t* a, int rank_rows, const int* tok, int cta, int ctas,
                                       float* part) {
    using S = Shape<MT, RT, TW>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int tw = warp % TW, kw = warp / TW;
    const int units = (p.K + 31) / 32;
    const int u0 = (int)((long long)units * cta / ctas), u1 = (int)((long long)units * (cta + 1) / ctas);
    const void* row[2 * MT];
    bool live[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int t = tok[tw * 16 * MT + i * 8 + g];
        live[i] = t >= 0;
        row[i] = static_cast<const uint8_t*>(p.x) + (size_t)max(t, 0) * p.ldx * (XF32 ? 4 : 2);
    }
    float acc[MT][RT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][r][i] = 0.0f;

#pragma unroll 2
    for (int u = u0 + kw; u < u1; u += S::kKWarps) {
        const int k = u * 32 + 8 * tq;
        const bool in = k < p.K;
        Chunk<XF32> x[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) load_x<XF32>(x[i], row[i], k, in && live[i], p.x_wide);
        uint4 w[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            w[r] = in && r * 8 + g < rank_rows ? __ldg(reinterpret_cast<const uint4*>(a + (size_t)(r * 8 + g) * p.K + k))
                                               : make_uint4(0, 0, 0, 0);
        if constexpr (XF32) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t lo[3][4], hi[3][4];  // rows g and g + 8
                split8(reinterpret_cast<const float*>(x[2 * m].w), lo);
                split8(reinterpret_cast<const float*>(x[2 * m + 1].w), hi);
#pragma unroll
                for (int j = 2; j >= 0; --j)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        mma_bf16(acc[m][r], lo[j][0], hi[j][0], lo[j][1], hi[j][1], w[r].x, w[r].y);
                        mma_bf16(acc[m][r], lo[j][2], hi[j][2], lo[j][3], hi[j][3], w[r].z, w[r].w);
                    }
            }
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t *lo = x[2 * m].w, *hi = x[2 * m + 1].w;
                    mma_bf16(acc[m][r], lo[0], hi[0], lo[1], hi[1], w[r].x, w[r].y);
                    mma_bf16(acc[m][r], lo[2], hi[2], lo[3], hi[3], w[r].z, w[r].w);
                }
        }
    }
    float* mine = part + ((size_t)kw * S::kTokens + tw * 16 * MT) * S::kPart;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float* q = mine + (m * 16 + g) * S::kPart + r * 8 + 2 * tq;
            *reinterpret_cast<float2*>(q) = make_float2(acc[m][r][0], acc[m][r][1]);
            *reinterpret_cast<float2*>(q + 8 * S::kPart) = make_float2(acc[m][r][2], acc[m][r][3]);
        }
}

// out for this CTA's columns, 32 a warp at a time, all tokens of the tile.
template <int MT, int RT, int TW>
__device__ __forceinline__ void expand(const Lora& p, const uint16_t* b, int rank, const int* tok, int cta, int ctas,
                                       const uint16_t* terms) {
    using S = Shape<MT, RT, TW>;
    constexpr bool kShort = RT <= 2;                 // at most 16 ranks: one MMA, 4 k a lane
    constexpr int KU = kShort ? 1 : RT / 4;          // else units of 32 k, two MMAs, 8 k a lane
    constexpr int W = kShort ? 2 : 4;                // words a lane and unit
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int units = (p.N + 31) / 32;
    const int u0 = (int)((long long)units * cta / ctas), u1 = (int)((long long)units * (cta + 1) / ctas);
    const int nterms = p.out_f32 ? 3 : 2;
    for (int u = u0 + warp; u < u1; u += kWarps) {
        uint32_t bw[4][KU][W];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = u * 32 + (g >> 1) * 8 + 2 * j + (g & 1);
#pragma unroll
            for (int q = 0; q < KU; ++q) {
                const int k = q * 32 + 2 * W * tq;
#pragma unroll
                for (int i = 0; i < W; ++i) bw[j][q][i] = 0u;
                if (n < p.N && k < rank) {
                    const uint16_t* at = b + (size_t)n * p.R + k;
                    if constexpr (kShort) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
                        bw[j][q][0] = v.x, bw[j][q][1] = v.y;
                    } else {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
                        bw[j][q][0] = v.x, bw[j][q][1] = v.y, bw[j][q][W - 2] = v.z, bw[j][q][W - 1] = v.w;
                    }
                    // what lies behind an adapter's rank is not its own, and may be NaN
                    if (rank < p.R) keep_first(bw[j][q], W, rank - k);
                }
            }
        }
        const int n0 = u * 32 + 8 * tq, count = p.N - n0;
#pragma unroll 1
        for (int m = 0; m < S::kTokens / 16; ++m) {
            const int t0 = tok[m * 16 + g], t1 = tok[m * 16 + 8 + g];
            if (__all_sync(0xFFFFFFFFu, t0 < 0 && t1 < 0)) continue;
            float r0[8], r1[8];
            load_out(p.residual, p.out_f32, (long long)t0 * p.ldr + n0, p.residual && t0 >= 0 ? count : 0, p.res_wide, r0);
            load_out(p.residual, p.out_f32, (long long)t1 * p.ldr + n0, p.residual && t1 >= 0 ? count : 0, p.res_wide, r1);
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll 1
            for (int e = nterms - 1; e >= 0; --e) {
                const uint16_t* v = terms + (size_t)e * S::kTermHalves + (m * 16 + g) * S::kTerm + 2 * W * tq;
#pragma unroll
                for (int q = 0; q < KU; ++q) {
                    uint32_t lo[4], hi[4];
                    if constexpr (kShort) {
                        const uint2 a = *reinterpret_cast<const uint2*>(v), c = *reinterpret_cast<const uint2*>(v + 8 * S::kTerm);
                        lo[0] = a.x, lo[1] = a.y, hi[0] = c.x, hi[1] = c.y;
                    } else {
                        const uint4 a = *reinterpret_cast<const uint4*>(v + q * 32),
                                    c = *reinterpret_cast<const uint4*>(v + 8 * S::kTerm + q * 32);
                        lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w, hi[0] = c.x, hi[1] = c.y, hi[2] = c.z, hi[3] = c.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int h = 0; h < W / 2; ++h)
                            mma_bf16(acc[j], lo[2 * h], hi[2 * h], lo[2 * h + 1], hi[2 * h + 1], bw[j][q][2 * h], bw[j][q][2 * h + 1]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r0[2 * j] += acc[j][0], r0[2 * j + 1] += acc[j][1];
                r1[2 * j] += acc[j][2], r1[2 * j + 1] += acc[j][3];
            }
            if (t0 >= 0) store_out(p.out, p.out_f32, (long long)t0 * p.ldo + n0, count, p.out_wide, r0);
            if (t1 >= 0) store_out(p.out, p.out_f32, (long long)t1 * p.ldo + n0, count, p.out_wide, r1);
        }
    }
}

template <int MT, int RT, int TW, bool XF32>
__global__ void __launch_bounds__(kThreads) lora_kernel(const __grid_constant__ Lora p) {
    using S = Shape<MT, RT, TW>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int tok[S::kTokens];
    pdl_begin();
    const int ctas = p.ctas, item = blockIdx.x / ctas, cta = blockIdx.x % ctas;
    if (item >= p.tiles) {
        copy_rows<kThreads>(p, (item - p.tiles) * kThreads, cta, ctas);
        pdl_end();
        return;
    }
    int used = __ldg(p.num_tiles);
    if (used < 0 || used > p.tiles / (p.tile_m / S::kTokens)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_index_error();
        used = 0;
    }
    // a tile of 128 is taken as two
    const int halves = p.tile_m / S::kTokens, tile = item / halves;
    if (tile >= used) return;
    const int adapter = __ldg(p.tile_expert + tile);
    if ((unsigned)adapter >= (unsigned)p.adapters) {
        if (threadIdx.x == 0) flag_index_error();
        return;
    }
    // (uniform over the cluster: its CTAs read the same words)
    const int rank = p.ranks ? min(max(__ldg(p.ranks + adapter), 0), p.R) : p.R;
    float* part = reinterpret_cast<float*>(smem);
    float* sum = part + S::kPartFloats;
    uint16_t* terms = reinterpret_cast<uint16_t*>(part);
    if (threadIdx.x < S::kTokens) {
        // (positions follow one another from tile to tile)
        int q = __ldg(p.sorted_pairs + (size_t)item * S::kTokens + threadIdx.x);
        if (q >= p.T) {
            flag_index_error();
            q = -1;
        }
        tok[threadIdx.x] = q;
    }
    __syncthreads();

    shrink<MT, RT, TW, XF32>(p, p.a + (size_t)adapter * p.R * p.K, rank, tok, cta, ctas, part);
    __syncthreads();
    for (int i = threadIdx.x; i < S::kTokens * S::kRanks; i += kThreads) {
        const int at = (i / S::kRanks) * S::kPart + i % S::kRanks;
        float v = part[at];
#pragma unroll
        for (int w = 1; w < S::kKWarps; ++w) v += part[at + w * S::kTokens * S::kPart];
        sum[at] = v;
    }
    if (ctas > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const float scale = p.scale ? __ldg(p.scale + adapter) : 1.0f;
    const int nterms = p.out_f32 ? 3 : 2;
    for (int i = threadIdx.x; i < S::kTokens * S::kRanks; i += kThreads) {
        const int t = i / S::kRanks, r = i % S::kRanks;
        const float* at = sum + t * S::kPart + r;
        float v = ctas > 1 ? ld_cluster(at, 0) : *at;
        for (int c = 1; c < ctas; ++c) v += ld_cluster(at, c);
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
    expand<MT, RT, TW>(p, p.b + (size_t)adapter * p.N * p.R, rank, tok, cta, ctas, terms);
    pdl_end();
    // a CTA's shared memory has to live until the others have read it
    if (ctas > 1) cluster_wait();
}

template <int MT, int RT, int TW, bool XF32>
cudaError_t launch_one(const Lora& p, int items, cudaStream_t s) {
    const auto kernel = lora_kernel<MT, RT, TW, XF32>;
    const size_t smem = Shape<MT, RT, TW>::kBytes;
    const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (err != cudaSuccess) return err;
    if (p.ctas == 1) return launch_pdl(kernel, dim3(items), dim3(kThreads), smem, s, p);
    return launch_pdl_cluster(kernel, dim3((unsigned)(items * p.ctas)), dim3(kThreads), smem, s, p.ctas, p);
}

template <int MT, int TW, bool XF32>
cudaError_t launch_ranks(const Lora& p, int items, cudaStream_t s) {
    if (p.R <= 16) return launch_one<MT, 2, TW, XF32>(p, items, s);
    if (p.R <= 32) return launch_one<MT, 4, TW, XF32>(p, items, s);
    if (p.R <= 64) return launch_one<MT, 8, TW, XF32>(p, items, s);
    return launch_one<MT, 16, TW, XF32>(p, items, s);
}

template <bool XF32>
cudaError_t launch_tile(const Lora& p, int items, cudaStream_t s) {
    if (p.tile_m == 16) return launch_ranks<1, 1, XF32>(p, items, s);
    if (p.tile_m == 32) return launch_ranks<2, 1, XF32>(p, items, s);
    return launch_ranks<2, 2, XF32>(p, items, s);
}

bool wide_rows(const void* p, int f32, long long ld) {
    return (uintptr_t)p % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

}  // namespace

bool lora_tile_supported(int tile_m) { return tile_m == 16 || tile_m == 32 || tile_m == 64 || tile_m == 128; }

// Tile height: tokens that share an adapter share its reads, so the height follows the
// tokens an adapter has on average, as long as there are tiles enough for the SMs.
int lora_tile_rule(int T, int adapters) {
    const int each = T / std::max(1, std::min(T, adapters));
    return each >= 96 && T >= 1024 ? 128 : each >= 64 && T >= 4096 ? 64 : each >= 32 && T >= 1024 ? 32 : 16;
}

cudaError_t launch_lora(const Lora& given, cudaStream_t s) {
    Lora p = given;
    // a used tile holds a token, and only an adapter's last one is not full
    p.tiles = (int)std::min<long long>({(long long)p.max_tiles, (long long)p.T,
                                        (long long)p.T / p.tile_m + std::min(p.adapters, p.T)});
    p.x_wide = wide_rows(p.x, p.x_f32, p.ldx);
    p.res_wide = p.residual && wide_rows(p.residual, p.out_f32, p.ldr);
    p.out_wide = wide_rows(p.out, p.out_f32, p.ldo);
    if (lora_prompt_supported(p)) return launch_lora_prompt(p, s);
    if (p.tile_m == 128) p.tiles *= 2;
    // CTAs a tile: about two for each SM in all
    const int widest = std::max(p.K, p.N);
    p.ctas = 8;
    while (p.ctas > 1 && ((long long)p.tiles * p.ctas > 2LL * num_sms() || p.ctas * 64 > widest)) p.ctas /= 2;
    const bool in_place = p.residual == p.out && p.ldr == p.ldo;
    const int items = p.tiles + (in_place ? 0 : (p.T + kThreads - 1) / kThreads);
    return p.x_f32 ? launch_tile<true>(p, items, s) : launch_tile<false>(p, items, s);
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
