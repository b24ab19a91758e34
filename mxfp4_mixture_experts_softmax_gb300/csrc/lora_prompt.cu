// lora_prompt.cu -- low-rank adapters beside a shared projection for prompts, on the 5th-generation
// tensor cores: tiles of 128 tokens of one adapter (moe_permute's grouping).
//
//   v = A[a] x_t (fp32),   out[t] = residual[t] + B[a] (scale[a] v)
//
// What has to move is x, the residual and the output once (192 MB for 8192 tokens of 4096 values: 32
// us); at rank 64 both products are a tenth of that at the tensor cores' rate, but as much as that
// through warp MMAs, whose operands pass the registers (lora.cu: 102 us).  So:
//   * a cluster of CTAs has a tile; its CTAs split the sum over K, join their parts of v through
//     distributed shared memory in rank order (each makes the sums of its share of the rows and gives them to
//     all), and split the N outputs.  One launch, no workspace;
//   * producer warp: A, B and x by TMA into a ring of 64-k stages (128-byte swizzle).  The tile's
//     tokens lie anywhere, but mostly one after another: where 32 or 8 do, one box fetches them, else
//     gathers of four rows (which alone, at 80 clocks each, take 42 us for 8192 tokens);
//   * MMA warp: D1[128 x ranks] += x A^T from shared memory; then, for each tile of outputs,
//     D2[128 x 128] = v B^T with v as the operand in tensor memory, two accumulators in turn;
//   * eight epilogue warps: four read D1, add the others' parts, scale and write v back to tensor
//     memory as two bf16 terms (2^-16 of v; three for an fp32 output, 2^-24).  All eight then take D2, each 32
//     rows and half of the columns.  Where its 32 tokens lie one after another, residual and output pass
//     as TMA boxes through a ring of the warp's own; else D2 passes through shared memory into rows, which
//     are loaded and stored 128 bytes at a time (that way alone: 55 us, the loads waiting for one another in L1).
//
// 8192 tokens of 4096 values, rank 64, eleven prompts: 49.5 us (4.3 TB/s); 32768 tokens, rank 16: 162 us (5.0
// TB/s).  About 15 us of the 49.5 are x's way in, 3 the joining of v, 22 the residual's and the output's, the rest
// the launch and the ends: with a tile a cluster these follow one another on an SM, and only many tiles let them overlap.
#include <algorithm>

#include "lora_device.cuh"
#include "mxf4.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kTile = 128, kWarps = 12, kThreads = kWarps * 32, kEpi0 = 4;
constexpr int kXBytes = kTile * 128;               // 64 k of the tile's tokens
constexpr int kRing = 128 * 1024;                  // phase 1's stages; then v's parts and B's stages
constexpr int kBOffset = 68 * 1024, kBBytes = 16 * 1024, kBStages = 3;
constexpr int kMaxStages = 6;
constexpr int kAhead = 4, kPieceBytes = 4096;       // an epilogue warp's ring of residual and output, 32 rows x 128 bytes
constexpr int kPitch = 68;                         // floats of a staged row of 64: rows of 8 lanes in separate banks
constexpr int kStaging = 68 * 1024;                // v's sums; then rings (and 8.5 KB where D2 is staged) of four warps
constexpr size_t kSmem = 1024 + kRing + kStaging;  // 1 KB to align
constexpr uint32_t kD2 = 0, kV = 256, kColumns = 512;  // tensor memory: D2 twice (D1 over the first), v's terms

__host__ __device__ constexpr uint32_t idesc_bf16(int N) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Four rows of a map whose box is one row, to `dst` and the three rows behind it.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* tmap, int c0, const int* row, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void st_cluster4(float* p, uint32_t rank, float4 v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// A box of shared memory to global memory, in the thread's current bulk group.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(c0),
                 "r"(c1), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// 16 bytes of the residual and the output, which no other thread touches: free of the order that the
// compiler keeps between accesses that may alias (an output that is its own residual is read before it is
// written, through the registers).
__device__ __forceinline__ uint4 ld_global(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void st_global(void* p, uint4 v) {
    asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Residual or output of 64 columns of the warp's 32 rows: lane l has V neighbouring columns of
// row pass * ROWS + l / (64 / V).
template <bool OF32>
struct Rows {
    static constexpr int kV = OF32 ? 4 : 8, kLanes = 64 / kV, kRows = 32 / kLanes, kPasses = 32 / kRows,
                         kSets = OF32 ? 1 : 2;  // pieces whose residual is on its way
    // Where a staged row has its column c (a multiple of 4): for bf16 the even fours first, so that the lanes
    // of a row, each with two neighbouring fours, read 128 bytes in a row twice.
    __device__ static __forceinline__ int place(int c) { return OF32 ? c : ((c >> 3) << 2) + ((c & 4) << 3); }
};

template <bool OF32>
__global__ void __launch_bounds__(kThreads, 1)
    lora_prompt_kernel(const __grid_constant__ Lora p, const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap x8_map, const __grid_constant__ CUtensorMap x32_map,
                       const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                       const __grid_constant__ CUtensorMap res_map, const __grid_constant__ CUtensorMap out_map) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], b_full[kBStages], b_empty[kBStages], d2_full[2],
        d2_empty[2], d1_full, v_ready, res_full[8][kAhead];
    __shared__ uint32_t tmem_slot;
    __shared__ int tok[kTile];

    pdl_begin();
    const int ctas = p.ctas, item = blockIdx.x / ctas, cta = blockIdx.x % ctas;
    if (item >= p.tiles) {
        copy_rows<kThreads>(p, (item - p.tiles) * kThreads, cta, ctas);
        pdl_end_block();
        return;
    }
    // (uniform over the cluster: its CTAs read the same words)
    int used = __ldg(p.num_tiles);
    if (used < 0 || used > p.tiles) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_index_error();
        used = 0;
    }
    if (item >= used) return;
    const int adapter = __ldg(p.tile_expert + item);
    if ((unsigned)adapter >= (unsigned)p.adapters) {
        if (threadIdx.x == 0) flag_index_error();
        return;
    }

    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Rp = (p.R + 15) & ~15;          // ranks as the MMA takes them
    const int NT = Rp <= 64 ? 128 : 64;       // outputs of a tile: B's stage is 16 KB either way
    const int blocks = Rp <= 64 ? 1 : 2;      // of 64 ranks
    const uint32_t stage_bytes = kXBytes + 128 * Rp;
    const int stages = min(kMaxStages, kRing / (int)stage_bytes);
    const int ks = (p.K + 63) / 64, nk = (ks - cta + ctas - 1) / ctas;
    const int tn = (p.N + NT - 1) / NT, nn = (tn - cta + ctas - 1) / ctas;
    const int terms = OF32 ? 3 : 2;
    // the warps that read a D2 buffer: all eight of a tile of 128 outputs, four (by the tile's parity) of one of 64
    const int readers = NT == 128 ? 8 : 4;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < kBStages; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&d2_full[i], 1), mbar_init(&d2_empty[i], readers);
        for (int i = 0; i < 8 * kAhead; ++i) mbar_init(&res_full[0][0] + i, 1);
        mbar_init(&d1_full, 1);
        mbar_init(&v_ready, 128);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < kTile) {
        int q = __ldg(p.sorted_pairs + (size_t)item * kTile + threadIdx.x);
        if (q >= p.T) {
            flag_index_error();
            q = -1;
        }
        tok[threadIdx.x] = q;
    }
    if (warp == 1) tmem_alloc<false>(&tmem_slot, kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const bool joins = ctas > 1;
    // The cluster meets twice: when the parts of v are there, and when their sums are.  Four warps write and
    // read them; the others arrive ahead and wait where they have nothing else to do.
    const bool sums = warp >= kEpi0 && warp < kEpi0 + 4;
    if (joins && !sums) cluster_arrive();
    const auto meet_once = [&] {
        if (joins) {
            cluster_wait();
            cluster_arrive();
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------- producer
        bool met = false;
        // Lane l has rows 4 l .. 4 l + 3.  A row without a token continues the one before (its outputs go nowhere;
        // a row behind the last token is zeros); where a whole piece has none, it is not fetched.
        int row[4], held = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row[i] = tok[4 * lane + i];
            held += row[i] >= 0;
        }
        int last = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) last = row[i] >= 0 ? row[i] - 4 * lane - i : last;  // token minus row
        // (rows without a token come last in a tile: the lanes before know where it continues)
        const uint32_t any = __ballot_sync(0xFFFFFFFFu, held > 0), below = any & ((2u << lane) - 1);
        const int before = __shfl_sync(0xFFFFFFFFu, last, below ? 31 - __clz((int)below) : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = row[i] >= 0 ? row[i] : max(before + 4 * lane + i, 0);
        const int next = __shfl_down_sync(0xFFFFFFFFu, row[0], 1);
        const bool inner = row[1] == row[0] + 1 && row[2] == row[1] + 1 && row[3] == row[2] + 1, outer = next == row[3] + 1;
        const uint32_t in_row = __ballot_sync(0xFFFFFFFFu, inner), on_row = __ballot_sync(0xFFFFFFFFu, outer);
        const int g32 = lane & ~7, g8 = lane & ~1;
        const bool run32 = ((in_row >> g32) & 0xFFu) == 0xFFu && ((on_row >> g32) & 0x7Fu) == 0x7Fu;
        const bool run8 = ((in_row >> g8) & 3u) == 3u && ((on_row >> g8) & 1u);
        const bool want32 = (any >> g32) & 0xFFu, want8 = (any >> g8) & 3u;
        // the rows that this lane fetches: 32, 8, 4 or none
        int rows = 0;
        if (run32)
            rows = want32 && (lane & 7) == 0 ? 32 : 0;
        else if (run8)
            rows = want8 && (lane & 1) == 0 ? 8 : 0;
        else
            rows = want8 ? 4 : 0;
        const uint32_t x_bytes = 128u * __reduce_add_sync(0xFFFFFFFFu, rows);
        if (rows == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) row[i] = min(row[i], p.T - 1);
        }
        bool ok = true;
        for (int i = 0, s = 0, parity = 1; i < nk && ok; ++i) {
            if (i >= stages) ok = mbar_wait_warp(&empty[s], parity);
            if (!ok) break;
            uint8_t* to = smem + (size_t)s * stage_bytes;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], x_bytes + 128 * p.R);
                tma_load_2d(smem_u32(to + kXBytes), &a_map, (cta + i * ctas) * 64, adapter * p.R, &full[s]);
            }
            __syncwarp();
            const uint32_t dst = smem_u32(to) + lane * 512;
            if (rows == 32)
                tma_load_2d(dst, &x32_map, (cta + i * ctas) * 64, row[0], &full[s]);
            else if (rows == 8)
                tma_load_2d(dst, &x8_map, (cta + i * ctas) * 64, row[0], &full[s]);
            else if (rows == 4)
                tma_gather4(dst, &x_map, (cta + i * ctas) * 64, row, &full[s]);
            if (++s == stages) s = 0, parity ^= 1;
        }
        __syncwarp();
        // B's stages lie where the last of those were
        ok = ok && mbar_wait_warp(&d1_full, 0);
        for (int i = 0; i < nn && ok; ++i) {
            const int s = i % kBStages;
            if (i == kBStages) {
                meet_once();
                met = true;
            }
            if (i >= kBStages) ok = mbar_wait_warp(&b_empty[s], ((i / kBStages) - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                uint8_t* to = smem + kBOffset + s * kBBytes;
                mbar_arrive_expect_tx(&b_full[s], kBBytes);
                for (int j = 0; j < blocks; ++j)
                    tma_load_2d(smem_u32(to + j * NT * 128), &b_map, j * 64, adapter * p.N + (cta + i * ctas) * NT, &b_full[s]);
            }
            __syncwarp();
        }
        if (!met) meet_once();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA
        bool ok = true;
        const uint32_t id1 = idesc_bf16(Rp), id2 = idesc_bf16(NT);
        // (a descriptor's low bits are its address in units of 16 bytes)
        const uint64_t x_desc = sdesc_sw128(smem_u32(smem)), a_desc = sdesc_sw128(smem_u32(smem + kXBytes)),
                       b_desc = sdesc_sw128(smem_u32(smem + kBOffset));
        for (int i = 0, s = 0, parity = 0; i < nk && ok; ++i) {
            ok = mbar_wait_warp(&full[s], parity);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                const uint64_t ad = x_desc + s * (stage_bytes >> 4), bd = a_desc + s * (stage_bytes >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(tmem + kD2, ad + 2 * k, bd + 2 * k, id1, (i | k) != 0);
                mma_commit(&empty[s]);
                if (i == nk - 1) mma_commit(&d1_full);
            }
            __syncwarp();
            if (++s == stages) s = 0, parity ^= 1;
        }
        if (nk == 0 && lane == 0) mbar_arrive(&d1_full);
        __syncwarp();
        meet_once();
        ok = ok && mbar_wait_warp(&v_ready, 0);
        tc_fence_after();
        for (int i = 0; i < nn && ok; ++i) {
            const int s = i % kBStages, buf = i & 1;
            if (i >= 2) ok = mbar_wait_warp(&d2_empty[buf], ((i >> 1) - 1) & 1);
            ok = ok && mbar_wait_warp(&b_full[s], (i / kBStages) & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                const uint32_t d = tmem + kD2 + buf * 128;
                const uint64_t bd = b_desc + s * (kBBytes >> 4);
                // v's smallest term first
                for (int e = terms - 1; e >= 0; --e) {
                    const uint32_t a = tmem + kV + e * (Rp / 2);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (16 * k < Rp) mma_ts(d, a + 8 * k, bd + (k >> 2) * (NT * 128 >> 4) + 2 * (k & 3), id2, e != terms - 1 || k != 0);
                }
                mma_commit(&b_empty[s]);
                mma_commit(&d2_full[buf]);
            }
            __syncwarp();
        }
    } else if (warp >= kEpi0) {
        // ------------------------------------------------------- epilogue
        const int ew = warp - kEpi0, quad = ew & 3, half = ew >> 2;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        bool ok = true;
        if (half == 0) {
            ok = mbar_wait_warp(&d1_full, 0);
            tc_fence_after();
            const int r = 32 * quad + lane;
            float* mine = reinterpret_cast<float*>(smem) + (size_t)r * (Rp + 4);
            if (ok) {
                for (int c = 0; c < Rp; c += 16) {
                    uint32_t w[16];
                    tmem_ld16_nowait(tmem + kD2 + lanes + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        *reinterpret_cast<uint4*>(mine + c + k) = nk > 0 ? make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3])
                                                                          : make_uint4(0, 0, 0, 0);
                }
            }
            // the sums over the CTAs, in rank order: each CTA makes those of 128 / ctas rows and gives them to all
            const float* sums_row = mine;
            if (joins) {
                float* parts = reinterpret_cast<float*>(smem);
                float* all = reinterpret_cast<float*>(smem + kRing);  // (where D2 is staged later)
                cluster_arrive();
                cluster_wait();
                const int quarter = Rp / 4, mine_rows = kTile / ctas, first_row = cta * mine_rows;
#pragma unroll 2
                for (int j = threadIdx.x - kEpi0 * 32; j < mine_rows * quarter; j += 128) {
                    const size_t at = (size_t)(first_row + j / quarter) * (Rp + 4) + 4 * (j % quarter);
                    float4 q[8], sum;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < ctas) q[c] = ld_cluster4(parts + at, c);
                    sum = q[0];
#pragma unroll
                    for (int c = 1; c < 8; ++c)
                        if (c < ctas) sum.x += q[c].x, sum.y += q[c].y, sum.z += q[c].z, sum.w += q[c].w;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < ctas) st_cluster4(all + at, c, sum);
                }
                __syncwarp();
                cluster_arrive();
                cluster_wait();
                sums_row = all + (size_t)r * (Rp + 4);
            }
            if (ok) {
                const float scale = p.scale ? __ldg(p.scale + adapter) : 1.0f;
                for (int c = 0; c < Rp; c += 16) {
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = sums_row[c + k];
                    uint32_t term[3][8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t h0, h1, m0, m1;
                        // (columns behind the rank hold what lay in shared memory)
                        const float a = split_bf16(c + 2 * k < p.R ? v[2 * k] * scale : 0.0f, h0);
                        const float b = split_bf16(c + 2 * k + 1 < p.R ? v[2 * k + 1] * scale : 0.0f, h1);
                        term[0][k] = h0 | (h1 << 16);
                        if (OF32) {
                            const float a2 = split_bf16(a, m0), b2 = split_bf16(b, m1);
                            term[1][k] = m0 | (m1 << 16);
                            term[2][k] = f32x2_to_bf16x2_bits(a2, b2);
                        } else {
                            term[1][k] = f32x2_to_bf16x2_bits(a, b);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < (OF32 ? 3 : 2); ++e)
                        tmem_st_cols<8>(tmem + kV + lanes + e * (Rp / 2) + c / 2, term[e]);
                }
                tmem_wait_st();
                tc_fence_before();
                // v's parts and sums have been read: their place goes to the TMA
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(&v_ready);
            }
        }
        // D2, 64 columns at a time.  The warp's 16 KB are v's parts (of the warps that sum them) or sums until v is ready.
        using W = Rows<OF32>;
        uint8_t* own = smem + (sums ? quad : 4 + quad) * (kAhead * kPieceBytes) + (sums ? 0 : kRing - 4 * kAhead * kPieceBytes);
        const int first = NT == 128 ? 0 : half, every = NT == 128 ? 1 : 2, at = NT == 128 ? 64 * half : 0;
        const int row0 = tok[32 * quad];
        const bool run = p.whole && __all_sync(0xFFFFFFFFu, tok[32 * quad + lane] == row0 + lane && row0 >= 0);
        if (run) {
            // 32 tokens one after another: residual and output pass as boxes of 32 rows x 128 bytes through a ring of the
            // warp's own, a lane its row; the sum is written where the residual lay.
            constexpr int kCols = OF32 ? 32 : 64, kPer = 64 / kCols;  // columns of a piece, pieces of 64 columns
            const int pieces = nn > first ? ((nn - first + every - 1) / every) * kPer : 0;
            const auto column_of = [&](int j) { return (cta + (first + (j / kPer) * every) * ctas) * NT + at + (j % kPer) * kCols; };
            const auto fetch = [&](int j) {
                if (lane != 0 || !p.residual || j >= pieces || column_of(j) >= p.N) return;
                const int b = j % kAhead;
                mbar_arrive_expect_tx(&res_full[ew][b], kPieceBytes);
                tma_load_2d(smem_u32(own + b * kPieceBytes), &res_map, column_of(j), row0, &res_full[ew][b]);
            };
            if (!sums) meet_once();
            ok = ok && mbar_wait_warp(&v_ready, 0);
            // (the sums were stored by the other CTAs' threads too)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (ok)
                for (int j = 0; j < kAhead; ++j) fetch(j);
            for (int j = 0; j < pieces && ok; ++j) {
                const int t = j / kPer, i = first + t * every, buf = i & 1, b = j % kAhead;
                if (j % kPer == 0) {
                    ok = mbar_wait_warp(&d2_full[buf], (i >> 1) & 1);
                    tc_fence_after();
                }
                if (ok && column_of(j) >= p.N) {  // the end of the last tile
                    if (j % kPer == kPer - 1 && lane == 0) mbar_arrive(&d2_empty[buf]);
                    continue;
                }
                if (p.residual) ok = mbar_wait_warp(&res_full[ew][b], (j / kAhead) & 1) && ok;
                if (!ok) break;
                uint8_t* row = own + b * kPieceBytes + lane * 128;
                const uint32_t from = tmem + kD2 + lanes + buf * 128 + at + (j % kPer) * kCols;
#pragma unroll
                for (int h = 0; h < kCols; h += 32) {
                    uint32_t d[32];
                    tmem_ld16_nowait(from + h, d);
                    tmem_ld16_nowait(from + h + 16, d + 16);
                    tmem_wait_ld();
                    if (h + 32 == kCols && j % kPer == kPer - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&d2_empty[buf]);
                    }
                    constexpr int kV = OF32 ? 4 : 8;  // columns of 16 bytes
#pragma unroll
                    for (int c = 0; c < 32; c += kV) {
                        // (the 128-byte swizzle: a row's pieces of 16 bytes by its number)
                        uint4* q = reinterpret_cast<uint4*>(row + ((((h + c) / kV) ^ (lane & 7)) << 4));
                        uint4 o = p.residual ? *q : make_uint4(0, 0, 0, 0);
                        const auto f = [&](int k) { return __uint_as_float(d[c + k]); };
                        if constexpr (OF32)
                            o = make_uint4(__float_as_uint(f(0) + __uint_as_float(o.x)), __float_as_uint(f(1) + __uint_as_float(o.y)),
                                           __float_as_uint(f(2) + __uint_as_float(o.z)), __float_as_uint(f(3) + __uint_as_float(o.w)));
                        else
                            o = make_uint4(f32x2_to_bf16x2_bits(f(0) + bf16_lo(o.x), f(1) + bf16_hi(o.x)),
                                           f32x2_to_bf16x2_bits(f(2) + bf16_lo(o.y), f(3) + bf16_hi(o.y)),
                                           f32x2_to_bf16x2_bits(f(4 % kV) + bf16_lo(o.z), f(5 % kV) + bf16_hi(o.z)),
                                           f32x2_to_bf16x2_bits(f(6 % kV) + bf16_lo(o.w), f(7 % kV) + bf16_hi(o.w)));
                        *q = o;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&out_map, column_of(j), row0, smem_u32(own + b * kPieceBytes));
                    // the piece before has been read: its place is free
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                }
                __syncwarp();
                if (j > 0) fetch(j - 1 + kAhead);
            }
            if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            __syncwarp();
        } else {
            float* stage = reinterpret_cast<float*>(own);
            const int col = (lane % W::kLanes) * W::kV, sub = lane / W::kLanes;
            const auto column = [&](int i) { return (cta + i * ctas) * NT + at + col; };
            // the lane's rows, one for each pass, and what it has of them
            int rows[W::kPasses];
#pragma unroll
            for (int k = 0; k < W::kPasses; ++k) rows[k] = tok[32 * quad + k * W::kRows + sub];
            uint4 res[W::kSets][W::kPasses];
#pragma unroll
            for (int a = 0; a < W::kSets; ++a)
#pragma unroll
                for (int k = 0; k < W::kPasses; ++k) res[a][k] = make_uint4(0, 0, 0, 0);
            // Without a choice for each load, which would wait for it: where there is no token or no output, what is
            // read lies in the first row or the last columns, and goes nowhere.
            const auto fetch = [&](uint4* to, int i) {
                if (!p.residual || i >= nn) return;
                const int n = min(column(i), p.N - W::kV);
#pragma unroll
                for (int k = 0; k < W::kPasses; ++k)
                    to[k] = ld_global(static_cast<const uint8_t*>(p.residual) + ((long long)max(rows[k], 0) * p.ldr + n) * (OF32 ? 4 : 2));
            };
#pragma unroll
            for (int a = 0; a < W::kSets; ++a) fetch(res[a], first + a * every);
            if (!sums) meet_once();
            for (int i = first; i < nn && ok; i += W::kSets * every) {
#pragma unroll
                for (int a = 0; a < W::kSets; ++a) {
                    const int j = i + a * every, buf = j & 1;
                    if (j >= nn || !ok) break;
                    ok = mbar_wait_warp(&d2_full[buf], (j >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t from = tmem + kD2 + lanes + buf * 128 + at;
#pragma unroll
                    for (int h = 0; h < 64; h += 32) {
                        uint32_t d[32];
                        tmem_ld16_nowait(from + h, d);
                        tmem_ld16_nowait(from + h + 16, d + 16);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            *reinterpret_cast<uint4*>(stage + lane * kPitch + W::place(h + c)) = make_uint4(d[c], d[c + 1], d[c + 2], d[c + 3]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d2_empty[buf]);
                    // all sums before the first store: stores that may alias what is read would part the passes
                    const int n = column(j);
#pragma unroll
                    for (int k = 0; k < W::kPasses; ++k) {
                        const float* line = stage + (k * W::kRows + sub) * kPitch;
                        const float4 u = *reinterpret_cast<const float4*>(line + W::place(col));
                        uint4& q = res[a][k];
                        if constexpr (OF32) {
                            q = make_uint4(__float_as_uint(u.x + __uint_as_float(q.x)), __float_as_uint(u.y + __uint_as_float(q.y)),
                                           __float_as_uint(u.z + __uint_as_float(q.z)), __float_as_uint(u.w + __uint_as_float(q.w)));
                        } else {
                            const float4 w = *reinterpret_cast<const float4*>(line + W::place(col + 4));
                            q = make_uint4(f32x2_to_bf16x2_bits(u.x + bf16_lo(q.x), u.y + bf16_hi(q.x)),
                                           f32x2_to_bf16x2_bits(u.z + bf16_lo(q.y), u.w + bf16_hi(q.y)),
                                           f32x2_to_bf16x2_bits(w.x + bf16_lo(q.z), w.y + bf16_hi(q.z)),
                                           f32x2_to_bf16x2_bits(w.z + bf16_lo(q.w), w.w + bf16_hi(q.w)));
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < W::kPasses; ++k)
                        if (rows[k] >= 0 && n < p.N)
                            st_global(static_cast<uint8_t*>(p.out) + ((long long)rows[k] * p.ldo + n) * (OF32 ? 4 : 2), res[a][k]);
                    if (!p.residual) {
#pragma unroll
                        for (int k = 0; k < W::kPasses; ++k) res[a][k] = make_uint4(0, 0, 0, 0);
                    }
                    fetch(res[a], j + W::kSets * every);
                }
            }
        }
    } else {
        meet_once();
    }
    // A wait that gave up has left its role's loop; everybody comes here all the same.  After the cluster's
    // second meeting no CTA reads or writes another's shared memory; the MMAs are done with tensor
    // memory (the epilogue has waited for every one of them).
    __syncwarp();
    if (joins && !sums) cluster_wait();
    tc_fence_before();
    __syncthreads();
    pdl_end();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<false>(tmem, kColumns);
}

template <bool OF32>
cudaError_t launch(const Lora& p, const CUtensorMap* x, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& res,
                   const CUtensorMap& out, int items, cudaStream_t s) {
    const auto kernel = lora_prompt_kernel<OF32>;
    const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmem);
    if (err != cudaSuccess) return err;
    if (p.ctas == 1) return launch_pdl(kernel, dim3((unsigned)items), dim3(kThreads), kSmem, s, p, x[0], x[1], x[2], a, b, res, out);
    return launch_pdl_cluster(kernel, dim3((unsigned)(items * p.ctas)), dim3(kThreads), kSmem, s, p.ctas, p, x[0], x[1], x[2], a, b, res, out);
}

}  // namespace

// Rows that TMA can fetch and the epilogue access 16 bytes at a time, whole ranks (B's columns behind
// a rank would be multiplied), coordinates of 31 bits.
bool lora_prompt_supported(const Lora& p) {
    return p.tile_m == kTile && !p.x_f32 && p.x_wide && p.ldx >= p.K && p.out_wide && (!p.residual || p.res_wide) &&
           p.N % 8 == 0 && !p.ranks && (long long)p.adapters * p.N < (1LL << 31) && p.ldx < (1LL << 38) &&
           p.ldo < (1LL << 37) && p.ldr < (1LL << 37);
}

cudaError_t launch_lora_prompt(const Lora& given, cudaStream_t s) {
    Lora p = given;
    CUtensorMap x[3], a, b, res, out;  // x by 1 (gathers), 8 and 32 rows
    const int NT = p.R <= 64 ? 128 : 64;
    cudaError_t err = cudaSuccess;
    for (int i = 0; i < 3 && err == cudaSuccess; ++i)
        err = encode_2d_map(&x[i], p.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.K, p.T, (uint64_t)p.ldx * 2, 64,
                            i == 0 ? 1 : i == 1 ? 8 : 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (err == cudaSuccess)
        err = encode_2d_map(&a, p.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.K, (uint64_t)p.adapters * p.R, (uint64_t)p.K * 2, 64,
                            p.R, CU_TENSOR_MAP_SWIZZLE_128B);
    if (err == cudaSuccess)
        err = encode_2d_map(&b, p.b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.R, (uint64_t)p.adapters * p.N, (uint64_t)p.R * 2, 64,
                            NT, CU_TENSOR_MAP_SWIZZLE_128B);
    // residual and output as boxes of 32 rows x 128 bytes, where no rows of the residual overlap
    p.whole = !p.residual || p.ldr >= p.N;
    const CUtensorMapDataType type = p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int size = p.out_f32 ? 4 : 2;
    if (err == cudaSuccess)
        err = encode_2d_map(&out, p.out, type, p.N, p.T, (uint64_t)p.ldo * size, 128 / size, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    res = out;
    if (err == cudaSuccess && p.residual && p.whole)
        err = encode_2d_map(&res, p.residual, type, p.N, p.T, (uint64_t)p.ldr * size, 128 / size, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (err != cudaSuccess) return err;
    // CTAs a tile: as many as one for each SM allows, for the tiles there are likely to be (clusters of 8
    // leave a sixth of the SMs out, clusters of 4 some).  In us with 1, 2, 4 and 8, 4096 -> 4096 at rank 64: 1024 tokens of
    // 2 adapters 68, 42, 26, 19; 2048 of 2 68, 42, 27, 36; 8192 of 11 71, 49, 57, 93; 16384 of 8 77, 93, 109, 167.
    const int likely = p.T / kTile + std::min(p.adapters, p.T / kTile + 1) / 2 + 1, sms = num_sms();
    p.ctas = 8;
    while (p.ctas > 1 && (likely * p.ctas > (p.ctas == 8 ? sms * 5 / 6 : p.ctas == 4 ? sms * 15 / 16 : sms) ||
                          p.ctas * 128 > std::max(p.K, p.N)))
        p.ctas /= 2;
    const bool in_place = p.residual == p.out && p.ldr == p.ldo;
    const int items = p.tiles + (in_place ? 0 : (p.T + kThreads - 1) / kThreads);
    return p.out_f32 ? launch<true>(p, x, a, b, res, out, items, s) : launch<false>(p, x, a, b, res, out, items, s);
}

cudaError_t read_device_error_lora_prompt(int* flag, int clear) {
    int wait = 0, index = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&wait, g_device_error, sizeof(int));
    if (err == cudaSuccess) err = cudaMemcpyFromSymbol(&index, g_index_error, sizeof(int));
    if (err != cudaSuccess) return err;
    *flag = (wait ? 1 : 0) | (index ? 2 : 0);
    if (!clear) return cudaSuccess;
    const int zero = 0;
    err = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
    return err == cudaSuccess ? cudaMemcpyToSymbol(g_index_error, &zero, sizeof(int)) : err;
}

}  // namespace moe
