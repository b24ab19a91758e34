// combine_norm.cu -- what lies between two blocks of a decoder, one pass over a
// token's row:
//
//   y = sum over the slots j ascending of y[t * slots + j]
//   u = [N(y; post_w)] [* act(gate)];   h' = beta h + alpha u;   n = N(h'; pre_w)
//   N(v; w) = v / sqrt(mean(v^2) + eps) * (w + w_offset)
//
// Everything is fp32 between the loads and the two stores; n is the norm of h' before
// its rounding to h_out.  The row stays in registers, so each value is read and
// written once and the kernel is bound by HBM where there are many tokens, by
// latency (launch, the loads, one or two block sums) where there are few.
#include <algorithm>

#include "moe_internal.h"

namespace moe {

namespace {

// V neighbouring values at p + i (elements), rows of bf16 or fp32.
template <int V>
__device__ __forceinline__ void load_values(const void* p, int f32, long long i, float* v) {
    if (f32) {
        const float* q = static_cast<const float*>(p) + i;
        if constexpr (V == 8) {
            const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else if constexpr (V == 4) {
            const float4 a = *reinterpret_cast<const float4*>(q);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        } else {
            v[0] = *q;
        }
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i;
        if constexpr (V == 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(q);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        } else if constexpr (V == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(q);
            v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
            v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
        } else {
            v[0] = __uint_as_float((uint32_t)*q << 16);
        }
    }
}

// A thread's CH chunks of a row of H values: c, c + step, ...; zeros behind its end.  The type is decided
// once and the addresses stay in the row, so that all loads are in flight together (with a
// branch around each: 250 us for 4000 rows of 2087, one load waiting for the other).
template <int V, int CH>
__device__ __forceinline__ void load_row(const void* p, int f32, long long row, int c, int step, int H, float (*v)[V]) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < CH; ++i) load_values<V>(p, 1, row + min(c + i * step, H - V), v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) load_values<V>(p, 0, row + min(c + i * step, H - V), v[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = c + i * step < H ? v[i][k] : 0.0f;
}

template <int V>
__device__ __forceinline__ void store_values(void* p, int f32, long long i, const float* v) {
    if (f32) {
        float* q = static_cast<float*>(p) + i;
        if constexpr (V == 1) {
            *q = v[0];
        } else {
#pragma unroll
            for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(q + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(q) = make_uint4(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]),
                                                      f32x2_to_bf16x2_bits(v[4], v[5]), f32x2_to_bf16x2_bits(v[6], v[7]));
        else if constexpr (V == 4)
            *reinterpret_cast<uint2*>(q) = make_uint2(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]));
        else
            *q = f32_to_bf16_bits(v[0]);
    }
}

// The sum over a row's threads, the same on each of them: one warp's, or the block's warps in order.
__device__ __forceinline__ float row_sum(float v, int warps, float* slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float gate_of(float z, int act) {
    if (act == 0) return z;
    const float e = expf(-fabsf(z));
    const float s = (z >= 0.0f ? 1.0f : e) / (1.0f + e);
    return act == 1 ? s : z * s;
}

// One row at a time: thread i of its p.row_warps warps has the chunks i, i + threads, ... of V values.
// Rows of one warp share a block of up to 8.
template <int V, int CH, int MOST>
__global__ void __launch_bounds__(MOST) combine_norm_kernel(const __grid_constant__ CombineNorm p) {
    __shared__ float sums[2][32];
    pdl_begin();
    const int threads = p.row_warps * 32, rank = p.row_warps == 1 ? threadIdx.x & 31 : threadIdx.x;
    const long long t = p.row_warps == 1 ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= p.T) return;
    const int step = threads * V, c0 = rank * V;
    float u[CH][V], h[CH][V];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] = 0.0f;
    if (p.h) load_row<V, CH>(p.h, p.h_f32, t * p.ldh, c0, step, p.H, h);
    // the slots in order, the loads of several together
    load_row<V, CH>(p.y, p.y_f32, t * p.slots * p.ldy, c0, step, p.H, u);
    if constexpr (V == 8 && CH == 1) {
        for (int j = 1; j < p.slots; j += 4) {
            float v[4][V];
#pragma unroll
            for (int a = 0; a < 4; ++a)
                if (j + a < p.slots && c0 < p.H) load_values<V>(p.y, p.y_f32, (t * p.slots + j + a) * p.ldy + c0, v[a]);
#pragma unroll
            for (int a = 0; a < 4; ++a)
                if (j + a < p.slots && c0 < p.H) {
#pragma unroll
                    for (int k = 0; k < V; ++k) u[0][k] += v[a][k];
                }
        }
    } else {
        for (int j = 1; j < p.slots; j += 2) {
            float v[2][CH][V];
            const bool both = j + 1 < p.slots;
            load_row<V, CH>(p.y, p.y_f32, (t * p.slots + j) * p.ldy, c0, step, p.H, v[0]);
            load_row<V, CH>(p.y, p.y_f32, (t * p.slots + j + (both ? 1 : 0)) * p.ldy, c0, step, p.H, v[1]);
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    u[i][k] += v[0][i][k];
                    if (both) u[i][k] += v[1][i][k];
                }
        }
    }
    const float inv = 1.0f / (float)p.H;
    if (p.post) {
        float w[CH][V];
        load_row<V, CH>(p.post_w, p.w_f32, 0, c0, step, p.H, w);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) q += u[i][k] * u[i][k];
        const float r = rsqrtf(row_sum(q, p.row_warps, sums[0]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) u[i][k] *= r * (w[i][k] + p.w_offset);
    }
    if (p.gate) {
        if (p.gate_cols == 1) {
            float z;
            load_values<1>(p.gate, p.gate_f32, t * p.ldg, &z);
            z = gate_of(z, p.act);
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] *= z;
        } else {
            float z[CH][V];
            load_row<V, CH>(p.gate, p.gate_f32, t * p.ldg, c0, step, p.H, z);
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] *= gate_of(z[i][k], p.act);
        }
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            // without a residual h is 0, and what beta is does not matter
            u[i][k] = p.h ? p.beta * h[i][k] + p.alpha * u[i][k] : p.alpha * u[i][k];
            if (c0 + i * step < p.H) q += u[i][k] * u[i][k];
        }
    if (p.h_out) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) store_values<V>(p.h_out, p.h_f32, t * p.ldho + c0 + i * step, u[i]);
    }
    if (p.n_out) {
        float w[CH][V];
        if (p.pre_w) load_row<V, CH>(p.pre_w, p.w_f32, 0, c0, step, p.H, w);
        const float r = rsqrtf(row_sum(q, p.row_warps, sums[1]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) {
#pragma unroll
                for (int k = 0; k < V; ++k) w[i][k] = u[i][k] * r * (p.pre_w ? w[i][k] + p.w_offset : 1.0f);
                store_values<V>(p.n_out, p.n_f32, t * p.ldn + c0 + i * step, w[i]);
            }
    }
    pdl_end_block();
}

// Eight values as they lie in memory.
template <bool F32>
struct Raw {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, long long i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) w[k] = q[k];
    }
    __device__ __forceinline__ void get(float* v) const {
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) {
            const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    v[4 * k + j] = __uint_as_float(x[j]);
                } else {
                    v[2 * j] = __uint_as_float(x[j] << 16);
                    v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                }
            }
        }
    }
};

// The sum over a block of up to 16 warps, in order; slots behind the last warp's hold 0.
__device__ __forceinline__ float block_sum(float v, int warps, float* slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < warps; w += 4) {
        const float4 s = *reinterpret_cast<const float4*>(slots + w);
        v += (s.x + s.y) + (s.z + s.w);
    }
    return v;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// factors[i] = alpha times the weight after the block times a gate that all rows share (if there
// is one: returned), factors[H + i] = the weight before the next block.  The caller synchronises.
__device__ __forceinline__ bool fill_factors(const CombineNorm& p, float* factors) {
    const bool shared_gate = p.gate && p.gate_cols != 1 && p.ldg == 0;
    for (int i = 8 * threadIdx.x; i < p.H; i += 8 * blockDim.x) {
        float f[8], w[8], v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = p.alpha, w[k] = 1.0f;
        if (p.post) {
            load_values<8>(p.post_w, p.w_f32, i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= v[k] + p.w_offset;
        }
        if (shared_gate) {
            load_values<8>(p.gate, p.gate_f32, i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= gate_of(v[k], p.act);
        }
        if (p.pre_w) {
            load_values<8>(p.pre_w, p.w_f32, i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = v[k] + p.w_offset;
        }
        store_values<8>(factors, 1, i, f);
        store_values<8>(factors + p.H, 1, i, w);
    }
    return shared_gate;
}

// Many short rows (up to 512 values), no slots.  A row has `lanes` lanes of a warp (8 to 32), and a
// thread two times 8 neighbouring values of it; rows are taken in turn, the next one's y and h loaded
// before the work on this one.  What is the same for every row -- alpha, the weights after the
// block and a gate that all rows share, as one factor, and the weights before the next one -- lies
// in shared memory.  262144 rows of 128, bf16: 50.5 us (5.3 TB/s), with an fp32 stream 64 (6.3 TB/s); 40000 rows 10.8 (3.8 TB/s).
// (79 registers a thread, with fp32 rows 87 to 109: three of the four blocks for each SM run at once, or two.)
constexpr int kShortRow = 512, kShortThreads = 256;
template <bool YF, bool HF>
__global__ void __launch_bounds__(kShortThreads) combine_norm_short_kernel(const __grid_constant__ CombineNorm p) {
    extern __shared__ __align__(16) float factors[];  // [2][H]
    pdl_begin();
    const int lanes = p.row_lanes, rows = kShortThreads / lanes, rank = threadIdx.x & (lanes - 1);
    const bool shared_gate = fill_factors(p, factors);
    __syncthreads();

    const int c[2] = {8 * rank, 8 * (rank + lanes)};
    const bool in[2] = {c[0] < p.H, c[1] < p.H};
    long long t = (long long)blockIdx.x * rows + threadIdx.x / lanes;
    const long long step = (long long)gridDim.x * rows;
    // (the rows of a block end their turns together: a warp's meet in the sums)
    const long long last = ((long long)p.T + rows - 1) / rows * rows;
    Raw<YF> y[2];
    Raw<HF> h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < (YF ? 2 : 1); ++k) y[i].w[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < (HF ? 2 : 1); ++k) h[i].w[k] = make_uint4(0, 0, 0, 0);
        if (in[i] && t < p.T) {
            y[i].load(p.y, t * p.ldy + c[i]);
            if (p.h) h[i].load(p.h, t * p.ldh + c[i]);
        }
    }
    const float inv = 1.0f / (float)p.H;
    for (; t < last; t += step) {
        const bool live = t < p.T;
        float u[2][8];
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            y[i].get(u[i]);
            if (in[i] && t + step < p.T) y[i].load(p.y, (t + step) * p.ldy + c[i]);
        }
        float f = 1.0f;
        if (p.post) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) q += u[i][k] * u[i][k];
            f = rsqrtf(lanes_sum(q, lanes) * inv + p.eps);
        }
        if (p.gate && !shared_gate && live) {
            if (p.gate_cols == 1) {
                float z;
                load_values<1>(p.gate, p.gate_f32, t * p.ldg, &z);
                f *= gate_of(z, p.act);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (in[i]) {
                        float z[8];
                        load_values<8>(p.gate, p.gate_f32, t * p.ldg + c[i], z);
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[i][k] *= gate_of(z[k], p.act);
                    }
            }
        }
        q = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float r[8];
            h[i].get(r);
            if (p.h && in[i] && t + step < p.T) h[i].load(p.h, (t + step) * p.ldh + c[i]);
            if (in[i]) {
                const float4 a = *reinterpret_cast<const float4*>(factors + c[i]), b = *reinterpret_cast<const float4*>(factors + c[i] + 4);
                const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    u[i][k] = p.h ? p.beta * r[k] + u[i][k] * f * w[k] : u[i][k] * f * w[k];
                    q += u[i][k] * u[i][k];
                }
                if (p.h_out && live) store_values<8>(p.h_out, p.h_f32, t * p.ldho + c[i], u[i]);
            }
        }
        if (p.n_out) {
            const float g = rsqrtf(lanes_sum(q, lanes) * inv + p.eps);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (in[i]) {
                    const float4 a = *reinterpret_cast<const float4*>(factors + p.H + c[i]),
                                 b = *reinterpret_cast<const float4*>(factors + p.H + c[i] + 4);
                    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[i][k] = u[i][k] * g * w[k];
                    if (live) store_values<8>(p.n_out, p.n_f32, t * p.ldn + c[i], u[i]);
                }
        }
    }
    pdl_end_block();
}

// Many longer rows, no slots.  A block takes rows in turn; one thread keeps the next rows' y, h and
// gate coming as bulk copies into a ring of p.stages in shared memory, so that HBM always has whole rows
// of every block outstanding (with the next row in registers instead: 62 us for 8192 rows of 4096 with
// norms on both sides, a row a block without turns: 76).  A thread has the chunks i and i + threads
// of 8 values.
constexpr int kStreamThreads = 512;
template <bool YF, bool HF>
__global__ void __launch_bounds__(kStreamThreads) combine_norm_stream_kernel(const __grid_constant__ CombineNorm p) {
    extern __shared__ __align__(16) float factors[];  // [2][H], then the ring
    __shared__ __align__(16) float sums[2][2][16];
    __shared__ __align__(8) uint64_t full[kCombineNormStages];
    pdl_begin();
    const int warps = blockDim.x >> 5;
    const uint32_t y_bytes = p.H * (YF ? 4 : 2), h_bytes = p.h ? p.H * (HF ? 4 : 2) : 0;
    const bool full_gate = p.gate && p.gate_cols != 1 && p.ldg != 0;
    const uint32_t g_bytes = full_gate ? p.H * (p.gate_f32 ? 4 : 2) : 0, stage_bytes = y_bytes + h_bytes + g_bytes;
    uint8_t* ring = reinterpret_cast<uint8_t*>(factors + 2 * p.H);
    if (threadIdx.x < 64) (&sums[0][0][0])[threadIdx.x] = 0.0f;
    const auto fetch = [&](long long t, int stage) {
        uint8_t* to = ring + (size_t)stage * stage_bytes;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        bulk_copy_g2s(smem_u32(to), static_cast<const uint8_t*>(p.y) + t * p.ldy * (YF ? 4 : 2), y_bytes, &full[stage]);
        if (h_bytes)
            bulk_copy_g2s(smem_u32(to + y_bytes), static_cast<const uint8_t*>(p.h) + t * p.ldh * (HF ? 4 : 2), h_bytes, &full[stage]);
        if (g_bytes)
            bulk_copy_g2s(smem_u32(to + y_bytes + h_bytes),
                          static_cast<const uint8_t*>(p.gate) + t * p.ldg * (p.gate_f32 ? 4 : 2), g_bytes, &full[stage]);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < p.stages; ++i) {
            const long long t = blockIdx.x + (long long)i * gridDim.x;
            if (t < p.T) fetch(t, i);
        }
    }
    __syncwarp();
    const bool shared_gate = fill_factors(p, factors);
    __syncthreads();

    const int c[2] = {8 * (int)threadIdx.x, 8 * (int)(threadIdx.x + blockDim.x)};
    const bool in[2] = {c[0] < p.H, c[1] < p.H};
    const float inv = 1.0f / (float)p.H;
    int stage = 0, parity = 0, turn = 0;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        // (a wait that gave up has raised the error flag; the row is then not what it should be, and the
        // block goes on so that its threads stay together)
        mbar_wait(&full[stage], parity);
        const uint8_t* from = ring + (size_t)stage * stage_bytes;
        float u[2][8], r[2][8];
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) u[i][k] = r[i][k] = 0.0f;
            if (in[i]) {
                load_values<8>(from, YF, c[i], u[i]);
                if (h_bytes) load_values<8>(from + y_bytes, HF, c[i], r[i]);
            }
        }
        float f = 1.0f;
        if (p.post) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) q += u[i][k] * u[i][k];
            f = rsqrtf(block_sum(q, warps, sums[turn][0]) * inv + p.eps);
        }
        if (full_gate) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (in[i]) {
                    float z[8];
                    load_values<8>(from + y_bytes + h_bytes, p.gate_f32, c[i], z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[i][k] *= gate_of(z[k], p.act);
                }
        } else if (p.gate && !shared_gate) {
            float z;
            load_values<1>(p.gate, p.gate_f32, t * p.ldg, &z);
            f *= gate_of(z, p.act);
        }
        q = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (in[i]) {
                float w[8];
                load_values<8>(factors, 1, c[i], w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    u[i][k] = h_bytes ? p.beta * r[i][k] + u[i][k] * f * w[k] : u[i][k] * f * w[k];
                    q += u[i][k] * u[i][k];
                }
            }
        // (every thread is past its reads of the stage when the sum is done)
        const float g = rsqrtf(block_sum(q, warps, sums[turn][1]) * inv + p.eps);
        if (threadIdx.x == 0 && t + (long long)p.stages * gridDim.x < p.T) fetch(t + (long long)p.stages * gridDim.x, stage);
        if (++stage == p.stages) stage = 0, parity ^= 1;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (in[i]) {
                if (p.h_out) store_values<8>(p.h_out, p.h_f32, t * p.ldho + c[i], u[i]);
                if (p.n_out) {
                    float w[8];
                    load_values<8>(factors + p.H, 1, c[i], w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[i][k] = u[i][k] * g * w[k];
                    store_values<8>(p.n_out, p.n_f32, t * p.ldn + c[i], u[i]);
                }
            }
    }
    pdl_end_block();
}

template <int V, int CH, int MOST>
cudaError_t launch(CombineNorm p, cudaStream_t s) {
    p.row_warps = ((p.H + V * CH - 1) / (V * CH) + 31) / 32;
    const int rows = p.row_warps == 1 ? std::min(8, p.T) : 1;
    return launch_pdl(combine_norm_kernel<V, CH, MOST>, dim3((unsigned)(((long long)p.T + rows - 1) / rows)),
                      dim3(p.row_warps * 32 * rows), 0, s, p);
}

template <bool YF, bool HF>
cudaError_t launch_short(CombineNorm p, cudaStream_t s) {
    p.row_lanes = 8;
    while (16 * p.row_lanes < p.H) p.row_lanes *= 2;
    const int rows = kShortThreads / p.row_lanes;
    const long long blocks = std::min<long long>(num_sms() * 4LL, ((long long)p.T + rows - 1) / rows);
    return launch_pdl(combine_norm_short_kernel<YF, HF>, dim3((unsigned)blocks), dim3(kShortThreads), 2 * sizeof(float) * p.H, s, p);
}

// The stream kernel's threads, blocks an SM and stages for these rows: up to 1024 threads an SM, as
// long as two stages fit each block, and the ring takes what is left.  0 stages: they do not fit.
struct StreamShape {
    int threads, per_sm, stages;
    size_t smem;
};
StreamShape stream_shape(const CombineNorm& p) {
    const bool full_gate = p.gate && p.gate_cols != 1 && p.ldg != 0;
    const size_t stage = (size_t)p.H * ((p.y_f32 ? 4 : 2) + (p.h ? (p.h_f32 ? 4 : 2) : 0) + (full_gate ? (p.gate_f32 ? 4 : 2) : 0));
    const size_t factors = 2 * sizeof(float) * p.H, most = 220 * 1024, fixed = 1024;  // a block's own 1 KB
    StreamShape r;
    r.threads = ((p.H / 8 + 1) / 2 + 31) / 32 * 32;
    r.per_sm = std::max(1, 1024 / r.threads);
    while (r.per_sm > 1 && (factors + 2 * stage + fixed) * r.per_sm > most) --r.per_sm;
    const size_t room = most / r.per_sm - fixed;
    r.stages = factors + 2 * stage > room ? 0 : (int)std::min<size_t>(kCombineNormStages, (room - factors) / stage);
    r.smem = factors + r.stages * stage;
    return r;
}

template <bool YF, bool HF>
cudaError_t launch_stream(CombineNorm p, const StreamShape& shape, cudaStream_t s) {
    const auto kernel = combine_norm_stream_kernel<YF, HF>;
    p.stages = shape.stages;
    const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), shape.smem + 1024);
    if (err != cudaSuccess) return err;
    return launch_pdl(kernel, dim3((unsigned)std::min<long long>((long long)num_sms() * shape.per_sm, p.T)), dim3(shape.threads),
                      shape.smem, s, p);
}

// Whether rows of this type, `ld` elements apart, can be read V values at a time.
bool vectors(const void* p, int f32, long long ld, int V) {
    const size_t bytes = f32 ? 16 : 2 * V;  // (fp32 in pieces of 16 bytes)
    return !p || ((uintptr_t)p % bytes == 0 && (size_t)(ld * (f32 ? 4 : 2)) % bytes == 0);
}

bool vectors(const CombineNorm& p, int V) {
    return p.H % V == 0 && vectors(p.y, p.y_f32, p.ldy, V) && vectors(p.h, p.h_f32, p.ldh, V) &&
           vectors(p.h_out, p.h_f32, p.ldho, V) && vectors(p.n_out, p.n_f32, p.ldn, V) &&
           vectors(p.post_w, p.w_f32, 0, V) && vectors(p.pre_w, p.w_f32, 0, V) &&
           (p.gate_cols == 1 || vectors(p.gate, p.gate_f32, p.ldg, V));
}

}  // namespace

cudaError_t launch_combine_norm(const CombineNorm& p, cudaStream_t s) {
    if (vectors(p, 8)) {
        // Without slots and with rows for several turns of every block, 32768 values an SM.  A row a block against turns,
        // in us: rows of 4096, 8192 values an SM 4.5 and 5.0, 16384 8.1 and 7.7, 32768 14.9 and 11.3, 262144 107 and 53;
        // rows of 128, 2048 values an SM 2.4 and 2.7, 8192 6.6 and 4.6, 32768 22.6 and 11.3.
        if (p.slots == 1 && (long long)p.T * p.H >= 2LL * 16 * 1024 * num_sms()) {
            if (p.H <= kShortRow) {
                if (p.y_f32) return p.h_f32 ? launch_short<true, true>(p, s) : launch_short<true, false>(p, s);
                return p.h_f32 ? launch_short<false, true>(p, s) : launch_short<false, false>(p, s);
            }
            const StreamShape shape = stream_shape(p);
            if (p.H <= 16 * kStreamThreads && shape.stages > 0) {
                if (p.y_f32) return p.h_f32 ? launch_stream<true, true>(p, shape, s) : launch_stream<true, false>(p, shape, s);
                return p.h_f32 ? launch_stream<false, true>(p, shape, s) : launch_stream<false, false>(p, shape, s);
            }
        }
        return p.H <= 8192 ? launch<8, 1, 1024>(p, s) : launch<8, 2, 1024>(p, s);
    }
    if (vectors(p, 4)) return p.H <= 4096 ? launch<4, 2, 512>(p, s) : launch<4, 4, 1024>(p, s);
    return p.H <= 4096 ? launch<1, 8, 512>(p, s) : launch<1, 16, 1024>(p, s);
}

cudaError_t read_device_error_norm(int* flag, int clear) {
    int wait = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&wait, g_device_error, sizeof(int));
    if (err != cudaSuccess) return err;
    *flag = wait ? 1 : 0;
    if (!clear) return cudaSuccess;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace moe
