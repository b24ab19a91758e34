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

// The sum over the block's threads, the same on each of them: warps in order.
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5;
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

// Thread i of the block has the chunks i, i + threads, ... of V values.
template <int V, int CH>
__global__ void __launch_bounds__(1024) combine_norm_kernel(const __grid_constant__ CombineNorm p) {
    __shared__ float sums[2][32];
    pdl_begin();
    const long long t = blockIdx.x;
    const int step = blockDim.x * V, c0 = threadIdx.x * V;
    float u[CH][V], h[CH][V];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) u[i][k] = h[i][k] = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
        if (c0 + i * step < p.H) load_values<V>(p.y, p.y_f32, t * p.slots * p.ldy + c0 + i * step, u[i]);
    if (p.h) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) load_values<V>(p.h, p.h_f32, t * p.ldh + c0 + i * step, h[i]);
    }
    for (int j = 1; j < p.slots; ++j) {
        float v[CH][V];
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) load_values<V>(p.y, p.y_f32, (t * p.slots + j) * p.ldy + c0 + i * step, v[i]);
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) {
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] += v[i][k];
            }
    }
    const float inv = 1.0f / (float)p.H;
    if (p.post) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) q += u[i][k] * u[i][k];
        const float r = 1.0f / sqrtf(block_sum(q, sums[0]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) {
                float w[V];
                load_values<V>(p.post_w, p.w_f32, c0 + i * step, w);
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] *= r * (w[k] + p.w_offset);
            }
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
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (c0 + i * step < p.H) {
                    float z[V];
                    load_values<V>(p.gate, p.gate_f32, t * p.ldg + c0 + i * step, z);
#pragma unroll
                    for (int k = 0; k < V; ++k) u[i][k] *= gate_of(z[k], p.act);
                }
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
        const float r = 1.0f / sqrtf(block_sum(q, sums[1]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c0 + i * step < p.H) {
                float w[V];
                if (p.pre_w) load_values<V>(p.pre_w, p.w_f32, c0 + i * step, w);
#pragma unroll
                for (int k = 0; k < V; ++k) w[k] = u[i][k] * r * (p.pre_w ? w[k] + p.w_offset : 1.0f);
                store_values<V>(p.n_out, p.n_f32, t * p.ldn + c0 + i * step, w);
            }
    }
    pdl_end();
}

template <int V, int CH>
cudaError_t launch(const CombineNorm& p, cudaStream_t s) {
    const int threads = ((p.H + V * CH - 1) / (V * CH) + 31) / 32 * 32;
    return launch_pdl(combine_norm_kernel<V, CH>, dim3(p.T), dim3(threads), 0, s, p);
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
    if (vectors(p, 8)) return p.H <= 256 ? launch<8, 1>(p, s) : launch<8, 2>(p, s);
    if (vectors(p, 4)) return p.H <= 512 ? launch<4, 2>(p, s) : launch<4, 4>(p, s);
    return p.H <= 1024 ? launch<1, 4>(p, s) : launch<1, 16>(p, s);
}

}  // namespace moe
