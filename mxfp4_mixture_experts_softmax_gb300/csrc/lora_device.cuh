// lora_device.cuh -- what the two kernels of the low-rank adapters share (lora.cu, lora_prompt.cu).
#pragma once

#include "moe_internal.h"

namespace moe {

// v = hi + the return value, hi the upper 16 bits (a bf16, exact); infinities and
// NaN stay whole in hi.
__device__ __forceinline__ float split_bf16(float v, uint32_t& hi) {
    const uint32_t b = __float_as_uint(v);
    if ((b & 0x7F800000u) == 0x7F800000u) {
        hi = (b & 0x007FFFFFu) ? 0x7FC0u : b >> 16;
        return 0.0f;
    }
    hi = b >> 16;
    return v - __uint_as_float(b & 0xFFFF0000u);
}

// Eight values of a row of `out`'s type from element n on; those from `count` on are not touched.
__device__ __forceinline__ void load_out(const void* base, int f32, long long i, int count, bool wide, float* v) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (f32) {
        const float* q = static_cast<const float*>(base) + i;
        if (wide && count >= 8) {
            const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) v[k] = q[k];
        }
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(base) + i;
        if (wide && count >= 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(q);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) v[k] = __uint_as_float((uint32_t)q[k] << 16);
        }
    }
}

__device__ __forceinline__ void store_out(void* base, int f32, long long i, int count, bool wide, const float* v) {
    if (f32) {
        float* q = static_cast<float*>(base) + i;
        if (wide && count >= 8) {
            *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) q[k] = v[k];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(base) + i;
        if (wide && count >= 8)
            *reinterpret_cast<uint4*>(q) = make_uint4(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]),
                                                      f32x2_to_bf16x2_bits(v[4], v[5]), f32x2_to_bf16x2_bits(v[6], v[7]));
        else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) q[k] = f32_to_bf16_bits(v[k]);
        }
    }
}

// Rows without an adapter among tokens [t0, t0 + THREADS): residual or zeros.  Each warp has 32 of
// the tokens and takes every ctas-th of their rows.
template <int THREADS>
__device__ __forceinline__ void copy_rows(const Lora& p, int t0, int cta, int ctas) {
    const int lane = threadIdx.x & 31, first = t0 + ((int)threadIdx.x & ~31);
    const bool bare = first + lane < p.T && __ldg(p.inv_pairs + first + lane) < 0;
    uint32_t rows = __ballot_sync(0xFFFFFFFFu, bare);
    for (int turn = 0; rows; ++turn) {
        const int t = first + __ffs((int)rows) - 1;
        rows &= rows - 1;
        if (turn % ctas != cta) continue;
        for (int n = 8 * lane; n < p.N; n += 256) {
            float v[8];
            load_out(p.residual, p.out_f32, (long long)t * p.ldr + n, p.residual ? p.N - n : 0, p.res_wide, v);
            store_out(p.out, p.out_f32, (long long)t * p.ldo + n, p.N - n, p.out_wide, v);
        }
    }
}

}  // namespace moe
