// mxf4.cuh -- MXFP4 x MXFP4 tensor-core helpers (tcgen05.mma kind::mxf4) and
// the device-side MXFP4 encoding, shared by the grouped expert GEMMs
// (ffn_mxfp4act.cu) and the dense product (linear_mxfp4.cu).
#pragma once

#include "moe_device.cuh"

namespace moe {

// Instruction descriptor, kind::mxf4: E2M1 x E2M1 -> fp32, E8M0 scales, both
// operands K-major, M x N, scale id `sf` for both operands.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf << 29);
}

// D (tensor memory) += A * B, both from shared memory, scale factors of A
// and B in tensor memory (block size 32 along K).
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// The CTA-pair form (issued by the pair's even CTA): M = 256, A and its scale
// factors from each CTA's own shared and tensor memory, B's N columns from the two
// CTAs' halves, B's scale factors complete in both.
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t* v);
template <>
__device__ __forceinline__ void tmem_st_cols<1>(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v[0]) : "memory");
}
template <>
__device__ __forceinline__ void tmem_st_cols<2>(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1])
                 : "memory");
}
template <>
__device__ __forceinline__ void tmem_st_cols<4>(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
template <>
__device__ __forceinline__ void tmem_st_cols<8>(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                 "r"(v[7])
                 : "memory");
}

// ------------------------------------------------------------ quantisation

// Two values -> one byte of E2M1 codes (lo in the low nibble), rounded to
// nearest even with saturation to +-6 by the hardware conversion.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Scale byte of a block whose largest magnitude is amax (>= 0):
// floor(log2 amax) - 2 + 127 = biased exponent - 2, clamped at 0 (zero and
// subnormal amax, and blocks whose exponent would fall below -127).
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    return (uint32_t)max((int)((__float_as_uint(amax) >> 23) & 0xFFu) - 2, 0);
}

// 2^-(sbyte - 127) as fp32 (sbyte <= 252, so the exponent field 254 - sbyte
// stays finite).
__device__ __forceinline__ float mx_inv_scale(uint32_t sbyte) {
    return __uint_as_float((254u - sbyte) << 23);
}

// Eight values times f -> four bytes of codes (v[0] in the lowest nibble).
__device__ __forceinline__ uint32_t e2m1x8(const float* v, float f) {
    return e2m1x2(v[0] * f, v[1] * f) | (e2m1x2(v[2] * f, v[3] * f) << 8) |
           (e2m1x2(v[4] * f, v[5] * f) << 16) | (e2m1x2(v[6] * f, v[7] * f) << 24);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(smem_u32(p)));
    return v;
}

}  // namespace moe
