// route_grouped.cu -- routing with softmax or sigmoid scores, a bias for
// balance and expert groups, one warp per token.
//
//   s = softmax(l) or 1 / (1 + e^-l);   c = s + b   (without b: ordered as l)
//   value of a group = its largest c, or the sum of its two largest
//   the `chosen` groups of the largest values stay; of their experts the K
//   largest c, in descending order;   w = scale * s [/ sum of the chosen s]
// Equal values go to the lower index everywhere.
//
// The choice has to be that of the exact values, so it is made on fp32 values
// whose error has a bound (kErr below), and a token with two values closer than
// twice that bound, where it matters, is chosen again on 64-bit values
// (choose64): one token in some hundreds.  Without a bias and with groups
// ranked by their largest expert the order is the logits' own and needs none of
// this.
//
// A group's experts lie in one lane or in neighbouring ones, so that group values
// are reductions over P = 32 / (groups rounded up to a power of two) lanes.
#include "moe_internal.h"
#include "route_device.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
    float v;
    if (BF16)
        v = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(row) + e) << 16);
    else
        v = __ldg(static_cast<const float*>(row) + e);
    return v == v ? v : -INFINITY;  // a NaN is never preferred
}

__device__ __forceinline__ float sigmoid32(float l) {
    // both forms keep their relative error where s is small
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

__device__ __forceinline__ double sigmoid64(double l) {
    const double e = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// Which experts a lane holds: slot i is expert first + stride * i of its group.
struct Lanes {
    int first, stride, count;  // count slots; none for lanes without a group
    int group, P;
    __device__ __forceinline__ int expert(int i) const { return first + stride * i; }
};

// The choice on 64-bit values: lane k returns the k-th chosen expert.  Kept
// out of line, its values in local memory: it runs for few tokens.
template <int VPL, bool BF16>
__device__ __noinline__ int choose64(const RouteGrouped& p, const void* row, const Lanes& L, float m, int lane) {
    double c[VPL];
    double z = 0.0;
    if (!p.sigmoid) {
        for (int i = 0; i < L.count; ++i) z += exp((double)load_logit<BF16>(row, L.expert(i)) - (double)m);
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
        if (!(z > 0.0)) z = 1.0;
    }
    double m1 = -INFINITY, m2 = -INFINITY;
    for (int i = 0; i < L.count; ++i) {
        const int e = L.expert(i);
        const double l = load_logit<BF16>(row, e);
        const double s = p.sigmoid ? sigmoid64(l) : exp(l - (double)m) / z;
        const double v = p.bias ? s + (double)__ldg(p.bias + e) : s;
        const double u = v == v ? v : -INFINITY;
        c[i] = p.bias ? u : l;
        const double a = p.bias || p.top == 2 ? u : l;  // what the groups are ranked by
        if (a > m1) {
            m2 = m1;
            m1 = a;
        } else if (a > m2) {
            m2 = a;
        }
    }
    bool kept = L.count > 0;
    if (p.groups > 1) {
        for (int o = 1; o < L.P; o <<= 1) {
            const double o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            m2 = fmax(fmin(m1, o1), fmax(m2, o2));
            m1 = fmax(m1, o1);
        }
        const double value = p.top == 2 ? m1 + m2 : m1;
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double other = __shfl_sync(kAll, value, g * L.P);
            before += other > value || (other == value && g < L.group);
        }
        kept = kept && before < p.chosen;
    }
    unsigned long long taken = 0;
    int mine = 0;
    for (int k = 0; k < p.K; ++k) {
        double best = -INFINITY;
        int at = 0x7FFFFFFF;
        if (kept)
            for (int i = 0; i < L.count; ++i)
                if (!((taken >> i) & 1ull) && (at == 0x7FFFFFFF || c[i] > best)) {
                    best = c[i];
                    at = L.expert(i);
                }
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(kAll, best, o);
            const int oa = __shfl_xor_sync(kAll, at, o);
            const bool other = oa != 0x7FFFFFFF && (at == 0x7FFFFFFF || ob > best || (ob == best && oa < at));
            best = other ? ob : best;
            at = other ? oa : at;
        }
        for (int i = 0; i < L.count; ++i)
            if (L.expert(i) == at) taken |= 1ull << i;
        if (lane == k) mine = at;
    }
    return mine;
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(256) route_grouped_kernel(const __grid_constant__ RouteGrouped p) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)t * p.ld * (BF16 ? 2 : 4);

    Lanes L;
    const int gs = p.E / p.groups;
    L.P = p.lanes;
    L.group = lane / L.P;
    L.stride = L.P;
    L.first = L.group * gs + lane % L.P;
    L.count = L.group < p.groups ? (gs - lane % L.P + L.P - 1) / L.P : 0;

    float l[VPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        l[i] = i < L.count ? load_logit<BF16>(row, L.expert(i)) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
    float z = 1.0f;
    // the scores are needed for the choice (otherwise only those of the chosen are)
    const bool scored = p.bias != nullptr || (p.groups > 1 && p.top == 2);
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) m = 0.0f;  // no finite logit: every p is 0
        if (scored || !p.renorm) {
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < L.count) z += expf(l[i] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
            if (!(z > 0.0f)) z = 1.0f;
        }
    }
    // The error of s in fp32: sigmoid: expf 1 ulp, sum and quotient half an ulp
    // each, so 2^-22 of s <= 1.  softmax: l - m rounds to 2^-24 |l - m| <= 2^-24 e^-1 z / p
    // of the largest p = 1 / z, expf and quotient as before, and z's sum of VPL
    // terms a lane and 5 levels errs by 2^-24 (VPL + 5) of itself.  Adding b rounds c to 2^-24 |c|.
    const float kErr = p.sigmoid ? 0x1p-22f : (VPL + 16) * 0x1p-24f / z;

    uint32_t key[VPL];
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float s = l[i], c = l[i];
        if (scored) {
            s = p.sigmoid ? sigmoid32(l[i]) : expf(l[i] - m) / z;
            if (p.bias) {
                s += i < L.count ? __ldg(p.bias + L.expert(i)) : 0.0f;
                if (!(s == s)) s = -INFINITY;
                c = s;
            }
        }
        key[i] = i < L.count ? order_key(c) : 0u;
        if (i < L.count) {
            m2 = fmaxf(fminf(m1, s), m2);
            m1 = fmaxf(m1, s);
        }
    }
    bool unsure = false;
    if (p.groups > 1) {
        for (int o = 1; o < L.P; o <<= 1) {
            const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        const float value = p.top == 2 ? m1 + m2 : m1;
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl_sync(kAll, value, g * L.P);
            before += other > value || (other == value && g < L.group);
        }
        const bool kept = before < p.chosen;
        if (scored) {
            // the last group that stays against the first that does not
            float lo = kept && L.count > 0 ? value : INFINITY, hi = !kept && L.count > 0 ? value : -INFINITY;
            float mag = L.count > 0 ? fabsf(m1) + (p.top == 2 ? fabsf(m2) : 0.0f) : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
                mag = fmaxf(mag, __shfl_xor_sync(kAll, mag, o));
            }
            // two values of two scores each; the sums' own roundings are relative to what is added
            unsure = !(lo - hi > 4.0f * kErr + 0x1p-22f * mag);
        }
        if (!kept) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = 0u;
        }
    }

    // K rounds: the largest key of the warp, then the lowest expert that holds it;
    // with a bias one round more, to see how near the next one is
    int my_id = 0, next_id = 0;
    uint32_t my_key = 0u, next = 0u;
    const int rounds = p.bias ? p.K + 1 : p.K;
    for (int k = 0; k < rounds; ++k) {
        uint32_t lm = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) lm = max(lm, key[i]);
        const uint32_t best = __reduce_max_sync(kAll, lm);
        uint32_t le = 0xFFFFFFFFu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            if (best != 0u && key[i] == best) le = (uint32_t)L.expert(i);
        const uint32_t e = __reduce_min_sync(kAll, le);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((uint32_t)L.expert(i) == e) key[i] = 0u;
        if (lane == k) {
            my_id = (int)e;
            my_key = best;
        }
        if (lane == k - 1) {
            next_id = (int)e;
            next = best;
        }
    }
    if (p.bias && lane < p.K && next != 0u) {
        const float a = key_to_float(my_key), b = key_to_float(next);
        // the difference of two infinities is NaN, which compares as near
        if (!(a - b > 2.0f * kErr + 0x1p-23f * (fabsf(a) + fabsf(b))))
            // the same logit and the same bias are equal, and in order already
            unsure = unsure || load_logit<BF16>(row, my_id) != load_logit<BF16>(row, next_id) ||
                     __ldg(p.bias + my_id) != __ldg(p.bias + next_id);
    }
    if (__any_sync(kAll, unsure)) my_id = choose64<VPL, BF16>(p, row, L, m, lane);

    const int Kt = p.K + p.shared;
    const bool mine = lane < p.K;
    const float lw = mine ? load_logit<BF16>(row, my_id) : -INFINITY;
    float w;
    if (p.renorm) {
        // the scores times a common factor that keeps their largest near 1: e^-top for
        // softmax, and for sigmoid where every chosen logit is negative
        float top = lw;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (p.sigmoid) top = fminf(top, 0.0f);
        if (top == -INFINITY) top = 0.0f;
        w = mine ? expf((p.sigmoid ? fminf(lw, 0.0f) : lw) - top) : 0.0f;
        if (p.sigmoid) w /= 1.0f + expf(-fabsf(lw));
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        w = sum > 0.0f ? w / sum : 0.0f;
    } else {
        w = p.sigmoid ? sigmoid32(lw) : expf(lw - m) / z;
    }
    if (mine) {
        p.ids[(size_t)t * Kt + lane] = my_id;
        p.w[(size_t)t * Kt + lane] = w * p.scale;
    }
    if (p.shared && lane == 0) {
        p.ids[(size_t)t * Kt + p.K] = p.E;
        p.w[(size_t)t * Kt + p.K] = p.shared_w ? __ldg(p.shared_w + t) : 1.0f;
    }
    pdl_end();
}

template <int VPL>
cudaError_t launch(const RouteGrouped& p, cudaStream_t s) {
    const int warps = 8;
    const dim3 grid((p.T + warps - 1) / warps);
    return p.bf16 ? launch_pdl(route_grouped_kernel<VPL, true>, grid, dim3(warps * 32), 0, s, p)
                  : launch_pdl(route_grouped_kernel<VPL, false>, grid, dim3(warps * 32), 0, s, p);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGrouped& given, cudaStream_t s) {
    RouteGrouped p = given;
    if (p.chosen == p.groups) p.groups = p.chosen = 1;  // every group stays
    p.lanes = 32;
    while (p.lanes > 1 && p.lanes * p.groups > 32) p.lanes /= 2;
    const int per_lane = (p.E / p.groups + p.lanes - 1) / p.lanes;
    if (per_lane <= 2) return launch<2>(p, s);
    if (per_lane <= 4) return launch<4>(p, s);
    if (per_lane <= 8) return launch<8>(p, s);
    if (per_lane <= 16) return launch<16>(p, s);
    if (per_lane <= 32) return launch<32>(p, s);
    return launch<64>(p, s);
}

}  // namespace moe
