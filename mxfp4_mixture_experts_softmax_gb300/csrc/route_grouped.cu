// route_grouped.cu -- routing with softmax or sigmoid scores, a bias for
// balance and expert groups, one warp per token.
//
//   s = softmax(l) or 1 / (1 + e^-l);   c = s + b   (without b: c = l)
//   value of a group = its largest c, or the sum of its two largest
//   the `chosen` groups of the largest values stay; of their experts the K
//   largest c, in descending order;   w = scale * s [/ sum of the chosen s]
// Equal values go to the lower index everywhere.
//
// The choice has to be that of the exact values.  It is made on fp32 values with a
// known error (kErr below); where two of them lie closer than that allows and it
// matters, the few experts concerned are compared in 64 bits (settle), which about
// one token in a hundred needs, or in rarer cases all of them (choose64).
//
// A group's experts lie in one lane or in neighbouring ones, P = (lanes of a token) /
// (groups rounded up to a power of two), so that group values are reductions over P
// lanes.  A lane sorts its values once, as 32-bit keys whose lowest bits name the slot, so
// that each of the K rounds is one maximum over the lanes' heads and one shift in the
// winning lane.  Two kernels: a warp a token, for any sizes; and for long batches of few
// experts 8 or 16 lanes a token, which share the instructions of the rounds and weights
// between 4 or 2 tokens and hand a token with a near-tie to the first one's code.
#include <algorithm>

#include "moe_internal.h"
#include "route_device.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.44269504f;
// From so many tokens on several share a warp.  In us, a warp a token against several: 64 experts, top-6, 2048 tokens 2.8 and
// 2.5, 4096 3.9 and 2.8, 32768 21 and 9.5; 256 in groups with a bias, top-8, 4096 8.3 and 11.8, 16384 20.5 and 19.9, 32768
// 37 and 28, 131072 133 and 76; 512 with a bias, top-10, 4096 14.0 and 15.9, 8192 20.7 and 19.5, 32768 60 and 40.
constexpr int kManyTokens = 4096, kManyWarps = 4;

__device__ __forceinline__ float not_nan(float v) { return v == v ? v : -INFINITY; }  // a NaN is never preferred

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
    return not_nan(BF16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(row) + e) << 16)
                        : __ldg(static_cast<const float*>(row) + e));
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Which experts a lane holds.  V neighbouring ones at a time: slot i is expert
// first + (i / V) * V * P + i % V, for i < count.
template <int V>
struct Lanes {
    int first, P, group, count;
    __device__ __forceinline__ int expert(int i) const { return first + (i / V) * V * P + i % V; }
};

struct Token {
    const void* row;
    float m;  // the largest logit (softmax)
};

// The 64-bit score of a logit, z the sum that softmax divides by.
__device__ __forceinline__ double score64(const RouteGrouped& p, double l, double m, double z) {
    if (!p.sigmoid) return exp(l - m) / z;
    const double e = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

template <int V, bool BF16>
__device__ __forceinline__ double sum64(const RouteGrouped& p, const Token& t, const Lanes<V>& L) {
    if (p.sigmoid) return 1.0;
    double z = 0.0;
#pragma unroll 4
    for (int i = 0; i < L.count; ++i) z += exp((double)load_logit<BF16>(t.row, L.expert(i)) - (double)t.m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    return z > 0.0 ? z : 1.0;
}

// The choice on 64-bit values of all experts: lane k returns the k-th chosen one.
// Out of line and its values in local memory: it runs for very few tokens.
template <int VPL, int V, bool BF16>
__device__ __noinline__ int choose64(const RouteGrouped& p, const Token& t, const Lanes<V>& L, int lane) {
    double c[VPL];
    const double z = sum64<V, BF16>(p, t, L);
    double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < L.count; ++i) {
        const int e = L.expert(i);
        const double l = load_logit<BF16>(t.row, e);
        double a = l;  // what the groups are ranked by
        if (p.bias || p.top == 2) a = score64(p, l, t.m, z);
        if (p.bias) a += (double)__ldg(p.bias + e);
        a = a == a ? a : -INFINITY;
        c[i] = p.bias ? a : l;
        m2 = fmax(fmin(m1, a), m2);
        m1 = fmax(m1, a);
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

// The order of the n candidates that lanes 0 .. n - 1 hold, by their exact values: lane k
// returns the k-th.  Without a bias the logits themselves are the values.  Softmax's
// denominator in fp32, whose inverse is good to z_err (which grows with the slots of a lane: see
// route_one), does for two experts unless it matters for their difference; then it is
// summed in 64 bits.
template <int V, bool BF16>
__device__ __noinline__ int settle(const RouteGrouped& p, const Token& t, const Lanes<V>& L, int id, int n, float inv_z, float z_err,
                                   int lane) {
    const bool in = lane < n;
    const double l = in ? (double)load_logit<BF16>(t.row, id) : -INFINITY;
    const double b = p.bias && in ? (double)__ldg(p.bias + id) : 0.0;
    double e = l, c = l;
    bool rough = false;
    if (p.bias) {
        e = score64(p, l, t.m, 1.0);
        rough = !p.sigmoid;
        c = p.sigmoid ? e + b : e * (double)inv_z + b;
        c = c == c ? c : -INFINITY;
    }
    for (int pass = 0; pass < 2; ++pass) {
        // Nearly in order: neighbours change places until none has to.  Any n values are in order after n phases
        // and two more see it, which bounds the loop whatever the values are.
        bool unclear = false;
        for (int phase = 0, still = 0; still < 2 && phase < 34; ++phase) {
            const int other = ((lane + phase) & 1) ? lane - 1 : lane + 1;
            const bool pair = in && other >= 0 && other < n;
            const double oc = __shfl_sync(kAll, c, other & 31), oe = __shfl_sync(kAll, e, other & 31);
            const int oid = __shfl_sync(kAll, id, other & 31);
            const bool above = oc > c || (oc == c && oid < id);  // the other belongs above this one
            if (rough) {
                const double tol = fabs(oe - e) * (double)z_err;
                unclear = unclear || (pair && tol > 0.0 && !(fabs(oc - c) > tol));
            }
            const bool move = pair && above == (other > lane);
            c = move ? oc : c;
            e = move ? oe : e;
            id = move ? oid : id;
            still = __any_sync(kAll, move) ? 0 : still + 1;
        }
        if (!__any_sync(kAll, unclear)) break;  // (never in the second pass)
        const double z = sum64<V, BF16>(p, t, L);
        c = in ? e / z + (double)__ldg(p.bias + id) : -INFINITY;
        c = c == c ? c : -INFINITY;
        rough = false;
    }
    return id;
}

// Whether a group stays, by exact values.  u1 and u2 are what this lane contributes: the
// largest two of its values.
__device__ __forceinline__ bool settle_ranks(const RouteGrouped& p, double u1, double u2, int P, int group) {
    for (int o = 1; o < P; o <<= 1) {
        const double o1 = __shfl_xor_sync(kAll, u1, o), o2 = __shfl_xor_sync(kAll, u2, o);
        u2 = fmax(fmin(u1, o1), fmax(u2, o2));
        u1 = fmax(u1, o1);
    }
    const double value = p.top == 2 ? u1 + u2 : u1;
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const double other = __shfl_sync(kAll, value, g * P);
        before += other > value || (other == value && g < group);
    }
    return before < p.chosen;
}

// Without a bias: the two largest logits m1 and m2 of a lane have the largest scores.
__device__ __noinline__ bool settle_groups(const RouteGrouped& p, float m, float m1, float m2, int P, int group) {
    return settle_ranks(p, score64(p, m1, m, 1.0), score64(p, m2, m, 1.0), P, group);
}

// With one: the two experts e1 and e2 (-1: none) that may be a lane's part of its group's largest two.
template <int V, bool BF16>
__device__ __noinline__ bool settle_biased(const RouteGrouped& p, const Token& t, const Lanes<V>& L, int e1, int e2) {
    const double z = sum64<V, BF16>(p, t, L);
    const double l1 = e1 >= 0 ? (double)load_logit<BF16>(t.row, e1) : -INFINITY;
    const double l2 = e2 >= 0 ? (double)load_logit<BF16>(t.row, e2) : -INFINITY;
    double u1 = score64(p, l1, t.m, z), u2 = score64(p, l2, t.m, z);
    u1 = e1 >= 0 ? u1 + (double)__ldg(p.bias + e1) : -INFINITY;
    u2 = e2 >= 0 ? u2 + (double)__ldg(p.bias + e2) : -INFINITY;
    return settle_ranks(p, fmax(u1, u2), fmin(u1, u2), L.P, L.group);
}

// Descending order of N keys (odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* key) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + k];
                        key[i + j] = max(a, b);
                        key[i + j + k] = min(a, b);
                    }
}

// c of a logit: what the choice goes by.
__device__ __forceinline__ float value32(const RouteGrouped& p, float l, float b, float m, float inv_z) {
    return p.sigmoid ? b + rcp(1.0f + ex2(-kLog2e * l)) : ex2((l - m) * kLog2e) * inv_z + b;
}

// A key that orders like the value, its lowest bits replaced.  (A sum that is NaN has the canonical
// positive pattern, so no key of an expert is 0.)
__device__ __forceinline__ uint32_t packed_key(float v, uint32_t low_bits, uint32_t low) {
    const uint32_t u = __float_as_uint(v);
    return ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & ~low_bits) | low;
}

// The value of such a key up to its lowest bits.  Keys below that of the lowest finite value are -inf's, which
// would be a NaN without its lowest bits, or empty.
__device__ __forceinline__ float cut_value(uint32_t key, uint32_t low_bits) {
    const uint32_t k = key & ~low_bits;
    return k < 0x00800000u ? -INFINITY : key_to_float(k);
}

// V neighbouring logits from expert e on.
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const void* row, int e, float* l) {
    if constexpr (V == 4 && BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + e));
        l[0] = __uint_as_float(w.x << 16), l[1] = __uint_as_float(w.x & 0xFFFF0000u);
        l[2] = __uint_as_float(w.y << 16), l[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else if constexpr (V == 4) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + e));
        l[0] = w.x, l[1] = w.y, l[2] = w.z, l[3] = w.w;
    } else {
        l[0] = load_logit<BF16>(row, e);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = fmaxf(l[i], -INFINITY);  // NaN becomes -inf
}

// e^(a - b) to the exponential's own error: what the difference loses by its rounding (2^-24 of it, 60 parts of 2^24 of
// the result at a distance of 60) comes back as a factor.
__device__ __forceinline__ float exp_difference(float a, float b) {
    const float d = a - b, t = d - a, lost = (a - (d - t)) - (b + t), v = expf(d);
    return fabsf(d) < INFINITY ? fmaf(v, lost, v) : v;
}

// Weights of the chosen experts and the stores, S lanes a token, lane k of them with the k-th
// expert (id, logit lw).  sum_all: softmax's denominator, where it is needed.
template <int S>
__device__ __forceinline__ void finish(const RouteGrouped& p, int t, int k, int id, float lw, float m, float sum_all) {
    const bool mine = k < p.K;
    float w;
    if (!mine) lw = -INFINITY;
    if (p.renorm) {
        // the scores times a common factor that keeps their largest near 1: e^-top for
        // softmax, and for sigmoid where every chosen logit is negative
        float top = lw;
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (p.sigmoid) top = fminf(top, 0.0f);
        if (top == -INFINITY) top = 0.0f;
        w = mine ? exp_difference(p.sigmoid ? fminf(lw, 0.0f) : lw, top) : 0.0f;
        if (p.sigmoid) w /= 1.0f + expf(-fabsf(lw));
        float sum = w;
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        w = sum > 0.0f ? w / sum : 0.0f;
    } else if (p.sigmoid) {
        const float e = expf(-fabsf(lw));
        w = (lw >= 0.0f ? 1.0f : e) / (1.0f + e);
    } else {
        w = sum_all > 0.0f ? exp_difference(lw, m) / sum_all : 0.0f;
    }
    const int Kt = p.K + p.shared;
    const size_t at = (size_t)t * Kt + k;
    if (mine && t < p.T) {
        p.ids[at] = id;
        p.w[at] = w * p.scale;
    }
    if (p.shared && k == S - 1 && t < p.T) {
        p.ids[at - k + p.K] = p.E;
        p.w[at - k + p.K] = p.shared_w ? __ldg(p.shared_w + t) : 1.0f;
    }
}

// One token, one warp.
template <int VPL, int V, bool BF16>
__device__ __forceinline__ void route_one(const RouteGrouped& p, int t, int lane) {
    // what the lowest bits of a key hold: its slot, the first one largest
    constexpr uint32_t kSlots = VPL - 1;
    Lanes<V> L;
    const int gs = p.group_size;
    L.P = 1 << p.lanes_log2;
    L.group = lane >> p.lanes_log2;
    const int piece = V * (lane & (L.P - 1));  // of V experts; the next one is V * P further
    L.first = L.group * gs + piece;
    L.count = L.group < p.groups && piece < gs ? ((gs - piece + V * L.P - 1) >> p.lanes_log2) / V * V : 0;
    const bool biased = p.bias != nullptr;
    Token tk;
    tk.row = static_cast<const uint8_t*>(p.logits) + (size_t)t * p.ld * (BF16 ? 2 : 4);
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i += V) {
        if (i < L.count) {
            load_logits<V, BF16>(tk.row, L.expert(i), c + i);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) c[i + k] = -INFINITY;
        }
    }
    float m = 0.0f, sum_all = 0.0f;
    if (!p.sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = fmaxf(m, c[i]);
        m = key_to_float(__reduce_max_sync(kAll, order_key(m)));
        if (m == -INFINITY) m = 0.0f;  // no finite logit: every p is 0
        if (!p.renorm) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum_all += expf(c[i] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum_all += __shfl_xor_sync(kAll, sum_all, o);
        }
    }
    tk.m = m;
    // c, and the error it has.  ex2.approx errs by 2^-22, its argument by the rounding of
    // (l - m) log2 e; rcp.approx by 2^-23.  sigmoid: a quarter of 2^-22 (its slope over e is at most
    // 1/4 of e), 2^-23 and a rounding of a value up to 1: 2^-22.  softmax: e / z with e = e^-d and an argument good to 2^-23 d, d e^-d <= 0.37; z, a sum
    // of VPL terms a lane and 5 levels, to (VPL + 9) 2^-24 of itself; all relative to the largest p, 1 / z.
    // Adding b rounds to 2^-24 |c| (the compares below allow for that).
    float inv_z = 1.0f, kErr = 0.0f;
    if (biased) {
        if (p.sigmoid) {
            kErr = 0x1p-22f;
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) z += ex2((c[i] - m) * kLog2e);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
            inv_z = z > 0.0f ? rcp(z) : 1.0f;
            kErr = (VPL + 24) * 0x1p-24f * inv_z;
        }
#pragma unroll
        for (int i = 0; i < VPL; i += V)
            if (i < L.count) {
                float b[4];
                if constexpr (V == 4) {
                    const float4 w = __ldg(reinterpret_cast<const float4*>(p.bias + L.expert(i)));
                    b[0] = w.x, b[1] = w.y, b[2] = w.z, b[3] = w.w;
                } else {
                    b[0] = __ldg(p.bias + L.expert(i));
                }
#pragma unroll
                for (int j = 0; j < V; ++j) c[i + j] = value32(p, c[i + j], b[j], m, inv_z);
            }
    }

    bool unsure = false, kept = true;
    if (p.groups > 1) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i < L.count) {
                m2 = fmaxf(fminf(m1, c[i]), m2);
                m1 = fmaxf(m1, c[i]);
            }
        const float own1 = m1, own2 = m2;
        for (int o = 1; o < L.P; o <<= 1) {
            const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        float value = m1, err = 0.0f;
        if (p.top == 2) {
            float s1 = m1, s2 = m2;
            if (!biased) {  // (a factor of 1 / z changes no order)
                s1 = value32(p, m1, 0.0f, m, 1.0f);
                s2 = value32(p, m2, 0.0f, m, 1.0f);
            }
            value = s1 + s2;
            err = biased ? 4.0f * kErr + 0x1p-22f * (fabsf(s1) + fabsf(s2)) : 0x1p-19f;
        } else if (biased) {
            err = 2.0f * kErr + 0x1p-22f * fabsf(m1);
        }
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl_sync(kAll, value, g << p.lanes_log2);
            before += other > value || (other == value && g < L.group);
        }
        kept = before < p.chosen;
        if (biased || p.top == 2) {
            // the last group that stays against the first that does not
            const bool real = L.group < p.groups;
            const float lo = key_to_float(__reduce_min_sync(kAll, real && kept ? order_key(value) : 0xFF800000u));
            const float hi = key_to_float(__reduce_max_sync(kAll, real && !kept ? order_key(value) : 0x007FFFFFu));
            const float most = __uint_as_float(__reduce_max_sync(kAll, real ? __float_as_uint(err) : 0u));
            if (!(lo - hi > most)) {
                if (!biased) {
                    kept = settle_groups(p, m, own1, own2, L.P, L.group);
                } else {
                    // of each lane those that may be among the group's largest two
                    const float least = (p.top == 2 ? m2 : m1) - most;
                    int e1 = -1, e2 = -1;
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (i < L.count && !(c[i] < least)) {
                            unsure = unsure || e2 >= 0 || !(fabsf(c[i]) < INFINITY);
                            e2 = e1;
                            e1 = L.expert(i);
                        }
                    unsure = __any_sync(kAll, unsure) != 0;
                    if (!unsure) kept = settle_biased<V, BF16>(p, tk, L, e1, e2);
                }
            }
        }
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = i < L.count ? packed_key(c[i], kSlots, kSlots - i) : 0u;
    sort_keys<VPL>(key);
    if (!kept) key[0] = 0u;

    // K rounds: the largest head of the warp, the lowest lane that has it.  Then the others that
    // may be among the K: whose value, which the key gives up to its lowest bits, may reach the
    // K-th's.
    uint32_t my_key = 0u;
    int from = 0, n = 0;
    for (;; ++n) {
        const uint32_t best = __reduce_max_sync(kAll, key[0]);
        if (n >= p.K) {
            if (best == 0u) break;
            const float lo = key_to_float(__shfl_sync(kAll, my_key, p.K - 1) & ~kSlots), hi = key_to_float(best | kSlots);
            const float tol = biased ? 2.0f * kErr + 0x1p-22f * (fabsf(lo) + fabsf(hi)) : 0.0f;
            if (lo - hi > tol) break;
            if (n == 32) {
                unsure = true;
                break;
            }
        }
        const int src = __ffs((int)__ballot_sync(kAll, key[0] == best)) - 1;
        if (lane == src) {
#pragma unroll
            for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
            key[VPL - 1] = 0u;
        }
        if (lane == n) {
            my_key = best;
            from = src;
        }
    }
    const int slot = (int)(kSlots - (my_key & kSlots));
    const int first = __shfl_sync(kAll, L.first, from);
    int id = lane < n ? first + ((slot / V * V) << p.lanes_log2) + slot % V : 0;

    // the candidates' values in full: their order stands if each is surely above the next, or
    // equal to it in logit and bias and lower in number
    float lw = lane < n ? load_logit<BF16>(tk.row, id) : -INFINITY;
    const float bw = biased && lane < n ? __ldg(p.bias + id) : 0.0f;
    const float cw = biased ? value32(p, lw, bw, m, inv_z) : lw;
    const float cn = __shfl_down_sync(kAll, cw, 1), ln = __shfl_down_sync(kAll, lw, 1), bn = __shfl_down_sync(kAll, bw, 1);
    const int idn = __shfl_down_sync(kAll, id, 1);
    const float tol = biased ? 2.0f * kErr + 0x1p-23f * (fabsf(cw) + fabsf(cn)) : 0.0f;
    const bool sure = cw - cn > tol || (!biased && cw > cn) || (lw == ln && bw == bn && id < idn);
    unsure = __any_sync(kAll, unsure) != 0;
    if (unsure || __any_sync(kAll, lane + 1 < n && !sure)) {
        id = unsure ? choose64<VPL, V, BF16>(p, tk, L, lane) : settle<V, BF16>(p, tk, L, id, n, inv_z, kErr, lane);
        if (lane < p.K) lw = load_logit<BF16>(tk.row, id);
    }
    finish<32>(p, t, lane, id, lw, m, sum_all);
}

template <int VPL, int V, bool BF16>
__global__ void __launch_bounds__(256) route_grouped_kernel(const __grid_constant__ RouteGrouped p) {
    pdl_begin();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t < p.T) route_one<VPL, V, BF16>(p, t, threadIdx.x & 31);
    pdl_end();
}

template <int VPL, bool BF16>
__device__ __noinline__ void route_again(const RouteGrouped& p, int t, int lane) {
    route_one<VPL, 4, BF16>(p, t, lane);
}

// S lanes a token (32 / S tokens a warp), VPL slots a lane, of which the 8 largest are kept.
// Needs K <= S, groups <= S, experts of a group in fours.  Eight blocks an SM, which leaves 64 registers:
// 131072 tokens with groups and a bias in 77 us, with the compiler's own choice in 90 (32768: the same).  A warp loads its
// tokens, works and ends, so it waits for memory: 37% of the issue slots are used at 32768 tokens, the main stall is that on loads.
template <int S, int VPL, bool BF16>
__global__ void __launch_bounds__(kManyWarps * 32, 8) route_grouped_many_kernel(const __grid_constant__ RouteGrouped p) {
    constexpr uint32_t kSlots = VPL - 1;
    constexpr int kSLog2 = S == 8 ? 3 : 4, kList = 8;
    pdl_begin();
    const int lane = threadIdx.x & 31, k = lane & (S - 1);  // lane k of its token
    const int tokens = 32 / S;
    const int t0 = (blockIdx.x * kManyWarps + (threadIdx.x >> 5)) * tokens;
    if (t0 >= p.T) return;
    const int t = t0 + lane / S;
    const bool live = t < p.T;

    const int log2P = p.lanes_log2 - (5 - kSLog2);
    Lanes<4> L;
    const int gs = p.group_size;
    L.P = 1 << log2P;
    L.group = k >> log2P;
    const int piece = 4 * (k & (L.P - 1));
    L.first = L.group * gs + piece;
    L.count = L.group < p.groups && piece < gs ? ((gs - piece + 4 * L.P - 1) >> log2P) / 4 * 4 : 0;
    const bool biased = p.bias != nullptr;
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)min(t, p.T - 1) * p.ld * (BF16 ? 2 : 4);
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
        if (i < L.count) {
            load_logits<4, BF16>(row, L.expert(i), c + i);
        } else {
            c[i] = c[i + 1] = c[i + 2] = c[i + 3] = -INFINITY;
        }
    }
    float m = 0.0f, sum_all = 0.0f;
    if (!p.sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = fmaxf(m, c[i]);
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) m = 0.0f;
        if (!p.renorm) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum_all += expf(c[i] - m);
#pragma unroll
            for (int o = S / 2; o > 0; o >>= 1) sum_all += __shfl_xor_sync(kAll, sum_all, o);
        }
    }
    // errors as in route_one
    float inv_z = 1.0f, kErr = 0.0f;
    if (biased) {
        if (p.sigmoid) {
            kErr = 0x1p-22f;
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) z += ex2((c[i] - m) * kLog2e);
#pragma unroll
            for (int o = S / 2; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
            inv_z = z > 0.0f ? rcp(z) : 1.0f;
            kErr = (VPL + 24) * 0x1p-24f * inv_z;
        }
#pragma unroll
        for (int i = 0; i < VPL; i += 4)
            if (i < L.count) {
                const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + L.expert(i)));
                c[i] = value32(p, c[i], b.x, m, inv_z);
                c[i + 1] = value32(p, c[i + 1], b.y, m, inv_z);
                c[i + 2] = value32(p, c[i + 2], b.z, m, inv_z);
                c[i + 3] = value32(p, c[i + 3], b.w, m, inv_z);
            }
    }
    // the lane's largest eight, in order: eights sorted, then two lists into one
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = i < L.count ? packed_key(c[i], kSlots, kSlots - i) : 0u;
#pragma unroll
    for (int i = 0; i < VPL; i += kList) sort_keys<kList>(key + i);
#pragma unroll
    for (int w = kList; w < VPL; w *= 2)
#pragma unroll
        for (int i = 0; i < VPL; i += 2 * w) {
            // the larger of the first's j-th and the second's j-th from its end: the largest eight of both
#pragma unroll
            for (int j = 0; j < kList; ++j) key[i + j] = max(key[i + j], key[i + w + kList - 1 - j]);
#pragma unroll
            for (int d = kList / 2; d > 0; d /= 2)
#pragma unroll
                for (int j = 0; j < kList; ++j)
                    if (!(j & d)) {
                        const uint32_t x = key[i + j], y = key[i + j + d];
                        key[i + j] = max(x, y);
                        key[i + j + d] = min(x, y);
                    }
        }

    bool unsure = false;
    if (p.groups > 1) {
        // group values from the keys, which give a value up to its lowest bits: 2^-23 kSlots of it
        const bool real = L.group < p.groups;
        float m1 = cut_value(key[0], kSlots), m2 = cut_value(key[1], kSlots);
        for (int o = 1; o < L.P; o <<= 1) {
            const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        constexpr float kCut = 2.0f * VPL * 0x1p-23f;
        const auto size = [](float v) { return v == -INFINITY ? 0.0f : fabsf(v); };  // (nothing is cut off -inf)
        float value = m1, err = 2.0f * kErr + kCut * size(m1);
        if (p.top == 2) {
            float s1 = m1, s2 = m2;
            if (!biased) {
                s1 = value32(p, m1, 0.0f, m, 1.0f);
                s2 = value32(p, m2, 0.0f, m, 1.0f);
                // a score's slope is at most 1/4 (sigmoid) or itself
                err = 0x1p-19f + kCut * (size(m1) + size(m2) + 2.0f * fabsf(m));
            } else {
                err = 4.0f * kErr + kCut * (fabsf(s1) + fabsf(s2));
            }
            value = s1 + s2;
        }
        if (!(value == value)) err = INFINITY;  // compares with it say nothing: the token is routed again
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl_sync(kAll, value, (lane & ~(S - 1)) + (g << log2P));
            before += other > value || (other == value && g < L.group);
        }
        const bool kept = before < p.chosen;
        float lo = real && kept ? value : INFINITY, hi = real && !kept ? value : -INFINITY, most = real ? err : 0.0f;
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
            most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        }
        unsure = !(lo - hi > most);
        if (!kept) key[0] = 0u;
    }

    // a lane whose eight are used up may have more: its token is routed again
    const uint32_t beyond = L.count > kList ? 0xFFFFFFFFu : 0u;
    uint32_t my_key = 0u;
    int from = 0;
    for (int n = 0;; ++n) {
        uint32_t best = key[0];
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kAll, best, o));
        if (n == p.K) {
            const uint32_t last = __shfl_sync(kAll, my_key, (lane & ~(S - 1)) + n - 1);
            const float lo = key_to_float(last & ~kSlots), hi = key_to_float(best | kSlots);
            const float tol = biased ? 2.0f * kErr + 0x1p-22f * (fabsf(lo) + fabsf(hi)) : 0.0f;
            unsure = unsure || (best != 0u && !(lo - hi > tol));
            break;
        }
        unsure = unsure || best == 0xFFFFFFFFu;
        const uint32_t held = __ballot_sync(kAll, key[0] == best) >> (lane & ~(S - 1));
        const int src = __ffs((int)(held & ((1u << S) - 1))) - 1;
        if (k == src) {
#pragma unroll
            for (int i = 0; i + 1 < kList; ++i) key[i] = key[i + 1];
            key[kList - 1] = beyond;
        }
        if (k == n) {
            my_key = best;
            from = src;
        }
    }
    const int slot = (int)(kSlots - (my_key & kSlots));
    const int first = __shfl_sync(kAll, L.first, (lane & ~(S - 1)) + from);
    const int id = k < p.K ? min(first + ((slot / 4 * 4) << log2P) + slot % 4, p.E - 1) : 0;
    const float lw = k < p.K ? load_logit<BF16>(row, id) : -INFINITY;
    {
        const float bw = biased && k < p.K ? __ldg(p.bias + id) : 0.0f;
        const float cw = biased ? value32(p, lw, bw, m, inv_z) : lw;
        const float cn = __shfl_down_sync(kAll, cw, 1), ln = __shfl_down_sync(kAll, lw, 1), bn = __shfl_down_sync(kAll, bw, 1);
        const int idn = __shfl_down_sync(kAll, id, 1);
        const float tol = biased ? 2.0f * kErr + 0x1p-23f * (fabsf(cw) + fabsf(cn)) : 0.0f;
        const bool sure = cw - cn > tol || (!biased && cw > cn) || (lw == ln && bw == bn && id < idn);
        unsure = unsure || (k + 1 < p.K && !sure);
    }
    const uint32_t again = __ballot_sync(kAll, unsure && live);
    const bool mine_again = (again >> (lane & ~(S - 1))) & ((1u << S) - 1);
    finish<S>(p, mine_again ? p.T : t, k, id, lw, m, sum_all);
    for (int j = 0; j < tokens; ++j)
        if ((again >> (j * S)) & ((1u << S) - 1)) route_again<S * VPL / 32, BF16>(p, t0 + j, lane);
    pdl_end();
}

template <int S, int VPL>
cudaError_t launch_many(const RouteGrouped& p, cudaStream_t s) {
    const int tokens = kManyWarps * 32 / S;
    const dim3 grid((p.T + tokens - 1) / tokens);
    return p.bf16 ? launch_pdl(route_grouped_many_kernel<S, VPL, true>, grid, dim3(kManyWarps * 32), 0, s, p)
                  : launch_pdl(route_grouped_many_kernel<S, VPL, false>, grid, dim3(kManyWarps * 32), 0, s, p);
}

template <int VPL, int V>
cudaError_t launch(const RouteGrouped& p, cudaStream_t s) {
    const dim3 grid((p.T + 7) / 8);
    return p.bf16 ? launch_pdl(route_grouped_kernel<VPL, V, true>, grid, dim3(256), 0, s, p)
                  : launch_pdl(route_grouped_kernel<VPL, V, false>, grid, dim3(256), 0, s, p);
}

template <int V>
cudaError_t launch_slots(const RouteGrouped& p, int slots, cudaStream_t s) {
    if (slots <= 4) return launch<4, V>(p, s);
    if (slots <= 8) return launch<8, V>(p, s);
    if (slots <= 16) return launch<16, V>(p, s);
    if (slots <= 32) return launch<32, V>(p, s);
    return launch<64, V>(p, s);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGrouped& given, cudaStream_t s) {
    RouteGrouped p = given;
    if (p.chosen == p.groups) p.groups = p.chosen = 1;  // every group stays
    p.group_size = p.E / p.groups;
    p.lanes_log2 = 5;
    while (p.lanes_log2 > 0 && (p.groups << p.lanes_log2) > 32) --p.lanes_log2;
    // 16 bytes (8 of bf16) at a time where rows and groups allow it and no lane gets more slots for it
    const int P = 1 << p.lanes_log2, wide = (p.group_size + 4 * P - 1) / (4 * P) * 4, one = (p.group_size + P - 1) / P;
    const bool can = p.group_size % 4 == 0 && p.ld % 4 == 0 && (uintptr_t)p.logits % (p.bf16 ? 8 : 16) == 0 &&
                     (uintptr_t)p.bias % 16 == 0;
    if (can && p.T >= kManyTokens) {
        // lanes a token and slots a lane of the other kernel: the narrowest that holds K and the groups
        for (int S = 8; S <= 16; S *= 2) {
            const int log2P = p.lanes_log2 - (S == 8 ? 2 : 1);
            if (p.K > S || log2P < 0) continue;
            const int slots = (p.group_size + (4 << log2P) - 1) / (4 << log2P) * 4;
            if (slots > 32) continue;
            if (S == 8) return slots <= 16 ? launch_many<8, 16>(p, s) : launch_many<8, 32>(p, s);
            return slots <= 16 ? launch_many<16, 16>(p, s) : launch_many<16, 32>(p, s);
        }
    }
    return can && wide <= std::max(one, 4) ? launch_slots<4>(p, wide, s) : launch_slots<1>(p, one, s);
}

}  // namespace moe
