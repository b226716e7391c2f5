// Route (gfx950): a token's experts and weights from its router logits, and the logits'
// gradient from the weights'.
//
// The choice.  A wave takes a token.  With LG = 64 / groups lanes (a power of two) to a group,
// lane l holds experts gs (l / LG) + LG j + l % LG of groups of gs experts: a group's highest
// keys meet in LG lanes.  A lane sorts its keys once; every round of the choice is then one maximum
// over the wave's first ones (DPP) and a shift in the lane that had it.  Keys are 32-bit integers
// that order as floats, whose low bits name j:
//   without bias and groups, the logits (16-bit ones exactly, ties too);
//   else fp32 scores (hardware exp2 and reciprocal) plus bias.  Each is within
//     2^-24 (C smax + |key|) of the exact key, with C = 6, smax = 1 for a sigmoid (argument,
//     exp2, sum, reciprocal; s (1 - s) |l| < 0.23) and C = 40, smax = the highest score for a
//     softmax of at most 1024 terms; and the low bits take up to 2^(BITS - 23) of it.
// Neighbours among the chosen, and the k-th and the rest, that lie nearer than both bounds are put
// in order in fp64, whose order is the definition's: of 16384 tokens over 320 experts, 2 have
// their groups and 21 their experts decided so (a whole choice in fp64 in their place made a call
// of 1024 tokens take 12 us instead of 6.6).
// Weights are fp64 of the chosen logits alone, rounded once, for four tokens at a time.
//
// Bound by issue: 445 vector instructions a token.  T=16384 over 320 experts in 8 groups: 18.4 us (51
// with fp64 keys and a maximum over all of them each round; 21.1 with every logit made sane and the
// search for near ones in the rounds up to k); T=64, no groups: 4.1 us, most of it the chain of one
// token.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "block.h"
#include "eights.h"

namespace moe {

// A logit as the definition takes it: NaN counts as -Inf, +Inf as the largest finite.
__device__ __forceinline__ float sane(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t el) {
    return sane(to_f32<DT>(static_cast<const typename Elem<DT>::type*>(p)[el]));
}

// ---------------------------------------------------------------------------
// Reductions over the wave through DPP (rows of 16 by shifts, then rows into rows); the result
// is the same in every lane.
// ---------------------------------------------------------------------------
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t none) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false);
}
// v combined with the lane that CTRL names, or with the neutral element.
template <int CTRL, int ROWS, typename F>
__device__ __forceinline__ uint32_t dpp_step(uint32_t v, uint32_t none, F f) { return f(v, dpp<CTRL, ROWS>(v, none)); }
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, F f) {
    v = dpp_step<0x111, 0xF>(v, none, f);                         // row_shr 1, 2, 4, 8
    v = dpp_step<0x112, 0xF>(v, none, f);
    v = dpp_step<0x114, 0xF>(v, none, f);
    v = dpp_step<0x118, 0xF>(v, none, f);
    v = dpp_step<0x142, 0xA>(v, none, f);                         // row_bcast 15 into rows 1, 3
    v = dpp_step<0x143, 0xC>(v, none, f);                         // row_bcast 31 into rows 2, 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
// Over the lanes of a group of LG (a power of two): lanes trade places within quads, then halves
// of eight and rows of sixteen mirror each other, whose lanes agree by then.
template <typename F>
__device__ __forceinline__ void group_steps(int LG, F f) {
    if (LG > 1) f([](uint32_t v) { return dpp<0xB1, 0xF>(v, v); });
    if (LG > 2) f([](uint32_t v) { return dpp<0x4E, 0xF>(v, v); });
    if (LG > 4) f([](uint32_t v) { return dpp<0x141, 0xF>(v, v); });
    if (LG > 8) f([](uint32_t v) { return dpp<0x140, 0xF>(v, v); });
    if (LG > 16) f([](uint32_t v) { return (uint32_t)__shfl_xor((int)v, 16, 64); });
    if (LG > 32) f([](uint32_t v) { return (uint32_t)__shfl_xor((int)v, 32, 64); });
}
__device__ __forceinline__ float wave_total(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = (uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32), 0u) << 32 | dpp<CTRL, ROWS>((uint32_t)u, 0u);
    return v + __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double wave_total(double v) {
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    v = dpp_add<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Integers that order as the floats do, -0 below +0; those below kKeys stand for no key (-Inf).
constexpr uint32_t kKeys = 0x00800000u;
__device__ __forceinline__ uint32_t order_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) {
    return __uint_as_float(u ^ ((uint32_t)~((int32_t)u >> 31) | 0x80000000u));
}
__device__ __forceinline__ float wave_top(float v) { return order_value(wave_max_u32(order_bits(v))); }

constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

enum RouteKind { kByLogit, kBySigmoid, kBySoftmax };              // what keys are made of

// A lane's experts: ids first + j * step, of group `group` (idle lanes: bias -Inf).
struct RouteLane {
    int shift, gs, group, first, step;                           // lanes to a group: 1 << shift
};

// ---------------------------------------------------------------------------
// In fp64, by the definition, where 32 bits leave the order open.
// ---------------------------------------------------------------------------
struct Softmax64 {
    float top;
    double sum;
};
template <int KIND, int VPL>
__device__ __forceinline__ Softmax64 softmax64(const float (&l)[VPL]) {
    Softmax64 z{-INFINITY, 1.0};
    if (KIND == kBySoftmax) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) z.top = fmaxf(z.top, l[j]);
        z.top = wave_top(z.top);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (l[j] > -INFINITY) sum += exp((double)l[j] - (double)z.top);
        z.sum = wave_total(sum);
    }
    return z;
}
template <int KIND>
__device__ __forceinline__ double key64(float l, float bias, const Softmax64& z) {
    if (!(l > -INFINITY)) return -INFINITY;
    if (KIND == kByLogit) return (double)l;
    return (KIND == kBySigmoid ? sigmoid64(l) : exp((double)l - (double)z.top) / z.sum) + (double)bias;
}

// Whether the lane's group is among the best.
template <int KIND, int VPL>
__device__ __forceinline__ bool group64(const RouteArgs& a, const double (&key)[VPL], const RouteLane& o) {
    const int LG = 1 << o.shift;
    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        b2 = fmax(b2, fmin(b1, key[j]));
        b1 = fmax(b1, key[j]);
    }
    for (int i = 1; i < LG; i <<= 1) {
        const double c1 = __shfl_xor(b1, i, 64), c2 = __shfl_xor(b2, i, 64);
        b2 = fmax(fmin(b1, c1), fmax(b2, c2));
        b1 = fmax(b1, c1);
    }
    if (a.group_keys == 2 && b2 > -INFINITY) b1 += b2;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
        const double other = __shfl(b1, g * LG, 64);
        ahead += other > b1 || (other == b1 && g < o.group) ? 1 : 0;
    }
    return ahead < a.top_groups;
}

// The choice among the experts of the lanes that are `in`: the q-th expert's id to lane slot + q
// (-1 stays).
template <int KIND, int VPL>
__device__ __forceinline__ void choose64(const RouteArgs& a, const float (&l)[VPL], const float (&bias)[VPL],
                                         const RouteLane& o, bool in, int slot, int& id) {
    const int lane = threadIdx.x & 63;
    const Softmax64 z = softmax64<KIND>(l);
    double key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = in ? key64<KIND>(l[j], bias[j], z) : -INFINITY;
    for (int q = 0; q < a.k; ++q) {
        double best = -INFINITY;
        int at = INT_MAX;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = o.first + j * o.step;
            }
#pragma unroll
        for (int i = 32; i > 0; i >>= 1) {
            const double b = __shfl_xor(best, i, 64);
            const int e = __shfl_xor(at, i, 64);
            if (b > best || (b == best && e < at)) {
                best = b;
                at = e;
            }
        }
        if (!(best > -INFINITY)) break;
        if (lane == slot + q) id = at;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (o.first + j * o.step == at) key[j] = -INFINITY;
    }
}

// The choice from the lane's logits l (by a sigmoid: as they lie in memory; else sane ones, -Inf in
// idle places): the q-th expert's id to lane slot + q (-1 stays).  32-bit keys, whose low BITS bits
// name j, lower ones first, give the candidates: the k highest and those that lie too near the
// k-th to be told from it.  Where two neighbours among them are too near, all candidates are put
// in order in fp64, a lane each.  EXACT (16-bit logits, which leave the low bits 0): every key as it
// is, so nothing is left open; equal ones go by j, then by lane, which is by id where all lanes
// are one group.
template <int DT, int KIND, int VPL>
__device__ __forceinline__ void choose(const RouteArgs& a, const typename Elem<DT>::type* row, const float (&l)[VPL],
                                       const float (&bias)[VPL], const RouteLane& o, int slot, int& id) {
    constexpr bool EXACT = KIND == kByLogit && DT != kF32;
    constexpr float U = 1.0f / (1 << 24);
    constexpr int BITS = VPL <= 1 ? 0 : (VPL <= 2 ? 1 : (VPL <= 8 ? 3 : 5)), MASK = (1 << BITS) - 1;
    constexpr float R = (2 * (1 << BITS) + 1.02f) * U;           // relative: the low bits, the bias's addition
    const int lane = threadIdx.x & 63, LG = 1 << o.shift;
    bool in = true;                                              // the lane's group may be chosen from
    float key[VPL], base = 0.f;                                  // base: C smax 2^-24
    if constexpr (KIND == kByLogit) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = l[j] + 0.0f;      // -0 is +0
    } else {
        float smax = 1.0f;
        if (KIND == kBySoftmax) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) top = fmaxf(top, l[j]);
            top = wave_top(top);
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                key[j] = l[j] > -INFINITY ? fast_exp(l[j] - top) : 0.f;
                sum += key[j];
            }
            smax = __builtin_amdgcn_rcpf(wave_total(sum));
        }
        base = (KIND == kBySigmoid ? 6.0f : 40.0f) * U * smax;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            key[j] = (KIND == kBySigmoid ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[j])) : key[j] * smax) + bias[j];
            if (!(l[j] > -INFINITY)) key[j] = -INFINITY;
        }
    }
    uint32_t u[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) u[j] = (order_bits(key[j]) & ~(uint32_t)MASK) | (uint32_t)(VPL - 1 - j);
    // a lane's keys, highest first: a group's two highest and every round's candidate are then at hand
    // (many keys a lane: the maximum of all each time)
    constexpr bool SORTED = VPL <= 8;
    if constexpr (SORTED) {
#pragma unroll
        for (int pass = 0; pass < VPL; ++pass)
#pragma unroll
            for (int j = pass & 1; j + 1 < VPL; j += 2) {
                const uint32_t x = u[j], y = u[j + 1];
                u[j] = x > y ? x : y;
                u[j + 1] = x > y ? y : x;
            }
    }
    if (KIND != kByLogit && a.top_groups < a.groups) {
        uint32_t u1 = u[0], u2 = SORTED ? u[1] : 0u;
        if (!SORTED) {
#pragma unroll
            for (int j = 1; j < VPL; ++j) {
                const uint32_t low = u1 < u[j] ? u1 : u[j];
                u2 = u2 > low ? u2 : low;
                u1 = u1 > u[j] ? u1 : u[j];
            }
        }
        group_steps(LG, [&](auto swap) {
            const uint32_t c1 = swap(u1), c2 = swap(u2), low = u1 < c1 ? u1 : c1, high = u2 > c2 ? u2 : c2;
            u2 = low > high ? low : high;
            u1 = u1 > c1 ? u1 : c1;
        });
        const bool any = u1 >= kKeys, two = a.group_keys == 2 && u2 >= kKeys;
        const float b1 = order_value(u1), b2 = two ? order_value(u2) : 0.f, own = b1 + b2;
        // what the sum may be off by; groups without keys come last
        const float off = (two ? 2.f : 1.f) * base + (fabsf(b1) + fabsf(b2)) * (R + 1.01f * U) + 1e-36f;
        const uint32_t sum = any ? order_bits(own) : 0u;
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g)
            ahead += (uint32_t)__builtin_amdgcn_readlane((int)sum, g << o.shift) > sum ? 1 : 0;
        const bool live = o.group < a.groups;
        in = ahead < a.top_groups;
        const uint32_t last_in = ~wave_max_u32(in && live ? ~(any ? order_bits(own - off) : 0u) : 0u);
        const uint32_t first_out = wave_max_u32(in || !live ? 0u : (any ? order_bits(own + off) : 1u));
        // (equal sums may let too many in; a key of +Inf or a sum past fp32 has no bound)
        if (!(last_in > first_out) ||
            __popcll(__builtin_amdgcn_ballot_w64(in && live)) != a.top_groups << o.shift ||
            __builtin_amdgcn_ballot_w64(any && !(fabsf(own) + off <= FLT_MAX))) {
            const Softmax64 z = softmax64<KIND>(l);
            double key[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = key64<KIND>(l[j], bias[j], z);
            in = group64<KIND>(a, key, o);
        }
        if (!in) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) u[j] = 0;
        }
    }
    uint32_t got = 0, from = 0;                                  // lane q: the q-th key and its lane
    int n = 0;
    uint32_t m, best;                                            // the lane's and the wave's highest key
    auto highest = [&]() {
        m = u[0];
        if (!SORTED) {
#pragma unroll
            for (int j = 1; j < VPL; ++j) m = m > u[j] ? m : u[j];
        }
        best = wave_max_u32(m);
        return best >= kKeys;
    };
    auto take = [&]() {                                          // it becomes the n-th
        const int w = __builtin_ctzll(__builtin_amdgcn_ballot_w64(m == best));
        if (lane == n) {
            got = best;
            from = (uint32_t)w;
        }
        const uint32_t mine = lane == w ? ~0u : 0u;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            // (as bits: the compiler would turn a choice of neighbours into a search for one)
            if (SORTED) u[j] = (u[j] & ~mine) | ((j + 1 < VPL ? u[j + 1] : 0u) & mine);
            else u[j] = u[j] == best ? u[j] & ~mine : u[j];
        }
    };
    for (; n < a.k && highest(); ++n) take();
    if (!EXACT && n == a.k) {                                    // and those too near to the k-th
        const float last = order_value((uint32_t)__builtin_amdgcn_readlane((int)got, n - 1));
        for (; highest(); ++n) {
            const float now = order_value(best);
            if (last - now > 2.f * base + (fabsf(last) + fabsf(now)) * R + 1e-36f) break;
            if (n == 64) break;                                  // too many
            take();
        }
    }
    if (n == 64) {
        choose64<KIND>(a, l, bias, o, in, slot, id);
        return;
    }
    const int at = lane < n ? (int)(from >> o.shift) * o.gs + (VPL - 1 - (int)(got & MASK)) * LG + (int)(from & (LG - 1)) : -1;
    if constexpr (!EXACT) {
        // every key further from the next than both may be off by?
        const uint32_t next = (uint32_t)__shfl_down((int)got, 1, 64);
        const float x = order_value(got), y = order_value(next);
        const bool open = lane + 1 < n && !(x - y > 2.f * base + (fabsf(x) + fabsf(y)) * R + 1e-36f);
        if (__ballot(open)) {
            const Softmax64 z = softmax64<KIND>(l);
            const double key = lane < n ? key64<KIND>(load_logit<DT>(row, at),
                                                      KIND != kByLogit && a.bias ? a.bias[at] : 0.f, z) : 0.0;
            const uint64_t bits = __builtin_bit_cast(uint64_t, key);
            int rank = 0;
            for (int c = 0; c < n; ++c) {
                const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), c);
                const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)bits, c);
                const double other = __builtin_bit_cast(double, hi << 32 | lo);
                rank += other > key || (other == key && __builtin_amdgcn_readlane(at, c) < at) ? 1 : 0;
            }
            for (int q = 0; q < a.k; ++q) {
                const uint64_t who = __ballot(lane < n && rank == q);
                if (!who) break;
                const int e = __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)who) - 1);
                if (lane == slot + q) id = e;
            }
            return;
        }
    }
    const int moved = __shfl(at, lane - slot, 64);
    if ((uint32_t)(lane - slot) < (uint32_t)a.k) id = moved;
}

// A wave takes `batch` tokens one after another; their weights, a token's in a segment of 16 (k up
// to 16) or 32 lanes, are then computed together.
template <int DT, int VPL, int KIND>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int shift, int gs, int batch) {
    const int lane = threadIdx.x & 63, LG = 1 << shift, group = lane >> shift, within = lane & (LG - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);       // (scalar row addresses)
    const int waves = blockDim.x >> 6, seg = a.k <= 16 ? 16 : 32, q = lane & (seg - 1), own = lane >> (a.k <= 16 ? 4 : 5);
    const RouteLane o{shift, gs, group, group * gs + within, LG};
    const bool whole = !a.sigmoid && !a.renormalize;             // weights need every expert's score
    const bool idle = group * gs >= a.E;
    typedef typename Elem<DT>::type L;
    float bias[VPL];
    uint32_t at[VPL];                                            // bytes to the lane's logits; idle places read the token's first
    bool here[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        here[j] = !idle && j * LG + within < gs;
        at[j] = here[j] ? (o.first + j * LG) * (uint32_t)sizeof(L) : 0u;
        bias[j] = !here[j] ? -INFINITY : (KIND != kByLogit && a.bias ? a.bias[o.first + j * LG] : 0.f);
        if (!(bias[j] > -INFINITY)) bias[j] = -INFINITY;         // NaN
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * waves + wave) * batch; t0 < a.T;
         t0 += (int64_t)gridDim.x * waves * batch) {
        int id = -1;
        float top = -INFINITY;
        double sum = 1.0;                                        // of the lane's token (cancels if renormalised)
        for (int b = 0; b < batch && t0 + b < a.T; ++b) {
            const L* row = static_cast<const L*>(a.logits) + (t0 + b) * a.ls;
            float l[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                l[j] = to_f32<DT>(*reinterpret_cast<const L*>(reinterpret_cast<const char*>(row) + at[j]));
            if (KIND != kBySigmoid) {                            // (there a bias or logit of NaN or -Inf shows in the key)
#pragma unroll
                for (int j = 0; j < VPL; ++j) l[j] = here[j] ? sane(l[j]) : -INFINITY;
            }
            choose<DT, KIND, VPL>(a, row, l, bias, o, b * seg, id);
            if (whole) {
                float t = -INFINITY;
#pragma unroll
                for (int j = 0; j < VPL; ++j) t = fmaxf(t, l[j]);
                t = wave_top(t);
                double y = 0.0;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (l[j] > -INFINITY) y += exp((double)l[j] - (double)t);
                y = wave_total(y);
                if (own == b) {
                    top = t;
                    sum = y;
                }
            }
        }
        const int64_t token = t0 + own;
        const float mine = id >= 0 ? load_logit<DT>(a.logits, token * a.ls + id) : -INFINITY;
        double s = 0.0;
        if (a.sigmoid) {
            if (id >= 0) s = sigmoid64(mine);
        } else {
            if (a.renormalize) {
                top = mine;
                group_steps(seg, [&](auto swap) { top = fmaxf(top, __uint_as_float(swap(__float_as_uint(top)))); });
            }
            if (id >= 0) s = exp((double)mine - (double)top) / sum;
        }
        if (a.renormalize) {
            double total = s;
            group_steps(seg, [&](auto swap) {
                const uint64_t u = __builtin_bit_cast(uint64_t, total);
                total += __builtin_bit_cast(double, (uint64_t)swap((uint32_t)(u >> 32)) << 32 | swap((uint32_t)u));
            });
            s = total > 0.0 ? s / total : 0.0;
        }
        if (q < a.k && own < batch && token < a.T) {
            a.ids[token * a.k + q] = id;
            a.w[token * a.k + q] = (float)((double)a.scale * s);
        }
    }
}

// A wave a token; few tokens over as many CUs.  (A grid holds fewer than 2^32 threads.)
static dim3 token_grid(int T, int waves) { return dim3((unsigned)std::min(((int64_t)T + waves - 1) / waves, (int64_t)1 << 20)); }

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    const bool grouped = a.top_groups < a.groups;
    const int kind = !a.bias && !grouped ? kByLogit : (a.sigmoid ? kBySigmoid : kBySoftmax);
    const int groups = grouped ? a.groups : 1, gs = a.E / groups;
    int shift = 6;
    while ((groups << shift) > 64) --shift;
    const int vpl = (gs + (1 << shift) - 1) >> shift;
    // few tokens: one a wave, a wave a block; many: as many a wave as their weights have room for
    // (groups, us with 1, 2, 4 a wave: T=4096 8.3 / 9.2 / 12.8, T=8192 12.8 / 11.8 / 14.4, T=16384 22.3 / 19.4
    // / 18.5, T=65536 76 / 65 / 61)
    const int waves = a.T <= 1024 ? 1 : 4, batch = a.T <= 4096 ? 1 : (a.k <= 16 && a.T >= 16384 ? 4 : 2);
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto run = [&](auto v) {
            constexpr int VPL = decltype(v)::value;
            auto go = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, token_grid(a.T, waves * batch), dim3(64 * waves), 0, s, a, shift, gs, batch);
            };
            if (kind == kByLogit) go(route_kernel<DT, VPL, kByLogit>);
            else if (kind == kBySigmoid) go(route_kernel<DT, VPL, kBySigmoid>);
            else go(route_kernel<DT, VPL, kBySoftmax>);
        };
        if (vpl <= 2) run(std::integral_constant<int, 2>{});
        else if (vpl <= 5) run(std::integral_constant<int, 5>{});
        else if (vpl <= 8) run(std::integral_constant<int, 8>{});
        else if (vpl <= 16) run(std::integral_constant<int, 16>{});
        else run(std::integral_constant<int, 32>{});
    });
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// gradient.  With p the chosen scores' shares (renormalised) and c the scale:
//   renormalised     dl_j = c p_j (dw_j - sum_i p_i dw_i), for sigmoid times 1 - s_j
//   sigmoid          dl_j = c dw_j s_j (1 - s_j)
//   softmax          dl_e = s_e (c dw_e - sum_j c s_j dw_j), every expert
// and 0 elsewhere.  A wave takes a token and writes its whole row, eight experts a lane (one,
// of fewer than eight); the chosen experts' values reach their lanes through LDS.
// ---------------------------------------------------------------------------
constexpr int kGradWaves = 4;

// exp(x) to about an ulp: the product's rounding is made good.
__device__ __forceinline__ float near_exp(float x) {
    x = fmaxf(x, -200.f);                                         // (0 from there on; no Inf - Inf below)
    const float t = x * kLog2e, r = fmaf(x, kLog2e, -t), e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, (r + x * 1.92596299e-8f) * 0.693147181f, e);   // (log2 e - kLog2e = 1.926e-8)
}

// What the wave's lanes have written to LDS is seen by all of them (LDS serves a wave in order).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

template <int DT, int N, int UPL, bool DENSE>
__global__ __launch_bounds__(64 * kGradWaves) void route_grad_kernel(RouteGradArgs a) {
    __shared__ __attribute__((aligned(16))) float lds[kGradWaves][UPL * 64 * N];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, units = unit_count<N>(a.E);
    float* row = lds[wave];
    for (int64_t token = (int64_t)blockIdx.x * waves + wave; token < a.T; token += (int64_t)gridDim.x * waves) {
        float l[UPL][N];
        if (DENSE) {
#pragma unroll
            for (int i = 0; i < UPL; ++i)
                if (lane + 64 * i < units)
                    load_unit<DT, N>(a.logits, token * a.ls + unit_begin<N>(lane + 64 * i, a.E), l[i]);
        }
        int id = -1;
        float dw = 0.f, mine = -INFINITY;
        if (lane < a.k) {
            id = a.ids[token * a.k + lane];
            if ((uint32_t)id >= (uint32_t)a.E) id = -1;
            if (id >= 0) {
                dw = a.dw[token * a.k + lane];
                mine = load_logit<DT>(a.logits, token * a.ls + id);
            }
        }
        float mean = 0.f, g = 0.f;                               // g: lane q's gradient
        if constexpr (DENSE) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < UPL; ++i)
                if (lane + 64 * i < units) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        l[i][e] = sane(l[i][e]);
                        top = fmaxf(top, l[i][e]);
                    }
                }
            top = wave_top(top);
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
                const int u = lane + 64 * i;
                if (u >= units) continue;
                const int old = u * N - unit_begin<N>(u, a.E);    // experts of the unit before
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    l[i][e] = l[i][e] > -INFINITY ? near_exp(l[i][e] - top) : 0.f;
                    if (e >= old) sum += l[i][e];
                }
            }
            sum = wave_total(sum);
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
            for (int i = 0; i < UPL; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) l[i][e] *= inv;       // scores
            g = a.scale * dw;
            mean = wave_total(id >= 0 && mine > -INFINITY ? near_exp(mine - top) * inv * g : 0.f);
        } else if (a.renormalize) {
            float p;
            if (a.sigmoid) {
                const double s = id >= 0 ? sigmoid64(mine) : 0.0, total = wave_total(s);
                p = total > 0.0 ? (float)(s / total) : 0.f;
            } else {
                const float top = wave_top(mine);
                p = id >= 0 && mine > -INFINITY ? expf(mine - top) : 0.f;
                const float total = wave_total(p);
                p = total > 0.f ? p / total : 0.f;
            }
            g = a.scale * p * (dw - wave_total(p * dw));
            if (a.sigmoid) g *= 1.0f / (1.0f + expf(mine));
        } else {
            g = id >= 0 ? a.scale * dw / (1.0f + expf(-mine)) / (1.0f + expf(mine)) : 0.f;
        }
        // slots of one expert: the first takes the sum, in slot order
        bool first = id >= 0;
        float total = 0.f;
        for (int q = 0; q < a.k; ++q) {
            const int other = __builtin_amdgcn_readlane(id, q);
            const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(g), q));
            total += other == id ? v : 0.f;
            first = first && (other != id || q >= lane);
        }
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) row[(i * 64 + lane) * N + e] = 0.f;
        wave_sync();
        if (first) row[id] = total;
        wave_sync();
#pragma unroll
        for (int i = 0; i < UPL; ++i) {
            const int u = lane + 64 * i;
            if (u >= units) continue;
            const int c = unit_begin<N>(u, a.E);
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = DENSE ? l[i][e] * (row[c + e] - mean) : row[c + e];
            store_unit<DT, N>(a.dlogits, token * a.ds + c, v);
        }
        wave_sync();
    }
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s) {
    const int waves = a.T <= 1024 ? 1 : kGradWaves;
    const bool dense = !a.sigmoid && !a.renormalize;
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto run = [&](auto n, auto upl) {
            constexpr int N = decltype(n)::value, UPL = decltype(upl)::value;
            if (dense)
                hipLaunchKernelGGL((route_grad_kernel<DT, N, UPL, true>), token_grid(a.T, waves), dim3(64 * waves), 0, s, a);
            else
                hipLaunchKernelGGL((route_grad_kernel<DT, N, UPL, false>), token_grid(a.T, waves), dim3(64 * waves), 0, s, a);
        };
        if (a.E < 8) run(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
        else if (a.E <= 512) run(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
    });
    return hipGetLastError();
}

}  // namespace moe
