// Route (gfx950): a token's experts and weights from its router logits, and the logits'
// gradient from the weights'.
//
// A wave takes a token.  With LG = 64 / groups lanes (a power of two) to a group, lane l
// holds experts gs (l / LG) + LG j + l % LG of groups of gs experts: a group's highest keys
// meet in LG lanes, and every round of the choice is one maximum over the wave.  Keys are
// compared in fp64: their order is then that of the definition (two different fp32 logits
// give scores whose fp32 roundings may tie or swap).
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

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
    return v;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

template <int DT, int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int LG, int gs) {
    const int lane = threadIdx.x & 63, group = lane / LG, within = lane & (LG - 1);
    const int waves = blockDim.x >> 6;
    const bool scored = a.bias || a.top_groups < a.groups;       // else keys order as the logits do
    for (int64_t token = (int64_t)blockIdx.x * waves + (threadIdx.x >> 6); token < a.T; token += (int64_t)gridDim.x * waves) {
    float l[VPL];
    int e[VPL];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int i = j * LG + within;
        e[j] = group < a.groups && i < gs ? group * gs + i : -1;
        l[j] = e[j] >= 0 ? load_logit<DT>(a.logits, token * a.ls + e[j]) : -INFINITY;
        top = fmaxf(top, l[j]);
    }
    double sum = 1.0;
    if (!a.sigmoid && (scored || !a.renormalize)) {
        top = wave_max_f32(top);
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (l[j] > -INFINITY) sum += exp((double)l[j] - (double)top);
        sum = wave_sum_f64(sum);
    }
    double key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        key[j] = (double)l[j];
        if (scored && l[j] > -INFINITY) {
            key[j] = a.sigmoid ? sigmoid64(l[j]) : exp((double)l[j] - (double)top) / sum;
            if (a.bias) {
                key[j] += (double)a.bias[e[j]];
                if (!(key[j] > -INFINITY)) key[j] = -INFINITY;   // NaN
            }
        }
    }
    if (a.top_groups < a.groups) {
        double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            b2 = fmax(b2, fmin(b1, key[j]));
            b1 = fmax(b1, key[j]);
        }
        for (int o = 1; o < LG; o <<= 1) {
            const double c1 = __shfl_xor(b1, o, 64), c2 = __shfl_xor(b2, o, 64);
            b2 = fmax(fmin(b1, c1), fmax(b2, c2));
            b1 = fmax(b1, c1);
        }
        if (a.group_keys == 2 && b2 > -INFINITY) b1 += b2;
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl(b1, g * LG, 64);
            ahead += other > b1 || (other == b1 && g < group) ? 1 : 0;
        }
        if (ahead >= a.top_groups) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = -INFINITY;
        }
    }
    int id = -1;                                                  // lane q: the q-th expert
    for (int q = 0; q < a.k; ++q) {
        double best = -INFINITY;
        int at = INT_MAX;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = e[j];
            }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double b = __shfl_xor(best, o, 64);
            const int i = __shfl_xor(at, o, 64);
            if (b > best || (b == best && i < at)) {
                best = b;
                at = i;
            }
        }
        if (!(best > -INFINITY)) break;
        if (lane == q) id = at;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e[j] == at) key[j] = -INFINITY;
    }
    // weights: lane q's
    const float mine = id >= 0 ? load_logit<DT>(a.logits, token * a.ls + id) : -INFINITY;
    double s = 0.0;
    if (a.sigmoid) {
        if (id >= 0) s = sigmoid64(mine);
    } else {
        if (a.renormalize) {
            top = wave_max_f32(mine);
            sum = 1.0;                                            // cancels
        }
        if (id >= 0) s = exp((double)mine - (double)top) / sum;
    }
    if (a.renormalize) {
        const double total = wave_sum_f64(s);
        s = total > 0.0 ? s / total : 0.0;
    }
    if (lane < a.k) {
        a.ids[token * a.k + lane] = id;
        a.w[token * a.k + lane] = (float)((double)a.scale * s);
    }
    }
}

// A wave a token; few tokens over as many CUs.  (A grid holds fewer than 2^32 threads.)
static dim3 token_grid(int T, int waves) { return dim3((unsigned)std::min(((int64_t)T + waves - 1) / waves, (int64_t)1 << 20)); }

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    int LG = 64;
    while (LG * a.groups > 64) LG >>= 1;
    const int gs = a.E / a.groups, vpl = (gs + LG - 1) / LG;
    const int waves = a.T <= 1024 ? 1 : 4;
    const dim3 grid = token_grid(a.T, waves);
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto run = [&](auto v) {
            hipLaunchKernelGGL((route_kernel<DT, decltype(v)::value>), grid, dim3(64 * waves), 0, s, a, LG, gs);
        };
        if (vpl <= 1) run(std::integral_constant<int, 1>{});
        else if (vpl <= 2) run(std::integral_constant<int, 2>{});
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
// and 0 elsewhere.  A wave takes a token; it writes the whole row.
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    for (int64_t token = (int64_t)blockIdx.x * waves + (threadIdx.x >> 6); token < a.T; token += (int64_t)gridDim.x * waves) {
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
    const bool dense = !a.sigmoid && !a.renormalize;
    float top = -INFINITY, sum = 0.f, g = 0.f, mean = 0.f;        // g: lane q's gradient
    if (dense) {
        for (int e = lane; e < a.E; e += 64) top = fmaxf(top, load_logit<DT>(a.logits, token * a.ls + e));
        top = wave_max_f32(top);
        for (int e = lane; e < a.E; e += 64) {
            const float l = load_logit<DT>(a.logits, token * a.ls + e);
            sum += l > -INFINITY ? expf(l - top) : 0.f;
        }
        sum = wave_sum_f32(sum);
        const float s = id >= 0 && mine > -INFINITY ? expf(mine - top) / sum : 0.f;
        g = a.scale * dw;
        mean = wave_sum_f32(s * g);
    } else if (a.renormalize) {
        float p;
        if (a.sigmoid) {
            const double s = id >= 0 ? sigmoid64(mine) : 0.0, total = wave_sum_f64(s);
            p = total > 0.0 ? (float)(s / total) : 0.f;
        } else {
            top = wave_max_f32(mine);
            p = id >= 0 && mine > -INFINITY ? expf(mine - top) : 0.f;
            const float total = wave_sum_f32(p);
            p = total > 0.f ? p / total : 0.f;
        }
        g = a.scale * p * (dw - wave_sum_f32(p * dw));
        if (a.sigmoid) g *= 1.0f / (1.0f + expf(mine));
    } else {
        g = id >= 0 ? a.scale * dw / (1.0f + expf(-mine)) / (1.0f + expf(mine)) : 0.f;
    }
    for (int e = lane; e < ((a.E + 63) & ~63); e += 64) {
        float v = 0.f;
        for (int q = 0; q < a.k; ++q) {
            const int at = __shfl(id, q, 64);
            const float add = __shfl(g, q, 64);
            v += at == e ? add : 0.f;
        }
        if (e >= a.E) continue;
        if (dense) {
            const float l = load_logit<DT>(a.logits, token * a.ls + e);
            v = l > -INFINITY ? expf(l - top) / sum * (v - mean) : 0.f;
        }
        static_cast<typename Elem<DT>::type*>(a.dlogits)[token * a.ds + e] = (typename Elem<DT>::type)from_f32<DT>(v);
    }
    }
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s) {
    const int waves = a.T <= 1024 ? 1 : 4;
    const dim3 grid = token_grid(a.T, waves);
    with_dtype(a.dtype, [&](auto dt) {
        hipLaunchKernelGGL((route_grad_kernel<decltype(dt)::value>), grid, dim3(64 * waves), 0, s, a);
    });
    return hipGetLastError();
}

}  // namespace moe
