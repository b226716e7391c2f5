// Residual addition and root-mean-square norm (gfx950), out in the rows' type and as MXFP8,
// and its gradients:
//   h = x + residual, r = 1 / sqrt(mean h^2 + eps), y = h r w
//   n = h r:  dx = r (w dy - n mean(w dy n)) + dh,   dw = sum over rows of dy n
// Bound by memory: a block keeps its row in registers between the sum and its use, so that
// every row is read once and written once.  T=8192, d=4096, bf16 with a residual, out in bf16 and
// MXFP8: 56 us, 5.4 TB/s (a large copy reaches 4.95); one row 3.1 us of kernel.
#include <algorithm>

#include "block.h"
#include "eights.h"
#include "mx_common.h"

namespace moe {

// The weight's elements, of a type of their own.
template <int N>
__device__ __forceinline__ void load_weight(const void* w, int dtype, int el, float (&f)[N]) {
    if (dtype == kBF16) load_unit<kBF16, N>(w, el, f);
    else if (dtype == kF16) load_unit<kF16, N>(w, el, f);
    else load_unit<kF32, N>(w, el, f);
}

// Sum of v over the block's threads, in every thread: lanes by halves, then waves in order.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum_f32(v);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    __syncthreads();                                     // red's previous readers are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
    for (int i = 1; i < waves; ++i) s += red[i];
    return s;
}

// A block a row; thread t takes units t, t + blockDim.x, ...
template <int DT, int N, int UPT>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a, int units) {
    __shared__ float red[16];
    const int tid = threadIdx.x, nt = blockDim.x;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        float h[UPT][N], ss = 0.f;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = tid + nt * i;
            if (u >= units) continue;
            const int c = unit_begin<N>(u, a.d), old = u * N - c;     // elements of the unit before
            load_unit<DT, N>(a.x, row * a.xs + c, h[i]);
            if (a.res) {
                float r[N];
                load_unit<DT, N>(a.res, row * a.ress + c, r);
#pragma unroll
                for (int e = 0; e < N; ++e) h[i][e] = round_to<DT>(h[i][e] + r[e]);
            }
            if (a.h) store_unit<DT, N>(a.h, row * a.hs + c, h[i]);
#pragma unroll
            for (int e = 0; e < N; ++e) ss += e >= old ? h[i][e] * h[i][e] : 0.f;
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red) / (float)a.d + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
        if (!a.y && !a.codes) continue;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = tid + nt * i;
            if (u >= units) continue;
            const int c = unit_begin<N>(u, a.d);
            float w[N], y[N];
            load_weight<N>(a.w, a.wdtype, c, w);
#pragma unroll
            for (int e = 0; e < N; ++e) y[e] = h[i][e] * rstd * w[e];
            if (a.y) store_unit<DT, N>(a.y, row * a.ys + c, y);
            if constexpr (N == 8) {
                if (a.codes) {                           // d is a multiple of 32: a quad of lanes holds a block
                    uint32_t sb;
                    const u32x2_t q = mx8_quantize8(y, sb);
                    __builtin_nontemporal_store(q, reinterpret_cast<u32x2_t*>(a.codes + row * a.d + c));
                    if ((u & 3) == 0) a.scales[(row * a.d + c) >> 5] = (uint8_t)sb;
                }
            }
        }
    }
}

// The units of a row to threads: units a thread (1, 2, 4 or 8) and threads of a block.
struct RowSplit {
    int upt, threads;
};
static RowSplit row_split(int units, int want) {
    int upt = want;
    while (upt < 8 && (units + upt - 1) / upt > 1024) upt *= 2;
    const int t = ((units + upt - 1) / upt + 63) & ~63;
    while (upt > 1 && (upt / 2) * t >= units) upt /= 2;
    return RowSplit{upt, t};
}

template <typename F>
static void with_upt(int upt, F f) {
    if (upt == 1) f(std::integral_constant<int, 1>{});
    else if (upt == 2) f(std::integral_constant<int, 2>{});
    else if (upt == 4) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 8>{});
}

// A grid holds fewer than 2^32 threads.
static unsigned row_blocks(int64_t n) { return (unsigned)(n < (1 << 21) ? n : (1 << 21)); }

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const dim3 grid(row_blocks(a.T));
        if (a.d < 8) {
            hipLaunchKernelGGL((norm_kernel<DT, 1, 1>), grid, dim3(64), 0, s, a, a.d);
            return;
        }
        const int units = unit_count<8>(a.d);
        const RowSplit r = row_split(units, units > 512 ? 2 : 1);    // (T=2048, d=8192: 24 us, 31 with one unit a thread)
        with_upt(r.upt, [&](auto upt) {
            hipLaunchKernelGGL((norm_kernel<DT, 8, decltype(upt)::value>), grid, dim3(r.threads), 0, s, a, units);
        });
    });
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// gradients.  A block is one or more teams of threads, a row each at a time; a thread keeps the
// weight's gradient of its columns in registers and has the next row's elements under way while
// it works on one.  The teams' sums meet in LDS, the blocks' in the workspace, [blocks][d], and a
// second kernel adds those, all in fixed orders.  T=8192, d=4096, bf16, with dh: 56 us, dx alone 49
// (5.5 TB/s; 68 and 53 with a row a block and no load ahead).
// ---------------------------------------------------------------------------
struct NormGradPlan {
    int upt, threads, teams, blocks;                     // units a thread; threads a row; rows at once; blocks
};
// Teams fill blocks of 1024 threads only when there are rows for 512 blocks of them: then few
// partial sums leave the card no emptier (T=8192, d=1024: 33 us with 4096 blocks of one, 18 so).
static NormGradPlan norm_grad_plan(int T, int d) {
    const RowSplit r = d < 8 ? RowSplit{1, 64} : row_split(unit_count<8>(d), 1);
    const int teams = r.upt > 1 ? 1 : std::max(1, std::min(1024 / r.threads, T / 512));
    return NormGradPlan{r.upt, r.threads, teams, std::min((T + teams - 1) / teams, 512)};
}

// The elements of a row's unit as they lie in memory.
template <int DT, int N>
struct RawUnit {
    typename Row<DT, (N > 1)>::Raw a, b;                 // (fp32: two halves)
    __device__ __forceinline__ void load(const void* base, int64_t el) {
        a = Row<DT, (N > 1)>::load(base, el);
        if constexpr (DT == kF32 && N > 1) b = Row<DT, true>::load(base, el + 4);
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (DT == kF32 && N > 1) return e < 4 ? Row<DT, true>::get(a, e) : Row<DT, true>::get(b, e - 4);
        else return Row<DT, (N > 1)>::get(a, e);
    }
};

template <int DT, int N, int UPT>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormGradArgs a, int units, int threads, int teams) {
    __shared__ float red[16], sums[UPT == 1 ? 1024 * N : 1];
    const int team = threadIdx.x / threads, tid = threadIdx.x - team * threads, wave = threadIdx.x >> 6;
    const int waves = threads >> 6;
    float dw[UPT][N];
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = 0.f;
    // the row's sum, in every thread of the team
    auto row_sum = [&](float s) {
        s = wave_sum_f32(s);
        if (waves == 1) return s;
        __syncthreads();                                 // red's previous readers are done
        if ((threadIdx.x & 63) == 0) red[wave] = s;
        __syncthreads();
        s = red[team * waves];
        for (int i = 1; i < waves; ++i) s += red[team * waves + i];
        return s;
    };
    const int64_t step = (int64_t)gridDim.x * teams;
    int64_t row = (int64_t)blockIdx.x * teams + team;
    // (every team takes as many turns as the first: the block's barriers are for all)
    if constexpr (UPT == 1) {
        const bool mine = tid < units;
        const int c = unit_begin<N>(mine ? tid : 0, a.d), old = tid * N - c;     // elements of the unit before
        float w[N];
        RawUnit<DT, N> h, g, dh;
        float rstd = 0.f;
        if (a.dx) load_weight<N>(a.w, a.wdtype, c, w);
        auto load = [&](int64_t r) {
            rstd = a.rstd[r];
            if (!mine) return;
            h.load(a.h, r * a.hs + c);
            g.load(a.dy, r * a.dys + c);
            if (a.dh) dh.load(a.dh, r * a.dhs + c);
        };
        if (row < a.T) load(row);
        for (int64_t first = (int64_t)blockIdx.x * teams; first < a.T; first += step, row += step) {
            const bool live = row < a.T && mine;
            float n[N], y[N], o[N], s = 0.f;
            const float r = rstd;
            if (live) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    n[e] = h.get(e) * r;
                    y[e] = g.get(e);
                    dw[0][e] = fmaf(y[e], n[e], dw[0][e]);
                    o[e] = a.dh ? dh.get(e) : 0.f;
                    if (a.dx) y[e] *= w[e];
                    if (e >= old) s = fmaf(y[e], n[e], s);
                }
            }
            if (row + step < a.T) load(row + step);
            if (!a.dx) continue;
            const float mean = row_sum(s) / (float)a.d;
            if (!live) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] += r * (y[e] - n[e] * mean);
            store_unit<DT, N>(a.dx, row * a.dxs + c, o);
        }
    } else {
        // wide rows (one team): read again for the second part, from the caches
        for (; row < a.T; row += step) {
            const float rstd = a.rstd[row];
            float mean = 0.f;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (part == 1 && !a.dx) break;
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < UPT; ++i) {
                    const int u = tid + threads * i;
                    if (u >= units) continue;
                    const int c = unit_begin<N>(u, a.d), old = u * N - c;
                    float n[N], y[N], w[N];
                    load_unit<DT, N>(a.h, row * a.hs + c, n);
                    load_unit<DT, N>(a.dy, row * a.dys + c, y);
                    if (a.dx) load_weight<N>(a.w, a.wdtype, c, w);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        n[e] *= rstd;
                        if (part == 0) dw[i][e] = fmaf(y[e], n[e], dw[i][e]);
                        if (a.dx) y[e] *= w[e];
                        if (part == 0 && e >= old) s = fmaf(y[e], n[e], s);
                    }
                    if (part == 0) continue;
                    if (a.dh) load_unit<DT, N>(a.dh, row * a.dhs + c, w);
#pragma unroll
                    for (int e = 0; e < N; ++e) y[e] = rstd * (y[e] - n[e] * mean) + (a.dh ? w[e] : 0.f);
                    store_unit<DT, N>(a.dx, row * a.dxs + c, y);
                }
                if (part == 0 && a.dx) mean = row_sum(s) / (float)a.d;
            }
        }
    }
    if (!a.dw) return;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        if (UPT == 1 && teams > 1) {
#pragma unroll
            for (int e = 0; e < N; ++e) sums[threadIdx.x + e * 1024] = dw[i][e];
            __syncthreads();
            for (int t = 1; t < teams && team == 0; ++t)
#pragma unroll
                for (int e = 0; e < N; ++e) dw[i][e] += sums[t * threads + tid + e * 1024];
        }
        const int u = tid + threads * i;
        if (team || u >= units) continue;
        const int c = unit_begin<N>(u, a.d), old = u * N - c;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e >= old) a.partial[(int64_t)blockIdx.x * a.d + c + e] = dw[i][e];
    }
}

// dw[c] = the sum over the blocks, in a fixed order: 32 columns a workgroup, 32 threads each.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float* partial, int blocks, int d, float* dw) {
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
    float s = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int b = part; b < blocks; b += 32) s += partial[(int64_t)b * d + c];
    }
    red[part][col] = s;
    __syncthreads();
    if (part == 0 && c < d) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += red[i][col];
        dw[c] = s;
    }
}

int norm_grad_blocks(int T, int d) { return norm_grad_plan(T, d).blocks; }

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
    const NormGradPlan p = norm_grad_plan(a.T, a.d);
    const dim3 grid(p.blocks), block(p.threads * p.teams);
    if (p.blocks > 0)
        with_dtype(a.dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            if (a.d < 8) {
                hipLaunchKernelGGL((norm_grad_kernel<DT, 1, 1>), grid, block, 0, s, a, a.d, p.threads, p.teams);
                return;
            }
            with_upt(p.upt, [&](auto upt) {
                hipLaunchKernelGGL((norm_grad_kernel<DT, 8, decltype(upt)::value>), grid, block, 0, s, a, unit_count<8>(a.d),
                                   p.threads, p.teams);
            });
        });
    if (a.dw)
        hipLaunchKernelGGL(norm_dweight_kernel, dim3((a.d + 31) / 32), dim3(1024), 0, s, a.partial, p.blocks, a.d, a.dw);
    return hipGetLastError();
}

}  // namespace moe
