// Residual addition and root-mean-square norm (gfx950), out in the rows' type and as MXFP8,
// and its gradients:
//   h = x + residual, r = 1 / sqrt(mean h^2 + eps), y = h r w
//   n = h r:  dx = r (w dy - n mean(w dy n)) + dh,   dw = sum over rows of dy n
// Bound by memory: a block keeps its row in registers between the sum and its use, so that
// every row is read once and written once.
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
        const RowSplit r = row_split(units, 1);
        with_upt(r.upt, [&](auto upt) {
            hipLaunchKernelGGL((norm_kernel<DT, 8, decltype(upt)::value>), grid, dim3(r.threads), 0, s, a, units);
        });
    });
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// gradients: a block takes rows one after another and keeps the weight's gradient of its
// columns in registers; its sums go to the workspace, [blocks][d], and a second kernel adds
// them in block order.
// ---------------------------------------------------------------------------
template <int DT, int N, int UPT>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormGradArgs a, int units) {
    __shared__ float red[16];
    const int tid = threadIdx.x, nt = blockDim.x;
    float dw[UPT][N];
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = 0.f;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const float rstd = a.rstd[row];
        float n[UPT][N], g[UPT][N], s = 0.f;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = tid + nt * i;
            if (u >= units) continue;
            const int c = unit_begin<N>(u, a.d), old = u * N - c;
            load_unit<DT, N>(a.h, row * a.hs + c, n[i]);
            load_unit<DT, N>(a.dy, row * a.dys + c, g[i]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                n[i][e] *= rstd;
                dw[i][e] = fmaf(g[i][e], n[i][e], dw[i][e]);
            }
            if (a.dx) {
                float w[N];
                load_weight<N>(a.w, a.wdtype, c, w);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    g[i][e] *= w[e];
                    s = e >= old ? fmaf(g[i][e], n[i][e], s) : s;
                }
            }
        }
        if (!a.dx) continue;
        const float mean = block_sum(s, red) / (float)a.d;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = tid + nt * i;
            if (u >= units) continue;
            const int c = unit_begin<N>(u, a.d);
            float o[N];
            if (a.dh) load_unit<DT, N>(a.dh, row * a.dhs + c, o);
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = rstd * (g[i][e] - n[i][e] * mean) + (a.dh ? o[e] : 0.f);
            store_unit<DT, N>(a.dx, row * a.dxs + c, o);
        }
    }
    if (!a.dw) return;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        const int u = tid + nt * i;
        if (u >= units) continue;
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

// Enough blocks to fill the card however narrow the rows, few enough that their sums stay a
// small part of the rows' bytes.
int norm_grad_blocks(int T, int d) {
    const int most = (1 << 22) / d;
    return T < 512 ? T : std::min(T, most < 512 ? 512 : (most > 4096 ? 4096 : most));
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
    const int blocks = norm_grad_blocks(a.T, a.d);
    if (blocks > 0)
        with_dtype(a.dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            if (a.d < 8) {
                hipLaunchKernelGGL((norm_grad_kernel<DT, 1, 1>), dim3(blocks), dim3(64), 0, s, a, a.d);
                return;
            }
            const int units = unit_count<8>(a.d);
            const RowSplit r = row_split(units, 2);
            with_upt(r.upt, [&](auto upt) {
                hipLaunchKernelGGL((norm_grad_kernel<DT, 8, decltype(upt)::value>), dim3(blocks), dim3(r.threads), 0,
                                   s, a, units);
            });
        });
    if (a.dw)
        hipLaunchKernelGGL(norm_dweight_kernel, dim3((a.d + 31) / 32), dim3(1024), 0, s, a.partial, blocks, a.d, a.dw);
    return hipGetLastError();
}

}  // namespace moe
