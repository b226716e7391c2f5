// SwiGLU between the products (gfx950): a = gate / (1 + exp(-gate)) * up, out in the rows'
// type and as MXFP8, the rows gate | up kept as MXFP8 for the way back, and its gradient:
//   s = 1 / (1 + exp(-gate)):  dgate = da up s (1 + gate (1 - s)),  dup = da gate s
// Bound by memory; eight columns a thread, each row read and written once.  65536 rows of F = 1024,
// bf16: there with a in bf16 and u kept 91-112 us, back from what was kept 105-125 us (5 TB/s; a large
// copy reaches 4.95).  The exponential and the division are the accurate ones, which the memory
// hides: a's MXFP8 codes are then those of the fp32 formula.
#include "block.h"
#include "eights.h"
#include "mx_common.h"

namespace moe {

// Rows that hold something: all, or up to the last group's end.
__device__ __forceinline__ int live_rows(const SwigluArgs& p) {
    return p.offsets ? min(max(p.offsets[p.G], 0), p.M) : p.M;
}

// Walks (row, unit) pairs of `units` units a row, `step` threads apart, without dividing.
struct Walk {
    int row, unit, drow, dunit;
    __device__ __forceinline__ Walk(int64_t first, int64_t step, int units) {
        row = (int)(first / units);
        unit = (int)(first - (int64_t)row * units);
        drow = (int)(step / units);
        dunit = (int)(step - (int64_t)drow * units);
    }
    __device__ __forceinline__ void next(int units) {
        row += drow;
        unit += dunit;
        if (unit >= units) {
            unit -= units;
            ++row;
        }
    }
};

template <int N>
__device__ __forceinline__ void store_mx8(const float (&f)[N], uint8_t* codes, uint8_t* scales, int64_t el) {
    if constexpr (N == 8) {
        uint32_t sb;
        const u32x2_t q = mx8_quantize8(f, sb);
        __builtin_nontemporal_store(q, reinterpret_cast<u32x2_t*>(codes + el));
        if ((threadIdx.x & 3) == 0) scales[el >> 5] = (uint8_t)sb;
    }
}

template <int DT, int N>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs p, int units) {
    const int n = live_rows(p);
    Walk w((int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256, units);
    // MXFP8: a row is whole quads of units, so a quad of lanes stays together
    for (; w.row < n; w.next(units)) {
        const int64_t r = w.row;
        const int c = unit_begin<N>(w.unit, p.F);
        float g[N], u[N];
        load_unit<DT, N>(p.u, r * p.us + c, g);
        load_unit<DT, N>(p.u, r * p.us + p.F + c, u);
        if (p.kept) {
            store_mx8<N>(g, p.kept, p.kept_s, r * 2 * p.F + c);
            store_mx8<N>(u, p.kept, p.kept_s, r * 2 * p.F + p.F + c);
        }
        if (!p.a && !p.codes) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) g[e] = g[e] / (1.0f + expf(-g[e])) * u[e];
        if (p.a) store_unit<DT, N>(p.a, r * p.as + c, g);
        if (p.codes) store_mx8<N>(g, p.codes, p.scales, r * p.F + c);
    }
}

template <int DT, int N, bool MX>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(SwigluArgs p, int units) {
    const int n = live_rows(p);
    Walk w((int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256, units);
    for (; w.row < n; w.next(units)) {
        const int64_t r = w.row;
        const int c = unit_begin<N>(w.unit, p.F);
        float g[N], u[N], da[N];
        if constexpr (MX) {
            const int64_t el = r * 2 * p.F + c;
            const uint8_t* k = static_cast<const uint8_t*>(p.u) + el;
            mx8_decode8(*reinterpret_cast<const u32x2_t*>(k), p.kept_s[el >> 5], g);
            mx8_decode8(*reinterpret_cast<const u32x2_t*>(k + p.F), p.kept_s[(el + p.F) >> 5], u);
        } else {
            load_unit<DT, N>(p.u, r * p.us + c, g);
            load_unit<DT, N>(p.u, r * p.us + p.F + c, u);
        }
        load_unit<DT, N>(p.a, r * p.as + c, da);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float s = 1.0f / (1.0f + expf(-g[e])), d = da[e] * s;
            da[e] = d * u[e] * (1.0f + g[e] * (1.0f - s));
            u[e] = d * g[e];
        }
        store_unit<DT, N>(p.du, r * p.dus + c, da);
        store_unit<DT, N>(p.du, r * p.dus + p.F + c, u);
    }
}

static unsigned swiglu_blocks(int64_t work) {
    const int64_t n = (work + 255) / 256;
    return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const int units = a.F < 8 ? a.F : unit_count<8>(a.F);
        const dim3 grid(swiglu_blocks((int64_t)a.M * units));
        if (a.F < 8) hipLaunchKernelGGL((swiglu_kernel<DT, 1>), grid, dim3(256), 0, s, a, units);
        else hipLaunchKernelGGL((swiglu_kernel<DT, 8>), grid, dim3(256), 0, s, a, units);
    });
    return hipGetLastError();
}

hipError_t launch_swiglu_grad(const SwigluArgs& a, hipStream_t s) {
    with_dtype(a.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const int units = a.F < 8 ? a.F : unit_count<8>(a.F);
        const dim3 grid(swiglu_blocks((int64_t)a.M * units));
        if (a.kept_s) hipLaunchKernelGGL((swiglu_grad_kernel<DT, 8, true>), grid, dim3(256), 0, s, a, units);
        else if (a.F < 8) hipLaunchKernelGGL((swiglu_grad_kernel<DT, 1, false>), grid, dim3(256), 0, s, a, units);
        else hipLaunchKernelGGL((swiglu_grad_kernel<DT, 8, false>), grid, dim3(256), 0, s, a, units);
    });
    return hipGetLastError();
}

}  // namespace moe
