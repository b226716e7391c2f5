// Rows in units of eight elements (device): a unit is loaded to fp32 and stored from it in
// 16 or 32 bytes.  Rows need no alignment; a row's last unit ends with the row and overlaps
// the one before.  Rows shorter than a unit are taken element by element (N = 1).
#pragma once
#include <type_traits>

#include "device_common.h"
#include "ops.h"
#include "rows.h"

namespace moe {

// Elements of a unit and its start, for rows of d elements.
template <int N>
__host__ __device__ inline int unit_count(int d) { return (d + N - 1) / N; }
template <int N>
__device__ __forceinline__ int unit_begin(int u, int d) { return min(u * N, d - N); }

template <int DT, int N>
__device__ __forceinline__ void load_unit(const void* base, int64_t el, float (&f)[N]) {
    typedef typename Elem<DT>::type E;
    if constexpr (N == 1) {
        f[0] = to_f32<DT>(static_cast<const E*>(base)[el]);
    } else if constexpr (DT == kF32) {
        const u32x4_any_t* p = reinterpret_cast<const u32x4_any_t*>(static_cast<const E*>(base) + el);
        const u32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(a[i]);
            f[4 + i] = __uint_as_float(b[i]);
        }
    } else {
        const u32x4_t v = *reinterpret_cast<const u32x4_any_t*>(static_cast<const E*>(base) + el);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = to_f32<DT>(v[i] & 0xFFFFu);
            f[2 * i + 1] = to_f32<DT>(v[i] >> 16);
        }
    }
}

// Two values rounded to a pair of 16-bit elements.
template <int DT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    return DT == kBF16 ? f32x2_to_bf16x2(a, b) : from_f32<DT>(a) | (from_f32<DT>(b) << 16);
}

// Streaming stores: what is written here is read by the next kernel at the earliest.
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t el, const float (&f)[8]) {
    typedef typename Elem<DT>::type E;
    u32x4_any_t* p = reinterpret_cast<u32x4_any_t*>(static_cast<E*>(base) + el);
    if constexpr (DT == kF32) {
        __builtin_nontemporal_store(u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                            __float_as_uint(f[3])}, p);
        __builtin_nontemporal_store(u32x4_t{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                            __float_as_uint(f[7])}, p + 1);
    } else {
        __builtin_nontemporal_store(u32x4_t{pack_pair<DT>(f[0], f[1]), pack_pair<DT>(f[2], f[3]),
                                            pack_pair<DT>(f[4], f[5]), pack_pair<DT>(f[6], f[7])}, p);
    }
}

template <int DT, int N>
__device__ __forceinline__ void store_unit(void* base, int64_t el, const float (&f)[N]) {
    if constexpr (N == 1) static_cast<typename Elem<DT>::type*>(base)[el] = (typename Elem<DT>::type)from_f32<DT>(f[0]);
    else store8<DT>(base, el, f);
}

// f rounded to the type and back.
template <int DT>
__device__ __forceinline__ float round_to(float f) { return to_f32<DT>(from_f32<DT>(f)); }

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Runs f with the type as a compile-time constant.
template <typename F>
inline void with_dtype(int dtype, F f) {
    if (dtype == kBF16) f(std::integral_constant<int, kBF16>{});
    else if (dtype == kF16) f(std::integral_constant<int, kF16>{});
    else f(std::integral_constant<int, kF32>{});
}

}  // namespace moe
