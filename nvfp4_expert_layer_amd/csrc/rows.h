// Rows of bf16, f16 or f32 elements of any alignment and width (device).
#pragma once
#include "device_common.h"
#include "ops.h"

namespace moe {

// ---------------------------------------------------------------------------
// Row elements: 16-byte units of VEC elements, or single elements (VEC 1) for rows
// shorter than a unit.  Unit u of a row of d elements starts at unit_start.
// ---------------------------------------------------------------------------
template <int DT> struct Elem;
template <> struct Elem<kBF16> { typedef uint16_t type; };
template <> struct Elem<kF16> { typedef uint16_t type; };
template <> struct Elem<kF32> { typedef uint32_t type; };

template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits) {
    if constexpr (DT == kBF16) return bf16_bits_to_f32(bits);
    else if constexpr (DT == kF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    else return __uint_as_float(bits);
}
template <int DT>
__device__ __forceinline__ uint32_t from_f32(float f) {
    if constexpr (DT == kBF16) return f32_to_bf16_rne(f);
    else if constexpr (DT == kF16) return f32_to_f16_bits(f);
    else return __float_as_uint(f);
}

template <int DT, bool VECTOR>
struct Row {
    typedef typename Elem<DT>::type E;
    static constexpr int VEC = VECTOR ? 16 / (int)sizeof(E) : 1;
    static __host__ __device__ int units(int d) { return (d + VEC - 1) / VEC; }
    static __device__ int unit_start(int u, int d) { return min(u * VEC, d - VEC); }
    struct Raw { uint32_t w[VECTOR ? 4 : 1]; };
    static __device__ __forceinline__ Raw load(const void* base, int64_t el) {
        Raw r;
        if constexpr (VECTOR) {
            const u32x4_t v = *reinterpret_cast<const u32x4_any_t*>(static_cast<const E*>(base) + el);
            r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
        } else {
            r.w[0] = static_cast<const E*>(base)[el];
        }
        return r;
    }
    static __device__ __forceinline__ float get(const Raw& r, int i) {
        if constexpr (!VECTOR || sizeof(E) == 4) return to_f32<DT>(r.w[i]);
        else return to_f32<DT>((i & 1) ? r.w[i / 2] >> 16 : r.w[i / 2] & 0xFFFFu);
    }
    // Streaming stores: a row is written once and read by the next kernel at the earliest
    // (T=8192, d=4096: gradient rows alone 149 -> 104 us, combine 116 -> 109 us).
    static __device__ __forceinline__ void store(void* base, int64_t el, const float (&f)[VEC]) {
        E* p = static_cast<E*>(base) + el;
        if constexpr (!VECTOR) {
            *p = (E)from_f32<DT>(f[0]);
        } else if constexpr (sizeof(E) == 4) {
            __builtin_nontemporal_store(u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                                __float_as_uint(f[3])},
                                        reinterpret_cast<u32x4_any_t*>(p));
        } else {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = DT == kBF16 ? f32x2_to_bf16x2(f[2 * i], f[2 * i + 1])
                                   : from_f32<DT>(f[2 * i]) | (from_f32<DT>(f[2 * i + 1]) << 16);
            __builtin_nontemporal_store(u32x4_t{o[0], o[1], o[2], o[3]}, reinterpret_cast<u32x4_any_t*>(p));
        }
    }
};

}  // namespace moe
