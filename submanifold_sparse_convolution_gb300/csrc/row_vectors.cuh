// Vectors of a row's elements: loads, stores and their conversion to and from
// fp32, for the kernels that walk rows in registers.
#pragma once
#include "rows.cuh"

namespace spconv {

// W consecutive elements as they lie in memory (W = 8 is one or two 16-byte loads).
template <typename T, int W>
struct alignas(sizeof(T) * W < 16 ? sizeof(T) * W : 16) Pack {
    T v[W];
};

// To fp32 and back (one rounding); pairs of bf16 take one instruction each.
template <int W>
__device__ __forceinline__ void unpack(const Pack<float, W>& p, float (&f)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) f[j] = p.v[j];
}
template <int W>
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, W>& p, float (&f)[W]) {
    if constexpr (W == 8) {
        const uint4 q = reinterpret_cast<const uint4&>(p);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(u[j] << 16);
            f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = __bfloat162float(p.v[j]);
    }
}
template <int W>
__device__ __forceinline__ void pack(const float (&f)[W], Pack<float, W>& p) {
#pragma unroll
    for (int j = 0; j < W; ++j) p.v[j] = f[j];
}
template <int W>
__device__ __forceinline__ void pack(const float (&f)[W], Pack<__nv_bfloat16, W>& p) {
    if constexpr (W == 8) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            u[j] = reinterpret_cast<const uint32_t&>(v);
        }
        reinterpret_cast<uint4&>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) p.v[j] = __float2bfloat16_rn(f[j]);
    }
}

// Four values as e4m3.
__device__ __forceinline__ uint32_t pack_e4m3(const float* v) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// W values to memory with W bytes' alignment.
template <int W>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, const float* v) {
    if (W == 8) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_e4m3(v), pack_e4m3(v + 4));
    } else if (W == 2) {
        *reinterpret_cast<uint16_t*>(dst) = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1 % W]), __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) dst[j] = __nv_cvt_float_to_fp8(v[j], __NV_SATFINITE, __NV_E4M3);
    }
}

// Calls f with the widest vectors (as a constant) that every row starts on: all
// is the addresses' and row strides' bits in bytes, or-ed together.
template <typename T, typename F>
int with_width(uintptr_t all, int32_t c, F&& f) {
    auto fits = [&](int w) { return c % w == 0 && all % (w * sizeof(T)) == 0; };
    if constexpr (sizeof(T) == 2) {
        if (fits(8)) return f(std::integral_constant<int, 8>());
    }
    if (fits(4)) return f(std::integral_constant<int, 4>());
    if (fits(2)) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>());
}

}  // namespace spconv
