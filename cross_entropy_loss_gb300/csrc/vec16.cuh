// 16-byte vectors of bf16 or fp32 elements (ES bytes each) as floats, for the kernels
// that stream rows.
#pragma once

#include "common.cuh"

namespace foak {

template <int ES>
struct Vec16 {
    static constexpr int N = 16 / ES;  // elements

    static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[N]) {
        if constexpr (ES == 2) {
            f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
            f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
        } else {
            f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
            f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
        }
    }
    // Rounded to nearest even: the one rounding of an output, half a step at most.
    static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
        if constexpr (ES == 2)
            return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7]));
        else
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ void load(const char* p, float (&f)[N]) { unpack(ld_global_v4(p), f); }
    static __device__ __forceinline__ void store(char* p, const float (&f)[N]) {
        *reinterpret_cast<uint4*>(p) = pack(f);
    }
    static __device__ __forceinline__ float load1(const char* p) {
        if constexpr (ES == 2)
            return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(p)) << 16);
        else
            return *reinterpret_cast<const float*>(p);
    }
};

}  // namespace foak
