// ep_types.cuh -- element types of the norm and router kernels (bf16, fp16, fp32): vectors of
// VEC elements moved as one access and widened to fp32.
#pragma once

#include <cuda_fp16.h>

#include "ep_common.cuh"

namespace ep {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// One rounding (to nearest even) from the fp32 the kernels compute in.
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

// VEC consecutive elements.  VEC * sizeof(T) is 16 (or 32, for fp32 parameters beside 16-bit
// data: two 16-byte accesses), or VEC is 1 and the address has the element's alignment only.
template <typename T, int VEC> struct alignas(VEC == 1 ? sizeof(T) : 16) Pack {
    T v[VEC];
    __device__ __forceinline__ float f(int i) const { return to_f32(v[i]); }
};

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> ld_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
// Read once: the streaming policy.
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> ld_pack_stream(const T *p) {
    if constexpr (VEC * sizeof(T) == 16) {
        const uint4 u = ld_stream(p);
        Pack<T, VEC> r;
        __builtin_memcpy(&r, &u, 16);
        return r;
    } else {
        return ld_pack<T, VEC>(p);
    }
}
template <typename T, int VEC> __device__ __forceinline__ void st_pack_stream(T *p, const float (&f)[VEC]) {
    Pack<T, VEC> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = from_f32<T>(f[i]);
    if constexpr (VEC * sizeof(T) == 16) {
        uint4 u;
        __builtin_memcpy(&u, &r, 16);
        st_stream(p, u);
    } else {
        *reinterpret_cast<Pack<T, VEC> *>(p) = r;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

}  // namespace ep
