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

// The two elements of a 32-bit word, and back.
__device__ __forceinline__ float2 word_to_f32(uint32_t w, __nv_bfloat16) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 word_to_f32(uint32_t w, __half) {
    __half2 h;
    __builtin_memcpy(&h, &w, 4);
    return __half22float2(h);
}
__device__ __forceinline__ uint32_t f32_to_word(float lo, float hi, __nv_bfloat16) { return pack_bf16x2(lo, hi); }
__device__ __forceinline__ uint32_t f32_to_word(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t w;
    __builtin_memcpy(&w, &h, 4);
    return w;
}

// VEC consecutive elements, aligned to their size up to 16 bytes (fp32 parameters beside 8 elements of
// 16-bit data take two 16-byte accesses); VEC = 1 needs the element's alignment only.
template <typename T, int VEC> struct alignas(VEC * sizeof(T) > 16 ? 16 : VEC * sizeof(T)) Pack {
    T v[VEC];
    __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
        if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
            uint32_t w[VEC / 2];
            __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 p = word_to_f32(w[i], T());
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = to_f32(v[i]);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[VEC]) {
        if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
            uint32_t w[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) w[i] = f32_to_word(f[2 * i], f[2 * i + 1], T());
            __builtin_memcpy(v, w, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(f[i]);
        }
    }
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
    r.pack(f);
    if constexpr (VEC * sizeof(T) == 16) {
        uint4 u;
        __builtin_memcpy(&u, &r, 16);
        st_stream(p, u);
    } else {
        *reinterpret_cast<Pack<T, VEC> *>(p) = r;
    }
}

// Two fp32 values in a 64-bit register, with one instruction for both.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 f2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(f32x2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
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
