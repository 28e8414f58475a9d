// rows_common.cuh -- loads, stores and reductions shared by the row-local operators
// (kernels_qknorm.cu, kernels_embed.cu, kernels_distill.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "rsa_internal.h"
#include "sm100_ptx.cuh"

namespace rsa {
namespace rows {

// N elements of T moved by one access: 16 bytes on aligned rows, one element otherwise.
template <typename T, int N>
struct Pack {
    static_assert(N * sizeof(T) == 16 || N == 1, "a 16-byte vector or one element");
    using Raw = typename std::conditional<N == 1, T, uint4>::type;
    Raw raw;

    __device__ __forceinline__ static Pack load(const T *p) {
        Pack v;
        v.raw = *reinterpret_cast<const Raw *>(p);
        return v;
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Raw *>(p) = raw; }
    __device__ __forceinline__ static Pack zero() {
        Pack v;
        if constexpr (N == 1)
            v.raw = T(0.f);
        else
            v.raw = make_uint4(0u, 0u, 0u, 0u);
        return v;
    }
    __device__ __forceinline__ void to(float (&f)[N]) const {
        if constexpr (N == 1) {
            f[0] = static_cast<float>(raw);
        } else if constexpr (sizeof(T) == 2) {
            // bf16 is the upper half of the fp32 number
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            f[0] = __uint_as_float(raw.x), f[1] = __uint_as_float(raw.y);
            f[2] = __uint_as_float(raw.z), f[3] = __uint_as_float(raw.w);
        }
    }
    // The same as pairs of neighbours, for the packed operations.
    __device__ __forceinline__ void to(float2 (&f)[N > 1 ? N / 2 : 1]) const {
        static_assert(N > 1, "a vector");
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
            f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
        }
    }
    __device__ __forceinline__ static Pack from(const float2 (&f)[N > 1 ? N / 2 : 1]) {
        static_assert(N > 1, "a vector");
        Pack v;
        if constexpr (sizeof(T) == 2)
            v.raw = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                               pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
        else
            v.raw = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                               __float_as_uint(f[1].x), __float_as_uint(f[1].y));
        return v;
    }
    __device__ __forceinline__ static Pack from(const float (&f)[N]) {
        Pack v;
        if constexpr (N == 1) {
            v.raw = T(f[0]);  // round to nearest even
        } else if constexpr (sizeof(T) == 2) {
            v.raw = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else {
            v.raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                               __float_as_uint(f[3]));
        }
        return v;
    }
};

// Two fp32 operations in one instruction (sm_100's packed fp32 forms), each rounded by itself.
__device__ __forceinline__ unsigned long long bits2(float2 v) {
    return *reinterpret_cast<unsigned long long *>(&v);
}
__device__ __forceinline__ float2 float2_of(unsigned long long b) {
    return *reinterpret_cast<float2 *>(&b);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 16 bytes global -> shared without a register, ordered by commit / wait groups of the thread.
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Element i of an index array of int32 or int64.
__device__ __forceinline__ long long index_at(const void *p, int is64, long long i) {
    return is64 ? static_cast<const long long *>(p)[i]
                : static_cast<long long>(static_cast<const int *>(p)[i]);
}

}  // namespace rows
}  // namespace rsa
