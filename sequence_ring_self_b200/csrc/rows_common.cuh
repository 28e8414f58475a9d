// rows_common.cuh -- loads, stores and reductions shared by the row-local operators
// (kernels_qknorm.cu, kernels_embed.cu, kernels_distill.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// Element i of an index array of int32 or int64.
__device__ __forceinline__ long long index_at(const void *p, int is64, long long i) {
    return is64 ? static_cast<const long long *>(p)[i]
                : static_cast<long long>(static_cast<const int *>(p)[i]);
}

}  // namespace rows
}  // namespace rsa
