// Shared by the dense-path operators (lb_quant.cu, lb_int8.cu, lb_logprobs.cu):
// element types, argument helpers.
#pragma once

#include "lb_internal.cuh"

namespace lb {

// The element type of an lb_dtype and its conversions.  Values are computed on
// in fp32; a store rounds once, to nearest even.
template <int DT> struct Elem;
template <> struct Elem<LB_F16> {
    using T = __half;
    static __device__ __forceinline__ float get(T v) { return __half2float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<LB_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<LB_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};

inline bool dtype_ok(int t) { return t == LB_F16 || t == LB_BF16 || t == LB_F32; }
inline size_t dtype_size(int t) { return t == LB_F32 ? 4 : 2; }
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// LB_OK when the current device is an sm_100 part.
inline lb_status dense_device_ok() {
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return LB_ERR_CUDA;
    return major == 10 ? LB_OK : LB_ERR_UNSUPPORTED;
}

// Calls f with the lb_dtype as a compile-time constant.
template <class F>
auto with_dtype(int t, F f) {
    if (t == LB_F16) return f(std::integral_constant<int, LB_F16>{});
    if (t == LB_BF16) return f(std::integral_constant<int, LB_BF16>{});
    return f(std::integral_constant<int, LB_F32>{});
}

}  // namespace lb
