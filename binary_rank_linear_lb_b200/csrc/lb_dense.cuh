// Shared by the dense-path operators (lb_quant.cu, lb_int8.cu, lb_logprobs.cu):
// element types, pair arithmetic, argument helpers.
#pragma once

#include <atomic>
#include <type_traits>

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

// Two fp32 at a time: sm_100 issues one instruction for both.
struct F2 { unsigned long long u; };
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v.u));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return r;
}

// The VE elements of a 16-byte piece as pairs, and back.
template <int DT> struct Piece;
template <> struct Piece<LB_F32> {
    static constexpr int VE = 4;
    static __device__ __forceinline__ void unpack(uint4 u, F2 (&v)[2]) {
        v[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
        v[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&v)[2]) {
        const float2 a = halves(v[0]), b = halves(v[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
};
template <> struct Piece<LB_BF16> {
    static constexpr int VE = 8;
    static __device__ __forceinline__ void unpack(uint4 u, F2 (&v)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&v)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 h = halves(v[i]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(h.x, h.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Piece<LB_F16> {
    static constexpr int VE = 8;
    static __device__ __forceinline__ void unpack(uint4 u, F2 (&v)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[i] = f2(f.x, f.y);
        }
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&v)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 h = halves(v[i]);
            const __half2 b = __floats2half2_rn(h.x, h.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

inline bool dtype_ok(int t) { return t == LB_F16 || t == LB_BF16 || t == LB_F32; }
inline size_t dtype_size(int t) { return t == LB_F32 ? 4 : 2; }
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The status of a call whose last runtime call returned e.  An error is reported here,
// so it is taken back from the runtime: other entry points ask that for their own.
inline lb_status dense_status(cudaError_t e) {
    if (e == cudaSuccess) return LB_OK;
    (void)cudaGetLastError();
    return LB_ERR_CUDA;
}

// LB_OK when the current device is an sm_100 part; its SM count.  (Asked once per
// device: two runtime calls are a tenth of a small call's time on the host.)
inline lb_status dense_device(int& sms) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];       // 0: not asked yet, -1: another part, else its SMs
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kDevices) return e == cudaSuccess ? LB_ERR_CUDA : dense_status(e);
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        int major = 0;
        cudaError_t a = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (a == cudaSuccess) a = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (a != cudaSuccess) return dense_status(a);
        if (major != 10) sms = -1;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    return sms > 0 ? LB_OK : LB_ERR_UNSUPPORTED;
}

// Programmatic dependent launch.  The kernels of the dense path follow one another
// on a stream; each lets the next one start while it still runs (grid_trigger),
// and touches global memory only after everything before it has completed and is
// visible (every thread calls grid_wait before its first access), so only launch
// latency and set-up overlap.  What a kernel reads may thus be written while it
// already runs, so it is read with ordinary loads, none through the read-only path.  333 x 5120 -> 13824 called back to back: 30.8 -> 29.0
// us; one token, 4096 -> 32000: 24.4 -> 22.7 us.
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches with that attribute; cluster: CTAs of a cluster (1: none).
template <class... P, class... A>
cudaError_t launch_dense(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t s, const A&... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Calls f with the lb_dtype as a compile-time constant.
template <class F>
auto with_dtype(int t, F f) {
    if (t == LB_F16) return f(std::integral_constant<int, LB_F16>{});
    if (t == LB_BF16) return f(std::integral_constant<int, LB_BF16>{});
    return f(std::integral_constant<int, LB_F32>{});
}

}  // namespace lb
