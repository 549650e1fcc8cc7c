// 8-bit rows with scales: lb_quantize_rows and lb_rmsnorm_quantize.
//
// Per row, with s the row as it is stored (x, or x + residual rounded to its
// type), v_i = s_i w_i and peak = max_i |v_i|:
//   q_i = rint(127 v_i / peak),  scale = size * peak / 127,
//   size = 1 / sqrt(mean(s^2) + eps) for the norm, 1 without it,
// so scale * q_i is the normalised row.  The norm's factor is the same for the
// whole row and cancels from q_i: the codes depend on v alone.
//
// Rounding.  Sums, products and quotients are computed in 64 bits (s_i w_i is
// exact there), so the codes are those of the exact quotient.
#include <cmath>

#include "lb_dense.cuh"

namespace lb {
namespace {

struct QuantArgs {
    const void* x;
    const void* residual;     // nullptr: none
    void* sum;                // x + residual (with residual only)
    const void* weight;       // nullptr: ones
    int8_t* q;
    float* scale;
    int64_t rows, ldx, ldr, lds, ldq;
    int cols;
    int norm;                 // 0: no norm (size 1)
    float eps;
};

constexpr int kQuantThreads = 256;
template <class T>
__device__ __forceinline__ T block_fold(T v, T* red, T (*op)(T, T)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kQuantThreads / 32; ++w) v = op(v, red[w]);
    return v;
}
__device__ __forceinline__ double add_d(double a, double b) { return a + b; }
// NaN wins, so that a row holding one has a NaN peak.
__device__ __forceinline__ double max_d(double a, double b) { return a != a ? a : b != b ? b : fmax(a, b); }

// One block per row, the row read three times (the later times from L2).
template <int DT, int WT>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const QuantArgs a) {
    using X = Elem<DT>;
    using W = Elem<WT>;
    using XT = typename X::T;
    using WTt = typename W::T;
    __shared__ double red[kQuantThreads / 32];
    const int64_t row = blockIdx.x;
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    const XT* r = a.residual ? static_cast<const XT*>(a.residual) + row * a.ldr : nullptr;
    XT* sum = a.residual ? static_cast<XT*>(a.sum) + row * a.lds : nullptr;
    const WTt* wt = static_cast<const WTt*>(a.weight);
    double ss = 0.0, peak = 0.0;
    for (int i = threadIdx.x; i < a.cols; i += kQuantThreads) {
        XT sv = x[i];
        if (r) {
            sv = X::put(X::get(sv) + X::get(r[i]));
            sum[i] = sv;
        }
        const double s = (double)X::get(sv);
        const double w = wt ? (double)W::get(wt[i]) : 1.0;
        ss += s * s;
        peak = max_d(peak, fabs(s * w));
    }
    ss = block_fold(ss, red, add_d);
    peak = block_fold(peak, red, max_d);
    const bool bad = !(peak <= 1.7976931348623157e308);
    const double size = a.norm ? 1.0 / sqrt(ss / a.cols + (double)a.eps) : 1.0;
    if (threadIdx.x == 0) a.scale[row] = bad ? NAN : peak > 0.0 ? (float)(peak * size / 127.0) : 0.0f;
    const XT* src = r ? sum : x;
    int8_t* q = a.q + row * a.ldq;
    for (int i = threadIdx.x; i < a.cols; i += kQuantThreads) {
        const float s = X::get(src[i]), w = wt ? W::get(wt[i]) : 1.0f;
        q[i] = bad || !(peak > 0.0) ? 0 : (int8_t)__double2int_rn((double)s * (double)w * 127.0 / peak);
    }
}

lb_status quant_call(const QuantArgs& a, int dt, int wt, cudaStream_t s) {
    const lb_status st = dense_device_ok();
    if (st != LB_OK) return st;
    with_dtype(dt, [&](auto d) {
        with_dtype(wt, [&](auto w) {
            quant_rows_kernel<d.value, w.value><<<(unsigned)a.rows, kQuantThreads, 0, s>>>(a);
        });
    });
    return cudaGetLastError() == cudaSuccess ? LB_OK : LB_ERR_CUDA;
}

bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
    return rows > 0 && cols > 0 && rows <= 0x7fffffff && cols <= (1 << 24) && ld >= cols &&
           ld <= ((int64_t)1 << 40);
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_quantize_rows(const void* x, lb_dtype x_dtype, int64_t rows, int64_t cols,
                                      int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                                      void* stream) {
    if (!x || !q || !scale || !dtype_ok(x_dtype)) return LB_ERR_INVALID_ARG;
    if (!matrix_ok(rows, cols, ldx) || !matrix_ok(rows, cols, ldq)) return LB_ERR_INVALID_ARG;
    if (!is_aligned(x, dtype_size(x_dtype)) || !is_aligned(scale, 4)) return LB_ERR_ALIGNMENT;
    QuantArgs a = {};
    a.x = x; a.q = q; a.scale = scale;
    a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldq = ldq;
    return quant_call(a, x_dtype, LB_F32, static_cast<cudaStream_t>(stream));
}

extern "C" lb_status lb_rmsnorm_quantize(const void* x, lb_dtype x_dtype, int64_t rows,
                                         int64_t cols, int64_t ldx, const void* residual,
                                         int64_t ldr, void* sum, int64_t lds, const void* weight,
                                         lb_dtype weight_dtype, float eps, int8_t* q, int64_t ldq,
                                         float* scale, void* stream) {
    if (!x || !q || !scale || !dtype_ok(x_dtype)) return LB_ERR_INVALID_ARG;
    if (weight && !dtype_ok(weight_dtype)) return LB_ERR_INVALID_ARG;
    if ((residual != nullptr) != (sum != nullptr)) return LB_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return LB_ERR_INVALID_ARG;
    if (!matrix_ok(rows, cols, ldx) || !matrix_ok(rows, cols, ldq)) return LB_ERR_INVALID_ARG;
    if (residual && (!matrix_ok(rows, cols, ldr) || !matrix_ok(rows, cols, lds)))
        return LB_ERR_INVALID_ARG;
    const size_t e = dtype_size(x_dtype);
    if (!is_aligned(x, e) || !is_aligned(scale, 4) || !is_aligned(residual, e) ||
        !is_aligned(sum, e) || (weight && !is_aligned(weight, dtype_size(weight_dtype))))
        return LB_ERR_ALIGNMENT;
    QuantArgs a = {};
    a.x = x; a.residual = residual; a.sum = sum; a.weight = weight; a.q = q; a.scale = scale;
    a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldq = ldq;
    a.norm = 1; a.eps = eps;
    return quant_call(a, x_dtype, weight ? weight_dtype : LB_F32, static_cast<cudaStream_t>(stream));
}
