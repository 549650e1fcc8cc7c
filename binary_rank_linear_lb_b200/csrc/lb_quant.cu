// 8-bit rows with scales: lb_quantize_rows and lb_rmsnorm_quantize.
//
// Per row, with s the row as it is stored (x, or x + residual rounded to its
// type), v_i = s_i w_i and peak = max_i |v_i|:
//   q_i = rint(127 v_i / peak),  scale = size * peak / 127,
//   size = 1 / sqrt(mean(s^2) + eps) for the norm, 1 without it,
// so scale * q_i is the normalised row.  The norm's factor is the same for the
// whole row and cancels from q_i: the codes depend on v alone.
//
// Rounding.  The codes are those of the exact quotient.  It is computed in fp32,
// where its error (see kBorder) can move it over the border between two codes,
// so quotients that near a border are computed again in 64 bits, where s_i w_i
// is exact.  peak is exact too: the fp32 products that share the largest value
// are compared again in 64 bits (unless no product rounds).  Rows whose peak or
// mean square leaves fp32's comfortable range, rows of zeros and rows with a
// NaN or an infinity are computed in 64 bits altogether.
//
// What bounds it: HBM.  A row is read once and kept in registers as v between
// the two halves (peak and mean square, then the codes): rows up to 1024 columns
// by one warp, up to 32768 by one block; wider ones read memory twice.
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
    int weight_type;          // lb_dtype of weight
    bool weight_wide;         // weight is 16-byte aligned
    bool inexact;             // s w can need more than fp32's 24 bits
    float eps;
};

// A quotient this near a half-integer is computed again in 64 bits.  In fp32 v,
// peak, 127 / peak and their product are each off by at most 2^-24 relative,
// together by 4 * 2^-24 * 127 = 2^-15.01 for a quotient of at most 127.
constexpr float kBorder = 1.0f / 16384.0f;
// Peaks and mean squares outside these are left to the 64-bit path (squares and
// reciprocals inside them are far from fp32's ends).
constexpr float kLow = 1e-30f, kHigh = 1e30f;

constexpr int kMaxThreads = 1024;
// With this many rows or fewer a row takes four times the threads (8 elements each
// instead of 32): its latency is what the call waits for.
constexpr int64_t kFewRows = 148;

// v[VE] = the VE elements at p, `n` of them inside the row (the rest 0).
template <int DT, int VE, bool VEC>
__device__ __forceinline__ void load_row(const typename Elem<DT>::T* p, int n, int stride, float (&v)[VE]) {
    using X = Elem<DT>;
    if constexpr (VEC) {
        if (n >= VE) {
            static_assert(VE * sizeof(typename X::T) == 16, "one 16-byte piece");
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const typename X::T* e = reinterpret_cast<const typename X::T*>(&u);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = X::get(e[i]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = i * (VEC ? 1 : stride) < n ? X::get(p[VEC ? i : i * stride]) : 0.0f;
}
template <int DT, int VE, bool VEC>
__device__ __forceinline__ void store_row(typename Elem<DT>::T* p, int n, int stride, const float (&v)[VE]) {
    using X = Elem<DT>;
    if constexpr (VEC) {
        if (n >= VE) {
            uint4 u;
            typename X::T* e = reinterpret_cast<typename X::T*>(&u);
#pragma unroll
            for (int i = 0; i < VE; ++i) e[i] = X::put(v[i]);
            *reinterpret_cast<uint4*>(p) = u;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i)
        if (i * (VEC ? 1 : stride) < n) p[VEC ? i : i * stride] = X::put(v[i]);
}

__device__ __forceinline__ float weight_at(const void* w, int wt, int i) {
    if (w == nullptr) return 1.0f;
    if (wt == LB_F16) return __half2float(static_cast<const __half*>(w)[i]);
    if (wt == LB_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
    return static_cast<const float*>(w)[i];
}
// The VE weights from column i (VEC: consecutive and 16-byte aligned pieces).
template <int VE, bool VEC>
__device__ __forceinline__ void load_weights(const void* w, int wt, int i, int n, int stride, bool wide,
                                             float (&v)[VE]) {
    if (VEC && wide && n >= VE) {
        if (wt == LB_F32) {
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + i + j));
                v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + i + j));
                const uint32_t h[2] = {u.x, u.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = wt == LB_F16
                                         ? __half22float2(*reinterpret_cast<const __half2*>(&h[k]))
                                         : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h[k]));
                    v[j + 2 * k] = f.x;
                    v[j + 2 * k + 1] = f.y;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        const int o = VEC ? j : j * stride;
        v[j] = o < n ? weight_at(w, wt, i + o) : 0.0f;
    }
}

// Folds over the threads of a row: a warp (red unused) or the block.
template <bool WARP, class T, class Op>
__device__ __forceinline__ T row_fold(T v, T none, T* red, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (!WARP) {
        const int nw = (int)blockDim.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();                           // red may still be read from the fold before
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < nw ? red[lane] : none;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    return v;
}
__device__ __forceinline__ double add_d(double a, double b) { return a + b; }
// NaN wins, so that a row holding one has a NaN peak.
__device__ __forceinline__ double max_d(double a, double b) { return a != a ? a : b != b ? b : fmax(a, b); }

__device__ __forceinline__ int code_d(double s, double w, double peak) {
    return __double2int_rn(s * w * 127.0 / peak);
}

// A row in 64 bits, from memory (its sums already written): every thread
// takes the columns first, first + step, ...
template <int DT, bool WARP>
__device__ __noinline__ void quant_row_64(const QuantArgs& a, int64_t row, int first, int step, double* red) {
    using X = Elem<DT>;
    const typename X::T* s = a.residual ? static_cast<const typename X::T*>(a.sum) + row * a.lds
                                        : static_cast<const typename X::T*>(a.x) + row * a.ldx;
    if constexpr (!WARP) __syncthreads();          // the row's sums were written by other threads
    else __syncwarp();
    double ss = 0.0, peak = 0.0;
    for (int i = first; i < a.cols; i += step) {
        const double v = (double)X::get(s[i]);
        ss += v * v;
        peak = max_d(peak, fabs(v * (double)weight_at(a.weight, a.weight_type, i)));
    }
    ss = row_fold<WARP>(ss, 0.0, red, add_d);
    peak = row_fold<WARP>(peak, 0.0, red, max_d);
    const bool bad = !(peak <= 1.7976931348623157e308);
    const double size = a.norm ? 1.0 / sqrt(ss / a.cols + (double)a.eps) : 1.0;
    if (first == 0) a.scale[row] = bad ? NAN : peak > 0.0 ? (float)(peak * size / 127.0) : 0.0f;
    int8_t* q = a.q + row * a.ldq;
    for (int i = first; i < a.cols; i += step)
        q[i] = bad || !(peak > 0.0)
                   ? 0
                   : (int8_t)code_d((double)X::get(s[i]), (double)weight_at(a.weight, a.weight_type, i), peak);
}

// C pieces of VE elements per thread.  VEC: a piece is 16 consecutive bytes;
// otherwise (pointers or pitches that are not multiples of 16) its elements are
// the row's threads apart, so that a warp still reads consecutive ones.
template <int DT, int C, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : kMaxThreads) quant_rows_kernel(const __grid_constant__ QuantArgs a) {
    using X = Elem<DT>;
    using T = typename X::T;
    constexpr int VE = 16 / (int)sizeof(T);
    __shared__ double red[WARP ? 1 : 32];
    const int tr = WARP ? 32 : (int)blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* sum = a.residual ? static_cast<T*>(a.sum) + row * a.lds : nullptr;
    const int estep = VEC ? 1 : tr;                // columns between a piece's elements
    auto at = [&](int c) { return VEC ? (c * tr + t) * VE : c * tr * VE + t; };   // a piece's first column

    // s, its squares, v = s w and the largest |v| (as bits: a NaN beats infinity)
    float v[C][VE];
    float ss = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = at(c), n = a.cols - i;
        if (n > 0) load_row<DT, VE, VEC>(x + i, n, estep, v[c]);
        else
#pragma unroll
            for (int e = 0; e < VE; ++e) v[c][e] = 0.0f;
    }
    if (r) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = at(c), n = a.cols - i;
            if (n <= 0) continue;
            float rv[VE];
            load_row<DT, VE, VEC>(r + i, n, estep, rv);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[c][e] = X::get(X::put(v[c][e] + rv[e]));
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = at(c), n = a.cols - i;
            if (n > 0) store_row<DT, VE, VEC>(sum + i, n, estep, v[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = at(c), n = a.cols - i;
        if (a.norm)
#pragma unroll
            for (int e = 0; e < VE; ++e) ss = fmaf(v[c][e], v[c][e], ss);
        if (a.weight && n > 0) {
            float w[VE];
            load_weights<VE, VEC>(a.weight, a.weight_type, i, n, estep, a.weight_wide, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[c][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) top = max(top, __float_as_uint(v[c][e]) & 0x7fffffffu);
    }
    // (the folds' scratch: one 8-byte word per warp)
    struct Pair { float ss; uint32_t top; };
    top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (!WARP) {
        Pair* pr = reinterpret_cast<Pair*>(red);
        const int nw = tr >> 5, lane = t & 31;
        if (lane == 0) pr[t >> 5] = Pair{ss, top};
        __syncthreads();
        const Pair mine = lane < nw ? pr[lane] : Pair{0.0f, 0u};
        ss = mine.ss;
        top = __reduce_max_sync(0xffffffffu, mine.top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float peak = __uint_as_float(top);
    const float ms = ss / (float)a.cols;
    if (!(peak >= kLow && peak <= kHigh) || (a.norm && !(ms >= kLow && ms <= kHigh))) {
        quant_row_64<DT, WARP>(a, row, t, tr, red);
        return;
    }
    // the exact peak: of the products that round to it, the largest in 64 bits
    const T* src = r ? sum : x;
    double exact = (double)peak;
    if (a.inexact) {
        exact = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (fabsf(v[c][e]) == peak) {
                    const int i = at(c) + e * estep;
                    exact = fmax(exact, fabs((double)X::get(src[i]) * (double)weight_at(a.weight, a.weight_type, i)));
                }
        exact = row_fold<WARP>(exact, 0.0, red, max_d);
    }
    if (t == 0) a.scale[row] = a.norm ? peak / (127.0f * sqrtf(ms + a.eps)) : peak / 127.0f;
    const float inv = 127.0f / peak;
    int8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = at(c), n = a.cols - i;
        int8_t code[VE];
        bool near = false;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float f = v[c][e] * inv, k = rintf(f);
            near |= fabsf(f - k) >= 0.5f - kBorder;
            code[e] = (int8_t)__float2int_rn(k);
        }
        if (near)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float f = v[c][e] * inv;
                const int o = i + e * estep;
                if (fabsf(f - rintf(f)) >= 0.5f - kBorder && o < a.cols)
                    code[e] = (int8_t)code_d((double)X::get(src[o]), (double)weight_at(a.weight, a.weight_type, o), exact);
            }
        if (n <= 0) continue;
        if (VEC && n >= VE) {
            uint32_t w[VE / 4];
#pragma unroll
            for (int e = 0; e < VE; e += 4)
                w[e / 4] = (uint32_t)(uint8_t)code[e] | (uint32_t)(uint8_t)code[e + 1] << 8 |
                           (uint32_t)(uint8_t)code[e + 2] << 16 | (uint32_t)(uint8_t)code[e + 3] << 24;
            if constexpr (VE == 8) *reinterpret_cast<uint2*>(q + i) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(q + i) = w[0];
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e * estep < n) q[i + e * estep] = code[e];
        }
    }
}

// Rows of more columns than a block's registers hold: one block per row, in 64
// bits, the row read twice.
template <int DT>
__global__ void __launch_bounds__(256) quant_wide_kernel(const __grid_constant__ QuantArgs a) {
    using X = Elem<DT>;
    __shared__ double red[32];
    const int64_t row = blockIdx.x;
    if (a.residual) {
        const typename X::T* x = static_cast<const typename X::T*>(a.x) + row * a.ldx;
        const typename X::T* r = static_cast<const typename X::T*>(a.residual) + row * a.ldr;
        typename X::T* sum = static_cast<typename X::T*>(a.sum) + row * a.lds;
        for (int i = threadIdx.x; i < a.cols; i += 256) sum[i] = X::put(X::get(x[i]) + X::get(r[i]));
    }
    quant_row_64<DT, false>(a, row, threadIdx.x, 256, red);
}

template <int DT, int C, bool VEC>
void launch_block(const QuantArgs& a, int per_piece, cudaStream_t s) {
    const int threads = ((a.cols + C * per_piece - 1) / (C * per_piece) + 31) / 32 * 32;
    quant_rows_kernel<DT, C, VEC, false><<<(unsigned)a.rows, threads, 0, s>>>(a);
}

template <int DT, bool VEC>
void launch_rows(const QuantArgs& a, cudaStream_t s) {
    constexpr int VE = 16 / (int)sizeof(typename Elem<DT>::T);
    constexpr int kFull = 32 / VE;                 // pieces of 32 elements
    constexpr int kFew = 8 / VE;                   // pieces of 8 elements
    if (a.cols <= 32 * 32) {
        const unsigned blocks = (unsigned)((a.rows + 7) / 8);
        if (a.cols <= 32 * 8) quant_rows_kernel<DT, kFew, VEC, true><<<blocks, 256, 0, s>>>(a);
        else quant_rows_kernel<DT, kFull, VEC, true><<<blocks, 256, 0, s>>>(a);
    } else if (a.cols <= kMaxThreads * 8 && a.rows <= kFewRows) {
        launch_block<DT, kFew, VEC>(a, VE, s);
    } else if (a.cols <= kMaxThreads * 32) {
        launch_block<DT, kFull, VEC>(a, VE, s);
    } else {
        quant_wide_kernel<DT><<<(unsigned)a.rows, 256, 0, s>>>(a);
    }
}

lb_status quant_call(QuantArgs a, int dt, cudaStream_t s) {
    const lb_status st = dense_device_ok();
    if (st != LB_OK) return st;
    const int64_t per16 = 16 / (int64_t)dtype_size(dt);        // elements in 16 bytes
    const bool vec = is_aligned(a.x, 16) && is_aligned(a.residual, 16) && is_aligned(a.sum, 16) &&
                     is_aligned(a.q, (size_t)per16) &&
                     (a.rows == 1 || (a.ldx % per16 == 0 && a.ldr % per16 == 0 && a.lds % per16 == 0 &&
                                      a.ldq % per16 == 0));
    a.weight_wide = is_aligned(a.weight, 16);
    // products that fp32 holds exactly: two 16-bit factors, or no weight
    a.inexact = a.weight && (dt == LB_F32 || a.weight_type == LB_F32);
    with_dtype(dt, [&](auto d) {
        if (vec) launch_rows<d.value, true>(a, s);
        else launch_rows<d.value, false>(a, s);
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
    return quant_call(a, x_dtype, static_cast<cudaStream_t>(stream));
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
    a.norm = 1; a.eps = eps; a.weight_type = weight_dtype;
    return quant_call(a, x_dtype, static_cast<cudaStream_t>(stream));
}
