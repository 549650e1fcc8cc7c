// lb_linear_int8: y[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k].
//
// The sum is exact (int32; in <= 131071 keeps it inside, since a product is at
// most 2^14).  y = (fp32(sum) * xs) * ws, rounded to y's type: fp32(sum) rounds
// sums past 2^24, and each factor once, so y is off by at most 3 * 2^-24
// relative before its own rounding.
#include "lb_dense.cuh"

namespace lb {
namespace {

struct Int8Args {
    const int8_t* x;
    const int8_t* w;
    const float* xs;
    const float* ws;
    void* y;
    int64_t ldx, ldw, ldy;
    int M, N, K;
};

// General kernel: any pitch and alignment.  64 x 64 outputs per block, 64
// columns of K at a time through shared memory (bytes loaded one by one, zero
// past the edges), four rows by four columns per thread with __dp4a.
constexpr int kGenTile = 64;
constexpr int kGenPitch = 17;                // words of a staged row (16 used), odd: no bank conflicts

template <int DT>
__global__ void __launch_bounds__(256) int8_general_kernel(const Int8Args a) {
    __shared__ int xt[kGenTile * kGenPitch], wt[kGenTile * kGenPitch];
    const int n_m = (a.M + kGenTile - 1) / kGenTile;
    const int m0 = (int)(blockIdx.x % n_m) * kGenTile, n0 = (int)(blockIdx.x / n_m) * kGenTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 64) {
        for (int i = threadIdx.x; i < kGenTile * 64; i += 256) {
            const int r = i >> 6, c = i & 63, k = k0 + c;
            int8_t xv = 0, wv = 0;
            if (k < a.K && m0 + r < a.M) xv = a.x[(int64_t)(m0 + r) * a.ldx + k];
            if (k < a.K && n0 + r < a.N) wv = a.w[(int64_t)(n0 + r) * a.ldw + k];
            reinterpret_cast<int8_t*>(xt + r * kGenPitch)[c] = xv;
            reinterpret_cast<int8_t*>(wt + r * kGenPitch)[c] = wv;
        }
        __syncthreads();
#pragma unroll 4
        for (int kk = 0; kk < 16; ++kk) {
            int xv[4], wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[i] = xt[(ty + 16 * i) * kGenPitch + kk];
                wv[i] = wt[(tx + 16 * i) * kGenPitch + kk];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
    using Y = Elem<DT>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty + 16 * i;
        if (m >= a.M) continue;
        const float xs = a.xs[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            if (n < a.N)
                static_cast<typename Y::T*>(a.y)[(int64_t)m * a.ldy + n] =
                    Y::put((float)acc[i][j] * xs * a.ws[n]);
        }
    }
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_linear_int8(const int8_t* xq, int64_t ldx, const float* xs, int64_t M,
                                    const int8_t* wq, int64_t ldw, const float* ws, int64_t in,
                                    int64_t out, void* y, lb_dtype y_dtype, int64_t ldy,
                                    void* stream) {
    if (!xq || !xs || !wq || !ws || !y || !dtype_ok(y_dtype)) return LB_ERR_INVALID_ARG;
    if (M <= 0 || in <= 0 || out <= 0 || M > (1 << 24) || out > (1 << 24) || in > 131071)
        return LB_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 32;
    if (ldx < in || ldw < in || ldy < out || ldx > most || ldw > most || ldy > most)
        return LB_ERR_INVALID_ARG;
    if (!is_aligned(xs, 4) || !is_aligned(ws, 4) || !is_aligned(y, dtype_size(y_dtype)))
        return LB_ERR_ALIGNMENT;
    const lb_status st = dense_device_ok();
    if (st != LB_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Int8Args a = {xq, wq, xs, ws, y, ldx, ldw, ldy, (int)M, (int)out, (int)in};
    const int64_t blocks = ((M + kGenTile - 1) / kGenTile) * ((out + kGenTile - 1) / kGenTile);
    if (blocks > 0x7fffffff) return LB_ERR_INVALID_ARG;
    with_dtype(y_dtype, [&](auto d) { int8_general_kernel<d.value><<<(unsigned)blocks, 256, 0, s>>>(a); });
    return cudaGetLastError() == cudaSuccess ? LB_OK : LB_ERR_CUDA;
}
