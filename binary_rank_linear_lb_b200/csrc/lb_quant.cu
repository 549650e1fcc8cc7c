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
// is exact (127 s_i w_i not always: above_border).  peak is exact too: the fp32
// products that share the largest value are compared again in 64 bits (unless no
// product rounds).  Rows whose peak or mean square leaves fp32's comfortable range,
// rows of zeros and rows with a NaN or an infinity are computed in 64 bits altogether.
//
// What bounds it: HBM.  A row is read once and kept in registers as v between
// the two halves (peak and mean square, then the codes): rows up to 1024 columns
// by one warp, up to 32768 by one block; wider ones read memory twice.  Codes of
// 32000 x 4096 bf16: 66 to 69 us, 5.7 to 6.0 TB/s (89 to 93% of the copy rate); norm of
// 4096 x 8192 bf16 with residual and sum: 42 to 44 us, 5.4 to 5.6 TB/s (83 to 87%).
// Rows off 16 bytes load each piece from two: 100000 x 777 bf16 105 us, x 776 61 us.
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
    bool q_wide;              // so are the codes of every piece, to their size
    bool inexact;             // s w can need more than fp32's 24 bits
    float eps;
};

// A quotient this near a half-integer is computed again in 64 bits.  v, peak and
// 127 / peak are each off by at most 2^-24 relative in fp32 (the product is not
// rounded before it is compared), together by 3 * 2^-24 * 127 = 2^-15.4 for a
// quotient of at most 127.
constexpr float kBorder = 1.0f / 32768.0f;
// Adding it rounds |f| < 2^22 to a whole number, ties to even, and leaves that in
// the low bits.
constexpr float kRound = 12582912.0f;              // 1.5 * 2^23
// Peaks and mean squares outside these are left to the 64-bit path (squares and
// reciprocals inside them are far from fp32's ends).
constexpr float kLow = 1e-30f, kHigh = 1e30f;

constexpr int kMaxThreads = 1024;

// max(m, |v.x|, |v.y|); NaN if one is.
__device__ __forceinline__ float max_abs(float m, F2 v) {
    const float2 h = halves(v);
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(h.x), "f"(h.y));
    return r;
}

constexpr int64_t kFewElems = (int64_t)1 << 21;    // what the SMs hold at 8 elements a thread

// Bytes m .. m + 15 of the 32 in lo, hi (0 < m < 16, the same for the whole row).
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, int m) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 7; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
    const uint32_t bits = 8u * (uint32_t)(m & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// The piece of VE elements from column i of a row (zeros past its end).  A row
// that does not start on 16 bytes is read in aligned 16-byte pairs that lie inside
// it and shifted; its ends element by element.
template <int DT, bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const typename Elem<DT>::T* row, int i, int cols) {
    using T = typename Elem<DT>::T;
    constexpr int VE = Piece<DT>::VE;
    const T* p = row + i;
    const int m = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15);
    if (i + VE <= cols) {
        if (m == 0) return *reinterpret_cast<const uint4*>(p);
        const int before = m / (int)sizeof(T);     // elements of the pair before the piece
        if (!ALIGNED && i >= before && i - before + 2 * VE <= cols) {
            const uint4* q = reinterpret_cast<const uint4*>(p - before);
            return shifted(q[0], q[1], m);
        }
    }
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (i >= cols) return u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (i + k < cols) e[k] = p[k];
    return u;
}

// Stores it.  Called by whole warps, lanes holding consecutive pieces: where the row
// is not aligned, a lane stores the aligned 16 bytes that end inside its piece (the
// lane before it gives the start), and what no such store covers goes element by element.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_piece(typename Elem<DT>::T* row, int i, int cols, uint4 u) {
    using T = typename Elem<DT>::T;
    constexpr int VE = Piece<DT>::VE;
    T* p = row + i;
    const T* e = reinterpret_cast<const T*>(&u);
    const bool whole = i + VE <= cols;
    int from = 0, to = VE;                         // elements left to store one by one
    if constexpr (ALIGNED) {
        if (whole) {
            *reinterpret_cast<uint4*>(p) = u;
            return;
        }
    } else {
        const int lane = threadIdx.x & 31, m = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        const int head = m ? (16 - m) / (int)sizeof(T) : VE;       // elements up to the next 16 bytes
        const uint4 prev = make_uint4(__shfl_up_sync(0xffffffffu, u.x, 1), __shfl_up_sync(0xffffffffu, u.y, 1),
                                      __shfl_up_sync(0xffffffffu, u.z, 1), __shfl_up_sync(0xffffffffu, u.w, 1));
        const bool next = __shfl_down_sync(0xffffffffu, whole ? 1 : 0, 1) != 0 && lane < 31;
        if (whole && m == 0) {
            *reinterpret_cast<uint4*>(p) = u;
            return;
        }
        if (whole && lane > 0) {                   // the last m bytes of the piece before, then this one's first
            *reinterpret_cast<uint4*>(p - m / (int)sizeof(T)) = shifted(prev, u, 16 - m);
            from = head;
        }
        if (whole && next) to = head;
    }
    if (i < cols)
#pragma unroll
        for (int k = 0; k < VE; ++k)
            if (k >= from && k < to && i + k < cols) p[k] = e[k];
}

__device__ __forceinline__ float weight_at(const void* w, int wt, int i) {
    if (w == nullptr) return 1.0f;
    if (wt == LB_F16) return __half2float(static_cast<const __half*>(w)[i]);
    if (wt == LB_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
    return static_cast<const float*>(w)[i];
}
// The weights of the piece of VE columns from i, as pairs.
template <int VE>
__device__ __forceinline__ void load_weights(const QuantArgs& a, int i, F2 (&v)[VE / 2]) {
    if (a.weight_wide && i + VE <= a.cols) {
        if (a.weight_type == LB_F32) {
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + i + j);
                v[j / 2] = f2(f.x, f.y);
                v[j / 2 + 1] = f2(f.z, f.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.weight) + i + j);
                const uint32_t h[2] = {u.x, u.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = a.weight_type == LB_F16
                                         ? __half22float2(*reinterpret_cast<const __half2*>(&h[k]))
                                         : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h[k]));
                    v[j / 2 + k] = f2(f.x, f.y);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < VE; j += 2)
        v[j / 2] = f2(i + j < a.cols ? weight_at(a.weight, a.weight_type, i + j) : 0.0f,
                      i + j + 1 < a.cols ? weight_at(a.weight, a.weight_type, i + j + 1) : 0.0f);
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

// The code of v where the quotient 127 |v| / peak is within 2^-13 of the border lo + 1/2: lo
// or lo + 1, ties to even, with v's sign.  For the norm of fp32 rows, as products of two
// fp32 have up to 48 bits: 127 v can need 55, rounds in code_d, and a tie may be missed.
// (All other products have 35 bits at most; 127 v is exact, and a quotient that is not on a
// border is at least 2^-44 from it and off by less than 2^-46.)  Here both sides are
// compared as they are: 127 |v| = p + e and (lo + 1/2) peak = p + d, where e, the rest of a
// product, and d, a difference of 42 bits at most, are exact.
__device__ __forceinline__ int above_border(double v, int lo, double peak) {
    const double p = 127.0 * fabs(v), e = fma(127.0, fabs(v), -p), d = fma(lo + 0.5, peak, -p);
    const int k = lo + (e > d || (e == d && (lo & 1)));
    return v < 0.0 ? -k : k;
}

// A row in 64 bits, from memory (its sums already written): every thread
// takes the columns first, first + step, ...
template <int DT, bool WARP, bool EXACT>
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
    if constexpr (EXACT) {
        if (bad || !(peak > 0.0)) {
            for (int i = first; i < a.cols; i += step) q[i] = 0;
            return;
        }
        const double inv = 127.0 / peak;
        for (int i = first; i < a.cols; i += step) {
            const double v = (double)X::get(s[i]) * (double)weight_at(a.weight, a.weight_type, i);
            const double quotient = v * inv;       // (off by less than 2^-45)
            q[i] = (int8_t)__double2int_rn(quotient);
            if (fabs(quotient - rint(quotient)) > 0.5 - 0x1p-40)
                q[i] = (int8_t)above_border(v, (int)fabs(quotient), peak);
        }
    } else {
        for (int i = first; i < a.cols; i += step)
            q[i] = bad || !(peak > 0.0)
                       ? 0
                       : (int8_t)code_d((double)X::get(s[i]), (double)weight_at(a.weight, a.weight_type, i), peak);
    }
}

// The code of column i again, in 64 bits (rare: a quotient that near a border
// comes up once in 16,000, and for v = peak / 2).
template <int DT, bool EXACT>
__device__ __noinline__ void settle_code(const QuantArgs& a, int64_t row, int i, double peak) {
    using X = Elem<DT>;
    const typename X::T* s = a.residual ? static_cast<const typename X::T*>(a.sum) + row * a.lds
                                        : static_cast<const typename X::T*>(a.x) + row * a.ldx;
    if constexpr (EXACT) {
        if (i < a.cols) {                          // (the quotient is within 2^-13 of a border in fp32 too)
            const double v = (double)X::get(s[i]) * (double)weight_at(a.weight, a.weight_type, i);
            a.q[row * a.ldq + i] = (int8_t)above_border(v, (int)(127.0f * fabsf((float)v) / (float)peak), peak);
        }
    } else {
        if (i < a.cols)
            a.q[row * a.ldq + i] =
                (int8_t)code_d((double)X::get(s[i]), (double)weight_at(a.weight, a.weight_type, i), peak);
    }
}

// C pieces of VE elements per thread; a warp per row (8 to a block) or a block
// per row.  The work is as much in the instructions as in the bytes (a 16-bit
// element comes and goes with 3 to 7 bytes), so everything runs on pairs and the
// codes take two pair instructions: v * 127 / peak + kRound holds the code in its
// low byte, and what it left over says how near the border was.  (Where a thread holds 32
// fp32 of a norm off 16 bytes one block an SM is asked for: left to itself the compiler
// makes room for two by 1.4 KB of spills.)
template <int DT, int C, bool ALIGNED, bool WARP, int THREADS, bool NORM>
__global__ void __launch_bounds__(THREADS, NORM && !ALIGNED && !WARP && DT == LB_F32 && C == 8 ? 1 : 0)
quant_rows_kernel(const __grid_constant__ QuantArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int VE = Piece<DT>::VE, P = VE / 2;
    __shared__ double red[WARP ? 1 : 32];
    __shared__ unsigned long long exact_bits[WARP ? 8 : 1];
    const int tr = WARP ? 32 : (int)blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    grid_trigger();
    grid_wait();
    if (WARP && row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    auto at = [&](int c) { return (c * tr + t) * VE; };              // a piece's first column

    uint4 raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = load_piece<DT, ALIGNED>(x, at(c), a.cols);
    // with 8 elements a thread (few rows) the weights are requested with the row
    constexpr bool kEarly = NORM && C * VE == 8;
    F2 we[kEarly ? C : 1][P];
    if constexpr (kEarly)
        if (a.weight)
#pragma unroll
            for (int c = 0; c < C; ++c) load_weights<VE>(a, at(c), we[c]);
    if (NORM && a.residual) {
        const T* r = static_cast<const T*>(a.residual) + row * a.ldr;
        T* sum = static_cast<T*>(a.sum) + row * a.lds;
        uint4 more[C];
#pragma unroll
        for (int c = 0; c < C; ++c) more[c] = load_piece<DT, ALIGNED>(r, at(c), a.cols);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            F2 xv[P], rv[P];
            Piece<DT>::unpack(raw[c], xv);
            Piece<DT>::unpack(more[c], rv);
#pragma unroll
            for (int i = 0; i < P; ++i) xv[i] = add2(xv[i], rv[i]);
            raw[c] = Piece<DT>::pack(xv);
            store_piece<DT, ALIGNED>(sum, at(c), a.cols, raw[c]);
        }
        __syncwarp();                              // (a lane may have stored part of its neighbour's piece)
    }
    // v = s w, the sum of s^2 and the largest |v|.  (Without a norm v is the row
    // itself and is unpacked again for the codes, which frees registers.)
    F2 v[NORM ? C : 1][P], sq = f2(0.0f, 0.0f);
    float top = 0.0f;
    const int slot = WARP ? threadIdx.x >> 5 : 0;
    if (t == 0) exact_bits[slot] = 0;              // (ordered before its use by the barriers below)
#pragma unroll
    for (int c = 0; c < C; ++c) {
        F2 (&vc)[P] = v[NORM ? c : 0];
        Piece<DT>::unpack(raw[c], vc);
        if (NORM) {
#pragma unroll
            for (int i = 0; i < P; ++i) sq = fma2(vc[i], vc[i], sq);
            if (a.weight) {
                F2 w[P];
                if constexpr (!kEarly) load_weights<VE>(a, at(c), w);
#pragma unroll
                for (int i = 0; i < P; ++i) vc[i] = mul2(vc[i], kEarly ? we[c][i] : w[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) top = max_abs(top, vc[i]);
    }
    float ss = halves(sq).x + halves(sq).y;
    // non-negative floats order like their bits, and a NaN comes last
    __syncwarp();
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (!WARP) {
        uint2* part = reinterpret_cast<uint2*>(red);
        const int nw = tr >> 5, lane = t & 31;
        if (lane == 0) part[t >> 5] = make_uint2(__float_as_uint(ss), bits);
        __syncthreads();
        const uint2 mine = lane < nw ? part[lane] : make_uint2(0u, 0u);
        ss = __uint_as_float(mine.x);
        bits = __reduce_max_sync(0xffffffffu, mine.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float peak = __uint_as_float(bits);
    const float ms = ss / (float)a.cols;
    if (!(peak >= kLow && peak <= kHigh) || (NORM && !(ms >= kLow && ms <= kHigh))) {
        quant_row_64<DT, WARP, NORM && DT == LB_F32>(a, row, t, tr, red);
        return;
    }
    // The exact peak: of the products that round to it, the largest in 64 bits.  It
    // is only needed where a code is near a border, so the threads that hold those
    // products leave it in shared memory and it is read after the codes.
    if (NORM && a.inexact) {
        const T* s = a.residual ? static_cast<const T*>(a.sum) + row * a.lds : x;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 h = halves(v[NORM ? c : 0][i]);
                if (fmaxf(fabsf(h.x), fabsf(h.y)) == peak)
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {
                        const int o = at(c) + 2 * i + e;
                        if (o < a.cols)          // (non-negative doubles order like their bits)
                            atomicMax(&exact_bits[slot],
                                      (unsigned long long)__double_as_longlong(fabs(
                                          (double)Elem<DT>::get(s[o]) *
                                          (double)weight_at(a.weight, a.weight_type, o))));
                    }
            }
    }
    if (t == 0) a.scale[row] = NORM ? peak / (127.0f * sqrtf(ms + a.eps)) : peak / 127.0f;
    const float inv = 127.0f / peak;
    const F2 inv2 = f2(inv, inv), round2 = f2(kRound, kRound), back2 = f2(-kRound, -kRound);
    const F2 minus2 = f2(-1.0f, -1.0f);
    int8_t* q = a.q + row * a.ldq;
    // Elements with a code near a border, a bit each.  Where 127 / peak is exact (a peak
    // of 127 * 2^n, common in 16-bit rows, with many values on borders) and so are the
    // products, nothing is in doubt: the rounding above is that of the exact quotient.
    const float limit = !a.inexact && fmaf(inv, peak, -127.0f) == 0.0f ? 1.0f : 0.5f - kBorder;
    uint32_t near = 0;
    static_assert(C * VE <= 32, "a bit for each element");
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = at(c), n = a.cols - i;
        F2 (&vc)[P] = v[NORM ? c : 0];
        if (!NORM) Piece<DT>::unpack(raw[c], vc);
        uint32_t code[VE];
        float rest = 0.0f;                         // the largest distance from a code
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const F2 k = fma2(vc[j], inv2, round2);
            const float2 h = halves(k);
            code[2 * j] = __float_as_uint(h.x);
            code[2 * j + 1] = __float_as_uint(h.y);
            const F2 whole = mul2(add2(k, back2), minus2);
            rest = max_abs(rest, fma2(vc[j], inv2, whole));
        }
        if (a.q_wide && n >= VE) {
            uint32_t w[VE / 4];
#pragma unroll
            for (int e = 0; e < VE; e += 4)
                w[e / 4] = prmt(prmt(code[e], code[e + 1], 0x0040u), prmt(code[e + 2], code[e + 3], 0x0040u), 0x5410u);
            if constexpr (VE == 8) *reinterpret_cast<uint2*>(q + i) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(q + i) = w[0];
        } else if (n > 0) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e < n) q[i + e] = (int8_t)code[e];
        }
        if (rest >= limit)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const F2 whole = mul2(add2(fma2(vc[j], inv2, round2), back2), minus2);
                const float2 h = halves(fma2(vc[j], inv2, whole));
                near |= (fabsf(h.x) >= limit ? 1u : 0u) << (c * VE + 2 * j);
                near |= (fabsf(h.y) >= limit ? 1u : 0u) << (c * VE + 2 * j + 1);
            }
    }
    double exact = (double)peak;
    if (NORM && a.inexact) {
        if constexpr (WARP) __syncwarp();
        else __syncthreads();
        exact = __longlong_as_double((long long)exact_bits[slot]);
    }
    while (near) {
        const int b = __ffs(near) - 1;
        near &= near - 1;
        settle_code<DT, NORM && DT == LB_F32>(a, row, at(b / VE) + b % VE, exact);
    }
}

// Rows of more columns than a block's registers hold: one block per row, in 64
// bits, the row read twice.  Bound by the 64-bit arithmetic and by loads of one
// element: 4096 x 40000 fp32 715 to 730 us, 1.1 TB/s (17% of the copy rate).
template <int DT, bool NORM>
__global__ void __launch_bounds__(256) quant_wide_kernel(const __grid_constant__ QuantArgs a) {
    using X = Elem<DT>;
    __shared__ double red[32];
    const int64_t row = blockIdx.x;
    grid_trigger();
    grid_wait();
    if (a.residual) {
        const typename X::T* x = static_cast<const typename X::T*>(a.x) + row * a.ldx;
        const typename X::T* r = static_cast<const typename X::T*>(a.residual) + row * a.ldr;
        typename X::T* sum = static_cast<typename X::T*>(a.sum) + row * a.lds;
        for (int i = threadIdx.x; i < a.cols; i += 256) sum[i] = X::put(X::get(x[i]) + X::get(r[i]));
    }
    quant_row_64<DT, false, NORM && DT == LB_F32>(a, row, threadIdx.x, 256, red);
}

template <int DT, int C, bool ALIGNED, int THREADS, bool NORM>
cudaError_t launch_block(const QuantArgs& a, cudaStream_t s) {
    constexpr int per_thread = C * Piece<DT>::VE;
    const int threads = ((a.cols + per_thread - 1) / per_thread + 31) / 32 * 32;
    return launch_dense(quant_rows_kernel<DT, C, ALIGNED, false, THREADS, NORM>, (unsigned)a.rows, threads, 0, 1, s, a);
}

// Elements per thread.  Fewer mean more threads, so more of a row in flight and a
// shorter path through it, but more of the work goes into the folds and, past 512
// threads, an SM runs out of registers.  Measured (us, 8 / 16 / 32 elements, with
// fp16 weights and a residual unless "plain"; the choice in brackets):
//   333 x 5120 bf16 [5.5] 6.0 6.9, fp32 [6.6] 7.8 9.6, plain bf16 [3.0] 3.5 3.8;
//   4096 x 4096 bf16 28.7 [25.2] 25.6, fp32 [37.7] 39.1 48.0, plain bf16 17.2 14.2 [12.7];
//   4096 x 8192 bf16 58.0 46.8 [44.5], fp32 73.5 [70.5] 81.1, plain bf16 35.1 27.1 [23.6].
template <int DT, bool ALIGNED, bool NORM>
cudaError_t launch_rows(const QuantArgs& a, cudaStream_t s) {
    constexpr int VE = Piece<DT>::VE;
    constexpr bool kWide = DT == LB_F32;           // 32 elements are 8 pieces
    if (a.cols <= 32 * 32) {                       // a warp per row
        auto kernel = a.cols <= 32 * 8    ? quant_rows_kernel<DT, 8 / VE, ALIGNED, true, 256, NORM>
                      : a.cols <= 32 * 16 ? quant_rows_kernel<DT, 16 / VE, ALIGNED, true, 256, NORM>
                                          : quant_rows_kernel<DT, 32 / VE, ALIGNED, true, 256, NORM>;
        return launch_dense(kernel, (unsigned)((a.rows + 7) / 8), 256, 0, 1, s, a);
    }
    if (a.cols <= kMaxThreads * 8 && (a.rows * a.cols <= kFewElems || (NORM && kWide && a.cols <= 4096)))
        return launch_block<DT, 8 / VE, ALIGNED, kMaxThreads, NORM>(a, s);
    if constexpr (NORM) {
        if (a.cols <= (kWide ? 8192 : 6144)) return launch_block<DT, 16 / VE, ALIGNED, 512, NORM>(a, s);
        if constexpr (kWide)
            if (a.cols <= kMaxThreads * 16) return launch_block<DT, 16 / VE, ALIGNED, kMaxThreads, NORM>(a, s);
    }
    if constexpr (!(NORM && kWide))
        if (a.cols <= 256 * 32) return launch_block<DT, 32 / VE, ALIGNED, 256, NORM>(a, s);
    if (a.cols <= kMaxThreads * 32) return launch_block<DT, 32 / VE, ALIGNED, kMaxThreads, NORM>(a, s);
    return launch_dense(quant_wide_kernel<DT, NORM>, (unsigned)a.rows, 256, 0, 1, s, a);
}

lb_status quant_call(QuantArgs a, int dt, cudaStream_t s) {
    int sms = 0;
    const lb_status st = dense_device(sms);
    if (st != LB_OK) return st;
    const int64_t per16 = 16 / (int64_t)dtype_size(dt);        // elements in 16 bytes
    const bool aligned = is_aligned(a.x, 16) && is_aligned(a.residual, 16) && is_aligned(a.sum, 16) &&
                         (a.rows == 1 || (a.ldx % per16 == 0 && a.ldr % per16 == 0 && a.lds % per16 == 0));
    a.q_wide = is_aligned(a.q, (size_t)per16) && (a.rows == 1 || a.ldq % per16 == 0);
    a.weight_wide = is_aligned(a.weight, 16);
    // products that fp32 holds exactly: two 16-bit factors, or no weight
    a.inexact = a.weight && (dt == LB_F32 || a.weight_type == LB_F32);
    const cudaError_t e = with_dtype(dt, [&](auto d) {
        if (a.norm) return aligned ? launch_rows<d.value, true, true>(a, s) : launch_rows<d.value, false, true>(a, s);
        return aligned ? launch_rows<d.value, true, false>(a, s) : launch_rows<d.value, false, false>(a, s);
    });
    return dense_status(e);
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
