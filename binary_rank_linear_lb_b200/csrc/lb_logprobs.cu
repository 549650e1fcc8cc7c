// lb_token_logprobs: per row x of logits, with m = max x and S = sum e^(x - m),
//   log p_i = (x_i - m) - log S,
//   entropy = -sum p_i log p_i = log S - sum e^(x - m) (x - m) / S,
// the log probabilities of the given tokens and of the `top` largest logits.
// Both terms of the entropy are >= 0, so nothing cancels.
//
// One pass.  Every thread keeps the running maximum, S and the entropy's sum of
// its 16-byte pieces (rescaled when the maximum grows, which after the first
// batches is rare), in powers of two: t = (x - m) log2 e, S = sum 2^t,
// A = sum 2^t t.  The threads' triples are folded at the end.  What bounds it:
// HBM for fp32, the exponentials (16 a clock and SM) and the instructions around
// them (about 5 an element) close behind for 16-bit logits.  4096 x 32000, top 5: fp32
// 98 to 103 us, 5.1 to 5.3 TB/s (79 to 83% of the copy rate); bf16 67 us, 3.9 TB/s (55
// us without alternatives: those cost a second look at some pieces and the ranking).
//
// The alternatives need no second pass either: the threads' maxima bound them.
// If `top` of the maxima of 64 groups of threads are >= T, the alternatives are
// among the logits >= T, and only threads whose maximum is >= T hold any: those
// few pieces are read again (from L2).  T is found by bisection over the groups'
// maxima, the candidates are ranked by counting.  Where many logits equal T (a mask that leaves
// few) only the first of those are taken; rows where too many lie above it, or
// with a NaN, take `top` rounds of a maximum instead.
//
// With few rows a row is split over a cluster of CTAs; the first one folds the
// others' results through distributed shared memory.
#include <cmath>

#include "lb_dense.cuh"

namespace lb {
namespace {

constexpr int kSplitThreads = 256;           // of each CTA of a split row
constexpr int kMaxTop = 32;
constexpr int kGroups = 64;                  // groups of threads whose maxima bound the alternatives
constexpr int kCandidates = 1024;            // logits >= T kept at most
constexpr int kLpCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// t below this is as good as -inf (2^t is 0), and unlike it can be multiplied by 0.
constexpr float kTiny = -200.0f;

struct LogprobArgs {
    const void* x;
    const int64_t* tokens;
    float* logprob;
    float* entropy;
    int64_t* top_id;
    float* top_logprob;
    int64_t ld;
    int vocab, top;
};

// Order of the alternatives as an unsigned key: larger logit first, NaN before
// everything, -0 equal to +0.  Key 0 is below every logit; 0xffffffff is left free, so
// that every entry (entry_of) is below ~0, where the rounds of a maximum start.
constexpr uint32_t kNanKey = 0xfffffffeu;           // (+inf: 0xff800000)
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return kNanKey;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == kNanKey ? NAN : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// Key and index as one number: larger is earlier (equal keys by rising index).
__device__ __forceinline__ unsigned long long entry_of(uint32_t key, int i) {
    return (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int entry_index(unsigned long long e) { return (int)(0xffffffffu - (uint32_t)e); }

__device__ __forceinline__ float exp2_fast(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
__device__ __forceinline__ float max3_nan(float a, F2 v) {
    const float2 h = halves(v);
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(h.x), "f"(h.y));
    return r;
}

// Running maximum and sums of a thread.
struct Stat {
    float m = -INFINITY, shift = 0.0f;             // shift: m, or 0 while m = -inf
    F2 S = {0ull}, A = {0ull};
    bool nan = false;

    template <int P>
    __device__ __forceinline__ void take(const F2 (&x)[P]) {
        float top = m;
#pragma unroll
        for (int i = 0; i < P; ++i) top = max3_nan(top, x[i]);
        if (!(top <= m)) {
            if (top != top) {
                nan = true;
            } else {
                if (m > -INFINITY) {
                    const float dt = fmaxf((m - top) * kLog2e, kTiny), c = exp2_fast(dt);
                    A = mul2(f2(c, c), fma2(S, f2(dt, dt), A));
                    S = mul2(f2(c, c), S);
                }
                m = shift = top;
            }
        }
        const F2 back = f2(-shift, -shift), l2e = f2(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 t = halves(mul2(add2(x[i], back), l2e));
            t.x = fmaxf(t.x, kTiny);
            t.y = fmaxf(t.y, kTiny);
            const F2 e = f2(exp2_fast(t.x), exp2_fast(t.y));
            S = add2(S, e);
            A = fma2(e, f2(t.x, t.y), A);
        }
    }
};

// Entries of cand[0 .. n) that come before `mine`.
__device__ __forceinline__ int rank_of(unsigned long long mine, const unsigned long long* cand, int n) {
    int before = 0, o = 0;
#pragma unroll 8
    for (; o + 1 < n; o += 2) {
        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cand + o);
        before += (c.x > mine) + (c.y > mine);
    }
    return o < n ? before + (cand[o] > mine) : before;
}

// The 32 largest of two falling lists of 32, in order: u holds the first, v the
// second from its end (their larger elements, lane by lane, are bitonic).
__device__ __forceinline__ unsigned long long merge_sorted(unsigned long long u, unsigned long long v) {
    unsigned long long x = u > v ? u : v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, x, o);
        x = (threadIdx.x & o) ? (x < y ? x : y) : (x > y ? x : y);
    }
    return x;
}

// What a CTA knows of its part of a row.
struct LpPart {
    float m, S, A;
    int nan;
    unsigned long long list[kMaxTop];              // its alternatives, in order (0: none left)
};

__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
    uint32_t p;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    return p;
}
__device__ __forceinline__ uint32_t ld_peer32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_peer64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A CTA per row, or `parts` CTAs (a cluster).  A row is read as the 16-byte
// pieces of memory that it touches; the first and the last may lie partly
// outside it and are read element by element.
template <int DT, bool SPLIT, int kLpThreads>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const __grid_constant__ LogprobArgs a, int parts) {
    using X = Elem<DT>;
    using T = typename X::T;
    constexpr int VE = Piece<DT>::VE, kLpWarps = kLpThreads / 32;
    static_assert(!SPLIT || kLpCluster / 2 <= kLpWarps - 1, "a warp merges two lists, the last folds the sums");
    constexpr int kBatch = 16 / VE;                // pieces of a batch: 16 logits
    __shared__ float fred[2][kLpWarps];
    __shared__ __align__(8) uint32_t group[kGroups];
    __shared__ int n_cand;
    __shared__ __align__(16) unsigned long long cand[kCandidates];
    __shared__ LpPart part;
    constexpr int kGroup = kLpThreads / kGroups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = SPLIT ? (int)(blockIdx.x % parts) : 0;
    const int64_t row = SPLIT ? blockIdx.x / parts : blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld;
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15) / (int)sizeof(T);
    const int n_pieces = (shift + a.vocab + VE - 1) / VE;
    const int p0 = SPLIT ? (int)((int64_t)n_pieces * rank / parts) : 0;
    const int p1 = SPLIT ? (int)((int64_t)n_pieces * (rank + 1) / parts) : n_pieces;

    grid_trigger();
    grid_wait();
    // the given token's logit is requested first
    int64_t tok = -1;
    float tok_x = 0.0f;
    if (threadIdx.x == 0 && rank == 0 && a.tokens) {
        tok = a.tokens[row];
        if (tok >= 0 && tok < a.vocab) tok_x = X::get(x[tok]);
    }
    if (threadIdx.x == 0) n_cand = 0;

    auto load = [&](int j) {
        const int i = j * VE - shift;
        if (i >= 0 && i + VE <= a.vocab && j < p1) return *reinterpret_cast<const uint4*>(x + i);
        const float none = -INFINITY;
        uint4 u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int k = 0; k < VE; ++k) e[k] = j < p1 && i + k >= 0 && i + k < a.vocab ? x[i + k] : X::put(none);
        return u;
    };

    // This thread's pieces are p0 + threadIdx.x + k * kLpThreads.  Those of a first
    // step that holds the row's partial first piece, and of the last batch, are
    // checked one by one; the batches between are whole for every thread.
    Stat st;
    int k = 0;
    auto step = [&] {
        const int j = p0 + (int)threadIdx.x + k * kLpThreads;
        if (j < p1) {
            F2 v[VE / 2];
            Piece<DT>::unpack(load(j), v);
            st.take(v);
        }
        ++k;
    };
    if (shift > 0 && p0 == 0) step();
    const int whole = min(p1, (shift + a.vocab) / VE);       // pieces below it end inside the row
    int batches = (whole - p0 - k * kLpThreads) / (kBatch * kLpThreads);
    if (batches > 0) {
        const uint4* p = reinterpret_cast<const uint4*>(x - shift) + p0 + threadIdx.x + k * kLpThreads;
        k += batches * kBatch;
        uint4 raw[kBatch];                         // the next batch is requested before one is taken
#pragma unroll
        for (int b = 0; b < kBatch; ++b) raw[b] = p[b * kLpThreads];
        while (true) {
            F2 v[8];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                F2 (&vb)[VE / 2] = *reinterpret_cast<F2 (*)[VE / 2]>(&v[b * VE / 2]);
                Piece<DT>::unpack(raw[b], vb);
            }
            p += kBatch * kLpThreads;
            if (--batches > 0)
#pragma unroll
                for (int b = 0; b < kBatch; ++b) raw[b] = p[b * kLpThreads];
            st.take(v);
            if (batches == 0) break;
        }
    }
    for (; p0 + k * kLpThreads < p1; k += kBatch) {
        const int j = p0 + (int)threadIdx.x + k * kLpThreads;
        uint4 raw[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) raw[b] = load(j + b * kLpThreads);
        if (j >= p1) break;
        F2 v[8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            F2 (&vb)[VE / 2] = *reinterpret_cast<F2 (*)[VE / 2]>(&v[b * VE / 2]);
            Piece<DT>::unpack(raw[b], vb);
        }
        st.take(v);
    }

    // fold: the row's maximum (as a key), then the sums relative to it
    const bool some = p0 + (int)threadIdx.x < p1;            // this thread holds logits
    const uint32_t key = some ? order_key(st.m) : 0u;
    {
        // maxima of a few threads each, which bound the alternatives, and the row's
        uint32_t g = key;
#pragma unroll
        for (int o = 1; o < kGroup; o *= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (lane % kGroup == 0) group[threadIdx.x / kGroup] = g;
    }
    const bool nan = __syncthreads_or(st.nan) != 0;
    const uint2 mine2 = *reinterpret_cast<const uint2*>(&group[2 * lane]);   // two groups a lane
    const uint32_t hi = __reduce_max_sync(0xffffffffu, max(mine2.x, mine2.y));
    const float M = hi ? key_value(hi) : -INFINITY;
    float S = halves(st.S).x + halves(st.S).y, A = halves(st.A).x + halves(st.A).y;
    if (M > -INFINITY) {
        const float dt = fmaxf((st.m - M) * kLog2e, kTiny), c = exp2_fast(dt);
        A = c * fmaf(S, dt, A);
        S *= c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, o);
        A += __shfl_xor_sync(0xffffffffu, A, o);
    }
    if (lane == 0) { fred[0][warp] = S; fred[1][warp] = A; }

    if (a.top > 0) {
        const int held = (n_pieces < p1 ? n_pieces : p1) - p0;             // pieces of this part
        bool rounds = nan;
        if (!rounds) {
            // T: at least `top` of the groups' maxima are >= T (0: every logit is a
            // candidate).  Every warp bisects on its own; any T with `top` to
            // top * 5 / 4 + 1 maxima above it will do.
            uint32_t T0 = 0;
            bool tied = false;                     // most groups share the lowest maximum
            const int full = ((held < kLpThreads ? held : kLpThreads) + kGroup - 1) / kGroup;   // groups with logits
            if (full >= a.top) {
                const uint32_t a0 = mine2.x ? mine2.x : 0xffffffffu, a1 = mine2.y ? mine2.y : 0xffffffffu;
                const uint32_t lo = T0 = __reduce_min_sync(0xffffffffu, min(a0, a1));
                uint32_t end = hi;
                while (T0 < end) {
                    const uint32_t mid = T0 + (end - T0 + 1) / 2;
                    const int c = __popc(__ballot_sync(0xffffffffu, mine2.x >= mid)) +
                                  __popc(__ballot_sync(0xffffffffu, mine2.y >= mid));
                    if (c >= a.top) {
                        T0 = mid;
                        if (c <= a.top + a.top / 4 + 1) break;
                    } else {
                        end = mid - 1;
                    }
                }
                tied = T0 == lo && full > a.top + a.top / 4 + 1;
            }
            // The logits >= from that the threads with a maximum >= from hold, read again:
            // by the thread itself where it has a few pieces (they are in L1), else by
            // its warp, a lane a piece and two threads at a time, which is one round
            // trip to L2 instead of one per batch.
            auto gather = [&](uint32_t from) {
                const float value = from == 0 ? -INFINITY : key_value(from);
                auto scan = [&](const uint4& raw, int j) {
                    F2 v[VE / 2];
                    Piece<DT>::unpack(raw, v);
                    float top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < VE / 2; ++q) top = max3_nan(top, v[q]);
                    if (top < value) return;
                    const int i = j * VE - shift;
#pragma unroll
                    for (int q = 0; q < VE; ++q) {
                        const float2 h = halves(v[q / 2]);
                        const float f = q & 1 ? h.y : h.x;
                        if (f >= value && i + q >= 0 && i + q < a.vocab) {
                            const int at = atomicAdd(&n_cand, 1);
                            if (at < kCandidates) cand[at] = entry_of(order_key(f), i + q);
                        }
                    }
                };
                const bool mine = some && key >= from;
                if (held <= 8 * kLpThreads) {
                    if (mine)
                        for (int j = p0 + (int)threadIdx.x; j < p1; j += 4 * kLpThreads) {
                            uint4 r[4];
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if (j + w * kLpThreads < p1) r[w] = load(j + w * kLpThreads);
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if (j + w * kLpThreads < p1) scan(r[w], j + w * kLpThreads);
                        }
                } else {
                    uint32_t who = __ballot_sync(0xffffffffu, mine);
                    while (who) {
                        const int l0 = __ffs(who) - 1;
                        who &= who - 1;
                        const int l1 = who ? __ffs(who) - 1 : -1;
                        who &= who - 1;
                        for (int j = p0 + warp * 32 + lane * kLpThreads; j - lane * kLpThreads < p1;
                             j += 32 * kLpThreads) {
                            const bool b0 = j + l0 < p1, b1 = l1 >= 0 && j + l1 < p1;
                            uint4 r0, r1;
                            if (b0) r0 = load(j + l0);
                            if (b1) r1 = load(j + l1);
                            if (b0) scan(r0, j + l0);
                            if (b1) scan(r1, j + l1);
                        }
                    }
                }
                __syncthreads();
            };
            if (!tied) gather(T0);
            if (tied || n_cand > kCandidates) {
                // Many equal T (a mask that leaves few, a constant row): take those above
                // it, and the first of the equal ones as a warp meets them in order.
                __syncthreads();
                if (threadIdx.x == 0) n_cand = 0;
                __syncthreads();
                gather(T0 + 1);
                const int above = n_cand;
                rounds = above > kCandidates - kMaxTop;
                __syncthreads();
                if (!rounds && warp == 0) {
                    int found = above;
                    for (int j = p0; j < p1 && found < a.top; j += 32) {
                        const uint4 raw = load(j + lane);
                        const T* e = reinterpret_cast<const T*>(&raw);
                        const int i = (j + lane) * VE - shift;
                        uint32_t equal = 0;
#pragma unroll
                        for (int k = 0; k < VE; ++k)
                            if (j + lane < p1 && i + k >= 0 && i + k < a.vocab && order_key(X::get(e[k])) == T0)
                                equal |= 1u << k;
                        int upto = __popc(equal);
#pragma unroll
                        for (int o = 1; o < 32; o *= 2) {
                            const int v = __shfl_up_sync(0xffffffffu, upto, o);
                            if (lane >= o) upto += v;
                        }
                        int at = found + upto - __popc(equal);
                        for (; equal && at < a.top; equal &= equal - 1) cand[at++] = entry_of(T0, i + __ffs(equal) - 1);
                        found += __shfl_sync(0xffffffffu, upto, 31);
                    }
                    if (lane == 0) n_cand = max(above, min(found, a.top));
                }
                __syncthreads();
            }
        }
        if (!rounds) {
            const int n = n_cand;
            for (int c = threadIdx.x; c < n; c += kLpThreads) {
                const unsigned long long mine = cand[c];
                const int before = rank_of(mine, cand, n);
                if (before < a.top) part.list[before] = mine;
            }
            if ((int)threadIdx.x >= n && (int)threadIdx.x < a.top) part.list[threadIdx.x] = 0;
        } else {
            // the largest entry below the one before it, `top` times
            unsigned long long last = ~0ull;
            for (int k = 0; k < a.top; ++k) {
                unsigned long long best = 0;
                for (int j = p0 + (int)threadIdx.x; j < p1; j += kLpThreads) {
                    const uint4 raw = load(j);
                    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
                    for (int q = 0; q < VE; ++q) {
                        const int i = j * VE - shift + q;
                        const unsigned long long c = entry_of(order_key(X::get(e[q])), i);
                        if (i >= 0 && i < a.vocab && c < last && c > best) best = c;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long c = __shfl_xor_sync(0xffffffffu, best, o);
                    best = c > best ? c : best;
                }
                __syncthreads();                                            // cand is free again
                if (lane == 0) cand[warp] = best;
                __syncthreads();
                for (int w = 0; w < kLpWarps; ++w) best = cand[w] > best ? cand[w] : best;
                last = best;
                if (threadIdx.x == 0) part.list[k] = best;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        S = A = 0.0f;
        for (int w = 0; w < kLpWarps; ++w) { S += fred[0][w]; A += fred[1][w]; }
        part.m = M; part.S = S; part.A = A; part.nan = nan;
    }
    __syncthreads();

    if constexpr (SPLIT) {
        // the first CTA gathers the others' parts
        cluster_sync();
        if (rank == 0) {
            const uint32_t base = (uint32_t)__cvta_generic_to_shared(&part);
            // the lists, in pairs: warp w merges those of CTAs 2w and 2w + 1, and so on
            if (a.top > 0) {
                unsigned long long best = 0;
                if (2 * warp < parts) {
                    const uint32_t la = base + (uint32_t)offsetof(LpPart, list);
                    const unsigned long long u = lane < a.top ? ld_peer64(peer(la + 8u * lane, 2 * warp)) : 0;
                    const unsigned long long v = 31 - lane < a.top ? ld_peer64(peer(la + 8u * (31 - lane), 2 * warp + 1)) : 0;
                    best = merge_sorted(u, v);
                }
                for (int n = parts / 2; n > 1; n /= 2) {             // n lists left, one a warp
                    if (warp < n) cand[32 * warp + lane] = best;
                    __syncthreads();
                    if (2 * warp < n) best = merge_sorted(cand[64 * warp + lane], cand[64 * warp + 63 - lane]);
                    __syncthreads();
                }
                if (warp == 0) cand[lane] = best;
            }
            float pm = -INFINITY, pS = 0.0f, pA = 0.0f;
            int pn = 0;
            if (warp == kLpWarps - 1) {
                if (lane < parts) {
                    pm = __uint_as_float(ld_peer32(peer(base + (uint32_t)offsetof(LpPart, m), lane)));
                    pS = __uint_as_float(ld_peer32(peer(base + (uint32_t)offsetof(LpPart, S), lane)));
                    pA = __uint_as_float(ld_peer32(peer(base + (uint32_t)offsetof(LpPart, A), lane)));
                    pn = (int)ld_peer32(peer(base + (uint32_t)offsetof(LpPart, nan), lane));
                }
                float all = pm;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
                if (all > -INFINITY) {
                    const float dt = fmaxf((pm - all) * kLog2e, kTiny), c = exp2_fast(dt);
                    pA = c * fmaf(pS, dt, pA);
                    pS *= c;
                }
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    pS += __shfl_xor_sync(0xffffffffu, pS, o);
                    pA += __shfl_xor_sync(0xffffffffu, pA, o);
                }
                pn = __any_sync(0xffffffffu, pn);
                pm = all;
            }
            __syncthreads();                                                // part is read by this CTA too
            if ((int)threadIdx.x < a.top) part.list[threadIdx.x] = cand[threadIdx.x];
            if (threadIdx.x == kLpThreads - 32) { part.m = pm; part.S = pS; part.A = pA; part.nan = pn; }
            __syncthreads();
        }
        cluster_sync();                                                     // (the others' parts have been read)
        if (rank != 0) return;
    }

    const float rm = part.m;
    const bool bad = part.nan || rm == INFINITY, empty = !bad && rm == -INFINITY;
    const float logS = logf(part.S);
    auto logprob = [&](float v) { return bad ? NAN : empty ? -INFINITY : (v - rm) - logS; };
    if (threadIdx.x == 0) {
        if (a.entropy) a.entropy[row] = bad ? NAN : empty ? 0.0f : logS - part.A * kLn2 / part.S;
        if (a.tokens) a.logprob[row] = tok < 0 ? 0.0f : tok >= a.vocab ? NAN : logprob(tok_x);
    }
    if ((int)threadIdx.x < a.top) {
        const unsigned long long e = part.list[threadIdx.x];
        a.top_id[row * a.top + threadIdx.x] = entry_index(e);
        a.top_logprob[row * a.top + threadIdx.x] = logprob(key_value((uint32_t)(e >> 32)));
    }
}

// CTAs of a row: until there is one per SM, in parts of at least 2048 logits.
// (Until two per SM: 77 rows of 32000 bf16 9.8 -> 9.0 us, but 150 rows 8.5 -> 12.1
// and 38 rows of 87371 10.7 -> 11.3.)
int row_parts(int64_t rows, int64_t vocab, int sms) {
    int parts = 1;
    while (parts < kLpCluster && rows * parts < sms && vocab / (parts * 2) >= 2048) parts *= 2;
    return parts;
}

template <int DT>
cudaError_t launch_logprobs(const LogprobArgs& a, int64_t rows, int sms, cudaStream_t s) {
    const int parts = row_parts(rows, a.vocab, sms);
    if (parts > 1)
        return launch_dense(logprobs_kernel<DT, true, kSplitThreads>, (unsigned)(rows * parts), kSplitThreads, 0,
                            (unsigned)parts, s, a, parts);
    // Threads of a row.  Rows that come in many waves and are short spend their time in
    // the folds: fewer threads a row put more rows on an SM, whose folds then overlap
    // others' loads.  Measured (us, 64 / 128 / 256 threads, top 5): 4096 x 4099 fp32 [22.6]
    // 28.4 39.0, 2500 x 5430 bf16 [15.0] 21.7 26.2; 4096 x 16000 fp32 58.9 [54.9] 61.5,
    // 600 x 2000 bf16 8.4 [6.0] 7.7, 4096 x 32000 bf16 [68] against 77; 1000 x 32000 fp32
    // 41.8 28.9 [27.8], 4096 x 32000 fp32 [96.9] against 99.7.
    const int64_t bytes = (int64_t)a.vocab * (int64_t)sizeof(typename Elem<DT>::T);
    const unsigned threads = rows >= 16 * (int64_t)sms && bytes <= 24 * 1024  ? 64
                             : rows >= 4 * (int64_t)sms && bytes <= 64 * 1024 ? 128
                                                                              : 256;
    auto kernel = threads == 64    ? logprobs_kernel<DT, false, 64>
                  : threads == 128 ? logprobs_kernel<DT, false, 128>
                                   : logprobs_kernel<DT, false, 256>;
    return launch_dense(kernel, (unsigned)rows, threads, 0, 1, s, a, 1);
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_token_logprobs(const void* logits, lb_dtype dtype, int64_t rows,
                                       int64_t vocab, int64_t ld, const int64_t* tokens,
                                       float* logprob, float* entropy, int top, int64_t* top_id,
                                       float* top_logprob, void* stream) {
    if (!logits || !dtype_ok(dtype)) return LB_ERR_INVALID_ARG;
    if (rows <= 0 || rows > 0x7fffffff || vocab <= 0 || vocab > (1 << 24) || ld < vocab ||
        ld > ((int64_t)1 << 40))
        return LB_ERR_INVALID_ARG;
    if ((tokens != nullptr) != (logprob != nullptr)) return LB_ERR_INVALID_ARG;
    if (top < 0 || top > kMaxTop || top > vocab) return LB_ERR_INVALID_ARG;
    if (top > 0 && (!top_id || !top_logprob)) return LB_ERR_INVALID_ARG;
    if (!tokens && !entropy && top == 0) return LB_ERR_INVALID_ARG;
    if (!is_aligned(logits, dtype_size(dtype)) || !is_aligned(tokens, 8) || !is_aligned(logprob, 4) ||
        !is_aligned(entropy, 4) || (top > 0 && (!is_aligned(top_id, 8) || !is_aligned(top_logprob, 4))))
        return LB_ERR_ALIGNMENT;
    int sms = 0;
    const lb_status st = dense_device(sms);
    if (st != LB_OK) return st;
    const LogprobArgs a = {logits, tokens, logprob, entropy, top_id, top_logprob, ld, (int)vocab, top};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        with_dtype(dtype, [&](auto d) { return launch_logprobs<d.value>(a, rows, sms, s); });
    return dense_status(e);
}
