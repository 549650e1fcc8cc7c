// lb_linear_int8: y[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k].
//
// The sum is exact (int32; in <= 131071 keeps it inside, since a product is at
// most 2^14).  y = (fp32(sum) * xs) * ws, rounded to y's type: fp32(sum) rounds
// sums past 2^24, and each factor once, so y is off by at most 3 * 2^-24
// relative before its own rounding.
#include <algorithm>

#include "lb_dense.cuh"
#include "lb_drain.h"

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

// General kernel: any pitch and alignment.  16 R tokens x 64 channels per block, 64
// columns of K at a time through two stages of shared memory, R tokens by four
// channels per thread with __dp4a.
//
// What bounds it: latency of a stage's loads with few blocks, reads of shared memory
// with many; two words are loaded for each one used.  4097 -> 32000, one token: 140 us
// (0.9 TB/s; rows on 16 bytes 21); 4097 -> 4096, 64 tokens 98 us, 512 tokens 256 us
// (67 TOP/s; 12 on 16 bytes).  Byte by byte these were 500, 216 and 485 us.
constexpr int kGenTile = 64;
constexpr int kGenPitch = 17;                // words of a staged row (16 used), odd: no bank conflicts

// Codes k .. k + 3 of a row of K that starts anywhere, 0 past its end, from the two
// aligned words that hold them.  A word is read only if it holds a code of the row.
__device__ __forceinline__ int codes_at(const int8_t* row, int k, int K) {
    if (k >= K) return 0;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    const int off = (int)(at & 3);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(at - off);
    const uint32_t lo = p[0], hi = off > 0 && k + 4 - off < K ? p[1] : 0;
    const uint32_t v = __funnelshift_r(lo, hi, 8 * off);
    return (int)(K - k < 4 ? v & ((1u << 8 * (K - k)) - 1) : v);
}

template <int DT, int R>
__global__ void __launch_bounds__(256) int8_general_kernel(const __grid_constant__ Int8Args a) {
    __shared__ int xt[2][16 * R * kGenPitch], wt[2][kGenTile * kGenPitch];
    const int n_m = (a.M + 16 * R - 1) / (16 * R);
    const int m0 = (int)(blockIdx.x % n_m) * (16 * R), n0 = (int)(blockIdx.x / n_m) * kGenTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    // Rows past the last are the last again: what they give is not stored.
    const int8_t* row[R + 4];
    int off[R + 4];
#pragma unroll
    for (int i = 0; i < R + 4; ++i) {
        const int m = m0 + ty + 16 * i, n = n0 + ty + 16 * (i - R);
        row[i] = i < R ? a.x + (int64_t)(m < a.M ? m : a.M - 1) * a.ldx : a.w + (int64_t)(n < a.N ? n : a.N - 1) * a.ldw;
        off[i] = (int)(reinterpret_cast<uintptr_t>(row[i]) & 3);
    }
    // Words tx of the next stage's rows.  While a code follows the stage's 64, both
    // aligned words of each hold codes of the row: all are requested without a
    // condition, which would make each load wait for the one before it.
    uint32_t lo[R + 4], hi[R + 4];
    const auto fetch = [&](int k0) {
        const int k = k0 + 4 * tx;
        if (k0 + 64 < a.K) {
#pragma unroll
            for (int i = 0; i < R + 4; ++i) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(row[i] + k - off[i]);
                lo[i] = p[0];
                hi[i] = p[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < R + 4; ++i) {
                const uint64_t v = (uint64_t)(uint32_t)codes_at(row[i], k, a.K) << 8 * off[i];
                lo[i] = (uint32_t)v;
                hi[i] = (uint32_t)(v >> 32);
            }
        }
    };
    grid_trigger();
    grid_wait();
    int acc[R][4] = {};
    fetch(0);
    for (int k0 = 0, stage = 0; k0 < a.K; k0 += 64, stage ^= 1) {
#pragma unroll
        for (int i = 0; i < R + 4; ++i) {
            const int v = (int)__funnelshift_r(lo[i], hi[i], 8 * off[i]);
            if (i < R) xt[stage][(ty + 16 * i) * kGenPitch + tx] = v;
            else wt[stage][(ty + 16 * (i - R)) * kGenPitch + tx] = v;
        }
        // Two stages: whoever is past this has read the other stage to its end.
        __syncthreads();
        if (k0 + 64 < a.K) fetch(k0 + 64);
#pragma unroll 4
        for (int kk = 0; kk < 16; ++kk) {
            int xv[R], wv[4];
#pragma unroll
            for (int i = 0; i < R; ++i) xv[i] = xt[stage][(ty + 16 * i) * kGenPitch + kk];
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[i] = wt[stage][(tx + 16 * i) * kGenPitch + kk];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
        }
    }
    using Y = Elem<DT>;
#pragma unroll
    for (int i = 0; i < R; ++i) {
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

// Tokens of a block's tile, 16 / 32 / 64, in us: 4097 -> 32000, 16 tokens [143] 170 245,
// 17 tokens 238 [170] 245, 32 tokens 240 [173] 248, 48 tokens 369 292 [250]; 4097 ->
// 4096, 32 tokens 103 [55] 106, 512 tokens 465 293 [256].
template <int DT, int R>
cudaError_t launch_general(const Int8Args& a, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.M + 16 * R - 1) / (16 * R) * (((int64_t)a.N + kGenTile - 1) / kGenTile);
    return launch_dense(int8_general_kernel<DT, R>, (unsigned)blocks, 256, 0, 1, s, a);
}

// ------------------------------------------------------------ one token
// The weights stream past once and __dp4a keeps up.  A warp takes two channels and,
// with few channels, a block's warps share their K (`parts`), so that every SM has
// some 100 KB of weights in flight; a lane holds 16 bytes of every row, 512
// contiguous bytes a warp, four such chunks requested together.  xq comes from L1.
//
// Against the tensor cores (us, weights from HBM): 4096 -> 32000 [21.4] 22.2, 8192
// -> 28672 [38.3] 38.9, 4096 -> 4096 [4.8] 6.8, 1024 -> 1024 [2.2] 3.6 (no barriers,
// TMEM and tensor maps to set up).  From two tokens on the products catch up with
// the loads: 4096 -> 32000 30.6 against [22.4], 4096 -> 4096 8.6 against [6.8].
// What bounds it: HBM, 6.1 to 6.3 TB/s (95 to 99% of the copy rate) at 4096 -> 32000.
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneCh = 2;                          // channels of a warp

__device__ __forceinline__ int dot16(int4 a, int4 b, int acc) {
    acc = __dp4a(a.x, b.x, acc);
    acc = __dp4a(a.y, b.y, acc);
    acc = __dp4a(a.z, b.z, acc);
    return __dp4a(a.w, b.w, acc);
}
__device__ __forceinline__ int4 ld_once(const int8_t* p) {
    int4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kOneThreads) int8_one_kernel(const __grid_constant__ Int8Args a, int parts) {
    using Y = Elem<DT>;
    __shared__ int part_sums[kOneWarps][kOneCh];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % parts;
    const int64_t n0 = ((int64_t)blockIdx.x * (kOneWarps / parts) + warp / parts) * kOneCh;
    const int chunks = a.K / 16;                   // whole 16-byte chunks of a row
    const int c0 = (int)((int64_t)chunks * part / parts), c1 = (int)((int64_t)chunks * (part + 1) / parts);
    const int4* x = reinterpret_cast<const int4*>(a.x);
    const int8_t* w[kOneCh];
#pragma unroll
    for (int i = 0; i < kOneCh; ++i) w[i] = a.w + (n0 + i < a.N ? n0 + i : a.N - 1) * a.ldw;
    grid_trigger();
    grid_wait();
    int acc[kOneCh] = {};
    constexpr int kAhead = 4;                      // chunks requested together
    int c = c0 + lane;
    for (; c + 32 * (kAhead - 1) < c1; c += 32 * kAhead) {
        int4 wv[kAhead][kOneCh];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int i = 0; i < kOneCh; ++i) wv[u][i] = ld_once(w[i] + 16 * (int64_t)(c + 32 * u));
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int4 xv = x[c + 32 * u];
#pragma unroll
            for (int i = 0; i < kOneCh; ++i) acc[i] = dot16(wv[u][i], xv, acc[i]);
        }
    }
    for (; c < c1; c += 32) {
        const int4 xv = x[c];
#pragma unroll
        for (int i = 0; i < kOneCh; ++i) acc[i] = dot16(ld_once(w[i] + 16 * (int64_t)c), xv, acc[i]);
    }
    if (part == parts - 1 && lane < a.K - 16 * chunks)             // the last bytes, one a lane
#pragma unroll
        for (int i = 0; i < kOneCh; ++i) acc[i] += (int)w[i][16 * chunks + lane] * (int)a.x[16 * chunks + lane];
#pragma unroll
    for (int i = 0; i < kOneCh; ++i) acc[i] = __reduce_add_sync(0xffffffffu, acc[i]);
    // lane i of the group's first warp stores channel n0 + i
    int sum = lane == 0 ? acc[0] : acc[1];
    static_assert(kOneCh == 2, "a lane per channel");
    if (parts > 1) {
        if (lane < kOneCh) part_sums[warp][lane] = sum;
        __syncthreads();
        if (part != 0) return;
        if (lane < kOneCh)
            for (int p = 1; p < parts; ++p) sum += part_sums[warp + p][lane];
    }
    const int64_t n = n0 + lane;
    if (lane < kOneCh && n < a.N) static_cast<typename Y::T*>(a.y)[n] = Y::put((float)sum * a.xs[0] * a.ws[n]);
}

template <int DT>
cudaError_t launch_one(const Int8Args& a, int sms, cudaStream_t s) {
    const int64_t groups = ((int64_t)a.N + kOneCh - 1) / kOneCh;
    int parts = 1;
    while (parts < kOneWarps && groups * parts < (int64_t)sms * 24 && a.K / (parts * 2) >= 512) parts *= 2;
    const int per_block = kOneWarps / parts;
    return launch_dense(int8_one_kernel<DT>, (unsigned)((groups + per_block - 1) / per_block), kOneThreads, 0, 1, s, a,
                        parts);
}

// ------------------------------------------------------------ tensor cores
// y^T tile = (128 channels of wq) x (nt tokens of xq): tcgen05.mma kind::i8, the
// weights as A, the tokens as B, int32 accumulators in TMEM.  The channels are
// the accumulator's lanes, so a column of it is one token's 128 channels: its
// store is contiguous in y without a transpose, whatever y's type, and a tile of
// few tokens costs a narrow MMA instead of 128 padded rows.
//
// One CTA per SM, persistent over tiles (tokens fastest, so the tiles that run
// together share their weights and the token rows stay in L2).  Warps 0-7 drain
// the accumulators, warp 8 loads (TMA, 128 bytes of K a stage, 128-byte swizzle;
// zeros past the edges), warp 9 owns TMEM and issues the MMAs.  Two accumulators:
// one tile is drained while the next is summed.
//
// What bounds it: HBM while the tokens are few (16 x 8192 -> 28672 bf16: 42.1 us a call,
// 5.6 TB/s, 87% of the copy rate; 39.5 us, 93%, in a graph), then what L2 gives an SM (see
// mma_plan), then the MMAs and the card's power limit (4096 x 8192 -> 32000, pairs of
// CTAs: 675 us, 3180 TOP/s in a burst, 94% of twice the bf16 burst rate; 780 to 800 us
// when it runs on).
//
// With few tiles the K blocks of a tile are split over a cluster of CTAs, which
// exchange their partial sums through distributed shared memory (each CTA folds
// and stores its share of the tokens).  Integer sums: the order does not matter.
//
// Every wait is bounded (about 2 s).  A CTA that gives up stores NaN for the
// tiles it could not finish and all after them, frees its TMEM and returns.
constexpr int kMmaThreads = 320;
constexpr int kDrainWarps = 8;
constexpr int kLoadWarp = 8;
constexpr int kIssueWarp = 9;
constexpr int kTileCh = 128;                       // channels of a tile
constexpr int kMaxTok = 256;                       // tokens of a tile at most
constexpr int kKBytes = 128;                       // K per stage
constexpr int kWBytes = kTileCh * kKBytes;         // 16 KB
constexpr int kMaxStages8 = 12;
constexpr int kTwoBlockTok = 160;                   // 3 stages of 2 x (16 + 20) KB
constexpr int kTwoBlockPair = 96;
constexpr int kSingleTok = 96;                      // up to here only single CTAs
constexpr int kPipeBytes = 216 * 1024;             // stages; then a split's partial sums
static_assert(kTileCh * (kMaxTok + 4) * 4 <= kPipeBytes, "partial sums");
constexpr int kMaxLgSplit = 3;                     // at most 8 CTAs share a tile
constexpr int kMaxSplit8 = 1 << kMaxLgSplit;
constexpr long long kWaitLimit8 = 4000000000LL;    // cycles (~2 s)

struct Ctl8 {
    uint64_t full[kMaxStages8], empty[kMaxStages8], acc_full[2], acc_empty[2];
    uint32_t tmem_base;
    int abort;
    alignas(16) float xbuf[kDrainWarps][32];       // token scales of the columns being stored
    int lost[kMaxSplit8];                          // split: CTA r of the cluster gave up
};
constexpr int kMmaSmem = kPipeBytes + (int)sizeof(Ctl8) + 1024;
static_assert(kMmaSmem <= 232448, "shared memory");

struct MmaPlan {
    int pair;             // two CTAs on a tile of 256 channels (else one, 128 channels)
    int nt;               // tokens per tile, a multiple of 16 (pairs: 32)
    int n_tok, n_ch;      // tiles along the tokens and the channels
    int kper;             // K blocks of 128 bytes a stage (1 or 2)
    int n_kb;             // stages of a tile's K
    int lg_split;         // log2 of the CTAs that share a tile's K blocks
    int stages, stage_bytes;
    int acc_cols;         // columns of one accumulator, a multiple of 32
    int tmem_cols;        // allocated: a power of two >= 2 acc_cols
};

__device__ __forceinline__ uint32_t s32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Whether a barrier's phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test8(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Waits for a barrier's phase; false when it gave up (bounded, about 2 s).  (Inline:
// around a call the loops' addresses and descriptors would leave the uniform registers.)
__device__ __forceinline__ bool wait8(Ctl8* c, uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int*>(&c->abort)) return false;
        if (clock64() - t0 > kWaitLimit8) {
            *reinterpret_cast<volatile int*>(&c->abort) = 1;
            return false;
        }
    }
}

// Shared-memory descriptor: K-major, 128-byte swizzle, 8-row atoms of 1024 bytes.
// The low word holds the address in 16-byte units.
constexpr uint64_t kDesc8 = (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
__device__ __forceinline__ uint64_t desc8(uint32_t saddr) { return kDesc8 | ((saddr & 0x3FFFFu) >> 4); }
// Instruction descriptor of kind::i8: int32 accumulator, signed A and B, both K-major.
__device__ __forceinline__ uint32_t idesc8(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ bool elect8() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void commit8(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before8() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after8() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes x 32 columns of the accumulator.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, int (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_arrive8() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait8() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr8(uint32_t addr, uint32_t rank) {
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    return p;
}
__device__ __forceinline__ void st_cluster8(uint32_t addr, int a, int b, int c, int d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_cluster8(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// Waits for the turn's accumulator and stores it, a warp a quarter of the lanes (lane =
// channel c0 + 32 (warp & 3) + lane) and every other 32 columns (tokens m0 ..).  The
// tokens' scales go through a shared buffer of the warp (xbuf, 32 floats) to be read
// four at a time: a shuffle a column shared the stores' queue.
template <int DT>
__device__ __forceinline__ void drain_tile(DrainTurn& turn, Ctl8* ctl, const Int8Args& a, uint32_t bar, uint32_t tacc,
                                           int c0, int m0, int nt, float* xbuf, int warp, int lane) {
    using Y = Elem<DT>;
    const int q = warp & 3, hw = warp >> 2, n = c0 + q * 32 + lane;
    float ws = n < a.N ? a.ws[n] : 0.0f;
    const int cols = min(nt, a.M - m0);
    float xl = lane < cols - 32 * hw ? a.xs[m0 + 32 * hw + lane] : 0.0f;
    // every lane waits; the warp goes on together (the TMEM loads are warp-wide)
    const bool ok =
        turn.full([&](uint32_t parity) { return __all_sync(0xffffffffu, wait8(ctl, bar, parity)) != 0; });
    fence_after8();
    if (!ok) ws = __int_as_float(0x7fc00000);      // NaN: the sums are not there
    tacc += (uint32_t)(q * 32) << 16;
    const int64_t ldy = a.ldy;
    for (int j = 32 * hw; j < cols; j += 64) {
        int v[32];
        __syncwarp();
        xbuf[lane] = xl;
        if (ok) tmem_ld8(tacc + (uint32_t)j, v);
        xl = lane < cols - (j + 64) ? a.xs[m0 + j + 64 + lane] : 0.0f;
        __syncwarp();
        typename Y::T* y = static_cast<typename Y::T*>(a.y) + (int64_t)(m0 + j) * ldy + n;
        const bool whole = j + 32 <= cols && c0 + kTileCh <= a.N;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 x4 = *reinterpret_cast<const float4*>(xbuf + i);
            const float xs[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const typename Y::T o = Y::put((float)v[i + k] * xs[k] * ws);
                if (whole || (j + i + k < cols && n < a.N)) *y = o;
                y += ldy;
            }
        }
    }
}

template <int DT, bool SPLIT, int KPER>
__global__ void __launch_bounds__(kMmaThreads, 1)
int8_mma_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                const __grid_constant__ Int8Args a, const __grid_constant__ MmaPlan p) {
    using Y = Elem<DT>;
    extern __shared__ __align__(1024) unsigned char dsm[];
    const uint32_t raw = s32(dsm);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* basep = dsm + (base - raw);
    Ctl8* ctl = reinterpret_cast<Ctl8*>(basep + kPipeBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = SPLIT ? p.lg_split : 0;         // a cluster has 2^lg CTAs
    const int rank = SPLIT ? (int)(blockIdx.x & ((1u << lg) - 1u)) : 0;
    const int first = (int)(blockIdx.x >> lg), step = (int)(gridDim.x >> lg);
    const int n_tok = p.n_tok, n_tiles = n_tok * p.n_ch, nt = p.nt;
    const int kb0 = (p.n_kb * rank) >> lg, kb1 = (p.n_kb * (rank + 1)) >> lg;
    const int stages = p.stages;
    const uint32_t stage_bytes = (uint32_t)p.stage_bytes;
    const uint32_t x_bytes = (uint32_t)(nt * kKBytes);             // the tokens of one K block
    const uint32_t full = s32(&ctl->full[0]), empty = s32(&ctl->empty[0]);
    const uint32_t acc_full = s32(&ctl->acc_full[0]), acc_empty = s32(&ctl->acc_empty[0]);

    grid_trigger();
    // The loading warp sets up the stages' barriers and requests the first stages
    // before anything else; TMEM and the other barriers follow meanwhile.  (It and
    // the issuing warp run their loops whole, with one lane elected for the
    // instructions: that keeps addresses and descriptors in uniform registers.  With
    // one lane inside a branch a tcgen05.mma took ~110 cycles to issue, now ~64.)
    int ls = 0, lkb = kb0, lt = first;             // its position: stage, K block, tile
    uint32_t lph = 1;                              // a fresh stage counts as empty
    int lc = (first / n_tok) * kTileCh, lm = (first % n_tok) * nt;
    auto load_stage = [&] {
        const uint32_t fb = full + 8u * (uint32_t)ls, sb = base + (uint32_t)ls * stage_bytes;
        if (elect8()) {
            mbar_expect_tx(fb, stage_bytes);
#pragma unroll
            for (int k = 0; k < KPER; ++k) {
                const int col = (lkb * KPER + k) * kKBytes;
                tma_load_2d(sb + k * kWBytes, &wmap, fb, col, lc);
                tma_load_2d(sb + KPER * kWBytes + (uint32_t)k * x_bytes, &xmap, fb, col, lm);
            }
        }
        __syncwarp();
        if (++ls == stages) { ls = 0; lph ^= 1; }
        if (++lkb == kb1) {
            lkb = kb0;
            lt += step;
            lc = (lt / n_tok) * kTileCh;
            lm = (lt % n_tok) * nt;
        }
    };
    if (warp == kLoadWarp) {
        if (lane < stages) {
            mbar_init(full + 8u * (uint32_t)lane, 1);
            mbar_init(empty + 8u * (uint32_t)lane, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        grid_wait();
        for (int s = 0; s < stages && lt < n_tiles; ++s) load_stage();
    }
    if (warp == kIssueWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(acc_full + 8u * i, 1);
                mbar_init(acc_empty + 8u * i, kDrainWarps);
            }
            ctl->abort = 0;
            for (int r = 0; r < kMaxSplit8; ++r) ctl->lost[r] = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(s32(&ctl->tmem_base)), "r"(p.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    fence_before8();
    __syncthreads();
    fence_after8();
    grid_wait();
    const uint32_t tmem = ctl->tmem_base;

    if (warp == kLoadWarp) {
        while (lt < n_tiles && __all_sync(0xffffffffu, wait8(ctl, empty + 8u * (uint32_t)ls, lph))) load_stage();
    } else if (warp == kIssueWarp) {
        const uint32_t id = idesc8(kTileCh, nt);
        const uint32_t acc_cols = (uint32_t)p.acc_cols;
        const uint64_t ad0 = desc8(base), bd0 = desc8(base + KPER * kWBytes);
        const uint32_t stage16 = stage_bytes / 16u, x16 = x_bytes / 16u;
        uint64_t ad = ad0, bd = bd0;               // the current stage's descriptors
        uint32_t ph = 0, fb = full, eb = empty;    // and barriers
        const uint32_t fb_end = full + 8u * (uint32_t)stages;
        int tl = 0;
        bool ok = true, ready = false;             // ready: the current stage is known to be full
        for (int t = first; t < n_tiles && ok; t += step, ++tl) {
            const uint32_t buf = tl & 1;
            if (!(ok = __all_sync(0xffffffffu, wait8(ctl, acc_empty + 8u * buf, ((tl >> 1) & 1) ^ 1)))) break;
            fence_after8();
            const uint32_t d = tmem + buf * acc_cols;
            uint32_t add = 0;                      // the tile's first product starts the sums
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!__all_sync(0xffffffffu, ready) && !(ok = __all_sync(0xffffffffu, wait8(ctl, fb, ph)))) break;
                fence_after8();
                if (elect8()) {
#pragma unroll
                    for (int k = 0; k < KPER; ++k)
#pragma unroll
                        for (int kk = 0; kk < kKBytes / 32; ++kk)
                            mma_i8(d, ad + (uint64_t)(k * (kWBytes / 16) + 2 * kk),
                                   bd + (uint64_t)((uint32_t)k * x16 + 2u * kk), id, k + kk ? 1u : add);
                    commit8(eb);
                }
                __syncwarp();
                add = 1;
                ad += stage16;
                bd += stage16;
                fb += 8u;
                eb += 8u;
                if (fb == fb_end) { fb = full; eb = empty; ph ^= 1; ad = ad0; bd = bd0; }
                ready = mbar_test8(fb, ph);        // (asked while the MMAs run)
            }
            if (ok && elect8()) commit8(acc_full + 8u * buf);
            __syncwarp();
        }
    } else if constexpr (SPLIT) {
        if (first < n_tiles) {                     // (a split call has one tile per cluster)
            // Once every CTA of the cluster has its sums (its stages are free then),
            // each gives the others their channels' partial sums: [source][channel]
            // [token], a channel's row padded to an odd number of 16-byte pieces.
            const int q = warp & 3, hw = warp >> 2;
            const bool ok = __all_sync(0xffffffffu, wait8(ctl, acc_full, 0));
            fence_after8();
            cluster_arrive8();
            cluster_wait8();
            const uint32_t per = (uint32_t)kTileCh >> lg;              // channels a CTA folds
            const uint32_t ch = (uint32_t)(q * 32 + lane), pitch = 4u * (uint32_t)(nt + 4);
            const uint32_t dst = peer_addr8(base + ((uint32_t)rank * per + (ch & (per - 1))) * pitch, ch >> (7 - lg));
            for (int j = 32 * hw; j < nt; j += 64) {
                int v[32];
                __syncwarp();
                if (ok) tmem_ld8(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)j, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (j + i < nt) st_cluster8(dst + 4u * (uint32_t)(j + i), v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            if (!ok && lane < (1 << lg)) st_cluster8(peer_addr8(s32(&ctl->lost[rank]), (uint32_t)lane), 1);
        }
    } else {
        DrainTurn turn;
        for (int t = first; t < n_tiles; t += step, turn.next()) {
            const uint32_t buf = turn.buf();
            drain_tile<DT>(turn, ctl, a, acc_full + 8u * buf, tmem + buf * (uint32_t)p.acc_cols,
                           (t / n_tok) * kTileCh, (t % n_tok) * nt, nt, ctl->xbuf[warp], warp, lane);
            fence_before8();
            __syncwarp();
            if (turn.alive && lane == 0) mbar_arrive(acc_empty + 8u * buf);
        }
    }
    if constexpr (SPLIT) {
        __syncwarp();
        if (warp >= kDrainWarps) {                 // (the draining warps have been through this one)
            cluster_arrive8();
            cluster_wait8();
        }
        cluster_arrive8();
        cluster_wait8();                           // all partial sums have arrived
        if (warp < kDrainWarps) {
            const int c0 = (first / n_tok) * kTileCh, m0 = (first % n_tok) * nt;
            const int per = kTileCh >> lg, parts = 1 << lg;
            const int ch = threadIdx.x & (per - 1), n = c0 + rank * per + ch;
            const uint32_t pitch = 4u * (uint32_t)(nt + 4);
            float ws = n < a.N ? a.ws[n] : 0.0f;
            for (int r = 0; r < parts; ++r)
                if (ctl->lost[r]) ws = __int_as_float(0x7fc00000);
            const int cols = min(nt, a.M - m0);
            const int4* red = reinterpret_cast<const int4*>(basep + (uint32_t)ch * pitch);
            const uint32_t part_step = (uint32_t)per * pitch / 16u;
            for (int j = 4 * (int)(threadIdx.x >> (7 - lg)); j < cols; j += 4 * ((kDrainWarps * 32) >> (7 - lg))) {
                float xs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) xs[i] = j + i < cols ? a.xs[m0 + j + i] : 0.0f;
                int4 v = red[j / 4];
                for (int r = 1; r < parts; ++r) {
                    const int4 o = red[(uint32_t)r * part_step + j / 4];
                    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                }
                if (n >= a.N) continue;
                typename Y::T* y = static_cast<typename Y::T*>(a.y) + (int64_t)(m0 + j) * a.ldy + n;
                const int vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j + i < cols) y[i * a.ldy] = Y::put((float)vv[i] * xs[i] * ws);
            }
        }
    }
    // Every role is done or has given up; copies still in flight after an abort
    // get time to land before the shared memory goes away, then TMEM is freed.
    __syncthreads();
    if (ctl->abort && threadIdx.x == 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000LL) { }
    }
    __syncthreads();
    if (warp == kIssueWarp) {
        fence_after8();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

// The same with two CTAs on a tile of 256 channels (tcgen05 cta_group::2): each
// loads its own 128 channels and half of the tokens, the first one issues the MMAs
// for both, and each drains its own channels.  A CTA then brings in 32 KB for a
// K block of 256 tokens instead of 48 KB.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];"
        :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Arrives on the barrier at this offset in both CTAs when the MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void arrive_peer8(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

template <int DT, int KPER>
__global__ void __launch_bounds__(kMmaThreads, 1)
int8_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                 const __grid_constant__ Int8Args a, const __grid_constant__ MmaPlan p) {
    extern __shared__ __align__(1024) unsigned char dsm[];
    const uint32_t raw = s32(dsm);
    const uint32_t base = (raw + 1023u) & ~1023u;
    Ctl8* ctl = reinterpret_cast<Ctl8*>(dsm + (base - raw) + kPipeBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1u);
    const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
    const int n_tok = p.n_tok, n_tiles = n_tok * p.n_ch, nt = p.nt, n_kb = p.n_kb;
    const int stages = p.stages;
    const uint32_t stage_bytes = (uint32_t)p.stage_bytes, x_bytes = (uint32_t)(nt / 2 * kKBytes);
    const uint32_t full = s32(&ctl->full[0]), empty = s32(&ctl->empty[0]);
    const uint32_t acc_full = s32(&ctl->acc_full[0]), acc_empty = s32(&ctl->acc_empty[0]);

    grid_trigger();
    if (warp == kLoadWarp) {
        if (lane < stages) {
            mbar_init(full + 8u * (uint32_t)lane, 1);
            mbar_init(empty + 8u * (uint32_t)lane, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssueWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(acc_full + 8u * i, 1);
                mbar_init(acc_empty + 8u * i, 2 * kDrainWarps);        // (the first CTA's; both drain)
            }
            ctl->abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(s32(&ctl->tmem_base)), "r"(p.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    fence_before8();
    __syncthreads();
    cluster_arrive8();
    cluster_wait8();                               // both CTAs' barriers are set up
    fence_after8();
    grid_wait();
    const uint32_t tmem = ctl->tmem_base;

    if (warp == kLoadWarp) {
        // both CTAs' copies count on the first CTA's barrier
        const uint32_t full0 = peer_addr8(full, 0);
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int t = first; t < n_tiles && ok; t += step) {
            const int c0 = (t / n_tok) * 2 * kTileCh + rank * kTileCh, m0 = (t % n_tok) * nt + rank * (nt / 2);
            for (int kb = 0; kb < n_kb; ++kb) {
                if (!(ok = __all_sync(0xffffffffu, wait8(ctl, empty + 8u * (uint32_t)s, ph)))) break;
                const uint32_t sb = base + (uint32_t)s * stage_bytes, fb = full0 + 8u * (uint32_t)s;
                if (elect8()) {
                    if (rank == 0) mbar_expect_tx(full + 8u * (uint32_t)s, 2u * stage_bytes);
#pragma unroll
                    for (int k = 0; k < KPER; ++k) {
                        const int col = (kb * KPER + k) * kKBytes;
                        tma_load_pair(sb + k * kWBytes, &wmap, fb, col, c0);
                        tma_load_pair(sb + KPER * kWBytes + (uint32_t)k * x_bytes, &xmap, fb, col, m0);
                    }
                }
                __syncwarp();
                if (++s == stages) { s = 0; ph ^= 1; }
            }
        }
    } else if (warp == kIssueWarp) {
        if (rank == 0) {
            const uint32_t id = idesc8(2 * kTileCh, nt);
            const uint32_t acc_cols = (uint32_t)p.acc_cols;
            const uint64_t ad0 = desc8(base), bd0 = desc8(base + KPER * kWBytes);
            const uint32_t stage16 = stage_bytes / 16u, x16 = x_bytes / 16u;
            uint64_t ad = ad0, bd = bd0;
            uint32_t ph = 0, fb = full, eb = empty;
            const uint32_t fb_end = full + 8u * (uint32_t)stages;
            int tl = 0;
            bool ok = true, ready = false;
            for (int t = first; t < n_tiles && ok; t += step, ++tl) {
                const uint32_t buf = tl & 1;
                if (!(ok = __all_sync(0xffffffffu, wait8(ctl, acc_empty + 8u * buf, ((tl >> 1) & 1) ^ 1)))) break;
                fence_after8();
                const uint32_t d = tmem + buf * acc_cols;
                uint32_t add = 0;
                for (int kb = 0; kb < n_kb; ++kb) {
                    if (!__all_sync(0xffffffffu, ready) && !(ok = __all_sync(0xffffffffu, wait8(ctl, fb, ph)))) break;
                    fence_after8();
                    if (elect8()) {
#pragma unroll
                        for (int k = 0; k < KPER; ++k)
#pragma unroll
                            for (int kk = 0; kk < kKBytes / 32; ++kk)
                                mma_i8_pair(d, ad + (uint64_t)(k * (kWBytes / 16) + 2 * kk),
                                            bd + (uint64_t)((uint32_t)k * x16 + 2u * kk), id, k + kk ? 1u : add);
                        commit_pair(eb);
                    }
                    __syncwarp();
                    add = 1;
                    ad += stage16;
                    bd += stage16;
                    fb += 8u;
                    eb += 8u;
                    if (fb == fb_end) { fb = full; eb = empty; ph ^= 1; ad = ad0; bd = bd0; }
                    ready = mbar_test8(fb, ph);
                }
                if (ok && elect8()) commit_pair(acc_full + 8u * buf);
                __syncwarp();
            }
        }
    } else {
        const uint32_t acc_empty0 = peer_addr8(acc_empty, 0);
        DrainTurn turn;
        for (int t = first; t < n_tiles; t += step, turn.next()) {
            const uint32_t buf = turn.buf();
            drain_tile<DT>(turn, ctl, a, acc_full + 8u * buf, tmem + buf * (uint32_t)p.acc_cols,
                           (t / n_tok) * 2 * kTileCh + rank * kTileCh, (t % n_tok) * nt, nt, ctl->xbuf[warp], warp, lane);
            fence_before8();
            __syncwarp();
            if (turn.alive && lane == 0) arrive_peer8(acc_empty0 + 8u * buf);
        }
    }
    __syncthreads();
    if (ctl->abort && threadIdx.x == 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000LL) { }
    }
    __syncthreads();
    cluster_arrive8();
    cluster_wait8();                               // neither CTA leaves while the other may signal it
    if (warp == kIssueWarp) {
        fence_after8();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

Encode encoder() {
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (dense_status(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r)) != LB_OK ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    return fn;
}

// int8 [rows][k] of pitch ld (a multiple of 16, 16-byte aligned), boxes of 128
// columns by box_rows rows in the 128-byte swizzle, zeros past the edges.
bool code_map(CUtensorMap* map, const int8_t* ptr, int64_t rows, int64_t k, int64_t ld, int box_rows) {
    const Encode enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)kKBytes, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(ptr), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The plan of a call on `sms` SMs: single CTAs or pairs, tokens per tile, K split.
// Each candidate is given its time in cycles and the shortest is taken.  A K block
// (128 bytes of K) of a tile costs what its operands take from L2 at 64 bytes a
// clock and SM, which is what every shape with several rounds measured (4096 ->
// 11008 at 1000 tokens, tiles of 208 tokens by single CTAs: 672 cycles a block by
// this rule, 38 us; pairs with 224 tokens: 480 cycles, 37 us; with 192, a fourth
// round, 40 us), and at least ~300 to issue.  A pair's K block of 256 tokens takes
// 512 cycles to bring in and 512 to multiply.  Then come the last tile's stores,
// ~25 cycles a token, or a split's exchange, ~3000 + 55 a token.
MmaPlan mma_plan(int64_t M, int64_t N, int64_t K, int sms) {
    MmaPlan best = {};
    int64_t best_cost = -1;
    const int64_t blocks = (K + kKBytes - 1) / kKBytes;
    const int64_t least = (M + kMaxTok - 1) / kMaxTok;             // token tiles at least
    for (int pair = 0; pair <= (M > kSingleTok ? 1 : 0); ++pair) {
        const int grain = pair ? 32 : 16, ch = pair ? 2 * kTileCh : kTileCh;
        const int64_t n_ch = (N + ch - 1) / ch, ctas = pair ? sms / 2 : sms;
        for (int64_t tok = least; tok < least + 8 && (tok - 1) * grain < M; ++tok) {
            const int nt = (int)((M + tok - 1) / tok + grain - 1) / grain * grain;
            const int64_t n_tok = (M + nt - 1) / nt, tiles = n_tok * n_ch;
            const int64_t block = std::max<int64_t>(300, pair ? 256 + nt : 2 * (kTileCh + nt));
            for (int lg = 0; lg <= (pair ? 0 : kMaxLgSplit); ++lg) {
                // (a split has a cluster per tile, all at once, and at least 4 blocks a part)
                if (lg > 0 && ((tiles << lg) > sms || (blocks >> lg) < 4)) break;
                const int64_t rounds = lg > 0 ? 1 : (tiles + ctas - 1) / ctas;
                const int64_t cost = rounds * ((blocks + (1 << lg) - 1) >> lg) * block +
                                     (lg > 0 ? 3000 + 55 * nt : 25 * nt);
                if (best_cost >= 0 && cost >= best_cost) continue;
                best_cost = cost;
                best.pair = pair;
                best.nt = nt;
                best.n_tok = (int)n_tok;
                best.n_ch = (int)n_ch;
                best.lg_split = lg;
            }
        }
    }
    MmaPlan p = best;
    const int x_rows = p.pair ? p.nt / 2 : p.nt;                    // tokens that one CTA loads
    // Two K blocks a stage halve the waits and commits: worth it while the tiles are
    // small (pairs of 64 tokens 12.7 -> 12.5 us, of 192 tokens 23.6 -> 26.2 us).
    p.kper = p.nt <= (p.pair ? kTwoBlockPair : kTwoBlockTok) ? 2 : 1;
    p.n_kb = (int)((K + p.kper * kKBytes - 1) / (p.kper * kKBytes));
    p.stage_bytes = p.kper * (kWBytes + x_rows * kKBytes);
    p.stages = std::min(kPipeBytes / p.stage_bytes, kMaxStages8);
    p.acc_cols = (p.nt + 31) / 32 * 32;
    p.tmem_cols = 64;
    while (p.tmem_cols < 2 * p.acc_cols) p.tmem_cols *= 2;
    return p;
}

template <int DT, bool SPLIT, int KPER>
cudaError_t launch_mma(const Int8Args& a, const MmaPlan& p, const CUtensorMap& wm, const CUtensorMap& xm,
                       int sms, cudaStream_t s) {
    const int64_t tiles = (int64_t)p.n_tok * p.n_ch;
    const cudaError_t e = cudaFuncSetAttribute(int8_mma_kernel<DT, SPLIT, KPER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem);
    if (e != cudaSuccess) return e;
    return launch_dense(int8_mma_kernel<DT, SPLIT, KPER>,
                        (unsigned)(SPLIT ? tiles << p.lg_split : std::min<int64_t>(tiles, sms)), kMmaThreads, kMmaSmem,
                        1u << p.lg_split, s, wm, xm, a, p);
}

template <int DT, int KPER>
cudaError_t launch_pair(const Int8Args& a, const MmaPlan& p, const CUtensorMap& wm, const CUtensorMap& xm,
                        int sms, cudaStream_t s) {
    const int64_t tiles = (int64_t)p.n_tok * p.n_ch;
    const cudaError_t e = cudaFuncSetAttribute(int8_pair_kernel<DT, KPER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem);
    if (e != cudaSuccess) return e;
    return launch_dense(int8_pair_kernel<DT, KPER>, (unsigned)(2 * std::min<int64_t>(tiles, sms / 2)), kMmaThreads,
                        kMmaSmem, 2, s, wm, xm, a, p);
}

// The tensor-core kernel reads rows through tensor maps: 16-byte pieces.
bool mma_ok(const Int8Args& a) {
    return is_aligned(a.x, 16) && is_aligned(a.w, 16) && (a.M == 1 || a.ldx % 16 == 0) &&
           (a.N == 1 || a.ldw % 16 == 0);
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_linear_int8(const int8_t* xq, int64_t ldx, const float* xs, int64_t M,
                                    const int8_t* wq, int64_t ldw, const float* ws, int64_t in,
                                    int64_t out, void* y, lb_dtype y_dtype, int64_t ldy,
                                    void* stream) {
    if (!xq || !xs || !wq || !ws || !y || !dtype_ok(y_dtype)) return LB_ERR_INVALID_ARG;
    if (M <= 0 || in <= 0 || out <= 0 || M > (1 << 24) || out > (1 << 24) || in > 131071 ||
        M * out > ((int64_t)1 << 40))
        return LB_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 32;
    if (ldx < in || ldw < in || ldy < out || ldx > most || ldw > most || ldy > most)
        return LB_ERR_INVALID_ARG;
    if (!is_aligned(xs, 4) || !is_aligned(ws, 4) || !is_aligned(y, dtype_size(y_dtype)))
        return LB_ERR_ALIGNMENT;
    int sms = 0;
    const lb_status st = dense_device(sms);
    if (st != LB_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Int8Args a = {xq, wq, xs, ws, y, ldx, ldw, ldy, (int)M, (int)out, (int)in};
    if (mma_ok(a)) {
        if (M == 1) {
            const cudaError_t e = with_dtype(y_dtype, [&](auto d) { return launch_one<d.value>(a, sms, s); });
            return dense_status(e);
        }
        const MmaPlan p = mma_plan(M, out, in, sms);
        CUtensorMap wm, xm;
        // (the pitch of a single channel is never used; the map wants a multiple of 16)
        if (!code_map(&wm, wq, out, in, out == 1 ? (in + 15) / 16 * 16 : ldw, kTileCh) ||
            !code_map(&xm, xq, M, in, ldx, p.pair ? p.nt / 2 : p.nt))
            return LB_ERR_CUDA;
        const cudaError_t e = with_dtype(y_dtype, [&](auto d) {
            if (p.pair && p.kper == 1) return launch_pair<d.value, 1>(a, p, wm, xm, sms, s);
            if (p.pair) return launch_pair<d.value, 2>(a, p, wm, xm, sms, s);
            if (p.kper == 1)
                return p.lg_split > 0 ? launch_mma<d.value, true, 1>(a, p, wm, xm, sms, s)
                                      : launch_mma<d.value, false, 1>(a, p, wm, xm, sms, s);
            return p.lg_split > 0 ? launch_mma<d.value, true, 2>(a, p, wm, xm, sms, s)
                                  : launch_mma<d.value, false, 2>(a, p, wm, xm, sms, s);
        });
        return dense_status(e);
    }
    const cudaError_t e = with_dtype(y_dtype, [&](auto d) {
        return M <= 16   ? launch_general<d.value, 1>(a, s)
               : M <= 32 ? launch_general<d.value, 2>(a, s)
                         : launch_general<d.value, 4>(a, s);
    });
    return dense_status(e);
}
