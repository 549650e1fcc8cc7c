// lb_linear_int8: y[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k].
//
// The sum is exact (int32; in <= 131071 keeps it inside, since a product is at
// most 2^14).  y = (fp32(sum) * xs) * ws, rounded to y's type: fp32(sum) rounds
// sums past 2^24, and each factor once, so y is off by at most 3 * 2^-24
// relative before its own rounding.
#include <algorithm>

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
// With few tiles the K blocks of a tile are split over a cluster of CTAs, which
// exchange their partial sums through distributed shared memory (each CTA folds
// and stores its share of the tokens).  Integer sums: the order does not matter.
//
// Every wait is bounded (about 2 s).  A CTA that gives up stores NaN for the
// tiles it could not finish, frees its TMEM and returns.
constexpr int kMmaThreads = 320;
constexpr int kDrainWarps = 8;
constexpr int kLoadWarp = 8;
constexpr int kIssueWarp = 9;
constexpr int kTileCh = 128;                       // channels of a tile
constexpr int kMaxTok = 256;                       // tokens of a tile at most
constexpr int kKBytes = 128;                       // K per stage
constexpr int kWBytes = kTileCh * kKBytes;         // 16 KB
constexpr int kMaxStages8 = 12;
constexpr int kPipeBytes = 216 * 1024;             // stages (and a split's partial sums)
constexpr int kMaxSplit8 = 8;
constexpr long long kWaitLimit8 = 4000000000LL;    // cycles (~2 s)

struct Ctl8 {
    uint64_t full[kMaxStages8], empty[kMaxStages8], acc_full[2], acc_empty[2];
    uint32_t tmem_base;
    int abort;
    int lost[kMaxSplit8];                          // split: CTA r of the cluster gave up
};
constexpr int kMmaSmem = kPipeBytes + (int)sizeof(Ctl8) + 1024;
static_assert(kMmaSmem <= 232448, "shared memory");

struct MmaPlan {
    int nt;               // tokens per tile, a multiple of 16
    int n_tok, n_ch;      // tiles along the tokens and the channels
    int n_kb;             // K blocks
    int split;            // CTAs of the cluster that share a tile's K blocks
    int stages, stage_bytes;
    int acc_cols;         // columns of one accumulator, a multiple of 32
    int tmem_cols;        // allocated: a power of two >= 2 acc_cols
};

__device__ __forceinline__ uint32_t s32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ bool wait8(Ctl8* c, uint64_t* bar, uint32_t parity) {
    const uint32_t a = s32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(a, parity)) return true;
        if (*reinterpret_cast<volatile int*>(&c->abort)) return false;
        if (clock64() - t0 > kWaitLimit8) {
            atomicExch(&c->abort, 1);
            return false;
        }
    }
}

// Shared-memory descriptor: K-major, 128-byte swizzle, 8-row atoms of 1024 bytes.
__device__ __forceinline__ uint64_t desc8(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}
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

__device__ __forceinline__ void cluster_sync8() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank8() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr8(uint32_t addr, uint32_t rank) {
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    return p;
}
__device__ __forceinline__ void st_cluster8(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

template <int DT, bool SPLIT>
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
    const int rank = SPLIT ? (int)cluster_rank8() : 0;
    const int parts = SPLIT ? p.split : 1;
    const int first = (int)blockIdx.x / parts, step = (int)gridDim.x / parts;
    const int n_tiles = p.n_tok * p.n_ch;
    const int kb0 = (int)((long long)p.n_kb * rank / parts);
    const int kb1 = (int)((long long)p.n_kb * (rank + 1) / parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(s32(&ctl->full[s]), 1);
            mbar_init(s32(&ctl->empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s32(&ctl->acc_full[i]), 1);
            mbar_init(s32(&ctl->acc_empty[i]), kDrainWarps);
        }
        ctl->abort = 0;
        for (int r = 0; r < kMaxSplit8; ++r) ctl->lost[r] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(s32(&ctl->tmem_base)), "r"(p.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before8();
    __syncthreads();
    fence_after8();
    if (SPLIT) cluster_sync8();                    // every CTA of the cluster runs before one writes to it
    const uint32_t tmem = ctl->tmem_base;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 1;                       // a fresh stage counts as empty
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += step) {
                const int c0 = (t / p.n_tok) * kTileCh, m0 = (t % p.n_tok) * p.nt;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = wait8(ctl, &ctl->empty[s], ph))) break;
                    const uint32_t fb = s32(&ctl->full[s]), sb = base + s * p.stage_bytes;
                    mbar_expect_tx(fb, kWBytes + p.nt * kKBytes);
                    tma_load_2d(sb, &wmap, fb, kb * kKBytes, c0);
                    tma_load_2d(sb + kWBytes, &xmap, fb, kb * kKBytes, m0);
                    if (++s == p.stages) { s = 0; ph ^= 1; }
                }
            }
        }
    } else if (warp == kIssueWarp) {
        if (lane == 0) {
            const uint32_t id = idesc8(kTileCh, p.nt);
            int s = 0, tl = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += step, ++tl) {
                const int buf = tl & 1;
                if (!(ok = wait8(ctl, &ctl->acc_empty[buf], ((tl >> 1) & 1) ^ 1))) break;
                fence_after8();
                const uint32_t d = tmem + (uint32_t)(buf * p.acc_cols);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = wait8(ctl, &ctl->full[s], ph))) break;
                    fence_after8();
                    const uint32_t sb = base + s * p.stage_bytes;
                    const uint64_t ad = desc8(sb), bd = desc8(sb + kWBytes);
#pragma unroll
                    for (int kk = 0; kk < kKBytes / 32; ++kk)
                        mma_i8(d, ad + 2ull * kk, bd + 2ull * kk, id, (kb != kb0) || kk != 0);
                    commit8(s32(&ctl->empty[s]));
                    if (++s == p.stages) { s = 0; ph ^= 1; }
                }
                if (ok) commit8(s32(&ctl->acc_full[buf]));
            }
        }
    } else {
        const int q = warp & 3, hw = warp >> 2;    // accumulator lanes 32q .. 32q + 31
        int tl = 0;
        for (int t = first; t < n_tiles; t += step, ++tl) {
            const int c0 = (t / p.n_tok) * kTileCh, m0 = (t % p.n_tok) * p.nt;
            const int buf = tl & 1;
            const int n = c0 + q * 32 + lane;
            const float ws = n < a.N ? __ldg(a.ws + n) : 0.0f;
            // every lane waits; the warp goes on together (the TMEM loads are warp-wide)
            const bool ok = __all_sync(0xffffffffu, wait8(ctl, &ctl->acc_full[buf], (tl >> 1) & 1));
            fence_after8();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * p.acc_cols);
            if constexpr (SPLIT) {
                // partial sums to the CTA that folds their tokens: [source][token][channel]
                const int per = p.nt / parts;
                const uint32_t red = base + p.stages * p.stage_bytes;
                for (int j = 32 * hw; j < p.nt; j += 64) {
                    int v[32];
                    __syncwarp();
                    if (ok) tmem_ld8(tacc + (uint32_t)j, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (j + i >= p.nt) break;
                        const int dst = (j + i) / per, col = (j + i) % per;
                        st_cluster8(peer_addr8(red + 4u * (uint32_t)((rank * per + col) * kTileCh + q * 32 + lane),
                                               (uint32_t)dst), v[i]);
                    }
                }
                if (!ok && lane < parts)
                    st_cluster8(peer_addr8(s32(&ctl->lost[rank]), (uint32_t)lane), 1);
                break;                             // (a split call has one tile per cluster)
            } else {
            for (int j = 32 * hw; j < p.nt; j += 64) {
                int v[32];
                __syncwarp();
                if (ok) tmem_ld8(tacc + (uint32_t)j, v);
                const float xl = m0 + j + lane < a.M ? __ldg(a.xs + m0 + j + lane) : 0.0f;
                typename Y::T* y = static_cast<typename Y::T*>(a.y) + (int64_t)(m0 + j) * a.ldy + n;
                const int cols = min(min(32, p.nt - j), a.M - (m0 + j));
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float xs = __shfl_sync(0xffffffffu, xl, i);
                    if (i < cols && n < a.N) *y = Y::put(ok ? (float)v[i] * xs * ws : __int_as_float(0x7fc00000));
                    y += a.ldy;
                }
            }
            fence_before8();
            __syncwarp();
            if (lane == 0) mbar_arrive(s32(&ctl->acc_empty[buf]));
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync8();                           // all partial sums have arrived
        if (first < n_tiles && warp < kDrainWarps) {
            const int c0 = (first / p.n_tok) * kTileCh, m0 = (first % p.n_tok) * p.nt;
            const int per = p.nt / parts;
            const int ch = threadIdx.x & (kTileCh - 1), n = c0 + ch;
            const int* red = reinterpret_cast<const int*>(basep + p.stages * p.stage_bytes);
            bool ok = true;
            for (int r = 0; r < parts; ++r) ok = ok && ctl->lost[r] == 0;
            const float ws = n < a.N ? __ldg(a.ws + n) : 0.0f;
            for (int col = threadIdx.x / kTileCh; col < per; col += kDrainWarps * 32 / kTileCh) {
                const int m = m0 + rank * per + col;
                if (n >= a.N || m >= a.M) continue;
                int v = 0;
                for (int r = 0; r < parts; ++r) v += red[(r * per + col) * kTileCh + ch];
                static_cast<typename Y::T*>(a.y)[(int64_t)m * a.ldy + n] =
                    Y::put(ok ? (float)v * __ldg(a.xs + m) * ws : __int_as_float(0x7fc00000));
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

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

Encode encoder() {
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
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

// Tiles, K split and stages of a call on `sms` SMs.
MmaPlan mma_plan(int64_t M, int64_t N, int64_t K, int sms) {
    MmaPlan p = {};
    p.n_tok = (int)((M + kMaxTok - 1) / kMaxTok);
    p.nt = (int)(((M + p.n_tok - 1) / p.n_tok + 15) / 16 * 16);
    p.n_tok = (int)((M + p.nt - 1) / p.nt);
    p.n_ch = (int)((N + kTileCh - 1) / kTileCh);
    p.n_kb = (int)((K + kKBytes - 1) / kKBytes);
    p.split = 1;
    const int64_t tiles = (int64_t)p.n_tok * p.n_ch;
    // halve the K range while the clusters fit the SMs and a part keeps 4 blocks
    while (p.split < kMaxSplit8 && tiles * p.split * 2 <= sms && p.n_kb / (p.split * 2) >= 4) p.split *= 2;
    const int red = p.split > 1 ? kTileCh * p.nt * 4 : 0;
    p.stage_bytes = kWBytes + p.nt * kKBytes;
    p.stages = (kPipeBytes - red) / p.stage_bytes;
    if (p.stages > kMaxStages8) p.stages = kMaxStages8;
    p.acc_cols = (p.nt + 31) / 32 * 32;
    p.tmem_cols = 64;
    while (p.tmem_cols < 2 * p.acc_cols) p.tmem_cols *= 2;
    return p;
}

template <int DT, bool SPLIT>
cudaError_t launch_mma(const Int8Args& a, const MmaPlan& p, const CUtensorMap& wm, const CUtensorMap& xm,
                       int sms, cudaStream_t s) {
    const int64_t tiles = (int64_t)p.n_tok * p.n_ch;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)p.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * p.split : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = kMmaSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT ? 1 : 0;
    cudaError_t e = cudaFuncSetAttribute(int8_mma_kernel<DT, SPLIT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, int8_mma_kernel<DT, SPLIT>, wm, xm, a, p);
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
    const lb_status st = dense_device_ok();
    if (st != LB_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Int8Args a = {xq, wq, xs, ws, y, ldx, ldw, ldy, (int)M, (int)out, (int)in};
    if (mma_ok(a)) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return LB_ERR_CUDA;
        const MmaPlan p = mma_plan(M, out, in, sms);
        CUtensorMap wm, xm;
        // (the pitch of a single row is never used; the map wants a multiple of 16)
        if (!code_map(&wm, wq, out, in, out == 1 ? (in + 15) / 16 * 16 : ldw, kTileCh) ||
            !code_map(&xm, xq, M, in, M == 1 ? (in + 15) / 16 * 16 : ldx, p.nt))
            return LB_ERR_CUDA;
        const cudaError_t e = with_dtype(y_dtype, [&](auto d) {
            return p.split > 1 ? launch_mma<d.value, true>(a, p, wm, xm, sms, s)
                               : launch_mma<d.value, false>(a, p, wm, xm, sms, s);
        });
        return e == cudaSuccess ? LB_OK : LB_ERR_CUDA;
    }
    const int64_t blocks = ((M + kGenTile - 1) / kGenTile) * ((out + kGenTile - 1) / kGenTile);
    with_dtype(y_dtype, [&](auto d) { int8_general_kernel<d.value><<<(unsigned)blocks, 256, 0, s>>>(a); });
    return cudaGetLastError() == cudaSuccess ? LB_OK : LB_ERR_CUDA;
}
