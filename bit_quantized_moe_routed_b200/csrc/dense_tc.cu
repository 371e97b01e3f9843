// dense_tc.cu -- products of the dense operators on the tensor cores, many
// rows: out[M][N] tiles of 256 x BN by pairs of SMs (tcgen05 cta_group::2).
//
// Mathematics: D = A B^T with A [M][K], B [N][K], each stored with K
// contiguous or (bf16) transposed with M / N contiguous; sums in f32 (bf16) or
// exact in s32 (int8).  The gated block multiplies A with two matrices at
// once: a pair's B tile is BN/2 rows of gate (loaded by the first SM) and the
// same BN/2 rows of up (by the second), so one accumulator row holds the gate
// and up sums of the same outputs and the epilogue forms silu(g) u, or the
// gradients dg, du, without another pass.  dx = dg Wg + du Wu runs its
// reduction over two segments into one accumulator; dWg and dWu are two
// batches over one B; the three gradients are one launch.
//
// Bound: the tensor cores.  Each K block of 128 bytes (64 bf16, 128 s8) is 16
// KB of A and BN/2 x 128 bytes of B per SM, loaded by TMA (128-byte swizzle)
// into a ring of stages; a pair reads every byte of its tile once per K block,
// so 256 x 256 tiles need 256 flop per byte from L2.  Roles per SM: warp 0
// loads, warp 1 of the first SM issues the MMAs for both, warps 4..11 run the
// epilogue of one accumulator while the MMAs fill the other (two of BN columns
// in tensor memory).  Persistent pairs walk the tiles in groups of 8 tile rows
// so that the tiles in flight share operands in L2; the longer tiles of a
// launch come first and the shorter ones even out what they leave.
//
// Every wait is bounded: a role that gives up raises the CTA's abort flag, the
// kernel drains its copies and MMAs, frees its tensor memory and raises the
// status word.
#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <mutex>
#include <utility>

#include "dense_tc.cuh"

namespace moeq {
namespace dense {
namespace {

using namespace umma;

constexpr int kTileM = 128;                 // rows of A per SM (a pair: 256)
constexpr int kABytes = kTileM * kRowBytes; // 16 KB
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kScaleBytes = 32 * 4;         // a chunk's int8 channel scales
constexpr int kStageOut = kEpiWarps * (4096 + kScaleBytes);
constexpr int kGroupM = 8;

// One product, or two of one shape over one B.
struct TcWork {
    CUtensorMap a[2], b[2];
    long long M, N;
    int kblocks;         // K blocks of one segment
    int nseg, nbatch;
    int mt, nt;          // tiles of one batch
    bool a_mn;           // A stored [K][M]
    void *out[2];
    long long old[2];
    bool vec_out;
    __host__ __device__ int tiles() const { return mt * nt * nbatch; }
    __host__ __device__ int kb_total() const { return kblocks * nseg; }
};
struct TcArgs {
    TcWork w[2];         // the longer tiles first
    int nwork;
    int extra;           // see TileWalk
    const float *a_scale, *b_scale[2];
    void *keep[2];
    long long kld;
    const void *dh;
    long long dhld;
    bool vec_keep, vec_dh;
    long long wait_cycles;
    uint32_t *status;
};

__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool I8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (I8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// Arrive on `bar` of both SMs once every MMA issued so far has completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

template <int BN>
struct Ring {
    static constexpr int kBBytes = BN / 2 * kRowBytes;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 6 : 7;
    static constexpr size_t kSmem = (size_t)kStages * kStage + kStageOut + 1024;
};

// The tiles of one pair.  Work 0 goes round the pairs; the pairs that get one
// tile less of it take `extra` tiles of work 1 first, then work 1 goes round.
struct TileWalk {
    const TcArgs &p;
    int pair, pairs, n0, r0, t = 0, phase = 0;
    int work = 0, z = 0, m = 0, n = 0;     // the current tile
    __device__ __forceinline__ TileWalk(const TcArgs &a, int pair_, int pairs_) : p(a), pair(pair_), pairs(pairs_) {
        n0 = a.w[0].tiles();
        r0 = n0 % pairs;
        t = pair;
    }
    __device__ __forceinline__ bool next() {
        if (phase == 0) {
            if (t < n0) {
                set(0, t);
                t += pairs;
                return true;
            }
            if (p.nwork == 1) return false;
            phase = 1;
            t = pair - r0;
        }
        const int n1 = p.w[1].tiles(), ahead = r0 ? (pairs - r0) * p.extra : 0;
        if (phase == 1) {
            if (t >= 0 && t < min(ahead, n1)) {
                set(1, t);
                t += pairs - r0;
                return true;
            }
            phase = 2;
            t = ahead + pair;
        }
        if (t >= n1) return false;
        set(1, t);
        t += pairs;
        return true;
    }
    // tile index -> batch, tile row, tile column: groups of kGroupM tile rows, row fastest
    __device__ __forceinline__ void set(int w, int i) {
        const int mt = p.w[w].mt, nt = p.w[w].nt;
        work = w;
        z = i / (mt * nt);
        i -= z * mt * nt;
        const int per = kGroupM * nt, g = i / per, first = g * kGroupM;
        const int rows = min(kGroupM, mt - first);
        i -= g * per;
        m = first + i % rows;
        n = i / rows;
    }
};

template <bool I8, bool B_MN, int EPI, int BN, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) product_tc_kernel(const __grid_constant__
                                                                                          TcArgs p) {
    typedef Ring<BN> R;
    constexpr int S = R::kStages;
    constexpr int kKE = I8 ? 128 : 64;                       // elements of a K block
    constexpr int kOutN = EPI == EPI_STORE ? BN : BN / 2;    // columns of out per tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *stage_out = smem + S * R::kStage;
    __shared__ alignas(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&done, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(2 * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // f(dst offset in a stage, map, x, y) for every box of K block kb of a tile
    auto boxes = [&](const TileWalk &at, const TcWork &w, int kb, auto f) {
        const int m0 = at.m * 2 * kTileM + (int)rank * kTileM;
        const int n0 = EPI == EPI_STORE ? at.n * BN + (int)rank * (BN / 2) : at.n * kOutN;
        const int seg = w.nseg > 1 && kb >= w.kblocks, k0 = (seg ? kb - w.kblocks : kb) * kKE;
        const CUtensorMap *ma = &w.a[w.nseg > 1 ? seg : at.z];
        const CUtensorMap *mb = &w.b[EPI == EPI_STORE ? seg : (int)rank];
        if (B_MN && w.a_mn) {
#pragma unroll
            for (int j = 0; j < kTileM / 64; ++j) f(j * 8192, ma, m0 + 64 * j, k0);
        } else {
            f(0, ma, k0, m0);
        }
        if (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) f(kABytes + j * 8192, mb, n0 + 64 * j, k0);
        } else {
            f(kABytes, mb, k0, n0);
        }
    };
    // the first stages' boxes on their way to L2 while the kernel before drains
    if (threadIdx.x == 0) {
        TileWalk at(p, pair, pairs);
        if (at.next())
            for (int kb = 0; kb < S && kb < p.w[at.work].kb_total(); ++kb)
                boxes(at, p.w[at.work], kb, [&](int, const CUtensorMap *map, int x, int y) { tma_prefetch_2d(map, x, y); });
    }
    pdl_wait_primary();
    pdl_launch_dependents();

    if (warp == 0 && lane == 0) {
        // ---- loads: this SM's 128 rows of A and its half of B, into the pair's barrier
        int c = 0;
        bool ok = true;
        for (TileWalk at(p, pair, pairs); ok && at.next();) {
            const TcWork &w = p.w[at.work];
            const int kb_total = w.kb_total();
            for (int kb = 0; kb < kb_total; ++kb, ++c) {
                const int s = c % S;
                if (c >= S && !wait_cluster(&empty[s], (uint32_t)((c / S - 1) & 1), &abort_flag, p.wait_cycles)) {
                    ok = false;
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * R::kStage);
                const uint32_t bar = in_cta(&full[s], 0);
                uint8_t *st = smem + s * R::kStage;
                boxes(at, w, kb, [&](int off, const CUtensorMap *map, int x, int y) { tma_load_pair(st + off, map, x, y, bar); });
            }
        }
        // the ring's last stages: consumed before this SM's shared memory goes away,
        // or, once a role has given up, landed long since (this SM cannot wait for
        // the pair's barrier)
        const long long t0 = clock64(), drain = ok && p.wait_cycles > kDrainCycles ? p.wait_cycles : kDrainCycles;
        for (int i = c > S ? c - S : 0; i < c; ++i)
            while (!test_wait_cluster(&empty[i % S], (uint32_t)((i / S) & 1)) && clock64() - t0 < drain) {
            }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- MMAs of the pair
        int c = 0, q = 0;
        bool ok = true;
        for (TileWalk at(p, pair, pairs); ok && at.next(); ++q) {
            const bool a_mn = B_MN && p.w[at.work].a_mn;
            const int kb_total = p.w[at.work].kb_total(), b = q & 1;
            const uint32_t id = a_mn ? idesc_dense<I8>(2 * kTileM, BN, true, B_MN) : idesc_dense<I8>(2 * kTileM, BN, false, B_MN);
            const uint64_t step = a_mn ? 2048 >> 4 : 32 >> 4;
            if (q >= 2 && !wait_cluster(&acc_empty[b], (uint32_t)(((q >> 1) - 1) & 1), &abort_flag, p.wait_cycles)) break;
            tc_fence_after();
            for (int kb = 0; kb < kb_total; ++kb, ++c) {
                const int s = c % S;
                if (!wait_cluster(&full[s], (uint32_t)((c / S) & 1), &abort_flag, p.wait_cycles)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint8_t *sa = smem + s * R::kStage, *sb = sa + kABytes;
                const uint64_t da = a_mn ? desc_mn_sw128(sa, 8192) : desc_sw128(sa);
                const uint64_t db = B_MN ? desc_mn_sw128(sb, 8192) : desc_sw128(sb);
#pragma unroll
                for (int k = 0; k < 4; ++k)   // 32 bytes of K each: 16 bf16 or 32 s8
                    mma_pair<I8>(tmem + b * BN, da + k * step,
                                 db + k * (B_MN ? 2048 >> 4 : 32 >> 4), id, (kb | k) != 0);
                commit_pair(&empty[s]);
            }
            if (ok) commit_pair(&acc_full[b]);
        }
        // MMAs in flight end before the tensor memory goes away, whichever role gives up and when
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&done))
                     : "memory");
        mbar_wait_bounded(&done, 0, kDrainCycles);
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads lanes 32 (w % 4).., columns by halves
        const int e = warp - 4, quad = e & 3, half = e >> 2;
        uint8_t *stage = stage_out + e * 4096;
        float *scales = reinterpret_cast<float *>(stage_out + kEpiWarps * 4096 + e * kScaleBytes);
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        int q = 0;
        for (TileWalk at(p, pair, pairs); at.next(); ++q) {
            const TcWork &w = p.w[at.work];
            const int b = q & 1;
            if (!warp_wait_abort(&acc_full[b], (uint32_t)((q >> 1) & 1), &abort_flag, p.wait_cycles)) break;
            tc_fence_after();
            const long long m0 = (long long)at.m * 2 * kTileM + rank * kTileM + quad * 32, n0 = (long long)at.n * kOutN;
            const int rows = (int)min(32LL, w.M - m0);
            const float sx = I8 && lane < rows ? __ldg(p.a_scale + m0 + lane) : 0.f;
            O *out = static_cast<O *>(w.out[at.z]);
#pragma unroll 1
            for (int c0 = half * (kOutN / 2); c0 < (half + 1) * (kOutN / 2); c0 += 32) {
                const long long n = n0 + c0;
                const int cols = (int)max(0LL, min(32LL, w.N - n));
                uint32_t r0[32], r1[32];
                tmem_ld32(lane_base + b * BN + c0, r0);
                if (EPI != EPI_STORE) tmem_ld32(lane_base + b * BN + BN / 2 + c0, r1);
                tmem_ld_wait();
                if (rows <= 0 || cols <= 0) continue;
                float g[32], u[32];
                if (I8) {   // one load of the channel scales a lane, read back as broadcasts
#pragma unroll
                    for (int h = 0; h < (EPI == EPI_STORE ? 1 : 2); ++h) {
                        __syncwarp();
                        scales[lane] = lane < cols ? __ldg(p.b_scale[h] + n + lane) : 0.f;
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (h == 0) g[i] = (float)(int)r0[i] * sx * scales[i];
                            else u[i] = (float)(int)r1[i] * sx * scales[i];
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        g[i] = __uint_as_float(r0[i]);
                        if (EPI != EPI_STORE) u[i] = __uint_as_float(r1[i]);
                    }
                }
                if (EPI == EPI_STORE) {
                    store_32x32<O>(stage, g, out + m0 * w.old[at.z] + n, w.old[at.z], rows, cols, w.vec_out);
                } else if (EPI == EPI_GLU) {
                    if (!I8 && p.keep[0]) {
                        store_32x32<O>(stage, g, static_cast<O *>(p.keep[0]) + m0 * p.kld + n, p.kld, rows, cols, p.vec_keep);
                        store_32x32<O>(stage, u, static_cast<O *>(p.keep[1]) + m0 * p.kld + n, p.kld, rows, cols, p.vec_keep);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) g[i] = silu<sizeof(O) == 2>(g[i]) * u[i];
                    store_32x32<O>(stage, g, out + m0 * w.old[0] + n, w.old[0], rows, cols, w.vec_out);
                } else {
                    if constexpr (sizeof(O) == 2) {
                        float d[32];
                        load_32x32(d, static_cast<const O *>(p.dh) + m0 * p.dhld + n, p.dhld, rows, w.N - n, n > 0, p.vec_dh);
#pragma unroll
                        for (int i = 0; i < 32; ++i) glu_grad<true>(g[i], u[i], d[i], g[i], u[i]);
                    }
                    store_32x32<O>(stage, g, static_cast<O *>(p.keep[0]) + m0 * p.kld + n, p.kld, rows, cols, p.vec_keep);
                    store_32x32<O>(stage, u, static_cast<O *>(p.keep[1]) + m0 * p.kld + n, p.kld, rows, cols, p.vec_keep);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(in_cta(&acc_empty[b], 0));
        }
    }
    tc_fence_before();
    __syncthreads();
    // the other SM's arrivals and loads have ended too (bounded waits above); the results need no order here
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    tc_fence_after();
    if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, FLAG_TIMEOUT);
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
}

template <bool I8, bool B_MN, int EPI, int BN, typename O>
cudaError_t launch_t(const Product *ps, int n, int sms, cudaStream_t s) {
    constexpr int kKE = I8 ? 128 : 64, es = I8 ? 1 : 2, so = (int)sizeof(O);
    constexpr int kOutN = EPI == EPI_STORE ? BN : BN / 2;
    typedef Ring<BN> R;
    TcArgs a{};
    cudaError_t e = cudaSuccess;
    a.nwork = n;
    for (int j = 0; j < n; ++j) {
        const Product &p = ps[j];
        TcWork &w = a.w[j];
        w.a_mn = p.a_t;
        const int na = p.nseg > 1 || p.nbatch > 1 ? 2 : 1, nb = EPI == EPI_STORE ? p.nseg : 2;
        for (int i = 0; i < na && e == cudaSuccess; ++i)
            e = p.a_t ? make_map(&w.a[i], p.a[i], p.K, p.M, p.ald, es, 64)
                      : make_map(&w.a[i], p.a[i], p.M, p.K, p.ald, es, kTileM);
        for (int i = 0; i < nb && e == cudaSuccess; ++i)
            e = B_MN ? make_map(&w.b[i], p.b[i], p.K, p.N, p.bld[i], es, 64)
                     : make_map(&w.b[i], p.b[i], p.N, p.K, p.bld[i], es, BN / 2);
        if (e != cudaSuccess) return e;
        w.M = p.M;
        w.N = p.N;
        w.kblocks = (int)((p.K + kKE - 1) / kKE);
        w.nseg = p.nseg;
        w.nbatch = p.nbatch;
        w.mt = (int)((p.M + 2 * kTileM - 1) / (2 * kTileM));
        w.nt = (int)((p.N + kOutN - 1) / kOutN);
        w.vec_out = true;
        for (int i = 0; i < 2; ++i) {
            w.out[i] = p.out[i];
            w.old[i] = p.old[i];
            if (p.out[i] && (((uintptr_t)p.out[i] & 15u) || (p.old[i] * so & 15))) w.vec_out = false;
        }
        if ((long long)w.mt * w.nt * w.nbatch > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
    }
    const Product &p = ps[0];
    for (int i = 0; i < 2; ++i) {
        a.b_scale[i] = p.b_scale[i];
        a.keep[i] = p.keep[i];
    }
    a.a_scale = p.a_scale;
    a.kld = p.kld;
    a.dh = p.dh;
    a.dhld = p.dhld;
    a.vec_keep = !((uintptr_t)p.keep[0] & 15u) && !((uintptr_t)p.keep[1] & 15u) && !(p.kld * so & 15);
    a.vec_dh = !((uintptr_t)p.dh & 15u) && !(p.dhld * so & 15);
    long long tiles = a.w[0].tiles();
    if (n > 1) {
        tiles += a.w[1].tiles();
        a.extra = a.w[0].kb_total() / a.w[1].kb_total();
    }
    a.wait_cycles = wait_cycles();
    e = status_word(&a.status);
    if (e != cudaSuccess) return e;
    const auto kernel = product_tc_kernel<I8, B_MN, EPI, BN, O>;
    {
        static std::mutex mu;
        static bool ready[64] = {};
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)R::kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    const int pairs = (int)std::min<long long>(tiles, sms / 2);
    return launch_pdl(kernel, dim3((unsigned)(2 * pairs)), kThreads, R::kSmem, 0, s, a);
}

template <bool I8, bool B_MN, int EPI, typename O>
cudaError_t launch_bn(const Product *ps, int n, cudaStream_t s) {
    int sms = 0, bn = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    tc_ns(ps, n, sms, &bn);
    return bn == 256 ? launch_t<I8, B_MN, EPI, 256, O>(ps, n, sms, s) : launch_t<I8, B_MN, EPI, 128, O>(ps, n, sms, s);
}

__device__ uint32_t g_status;

}  // namespace

cudaError_t status_word(uint32_t **p) {
    static std::mutex mu;
    static uint32_t *at[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && at[dev]) {
        *p = at[dev];
        return cudaSuccess;
    }
    void *q = nullptr;
    e = cudaGetSymbolAddress(&q, g_status);
    if (e == cudaSuccess) {
        *p = static_cast<uint32_t *>(q);
        if (dev < 64) at[dev] = *p;
    }
    return e;
}

namespace {
std::atomic<long long> g_wait_cycles{0};   // 0: not read yet
}
void read_wait_cycles() {
    const char *e = std::getenv("MOEQ_TEST_WAIT_CYCLES");
    const long long v = e ? std::atoll(e) : 0;
    g_wait_cycles.store(v > 0 ? v : kWaitCycles, std::memory_order_relaxed);
}
long long wait_cycles() {
    if (!g_wait_cycles.load(std::memory_order_relaxed)) read_wait_cycles();
    return g_wait_cycles.load(std::memory_order_relaxed);
}

cudaError_t sm_count(int *n) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
    return e;
}

namespace {
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
                   const cuuint64_t *strides, const cuuint32_t *box) {
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
        f = reinterpret_cast<EncodeFn>(p);
        fn.store(f, std::memory_order_release);
    }
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = f(map, type, rank, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
}  // namespace

cudaError_t make_map(CUtensorMap *map, const void *base, long long rows, long long cols, long long ld, int es,
                     int box_rows) {
    // a single row has no stride of its own
    const long long pitch = rows > 1 ? ld * es : (cols * es + 15) / 16 * 16;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / es), (cuuint32_t)box_rows};
    return encode(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
                  box);
}

cudaError_t make_planes_map(CUtensorMap *map, const Planes &m, int box_rows, int box_planes) {
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, 3};
    const cuuint64_t strides[2] = {(cuuint64_t)m.ld * 2, (cuuint64_t)(m.rows * m.ld) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_planes};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, m.p, dims, strides, box);
}

// Measured: a K block of a 256-column tile takes 300 ns with most pairs busy, of
// a 128-column tile 250 (both are fed at 38 to 47 bytes a clock and SM from L2,
// and the narrow tile needs 1.5 times the bytes per flop), and a tile no less
// than its epilogue, 1.5 or 0.8 us.
long long tc_ns(const Product *ps, int n, int sms, int *bn) {
    const long long pairs = sms / 2;
    long long best = 0;
    for (int h = 0; h < 2; ++h) {
        const long long cols = (ps[0].epi == EPI_STORE ? 256 : 128) >> h;
        long long work = 0, longest = 0, least = 0;   // of all tiles; of the rounds of one product; of its last tiles
        for (int j = 0; j < n; ++j) {
            const int ke = ps[j].in_dtype == kI8 ? 128 : 64;
            const long long tiles = (ps[j].M + 255) / 256 * ((ps[j].N + cols - 1) / cols) * ps[j].nbatch;
            const long long tile = std::max<long long>((ps[j].K + ke - 1) / ke * ps[j].nseg * (h ? 250 : 300), h ? 800 : 1500);
            work += tiles * tile;
            longest = std::max(longest, (tiles + pairs - 1) / pairs * tile);
            least = j ? std::min(least, tile) : tile;
        }
        const long long t = std::max(longest, (work + pairs * least - 1) / (pairs * least) * least);
        if (h == 0 || t < best) {
            best = t;
            *bn = h ? 128 : 256;
        }
    }
    return best;
}

cudaError_t launch_product_tc(const Product &p, cudaStream_t s) {
    typedef __nv_bfloat16 B;
    if (p.keep_f32) return cudaErrorInvalidValue;   // keep is written in out_dtype
    if (p.in_dtype == kI8) {
        if (p.epi == EPI_GLU)
            return p.out_dtype == MOEQ_ACT_F32 ? launch_bn<true, false, EPI_GLU, float>(&p, 1, s)
                                               : launch_bn<true, false, EPI_GLU, B>(&p, 1, s);
        return p.out_dtype == MOEQ_ACT_F32 ? launch_bn<true, false, EPI_STORE, float>(&p, 1, s)
                                           : launch_bn<true, false, EPI_STORE, B>(&p, 1, s);
    }
    if (p.epi == EPI_GLU) return launch_bn<false, false, EPI_GLU, B>(&p, 1, s);
    return launch_bn<false, false, EPI_GLU_BWD, B>(&p, 1, s);
}

cudaError_t launch_gradients_tc(const Product *dx, const Product *dw, cudaStream_t s) {
    Product p[2];
    int n = 0;
    if (dw) p[n++] = *dw;
    if (dx) p[n++] = *dx;
    if (n == 2 && (p[0].K + 63) / 64 < (p[1].K + 63) / 64 * p[1].nseg) std::swap(p[0], p[1]);   // longer tiles first
    return launch_bn<false, true, EPI_STORE, __nv_bfloat16>(p, n, s);
}

}  // namespace dense
}  // namespace moeq
