// dense_skinny.cu -- products of the dense operators on the tensor cores where
// the 256-row tiles of dense_tc.cu would be few and long: tiles of 128 weight
// rows, K split over a cluster.
//
// The roles of the operands are swapped: the weights are the MMA's M = 128
// rows, the tokens its N = 16..128 columns, so nothing is computed for rows
// that are not there.  The gated block's tile is 64 gate rows and the 64 up
// rows of the same outputs.
//
// Bound: HBM (the weights' bytes) as long as the tiles cover the SMs.  Few
// rows of tiles are made up for by splitting K over the S CTAs of a cluster,
// each with its own ring of TMA stages, so that nearly a whole CTA's share of
// the weights is in flight at once.  The CTAs' partial sums meet in
// distributed shared memory: each CTA leaves its accumulator in its own shared
// memory and, after a cluster barrier, adds up the S partials of its share of
// the tokens in rank order (no atomics, the result does not depend on timing;
// int8 sums stay exact in s32), applies scales or the activation and writes
// 256 contiguous bytes a token.
#include <algorithm>
#include <mutex>

#include "dense_tc.cuh"

namespace moeq {
namespace dense {
namespace {

using namespace umma;

constexpr int kThreads = 256;
constexpr int kABytes = kT * kRowBytes;   // 16 KB
constexpr int kMaxStages = 12;
constexpr int kSmemMax = 108 * 1024;      // two CTAs of an SM: the next kernel's wait beside this one's

struct SkinnyArgs {
    CUtensorMap a[2], b[2];    // weights (gate / up, or segments), tokens (segments, or batches)
    int T, N;                  // tokens, outputs
    int kblocks, nseg, nbatch;
    int nt;                    // tokens per tile: 16, 32, 64 or 128
    int ttiles;
    int split;                 // CTAs of a cluster
    int stages;
    const float *a_scale, *b_scale[2];   // per token, per weight row
    void *out[2];              // per batch
    long long old[2];
    void *keep[2];
    long long kld;
    const void *dh;
    long long dhld;
    long long wait_cycles;
    uint32_t *status;
};

// Tokens per tile and CTAs that share a tile's K: doubled while the tiles do
// not cover the SMs and every CTA keeps two K blocks.  Clusters of 8 only when
// there are few: 16 of them do not run at once (a GPC's SMs divided by 8), and
// the second round cost more than the split gave (4096 x 4096 x 2048 gated, 64
// tokens: 26 us with 16 clusters of 8).
struct SkinnyShape {
    int nt, split;
};
SkinnyShape skinny_shape(const Product &p, long long row_tiles, long long kblocks, int sms) {
    const long long T = p.M;
    SkinnyShape r;
    r.nt = T <= 16 && !p.a_t ? 16 : (T <= 32 && !p.a_t ? 32 : (T <= 64 ? 64 : 128));   // transposed: whole 64-element rows
    const long long tiles = (T + r.nt - 1) / r.nt * row_tiles * p.nbatch;
    r.split = 1;
    while (r.split < (tiles <= 8 ? 8 : 4) && tiles * r.split * 2 <= sms && kblocks >= r.split * 4) r.split *= 2;
    return r;
}

template <bool I8>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (I8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
__device__ __forceinline__ uint4 ld_cluster(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
template <bool I8>
__device__ __forceinline__ void add4(uint32_t s[4], const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = I8 ? s[i] + w[i] : __float_as_uint(__uint_as_float(s[i]) + __uint_as_float(w[i]));
}

template <bool I8, bool A_MN, bool B_MN, int EPI, typename O>
__global__ void __launch_bounds__(kThreads, 1) product_skinny_kernel(const __grid_constant__ SkinnyArgs p) {
    constexpr int kRows = EPI == EPI_STORE ? kT : kT / 2;   // outputs of a tile
    constexpr int kKE = I8 ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ alignas(8) uint64_t full[kMaxStages], empty[kMaxStages], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int row_tiles = (p.N + kRows - 1) / kRows, tile = blockIdx.x / p.split;
    const int t0 = (tile % p.ttiles) * p.nt, n0 = (tile / p.ttiles % row_tiles) * kRows, z = tile / p.ttiles / row_tiles;
    const int S = p.stages, stage_bytes = kABytes + p.nt * kRowBytes;
    const int total = p.kblocks * p.nseg, share = (total + p.split - 1) / p.split;
    const int kb0 = min(total, rank * share), kb1 = min(total, kb0 + share);
    const int cols = p.nt < 32 ? 32 : p.nt;   // a power of two
    int issued = 0;
    auto load = [&](int c) {
        const int kb = kb0 + c, s = c % S, seg = p.nseg > 1 && kb >= p.kblocks, k0 = (seg ? kb - p.kblocks : kb) * kKE;
        uint8_t *st = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        if (EPI != EPI_STORE) {
            tma_load_2d(st, &p.a[0], k0, n0, &full[s]);
            tma_load_2d(st + kABytes / 2, &p.a[1], k0, n0, &full[s]);
        } else if (A_MN) {
            tma_load_2d(st, &p.a[seg], n0, k0, &full[s]);
            tma_load_2d(st + 8192, &p.a[seg], n0 + 64, k0, &full[s]);
        } else {
            tma_load_2d(st, &p.a[seg], k0, n0, &full[s]);
        }
        const CUtensorMap *mb = &p.b[p.nbatch > 1 ? z : seg];
        if (B_MN) {
            for (int j = 0; j < p.nt / 64; ++j) tma_load_2d(st + kABytes + j * 8192, mb, t0 + 64 * j, k0, &full[s]);
        } else {
            tma_load_2d(st + kABytes, mb, k0, t0, &full[s]);
        }
        ++issued;
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        abort_flag = 0;
        mbar_fence_init();
        // weights of the ring's first round on their way to L2 while the kernel before drains
        for (int c = 0; c < S && c < kb1 - kb0; ++c) {
            const int kb = kb0 + c, seg = p.nseg > 1 && kb >= p.kblocks, k0 = (seg ? kb - p.kblocks : kb) * kKE;
            if (EPI != EPI_STORE) {
                tma_prefetch_2d(&p.a[0], k0, n0);
                tma_prefetch_2d(&p.a[1], k0, n0);
            } else if (A_MN) {
                tma_prefetch_2d(&p.a[seg], n0, k0);
                tma_prefetch_2d(&p.a[seg], n0 + 64, k0);
            } else {
                tma_prefetch_2d(&p.a[seg], k0, n0);
            }
        }
        pdl_wait_primary();
        while (issued < S && issued < kb1 - kb0) load(issued);   // the ring's first round waits for nothing
    }
    if (warp == 2) tc_alloc(&tmem_slot, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_primary();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;

    if (warp == 0 && lane == 0) {
        while (issued < kb1 - kb0) {
            if (!wait_cluster(&empty[issued % S], (uint32_t)((issued / S - 1) & 1), &abort_flag, p.wait_cycles)) break;
            load(issued);
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t id = idesc_dense<I8>(kT, p.nt, A_MN, B_MN);
        for (int c = 0; c < kb1 - kb0; ++c) {
            const int s = c % S;
            if (!wait_cluster(&full[s], (uint32_t)((c / S) & 1), &abort_flag, p.wait_cycles)) break;
            tc_fence_after();
            const uint8_t *st = smem + s * stage_bytes;
            const uint64_t da = A_MN ? desc_mn_sw128(st, 8192) : desc_sw128(st);
            const uint64_t db = B_MN ? desc_mn_sw128(st + kABytes, 8192) : desc_sw128(st + kABytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_one<I8>(tmem, da + k * (A_MN ? 2048 >> 4 : 32 >> 4), db + k * (B_MN ? 2048 >> 4 : 32 >> 4), id,
                             (uint32_t)(c | k) != 0);
            tc_commit(&empty[s]);
        }
        tc_commit(&done);
    }
    __syncwarp();   // the other lanes of the issuing warps do not poll beside them
    // ---- this CTA's sums into its shared memory, [token][row]: the ring is
    // free once every MMA has completed (every load has been consumed by then)
    const bool ok = mbar_wait_abort(&done, 0, &abort_flag, p.wait_cycles);
    if (!ok) mbar_wait_bounded(&done, 0, kDrainCycles);
    __syncthreads();
    if (abort_flag) {   // every wait is behind: the same for all. Copies that nobody waited for land first
        if (threadIdx.x == 0) drain_stages(full, S, issued);
        __syncthreads();
    }
    tc_fence_after();
    uint32_t *part = reinterpret_cast<uint32_t *>(smem);
    if (warp >= 4) {
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16);
        for (int c0 = 0; c0 < p.nt; c0 += 16) {
            float v[16];
            tc_ld16(base + c0, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c0 + i) * kT + row] = kb1 > kb0 ? __float_as_uint(v[i]) : 0u;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tc_dealloc(tmem, cols);
    }
    if (p.split > 1) cluster_sync();

    // ---- this CTA's share of the tokens: four outputs a lane, whole tokens (or
    // with the gated block's 64 outputs, two tokens) a warp
    constexpr int NA = EPI == EPI_STORE ? 1 : 2, kLanes = kRows / 4;   // sums of an output; lanes of a token
    const int per = p.nt / p.split;                                    // tokens
    for (int i = threadIdx.x / kLanes; i < per; i += kThreads / kLanes) {
        const int lt = rank * per + i, tok = t0 + lt, r4 = (threadIdx.x % kLanes) * 4, n = n0 + r4;
        uint32_t s[NA][4];
#pragma unroll
        for (int a = 0; a < NA; ++a) s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0;
        if (tok < p.T) {
            if (p.split > 1) {
#pragma unroll 4
                for (int r = 0; r < p.split; ++r)
#pragma unroll
                    for (int a = 0; a < NA; ++a) add4<I8>(s[a], ld_cluster(in_cta(part + lt * kT + a * kRows + r4, r)));
            } else {
#pragma unroll
                for (int a = 0; a < NA; ++a)
                    add4<I8>(s[a], *reinterpret_cast<const uint4 *>(part + lt * kT + a * kRows + r4));
            }
            float v[NA][4];
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[a][j] = I8 ? (float)(int)s[a][j] * __ldg(p.a_scale + tok) * (n + j < p.N ? __ldg(p.b_scale[a] + n + j) : 0.f)
                                 : __uint_as_float(s[a][j]);
            auto put = [&](void *dst, long long ld, const float *w) {
                O *d = static_cast<O *>(dst) + (long long)tok * ld + n;
                if (n + 4 <= p.N && !((uintptr_t)d & (4 * sizeof(O) - 1))) {
                    alignas(16) O e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) st_elem(e + j, w[j]);
                    if (sizeof(O) == 4) *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(e);
                    else *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<const uint2 *>(e);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < p.N) st_elem(d + j, w[j]);
                }
            };
            if (EPI == EPI_STORE) {
                put(p.out[z], p.old[z], v[0]);
            } else if (EPI == EPI_GLU) {
                if (!I8 && p.keep[0]) {
                    put(p.keep[0], p.kld, v[0]);
                    put(p.keep[1], p.kld, v[NA - 1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[0][j] = silu<sizeof(O) == 2>(v[0][j]) * v[NA - 1][j];
                put(p.out[0], p.old[0], v[0]);
            } else {
                const O *dh = static_cast<const O *>(p.dh) + (long long)tok * p.dhld + n;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = n + j < p.N ? ld_elem(dh + j) : 0.f;
                    glu_grad<sizeof(O) == 2>(v[0][j], v[NA - 1][j], d, v[0][j], v[NA - 1][j]);
                }
                put(p.keep[0], p.kld, v[0]);
                put(p.keep[1], p.kld, v[NA - 1]);
            }
        }
    }
    // no CTA leaves while another reads its shared memory; the stores above need no order
    __syncwarp();
    if (p.split > 1)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, FLAG_TIMEOUT);
}

template <bool I8, bool A_MN, bool B_MN, int EPI, typename O>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    constexpr int kRows = EPI == EPI_STORE ? kT : kT / 2, es = I8 ? 1 : 2, kKE = I8 ? 128 : 64;
    SkinnyArgs a{};
    a.T = (int)p.M;
    a.N = (int)p.N;
    a.kblocks = (int)((p.K + kKE - 1) / kKE);
    a.nseg = p.nseg;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const SkinnyShape sh = skinny_shape(p, (p.N + kRows - 1) / kRows, (long long)a.kblocks * a.nseg, sms);
    a.nt = sh.nt;
    a.split = sh.split;
    a.ttiles = (int)((p.M + a.nt - 1) / a.nt);
    const int na = EPI == EPI_STORE ? p.nseg : 2;
    for (int i = 0; i < na && e == cudaSuccess; ++i)
        e = A_MN ? make_map(&a.a[i], p.b[i], p.K, p.N, p.bld[i], es, 64)
                 : make_map(&a.a[i], p.b[i], p.N, p.K, p.bld[i], es, kRows);
    a.nbatch = p.nbatch;
    for (int i = 0; i < std::max(p.nseg, p.nbatch) && e == cudaSuccess; ++i)
        e = B_MN ? make_map(&a.b[i], p.a[i], p.K, p.M, p.ald, es, 64) : make_map(&a.b[i], p.a[i], p.M, p.K, p.ald, es, a.nt);
    if (e == cudaSuccess) e = status_word(&a.status);
    if (e != cudaSuccess) return e;
    a.wait_cycles = wait_cycles();
    a.a_scale = p.a_scale;
    for (int i = 0; i < 2; ++i) {
        a.b_scale[i] = p.b_scale[i];
        a.keep[i] = p.keep[i];
        a.out[i] = p.out[i];
        a.old[i] = p.old[i];
    }
    a.kld = p.kld;
    a.dh = p.dh;
    a.dhld = p.dhld;
    const int stage = kABytes + a.nt * kRowBytes;
    const int share = (a.kblocks * a.nseg + a.split - 1) / a.split;
    a.stages = std::max(1, std::min(std::min(kMaxStages, share), kSmemMax / stage));
    const size_t smem = 1024 + (size_t)std::max(a.stages * stage, a.nt * kT * 4);
    const auto kernel = product_skinny_kernel<I8, A_MN, B_MN, EPI, O>;
    {
        static std::mutex mu;
        static bool ready[64] = {};
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax + 1024);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    const dim3 grid((unsigned)(a.ttiles * ((a.N + kRows - 1) / kRows) * a.nbatch * a.split));
    return launch_pdl(kernel, grid, kThreads, smem, a.split, s, a);
}

}  // namespace

// Measured: 430 ns a K block of a CTA (the feed of its 24 to 32 KB), 0.7 us for
// the cluster's exchange, 2.5 us for the start and end of every further round.
long long skinny_ns(const Product &p, int sms) {
    const int ke = p.in_dtype == kI8 ? 128 : 64;
    const long long rows = p.epi == EPI_STORE ? kT : kT / 2, row_tiles = (p.N + rows - 1) / rows;
    const long long kb = (p.K + ke - 1) / ke * p.nseg;
    const SkinnyShape sh = skinny_shape(p, row_tiles, kb, sms);
    const long long tiles = (p.M + sh.nt - 1) / sh.nt * row_tiles * p.nbatch;
    const long long rounds = (tiles * sh.split + sms - 1) / sms;
    return rounds * ((kb + sh.split - 1) / sh.split) * 430 + 700 + (rounds - 1) * 2500;
}

cudaError_t launch_product_skinny(const Product &p, cudaStream_t s) {
    typedef __nv_bfloat16 B;
    if (p.keep_f32) return cudaErrorInvalidValue;   // keep is written in out_dtype
    if (p.in_dtype == kI8) {
        if (p.epi == EPI_GLU)
            return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, false, false, EPI_GLU, float>(p, s)
                                               : launch_t<true, false, false, EPI_GLU, B>(p, s);
        return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, false, false, EPI_STORE, float>(p, s)
                                           : launch_t<true, false, false, EPI_STORE, B>(p, s);
    }
    if (p.epi == EPI_GLU) return launch_t<false, false, false, EPI_GLU, B>(p, s);
    if (p.epi == EPI_GLU_BWD) return launch_t<false, false, false, EPI_GLU_BWD, B>(p, s);
    return p.a_t ? launch_t<false, true, true, EPI_STORE, B>(p, s) : launch_t<false, true, false, EPI_STORE, B>(p, s);
}

}  // namespace dense
}  // namespace moeq
