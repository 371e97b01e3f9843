// dense_planes.cu -- f32 products of the dense operators on the tensor cores,
// from bf16 planes: x = hi + mid + lo, each part the nearest bf16 of what is
// left (8 significand bits a part; a bf16's smallest step is 2^-133, so the three
// hold all 24 bits of an f32 of 2^-110 and above).
//
// Mathematics: x w ~ hi hi + (hi mid + mid hi + hi lo + lo hi + mid mid); the
// products left out are below 2^-24 of |x w| (2^-27.5 rms).  The tensor core adds in f32 with
// truncation, which in a long sum loses about 2^-24 of the running value a
// step of 16 products, always towards zero (measured on sums of normal values:
// 9e-8 relative after 64 products, 6e-7 after 512, 4.8e-6 after 4096).  So the
// hi hi sum runs over kChunk K blocks (128 products) only and is then added to
// the total on the f32 units, two accumulators taking turns; the five small
// products share an accumulator of their own that is 2^-8 as large and is left
// to run.
//
// Bound: the tensor cores at six bf16 products an f32 one, and the feed of the
// planes (72 KB a K block for 128 x 64 outputs).  As in dense_skinny.cu a tile
// is 128 rows of one operand (64 gate and 64 up rows of the same outputs for
// the gated block) by 64 of the other, K is split over a cluster where the
// tiles do not cover the SMs, and the CTAs' sums meet in distributed shared
// memory in rank order.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "dense_tc.cuh"

namespace moeq {
namespace dense {
namespace {

using namespace umma;

constexpr int kThreads = 256;
constexpr int kNT = 64;                          // rows of B a tile
constexpr int kABytes = 3 * kT * kRowBytes;      // 48 KB: three planes
constexpr int kBBytes = 3 * kNT * kRowBytes;     // 24 KB
constexpr int kStage = kABytes + kBBytes;
constexpr int kStages = 3;
constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
constexpr int kChunk = 2;                        // K blocks of a hi hi sum
constexpr int kTmem = 256;                       // columns: hi hi twice, the small products, unused

struct PlanesWork {
    CUtensorMap a[2], b[2];    // A: gate / up, or segments; B: segments, or batches
    long long M, N;            // rows of B (rows of out), rows of A (columns of out)
    int kblocks, nseg, nbatch;
    int mtiles, ntiles, split; // split: CTAs that share a tile's K
    bool b_mn;                 // B stored [K][M]
    void *out[2];
    long long old[2];
};
struct PlanesArgs {
    PlanesWork w[2];           // dx and dW in one launch, or one work
    int clusters0, size;       // clusters of work 0; CTAs of a cluster: size / split tiles of a work
    void *keep[2];             // EPI_GLU: f32; EPI_GLU_BWD: planes
    long long kld, kplane;
    const float *dh;
    long long dhld;
    long long wait_cycles;
    uint32_t *status;
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The three parts of x.  An infinity or NaN is its own first part; a finite x
// whose nearest bf16 is infinite is cut off instead.
__device__ __forceinline__ void planes_of(float x, __nv_bfloat16 p[3]) {
    const uint32_t bits = __float_as_uint(x);
    const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
    p[0] = __float2bfloat16_rn(x);
    if (finite && (__bfloat16_as_ushort(p[0]) & 0x7F80u) == 0x7F80u) p[0] = __ushort_as_bfloat16((unsigned short)(bits >> 16));
    const float r = finite ? x - __bfloat162float(p[0]) : 0.f;
    p[1] = __float2bfloat16_rn(r);
    p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}
// p[0..3] of 4 consecutive outputs into the planes at d, d + plane, d + 2 plane
__device__ __forceinline__ void put_planes(__nv_bfloat16 *d, long long plane, const float v[4], int cols) {
    __nv_bfloat16 p[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) planes_of(v[j], p[j]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < cols) d[q * plane + j] = p[j][q];
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 1) product_planes_kernel(const __grid_constant__ PlanesArgs p) {
    constexpr bool A_MN = EPI == EPI_STORE;                 // dx, dW: A stored [K][N]
    constexpr int kRows = EPI == EPI_STORE ? kT : kT / 2;   // outputs (columns of out) of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ alignas(8) uint64_t full[kStages], empty[kStages], main_full[2], main_empty[2], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int in_cluster = p.size > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / p.size;
    const PlanesWork &w = p.w[cluster >= p.clusters0];
    const bool b_mn = A_MN && w.b_mn;
    const int split = w.split, rank = in_cluster % split, first = in_cluster - rank;   // first: the tile's first CTA
    int tile = (cluster >= p.clusters0 ? cluster - p.clusters0 : cluster) * (p.size / split) + in_cluster / split;
    const bool live = tile < w.mtiles * w.ntiles * w.nbatch;   // a cluster's last tiles may not be there
    const int m0 = tile % w.mtiles * kNT;
    tile /= w.mtiles;
    const int n0 = tile % w.ntiles * kRows, z = live ? tile / w.ntiles : 0;
    const int total = live ? w.kblocks * w.nseg : 0, share = (total + split - 1) / split;
    const int kb0 = min(total, rank * share), kbs = min(total, kb0 + share) - kb0;
    const int chunks = (kbs + kChunk - 1) / kChunk;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&main_full[i], 1);
            mbar_init(&main_empty[i], 4);
        }
        mbar_init(&done, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 2) tc_alloc(&tmem_slot, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_primary();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;
    float tot[kNT];
#pragma unroll
    for (int i = 0; i < kNT; ++i) tot[i] = 0.f;

    int issued = 0;   // loads, by thread 0
    if (warp == 0 && lane == 0) {
        for (; issued < kbs; ++issued) {
            const int c = issued, s = c % kStages, kb = kb0 + c, seg = w.nseg > 1 && kb >= w.kblocks, k0 = (seg ? kb - w.kblocks : kb) * 64;
            if (c >= kStages && !wait_cluster(&empty[s], (uint32_t)((c / kStages - 1) & 1), &abort_flag, p.wait_cycles)) break;
            uint8_t *sa = smem + s * kStage, *sb = sa + kABytes;
            mbar_arrive_expect_tx(&full[s], kStage);
            if (A_MN) {   // [64 columns][plane][64 rows of K]
                tma_load_3d(sa, &w.a[seg], n0, k0, 0, &full[s]);
                tma_load_3d(sa + kABytes / 2, &w.a[seg], n0 + 64, k0, 0, &full[s]);
            } else {      // [plane][gate rows, up rows]
#pragma unroll
                for (int q = 0; q < 3; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(sa + q * (kABytes / 3) + h * (kABytes / 6), &w.a[h], k0, n0, q, &full[s]);
            }
            const CUtensorMap *mb = &w.b[w.nbatch > 1 ? z : seg];
            if (b_mn) tma_load_3d(sb, mb, m0, k0, 0, &full[s]);
            else tma_load_3d(sb, mb, k0, m0, 0, &full[s]);
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t id = b_mn ? idesc_dense<false>(kT, kNT, A_MN, true) : idesc_dense<false>(kT, kNT, A_MN, false);
        const uint64_t bstep = b_mn ? 2048 >> 4 : 32 >> 4;
        bool ok = true;
        for (int c = 0; ok && c < kbs; ++c) {
            const int s = c % kStages, q = c / kChunk, buf = q & 1;
            if (c % kChunk == 0 && q >= 2 &&
                !wait_cluster(&main_empty[buf], (uint32_t)(((q >> 1) - 1) & 1), &abort_flag, p.wait_cycles))
                break;
            if (!wait_cluster(&full[s], (uint32_t)((c / kStages) & 1), &abort_flag, p.wait_cycles)) break;
            tc_fence_after();
            const uint8_t *sa = smem + s * kStage, *sb = sa + kABytes;
            uint64_t da[3], db[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                da[i] = A_MN ? desc_mn_sw128(sa + i * 8192, kABytes / 2) : desc_sw128(sa + i * (kABytes / 3));
                db[i] = b_mn ? desc_mn_sw128(sb + i * 8192, 8192) : desc_sw128(sb + i * 8192);
            }
            // (part of A, part of B): the small products, then hi hi
            constexpr int pa[6] = {1, 0, 2, 0, 1, 0}, pb[6] = {1, 2, 0, 1, 0, 0};
#pragma unroll
            for (int o = 0; o < 6; ++o)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16(o == 5 ? tmem + buf * kNT : tmem + 2 * kNT, da[pa[o]] + k * (A_MN ? 2048 >> 4 : 32 >> 4),
                             db[pb[o]] + k * bstep, id,
                             o == 5 ? (uint32_t)(c % kChunk | k) != 0 : (uint32_t)(c | o | k) != 0);
            tc_commit(&empty[s]);
            if (c % kChunk == kChunk - 1 || c == kbs - 1) tc_commit(&main_full[buf]);
        }
        tc_commit(&done);
    } else if (warp >= 4) {
        const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        for (int q = 0; q < chunks; ++q) {
            if (!warp_wait_abort(&main_full[q & 1], (uint32_t)((q >> 1) & 1), &abort_flag, p.wait_cycles)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < kNT / 32; ++h) {
                uint32_t r[32];
                tmem_ld32(base + (q & 1) * kNT + 32 * h, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) tot[32 * h + i] += __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&main_empty[q & 1]);
        }
    }
    __syncwarp();
    const bool ok = mbar_wait_abort(&done, 0, &abort_flag, p.wait_cycles);
    if (!ok) mbar_wait_bounded(&done, 0, kDrainCycles);
    __syncthreads();   // every load has been consumed: the ring is free
    if (abort_flag) {   // or not: copies that nobody waited for land first. Every wait is behind: the same for all
        if (threadIdx.x == 0) drain_stages(full, kStages, issued);
        __syncthreads();
    }
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);   // [row of B][row of A]
    if (warp >= 4) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 2 * kNT;
#pragma unroll
        for (int h = 0; h < kNT / 32; ++h) {
            uint32_t r[32];
            tmem_ld32(base + 32 * h, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                part[(32 * h + i) * kT + row] = kbs > 0 ? tot[32 * h + i] + __uint_as_float(r[i]) : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tc_dealloc(tmem, kTmem);
    }
    if (p.size > 1) cluster_sync();

    // ---- this CTA's share of the rows of out: four columns a lane
    constexpr int NA = EPI == EPI_STORE ? 1 : 2, kLanes = kRows / 4;
    const int per = live ? kNT / split : 0;
    for (int i = threadIdx.x / kLanes; i < per; i += kThreads / kLanes) {
        const int lm = rank * per + i, r4 = (threadIdx.x % kLanes) * 4;
        const long long m = m0 + lm, n = n0 + r4;
        const int cols = (int)min(4LL, w.N - n);
        if (m >= w.M) continue;
        float v[NA][4] = {};
        for (int r = 0; r < split; ++r)
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                const float *src = part + lm * kT + a * kRows + r4;
                const float4 q = split > 1 ? ld_cluster_f4(in_cta(src, first + r)) : *reinterpret_cast<const float4 *>(src);
                v[a][0] += q.x, v[a][1] += q.y, v[a][2] += q.z, v[a][3] += q.w;
            }
        auto put = [&](void *dst, long long ld, const float *q) {
            float *d = static_cast<float *>(dst) + m * ld + n;
            if (cols == 4 && !((uintptr_t)d & 15u)) *reinterpret_cast<float4 *>(d) = make_float4(q[0], q[1], q[2], q[3]);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < cols) d[j] = q[j];
        };
        if (EPI == EPI_STORE) put(w.out[z], w.old[z], v[0]);
        if (EPI == EPI_GLU) {
            if (p.keep[0]) {
                put(p.keep[0], p.kld, v[0]);
                put(p.keep[1], p.kld, v[NA - 1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[0][j] = silu<false>(v[0][j]) * v[NA - 1][j];
            put(w.out[0], w.old[0], v[0]);
        }
        if (EPI == EPI_GLU_BWD) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                glu_grad<false>(v[0][j], v[NA - 1][j], j < cols ? __ldg(p.dh + m * p.dhld + n + j) : 0.f, v[0][j],
                                v[NA - 1][j]);
            put_planes(static_cast<__nv_bfloat16 *>(p.keep[0]) + m * p.kld + n, p.kplane, v[0], cols);
            put_planes(static_cast<__nv_bfloat16 *>(p.keep[1]) + m * p.kld + n, p.kplane, v[NA - 1], cols);
        }
    }
    __syncwarp();
    if (p.size > 1)   // no CTA leaves while another reads its shared memory
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, FLAG_TIMEOUT);
}

template <int EPI>
cudaError_t launch_t(const PlanesProduct *ps, int nwork, cudaStream_t s) {
    constexpr int kRows = EPI == EPI_STORE ? kT : kT / 2;
    PlanesArgs a{};
    int sms = 0;
    cudaError_t e = status_word(&a.status);
    if (e == cudaSuccess) e = sm_count(&sms);
    a.wait_cycles = wait_cycles();
    a.size = 1;
    for (int j = 0; j < nwork && e == cudaSuccess; ++j) {
        const PlanesProduct &p = ps[j];
        PlanesWork &w = a.w[j];
        const int na = EPI == EPI_STORE ? p.nseg : 2, nb = std::max(p.nseg, p.nbatch);
        for (int i = 0; i < na && e == cudaSuccess; ++i)
            e = EPI == EPI_STORE ? make_planes_map(&w.a[i], p.b[i], 64, 3) : make_planes_map(&w.a[i], p.b[i], kRows, 1);
        for (int i = 0; i < nb && e == cudaSuccess; ++i) e = make_planes_map(&w.b[i], p.a[i], 64, 3);
        w.M = p.M;
        w.N = p.N;
        w.kblocks = (int)((p.K + 63) / 64);
        w.nseg = p.nseg;
        w.nbatch = p.nbatch;
        w.b_mn = p.a_t;
        w.mtiles = (int)((p.M + kNT - 1) / kNT);
        w.ntiles = (int)((p.N + kRows - 1) / kRows);
        const long long tiles = (long long)w.mtiles * w.ntiles * p.nbatch;
        if (tiles > 0x0FFFFFFF) return cudaErrorInvalidConfiguration;
        // of its own sizes alone: what else a launch computes changes no bits
        w.split = 1;
        while (w.split < (tiles <= 8 ? 8 : 4) && tiles * w.split * 2 <= sms && (long long)w.kblocks * w.nseg >= w.split * 2)
            w.split *= 2;
        a.size = std::max(a.size, w.split);
        for (int i = 0; i < 2; ++i) {
            w.out[i] = p.out[i];
            w.old[i] = p.old[i];
        }
    }
    if (e != cudaSuccess) return e;
    long long clusters = 0;
    for (int j = 0; j < nwork; ++j) {
        const int per = a.size / a.w[j].split, tiles = a.w[j].mtiles * a.w[j].ntiles * a.w[j].nbatch;
        clusters += (tiles + per - 1) / per;
        if (j == 0) a.clusters0 = (int)clusters;
    }
    const PlanesProduct &p = ps[0];
    for (int i = 0; i < 2; ++i) a.keep[i] = p.keep[i];
    a.kld = p.kld;
    a.kplane = p.kplane;
    a.dh = p.dh;
    a.dhld = p.dhld;
    const auto kernel = product_planes_kernel<EPI>;
    {
        static std::mutex mu;
        static bool ready[64] = {};
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    return launch_pdl(kernel, dim3((unsigned)(clusters * a.size)), kThreads, kSmem, a.size, s, a);
}

struct SplitArgs {
    const float *src[3];
    __nv_bfloat16 *dst[3];
    long long ld[3], dst_ld[3], rows[3];
    int cols[3];
};
// f32 matrices into their planes, four columns a thread (bandwidth bound: 4
// bytes in, 6 out an element)
__global__ void __launch_bounds__(128) split_kernel(const __grid_constant__ SplitArgs p) {
    const int z = blockIdx.z, c = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (c >= p.cols[z]) return;
    const long long plane = p.rows[z] * p.dst_ld[z];
    for (long long r = blockIdx.y * blockDim.y + threadIdx.y; r < p.rows[z]; r += gridDim.y * blockDim.y) {
        const float *s = p.src[z] + r * p.ld[z] + c;
        float v[4];
        if (c + 4 <= p.cols[z] && !((uintptr_t)s & 15u)) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(s));
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = c + i < p.cols[z] ? __ldg(s + i) : 0.f;
        }
        alignas(8) __nv_bfloat16 q[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat16 t[3];
            planes_of(v[i], t);
            q[0][i] = t[0], q[1][i] = t[1], q[2][i] = t[2];
        }
        __nv_bfloat16 *d = p.dst[z] + r * p.dst_ld[z] + c;   // the padded row holds whole pieces
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(d + i * plane) = *reinterpret_cast<const uint2 *>(q[i]);
    }
}

// the gradients of kept projections, into planes
__global__ void __launch_bounds__(128) dgate_planes_kernel(const float *__restrict__ dh, long long dhld,
                                                           const float *__restrict__ g, const float *__restrict__ u,
                                                           __nv_bfloat16 *__restrict__ dg, __nv_bfloat16 *__restrict__ du,
                                                           long long ld, long long M, long long N) {
    const long long n = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 4;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (n >= N) return;
    const int cols = (int)min(4LL, N - n);
    for (long long m = blockIdx.y * blockDim.y + threadIdx.y; m < M; m += gridDim.y * blockDim.y) {
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = b[j] = 0.f;
            if (j < cols)
                glu_grad<false>(__ldg(g + m * N + n + j), __ldg(u + m * N + n + j), __ldg(dh + m * dhld + n + j), a[j], b[j]);
        }
        put_planes(dg + m * ld + n, M * ld, a, cols);
        put_planes(du + m * ld + n, M * ld, b, cols);
    }
}

}  // namespace

cudaError_t launch_split(const Copy *c, int n, cudaStream_t s) {
    SplitArgs a{};
    long long pieces = 1, rows = 1;
    for (int i = 0; i < n; ++i) {
        a.src[i] = static_cast<const float *>(c[i].src);
        a.dst[i] = static_cast<__nv_bfloat16 *>(c[i].dst);
        a.ld[i] = c[i].ld;
        a.dst_ld[i] = c[i].dst_ld;
        a.rows[i] = c[i].rows;
        a.cols[i] = (int)c[i].cols;
        pieces = std::max<long long>(pieces, (c[i].cols + 3) / 4);
        rows = std::max(rows, c[i].rows);
    }
    const RowGrid g(rows, pieces, n);
    return launch_pdl(split_kernel, g.grid, g.block, 0, 0, s, a);
}

cudaError_t launch_dgate_planes(const float *dh, long long dhld, const float *gu, void *dg, void *du, long long ld,
                                long long M, long long N, cudaStream_t s) {
    const RowGrid r(M, (N + 3) / 4);
    return launch_pdl(dgate_planes_kernel, r.grid, r.block, 0, 0, s, dh, dhld, gu, gu + M * N, static_cast<__nv_bfloat16 *>(dg),
                      static_cast<__nv_bfloat16 *>(du), ld, M, N);
}

cudaError_t launch_product_planes(const PlanesProduct &p, cudaStream_t s) {
    return p.epi == EPI_GLU ? launch_t<EPI_GLU>(&p, 1, s) : launch_t<EPI_GLU_BWD>(&p, 1, s);
}
cudaError_t launch_gradients_planes(const PlanesProduct *p, int n, cudaStream_t s) { return launch_t<EPI_STORE>(p, n, s); }

}  // namespace dense
}  // namespace moeq
