// dense_simt.cu -- f32 products of the dense operators (any sizes, strides and
// alignment), and the elementwise steps around the products.
//
// Bound: the f32 units (128 fma a clock and SM; fma.rn.f32x2 does two with one
// instruction, which leaves issue slots for the shared-memory loads).  A CTA
// of 256 threads computes a tile of 16 TM x 64 outputs (32 gate and the 32 up
// of the same outputs for the gated block), TM x 4 a thread, from slices of 16
// along K that are copied into a ring of shared-memory stages (4-byte
// asynchronous copies: any stride and alignment, transposed on the way).  TM = 8 reads 3 x 16 bytes of shared memory for 32 fma; TM =
// 4 and 2 give small products more tiles.  Sums run over at most 256 products
// before they are added to the total: the error of a sum of K terms grows like
// K / 256 + 256 half-ulps instead of K.
#include <algorithm>

#include "dense.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kBN = 64, kBK = 16, kThreads = 256;
constexpr int kChunk = 256 / kBK;   // slices of a partial sum
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 twice(float a) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(a));
    return d;
}

__device__ __forceinline__ void copy4(float *dst, const float *src, bool in) {   // zero where !in
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// This thread's elements of a slice [ROWS][kBK] of a matrix stored [rows][K]
// (or [K][rows] if TR), consecutive threads along the contiguous axis: element
// i lies i steps from the first, in global and in shared memory.
template <bool TR, int ROWS>
struct Slice {
    static constexpr int kN = ROWS * kBK / kThreads;
    static constexpr int kRowStep = TR ? 0 : kThreads / kBK, kKStep = TR ? kThreads / ROWS : 0;
    const float *g = nullptr;
    long long step = 0, slice = 0;
    int r = 0, k = 0, rows_in = 0;
    __device__ __forceinline__ void start(const void *base, long long ld, long long r0, long long rows) {
        r = TR ? threadIdx.x % ROWS : threadIdx.x / kBK;
        k = TR ? threadIdx.x / ROWS : threadIdx.x % kBK;
        rows_in = (int)min((long long)ROWS, rows - r0);
        // rows outside are not read: their addresses stay inside the first row
        g = static_cast<const float *>(base) + (TR ? (long long)k * ld + r0 + (r < rows_in ? r : 0)
                                                   : (r0 + (r < rows_in ? r : 0)) * ld + k);
        step = TR ? (long long)kKStep * ld : (long long)kRowStep * ld;
        slice = TR ? (long long)kBK * ld : kBK;
    }
    // k_left: columns of K left from the slice's first
    template <typename F>
    __device__ __forceinline__ void copy(long long k_left, F dst) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const bool in = r + i * kRowStep < rows_in && k + i * kKStep < k_left;
            copy4(dst(r + i * kRowStep, k + i * kKStep), in ? g + i * step : g, in);
        }
    }
    __device__ __forceinline__ void next() { g += slice; }
};

template <int EPI, bool TA, bool TB, int TM>
__global__ void __launch_bounds__(kThreads, 2) product_simt_kernel(const __grid_constant__ Product p) {
    constexpr int NB = EPI == EPI_STORE ? 1 : 2, kRows = kBN / NB, BM = 16 * TM;
    constexpr int kLdA = BM + 4, kLdB = kBN + 4, kStages = TM == 8 ? 3 : 4;
    __shared__ alignas(16) float sa[kStages][kBK][kLdA], sb[kStages][kBK][kLdB];
    const long long mt = (p.M + BM - 1) / BM;
    const int z = (int)(blockIdx.x / mt);
    const long long m0 = (blockIdx.x % mt) * BM, n0 = (long long)blockIdx.y * kRows;
    const int tm = (threadIdx.x / 16) * TM, tn = threadIdx.x % 16;
    f32x2 tot[TM / 2][4], acc[TM / 2][4];
#pragma unroll
    for (int i = 0; i < TM / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][j] = acc[i][j] = 0;
    Slice<TA, BM> xa;
    Slice<TB, kRows> xb[NB];
    const int per = (int)((p.K + kBK - 1) / kBK), slices = per * p.nseg;
    int loaded = 0;
    long long k_left = 0;
    auto load = [&]() {   // the next slice, into its stage; an empty group past the last
        if (loaded < slices) {
            if (loaded == 0 || loaded == per) {
                const int seg = loaded == 0 ? 0 : 1;
                k_left = p.K;
                xa.start(p.a[p.nseg > 1 ? seg : z], p.ald, m0, p.M);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int bi = NB == 2 ? b : seg;
                    xb[b].start(p.b[bi], p.bld[bi], n0, p.N);
                }
            }
            const int st = loaded % kStages;
            xa.copy(k_left, [&](int r, int k) { return &sa[st][k][r]; });
            xa.next();
#pragma unroll
            for (int b = 0; b < NB; ++b) {   // gated block: two gate and two up columns side by side
                xb[b].copy(k_left, [&](int r, int k) { return &sb[st][k][NB == 1 ? r : (r >> 1) * 4 + 2 * b + (r & 1)]; });
                xb[b].next();
            }
            k_left -= kBK;
            ++loaded;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    pdl_wait_primary();
    pdl_launch_dependents();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load();
    for (int i = 0; i < slices; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();   // slice i has arrived for all; all are done with slice i - 1's stage
        load();
        const int st = i % kStages;
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            f32x2 av[TM / 2];
            if (TM >= 4) {
#pragma unroll
                for (int q = 0; q < TM / 4; ++q) {
                    const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sa[st][k][tm + 4 * q]);
                    av[(2 * q) % (TM / 2)] = w.x;
                    av[(2 * q + 1) % (TM / 2)] = w.y;
                }
            } else {
                av[0] = *reinterpret_cast<const f32x2 *>(&sa[st][k][tm]);
            }
            const float4 bv = *reinterpret_cast<const float4 *>(&sb[st][k][4 * tn]);
            const f32x2 b2[4] = {twice(bv.x), twice(bv.y), twice(bv.z), twice(bv.w)};
#pragma unroll
            for (int q = 0; q < TM / 2; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][j] = fma2(av[q], b2[j], acc[q][j]);
        }
        if ((i + 1) % kChunk == 0 || i + 1 == slices) {
#pragma unroll
            for (int q = 0; q < TM / 2; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) tot[q][j] = add2(tot[q][j], acc[q][j]), acc[q][j] = 0;
        }
    }
    float *out = static_cast<float *>(p.out[z]);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const long long m = m0 + tm + i;
        if (m >= p.M) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float((uint32_t)(i & 1 ? tot[i / 2][j] >> 32 : tot[i / 2][j]));
#pragma unroll
        for (int j = 0; j < 4 / NB; ++j) {
            const long long n = n0 + tn * (4 / NB) + j;
            if (n >= p.N) continue;
            if (EPI == EPI_STORE) out[m * p.old[z] + n] = v[j];
            if (EPI == EPI_GLU) {
                out[m * p.old[z] + n] = silu<false>(v[j]) * v[2 + (j & 1)];
                if (p.keep[0]) {
                    static_cast<float *>(p.keep[0])[m * p.kld + n] = v[j];
                    static_cast<float *>(p.keep[1])[m * p.kld + n] = v[2 + (j & 1)];
                }
            }
            if (EPI == EPI_GLU_BWD) {
                float dg, du;
                glu_grad<false>(v[j], v[2 + (j & 1)], __ldg(static_cast<const float *>(p.dh) + m * p.dhld + n), dg, du);
                static_cast<float *>(p.keep[0])[m * p.kld + n] = dg;
                static_cast<float *>(p.keep[1])[m * p.kld + n] = du;
            }
        }
    }
}

template <int EPI, bool TA, bool TB>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    constexpr int kRows = EPI == EPI_STORE ? kBN : kBN / 2;
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long nt = (p.N + kRows - 1) / kRows;
    auto tiles = [&](int tm) { return (p.M + 16 * tm - 1) / (16 * tm) * p.nbatch * nt; };
    const int tm = tiles(8) >= sms ? 8 : (tiles(4) >= sms ? 4 : 2);
    const long long mt = (p.M + 16 * tm - 1) / (16 * tm) * p.nbatch;
    if (mt > 0x7FFFFFFFLL || nt > 65535) return cudaErrorInvalidConfiguration;
    const auto kernel = tm == 8 ? product_simt_kernel<EPI, TA, TB, 8>
                                : (tm == 4 ? product_simt_kernel<EPI, TA, TB, 4> : product_simt_kernel<EPI, TA, TB, 2>);
    return launch_pdl(kernel, dim3((unsigned)mt, (unsigned)nt), kThreads, 0, 0, s, p);
}

// Copies of up to three matrices into rows that start on 16 bytes, 16 bytes a
// thread, read in aligned words and shifted (bandwidth bound: the matrices once
// in, once out).
struct PackArgs {
    const uint8_t *src[3];
    uint8_t *dst[3];
    long long ld[3], dst_ld[3], rows[3];   // bytes
    int cols[3];                           // bytes
};
__global__ void __launch_bounds__(128) pack_kernel(const __grid_constant__ PackArgs p) {
    const int z = blockIdx.z, c = (blockIdx.x * 128 + threadIdx.x) * 16;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (c >= p.cols[z]) return;
    for (long long r = blockIdx.y; r < p.rows[z]; r += gridDim.y) {
        uint32_t w[4];
        load16_any(p.src[z] + r * p.ld[z] + c, p.cols[z] - c, c > 0, w);
        *reinterpret_cast<uint4 *>(p.dst[z] + r * p.dst_ld[z] + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// dg, du from kept projections.  Bandwidth bound: three reads and two writes of
// an element each; VEC: 16 bytes of every array a thread (all rows on 16-byte
// addresses), else one element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) glu_dgate_kernel(const T *__restrict__ dh, long long dhld, const T *__restrict__ g,
                                                        const T *__restrict__ u, T *__restrict__ dg, T *__restrict__ du,
                                                        long long ld, long long M, long long N) {
    constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
    constexpr bool kFast = sizeof(T) == 2;
    const long long n = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * kPer;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (n >= N) return;
    for (long long m = blockIdx.y; m < M; m += gridDim.y) {
        alignas(16) T a[kPer], b[kPer], d[kPer];
        if (VEC) {
            *reinterpret_cast<uint4 *>(a) = __ldg(reinterpret_cast<const uint4 *>(g + m * N + n));
            *reinterpret_cast<uint4 *>(b) = __ldg(reinterpret_cast<const uint4 *>(u + m * N + n));
            *reinterpret_cast<uint4 *>(d) = __ldg(reinterpret_cast<const uint4 *>(dh + m * dhld + n));
        } else {
            a[0] = g[m * N + n], b[0] = u[m * N + n], d[0] = dh[m * dhld + n];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float x, y;
            glu_grad<kFast>((float)a[i], (float)b[i], (float)d[i], x, y);
            st_elem(a + i, x);
            st_elem(b + i, y);
        }
        if (VEC) {
            *reinterpret_cast<uint4 *>(dg + m * ld + n) = *reinterpret_cast<const uint4 *>(a);
            *reinterpret_cast<uint4 *>(du + m * ld + n) = *reinterpret_cast<const uint4 *>(b);
        } else {
            dg[m * ld + n] = a[0], du[m * ld + n] = b[0];
        }
    }
}
template <typename T>
cudaError_t launch_dgate_t(const T *dh, long long dhld, const T *gu, T *dg, T *du, long long ld, long long M, long long N,
                           cudaStream_t s) {
    constexpr int kPer = 16 / sizeof(T);
    // dg, du: the workspace's aligned planes
    const bool vec = !((uintptr_t)dh & 15u) && !(dhld % kPer) && !((uintptr_t)gu & 15u) && !(N % kPer);
    const long long per = vec ? 256 * kPer : 256;
    const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)(M < 32768 ? M : 32768));
    return launch_pdl(vec ? glu_dgate_kernel<T, true> : glu_dgate_kernel<T, false>, grid, 256, 0, 0, s, dh, dhld, gu,
                      gu + M * N, dg, du, ld, M, N);
}

}  // namespace

cudaError_t launch_product_simt(const Product &p, cudaStream_t s) {
    if (p.epi == EPI_GLU) return launch_t<EPI_GLU, false, false>(p, s);
    if (p.epi == EPI_GLU_BWD) return launch_t<EPI_GLU_BWD, false, false>(p, s);
    return p.a_t ? launch_t<EPI_STORE, true, true>(p, s) : launch_t<EPI_STORE, false, true>(p, s);
}

cudaError_t launch_pack(const Copy *c, int n, int es, cudaStream_t s) {
    PackArgs a{};
    long long pieces = 1, rows = 1;
    for (int i = 0; i < n; ++i) {
        a.src[i] = static_cast<const uint8_t *>(c[i].src);
        a.dst[i] = static_cast<uint8_t *>(c[i].dst);
        a.ld[i] = c[i].ld * es;
        a.dst_ld[i] = c[i].dst_ld * es;
        a.rows[i] = c[i].rows;
        a.cols[i] = (int)(c[i].cols * es);
        pieces = std::max<long long>(pieces, (a.cols[i] + 15) / 16);
        rows = std::max(rows, std::min<long long>(c[i].rows, 16384));
    }
    return launch_pdl(pack_kernel, dim3((unsigned)((pieces + 127) / 128), (unsigned)rows, (unsigned)n), 128, 0, 0, s, a);
}

cudaError_t launch_glu_dgate(const void *dh, long long dhld, const void *gu, void *dg, void *du, long long ld,
                             long long M, long long N, int dtype, cudaStream_t s) {
    typedef __nv_bfloat16 B;
    if (dtype == MOEQ_ACT_F32)
        return launch_dgate_t(static_cast<const float *>(dh), dhld, static_cast<const float *>(gu),
                              static_cast<float *>(dg), static_cast<float *>(du), ld, M, N, s);
    return launch_dgate_t(static_cast<const B *>(dh), dhld, static_cast<const B *>(gu), static_cast<B *>(dg),
                          static_cast<B *>(du), ld, M, N, s);
}

}  // namespace dense
}  // namespace moeq
