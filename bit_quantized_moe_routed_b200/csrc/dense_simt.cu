// dense_simt.cu -- f32 products of the dense operators (any sizes, strides and
// alignment), and the elementwise steps around the products.
//
// One CTA computes a 64 x 64 tile of out (two of them for the gated block,
// gate and up, which share A) from 16-deep slices of A and B in shared
// memory, 4 x 4 outputs a thread.  Sums run over at most 256 products before
// they are added to the total, so the rounding error of an f32 sum of K terms
// grows like K / 256 + 256 half-ulps instead of K.
#include "dense.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kBM = 64, kBN = 64, kBK = 16, kThreads = 256;
constexpr int kChunk = 256;

// slice [rows][kBK] of a matrix stored [rows][K] (or [K][rows] if TR) into s[k][row]
template <bool TR>
__device__ __forceinline__ void load_slice(float (*s)[kBM + 4], const float *g, long long ld, long long r0, long long rows,
                                           long long k0, long long K) {
    for (int i = threadIdx.x; i < kBM * kBK; i += kThreads) {
        const int r = TR ? i % kBM : i / kBK, k = TR ? i / kBM : i % kBK;
        const long long gr = r0 + r, gk = k0 + k;
        float v = 0.f;
        if (gr < rows && gk < K) v = __ldg(TR ? g + gk * ld + gr : g + gr * ld + gk);
        s[k][r] = v;
    }
}

template <int EPI, bool TA, bool TB>
__global__ void __launch_bounds__(kThreads) product_simt_kernel(Product p) {
    constexpr int NB = EPI == EPI_STORE ? 1 : 2;
    __shared__ float sa[kBK][kBM + 4], sb[NB][kBK][kBN + 4];
    const long long mt = (p.M + kBM - 1) / kBM;
    const int z = (int)(blockIdx.x / mt);
    const long long m0 = (blockIdx.x % mt) * kBM, n0 = (long long)blockIdx.y * kBN;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    float tot[NB][4][4], acc[NB][4][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) tot[b][i][j] = 0, acc[b][i][j] = 0;
    pdl_wait_primary();
    pdl_launch_dependents();
    for (int sgm = 0; sgm < p.nseg; ++sgm) {
        const float *a = static_cast<const float *>(p.a[p.nseg > 1 ? sgm : z]);
        for (long long k0 = 0; k0 < p.K; k0 += kBK) {
            load_slice<TA>(sa, a, p.ald, m0, p.M, k0, p.K);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int bi = NB == 2 ? b : (p.nseg > 1 ? sgm : 0);
                load_slice<TB>(sb[b], static_cast<const float *>(p.b[bi]), p.bld[bi], n0, p.N, k0, p.K);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kBK; ++k) {
                float av[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) av[i] = sa[k][tm + i];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float bv = sb[b][k][tn + j];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][i][j] += av[i] * bv;
                    }
            }
            __syncthreads();
            if ((k0 + kBK) % kChunk == 0 || k0 + kBK >= p.K) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) tot[b][i][j] += acc[b][i][j], acc[b][i][j] = 0;
            }
        }
    }
    float *out = static_cast<float *>(p.out[z]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long m = m0 + tm + i;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long n = n0 + tn + j;
            if (n >= p.N) continue;
            float v[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                v[b] = tot[b][i][j];
            }
            if (EPI == EPI_STORE) st_elem(out + m * p.old[z] + n, v[0]);
            if (EPI == EPI_GLU) {
                st_elem(out + m * p.old[z] + n, silu<false>(v[0]) * v[NB - 1]);
                if (p.keep[0]) {
                    st_elem(static_cast<float *>(p.keep[0]) + m * p.kld + n, v[0]);
                    st_elem(static_cast<float *>(p.keep[1]) + m * p.kld + n, v[NB - 1]);
                }
            }
            if (EPI == EPI_GLU_BWD) {
                float dg, du;
                glu_grad<false>(v[0], v[NB - 1], dense::ld_elem(static_cast<const float *>(p.dh) + m * p.dhld + n), dg, du);
                st_elem(static_cast<float *>(p.keep[0]) + m * p.kld + n, dg);
                st_elem(static_cast<float *>(p.keep[1]) + m * p.kld + n, du);
            }
        }
    }
}

template <int EPI, bool TA, bool TB>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    const long long mt = (p.M + kBM - 1) / kBM, nt = (p.N + kBN - 1) / kBN;
    if (mt * p.nbatch > 0x7FFFFFFFLL || nt > 65535) return cudaErrorInvalidConfiguration;
    return launch_pdl(product_simt_kernel<EPI, TA, TB>, dim3((unsigned)(mt * p.nbatch), (unsigned)nt), kThreads, 0, 0, s, p);
}

// Copy into rows with 16-byte aligned starts: one 16-byte piece a thread
template <typename T>
__global__ void pack_kernel(const T *__restrict__ src, long long ld, uint8_t *__restrict__ dst, long long dst_ld,
                            long long rows, long long cols) {
    constexpr int kPer = 16 / sizeof(T);
    const long long c = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * kPer;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (c >= cols) return;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        const T *p = src + r * ld + c;
        alignas(16) T v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = c + i < cols ? __ldg(p + i) : (T)0;
        *reinterpret_cast<uint4 *>(dst + (r * dst_ld + c) * sizeof(T)) = *reinterpret_cast<const uint4 *>(v);
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

cudaError_t launch_pack(const void *src, long long ld, void *dst, long long dst_ld, long long rows, long long cols,
                        int es, cudaStream_t s) {
    const long long pieces = (cols * es + 15) / 16;
    const dim3 grid((unsigned)((pieces + 127) / 128), (unsigned)(rows < 32768 ? rows : 32768));
    uint8_t *d = static_cast<uint8_t *>(dst);
    if (es == 1)
        return launch_pdl(pack_kernel<int8_t>, grid, 128, 0, 0, s, static_cast<const int8_t *>(src), ld, d, dst_ld, rows, cols);
    return launch_pdl(pack_kernel<uint16_t>, grid, 128, 0, 0, s, static_cast<const uint16_t *>(src), ld, d, dst_ld, rows,
                      cols);
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
