// dense_simt.cu -- products of the dense operators on the f32 / int32 units:
// any sizes, strides and alignment.
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

template <typename T> struct Acc { typedef float type; };
template <> struct Acc<int8_t> { typedef int type; };
__device__ __forceinline__ int ld_elem(const int8_t *p) { return __ldg(p); }
__device__ __forceinline__ float ld_any(const float *p) { return dense::ld_elem(p); }
__device__ __forceinline__ float ld_any(const __nv_bfloat16 *p) { return dense::ld_elem(p); }
__device__ __forceinline__ int ld_any(const int8_t *p) { return (int)__ldg(p); }

// slice [rows][kBK] of a matrix stored [rows][K] (or [K][rows] if TR) into s[k][row]
template <typename T, bool TR, typename E>
__device__ __forceinline__ void load_slice(E (*s)[kBM + 4], const T *g, long long ld, long long r0, long long rows,
                                           long long k0, long long K) {
    for (int i = threadIdx.x; i < kBM * kBK; i += kThreads) {
        const int r = TR ? i % kBM : i / kBK, k = TR ? i / kBM : i % kBK;
        const long long gr = r0 + r, gk = k0 + k;
        E v = 0;
        if (gr < rows && gk < K) v = ld_any(TR ? g + gk * ld + gr : g + gr * ld + gk);
        s[k][r] = v;
    }
}

template <typename T, typename O, int EPI, bool TA, bool TB>
__global__ void __launch_bounds__(kThreads) product_simt_kernel(Product p) {
    typedef typename Acc<T>::type E;
    constexpr int NB = EPI == EPI_STORE ? 1 : 2;
    __shared__ E sa[kBK][kBM + 4], sb[NB][kBK][kBN + 4];
    const long long mt = (p.M + kBM - 1) / kBM;
    const int z = (int)(blockIdx.x / mt);
    const long long m0 = (blockIdx.x % mt) * kBM, n0 = (long long)blockIdx.y * kBN;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    E tot[NB][4][4], acc[NB][4][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) tot[b][i][j] = 0, acc[b][i][j] = 0;
    for (int sgm = 0; sgm < p.nseg; ++sgm) {
        const T *a = static_cast<const T *>(p.a[p.nseg > 1 ? sgm : z]);
        for (long long k0 = 0; k0 < p.K; k0 += kBK) {
            load_slice<T, TA>(sa, a, p.ald, m0, p.M, k0, p.K);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int bi = NB == 2 ? b : (p.nseg > 1 ? sgm : 0);
                load_slice<T, TB>(sb[b], static_cast<const T *>(p.b[bi]), p.bld[bi], n0, p.N, k0, p.K);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kBK; ++k) {
                E av[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) av[i] = sa[k][tm + i];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const E bv = sb[b][k][tn + j];
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
    O *out = static_cast<O *>(p.out[z]);
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
                v[b] = (float)tot[b][i][j];
                if (sizeof(T) == 1) v[b] = v[b] * __ldg(p.a_scale + m) * __ldg(p.b_scale[b] + n);
            }
            if (EPI == EPI_STORE) st_elem(out + m * p.old[z] + n, v[0]);
            if (EPI == EPI_GLU) {
                st_elem(out + m * p.old[z] + n, silu_f32(v[0]) * v[NB - 1]);
                if (p.keep[0]) {
                    st_elem(static_cast<O *>(p.keep[0]) + m * p.kld + n, v[0]);
                    st_elem(static_cast<O *>(p.keep[1]) + m * p.kld + n, v[NB - 1]);
                }
            }
            if (EPI == EPI_GLU_BWD) {
                float dg, du;
                glu_grad(v[0], v[NB - 1], dense::ld_elem(static_cast<const O *>(p.dh) + m * p.dhld + n), dg, du);
                st_elem(static_cast<O *>(p.keep[0]) + m * p.kld + n, dg);
                st_elem(static_cast<O *>(p.keep[1]) + m * p.kld + n, du);
            }
        }
    }
}

template <typename T, typename O>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    const long long mt = (p.M + kBM - 1) / kBM, nt = (p.N + kBN - 1) / kBN;
    if (mt * p.nbatch > 0x7FFFFFFFLL || nt > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(mt * p.nbatch), (unsigned)nt);
    if (p.epi == EPI_GLU) product_simt_kernel<T, O, EPI_GLU, false, false><<<grid, kThreads, 0, s>>>(p);
    else if (sizeof(T) == 1) product_simt_kernel<T, O, EPI_STORE, false, false><<<grid, kThreads, 0, s>>>(p);
    else if (p.epi == EPI_GLU_BWD) {
        if constexpr (sizeof(T) > 1) product_simt_kernel<T, O, EPI_GLU_BWD, false, false><<<grid, kThreads, 0, s>>>(p);
    } else if (p.a_t) {
        if constexpr (sizeof(T) > 1) product_simt_kernel<T, O, EPI_STORE, true, true><<<grid, kThreads, 0, s>>>(p);
    } else {
        if constexpr (sizeof(T) > 1) product_simt_kernel<T, O, EPI_STORE, false, true><<<grid, kThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// dg, du from kept projections: bandwidth bound, one element a thread
template <typename T>
__global__ void glu_dgate_kernel(const T *__restrict__ dh, long long dhld, const T *__restrict__ g,
                                 const T *__restrict__ u, T *__restrict__ dg, T *__restrict__ du, long long ld,
                                 long long M, long long N) {
    const long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= N) return;
    for (long long m = blockIdx.y; m < M; m += gridDim.y) {
        float a, b;
        glu_grad(dense::ld_elem(g + m * N + n), dense::ld_elem(u + m * N + n), dense::ld_elem(dh + m * dhld + n), a, b);
        st_elem(dg + m * ld + n, a);
        st_elem(du + m * ld + n, b);
    }
}

}  // namespace

cudaError_t launch_product_simt(const Product &p, cudaStream_t s) {
    if (p.M <= 0 || p.N <= 0) return cudaSuccess;
    if (p.in_dtype == kI8)
        return p.out_dtype == MOEQ_ACT_F32 ? launch_t<int8_t, float>(p, s) : launch_t<int8_t, __nv_bfloat16>(p, s);
    return p.in_dtype == MOEQ_ACT_F32 ? launch_t<float, float>(p, s) : launch_t<__nv_bfloat16, __nv_bfloat16>(p, s);
}

cudaError_t launch_glu_dgate(const void *dh, long long dhld, const void *gu, void *dg, void *du, long long ld,
                             long long M, long long N, int dtype, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)(M < 32768 ? M : 32768));
    if (dtype == MOEQ_ACT_F32) {
        const float *g = static_cast<const float *>(gu);
        glu_dgate_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float *>(dh), dhld, g, g + M * N,
                                                     static_cast<float *>(dg), static_cast<float *>(du), ld, M, N);
    } else {
        const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(gu);
        glu_dgate_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
            static_cast<const __nv_bfloat16 *>(dh), dhld, g, g + M * N, static_cast<__nv_bfloat16 *>(dg),
            static_cast<__nv_bfloat16 *>(du), ld, M, N);
    }
    return cudaGetLastError();
}

}  // namespace dense
}  // namespace moeq
