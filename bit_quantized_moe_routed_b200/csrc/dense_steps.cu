// dense_steps.cu -- elementwise steps around the products of the dense
// operators: copies of operands into aligned rows, the gates' gradients (bf16).
#include <algorithm>

#include "dense.cuh"

namespace moeq {
namespace dense {
namespace {

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
    const int z = blockIdx.z, c = (blockIdx.x * blockDim.x + threadIdx.x) * 16;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (c >= p.cols[z]) return;
    for (long long r = blockIdx.y * blockDim.y + threadIdx.y; r < p.rows[z]; r += gridDim.y * blockDim.y) {
        uint32_t w[4];
        load16_any(p.src[z] + r * p.ld[z] + c, p.cols[z] - c, c > 0, w);
        *reinterpret_cast<uint4 *>(p.dst[z] + r * p.dst_ld[z] + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

typedef __nv_bfloat16 T;

// dg, du from kept projections.  Bandwidth bound: three reads and two writes of
// an element each; VEC: 16 bytes of every array a thread (all rows on 16-byte
// addresses), else one element.
template <bool VEC>
__global__ void __launch_bounds__(128) glu_dgate_kernel(const T *__restrict__ dh, long long dhld, const T *__restrict__ g,
                                                        const T *__restrict__ u, T *__restrict__ dg, T *__restrict__ du,
                                                        long long ld, long long M, long long N) {
    constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
    const long long n = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * kPer;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (n >= N) return;
    for (long long m = blockIdx.y * blockDim.y + threadIdx.y; m < M; m += gridDim.y * blockDim.y) {
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
            glu_grad<true>((float)a[i], (float)b[i], (float)d[i], x, y);
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
}  // namespace

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
        rows = std::max(rows, c[i].rows);
    }
    const RowGrid g(rows, pieces, n);
    return launch_pdl(pack_kernel, g.grid, g.block, 0, 0, s, a);
}

cudaError_t launch_glu_dgate(const void *dh_, long long dhld, const void *gu_, void *dg_, void *du_, long long ld,
                             long long M, long long N, cudaStream_t s) {
    const T *dh = static_cast<const T *>(dh_), *gu = static_cast<const T *>(gu_);
    T *dg = static_cast<T *>(dg_), *du = static_cast<T *>(du_);   // the workspace's aligned planes
    constexpr int kPer = 16 / sizeof(T);
    const bool vec = !((uintptr_t)dh & 15u) && !(dhld % kPer) && !((uintptr_t)gu & 15u) && !(N % kPer);
    const RowGrid r(M, vec ? N / kPer : N);
    return launch_pdl(vec ? glu_dgate_kernel<true> : glu_dgate_kernel<false>, r.grid, r.block, 0, 0, s, dh, dhld, gu, gu + M * N,
                      dg, du, ld, M, N);
}

}  // namespace dense
}  // namespace moeq
