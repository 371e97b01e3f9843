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
// an element each, eight elements a thread (VEC: rows on 16-byte addresses, else
// words shifted into place).
template <bool VEC>
__global__ void __launch_bounds__(128) glu_dgate_kernel(const T *__restrict__ dh, long long dhld, const T *__restrict__ g,
                                                        const T *__restrict__ u, T *__restrict__ dg, T *__restrict__ du,
                                                        long long ld, long long M, long long N) {
    const long long n = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 8;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (n >= N) return;
    const int left = (int)min(8LL, N - n) * 2;   // bytes of the row; the rest of the padded row gets zeros' gradients
    for (long long m = blockIdx.y * blockDim.y + threadIdx.y; m < M; m += gridDim.y * blockDim.y) {
        uint32_t a[4], b[4], d[4];
        auto read = [&](const T *p, uint32_t w[4]) {
            if (VEC) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {   // up to 4 bytes of the row beyond the 16: whole words where they are there
                load16_any(reinterpret_cast<const uint8_t *>(p), (int)min(32LL, (N - n) * 2), n > 0, w);
            }
        };
        read(g + m * N + n, a);
        read(u + m * N + n, b);
        read(dh + m * dhld + n, d);
        if (!VEC && left < 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t keep = 4 * i + 4 <= left ? 0xFFFFFFFFu : (4 * i + 2 <= left ? 0xFFFFu : 0u);
                a[i] &= keep, b[i] &= keep, d[i] &= keep;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[2], y[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sh = 16 * h;
                glu_grad<true>(bf16_bits_to_f32(a[i] >> sh & 0xFFFFu), bf16_bits_to_f32(b[i] >> sh & 0xFFFFu),
                               bf16_bits_to_f32(d[i] >> sh & 0xFFFFu), x[h], y[h]);
            }
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[0], x[1]), q = __floats2bfloat162_rn(y[0], y[1]);
            a[i] = *reinterpret_cast<const uint32_t *>(&p);
            b[i] = *reinterpret_cast<const uint32_t *>(&q);
        }
        *reinterpret_cast<uint4 *>(dg + m * ld + n) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4 *>(du + m * ld + n) = make_uint4(b[0], b[1], b[2], b[3]);
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
    const bool vec = !((uintptr_t)dh & 15u) && !(dhld % 8) && !((uintptr_t)gu & 15u) && !(N % 8);
    const RowGrid r(M, (N + 7) / 8);
    return launch_pdl(vec ? glu_dgate_kernel<true> : glu_dgate_kernel<false>, r.grid, r.block, 0, 0, s, dh, dhld, gu, gu + M * N,
                      dg, du, ld, M, N);
}

}  // namespace dense
}  // namespace moeq
