// dense_few.cu -- the gated block's gradients for up to 4 tokens (bf16), on the
// f32 units from f32 gate gradients.
//
//   dx[t][h] = sum_n dg[t][n] Wg[n][h] + du[t][n] Wu[n][h],   dW_i[n][h] = sum_t d_i[t][n] x[t][h]
//
// With few tokens a sum has few terms, and rounding dg and du to bf16 (as the
// tensor-core kernels do) could show in the result as more than the rounding of
// the result itself; here nothing is rounded before it.  Bound: HBM, the weights
// read once for dx, the gradients written once for dW (4096 x 2048: 10.2 us; the
// products of 4 tokens take the f32 units 3.7).  Measured there, 1 token, weights
// from HBM: 19.7 us with kept projections, 20.6 without.  The first loads wait a
// DRAM latency behind the kernel before, and where inter is far above hidden few
// blocks share long sums.
//
// One launch.  dx: a cluster of 1 to 8 blocks takes 64 columns, a block every so
// many chunks of 256 rows n; 8 threads side by side read a row's 128 bytes, the
// block's 32 groups of them a row each, and the sums meet by shuffles, in shared
// memory and over the cluster, in a fixed order.  dW: a thread keeps x of 8
// columns in registers and writes 8 rows of each gradient.  dg and du of a chunk
// lie in shared memory as [n][t].  Any strides and alignment.
#include <cooperative_groups.h>

#include "dense.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCols = 64, kGroups = kThreads / (kCols / 8);   // dx: columns a block, rows at a time
constexpr int kRowsN = 8;                                     // dW: rows a thread
constexpr int kChunk = 256;                                   // rows of dg, du held
typedef __nv_bfloat16 B;

struct FewArgs {
    const float *d[2];        // dg, du [T][dld]
    long long dld;
    const B *x, *w[2];
    long long ldx, ldw[2];
    B *dx, *dw[2];
    long long lddx, lddw[2];
    int T, H, I;
    int dx_blocks;            // blocks of dx, whole clusters; the rest are dW's
    int split;                // blocks of a cluster
    int tx, hblocks;          // dW: threads along the columns, blocks along them
    bool vec_x, vec_dw;
};

// 8 elements at p, `left` (elements, any value) of which are in the row, zeros beyond
__device__ __forceinline__ void load8(const B *p, int left, bool before, bool vec, float v[8]) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (vec && left >= 8) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if (left > 0) {
        load16_any(reinterpret_cast<const uint8_t *>(p), left * 2, before, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// dg and du of rows n0 .. n0 + kChunk to shared memory, zeros beyond T and I
template <int NT>
__device__ __forceinline__ void stage(const FewArgs &p, int n0, float (*d)[kChunk][NT]) {
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int n = n0 + threadIdx.x;
            d[m][threadIdx.x][t] = t < p.T && n < p.I ? __ldg(p.d[m] + t * p.dld + n) : 0.f;
        }
}

template <int NT, bool VEC>
__global__ void __launch_bounds__(kThreads) few_gradients_kernel(const __grid_constant__ FewArgs p) {
    static_assert(kChunk == kThreads, "one row a thread to stage");
    __shared__ alignas(16) float d[2][kChunk][NT];
    __shared__ float part[kWarps][NT][kCols];
    __shared__ float own[NT * kCols];
    pdl_wait_primary();
    pdl_launch_dependents();
    if ((int)blockIdx.x < p.dx_blocks) {
        const int hq = threadIdx.x & 7, nl = threadIdx.x >> 3, rank = blockIdx.x % p.split;
        const int h0 = blockIdx.x / p.split * kCols, h = h0 + 8 * hq;
        float acc[NT][8] = {};
        for (int n0 = rank * kChunk; n0 < p.I; n0 += p.split * kChunk) {
            __syncthreads();
            stage<NT>(p, n0, d);
            __syncthreads();
            for (int m = 0; m < 2; ++m) {
                const B *w = p.w[m] + (long long)(n0 + nl) * p.ldw[m] + h;
#pragma unroll(VEC ? 8 : 2)
                for (int r = 0; r < kChunk / kGroups; ++r) {
                    const int n = nl + r * kGroups;
                    float v[8];
                    load8(w + (long long)r * kGroups * p.ldw[m], n0 + n < p.I ? p.H - h : 0, h > 0, VEC, v);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float e = d[m][n][t];
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(e, v[j], acc[t][j]);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int o = 8; o < 32; o *= 2) acc[t][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[t][j], o);
                if ((threadIdx.x & 31) < 8) part[threadIdx.x >> 5][t][8 * hq + j] = acc[t][j];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < NT * kCols; i += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += part[w][i / kCols][i % kCols];
            own[i] = s;
        }
        const cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
        cl.sync();   // dx_blocks is whole clusters: all of a cluster's blocks come here
        for (int i = rank * kThreads + threadIdx.x; i < NT * kCols; i += p.split * kThreads) {
            const int t = i / kCols, c = h0 + i % kCols;
            float s = 0.f;
            for (int r = 0; r < p.split; ++r) s += cl.map_shared_rank(own, r)[i];
            if (t < p.T && c < p.H) p.dx[t * p.lddx + c] = __float2bfloat16_rn(s);
        }
        cl.sync();   // no block leaves while others read its sums
        return;
    }
    const int b = blockIdx.x - p.dx_blocks, ty = kThreads / p.tx;
    const int h = ((b % p.hblocks) * p.tx + threadIdx.x % p.tx) * 8;
    const int nb = b / p.hblocks * ty * kRowsN, nl = threadIdx.x / p.tx * kRowsN;   // nl + kRowsN <= kChunk
    if (nb >= p.I) return;   // blocks that fill up the last cluster
    stage<NT>(p, nb, d);
    __syncthreads();
    if (h >= p.H) return;
    float x[NT][8];
#pragma unroll
    for (int t = 0; t < NT; ++t) load8(p.x + (t < p.T ? t : 0) * p.ldx + h, t < p.T ? p.H - h : 0, h > 0, p.vec_x, x[t]);
    for (int m = 0; m < 2; ++m)
        for (int r = 0; r < kRowsN && nb + nl + r < p.I; ++r) {
            float acc[8] = {};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float e = d[m][nl + r][t];
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(e, x[t][j], acc[j]);
            }
            B *o = p.dw[m] + (long long)(nb + nl + r) * p.lddw[m] + h;
            alignas(16) B q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = __float2bfloat16_rn(acc[j]);
            if (p.vec_dw && h + 8 <= p.H) {
                *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(q);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (h + j < p.H) o[j] = q[j];
            }
        }
}

template <int NT>
cudaError_t launch_nt(const FewArgs &a, bool vec, long long blocks, cudaStream_t s) {
    return launch_pdl(vec ? few_gradients_kernel<NT, true> : few_gradients_kernel<NT, false>, dim3((unsigned)blocks), kThreads,
                      0, a.split, s, a);
}

// f32 gradients of kept projections
__global__ void __launch_bounds__(256) dgate_f32_kernel(const B *__restrict__ dh, long long dhld, const B *__restrict__ g,
                                                        const B *__restrict__ u, float *__restrict__ dg,
                                                        float *__restrict__ du, long long ld, int N) {
    const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (n >= N) return;
    glu_grad<false>(ld_elem(g + (long long)t * N + n), ld_elem(u + (long long)t * N + n), ld_elem(dh + t * dhld + n),
                    dg[t * ld + n], du[t * ld + n]);
}

}  // namespace

cudaError_t launch_dgate_f32(const void *dh, long long dhld, const void *gu, float *dg, float *du, long long ld, int T, int N,
                             cudaStream_t s) {
    const B *g = static_cast<const B *>(gu);
    return launch_pdl(dgate_f32_kernel, dim3((unsigned)((N + 255) / 256), (unsigned)T), 256, 0, 0, s,
                      static_cast<const B *>(dh), dhld, g, g + (long long)T * N, dg, du, ld, N);
}

cudaError_t launch_few_gradients(const Product *px, const Product *pw, const float *dg, const float *du, long long dld,
                                 cudaStream_t s) {
    FewArgs a{};
    bool vec = true;
    a.split = 1;
    a.d[0] = dg;
    a.d[1] = du;
    a.dld = dld;
    auto rows16 = [](const void *p, long long ld) { return !((uintptr_t)p & 15u) && !(ld & 7); };
    if (px) {
        a.T = (int)px->M;
        a.H = (int)px->N;
        a.I = (int)px->K;
        for (int i = 0; i < 2; ++i) {
            a.w[i] = static_cast<const B *>(px->b[i]);
            a.ldw[i] = px->bld[i];
            vec = vec && rows16(px->b[i], px->bld[i]);
        }
        a.dx = static_cast<B *>(px->out[0]);
        a.lddx = px->old[0];
        // split while blocks are few and have more than a chunk each
        const int tiles = (a.H + kCols - 1) / kCols;
        while (a.split < 8 && tiles * a.split < 592 && a.split * kChunk < a.I) a.split *= 2;
        a.dx_blocks = tiles * a.split;
    }
    long long blocks = a.dx_blocks;
    if (pw) {
        a.T = (int)pw->K;
        a.H = (int)pw->N;
        a.I = (int)pw->M;
        a.x = static_cast<const B *>(pw->b[0]);
        a.ldx = pw->bld[0];
        a.vec_x = rows16(a.x, a.ldx);
        a.vec_dw = true;
        for (int i = 0; i < 2; ++i) {
            a.dw[i] = static_cast<B *>(pw->out[i]);
            a.lddw[i] = pw->old[i];
            a.vec_dw = a.vec_dw && rows16(pw->out[i], pw->old[i]);
        }
        a.tx = 8;
        while (a.tx < kThreads && a.tx * 8 < a.H) a.tx *= 2;
        a.hblocks = (a.H + 8 * a.tx - 1) / (8 * a.tx);
        const int rows = kThreads / a.tx * kRowsN;
        blocks += (long long)a.hblocks * ((a.I + rows - 1) / rows);
    }
    blocks = (blocks + a.split - 1) / a.split * a.split;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (a.T <= 1) return launch_nt<1>(a, vec, blocks, s);
    return a.T <= 2 ? launch_nt<2>(a, vec, blocks, s) : launch_nt<4>(a, vec, blocks, s);
}

}  // namespace dense
}  // namespace moeq
