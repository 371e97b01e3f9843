// dense_stream.cu -- products of the dense operators for a few rows of A (the
// tokens of a decode step): the weights stream once through registers.
//
// Bound: HBM, the bytes of the weights.  A CTA takes 16 weight rows (8 gate
// and the 8 up rows of the same outputs for the gated block) over all of K;
// its warps split K.  A lane loads 16 consecutive bytes of a row, which are
// the A fragments of two tensor-core steps under a permutation of K that x
// shares (the sum does not depend on the order of K), so the weights go from
// HBM to mma.sync without shared memory, kChunk 64-byte blocks (2 kChunk
// loads of 16 bytes) a lane in flight.  The tokens are the N = 8 columns of
// the step.  tcgen05 would need the weights in shared memory first and pads N
// to its M; at 8 columns the legacy path leaves the tensor cores far from
// their limit.  A lane ends with the gate and the up sum of the same outputs;
// the warps' partial sums meet in shared memory in a fixed order.
//
// Operands at any address and row stride: rows that do not start on 16 bytes
// are read in aligned 4-byte words and shifted.
#include "dense_tc.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kChunk = 8;      // 64-byte blocks of K a warp has in flight

struct StreamArgs {
    const uint8_t *w[2];
    long long ldw[2];          // bytes
    const uint8_t *x;
    long long ldx;             // bytes
    int T, N;
    int kbytes;                // of a row
    const float *a_scale, *b_scale[2];
    void *out;
    long long old;
    void *keep[2];
    long long kld;
};

// 16 bytes at p, of which `left` (any value) are inside the row; zeros beyond.
template <bool VEC>
__device__ __forceinline__ uint4 load16(const uint8_t *p, int left, bool first) {
    if (left <= 0) return make_uint4(0, 0, 0, 0);
    if (VEC && left >= 16) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
    const int off = (int)((uintptr_t)p & 3);
    if (!VEC && left >= 20 && !(first && off)) {   // whole words of the row around the 16 bytes
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
        uint32_t a = __ldg(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = off ? __ldg(q + i + 1) : 0u;
            const uint32_t c = off ? b : (i < 3 ? __ldg(q + i + 1) : 0u);
            w[i] = off ? __funnelshift_r(a, b, 8 * off) : a;
            a = c;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * i + j < left) w[i] |= (uint32_t)__ldg(p + 4 * i + j) << (8 * j);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool I8> struct Sum { typedef float type; };
template <> struct Sum<true> { typedef int type; };

__device__ __forceinline__ void step(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void step(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 tokens
template <bool I8, int EPI, int NT, bool VEC, typename O>
__global__ void __launch_bounds__(kThreads, 2) product_stream_kernel(const __grid_constant__ StreamArgs p) {
    typedef typename Sum<I8>::type E;
    __shared__ E part[kWarps][NT][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int per = EPI == EPI_STORE ? 16 : 8;            // outputs of a group
    const int n0 = blockIdx.x * per;
    const int r0 = n0 + g, r1 = EPI == EPI_STORE ? n0 + 8 + g : n0 + g;
    const uint8_t *w0 = p.w[0] + (long long)min(r0, p.N - 1) * p.ldw[0];
    const uint8_t *w1 = EPI == EPI_STORE ? p.w[0] + (long long)min(r1, p.N - 1) * p.ldw[0]
                                         : p.w[1] + (long long)min(r1, p.N - 1) * p.ldw[1];
    const int k0 = r0 < p.N ? p.kbytes : 0, k1 = r1 < p.N ? p.kbytes : 0;
    E c[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0;
    const int blocks = (p.kbytes + 63) / 64, share = (blocks + kWarps - 1) / kWarps;
    const int b_end = min(blocks, (warp + 1) * share);
    for (int b0 = warp * share; b0 < b_end; b0 += kChunk) {
        uint4 a[kChunk][2];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const int k = (b0 + j) * 64 + 16 * t;
            const bool in = b0 + j < b_end;
            a[j][0] = load16<VEC>(w0 + k, in ? k0 - k : 0, k == 0);
            a[j][1] = load16<VEC>(w1 + k, in ? k1 - k : 0, k == 0);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const int k = (b0 + j) * 64 + 16 * t;
            if (b0 + j >= b_end) break;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int tok = 8 * i + g;
                const uint4 x = load16<VEC>(p.x + (long long)min(tok, p.T - 1) * p.ldx + k, tok < p.T ? p.kbytes - k : 0,
                                            k == 0);
                step(c[i], a[j][0].x, a[j][1].x, a[j][0].y, a[j][1].y, x.x, x.y);
                step(c[i], a[j][0].z, a[j][1].z, a[j][0].w, a[j][1].w, x.z, x.w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[warp][i][q][lane] = c[i][q];
    __syncthreads();
    // output o of the group's 8 NT tokens: the lane and component that hold it
    for (int o = threadIdx.x; o < per * 8 * NT; o += kThreads) {
        const int r = o % per, tok = o / per, n = n0 + r;
        if (tok >= p.T || n >= p.N) continue;
        const int i = tok >> 3, src = (r & 7) * 4 + ((tok & 7) >> 1), q = (tok & 1) + (r >> 3) * 2;
        E s0 = 0, s1 = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s0 += part[w][i][q][src];
            if (EPI == EPI_GLU) s1 += part[w][i][q + 2][src];
        }
        float v0 = (float)s0, v1 = (float)s1;
        if (I8) {
            const float sx = __ldg(p.a_scale + tok);
            v0 = v0 * sx * __ldg(p.b_scale[0] + n);
            if (EPI == EPI_GLU) v1 = v1 * sx * __ldg(p.b_scale[1] + n);
        }
        O *out = static_cast<O *>(p.out) + (long long)tok * p.old + n;
        if (EPI == EPI_GLU) {
            st_elem(out, silu<sizeof(O) == 2>(v0) * v1);
            if (!I8 && p.keep[0]) {
                st_elem(static_cast<O *>(p.keep[0]) + (long long)tok * p.kld + n, v0);
                st_elem(static_cast<O *>(p.keep[1]) + (long long)tok * p.kld + n, v1);
            }
        } else {
            st_elem(out, v0);
        }
    }
}

template <bool I8, int EPI, typename O>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    const int es = I8 ? 1 : 2;
    StreamArgs a{};
    bool vec = !((uintptr_t)p.a[0] & 15u) && !((p.ald * es) & 15);
    for (int i = 0; i < (EPI == EPI_GLU ? 2 : 1); ++i) {
        a.w[i] = static_cast<const uint8_t *>(p.b[i]);
        a.ldw[i] = p.bld[i] * es;
        a.b_scale[i] = p.b_scale[i];
        a.keep[i] = p.keep[i];
        vec = vec && !((uintptr_t)p.b[i] & 15u) && !(a.ldw[i] & 15);
    }
    if (EPI == EPI_GLU) a.keep[1] = p.keep[1];
    a.x = static_cast<const uint8_t *>(p.a[0]);
    a.ldx = p.ald * es;
    a.T = (int)p.M;
    a.N = (int)p.N;
    a.kbytes = (int)(p.K * es);
    a.a_scale = p.a_scale;
    a.out = p.out[0];
    a.old = p.old[0];
    a.kld = p.kld;
    const int per = EPI == EPI_STORE ? 16 : 8;
    const int grid = (a.N + per - 1) / per;
    if (a.T <= 8) {
        if (vec) product_stream_kernel<I8, EPI, 1, true, O><<<grid, kThreads, 0, s>>>(a);
        else product_stream_kernel<I8, EPI, 1, false, O><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (vec) product_stream_kernel<I8, EPI, 2, true, O><<<grid, kThreads, 0, s>>>(a);
        else product_stream_kernel<I8, EPI, 2, false, O><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

bool stream_supported(const Product &p) {
    return p.M <= kStreamRows && p.in_dtype != MOEQ_ACT_F32 && !p.a_t && !p.b_t && p.epi != EPI_GLU_BWD;
}

cudaError_t launch_product_stream(const Product &p, cudaStream_t s) {
    if (p.in_dtype == kI8) {
        if (p.epi == EPI_GLU)
            return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, EPI_GLU, float>(p, s)
                                               : launch_t<true, EPI_GLU, __nv_bfloat16>(p, s);
        return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, EPI_STORE, float>(p, s)
                                           : launch_t<true, EPI_STORE, __nv_bfloat16>(p, s);
    }
    return launch_t<false, EPI_GLU, __nv_bfloat16>(p, s);
}

}  // namespace dense
}  // namespace moeq
