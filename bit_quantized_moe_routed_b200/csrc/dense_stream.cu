// dense_stream.cu -- products of the dense operators for a few rows of A (the
// tokens of a decode step): the weights stream once through registers.
//
// Bound: HBM, the bytes of the weights.  A CTA takes 16 weight rows (8 gate
// and the 8 up rows of the same outputs for the gated block) over all of K;
// its warps split K.  A lane loads 32 consecutive bytes of a row, which are
// the A fragments of four tensor-core steps under a permutation of K that x
// shares (the sum does not depend on the order of K), so the weights go from
// HBM to mma.sync without shared memory, kChunk = 4 blocks of 128 bytes of K (8
// loads of 32 bytes a lane) always in flight.  The tokens are the N = 8 columns of
// a step, two steps for up to 16.  tcgen05 would need the weights in shared memory first and pads N
// to its M; at 8 columns the legacy path leaves the tensor cores far from
// their limit.  A lane ends with the gate and the up sum of the same outputs;
// the warps' partial sums meet in shared memory in a fixed order.
//
// Operands at any address and row stride: rows on 32 bytes are read 32 bytes
// at a time, rows on 16 bytes 16, others in the three aligned 16-byte pieces
// around the 32 bytes, shifted into place.
#include <type_traits>

#include "dense_tc.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

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
    const void *dh;
    long long dhld;
};

// The 32 bytes a lane takes of a row's 128-byte block, `left` of which (any
// value) are in the row; zeros beyond.  ALIGN: 32 or 16 (base, row stride and
// row length are multiples of it, so a piece is inside the row or not) or 0
// (anything; before / after: the bytes up to 15 before and 47 behind p are the
// matrix's too, whatever they hold).  The loads go into kWords words and are
// put in place by settle() when they are used: shifting them at once would wait
// for each in turn (24 against 17 us at 1 x 4095 x 2048).
template <int ALIGN>
struct Piece {
    static constexpr int kWords = ALIGN ? 8 : 12;
    uint32_t v[kWords];
    __device__ __forceinline__ static bool whole(const uint8_t *p, int left, bool before, bool after) {
        const int off = (int)((uintptr_t)p & 15);
        return left > 0 && (after || left >= 48 - off) && (before || !off);
    }
    __device__ __forceinline__ void load(const uint8_t *p, int left, bool before, bool after) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = 0;
        if (ALIGN == 32 && left > 0)
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                         : "l"(p));
        if (ALIGN == 16) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (left > 16 * h) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p) + h);
                    v[4 * h] = q.x, v[4 * h + 1] = q.y, v[4 * h + 2] = q.z, v[4 * h + 3] = q.w;
                }
        }
        if (ALIGN == 0 && whole(p, left, before, after)) {
            const uint4 *a = reinterpret_cast<const uint4 *>((uintptr_t)p & ~(uintptr_t)15);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint4 q = __ldg(a + i);
                v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
            }
        }
    }
    __device__ __forceinline__ void settle(const uint8_t *p, int left, bool before, bool after) {
        if (ALIGN) return;
        if (left <= 0) return;   // zeros
        if (!whole(p, left, before, after)) {
            load16_any(p, left, before, v);
            load16_any(p + 16, left - 16, true, v + 4);
            return;
        }
        const int off = (int)((uintptr_t)p & 15);
        const bool two = off & 8, one = off & 4;
#pragma unroll
        for (int i = 0; i < 10; ++i) v[i] = two ? v[(i + 2) % kWords] : v[i];
#pragma unroll
        for (int i = 0; i < 9; ++i) v[i] = one ? v[(i + 1) % kWords] : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = left - 4 * i;
            v[i] = __funnelshift_r(v[i], v[(i + 1) % kWords], 8 * (off & 3)) &
                   (n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u));
        }
    }
};

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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
template <bool I8, int EPI, int ALIGN, int NT, typename O>
__global__ void __launch_bounds__(kThreads, 2) product_stream_kernel(const __grid_constant__ StreamArgs p) {
    typedef typename Sum<I8>::type E;
    __shared__ E part[kWarps][NT][4][32];
    constexpr int kChunk = ALIGN ? 4 : 2;                 // 128-byte blocks of K a warp has in flight
    constexpr int kAhead = NT == 1 ? 2 : 1;               // blocks by which the tokens are loaded ahead
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
    const int blocks = (p.kbytes + 127) / 128, share = (blocks + kWarps - 1) / kWarps;
    const int b_first = warp * share, b_end = min(blocks, (warp + 1) * share);
    Piece<ALIGN> a[kChunk][2], xr[kAhead][NT];
    // unaligned rows: whether other rows of the matrix lie before and behind this
    // lane's (strides of 48 bytes at least)
    const bool wide0 = p.ldw[0] >= 48, wide1 = (EPI == EPI_STORE ? p.ldw[0] : p.ldw[1]) >= 48;
    auto of_w = [&](int b, auto f0, auto f1) {   // f(address, bytes left, before, after) of this lane's rows at block b
        const int k = b * 128 + 32 * t;
        const bool in = b < b_end;
        f0(w0 + k, in ? k0 - k : 0, k > 0 || (wide0 && r0 > 0), wide0 && r0 < p.N - 1);
        f1(w1 + k, in ? k1 - k : 0, k > 0 || (wide1 && r1 > 0), wide1 && r1 < p.N - 1);
    };
    auto of_x = [&](int b, int i, auto f) {
        const int k = b * 128 + 32 * t, tok = 8 * i + g;
        f(p.x + (long long)min(tok, p.T - 1) * p.ldx + k, b < b_end && tok < p.T ? p.kbytes - k : 0,
          k > 0 || (p.ldx >= 48 && tok > 0), p.ldx >= 48 && tok < p.T - 1);
    };
    auto load_w = [&](int j, int b) {
        of_w(b, [&](auto... v) { a[j][0].load(v...); }, [&](auto... v) { a[j][1].load(v...); });
    };
    auto load_x = [&](int j, int b) {
#pragma unroll
        for (int i = 0; i < NT; ++i) of_x(b, i, [&](auto... v) { xr[j][i].load(v...); });
    };
    // the first blocks on their way to L2 while the kernel before drains
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
        const int k = (b_first + j) * 128 + 32 * t;
        if (b_first + j < b_end && k < k0) prefetch_l2(w0 + k);
        if (b_first + j < b_end && k < k1) prefetch_l2(w1 + k);
    }
    pdl_wait_primary();
    pdl_launch_dependents();
#pragma unroll
    for (int j = 0; j < kChunk; ++j) load_w(j, b_first + j);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load_x(j, b_first + j);
    for (int b0 = b_first; b0 < b_end; b0 += kChunk) {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {   // a block past the share's end is zeros on both sides
            of_w(b0 + j, [&](auto... v) { a[j][0].settle(v...); }, [&](auto... v) { a[j][1].settle(v...); });
            const uint32_t *w = a[j][0].v, *u = a[j][1].v;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                of_x(b0 + j, i, [&](auto... v) { xr[j % kAhead][i].settle(v...); });
                const uint32_t *x = xr[j % kAhead][i].v;
#pragma unroll
                for (int q = 0; q < 8; q += 2) step(c[i], w[q], u[q], w[q + 1], u[q + 1], x[q], x[q + 1]);
            }
            load_w(j, b0 + kChunk + j);
            load_x(j % kAhead, b0 + kAhead + j);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[warp][i][q][lane] = c[i][q];
    __syncthreads();
    // one output a thread: the lane and component that hold its sums
    const int r = threadIdx.x % per, tok = threadIdx.x / per, n = n0 + r;
    if (tok < p.T && n < p.N) {
        const int i = tok >> 3, src = (r & 7) * 4 + ((tok & 7) >> 1), q = (tok & 1) + (r >> 3) * 2;
        E s0 = 0, s1 = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s0 += part[w][i][q][src];
            if (EPI != EPI_STORE) s1 += part[w][i][q + 2][src];
        }
        float v0 = (float)s0, v1 = (float)s1;
        if (I8) {
            const float sx = __ldg(p.a_scale + tok);
            v0 = v0 * sx * __ldg(p.b_scale[0] + n);
            if (EPI != EPI_STORE) v1 = v1 * sx * __ldg(p.b_scale[1] + n);
        }
        O *out = static_cast<O *>(p.out) + (long long)tok * p.old + n;
        if (EPI == EPI_GLU) {
            st_elem(out, silu<sizeof(O) == 2>(v0) * v1);
            if (!I8 && p.keep[0]) {
                st_elem(static_cast<O *>(p.keep[0]) + (long long)tok * p.kld + n, v0);
                st_elem(static_cast<O *>(p.keep[1]) + (long long)tok * p.kld + n, v1);
            }
        } else if (EPI == EPI_GLU_BWD) {   // f32, as the gradients of few tokens take them
            float dg, du;
            glu_grad<false>(v0, v1, ld_elem(static_cast<const __nv_bfloat16 *>(p.dh) + (long long)tok * p.dhld + n), dg, du);
            static_cast<float *>(p.keep[0])[(long long)tok * p.kld + n] = dg;
            static_cast<float *>(p.keep[1])[(long long)tok * p.kld + n] = du;
        } else {
            st_elem(out, v0);
        }
    }
}

template <bool I8, int EPI, typename O>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    const int es = I8 ? 1 : 2;
    StreamArgs a{};
    // the alignment that every row of every operand has
    unsigned long long low = (uintptr_t)p.a[0] | (p.M > 1 ? p.ald * es : 0) | p.K * es;
    for (int i = 0; i < (EPI != EPI_STORE ? 2 : 1); ++i) {
        a.w[i] = static_cast<const uint8_t *>(p.b[i]);
        a.ldw[i] = p.bld[i] * es;
        a.b_scale[i] = p.b_scale[i];
        a.keep[i] = p.keep[i];
        low |= (uintptr_t)p.b[i] | (p.N > 1 ? a.ldw[i] : 0);
    }
    a.x = static_cast<const uint8_t *>(p.a[0]);
    a.ldx = p.ald * es;
    a.T = (int)p.M;
    a.N = (int)p.N;
    a.kbytes = (int)(p.K * es);
    a.a_scale = p.a_scale;
    a.out = p.out[0];
    a.old = p.old[0];
    a.kld = p.kld;
    a.dh = p.dh;
    a.dhld = p.dhld;
    const int per = EPI == EPI_STORE ? 16 : 8;
    const int grid = (a.N + per - 1) / per;
    auto pick = [&](auto align) {
        constexpr int A = decltype(align)::value;
        if constexpr (EPI == EPI_GLU_BWD) return product_stream_kernel<I8, EPI, A, 1, O>;
        else return a.T <= 8 ? product_stream_kernel<I8, EPI, A, 1, O> : product_stream_kernel<I8, EPI, A, 2, O>;
    };
    const auto kernel = !(low & 31) ? pick(std::integral_constant<int, 32>{})
                                    : (!(low & 15) ? pick(std::integral_constant<int, 16>{})
                                                   : pick(std::integral_constant<int, 0>{}));
    return launch_pdl(kernel, dim3((unsigned)grid), kThreads, 0, 0, s, a);
}

}  // namespace

cudaError_t launch_product_stream(const Product &p, cudaStream_t s) {
    if (!stream_supported(p)) return cudaErrorInvalidValue;
    if (p.in_dtype == kI8) {
        if (p.epi == EPI_GLU)
            return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, EPI_GLU, float>(p, s)
                                               : launch_t<true, EPI_GLU, __nv_bfloat16>(p, s);
        return p.out_dtype == MOEQ_ACT_F32 ? launch_t<true, EPI_STORE, float>(p, s)
                                           : launch_t<true, EPI_STORE, __nv_bfloat16>(p, s);
    }
    return p.epi == EPI_GLU_BWD ? launch_t<false, EPI_GLU_BWD, __nv_bfloat16>(p, s) : launch_t<false, EPI_GLU, __nv_bfloat16>(p, s);
}

}  // namespace dense
}  // namespace moeq
