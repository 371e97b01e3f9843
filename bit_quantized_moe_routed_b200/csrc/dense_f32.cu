// dense_f32.cu -- f32 products of the dense operators (any sizes, strides and
// alignment), and the elementwise steps around the products.
//
// A product of f32 numbers is made of tensor-core products of 11-bit (tf32)
// parts: x = hi + lo with hi the top 11 significand bits and lo = x - hi
// (exact, 13 bits, rounded to 11 for the tensor core), and x w ~ hi_x hi_w +
// hi_x lo_w + lo_x hi_w.  The parts left out are at most 2^-21 (lo's rounding,
// twice) and 2^-20 (lo lo) of |x w|.  The tensor core adds in f32 with
// truncation, so its sums run over one slice of 32 products of each kind only
// and are then added to the total on the f32 units: a sum of K terms is off by
// about (K / 32 + 32) 2^-24 of the sum of magnitudes, at random.
// (tcgen05 keeps its sums in tensor memory, where taking them out every 32
// products would cost more than the products; mma.sync leaves them in
// registers.)
//
// Bound: the tensor cores' tf32 rate through mma.sync, a third of it for the
// three products.  A CTA of 4 warps computes 32 WM x 64 outputs (32 gate and
// the 32 up of the same outputs for the gated block: a lane holds both), a
// warp 16 WM x 32, from slices of 32 along K in a ring of shared-memory
// stages.  An operand with K contiguous lies [row][k] there, a transposed one
// [k][row], with row pitches that keep the fragments' 4-byte loads free of
// bank conflicts; copies are asynchronous, 16 bytes where the rows start on 16
// bytes, else 4.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "dense.cuh"

namespace moeq {
namespace dense {
namespace {

constexpr int kBN = 64, kBK = 32, kStages = 3;

template <int BYTES>
__device__ __forceinline__ void copy(float *dst, const float *src, int bytes) {   // zeros behind the first `bytes`
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
// Slices of ROWS rows by kBK of a matrix stored [rows][K], or [K][rows] if TR,
// in shared memory as stored: [ROWS][kPitch] or [kBK][kPitch].
template <bool TR, int ROWS, int kThreads>
struct Slice {
    static constexpr int kPitch = TR ? ROWS + 8 : kBK + 4;            // 8 or 4 mod 32: see at()
    static constexpr int kFloats = (TR ? kBK : ROWS) * kPitch;
    static constexpr int kInner = TR ? ROWS : kBK;                    // contiguous elements
    static constexpr int kPieces = ROWS * kBK / 4;
    static_assert(ROWS * kBK % kThreads == 0, "whole rounds of 4-byte copies");
    const float *g = nullptr;
    long long ld = 0;
    int rows = 0;      // inside the matrix
    bool vec = false;
    __device__ __forceinline__ void start(const void *base, long long ld_, long long r0, long long all) {
        ld = ld_;
        rows = (int)min((long long)ROWS, all - r0);
        g = static_cast<const float *>(base) + (TR ? r0 : r0 * ld);
        vec = !((uintptr_t)base & 15u) && !(ld & 3);
    }
    // k_left: columns of K left from the slice's first; nothing outside is read
    __device__ __forceinline__ void load(float *s, int k_left) {
        const int inner = TR ? rows : k_left, outer = TR ? k_left : rows;
        if (vec) {
#pragma unroll
            for (int i = 0; i < (kPieces + kThreads - 1) / kThreads; ++i) {
                const int e = i * kThreads + threadIdx.x;
                if (kPieces % kThreads && e >= kPieces) break;
                const int o = e / (kInner / 4), c = e % (kInner / 4) * 4;
                const int in = o < outer ? max(0, min(4, inner - c)) : 0;
                copy<16>(s + o * kPitch + c, in ? g + (long long)o * ld + c : g, in * 4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < ROWS * kBK / kThreads; ++i) {
                const int e = i * kThreads + threadIdx.x, o = e / kInner, c = e % kInner;
                const bool in = o < outer && c < inner;
                copy<4>(s + o * kPitch + c, in ? g + (long long)o * ld + c : g, in ? 4 : 0);
            }
        }
        g += TR ? kBK * ld : kBK;
    }
    __device__ __forceinline__ static float at(const float *s, int r, int k) { return TR ? s[k * kPitch + r] : s[r * kPitch + k]; }
};
// The tf32 parts of x: hi exactly, lo rounded (to nearest, halves away).
__device__ __forceinline__ void parts(float x, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(x) & 0xFFFFE000u;
    const float d = x - __uint_as_float(hi);
    lo = (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? 0u : __float_as_uint(d) + 0x1000u;   // inf: no second part
    if ((__float_as_uint(x) & 0x7FFFFFFFu) > 0x7F800000u) hi = 0x7FC00000u;                       // NaN stays one
}
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], const uint32_t b[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <bool TA, bool TB, int NB, int WM, int KG>
struct Layout {
    typedef Slice<TA, 32 * WM, 128 * KG> A;
    typedef Slice<TB, kBN / NB, 128 * KG> B;
    static constexpr int kStage = A::kFloats + NB * B::kFloats;
    static constexpr size_t kSmem = (size_t)kStages * kStage * 4;
};

template <int EPI, bool TA, bool TB, int WM, int KG>
__global__ void __launch_bounds__(128 * KG) product_f32_kernel(const __grid_constant__ Product p) {
    constexpr int NB = EPI == EPI_STORE ? 1 : 2, kRows = kBN / NB, BM = 32 * WM;
    typedef Layout<TA, TB, NB, WM, KG> L;
    extern __shared__ __align__(16) float smem_f[];
    const long long mt = (p.M + BM - 1) / BM;
    const int z = (int)(blockIdx.x / mt);
    const long long m0 = (blockIdx.x % mt) * BM, n0 = (long long)blockIdx.y * kRows;
    const int warp = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wm = (warp & 1) * 16 * WM, wn = (warp >> 1) * (kRows / 2);   // this warp's first row and column
    constexpr int kNT = kRows / 16;                                        // tiles of 8 columns of each B
    float acc[WM][NB][kNT][4], tot[WM][NB][kNT][4];
#pragma unroll
    for (int i = 0; i < WM * NB * kNT * 4; ++i) (&acc[0][0][0][0])[i] = (&tot[0][0][0][0])[i] = 0.f;
    typename L::A xa;
    typename L::B xb[NB];
    const int per = (int)((p.K + kBK - 1) / kBK), slices = per * p.nseg;
    int loaded = 0, k_left = 0;
    auto load = [&]() {   // the next slice, into its stage; an empty group past the last
        if (loaded < slices) {
            if (loaded == 0 || loaded == per) {
                const int seg = loaded == 0 ? 0 : 1;
                k_left = (int)p.K;
                xa.start(p.a[p.nseg > 1 ? seg : z], p.ald, m0, p.M);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int bi = NB == 2 ? b : seg;
                    xb[b].start(p.b[bi], p.bld[bi], n0, p.N);
                }
            }
            float *s = smem_f + loaded % kStages * L::kStage;
            xa.load(s, k_left);
#pragma unroll
            for (int b = 0; b < NB; ++b) xb[b].load(s + L::A::kFloats + b * L::B::kFloats, k_left);
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
        const float *a = smem_f + i % kStages * L::kStage, *b = a + L::A::kFloats;
#pragma unroll
        for (int kk = 0; kk < kBK; kk += 8 * KG) {
            const int k = kk + 8 * group;
            uint32_t ah[WM][4], al[WM][4], bh[NB][kNT][2], bl[NB][kNT][2];
#pragma unroll
            for (int q = 0; q < WM; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    parts(L::A::at(a, wm + 16 * q + g + 8 * (e & 1), k + t + 4 * (e >> 1)), ah[q][e], al[q][e]);
#pragma unroll
            for (int h = 0; h < NB; ++h)
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        parts(L::B::at(b + h * L::B::kFloats, wn + 8 * j + g, k + t + 4 * e), bh[h][j][e], bl[h][j][e]);
            // the small products first; tiles innermost: their steps do not wait for one another
#pragma unroll
            for (int o = 0; o < 3; ++o)
#pragma unroll
                for (int q = 0; q < WM; ++q)
#pragma unroll
                    for (int h = 0; h < NB; ++h)
#pragma unroll
                        for (int j = 0; j < kNT; ++j) mma(acc[q][h][j], o == 0 ? al[q] : ah[q], o == 1 ? bl[h][j] : bh[h][j]);
        }
#pragma unroll
        for (int e = 0; e < WM * NB * kNT * 4; ++e) {
            (&tot[0][0][0][0])[e] += (&acc[0][0][0][0])[e];
            (&acc[0][0][0][0])[e] = 0.f;
        }
    }
    if (KG > 1) {   // the groups' sums, in group order
        constexpr int kSums = WM * NB * kNT * 4;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float *part = smem_f + (threadIdx.x & 127);
        if (group > 0)
#pragma unroll
            for (int e = 0; e < kSums; ++e) part[((group - 1) * kSums + e) * 128] = (&tot[0][0][0][0])[e];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int r = 0; r < KG - 1; ++r)
#pragma unroll
            for (int e = 0; e < kSums; ++e) (&tot[0][0][0][0])[e] += part[(r * kSums + e) * 128];
    }
    float *out = static_cast<float *>(p.out[z]);
#pragma unroll
    for (int q = 0; q < WM; ++q)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const long long m = m0 + wm + 16 * q + g + 8 * (e >> 1), n = n0 + wn + 8 * j + 2 * t + (e & 1);
                if (m >= p.M || n >= p.N) continue;
                const float v = tot[q][0][j][e], u = tot[q][NB - 1][j][e];
                if (EPI == EPI_STORE) out[m * p.old[z] + n] = v;
                if (EPI == EPI_GLU) {
                    out[m * p.old[z] + n] = silu<false>(v) * u;
                    if (p.keep[0]) {
                        static_cast<float *>(p.keep[0])[m * p.kld + n] = v;
                        static_cast<float *>(p.keep[1])[m * p.kld + n] = u;
                    }
                }
                if (EPI == EPI_GLU_BWD) {
                    float dg, du;
                    glu_grad<false>(v, u, __ldg(static_cast<const float *>(p.dh) + m * p.dhld + n), dg, du);
                    static_cast<float *>(p.keep[0])[m * p.kld + n] = dg;
                    static_cast<float *>(p.keep[1])[m * p.kld + n] = du;
                }
            }
}

template <int EPI, bool TA, bool TB, int WM, int KG>
cudaError_t launch_wm(const Product &p, long long mt, long long nt, cudaStream_t s) {
    typedef Layout<TA, TB, EPI == EPI_STORE ? 1 : 2, WM, KG> L;
    static_assert(L::kSmem >= (size_t)(KG - 1) * WM * 16 * 4 * 128, "the groups' sums fit the ring");
    const auto kernel = product_f32_kernel<EPI, TA, TB, WM, KG>;
    static std::mutex mu;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    return launch_pdl(kernel, dim3((unsigned)mt, (unsigned)nt), 128 * KG, L::kSmem, 0, s, p);
}
template <int EPI, bool TA, bool TB>
cudaError_t launch_t(const Product &p, cudaStream_t s) {
    constexpr int kRows = EPI == EPI_STORE ? kBN : kBN / 2;
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long nt = (p.N + kRows - 1) / kRows;
    auto rows = [&](int wm) { return (p.M + 32 * wm - 1) / (32 * wm) * p.nbatch; };
    const int wm = rows(2) * nt >= 2 * sms ? 2 : 1;
    if (rows(wm) > 0x7FFFFFFFLL || nt > 65535) return cudaErrorInvalidConfiguration;
    return wm == 2 ? launch_wm<EPI, TA, TB, 2, 1>(p, rows(2), nt, s) : launch_wm<EPI, TA, TB, 1, 4>(p, rows(1), nt, s);
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

cudaError_t launch_product_f32(const Product &p, cudaStream_t s) {
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
