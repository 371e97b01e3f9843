// quant_i8.cu -- rows to 8-bit integers with one scale each: the operands of
// the int8 products (activations per token, weights per output channel).
//
//   a = max |x|,  scale = a / 127,  q = rne(127 x / a)
//
// The integer is defined on the exact quotient, so that it does not depend on
// how the quotient is formed.
// bf16: 127 x has 15 significand bits and a 8, so the quotient is a half or at
// least 1 / 510 away from every half.  t0 = 127 x (1 / a), then t = t0 + (127 x -
// t0 a) (1 / a) in two fma: t differs from the quotient by 2^-46 of it before
// its own rounding, so a half comes out exactly and rint(t) is the integer.
// f32: t = x (127 / a) is off by at most 127 * 3 * 2^-24 < 2.3e-5 (two roundings
// of half an ulp, with the margin of one more), so rint(t) is the integer
// unless t lies within 3e-5 of a half h.  There the sign of 127 x - h a decides,
// exactly: with p = rn(h a) and e = h a - p (one fma, exact), 127 x - p is exact
// in one fma too (127 x and p agree to within 2^-18, and their difference is a
// multiple of half an ulp of a or x), so 127 x is above, at or below the half as
// 127 x - p is above, at or below e.
// Rows whose a leaves the range in which these products are normal take f64 for
// every element: 127 x has at most 31 significand bits, and its f64 quotient by
// a 24-bit value is a half exactly when the true one is and otherwise on the
// same side of it.
//
// Bound: HBM.  A row is read once (its vectors stay in registers, as loaded,
// between the maximum and the rounding; longer rows are read again from L2)
// and written once.  Rows of up to 1024 columns take a warp each, up to 4096
// four warps, longer ones eight.
#include <type_traits>

#include "dense.cuh"

namespace moeq {
namespace {

constexpr int kQThreads = 256;
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, held in the low bits

// Eight elements as loaded, and as f32.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 a;
    static constexpr int kKeep = 4;     // vectors a thread keeps: 16 registers
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? a.x : (i < 4 ? a.y : (i < 6 ? a.z : a.w));
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
    // max of |x| as bits (of f32): ordered like the values, NaN above infinity
    __device__ __forceinline__ uint32_t amax() const {
        const uint32_t k = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
        return max(m >> 16, m & 0xFFFFu) << 16;
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    static constexpr int kKeep = 4;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ float get(int i) const {
        const float4 &v = i < 4 ? a : b;
        return (i & 3) == 0 ? v.x : ((i & 3) == 1 ? v.y : ((i & 3) == 2 ? v.z : v.w));
    }
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(get(i)) & 0x7FFFFFFFu);
        return m;
    }
};

struct RowScale {
    float a, inv;   // inv: 1 / a (bf16) or 127 / a (f32)
};
constexpr float kSure = 0.49997f;       // |t - rint(t)| up to which rint(t) is sure
__device__ __forceinline__ int quant_wide(float x, float a) { return (int)rint((double)x * 127.0 / (double)a); }
// t = x r.inv with |t - rint(t)| > kSure: which side of the half next to t
__device__ __forceinline__ int quant_half(float x, float t, float a) {
    const float n = rintf(t), h = n + copysignf(0.5f, t - n);
    const float p = h * a, e = fmaf(h, a, -p), d = fmaf(x, 127.0f, -p);
    const int k = (int)floorf(h);
    return d > e ? k + 1 : (d < e ? k : k + (k & 1));
}
// bf16: the quotient, exact where it is a half (see above)
__device__ __forceinline__ float quotient(float x, const RowScale &r) {
    const float v = 127.0f * x, t0 = v * r.inv;
    return fmaf(fmaf(-t0, r.a, v), r.inv, t0);
}
template <typename T>
__device__ __forceinline__ int quant1(float x, const RowScale &r) {
    if (sizeof(T) == 2) return (int)rintf(quotient(x, r));
    const float t = x * r.inv, n = rintf(t);
    return fabsf(t - n) > kSure ? quant_half(x, t, r.a) : (int)n;
}
template <typename T>
__device__ __forceinline__ uint2 quant8(const Vec8<T> &v, const RowScale &r) {
    uint32_t w[2];
    float far = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = v.get(4 * h + i), t = sizeof(T) == 2 ? quotient(x, r) : x * r.inv, mm = t + kMagic;
            if (sizeof(T) == 4) far = fmaxf(far, fabsf(t - (mm - kMagic)));
            m[i] = __float_as_uint(mm);
        }
        w[h] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
    }
    if (sizeof(T) == 4 && far > kSure) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t q = (uint32_t)quant1<T>(v.get(i), r) & 0xFFu;
            w[i >> 2] = (w[i >> 2] & ~(0xFFu << (8 * (i & 3)))) | (q << (8 * (i & 3)));
        }
    }
    return make_uint2(w[0], w[1]);
}

// TPR threads per row, VEC: 16-byte aligned rows of x, 8-byte aligned rows of q
template <typename T, int TPR, bool VEC>
__global__ void __launch_bounds__(kQThreads) quant_i8_kernel(const T *__restrict__ x, long long ldx, int rows, int cols,
                                                             int8_t *__restrict__ q, long long ldq,
                                                             float *__restrict__ scale) {
    constexpr int kKeep = Vec8<T>::kKeep, kWarps = TPR / 32;
    __shared__ uint32_t part[kQThreads / 32];
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (kQThreads / TPR) + threadIdx.x / TPR;
    const bool live = row < rows;
    const T *xr = x + (live ? row : 0) * ldx;
    const int nv = VEC && live ? cols / 8 : 0;     // whole vectors; the rest by element
    Vec8<T> keep[kKeep];
    uint32_t m = 0;
    pdl_wait_primary();
    pdl_launch_dependents();
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
        if (t + j * TPR < nv) keep[j].load(xr + 8LL * (t + j * TPR));
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
        if (t + j * TPR < nv) m = max(m, keep[j].amax());
    for (int v = t + kKeep * TPR; v < nv; v += TPR) {
        Vec8<T> e;
        e.load(xr + 8LL * v);
        m = max(m, e.amax());
    }
    if (live)
        for (int c = 8 * nv + t; c < cols; c += TPR)
            m = max(m, __float_as_uint(dense::ld_elem(xr + c)) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        const int first = (threadIdx.x / TPR) * kWarps;
        m = part[first];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) m = max(m, part[first + i]);
    }
    if (!live) return;
    const bool finite = m < 0x7F800000u;
    RowScale r;
    r.a = __uint_as_float(m);
    r.inv = (sizeof(T) == 2 ? 1.0f : 127.0f) / r.a;
    if (t == 0) scale[row] = finite ? r.a / 127.0f : __uint_as_float(0x7FC00000u);
    const bool zero = !finite || m == 0;
    int8_t *qr = q + row * ldq;
    if (!zero && !(r.a > 1e-30f && r.a < 1e36f)) {   // products of such a row leave f32's normal range
#pragma unroll 1
        for (int c = t; c < cols; c += TPR) qr[c] = (int8_t)quant_wide(dense::ld_elem(xr + c), r.a);
        return;
    }
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int v = t + j * TPR;
        if (v < nv) *reinterpret_cast<uint2 *>(qr + 8LL * v) = zero ? make_uint2(0, 0) : quant8(keep[j], r);
    }
    for (int v = t + kKeep * TPR; v < nv; v += TPR) {
        Vec8<T> e;
        e.load(xr + 8LL * v);
        *reinterpret_cast<uint2 *>(qr + 8LL * v) = zero ? make_uint2(0, 0) : quant8(e, r);
    }
    for (int c = 8 * nv + t; c < cols; c += TPR) qr[c] = zero ? 0 : (int8_t)quant1<T>(dense::ld_elem(xr + c), r);
}

template <typename T>
cudaError_t launch(const void *x, int rows, int cols, long long ldx, int8_t *q, long long ldq, float *scale,
                   cudaStream_t s) {
    const T *xt = static_cast<const T *>(x);
    const bool vec = !((uintptr_t)x & 15u) && !((ldx * sizeof(T)) & 15u) && !((uintptr_t)q & 7u) && !(ldq & 7);
    auto run = [&](auto tpr) {
        constexpr int kTpr = decltype(tpr)::value;
        const long long per = kQThreads / kTpr, grid = (rows + per - 1) / per;   // rows reach 2^31 - 1
        return dense::launch_pdl(vec ? quant_i8_kernel<T, kTpr, true> : quant_i8_kernel<T, kTpr, false>, dim3((unsigned)grid),
                                 kQThreads, 0, 0, s, xt, ldx, rows, cols, q, ldq, scale);
    };
    if (cols <= 1024) return run(std::integral_constant<int, 32>{});
    if (cols <= 4096) return run(std::integral_constant<int, 128>{});
    return run(std::integral_constant<int, 256>{});
}

}  // namespace

cudaError_t launch_quant_i8(const void *x, int dtype, int rows, int cols, long long ldx, int8_t *q, long long ldq,
                            float *scale, cudaStream_t s) {
    return dtype == MOEQ_ACT_F32 ? launch<float>(x, rows, cols, ldx, q, ldq, scale, s)
                                 : launch<__nv_bfloat16>(x, rows, cols, ldx, q, ldq, scale, s);
}

}  // namespace moeq
