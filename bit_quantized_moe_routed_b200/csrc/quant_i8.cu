// quant_i8.cu -- rows to 8-bit integers with one scale each: the operands of
// the int8 products (activations per token, weights per output channel).
//
//   a = max |x|,  scale = a / 127,  q = rne(127 x / a)
//
// The integer is defined on the exact quotient, so that it does not depend on
// how the quotient is formed.  t = x (127 / a) in f32 is off by at most
// 127 * 3 * 2^-24 < 2.3e-5 (two roundings of a half ulp each, one of them
// relative to 127 / a, with the margin of one more), so rint(t) is that
// integer unless t lies within 1e-4 of a half; there (about one element in
// 5000, and every exact half) the quotient is formed in f64: 127 x has at
// most 31 significand bits and the f64 quotient of it by a 24-bit value
// equals a half exactly when the true one does and otherwise stays on its
// side of it (they differ by at least 2^-25, f64 rounds at 2^-47).  Rows
// whose a leaves the range in which 127 / a and x (127 / a) are normal take
// f64 for every element.
//
// Bound: HBM.  A row is read once (kept in registers between the maximum and
// the rounding up to kKeep vectors a thread, read again from L2 beyond that)
// and written once.  Rows of up to 1024 columns take a warp each (no block
// barrier, eight rows in flight per CTA), longer ones a CTA.
#include "dense.cuh"

namespace moeq {
namespace {

constexpr int kQThreads = 256;
constexpr int kKeep = 4;   // vectors of 8 elements a thread keeps

__device__ __forceinline__ void load8(const float *p, float v[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float v[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

struct RowScale {
    float a, inv;
    bool wide;   // take f64 for every element
};
__device__ __forceinline__ int quant1(float x, const RowScale &r) {
    if (!r.wide) {
        const float t = x * r.inv, q = rintf(t);
        if (fabsf(fabsf(t - q) - 0.5f) > 1e-4f) return (int)q;
    }
    return (int)rint((double)x * 127.0 / (double)r.a);
}

// TPR threads per row, VEC: 16-byte aligned rows of x, 8-byte aligned rows of q
template <typename T, int TPR, bool VEC>
__global__ void __launch_bounds__(kQThreads) quant_i8_kernel(const T *__restrict__ x, long long ldx, int rows, int cols,
                                                             int8_t *__restrict__ q, long long ldq,
                                                             float *__restrict__ scale) {
    __shared__ uint32_t part[kQThreads / 32];
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (kQThreads / TPR) + threadIdx.x / TPR;
    const bool live = row < rows;
    const T *xr = x + (live ? row : 0) * ldx;
    const int nv = VEC ? cols / 8 : 0;     // whole vectors; the rest by element
    float keep[kKeep][8];
    uint32_t m = 0;   // |x| as bits: ordered like the values, NaN above infinity
    if (live) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            const int v = t + j * TPR;
            if (v < nv) {
                load8(xr + 8LL * v, keep[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(keep[j][i]) & 0x7FFFFFFFu);
            }
        }
        for (int v = t + kKeep * TPR; v < nv; v += TPR) {
            float e[8];
            load8(xr + 8LL * v, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(e[i]) & 0x7FFFFFFFu);
        }
        for (int c = 8 * nv + t; c < cols; c += TPR)
            m = max(m, __float_as_uint(dense::ld_elem(xr + c)) & 0x7FFFFFFFu);
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int i = 1; i < kQThreads / 32; ++i) m = max(m, part[i]);
    }
    if (!live) return;
    const bool finite = m < 0x7F800000u;
    RowScale r;
    r.a = __uint_as_float(m);
    r.inv = 127.0f / r.a;
    r.wide = !(r.a > 1e-30f && r.a < 1e36f);
    if (t == 0) scale[row] = finite ? r.a / 127.0f : __uint_as_float(0x7FC00000u);
    const bool zero = !finite || m == 0;
    int8_t *qr = q + row * ldq;
    auto put8 = [&](int v, const float e[8]) {
        uint32_t w[2] = {0, 0};
        if (!zero) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)quant1(e[i], r) & 0xFFu) << (8 * (i & 3));
        }
        *reinterpret_cast<uint2 *>(qr + 8LL * v) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int v = t + j * TPR;
        if (v < nv) put8(v, keep[j]);
    }
    for (int v = t + kKeep * TPR; v < nv; v += TPR) {
        float e[8];
        load8(xr + 8LL * v, e);
        put8(v, e);
    }
    for (int c = 8 * nv + t; c < cols; c += TPR) qr[c] = zero ? 0 : (int8_t)quant1(dense::ld_elem(xr + c), r);
}

template <typename T>
cudaError_t launch(const void *x, int rows, int cols, long long ldx, int8_t *q, long long ldq, float *scale,
                   cudaStream_t s) {
    const T *xt = static_cast<const T *>(x);
    const bool vec = !((uintptr_t)x & 15u) && !((ldx * sizeof(T)) & 15u) && !((uintptr_t)q & 7u) && !(ldq & 7);
    if (cols <= 1024) {
        const int grid = (rows + kQThreads / 32 - 1) / (kQThreads / 32);
        if (vec) quant_i8_kernel<T, 32, true><<<grid, kQThreads, 0, s>>>(xt, ldx, rows, cols, q, ldq, scale);
        else quant_i8_kernel<T, 32, false><<<grid, kQThreads, 0, s>>>(xt, ldx, rows, cols, q, ldq, scale);
    } else {
        if (vec) quant_i8_kernel<T, kQThreads, true><<<rows, kQThreads, 0, s>>>(xt, ldx, rows, cols, q, ldq, scale);
        else quant_i8_kernel<T, kQThreads, false><<<rows, kQThreads, 0, s>>>(xt, ldx, rows, cols, q, ldq, scale);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_i8(const void *x, int dtype, int rows, int cols, long long ldx, int8_t *q, long long ldq,
                            float *scale, cudaStream_t s) {
    return dtype == MOEQ_ACT_F32 ? launch<float>(x, rows, cols, ldx, q, ldq, scale, s)
                                 : launch<__nv_bfloat16>(x, rows, cols, ldx, q, ldq, scale, s);
}

}  // namespace moeq
