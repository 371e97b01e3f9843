// dense.cuh -- what the kernels of the dense operators (quant_i8.cu,
// dense_*.cu) and their entry points (dense_api.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "async.cuh"
#include "internal.cuh"

namespace moeq {
namespace dense {

// What a product kernel does with its sums.
enum Epi : int {
    EPI_STORE = 0,    // out = acc (scaled for int8)
    EPI_GLU = 1,      // out = silu(acc0) acc1; keep[0/1] = acc0 / acc1 where given
    EPI_GLU_BWD = 2   // keep[0/1] = gradients of acc0 / acc1 for the gradient dh of silu(acc0) acc1
};

// out[z] = sum over segments s of A_s B_s^T, or with two B (EPI_GLU*) both
// products of one A.  All strides in elements.
struct Product {
    // rows of A (M) and of B (N), reduction length of one segment
    long long M = 0, N = 0, K = 0;
    int nseg = 1;     // segments along the reduction (dx: gate, then up)
    int nbatch = 1;   // independent products of one B (dW: gate, up)
    const void *a[2] = {nullptr, nullptr};   // per segment, or per batch
    long long ald = 0;
    bool a_t = false;                        // A is stored [K][M]
    const void *b[2] = {nullptr, nullptr};   // per segment, or gate / up
    long long bld[2] = {0, 0};
    bool b_t = false;                        // B is stored [K][N]
    const float *a_scale = nullptr;          // int8: [M]
    const float *b_scale[2] = {nullptr, nullptr};   // int8: [N]
    void *out[2] = {nullptr, nullptr};       // per batch
    long long old[2] = {0, 0};
    void *keep[2] = {nullptr, nullptr};      // [M][N] planes, row stride kld
    bool keep_f32 = false;                   // EPI_GLU_BWD of bf16: keep is f32 (dense_stream.cu alone writes it so)
    long long kld = 0;
    const void *dh = nullptr;                // [M][N], row stride dhld (EPI_GLU_BWD)
    long long dhld = 0;
    int in_dtype = MOEQ_ACT_F32;             // moeq_dtype, or kI8
    int out_dtype = MOEQ_ACT_F32;            // of out, keep and dh
    int epi = EPI_STORE;
};
constexpr int kI8 = 100;

// sigmoid(g) = 1 / (1 + e^-g) and silu(g) = g sigmoid(g), from z = e^-|g|, which
// does not overflow: for g < 0 they are z / (1 + z) and g z / (1 + z), so that
// they fall off gradually (silu(-90) = -7e-38) instead of becoming 0 where e^-g
// leaves f32.  For bf16 results the exponential and the divide (by 1 to 2) are
// the hardware's approximations: off by at most 2 ulp each and by |g| 2^-23 (the
// rounding of g log2 e in the exponent), below 2^-16 as long as z is normal,
// against the 2^-9 of the rounding that follows.  The IEEE divide and expf made
// the gated epilogue 10 us longer at 2048 x 4096 x 2048.
template <bool FAST>
__device__ __forceinline__ float over_1_plus_z(float g, float at_plus, float at_minus) {   // (g < 0 ? at_minus z : at_plus) / (1 + z)
    const float z = FAST ? __expf(-fabsf(g)) : expf(-fabsf(g)), n = g < 0.f ? at_minus * z : at_plus;
    return FAST ? __fdividef(n, 1.0f + z) : n / (1.0f + z);
}
template <bool FAST>
__device__ __forceinline__ float sigmoid_f32(float g) {
    return over_1_plus_z<FAST>(g, 1.0f, 1.0f);
}
template <bool FAST>
__device__ __forceinline__ float silu(float g) {
    return over_1_plus_z<FAST>(g, g, g);
}
// dg and du for the gradient dh of silu(g) u
template <bool FAST>
__device__ __forceinline__ void glu_grad(float g, float u, float dh, float &dg, float &du) {
    const float s = sigmoid_f32<FAST>(g);
    dg = dh * u * (s * (1.0f + g * (1.0f - s)));
    du = dh * (g * s);
}

__device__ __forceinline__ float ld_elem(const float *p) { return __ldg(p); }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16 *p) {
    return bf16_bits_to_f32(__ldg(reinterpret_cast<const unsigned short *>(p)));
}
__device__ __forceinline__ void st_elem(float *p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes at any address p, of which `left` (any value) are inside the row
// and `before` say whether bytes before p are; zeros beyond.
__device__ __forceinline__ void load16_any(const uint8_t *p, int left, bool before, uint32_t w[4]) {
    const int off = (int)((uintptr_t)p & 3);
    if (left >= 20 && (before || !off)) {   // whole words of the row around the 16 bytes
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
        uint32_t v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = __ldg(q + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 8 * off);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * i + j < left) w[i] |= (uint32_t)__ldg(p + 4 * i + j) << (8 * j);
    }
}
// Launch as a programmatic dependent of the kernel before it on the stream:
// the kernel may start while that one drains, and waits for it (pdl_wait_primary)
// before it touches global memory.  cluster: CTAs of a cluster, 0 for the
// kernel's own.
template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Blocks of 128 threads for a pass over `rows` rows of `pieces` pieces each:
// narrow rows share a block.  A thread takes piece blockIdx.x * blockDim.x +
// threadIdx.x of rows blockIdx.y * blockDim.y + threadIdx.y.
struct RowGrid {
    dim3 grid, block;
    RowGrid(long long rows, long long pieces, int z = 1) {
        unsigned x = 4;
        while (x < 128 && x < pieces) x *= 2;
        block = dim3(x, 128 / x);
        const long long y = (rows + block.y - 1) / block.y;
        grid = dim3((unsigned)((pieces + x - 1) / x), (unsigned)(y < 16384 ? y : 16384), (unsigned)z);
    }
};

// ---- launchers ----
// bf16 and int8: A and B with 16-byte aligned bases and row strides (dense_tc.cu)
cudaError_t launch_product_tc(const Product &p, cudaStream_t s);
// dx and dW (both weights') in one launch, either of them NULL; bf16, operands
// as for launch_product_tc
cudaError_t launch_gradients_tc(const Product *dx, const Product *dw, cudaStream_t s);
// bf16 and int8, at most kStreamRows rows of A, any strides and alignment
// (dense_stream.cu); EPI_GLU_BWD: where keep is f32, at most kFewRows rows
constexpr int kStreamRows = 16, kFewRows = 4;
inline bool stream_supported(const Product &p) {
    return (p.epi == EPI_GLU_BWD ? p.keep_f32 && p.M <= kFewRows : p.M <= kStreamRows) && p.in_dtype != MOEQ_ACT_F32 && !p.a_t &&
           !p.b_t;
}
cudaError_t launch_product_stream(const Product &p, cudaStream_t s);
// bf16 and int8, K split over clusters; operands as for launch_product_tc
// (dense_skinny.cu)
cudaError_t launch_product_skinny(const Product &p, cudaStream_t s);
// Estimated time of either in ns, without a launch's common 5.5 us (bn: the tile width)
long long tc_ns(const Product *ps, int n, int sms, int *bn);
long long skinny_ns(const Product &p, int sms);
// dst (16-byte aligned base and row stride) = src, rows x cols of es-byte
// elements, strides in elements; up to three at once.
struct Copy {
    const void *src;
    long long ld;
    void *dst;
    long long dst_ld, rows, cols;
};
cudaError_t launch_pack(const Copy *c, int n, int es, cudaStream_t s);
// bf16, at most kFewRows tokens, any strides and alignment: both gradients from
// f32 gate gradients dg, du [T][dld] (dense_few.cu).  px, pw: dx and dW as for
// launch_gradients_tc, either of them NULL; their A is not read.
cudaError_t launch_few_gradients(const Product *px, const Product *pw, const float *dg, const float *du, long long dld,
                                 cudaStream_t s);
cudaError_t launch_dgate_f32(const void *dh, long long dhld, const void *gu, float *dg, float *du, long long ld, int T, int N,
                             cudaStream_t s);
// f32 products from bf16 planes (dense_planes.cu).  A matrix's planes: bf16
// [3][rows][ld], ld a multiple of 64.
struct Planes {
    const void *p = nullptr;
    long long rows = 0, cols = 0, ld = 0;
};
struct PlanesProduct {   // as Product
    long long M = 0, N = 0, K = 0;
    int nseg = 1, nbatch = 1;
    Planes a[2], b[2];           // a: per segment, or per batch; b: per segment, or gate / up
    bool a_t = false;            // a stored [K][M]; b is [K][N] but for the gated block
    void *out[2] = {nullptr, nullptr};
    long long old[2] = {0, 0};
    void *keep[2] = {nullptr, nullptr};   // f32 (EPI_GLU), or planes with `kplane` elements between them
    long long kld = 0, kplane = 0;
    const float *dh = nullptr;
    long long dhld = 0;
    int epi = EPI_STORE;
};
cudaError_t launch_product_planes(const PlanesProduct &p, cudaStream_t s);              // the gated block
cudaError_t launch_gradients_planes(const PlanesProduct *p, int n, cudaStream_t s);    // dx, dW, or both in one launch
cudaError_t launch_split(const Copy *c, int n, cudaStream_t s);   // dst: planes
cudaError_t launch_dgate_planes(const float *dh, long long dhld, const float *gu, void *dg, void *du, long long ld,
                                long long M, long long N, cudaStream_t s);
// SMs of the current device; address of its status word (dense_tc.cu).
cudaError_t sm_count(int *n);
cudaError_t status_word(uint32_t **p);
// Read the limit of the kernels' waits from the environment again (dense_tc.cu).
void read_wait_cycles();
// dg, du (row stride ld) = the gradients of the kept projections gu [2][M][N], bf16
cudaError_t launch_glu_dgate(const void *dh, long long dhld, const void *gu, void *dg, void *du, long long ld,
                             long long M, long long N, cudaStream_t s);

}  // namespace dense
}  // namespace moeq
