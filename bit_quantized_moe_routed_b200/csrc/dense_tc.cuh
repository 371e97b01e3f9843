// dense_tc.cuh -- what the tensor-core kernels of the dense operators share:
// tensor maps over strided matrices, descriptors, cluster helpers and the
// staged store of an output tile.
#pragma once

#include <cuda.h>

#include "async.cuh"
#include "dense.cuh"
#include "umma.cuh"

namespace moeq {
namespace dense {

constexpr int kRowBytes = 128;                  // bytes of K (or of 64 bf16 rows) a shared-memory row holds
constexpr long long kWaitCycles = 2000000000LL; // limit of every wait between roles: about a second

// The limit that a launch gives its kernel: kWaitCycles, or MOEQ_TEST_WAIT_CYCLES
// of the environment, read at the first call and when the status word is cleared
// (tests let a wait run out that way).
long long wait_cycles();

// Tensor map over a rows x cols matrix (row stride ld, elements of es bytes),
// 128-byte swizzle, boxes of box_rows x 128 bytes; reads outside give zeros.
// The base and the row stride are multiples of 16 bytes.
cudaError_t make_map(CUtensorMap *map, const void *base, long long rows, long long cols, long long ld, int es,
                     int box_rows);
// Tensor map over a matrix's planes, 128-byte swizzle, boxes of 64 columns x
// box_rows x box_planes; reads outside give zeros.
cudaError_t make_planes_map(CUtensorMap *map, const Planes &m, int box_rows, int box_planes);

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool test_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Bounded wait that also ends when another role of the CTA has given up.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort_flag, long long max_cycles) {
    if (test_wait_cluster(bar, parity)) return true;
    const long long t0 = clock64();
    while (!test_wait_cluster(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > max_cycles) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
// mbar_wait_abort by a whole warp: it gives up as one, as the tensor memory
// loads that follow are instructions of the warp.
__device__ __forceinline__ bool warp_wait_abort(uint64_t *bar, uint32_t parity, volatile int *abort_flag, long long max_cycles) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_abort(bar, parity, abort_flag, max_cycles));
}

// Shared-memory descriptor of an operand whose 128-byte rows run along M or
// N (stored [K][M]): 128-byte swizzle, blocks of 64 elements `lbo` bytes
// apart, groups of 8 K-rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn_sw128(const void *p, uint32_t lbo) {
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 x bf16 -> f32, or s8 x s8 -> s32.
template <bool I8>
__host__ __device__ constexpr uint32_t idesc_dense(int m, int n, bool a_mn, bool b_mn) {
    return (I8 ? (2u << 4) : (1u << 4)) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// 32 consecutive columns of this warp's 32 lanes, still in flight: follow
// with tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t r[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Write 32 rows x 32 columns, one row a lane, through the warp's 4 KB of
// shared memory, so that global stores cover whole 64- or 128-byte pieces of
// a row.  16-byte pieces are XOR-swizzled by row (no bank conflicts in either
// direction).  rows, cols: how many are inside the matrix (any value).
// vec: dst and its row stride are multiples of 16 bytes.
template <typename O>
__device__ __forceinline__ void store_32x32(uint8_t *stage, const float v[32], O *dst, long long ld, int rows, int cols,
                                            bool vec) {
    const int lane = threadIdx.x & 31;
    constexpr int kPieces = sizeof(O) * 32 / 16;          // 16-byte pieces of a row: 4 (bf16) or 8 (f32)
    constexpr int kPer = 16 / sizeof(O);
    auto slot = [&](int r, int c) {
        return kPieces == 8 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    };
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sizeof(O) == 4) w[i] = __float_as_uint(v[c * 4 + (i & 3)]);
            else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[(c * 8 + 2 * i) & 31], v[(c * 8 + 2 * i + 1) & 31]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        *reinterpret_cast<uint4 *>(stage + slot(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (vec) {
        const int c = lane % kPieces;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 32 / kPieces) {
            const int r = r0 + lane / kPieces;
            if (r >= rows || c * kPer >= cols) continue;
            const uint4 w = *reinterpret_cast<const uint4 *>(stage + slot(r, c));
            O *d = dst + (long long)r * ld + c * kPer;
            if (c * kPer + kPer <= cols) *reinterpret_cast<uint4 *>(d) = w;
            else {
                const O *e = reinterpret_cast<const O *>(&w);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (c * kPer + i < cols) d[i] = e[i];
            }
        }
    } else if (lane < cols) {   // one element a lane, one row at a time
        for (int r = 0; r < min(rows, 32); ++r)
            dst[(long long)r * ld + lane] = *reinterpret_cast<const O *>(stage + slot(r, lane / kPer) + lane % kPer * sizeof(O));
    }
}
// A lane's row of 32 x 32 bf16 elements at src into v, zeros outside.  left:
// elements of a row from src on; before: whether a row has some before src.
__device__ __forceinline__ void load_32x32(float v[32], const __nv_bfloat16 *src, long long ld, int rows, long long left,
                                           bool before, bool vec) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *row = src + (long long)(lane < rows ? lane : 0) * ld;
    uint4 w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int in = lane < rows ? (int)max(0LL, min(64LL, (left - 8 * c) * 2)) : 0;   // bytes of the row
        if (vec && in >= 16) w[c] = __ldg(reinterpret_cast<const uint4 *>(row) + c);
        else {
            uint32_t u[4];
            load16_any(reinterpret_cast<const uint8_t *>(row + 8 * c), in, before || c > 0, u);
            w[c] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * c + i] = bf16_bits_to_f32(i & 1 ? u[i >> 1] >> 16 : u[i >> 1] & 0xFFFFu);
    }
}

}  // namespace dense
}  // namespace moeq
