// The launches of moeq_quant_i8 on the host: cudaLaunchKernelExC is wrapped by
// one that prints the grid.  Reads "n_rows n_cols" from stdin.
#include <cuda_runtime.h>

#include <cstdio>

#include "moeq.h"

extern "C" cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **) {
    std::printf("%u %u %u %u\n", c->gridDim.x, c->gridDim.y, c->gridDim.z, c->blockDim.x);
    return cudaSuccess;
}

int main() {
    int rows, cols;
    while (std::scanf("%d %d", &rows, &cols) == 2)
        if (moeq_quant_i8(reinterpret_cast<void *>(1ll << 40), MOEQ_ACT_BF16, rows, cols, cols, reinterpret_cast<int8_t *>(1ll << 50),
                          cols, reinterpret_cast<float *>(1ll << 52), nullptr) != MOEQ_OK)
            std::printf("refused\n");
    return 0;
}
