// The entry points of the dense operators (dense_api.cu) over launchers that
// launch nothing: each notes what its kernel would write and read, so that the
// workspace's layout, the kernels chosen and the types they exchange can be
// checked on the host.
//
// Reads cases "T H I off16 dtype gu dx dw faster" from stdin (off16: rows that do not start on
// 16 bytes; faster: the kernel whose estimate is the smaller one, 0 tiles, 1
// clusters), prints "ok" or what is wrong with each.
#include <stdint.h>

#include <cstdio>
#include <string>
#include <vector>

#include "dense.cuh"

namespace {

struct Region {
    const char *p;
    long long ld, rows, cols;
    int es;
    bool has(const void *q, long long ld_, long long rows_, long long cols_, int es_) const {
        return p == q && ld == ld_ && rows == rows_ && cols == cols_ && es == es_;
    }
};
const char *g_ws;
long long g_bytes;
int g_faster;
std::vector<Region> g_written;   // in the workspace, by the steps so far
std::string g_wrong;

void wrong(const std::string &s) {
    if (g_wrong.empty()) g_wrong = s;
}
void write(const char *who, const void *p, long long ld, long long rows, long long cols, int es) {
    const char *b = static_cast<const char *>(p), *e = b + ((rows - 1) * ld + cols) * es;
    if (b < g_ws || e > g_ws + g_bytes)
        wrong(std::string(who) + " writes to byte " + std::to_string(e - g_ws) + " of a workspace of " + std::to_string(g_bytes));
    for (const Region &r : g_written)
        if (b < r.p + ((r.rows - 1) * r.ld + r.cols) * r.es && r.p < e) wrong(std::string(who) + " writes over another part");
    g_written.push_back(Region{b, ld, rows, cols, es});
}
// what lies in the workspace is read as it was written
void read(const char *who, const void *p, long long ld, long long rows, long long cols, int es) {
    const char *b = static_cast<const char *>(p);
    if (b < g_ws || b >= g_ws + g_bytes) return;
    for (const Region &r : g_written)
        if (r.has(p, ld, rows, cols, es)) return;
    wrong(std::string(who) + " reads what no step has written so");
}

}  // namespace

namespace moeq {
cudaError_t launch_quant_i8(const void *, int, int, int, long long, int8_t *, long long, float *, cudaStream_t) {
    return cudaSuccess;
}
namespace dense {

// the operands and the gate gradients of a product whose kernel holds dg and du in `es` bytes
void product(const char *who, const Product &p, int es) {
    for (int i = 0; i < 2; ++i) {
        if (p.a[i] && !p.a_t) read(who, p.a[i], p.ald, p.M, p.K, 2);
        if (p.a[i] && p.a_t) read(who, p.a[i], p.ald, p.K, p.M, 2);
        if (p.b[i] && !p.b_t) read(who, p.b[i], p.bld[i], p.N, p.K, 2);
        if (p.b[i] && p.b_t) read(who, p.b[i], p.bld[i], p.K, p.N, 2);
    }
    if (p.epi == EPI_GLU_BWD)
        for (int i = 0; i < 2; ++i) write(who, p.keep[i], p.kld, p.M, p.N, es);
}
cudaError_t launch_product_stream(const Product &p, cudaStream_t) {
    product("stream kernel", p, 4);
    return cudaSuccess;
}
cudaError_t launch_product_tc(const Product &p, cudaStream_t) {
    product("tile kernel", p, 2);
    return cudaSuccess;
}
cudaError_t launch_product_skinny(const Product &p, cudaStream_t) {
    product("cluster kernel", p, 2);
    return cudaSuccess;
}
cudaError_t launch_gradients_tc(const Product *dx, const Product *dw, cudaStream_t) {
    if (dx) product("tile kernel, dx", *dx, 2);
    if (dw) product("tile kernel, dW", *dw, 2);
    return cudaSuccess;
}
long long tc_ns(const Product *, int, int, int *bn) {
    *bn = 256;
    return 100000;
}
long long skinny_ns(const Product &, int) { return g_faster ? 1000 : 1000000; }
cudaError_t launch_pack(const Copy *c, int n, int es, cudaStream_t) {
    for (int i = 0; i < n; ++i) write("pack", c[i].dst, c[i].dst_ld, c[i].rows, c[i].cols, es);
    return cudaSuccess;
}
cudaError_t launch_few_gradients(const Product *px, const Product *pw, const float *dg, const float *du, long long dld,
                                 cudaStream_t) {
    const long long T = px ? px->M : pw->K, I = px ? px->K : pw->M;
    read("few-token kernel", dg, dld, T, I, 4);
    read("few-token kernel", du, dld, T, I, 4);
    return cudaSuccess;
}
cudaError_t launch_dgate_f32(const void *, long long, const void *, float *dg, float *du, long long ld, int T, int N,
                             cudaStream_t) {
    write("f32 gate gradients", dg, ld, T, N, 4);
    write("f32 gate gradients", du, ld, T, N, 4);
    return cudaSuccess;
}
cudaError_t launch_glu_dgate(const void *, long long, const void *, void *dg, void *du, long long ld, long long M, long long N,
                             cudaStream_t) {
    write("bf16 gate gradients", dg, ld, M, N, 2);
    write("bf16 gate gradients", du, ld, M, N, 2);
    return cudaSuccess;
}
// planes: [3][rows][ld] bf16
void planes(const char *who, const Planes &m) {
    if (m.p) read(who, m.p, m.ld, 3 * m.rows, m.cols, 2);
}
void planes_product(const char *who, const PlanesProduct &p) {
    for (int i = 0; i < 2; ++i) {
        planes(who, p.a[i]);
        planes(who, p.b[i]);
    }
    if (p.epi != EPI_GLU_BWD) return;
    if (p.kplane != p.M * p.kld) wrong("planes of dg, du not one behind the other");
    for (int i = 0; i < 2; ++i) write(who, p.keep[i], p.kld, 3 * p.M, p.N, 2);
}
cudaError_t launch_product_planes(const PlanesProduct &p, cudaStream_t) {
    planes_product("planes kernel", p);
    return cudaSuccess;
}
cudaError_t launch_gradients_planes(const PlanesProduct *p, int n, cudaStream_t) {
    for (int i = 0; i < n; ++i) planes_product("planes kernel, gradients", p[i]);
    return cudaSuccess;
}
cudaError_t launch_split(const Copy *c, int n, cudaStream_t) {
    for (int i = 0; i < n; ++i) write("split", c[i].dst, c[i].dst_ld, 3 * c[i].rows, c[i].cols, 2);
    return cudaSuccess;
}
cudaError_t launch_dgate_planes(const float *, long long, const float *, void *dg, void *du, long long ld, long long M,
                                long long N, cudaStream_t) {
    write("gate gradients in planes", dg, ld, 3 * M, N, 2);
    write("gate gradients in planes", du, ld, 3 * M, N, 2);
    return cudaSuccess;
}
cudaError_t sm_count(int *n) {
    *n = 148;
    return cudaSuccess;
}
cudaError_t status_word(uint32_t **p) {
    static uint32_t w;
    *p = &w;
    return cudaSuccess;
}

void read_wait_cycles() {}

}  // namespace dense
}  // namespace moeq

int main() {
    long long T, H, I;
    int off16, dtype, gu, dx, dw;
    while (std::scanf("%lld %lld %lld %d %d %d %d %d %d", &T, &H, &I, &off16, &dtype, &gu, &dx, &dw, &g_faster) == 9) {
        // made-up addresses, far apart
        auto at = [](int i) { return reinterpret_cast<char *>((uintptr_t)(i + 1) << 40); };
        const long long pad = off16 ? 3 : 0, ldh = (H + 7) / 8 * 8 + pad, ldi = (I + 7) / 8 * 8 + pad;
        moeq_glu_args a{};
        a.n_tokens = (int32_t)T;
        a.hidden = (int32_t)H;
        a.inter = (int32_t)I;
        a.dtype = dtype;
        a.x = at(0);
        a.w[0] = at(1);
        a.w[1] = at(2);
        a.ldx = a.ldw[0] = a.ldw[1] = a.lddx = a.lddw[0] = a.lddw[1] = ldh;
        a.gu = gu ? at(3) : nullptr;
        a.dh = at(4);
        a.lddh = ldi;
        if (dx) a.dx = at(5);
        if (dw) a.dw[0] = at(6), a.dw[1] = at(7);
        g_ws = at(8);
        g_bytes = moeq_glu_workspace(&a, 1);
        a.workspace = at(8);
        a.workspace_bytes = g_bytes;
        g_written.clear();
        g_wrong.clear();
        if (g_bytes < 0 || moeq_glu_backward(&a, nullptr) != MOEQ_OK) wrong("refused");
        std::printf("%s\n", g_wrong.empty() ? "ok" : g_wrong.c_str());
    }
    return 0;
}
