// dense_api.cu -- entry points of the dense operators: argument checks, the
// workspace's layout and the choice of kernels.  See include/moeq.h for what
// each call computes.
#include <algorithm>
#include <mutex>

#include "dense.cuh"

namespace moeq {

cudaError_t launch_quant_i8(const void *x, int dtype, int rows, int cols, long long ldx, int8_t *q, long long ldq,
                            float *scale, cudaStream_t s);

namespace dense {
namespace {

constexpr long long kMaxDim = 1LL << 20;      // hidden, inter, n_out
constexpr int kMaxTokens = 1 << 30;           // and columns of moeq_quant_i8
constexpr long long kMaxLd = 1LL << 36;
constexpr int kMaxI8K = 131071;               // 2^14 K < 2^31

bool known_dtype(int d) { return d == MOEQ_ACT_F32 || d == MOEQ_ACT_BF16; }
int elem_size(int d) { return d == MOEQ_ACT_F32 ? 4 : (d == MOEQ_ACT_BF16 ? 2 : 1); }

// A rows x cols array with row stride ld, in bytes.
struct Span {
    uintptr_t p = 0;
    unsigned long long row = 0, ld = 0, rows = 0;
    Span() {}
    Span(const void *q, long long rows_, long long cols, long long ld_, int es)
        : p((uintptr_t)q), row((unsigned long long)cols * es), ld((unsigned long long)ld_ * es),
          rows((unsigned long long)rows_) {}
    bool empty() const { return !p || !rows || !row; }
    uintptr_t end() const { return p + (rows - 1) * ld + row; }
};
// Whether two arrays share a byte.  Arrays of one row stride whose column
// windows are disjoint (slices of one buffer) do not.
bool overlap(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.end() <= b.p || b.end() <= a.p) return false;
    if (a.ld == b.ld && a.rows > 1 && b.rows > 1) {
        const unsigned long long d = a.p <= b.p ? (b.p - a.p) % a.ld : a.ld - 1 - ((a.p - b.p - 1) % a.ld);
        return d < a.row || d + b.row > a.ld;
    }
    return true;
}
template <int N, int M>
bool any_overlap(const Span (&outs)[N], const Span (&ins)[M]) {
    for (int i = 0; i < N; ++i) {
        for (int j = 0; j < M; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < N; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}
bool matrix_ok(const void *p, long long cols, long long ld, int es) {
    return p && ld >= cols && ld <= kMaxLd && !((uintptr_t)p % es);
}
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

moeq_status done(cudaError_t e) { return e == cudaSuccess ? MOEQ_OK : MOEQ_ERR_CUDA; }

// An operand of the tensor-core kernels that does not start its rows on
// 16-byte addresses is copied into the workspace with padded rows first.
struct Packed {
    size_t bytes = 0;          // 0: used where it lies
    long long ld = 0;
    Packed() {}
    Packed(const void *p, long long rows, long long cols, long long ld_, int es) {
        if (!((uintptr_t)p & 15u) && (rows <= 1 || !((ld_ * es) & 15))) return;
        ld = (cols * es + 127) / 128 * 128 / es;
        bytes = round256((size_t)rows * ld * es);
    }
    static Packed planes(long long rows, long long cols) {
        Packed k;
        k.ld = (cols + 63) / 64 * 64;
        k.bytes = round256((size_t)3 * rows * k.ld * 2);
        return k;
    }
};
// The workspace's parts, in the order they lie in it.  planes: f32 operands are
// multiplied as bf16 planes, which x, w and dgu then hold.
struct Plan {
    bool planes = false, few = false;   // few: dgu is f32 [2][T][dgu_ld] (dense_few.cu)
    Packed x, w[2];
    size_t dgu = 0;            // gradients of the projections, [2][T][dgu_ld] (or [2] planes of them)
    long long dgu_ld = 0;
    size_t total() const { return x.bytes + w[0].bytes + w[1].bytes + dgu; }
};
// The copies of a call's packed operands: add() says where an operand lies for
// the kernels (itself, or the next part of the workspace), run() makes the
// copies in one launch.
struct Packing {
    char *ws;
    int es;
    Copy c[3];
    int n = 0;
    Packing(void *workspace, int es_) : ws((char *)workspace), es(es_) {}
    void add(const Packed &k, const void *&p, long long &ld, long long rows, long long cols) {
        if (!k.bytes) return;
        c[n++] = Copy{p, ld, ws, k.ld, rows, cols};
        p = ws;
        ld = k.ld;
        ws += k.bytes;
    }
    cudaError_t run(cudaStream_t s, bool planes = false) const {
        return !n ? cudaSuccess : (planes ? launch_split(c, n, s) : launch_pack(c, n, es, s));
    }
};
// The same product of operands that lie as planes
PlanesProduct of_planes(const Product &p) {
    PlanesProduct q;
    q.M = p.M;
    q.N = p.N;
    q.K = p.K;
    q.nseg = p.nseg;
    q.nbatch = p.nbatch;
    q.a_t = p.a_t;
    for (int i = 0; i < 2; ++i) {
        if (p.a[i]) q.a[i] = Planes{p.a[i], p.a_t ? p.K : p.M, p.a_t ? p.M : p.K, p.ald};
        if (p.b[i]) q.b[i] = Planes{p.b[i], p.b_t ? p.K : p.N, p.b_t ? p.N : p.K, p.bld[i]};
        q.out[i] = p.out[i];
        q.old[i] = p.old[i];
        q.keep[i] = p.keep[i];
    }
    q.kld = p.kld;
    q.kplane = p.M * p.kld;
    q.dh = static_cast<const float *>(p.dh);
    q.dhld = p.dhld;
    q.epi = p.epi;
    return q;
}
cudaError_t launch_product(const Product &p, cudaStream_t s) {
    if (stream_supported(p)) return launch_product_stream(p, s);
    int sms = 0, bn = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    return skinny_ns(p, sms) < tc_ns(&p, 1, sms, &bn) ? launch_product_skinny(p, s) : launch_product_tc(p, s);
}

cudaError_t launch_gradients(const Product *dx, const Product *dw, cudaStream_t s) {
    // one of them by clusters where that saves more than a launch of its own
    // costs; neither choice depends on the other, so that asking for less changes
    // no bits
    int sms = 0, bn = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    for (const Product **p : {&dx, &dw}) {
        if (!*p || skinny_ns(**p, sms) + 3000 >= tc_ns(*p, 1, sms, &bn)) continue;
        e = launch_product_skinny(**p, s);
        *p = nullptr;
        if (e != cudaSuccess) return e;
    }
    if (!dx && !dw) return cudaSuccess;
    return launch_gradients_tc(dx, dw, s);
}

bool i8_args_ok(const moeq_i8_args *a, int nw) {
    if (!a || (nw != 1 && nw != 2) || a->n_tokens < 0 || a->n_tokens > kMaxTokens || a->n_in < 1 || a->n_in > kMaxI8K || a->n_out < 1 ||
        a->n_out > kMaxDim || !known_dtype(a->out_dtype))
        return false;
    const bool any = a->n_tokens > 0;   // the arrays of no tokens may be NULL
    if (any && (!matrix_ok(a->x, a->n_in, a->ldx, 1) || !a->x_scale || ((uintptr_t)a->x_scale & 3u) ||
                !matrix_ok(a->out, a->n_out, a->ldo, elem_size(a->out_dtype))))
        return false;
    for (int i = 0; i < nw; ++i)
        if (!matrix_ok(a->w[i], a->n_in, a->ldw[i], 1) || !a->w_scale[i] || ((uintptr_t)a->w_scale[i] & 3u))
            return false;
    if (nw == 1 && (a->w[1] || a->ldw[1] || a->w_scale[1])) return false;
    return true;
}
Plan plan_i8(const moeq_i8_args *a, int nw) {
    Plan p;
    if (a->n_tokens <= kStreamRows) return p;
    p.x = Packed(a->x, a->n_tokens, a->n_in, a->ldx, 1);
    for (int i = 0; i < nw; ++i) p.w[i] = Packed(a->w[i], a->n_out, a->n_in, a->ldw[i], 1);
    return p;
}

bool glu_args_ok(const moeq_glu_args *a, bool backward) {
    if (!a || a->n_tokens < 0 || a->n_tokens > kMaxTokens || a->hidden < 1 || a->hidden > kMaxDim || a->inter < 1 || a->inter > kMaxDim ||
        !known_dtype(a->dtype))
        return false;
    const int es = elem_size(a->dtype);
    const bool any = a->n_tokens > 0;
    if (any && !matrix_ok(a->x, a->hidden, a->ldx, es)) return false;
    for (int i = 0; i < 2; ++i)
        if (!matrix_ok(a->w[i], a->hidden, a->ldw[i], es)) return false;
    if ((uintptr_t)a->gu % es) return false;
    if (!backward) return !any || matrix_ok(a->h, a->inter, a->ldh, es);
    if (any && !matrix_ok(a->dh, a->inter, a->lddh, es)) return false;
    if ((a->dw[0] == nullptr) != (a->dw[1] == nullptr)) return false;
    if (!a->dx && !a->dw[0] && any) return false;
    if (a->dx && !matrix_ok(a->dx, a->hidden, a->lddx, es)) return false;
    for (int i = 0; i < 2; ++i)
        if (a->dw[i] && !matrix_ok(a->dw[i], a->hidden, a->lddw[i], es)) return false;
    return true;
}
// The gradients of few tokens by dense_few.cu, or on the tensor cores.  Back-to-back
// calls on weights that come from HBM, us, dense_few.cu against tensor cores:
//   1 token, kept  1024 x 1024 14.3 against 13.3; 4096 x 1024 16.3, 19.6; 4096 x 2048
//     19.7, 32.3; 4096 x 4096 34.9, 45.0; 4096 x 11008 92, 101 (2 tokens the same)
//   1 token, recomputed  1024 x 1024 11.8, 16.2; 4096 x 2048 20.6, 40.5; 4096 x 4096
//     45.0, 60.0; 4096 x 11008 125, 170
//   4 tokens, kept  1024 x 1024 15.2, 13.4; 4096 x 2048 32.9, 32.4; 4096 x 4096 58.2, 45.4
//   4 tokens, recomputed  4096 x 2048 29.2, 40.4; 4096 x 4096 60.7, 60.8; 4096 x 11008 186, 159
// so at any size for 2 tokens, for 4 up to 2^23 (kept) or 2^24.
//   few columns of dx and long sums, 1 token, kept  1024 x 4096 26.3, 22.1 (weights in L2:
//     12.0, 21.5); 512 x 8192 41, 27; 64 x 65536 264, 115; recomputed  512 x 8192 33, 45;
//     256 x 16384 53, 58; 128 x 32768 97, 92; 64 x 65536 185, 157
// so up to inter = 4 hidden, or 64 hidden where the projections were just computed and
// the weights lie in L2; small ones (64 x 8192 36, 22; in L2 16, 22) in f32 all the same.
//   rows off 16 bytes, 1 token  kept 77 x 69 6.8, 8.5; 99 x 130 11.7, 8.6; 255 x 255 13.4,
//     9.5; 576 x 640 20.7, 15.0; recomputed 77 x 69 9.8, 12.6; 255 x 255 16.4, 14.4; 1000 x
//     517 26.0, 17.3; 4096 x 2048 111, 66
// There the elements go one by one and the time alone would end it at 2^13; up to 2^16 it
// costs at most 6 us, which f32 dg and du are taken to be worth.
// Only what both gradients need decides, so that asking for one changes no bits.
bool few_tokens(const moeq_glu_args *a) {
    if (a->dtype != MOEQ_ACT_BF16 || a->n_tokens > kFewRows) return false;
    auto rows16 = [](const void *p, long long ld) { return !((uintptr_t)p & 15u) && !(ld & 7); };
    const bool aligned = rows16(a->x, a->ldx) && rows16(a->w[0], a->ldw[0]) && rows16(a->w[1], a->ldw[1]);
    const long long size = (long long)a->hidden * a->inter;
    if (!aligned) return size <= 1 << 16;
    const bool kept = a->gu != nullptr;
    return size <= 1 << 19 ||
           (a->inter <= (kept ? 4LL : 64LL) * a->hidden && (a->n_tokens <= 2 || size <= (kept ? 1 << 23 : 1 << 24)));
}

Plan plan_glu(const moeq_glu_args *a, bool backward) {
    Plan p;
    if (a->n_tokens == 0) return p;
    p.few = backward && few_tokens(a);
    if (a->dtype == MOEQ_ACT_BF16 && !p.few && (backward || a->n_tokens > kStreamRows)) {
        if (!backward || !a->gu || a->dw[0]) p.x = Packed(a->x, a->n_tokens, a->hidden, a->ldx, 2);
        if (!backward || !a->gu || a->dx)
            for (int i = 0; i < 2; ++i) p.w[i] = Packed(a->w[i], a->inter, a->hidden, a->ldw[i], 2);
    }
    p.planes = a->dtype == MOEQ_ACT_F32;
    if (p.planes) {
        if (!backward || !a->gu || a->dw[0]) p.x = Packed::planes(a->n_tokens, a->hidden);
        if (!backward || !a->gu || a->dx) p.w[0] = p.w[1] = Packed::planes(a->inter, a->hidden);
    }
    if (!backward) return p;
    p.dgu_ld = (a->inter + 63) / 64 * 64;
    p.dgu = round256((size_t)2 * a->n_tokens * p.dgu_ld * (p.planes ? 6 : (p.few ? 4 : 2)));
    return p;
}

bool workspace_ok(const void *ws, long long bytes, const Plan &p) {
    return p.total() == 0 || (ws && !((uintptr_t)ws & 255u) && bytes >= 0 && (size_t)bytes >= p.total());
}

moeq_status run_i8(const moeq_i8_args *a, int nw, cudaStream_t s) {
    if (!i8_args_ok(a, nw)) return MOEQ_ERR_INVALID_ARGUMENT;
    if (a->n_tokens == 0) return MOEQ_OK;
    const Plan plan = plan_i8(a, nw);
    if (!workspace_ok(a->workspace, a->workspace_bytes, plan)) return MOEQ_ERR_INVALID_ARGUMENT;
    const long long T = a->n_tokens, N = a->n_out, K = a->n_in;
    const Span outs[2] = {Span(a->out, T, N, a->ldo, elem_size(a->out_dtype)),
                          Span(a->workspace, 1, (long long)plan.total(), (long long)plan.total(), 1)};
    const Span ins[6] = {Span(a->x, T, K, a->ldx, 1),         Span(a->w[0], N, K, a->ldw[0], 1),
                         Span(a->w[1], N, K, a->ldw[1], 1),   Span(a->x_scale, 1, T, T, 4),
                         Span(a->w_scale[0], 1, N, N, 4),     Span(a->w_scale[1], 1, N, N, 4)};
    if (any_overlap(outs, ins)) return MOEQ_ERR_INVALID_ARGUMENT;
    Product p;
    p.M = T;
    p.N = N;
    p.K = K;
    p.a[0] = a->x;
    p.ald = a->ldx;
    p.a_scale = a->x_scale;
    for (int i = 0; i < nw; ++i) {
        p.b[i] = a->w[i];
        p.bld[i] = a->ldw[i];
        p.b_scale[i] = a->w_scale[i];
    }
    p.out[0] = a->out;
    p.old[0] = a->ldo;
    p.in_dtype = kI8;
    p.out_dtype = a->out_dtype;
    p.epi = nw == 2 ? EPI_GLU : EPI_STORE;
    Packing pk(a->workspace, 1);
    pk.add(plan.x, p.a[0], p.ald, T, K);
    for (int i = 0; i < nw; ++i) pk.add(plan.w[i], p.b[i], p.bld[i], N, K);
    const cudaError_t e = pk.run(s);
    return done(e == cudaSuccess ? launch_product(p, s) : e);
}

}  // namespace
}  // namespace dense
}  // namespace moeq

using namespace moeq;
using namespace moeq::dense;

extern "C" moeq_status moeq_quant_i8(const void *x, int32_t dtype, int32_t n_rows, int32_t n_cols, int64_t ldx,
                                     int8_t *q, int64_t ldq, float *scale, void *stream) {
    if (!known_dtype(dtype) || n_rows < 0 || n_cols < 1 || n_cols > kMaxTokens) return MOEQ_ERR_INVALID_ARGUMENT;
    if (n_rows == 0) return MOEQ_OK;
    const int es = elem_size(dtype);
    if (!matrix_ok(x, n_cols, ldx, es) || !matrix_ok(q, n_cols, ldq, 1) || !scale || ((uintptr_t)scale & 3u))
        return MOEQ_ERR_INVALID_ARGUMENT;
    const Span outs[2] = {Span(q, n_rows, n_cols, ldq, 1), Span(scale, 1, n_rows, n_rows, 4)};
    const Span ins[1] = {Span(x, n_rows, n_cols, ldx, es)};
    if (any_overlap(outs, ins)) return MOEQ_ERR_INVALID_ARGUMENT;
    return done(launch_quant_i8(x, dtype, n_rows, n_cols, ldx, q, ldq, scale, (cudaStream_t)stream));
}

extern "C" moeq_status moeq_matmul_i8(const moeq_i8_args *a, void *stream) {
    return run_i8(a, 1, (cudaStream_t)stream);
}
extern "C" moeq_status moeq_glu_i8(const moeq_i8_args *a, void *stream) { return run_i8(a, 2, (cudaStream_t)stream); }
extern "C" int64_t moeq_i8_workspace(const moeq_i8_args *a, int32_t n_w) {
    return i8_args_ok(a, n_w) ? (int64_t)plan_i8(a, n_w).total() : -1;
}

extern "C" int64_t moeq_glu_workspace(const moeq_glu_args *a, int32_t backward) {
    if ((backward != 0 && backward != 1) || !glu_args_ok(a, backward == 1)) return -1;
    return (int64_t)plan_glu(a, backward == 1).total();
}

extern "C" moeq_status moeq_glu(const moeq_glu_args *a, void *stream) {
    if (!glu_args_ok(a, false)) return MOEQ_ERR_INVALID_ARGUMENT;
    if (a->n_tokens == 0) return MOEQ_OK;
    const Plan plan = plan_glu(a, false);
    if (!workspace_ok(a->workspace, a->workspace_bytes, plan)) return MOEQ_ERR_INVALID_ARGUMENT;
    const long long T = a->n_tokens, H = a->hidden, I = a->inter;
    const int es = elem_size(a->dtype);
    const Span outs[3] = {Span(a->h, T, I, a->ldh, es), Span(a->gu, 2 * T, I, I, es),
                          Span(a->workspace, 1, (long long)plan.total(), (long long)plan.total(), 1)};
    const Span ins[3] = {Span(a->x, T, H, a->ldx, es), Span(a->w[0], I, H, a->ldw[0], es),
                         Span(a->w[1], I, H, a->ldw[1], es)};
    if (any_overlap(outs, ins)) return MOEQ_ERR_INVALID_ARGUMENT;
    Product p;
    p.M = T;
    p.N = I;
    p.K = H;
    p.a[0] = a->x;
    p.ald = a->ldx;
    for (int i = 0; i < 2; ++i) {
        p.b[i] = a->w[i];
        p.bld[i] = a->ldw[i];
        if (a->gu) p.keep[i] = (char *)a->gu + (size_t)i * T * I * es;
    }
    p.kld = I;
    p.out[0] = a->h;
    p.old[0] = a->ldh;
    p.in_dtype = p.out_dtype = a->dtype;
    p.epi = EPI_GLU;
    const cudaStream_t s = (cudaStream_t)stream;
    Packing pk(a->workspace, es);
    pk.add(plan.x, p.a[0], p.ald, T, H);
    for (int i = 0; i < 2; ++i) pk.add(plan.w[i], p.b[i], p.bld[i], I, H);
    const cudaError_t e = pk.run(s, plan.planes);
    if (e != cudaSuccess) return MOEQ_ERR_CUDA;
    if (plan.planes) {
        return done(launch_product_planes(of_planes(p), s));
    }
    return done(launch_product(p, s));
}

extern "C" moeq_status moeq_glu_backward(const moeq_glu_args *a, void *stream) {
    if (!glu_args_ok(a, true)) return MOEQ_ERR_INVALID_ARGUMENT;
    const cudaStream_t s = (cudaStream_t)stream;
    const long long T = a->n_tokens, H = a->hidden, I = a->inter;
    const int es = elem_size(a->dtype);
    const Plan plan = plan_glu(a, true);
    if (!workspace_ok(a->workspace, a->workspace_bytes, plan)) return MOEQ_ERR_INVALID_ARGUMENT;
    const Span outs[4] = {Span(a->dx, T, H, a->lddx, es), Span(a->dw[0], I, H, a->lddw[0], es),
                          Span(a->dw[1], I, H, a->lddw[1], es),
                          Span(a->workspace, 1, (long long)plan.total(), (long long)plan.total(), 1)};
    const Span ins[5] = {Span(a->x, T, H, a->ldx, es), Span(a->w[0], I, H, a->ldw[0], es),
                         Span(a->w[1], I, H, a->ldw[1], es), Span(a->gu, 2 * T, I, I, es),
                         Span(a->dh, T, I, a->lddh, es)};
    if (any_overlap(outs, ins)) return MOEQ_ERR_INVALID_ARGUMENT;
    if (T == 0) {
        for (int i = 0; i < 2 && a->dw[i]; ++i) {
            const cudaError_t e = cudaMemset2DAsync(a->dw[i], (size_t)a->lddw[i] * es, 0, (size_t)H * es, (size_t)I, s);
            if (e != cudaSuccess) return MOEQ_ERR_CUDA;
        }
        return MOEQ_OK;
    }
    const void *x = a->x, *w[2] = {a->w[0], a->w[1]};
    long long ldx = a->ldx, ldw[2] = {a->ldw[0], a->ldw[1]};
    Packing pk(a->workspace, es);
    pk.add(plan.x, x, ldx, T, H);
    for (int i = 0; i < 2; ++i) pk.add(plan.w[i], w[i], ldw[i], I, H);
    cudaError_t e = pk.run(s, plan.planes);
    if (e != cudaSuccess) return MOEQ_ERR_CUDA;
    char *dg = pk.ws, *du = dg + (size_t)T * plan.dgu_ld * (plan.planes ? 6 : (plan.few ? 4 : es));
    if (a->gu && plan.few) {
        e = launch_dgate_f32(a->dh, a->lddh, a->gu, (float *)dg, (float *)du, plan.dgu_ld, (int)T, (int)I, s);
    } else if (a->gu && plan.planes) {
        e = launch_dgate_planes(static_cast<const float *>(a->dh), a->lddh, static_cast<const float *>(a->gu), dg, du,
                                plan.dgu_ld, T, I, s);
    } else if (a->gu) {
        e = launch_glu_dgate(a->dh, a->lddh, a->gu, dg, du, plan.dgu_ld, T, I, s);
    } else {
        Product p;
        p.M = T;
        p.N = I;
        p.K = H;
        p.a[0] = x;
        p.ald = ldx;
        for (int i = 0; i < 2; ++i) {
            p.b[i] = w[i];
            p.bld[i] = ldw[i];
        }
        p.keep[0] = dg;
        p.keep[1] = du;
        p.keep_f32 = plan.few;   // the plan has sized them; the kernel follows
        p.kld = plan.dgu_ld;
        p.dh = a->dh;
        p.dhld = a->lddh;
        p.in_dtype = p.out_dtype = a->dtype;
        p.epi = EPI_GLU_BWD;
        e = plan.planes ? launch_product_planes(of_planes(p), s) : launch_product(p, s);
    }
    if (e != cudaSuccess) return MOEQ_ERR_CUDA;
    Product px, pw;
    // dx = dg W_gate + du W_up: two segments along the reduction
    px.M = T;
    px.N = H;
    px.K = I;
    px.nseg = 2;
    px.b_t = true;
    px.out[0] = a->dx;
    px.old[0] = a->lddx;
    // dW_i = d_i^T x: two products of one B
    pw.M = I;
    pw.N = H;
    pw.K = T;
    pw.nbatch = 2;
    pw.a_t = pw.b_t = true;
    pw.b[0] = x;
    pw.bld[0] = ldx;
    px.a[0] = pw.a[0] = dg;
    px.a[1] = pw.a[1] = du;
    px.ald = pw.ald = plan.dgu_ld;
    px.in_dtype = px.out_dtype = pw.in_dtype = pw.out_dtype = a->dtype;
    for (int i = 0; i < 2; ++i) {
        px.b[i] = w[i];
        px.bld[i] = ldw[i];
        pw.out[i] = a->dw[i];
        pw.old[i] = a->lddw[i];
    }
    if (plan.few)
        return done(launch_few_gradients(a->dx ? &px : nullptr, a->dw[0] ? &pw : nullptr, (const float *)dg,
                                         (const float *)du, plan.dgu_ld, s));
    if (plan.planes) {
        PlanesProduct both[2];
        int n = 0;
        if (a->dx) both[n++] = of_planes(px);
        if (a->dw[0]) both[n++] = of_planes(pw);
        return done(launch_gradients_planes(both, n, s));
    }
    return done(launch_gradients(a->dx ? &px : nullptr, a->dw[0] ? &pw : nullptr, s));
}

extern "C" moeq_status moeq_dense_status(int32_t clear) {
    uint32_t *at = nullptr, w = 0;
    if (status_word(&at) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return MOEQ_ERR_CUDA;
    if (cudaMemcpy(&w, at, sizeof(w), cudaMemcpyDeviceToHost) != cudaSuccess) return MOEQ_ERR_CUDA;
    if (clear) read_wait_cycles();
    if (clear && w && (cudaMemset(at, 0, sizeof(w)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)) return MOEQ_ERR_CUDA;
    return w ? MOEQ_ERR_TIMEOUT : MOEQ_OK;
}
