"""The dense operators at the ends of their ranges: the largest numbers of rows, tokens, hidden and inter, the smallest
values, tensors that are not what their memory holds."""
import pytest

from _gpu_util import torch_mod
from test_gpu_dense import (EPS, MISC, backward_refs, check, int_sum, mat, moeq, projections,  # noqa: F401  (moeq: the
                            sigmoid)                                                           # fixture)

pytestmark = pytest.mark.gpu


def test_quant_i8_of_the_most_rows(moeq):
    """2^31 - 1 rows of one element: each is its row's largest, so q = 127 sign(x), scale = |x| / 127."""
    torch = torch_mod()
    n, piece = 2**31 - 1, 1 << 28
    x = torch.empty((n, 1), dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.zeros((n, 1), dtype=torch.int8, device="cuda")
    scale = torch.full((n,), -1.0, device="cuda")
    moeq.quant_i8(x, q=q, scale=scale)
    for i in range(0, n, piece):
        v = x[i:i + piece, 0].float()
        assert torch.equal(q[i:i + piece, 0], (127 * v.sign()).to(torch.int8))
        # f64 quotients of f32 values round to the f32 quotient; a / 127 in f32 torch takes as a product with 1 / 127
        assert torch.equal(scale[i:i + piece], (v.double().abs() / 127).float())


@pytest.mark.parametrize("T", [3, 16, 40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_silu_falls_off_gradually(moeq, dtype, T):
    """Gates from -80 to -104, where e^-g leaves f32 (at -88.7) and silu(g) the normal range (at -92), through every
    kernel of the block (few tokens, cluster, tiles, f32), forward and backward.  With z = e^g the values are g z and
    z (1 + g) to within z^2.  z is off by |g| 2^-23 + 2 ulp < 1.3e-5 and in the subnormal range by a few of its steps
    of 2^-149; the divide and the products add 2 + 3 ulp; then the result's own rounding, whose steps end at 2^-133 for
    bf16, as those of the gate gradients do in both types (f32: their bf16 parts)."""
    torch = torch_mod()
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    half, step = {"bf16": (2.0 ** -8, 2.0 ** -133), "f32": (2.0 ** -24, 2.0 ** -149)}[dtype]
    H, I = 64, 48
    gates = -80 - 0.5 * torch.arange(I, device="cuda", dtype=torch.float32)      # exact in bf16
    x, wg, wu = (torch.zeros(s, device="cuda", dtype=dt) for s in ((T, H), (I, H), (I, H)))
    x[:, 0], x[:, 1] = 1, 1
    wg[:, 0], wu[:, 1] = gates.to(dt), 1
    h, gu = moeq.glu(x, wg, wu, save=True)
    g = gates.double()
    s = torch.exp(g) / (1 + torch.exp(g))
    assert torch.equal(gu[0].double(), g.expand(T, I)) and (gu[1] == 1).all()

    def close(got, want, what, step=step):
        rel = 1.3e-5 + 16 * 2.0 ** -23
        bound = want.abs() * (rel + half) + 8 * g.abs() * 2.0 ** -149 + step
        bad = (got.double() - want).abs() > bound
        assert not bad.any(), f"{what}: {got[bad][:4].tolist()}, not {want.expand_as(got)[bad][:4].tolist()}"
    close(h, g * s, "h")
    # rows of dh with one token each: dW_up = silu(g) at x's 1, dW_gate = s (1 + g (1 - s)) there
    dh = torch.zeros((T, I), device="cuda", dtype=dt)
    dh[T // 2] = 1
    for kept in (gu, None):
        _, dwg, dwu = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dx=False)
        # dg and du may be rounded to the type once more on the way
        close(dwg[:, 0], s * (1 + g * (1 - s)), "dwg", 2.0 ** -132)
        close(dwu[:, 1], g * s, "dwu", 2.0 ** -132)


def test_tensors_with_the_negative_bit_are_refused(moeq):
    """Their memory holds the values with the sign turned."""
    torch = torch_mod()
    x, w = mat(4, 64, "bf16", 1), mat(32, 64, "bf16", 2)
    dh = mat(4, 32, "bf16", 3)
    n = torch._neg_view
    q, s = moeq.quant_i8(w)
    for call in (lambda: moeq.quant_i8(n(x)), lambda: moeq.glu(n(x), w, w), lambda: moeq.glu(x, w, n(w)),
                 lambda: moeq.glu(x, w, w, out=n(dh)), lambda: moeq.glu_backward(n(dh), x, w, w),
                 lambda: moeq.matmul_i8(q, n(s), q, s), lambda: moeq.matmul_i8(q, s, q, n(s))):
        with pytest.raises(moeq.MoeqError):
            call()
    assert torch.equal(moeq.glu(n(x).resolve_neg(), w, w), moeq.glu(-x, w, w))


MOST = 1 << 20     # hidden and inter


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", [(1, MOST, 3), (4, MOST, 2), (16, MOST, 5), (40, MOST, 3), (300, MOST - 1, 2), (1, 5, MOST),
                                   (4, 8, MOST), (16, 3, MOST), (40, 8, MOST - 3), (300, 2, MOST), ((1 << 24) + 3, 8, 8),
                                   ((1 << 22) + 1, 3, 17)])
def test_the_largest_sizes(moeq, T, H, I, dtype):
    """Element by element within bounds that grow with the sums' length, and in the norm within what the errors leave
    of them together: bf16 rounds a result and a gate gradient by at most 2^-8 / sqrt(3) each; a tensor-core step of 16
    products cuts off up to 2^-24 of the running value on average, in the projections and in the gradients' sums.  f32:
    1e-6 for sums of 4096 (test_gpu_dense_f32.py), the joins of pieces of 128 by 2^-25 each and independently, the five
    small products below 2^-8 of that cut-off; three sums behind one another."""
    torch = torch_mod()
    x, dh = mat(T, H, dtype, 1), mat(T, I, dtype, 2, scale=0.1)
    wg, wu = mat(I, H, dtype, 3, scale=1.3 / H ** 0.5), mat(I, H, dtype, 4, scale=1.3 / H ** 0.5)
    g, u, eg, eu = projections(x, wg, wu)
    h, gu = moeq.glu(x, wg, wu, save=True)
    ref = g * sigmoid(g) * u
    hb = 1.1 * eg * (u.abs() + eu) + (g * sigmoid(g)).abs() * eu
    check(h, ref, hb + (ref.abs() + hb) * (MISC + EPS[dtype] * 1.001), "h")
    del ref, hb, h
    zero = torch.zeros_like(g)
    L = max(T, H, 2 * I)
    near = {"bf16": 3.2e-3 + 2 * L / 16 * 2.0 ** -24,
            "f32": 3 * (1e-6 + (L / 128) ** 0.5 * 2.0 ** -25 + 5 * L / 16 * 2.0 ** -32)}[dtype]
    for kept, pr in ((gu, (gu[0].double(), gu[1].double(), zero, zero)), (None, (g, u, eg, eu))):
        got = moeq.glu_backward(dh, x, wg, wu, gu=kept)
        for o, (want, bound), what in zip(got, backward_refs(dh, x, wg, wu, *pr, dtype), ("dx", "dwg", "dwu")):
            check(o, want, bound, what + (" (kept)" if kept is not None else ""))
            e = ((o.double() - want).norm() / want.norm()).item()
            assert e <= near, (what, e)


@pytest.mark.parametrize("T,K,N", [(1, 131071, 5), (16, 131071, 3), (40, 131071, 2), (300, 131071, 2), (1, 5, MOST), (16, 3, MOST),
                                   (40, 17, MOST), (300, 16, MOST - 1), ((1 << 24) + 3, 16, 5)])
def test_the_largest_int8_sizes(moeq, T, K, N):
    torch = torch_mod()
    x, w = mat(T, K, "i8", 1), mat(N, K, "i8", 2)
    sx, sw = (torch.rand(n, device="cuda") * 1e-2 + 1e-4 for n in (T, N))
    out = moeq.matmul_i8(x, sx, w, sw, dtype="f32")
    step = max(1, (1 << 26) // N)
    for t in range(0, T, step):
        ref = int_sum(x[t:t + step], w) * sx[t:t + step].double()[:, None] * sw.double()
        check(out[t:t + step], ref, ref.abs() * 3.01 * 2.0 ** -24, "matmul_i8")


def test_no_tokens_and_rows_far_apart(moeq):
    """dW of no tokens is zero, with rows 2 GB and more apart too; what lies between them stays."""
    torch = torch_mod()
    ld = (1 << 30) + 64
    buf = torch.full((2 * ld + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = buf.as_strided((3, 64), (ld, 1)), buf.as_strided((3, 64), (ld, 1), 64)
    w = mat(3, 64, "bf16", 1)
    moeq.glu_backward(mat(0, 3, "bf16", 2), mat(0, 64, "bf16", 3), w, w, dw_gate=dwg, dw_up=dwu, need_dx=False)
    assert not dwg.any() and not dwu.any()
    assert all(bool((buf[i * ld + 128:(i + 1) * ld] == 7).all()) for i in range(2))
