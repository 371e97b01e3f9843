"""The dense operators (row quantisation, int8 products, the gated block and
its backward pass) against their definitions in 64 bits.

Error bounds.  A sum of K products accumulated in f32 is off by at most
gamma(K) sum_k |a_k b_k|: the kernels add at most 256 products one by one
(the first term, one ulp of the running sum each, no matter whether an adder
rounds or truncates), or 8 at least per tensor-core step, and then the partial
sums.  A rounding to bf16 is off by at most 2^-8 of the value, one to f32 by
2^-24.  exp and the divide add a few 2^-23.  The bounds below carry these
through the formulas element by element; nothing in them is fitted."""
import numpy as np
import pytest

from _gpu_util import torch_mod

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
MISC = 16 * 2.0 ** -23      # expf (2 ulp), divides, a handful of f32 products


def gamma(K):
    return (min(K, 256) + K / 8 + 32) * 2.0 ** -23


@pytest.fixture(scope="module")
def moeq():
    from bit_quantized_moe_routed_b200 import moeq as m
    yield m
    assert m.dense_status() == m.OK


def dt_of(name):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}[name]


def mat(rows, cols, dtype, seed, scale=1.0, pad=0, off=0):
    """A random matrix inside a wider buffer: `off` columns before, `pad` after each row."""
    torch = torch_mod()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if dtype == "i8":
        buf = torch.randint(-127, 128, (rows, cols + pad + off), generator=g, device="cuda", dtype=torch.int8)
    else:
        buf = (torch.randn((rows, cols + pad + off), generator=g, device="cuda") * scale).to(dt_of(dtype))
    return buf[:, off:off + cols]


def framed(rows, cols, dtype, pad=0, off=0):
    """(output view, check that nothing around it was written)"""
    torch = torch_mod()
    mark = 77 if dtype == "i8" else 77.0
    buf = torch.full((rows + 2, cols + pad + off), mark, dtype=dt_of(dtype), device="cuda")

    def untouched():
        frame = buf.clone()
        frame[1:1 + rows, off:off + cols] = mark
        return bool((frame == mark).all())
    return buf[1:1 + rows, off:off + cols], untouched


def sigmoid(g):
    torch = torch_mod()
    return 1 / (1 + torch.exp(-g))


def check(got, ref, bound, what):
    torch = torch_mod()
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - ref).abs() - bound
    assert bad.max().item() <= 0, (f"{what}: {int((bad > 0).sum())} of {bad.numel()} values outside their bound, worst "
                                   f"{((got - ref).abs() / (bound + 1e-300)).max().item():.2f} times it")


# ---------------------------------------------------------------- quantiser
def quant_ref(x):
    v = x.double().cpu().numpy()
    a = np.abs(v).max(axis=1, keepdims=True)
    # 127 v is exact in f64 (31 bits); its f64 quotient by a 24-bit value lies
    # on the true quotient's side of a half (see quant_i8.cu)
    q = np.rint(v * 127.0 / np.where(a > 0, a, 1.0))
    return q.astype(np.int8), (a[:, 0].astype(np.float32) / np.float32(127)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,pad,off", [(1, 1, 0, 0), (1, 4096, 0, 0), (3, 7, 0, 0), (9, 64, 8, 0), (8, 1024, 0, 0),
                                         (5, 1025, 0, 0), (33, 1111, 5, 3), (7, 8191, 1, 0), (2, 9000, 0, 0),
                                         (2, 70000, 0, 0), (300, 256, 0, 8), (1000, 2048, 0, 0)])
def test_quant_i8(moeq, dtype, M, K, pad, off):
    torch = torch_mod()
    x = mat(M, K, dtype, 1, pad=pad, off=off)
    x[0] *= 3e-3
    if M > 2:
        x[1] = 0
    q, untouched = framed(M, K, "i8", pad, off)
    sc = torch.full((M,), 5.0, device="cuda")
    moeq.quant_i8(x, q=q, scale=sc)
    rq, rs = quant_ref(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(sc.cpu().numpy(), rs)
    assert untouched()


def test_quant_i8_halves_go_to_the_even_integer(moeq):
    torch = torch_mod()
    # x / a = (2 j + 1) / 254 for every j: all exact halves, for a = 127 and a = 2^-7 * 127
    for s in (1.0, 2.0 ** -7, 2.0 ** 90):
        half = torch.arange(-126, 127, device="cuda", dtype=torch.float32) + 0.5
        x = (torch.cat([half, torch.tensor([127.0], device="cuda")]) * s)[None]
        q, sc = moeq.quant_i8(x)
        want = np.append(np.rint(np.arange(-126, 127) + 0.5), 127).astype(np.int8)
        assert np.array_equal(q[0].cpu().numpy(), want)
        # the neighbours of the halves go to their side
        up = torch.nextafter(x, torch.full_like(x, float("inf")))
        up[0, -1] = x[0, -1]
        q, _ = moeq.quant_i8(up)
        assert np.array_equal(q[0, :-1].cpu().numpy(), np.arange(-125, 128))
        down = torch.nextafter(x, torch.full_like(x, -float("inf")))
        down[0, -1] = x[0, -1]
        q, _ = moeq.quant_i8(down)
        assert np.array_equal(q[0, :-1].cpu().numpy(), np.arange(-126, 127))


def test_quant_i8_extreme_rows(moeq):
    torch = torch_mod()
    x = mat(8, 512, "f32", 2)
    x[0] *= 1e38 / x[0].abs().max()
    x[1] *= 3e-39           # subnormal values
    x[2] = 0
    x[2, 5] = 2.0 ** -149   # the smallest
    x[3, 100] = float("nan")
    x[4, 511] = float("inf")
    x[5, 0] = -float("inf")
    x[6] = -0.0
    q, sc = moeq.quant_i8(x)
    ok = [0, 1, 2, 6, 7]
    rq, rs = quant_ref(x[ok])
    assert np.array_equal(q[ok].cpu().numpy(), rq) and np.array_equal(sc[ok].cpu().numpy(), rs)
    assert torch.isnan(sc[3:6]).all() and (q[3:6] == 0).all()
    # such rows make their products NaN, and only theirs
    w = mat(16, 512, "i8", 3)
    out = moeq.matmul_i8(q, sc, w, torch.ones(16, device="cuda"), dtype="f32")
    assert torch.isnan(out[3:6]).all() and torch.isfinite(out[[1, 2, 6, 7]]).all()
    # row 0's scale is 1e38 / 127 = 7.9e35: a sum of integers beyond 3.4e38 / 7.9e35 = 433 overflows f32
    exact = (q[0].double() @ w.double().t()) * sc[0].double()
    over = exact.abs() > 3.4028236e38
    assert over.any() and torch.equal(torch.isinf(out[0]), over) and (torch.sign(out[0]) == torch.sign(exact)).all()


# ------------------------------------------------------------- int8 products
def int_sum(x, w):
    return x.double() @ w.double().t()     # exact: every partial sum is below 2^53


SIZES = [  # T, K, N, pad, off
    (1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (1, 4096, 2048, 0, 0), (2, 100, 33, 0, 0), (3, 131, 70, 1, 1),
    (4, 2048, 130, 16, 0), (7, 999, 517, 0, 0), (8, 4096, 4096, 0, 0), (8, 256, 129, 16, 16), (9, 512, 256, 0, 0),
    (16, 1024, 384, 0, 0), (17, 272, 200, 0, 0), (31, 640, 1000, 0, 0), (64, 4096, 2048, 0, 0), (65, 384, 300, 32, 0),
    (128, 2048, 512, 0, 0), (129, 640, 257, 0, 0), (200, 130, 64, 3, 0), (256, 128, 256, 0, 0), (257, 1000, 517, 0, 0),
    (511, 777, 640, 0, 0), (777, 1111, 1003, 5, 0), (1024, 1024, 1024, 0, 0), (1500, 64, 72, 0, 0), (2048, 33, 128, 0, 0),
    (2048, 4096, 2048, 0, 0), (4097, 70, 66, 0, 0), (8192, 64, 200, 8, 0), (6000, 200, 16, 0, 0),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,pad,off", SIZES)
def test_int8_products(moeq, T, K, N, pad, off, out):
    torch = torch_mod()
    x, w, w2 = mat(T, K, "i8", 4, pad=pad, off=off), mat(N, K, "i8", 5, pad=pad, off=off), mat(N, K, "i8", 6, pad=pad)
    sx, sw, sw2 = (mat(1, n, "f32", 7 + i).abs()[0] * 1e-2 / K ** 0.25 + 1e-4 for i, n in enumerate((T, N, N)))
    sx, sw, sw2 = sx.contiguous(), sw.contiguous(), sw2.contiguous()
    o, untouched = framed(T, N, out, pad, off)
    moeq.matmul_i8(x, sx, w, sw, out=o)
    acc = int_sum(x, w)
    ref = acc * sx.double()[:, None] * sw.double()
    # one rounding of the integer, two products, then the output's own (nothing
    # but these: the sum is exact)
    scaled = 3.01 * 2.0 ** -24
    check(o, ref, ref.abs() * (scaled + (0 if out == "f32" else EPS["bf16"] * 1.001)), "matmul_i8")
    assert untouched()
    o, untouched = framed(T, N, out, pad, off)
    moeq.glu_i8(x, sx, w, sw, w2, sw2, out=o)
    u = int_sum(x, w2) * sx.double()[:, None] * sw2.double()
    h = ref * sigmoid(ref) * u
    # |d silu| <= 1.1 |d g|
    bound = 1.1 * ref.abs() * scaled * u.abs() + h.abs() * (scaled + MISC + EPS[out] * 1.001)
    check(o, h, bound, "glu_i8")
    assert untouched()


def test_int8_largest_values_do_not_overflow(moeq):
    torch = torch_mod()
    K = 131071
    x = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(5, device="cuda")
    for T in (1, 3):
        out = moeq.matmul_i8(x[:T], one[:T].clone(), w, one, dtype="f32")
        want = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K] + [128.0 * 128 * K] * 3, dtype=torch.float64)
        assert torch.equal(out.cpu(), want.float().expand(T, 5))
    # and through the tensor cores' row counts
    xl = torch.full((300, K), -128, dtype=torch.int8, device="cuda")
    out = moeq.matmul_i8(xl, torch.ones(300, device="cuda"), w, one, dtype="f32")
    assert torch.equal(out.cpu(), want.float().expand(300, 5))


# -------------------------------------------------------------- gated block
def projections(x, wg, wu):
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    gm = gamma(x.shape[1])
    return g, u, gm * (x.abs() @ wg.abs().t()), gm * (x.abs() @ wu.abs().t())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,pad,off", SIZES)
def test_glu(moeq, T, H, I, pad, off, dtype):
    torch = torch_mod()
    x = mat(T, H, dtype, 11, pad=pad, off=off)
    both = mat(2 * I, H, dtype, 12, scale=1.3 / H ** 0.5, pad=pad, off=off)     # both projections in one buffer
    wg, wu = both[:I], both[I:]
    g, u, eg, eu = projections(x, wg, wu)
    h = g * sigmoid(g) * u
    hb = 1.1 * eg * (u.abs() + eu) + (g * sigmoid(g)).abs() * eu
    hb = hb + (h.abs() + hb) * (MISC + EPS[dtype] * 1.001)
    o, untouched = framed(T, I, dtype, pad, off)
    r = moeq.glu(x, wg, wu, out=o)
    assert r is o
    check(o, h, hb, "h")
    assert untouched()
    # the kept projections do not change h
    h2, gu = moeq.glu(x, wg, wu, save=True)
    check(h2, h, hb, "h (with gu)")
    for got, ref, e, what in ((gu[0], g, eg, "g"), (gu[1], u, eu, "u")):
        check(got, ref, e + (ref.abs() + e) * EPS[dtype] * 1.001, what)


def backward_refs(dh, x, wg, wu, g, u, eg, eu, dtype, inner=None):
    """Gradients in f64 and their bounds, from projections known to within eg, eu.
    inner: the type that dg and du are held in, dtype without it."""
    inner = EPS[inner or dtype]
    s = sigmoid(g)
    ds = s * (1 + g * (1 - s))               # |ds| <= 1.1, |d ds / dg| <= 0.5
    dh, x, wg, wu = dh.double(), x.double(), wg.double(), wu.double()
    dg, du = dh * u * ds, dh * g * s
    bg = dh.abs() * (1.1 * eu + 0.5 * eg * (u.abs() + eu))
    bu = dh.abs() * 1.1 * eg
    # evaluation in f32: ds is a sum of terms up to s (1 + |g|)
    bg = bg + MISC * (dh * u).abs() * s * (1 + g.abs())
    bu = bu + MISC * du.abs()
    bg, bu = bg + (dg.abs() + bg) * inner * 1.001, bu + (du.abs() + bu) * inner * 1.001
    gx, gt = gamma(2 * g.shape[1]), gamma(x.shape[0])
    out = []
    for ref, e, sm, gm in (
            (dg @ wg + du @ wu, bg @ wg.abs() + bu @ wu.abs(), (dg.abs() + bg) @ wg.abs() + (du.abs() + bu) @ wu.abs(), gx),
            (dg.t() @ x, bg.t() @ x.abs(), (dg.abs() + bg).t() @ x.abs(), gt),
            (du.t() @ x, bu.t() @ x.abs(), (du.abs() + bu).t() @ x.abs(), gt)):
        e = e + gm * sm
        out.append((ref, e + (ref.abs() + e) * EPS[dtype] * 1.001))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,pad,off", SIZES)
def test_glu_backward(moeq, T, H, I, pad, off, dtype):
    torch = torch_mod()
    x = mat(T, H, dtype, 21, pad=pad, off=off)
    wg, wu = mat(I, H, dtype, 22, scale=1.3 / H ** 0.5, pad=pad), mat(I, H, dtype, 23, scale=1.3 / H ** 0.5, off=off)
    dh = mat(T, I, dtype, 24, scale=0.1, pad=pad, off=off)
    g, u, eg, eu = projections(x, wg, wu)
    gu = torch.stack([g, u]).to(dt_of(dtype))
    zero = torch.zeros_like(g)
    for kept, pr in ((gu, (gu[0].double(), gu[1].double(), zero, zero)), (None, (g, u, eg, eu))):
        outs = [framed(T, H, dtype, pad, off), framed(I, H, dtype, pad, off), framed(I, H, dtype, pad)]
        got = moeq.glu_backward(dh, x, wg, wu, gu=kept, dx=outs[0][0], dw_gate=outs[1][0], dw_up=outs[2][0])
        for o, (ref, bound), what, fr in zip(got, backward_refs(dh, x, wg, wu, *pr, dtype), ("dx", "dwg", "dwu"), outs):
            check(o, ref, bound, what + (" (kept)" if kept is not None else ""))
            assert fr[1](), what
        # a gradient that is left out does not change the others
        dx, n1, n2 = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dw=False)
        assert n1 is None and n2 is None and torch.equal(dx, got[0])
        n0, d1, d2 = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dx=False)
        assert n0 is None and torch.equal(d1, got[1]) and torch.equal(d2, got[2])


FEW = [  # T, H, I, pad, off
    (1, 1, 1, 0, 0), (1, 200, 69, 3, 0), (2, 64, 138, 0, 0), (3, 131, 70, 1, 1), (4, 1000, 513, 0, 0), (3, 40, 1030, 8, 8),
    (4, 99, 317, 0, 3), (2, 576, 640, 0, 0), (4, 31, 9, 0, 0), (3, 15, 2100, 2, 0), (4, 64, 8000, 0, 0),
]


@pytest.mark.parametrize("T,H,I,pad,off", FEW)
def test_glu_backward_of_few_tokens_rounds_once(moeq, T, H, I, pad, off):
    """Up to 4 bf16 tokens, small weights: dg and du stay f32, so that the only rounding to
    bf16 is the result's; empty rows of dh stay empty."""
    torch = torch_mod()
    x = mat(T, H, "bf16", 31, pad=pad, off=off)
    wg, wu = mat(I, H, "bf16", 32, scale=1.3 / H ** 0.5, pad=pad), mat(I, H, "bf16", 33, scale=1.3 / H ** 0.5, off=off)
    dh = mat(T, I, "bf16", 34, scale=0.1, pad=pad, off=off)
    dh[T // 2] = 0
    g, u, eg, eu = projections(x, wg, wu)
    gu = torch.stack([g, u]).to(torch.bfloat16)
    zero = torch.zeros_like(g)
    for kept, pr in ((gu, (gu[0].double(), gu[1].double(), zero, zero)), (None, (g, u, eg, eu))):
        outs = [framed(T, H, "bf16", pad, off), framed(I, H, "bf16", pad, off), framed(I, H, "bf16", pad)]
        got = moeq.glu_backward(dh, x, wg, wu, gu=kept, dx=outs[0][0], dw_gate=outs[1][0], dw_up=outs[2][0])
        refs = backward_refs(dh, x, wg, wu, *pr, "bf16", inner="f32")
        for o, (ref, bound), what, fr in zip(got, refs, ("dx", "dwg", "dwu"), outs):
            check(o, ref, bound, what + (" (kept)" if kept is not None else ""))
            assert fr[1](), what
        assert (got[0][T // 2] == 0).all()
        dx, _, _ = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dw=False)
        _, d1, d2 = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dx=False)
        assert torch.equal(dx, got[0]) and torch.equal(d1, got[1]) and torch.equal(d2, got[2])


def test_glu_gradients_against_differences(moeq):
    """f32: the directional derivative of sum(c * h) along random directions of
    x, Wg and Wu against central differences of the forward pass itself."""
    torch = torch_mod()
    T, H, I = 37, 90, 55
    x, wg, wu = mat(T, H, "f32", 31), mat(I, H, "f32", 32, scale=0.1), mat(I, H, "f32", 33, scale=0.1)
    c = mat(T, I, "f32", 34)
    h, gu = moeq.glu(x, wg, wu, save=True)
    grads = moeq.glu_backward(c, x, wg, wu, gu=gu)
    step = 2.0 ** -6
    for k, (t, gr) in enumerate(zip((x, wg, wu), grads)):
        d = mat(*t.shape, "f32", 40 + k, scale=float(t.std()) * 0.3)
        args = [x, wg, wu]
        vals = []
        for sgn in (2, 1, -1, -2):
            args[k] = (t.double() + sgn * step * d.double()).float()
            vals.append((c.double() * moeq.glu(*args).double()).sum().item())
        # fourth-order central difference: truncation ~ step^4, rounding ~ 2^-24 |c| |h| / step
        fd = (8 * (vals[1] - vals[2]) - (vals[0] - vals[3])) / (12 * step)
        an = (gr.double() * d.double()).sum().item()
        noise = 2 * (EPS["f32"] * (H + 8)) * (c.double().abs() * gu[1].double().abs()).sum().item() / step
        assert abs(fd - an) <= noise + 1e-4 * (gr.double() * d.double()).abs().sum().item(), (k, fd, an)


def test_glu_saturated_gates(moeq):
    """Gates far out on both sides: silu is 0 or the identity, nothing overflows."""
    torch = torch_mod()
    for dtype in ("bf16", "f32"):
        x = torch.zeros((20, 64), dtype=dt_of(dtype), device="cuda")
        x[:, 0] = torch.tensor([0.0, 1, -1, 20, -20, 80, -80, 90, -90, 104, -104, 200, -200, 1e4, -1e4, 1e30, -1e30, 3e38,
                                -3e38, 0.5], device="cuda").to(dt_of(dtype))
        wg = torch.zeros((8, 64), dtype=dt_of(dtype), device="cuda")
        wu = torch.zeros((8, 64), dtype=dt_of(dtype), device="cuda")
        wg[:, 0] = 1
        x[:, 1] = 1
        wu[:, 1] = 2
        h = moeq.glu(x, wg, wu)
        g = x[:, 0].double()
        ref = (g * sigmoid(g) * 2)[:, None].expand(20, 8)
        fin = ref.abs() < 3e38
        # e^-g leaves f32 below g = -ln(2^128) = -88.73, where silu(g) is taken as 0: there
        # |silu(g) u| <= 88.73 * 2^-128 * 2 = 5.3e-37 (g e^g falls towards -infinity)
        lost = 88.73 * 2.0 ** -128 * 2
        check(torch.where(fin, h.double(), torch.zeros_like(ref)), torch.where(fin, ref, torch.zeros_like(ref)),
              ref.abs() * (MISC + EPS[dtype] * 1.001) + lost, "h")
        dh = torch.ones_like(h)
        for gu in (None, moeq.glu(x, wg, wu, save=True)[1]):
            dx, dwg, dwu = moeq.glu_backward(dh, x, wg, wu, gu=gu)
            # dx[:, 1] sums 8 rows of silu(g) * 2: beyond f32 for the gate of 3e38 alone
            over = torch.zeros_like(dx, dtype=torch.bool)
            over[:, 1] = 16 * g * sigmoid(g) > 3.4028236e38
            assert over.sum() == 1
            assert torch.equal(torch.isinf(dx), over) and not torch.isnan(dx).any()
            assert not torch.isnan(dwg).any() and not torch.isnan(dwu).any()


# ------------------------------------------------- how a program uses them
def test_int8_block_as_a_program_runs_it(moeq):
    """Quantise, gated block, quantise, projection: each step's result against
    its definition on the step's own inputs, and the chain against f64."""
    torch = torch_mod()
    for T in (1, 5, 64, 300):
        x = mat(T, 512, "bf16", 51)
        wg, wu, wd = (mat(n, k, "f32", 52 + i, scale=1.5 / k ** 0.5) for i, (n, k) in
                      enumerate(((384, 512), (384, 512), (512, 384))))
        (qg, sg), (qu, su), (qd, sd) = (moeq.quant_i8(w) for w in (wg, wu, wd))
        q, s = moeq.quant_i8(x)
        h = moeq.glu_i8(q, s, qg, sg, qu, su)
        qh, sh = moeq.quant_i8(h)
        y = moeq.matmul_i8(qh, sh, qd, sd, dtype="f32")
        assert np.array_equal(qh.cpu().numpy(), quant_ref(h)[0])
        ref = int_sum(qh, qd) * sh.double()[:, None] * sd.double()
        check(y, ref, ref.abs() * 3.01 * 2.0 ** -24, "y")
        # each quantisation is off by half a step, a / 254 of the row's largest
        g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
        def err(a, wt):
            return ((a.double().abs().amax(1)[:, None] / 254) * wt.double().abs().sum(1) +
                    a.double().abs().sum(1)[:, None] * (wt.double().abs().amax(1) / 254) * (1 + 1 / 127))
        eg, eu = err(x, wg), err(x, wu)
        hr = g * sigmoid(g) * u
        eh = 1.1 * eg * (u.abs() + eu) + (g * sigmoid(g)).abs() * eu
        eh = eh + (hr.abs() + eh) * EPS["bf16"] * 1.01
        yr = hr @ wd.double().t()
        check(y, yr, 1.01 * (eh @ wd.double().abs().t() + err(h, wd)), "chain")


def test_training_step_lowers_nothing_by_itself_but_runs(moeq):
    """Forward, loss, backward and an update of the block inside torch, its
    gradients those of torch's own differentiation in f64."""
    torch = torch_mod()
    T, H, I = 50, 96, 64
    x, wg, wu = mat(T, H, "f32", 61), mat(I, H, "f32", 62, scale=0.1), mat(I, H, "f32", 63, scale=0.1)
    wd = mat(H, I, "f32", 64, scale=0.1)
    h, gu = moeq.glu(x, wg, wu, save=True)
    dy = mat(T, H, "f32", 65)
    grads = moeq.glu_backward((dy.double() @ wd.double()).float(), x, wg, wu, gu=gu)
    leaves = [t.double().requires_grad_() for t in (x, wg, wu)]
    z = torch.nn.functional.silu(leaves[0] @ leaves[1].t()) * (leaves[0] @ leaves[2].t())
    ((z @ wd.double().t()) * dy.double()).sum().backward()
    for got, leaf in zip(grads, leaves):
        assert (got.double() - leaf.grad).norm() <= 1e-5 * leaf.grad.norm()


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_captured_replayed_and_eager_calls_agree(moeq, T):
    """Two captured graphs with workspaces of their own and eager calls in
    between; inputs change between replays."""
    torch = torch_mod()
    H, I = 328, 200
    x, dh = mat(T, H, "bf16", 71), mat(T, I, "bf16", 72, scale=0.1)
    wg, wu = mat(I, H, "bf16", 73, scale=0.07), mat(I, H, "bf16", 74, scale=0.07)
    qg, sg = moeq.quant_i8(wg)
    qu, su = moeq.quant_i8(wu)

    def step():
        h, gu = moeq.glu(x, wg, wu, save=True)
        g = moeq.glu_backward(dh, x, wg, wu, gu=gu)
        q, s = moeq.quant_i8(x)
        return (h, gu) + tuple(g) + (moeq.glu_i8(q, s, qg, sg, qu, su),)
    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    for gr, o in zip(graphs, outs):
        gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, eager))
    x.mul_(-0.5)
    dh.mul_(2)
    want = [t.clone() for t in step()]
    graphs[0].replay()
    graphs[1].replay()
    step()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_streams_and_results_do_not_depend_on_each_other(moeq):
    """Calls on two streams at once, each with its own inputs, against the same
    calls one after the other; repeated calls give the same bits."""
    torch = torch_mod()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for i in range(2):
        T = (700, 33)[i]
        sets.append((mat(T, 640, "bf16", 81 + i), mat(320, 640, "bf16", 83 + i, scale=0.05),
                     mat(320, 640, "bf16", 85 + i, scale=0.05), mat(T, 320, "bf16", 87 + i)))
    want = [(moeq.glu(x, a, b), moeq.glu_backward(d, x, a, b)) for x, a, b, d in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st, (x, a, b, d) in zip(streams, sets):
            got.append((moeq.glu(x, a, b, stream=st), moeq.glu_backward(d, x, a, b, stream=st)))
    torch.cuda.synchronize()
    for i, (h, g) in enumerate(got):
        assert torch.equal(h, want[i % 2][0]) and all(torch.equal(p, q) for p, q in zip(g, want[i % 2][1]))


def test_column_windows_of_one_buffer(moeq):
    """x and h side by side in one buffer: not an overlap; a shifted window is one."""
    torch = torch_mod()
    buf = mat(40, 256 + 128, "bf16", 91)
    x, h = buf[:, :256], buf[:, 256:]
    wg, wu = mat(128, 256, "bf16", 92, scale=0.1), mat(128, 256, "bf16", 93, scale=0.1)
    want = moeq.glu(x.clone(), wg, wu)
    before = x.clone()
    moeq.glu(x, wg, wu, out=h)
    assert torch.equal(h, want) and torch.equal(x, before)
    with pytest.raises(moeq.MoeqError):
        moeq.glu(x, wg, wu, out=buf[:, 200:328])


def test_no_tokens(moeq):
    torch = torch_mod()
    x, wg, wu = mat(0, 64, "bf16", 1), mat(32, 64, "bf16", 2), mat(32, 64, "bf16", 3)
    assert moeq.glu(x, wg, wu).shape == (0, 32)
    dx, dwg, dwu = moeq.glu_backward(mat(0, 32, "bf16", 4), x, wg, wu)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()
    q, s = moeq.quant_i8(x)
    assert moeq.matmul_i8(q, s, mat(32, 64, "i8", 5), torch.ones(32, device="cuda")).shape == (0, 32)


def test_the_binding_refuses(moeq):
    torch = torch_mod()
    x, w = mat(4, 64, "bf16", 1), mat(32, 64, "bf16", 2)
    q, s = moeq.quant_i8(x)
    qw, sw = moeq.quant_i8(w)
    bad = [
        lambda: moeq.glu(x, w, w[:16]), lambda: moeq.glu(x, w, w.float()), lambda: moeq.glu(x.half(), w, w),
        lambda: moeq.glu(x, w.t(), w.t()), lambda: moeq.glu(x[0], w, w), lambda: moeq.glu(x, w, w.cpu()),
        lambda: moeq.glu(x, w, w, out=torch.empty(4, 31, dtype=x.dtype, device="cuda")),
        lambda: moeq.glu(x, w, w, gu=torch.empty(2, 4, 31, dtype=x.dtype, device="cuda")),
        lambda: moeq.glu(x[:1].expand(4, 64), w, w),
        lambda: moeq.glu_backward(x, x, w, w), lambda: moeq.glu_backward(mat(4, 32, "bf16", 1), x, w, w, need_dx=False,
                                                                        need_dw=False),
        lambda: moeq.glu_backward(mat(4, 32, "bf16", 1), x, w, w, workspace=torch.empty(16, device="cuda")),
        lambda: moeq.matmul_i8(x, s, qw, sw), lambda: moeq.matmul_i8(q, s, qw, sw[:31]),
        lambda: moeq.matmul_i8(q, s.double(), qw, sw), lambda: moeq.matmul_i8(q, s, qw, sw, dtype="f16"),
        lambda: moeq.matmul_i8(q, s, qw[:, :32], sw), lambda: moeq.quant_i8(x.half()), lambda: moeq.quant_i8(x[0]),
        lambda: moeq.quant_i8(x.t()), lambda: moeq.glu_i8(q, s, qw, sw, qw[:8], sw),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(moeq.MoeqError):
            call()
            raise AssertionError(f"call {k} was taken")


# --------------------------------------------------- what the kernels' rules rest on
def test_quant_i8_every_pair_of_bf16_significands(moeq):
    """bf16 quotients: every significand of x against every one of the row's
    largest, ten binades down: exact halves among them go to the even integer."""
    torch = torch_mod()
    m = torch.arange(128, 256, dtype=torch.float64)
    top = m[:, None]
    x = torch.cat([m * 2.0 ** -j for j in range(11)])[None].expand(128, -1)
    x = torch.where(x <= top, x, torch.zeros_like(x))
    rows = torch.cat([x, -x, top], dim=1).to(torch.bfloat16).cuda()
    q, s = moeq.quant_i8(rows)
    rq, rs = quant_ref(rows)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    t = rows.double().cpu().numpy() * 127 / rows.double().abs().amax(1, keepdim=True).cpu().numpy()
    # halves did occur: for a = 254 alone t = x / 2, a half for the 63 odd x below it and their negatives
    assert (np.abs(t - np.trunc(t)) == 0.5).sum() >= 126


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 100, 256, 257, 1000])
def test_tokens_do_not_see_each_other(moeq, T):
    """A NaN or an infinity in one token's row stays in that token's results."""
    torch = torch_mod()
    H, I = 200, 136
    for dtype in ("bf16", "f32"):
        x, wg, wu = mat(T, H, dtype, 1), mat(I, H, dtype, 2, scale=0.1), mat(I, H, dtype, 3, scale=0.1)
        want = moeq.glu(x, wg, wu)
        y = x.clone()
        y[T // 2, 7] = float("nan")
        y[0, 0] = float("inf") if T > 1 else float("nan")
        got = moeq.glu(y, wg, wu)
        rows = [r for r in range(T) if r not in (0, T // 2)]
        assert torch.equal(got[rows], want[rows])
        assert torch.isnan(got[T // 2]).all()
        # nor does a weight row's
        w2 = wg.clone()
        w2[5, 3] = float("nan")
        got = moeq.glu(x, w2, wu)
        cols = [c for c in range(I) if c != 5]
        assert torch.equal(got[:, cols], want[:, cols]) and torch.isnan(got[:, 5]).all()


def test_f32_parts_keep_their_exactness(moeq):
    """f32 operands with up to 8 significand bits are single parts: products
    and short sums of them are exact, whatever the sizes and alignment."""
    torch = torch_mod()
    for T, H, I in ((3, 32, 40), (70, 31, 65), (300, 32, 100)):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        x = torch.randint(-31, 32, (T, H), generator=g, device="cuda").float()
        wg, wu = (torch.randint(-31, 32, (I, H), generator=g, device="cuda").float() for _ in range(2))
        _, gu = moeq.glu(x, wg, wu, save=True)      # |sums| <= 32 * 961 < 2^24
        assert torch.equal(gu[0].double(), x.double() @ wg.double().t())
        assert torch.equal(gu[1].double(), x.double() @ wu.double().t())


def test_f32_values_near_the_ends_of_the_range(moeq):
    """Finite values whose nearest bf16 is infinite, and small ones, keep their
    accuracy: scaling an operand by a power of two scales the projections."""
    torch = torch_mod()
    for T in (2, 40, 300):
        x, w = mat(T, 96, "f32", 5), mat(50, 96, "f32", 6, scale=0.2)
        x = x / x.abs().max()                       # largest 1: times 3.4028e38 it is near the largest f32
        for sx, sw in ((3.4028e38, 2.0 ** -100), (2.0 ** 60, 2.0 ** -90), (2.0 ** -60, 2.0 ** -40)):
            y, v = x * sx, w * sw
            _, gu = moeq.glu(y, v, v, save=True)
            g, u, eg, eu = projections(y, v, v)
            check(gu[0], g, eg + (g.abs() + eg) * EPS["f32"] * 1.001, f"g at {sx} {sw}")


def test_wide_rows_far_apart(moeq):
    """Offsets beyond 2^31 elements: a few rows of a buffer with a huge row stride."""
    torch = torch_mod()
    ld = (1 << 30) + 64
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 64), (ld, 1))
    h = buf.as_strided((3, 48), (ld, 1), 4096)
    src = mat(3, 64, "bf16", 1)
    x.copy_(src)
    wg, wu = mat(48, 64, "bf16", 2, scale=0.2), mat(48, 64, "bf16", 3, scale=0.2)
    want = moeq.glu(src, wg, wu)
    moeq.glu(x, wg, wu, out=h)
    assert torch.equal(h, want)
    # the same rows as the dense kernels' weights (20 tokens: tensor maps with this stride)
    y = mat(20, 64, "bf16", 4)
    for t in (y, y[:2]):
        a, b = moeq.glu(t, src, src), moeq.glu(t, x, x)
        assert torch.equal(a, b)
    q, s = moeq.quant_i8(x)
    assert np.array_equal(q.cpu().numpy(), quant_ref(src)[0])
    del buf


def test_first_calls_inside_a_capture():
    """A process whose first calls of the dense operators are captured ones."""
    import subprocess
    import sys
    code = """
import torch
from bit_quantized_moe_routed_b200 import moeq
g = torch.Generator(device="cuda"); g.manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
sets = [(r(T, 136), r(72, 136) * 0.1, r(72, 136) * 0.1, r(T, 72)) for T in (2, 40, 300)]
def step(x, a, b, d):
    h, gu = moeq.glu(x, a, b, save=True)
    q, s = moeq.quant_i8(x)
    qa, sa = moeq.quant_i8(a)
    return (h, gu) + tuple(moeq.glu_backward(d, x, a, b, gu=gu)) + (moeq.matmul_i8(q, s, qa, sa), moeq.glu(x.float(), a.float(), b.float()))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = [step(*s) for s in sets]
graph.replay()
torch.cuda.synchronize()
for s, o in zip(sets, got):
    assert all(torch.equal(p, q) for p, q in zip(step(*s), o))
print("captured ok")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr
