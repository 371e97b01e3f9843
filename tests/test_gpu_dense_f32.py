"""f32 products of the dense operators: what their accuracy rests on.  The kernels
multiply three bf16 parts of each operand (hi + mid + lo = 24 bits) in six products
of parts and sum the leading one in pieces of 128 terms.  Bounds that hold for any
f32 sum would pass with a part missing; these tests would not."""
import pytest

from _gpu_util import torch_mod
from test_gpu_dense import mat, moeq  # noqa: F401  (moeq: the fixture)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 40, 33), (3, 64, 40), (70, 1000, 200), (129, 130, 517), (300, 333, 64), (40, 4096, 96)]   # T, H, I


def picks(rows, cols, seed):
    """[rows][cols] with one power of two in each row and each one's place and value: products with it only pick and
    scale, so that every sum has one term and an f32 result is exact."""
    torch = torch_mod()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    at = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    at[0], at[-1] = 0, cols - 1
    v = 2.0 ** torch.randint(-3, 4, (rows,), generator=g, device="cuda").float()
    m = torch.zeros((rows, cols), device="cuda")
    m[torch.arange(rows, device="cuda"), at] = v
    return m, at, v[:, None]


def values(rows, cols, seed, device="cuda"):
    """Random values, each with something in all three of its parts: 129..255 in hi, a fraction of 128..254 / 512 in
    mid, an odd number up to 63 of 2^-16 in lo, the signs of the parts and a power of two at random."""
    torch = torch_mod() if device == "cuda" else __import__("torch")
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def r(lo, hi):
        return torch.randint(lo, hi, (rows, cols), generator=g, device=device).float()
    hi, mid, lo = r(129, 256), r(128, 255) / 512 * (2 * r(0, 2) - 1), (2 * r(0, 32) + 1) / 65536 * (2 * r(0, 2) - 1)
    v = (hi + mid + lo) * (2 * r(0, 2) - 1) * 2 ** r(-10, -4)
    a = v.bfloat16().float()
    b = (v - a).bfloat16().float()
    c = v - a - b
    assert (b != 0).all() and (c != 0).all() and torch.equal(c.bfloat16().float(), c)
    return v


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_projections_keep_all_bits_of_either_operand(moeq, T, H, I):
    torch = torch_mod()
    x, at, v = picks(T, H, 1)
    wg, wu = values(I, H, 2), values(I, H, 3)
    _, gu = moeq.glu(x, wg, wu, save=True)
    assert torch.equal(gu[0], wg[:, at].t() * v) and torch.equal(gu[1], wu[:, at].t() * v)
    x = values(T, H, 4)
    (wg, ag, vg), (wu, au, vu) = picks(I, H, 5), picks(I, H, 6)
    _, gu = moeq.glu(x, wg, wu, save=True)
    assert torch.equal(gu[0], x[:, ag] * vg.t()) and torch.equal(gu[1], x[:, au] * vu.t())


def test_middle_parts_are_multiplied(moeq):
    """(1 + 2^-9)^2 = 1 + 2^-8 + 2^-18: hi is 1 and mid 2^-9 of both."""
    torch = torch_mod()
    for T, H, I in SHAPES:
        x, w = torch.zeros((T, H), device="cuda"), torch.zeros((I, H), device="cuda")
        x[:, H // 2] = w[:, H // 2] = 1 + 2.0 ** -9
        _, gu = moeq.glu(x, w, -w, save=True)
        want = 1 + 2.0 ** -8 + 2.0 ** -18
        assert (gu[0] == want).all() and (gu[1] == -want).all()


def gates(T, I, up):
    """Kept projections for which dg = dh, du = 0 (g = 0, u = 2: silu'(0) = 1/2), or du = 128 dh, dg = 0 (g = 128, u = 0)."""
    torch = torch_mod()
    gu = torch.zeros((2, T, I), device="cuda")
    gu[0 if up else 1] = 128 if up else 2
    return gu, 128.0 if up else 1.0


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_gradients_keep_all_bits_of_either_operand(moeq, T, H, I, up):
    torch = torch_mod()
    gu, k = gates(T, I, up)
    x, w = values(T, H, 11), [values(I, H, 12), values(I, H, 13)]
    # dh picks: a row of W for each token's dx, rows of x for dW
    dh, at, v = picks(T, I, 14)
    dx, _, _ = moeq.glu_backward(dh, x, *w, gu=gu)
    assert torch.equal(dx, w[up][at] * v * k)
    pt, at, v = picks(I, T, 15)
    dh = pt.t().contiguous()
    dw = moeq.glu_backward(dh, x, *w, gu=gu)[1:]
    assert torch.equal(dw[up], x[at] * v * k) and not dw[not up].any()
    # W and x pick from dh
    dh = values(T, I, 16)
    wt, at, v = picks(H, I, 17)
    w[up] = wt.t().contiguous()
    dx, _, _ = moeq.glu_backward(dh, x, *w, gu=gu)
    assert torch.equal(dx, dh[:, at] * v.t() * k)
    xt, at, v = picks(H, T, 18)
    dw = moeq.glu_backward(dh, xt.t().contiguous(), *w, gu=gu)[1:]
    assert torch.equal(dw[up], (dh[at] * v * k).t())


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_recomputed_gate_gradients_keep_all_bits(moeq, T, H, I):
    """x is the first unit vector, Wg's first column 0 and Wu's 2: g = 0, u = 2 and dg = dh again, through the epilogue
    that writes dg in parts."""
    torch = torch_mod()
    x = torch.zeros((T, H), device="cuda")
    x[:, 0] = 1
    wg, wu = values(I, H, 21), values(I, H, 22)
    wg[:, 0], wu[:, 0] = 0, 2
    dh, at, v = picks(T, I, 23)
    dx, _, _ = moeq.glu_backward(dh, x, wg, wu)
    assert torch.equal(dx, wg[at] * v)
    pt, at, _ = picks(I, T, 24)
    dh = (pt != 0).t() * values(T, I, 25)      # one value a column
    _, dwg, dwu = moeq.glu_backward(dh.contiguous(), x, wg, wu)
    assert torch.equal(dwg[:, 0], dh.sum(0)) and not dwg[:, 1:].any() and not dwu.any()


@pytest.mark.parametrize("K", [64, 520, 1000, 4096])
def test_long_sums_of_one_sign(moeq, K):
    """Sums of positive terms, where what an adder cuts off adds up.  The tensor core cuts off 2^-24 of the running
    value a step of 16 terms on average; in a piece of 128 the running value is 9/16 of the last on average: 8 * 9/16 *
    2^-24 = 2.7e-7 at most.  Joining the K / 128 pieces rounds by 2^-25 on average each, independently: 1.7e-7 at 4096.
    The five small products' sum is below 2^-8 of the whole (its terms have either sign), 5 K / 16 steps: below 1.5e-7.
    In all below 1e-6; unbroken sums of 4096 would lose 128 steps' average value, 256 * 2^-24 / 2 = 7.6e-6 (1000: 1.9e-6,
    520: 9.7e-7)."""
    torch = torch_mod()

    def near(got, want, what):
        e = ((got.double() - want).norm() / want.norm()).item()
        assert e < (1e-6 if K > 520 else 6e-7), f"{what}: {e:.2e}"
    T, I = 96, 80
    x, wg, wu = (mat(n, K, "f32", s).abs() for n, s in ((T, 31), (I, 32), (I, 33)))
    _, gu = moeq.glu(x, wg, wu, save=True)
    near(gu[0], x.double() @ wg.double().t(), "g")
    near(gu[1], x.double() @ wu.double().t(), "u")
    # dx over K outputs, dW over K tokens
    H = 72
    for up in (False, True):
        k = gates(1, 1, up)[1]
        w, x, dh = [mat(K, H, "f32", 34).abs(), mat(K, H, "f32", 35).abs()], mat(T, H, "f32", 36), mat(T, K, "f32", 37).abs()
        dx, _, _ = moeq.glu_backward(dh, x, *w, gu=gates(T, K, up)[0], need_dw=False)
        near(dx, dh.double() @ w[up].double() * k, "dx")
        w, x, dh = [mat(I, H, "f32", 38), mat(I, H, "f32", 39)], mat(K, H, "f32", 40).abs(), mat(K, I, "f32", 41).abs()
        dw = moeq.glu_backward(dh, x, *w, gu=gates(K, I, up)[0], need_dx=False)[1:]
        near(dw[up], dh.double().t() @ x.double() * k, "dW")
