"""The backward pass of the gated block for a few bf16 tokens on both sides of
the limits between its kernels, against f64 and with marks around everything
that a call may write."""
import pytest

from _gpu_util import torch_mod
from test_gpu_dense import backward_refs, check, framed, mat, moeq, projections  # noqa: F401  (moeq: the fixture)

pytestmark = pytest.mark.gpu


def workspace_of(moeq, dh, x, wg, wu, gu, outs):
    """(a workspace of exactly the size that the query names, inside a marked buffer; check of the marks)"""
    torch = torch_mod()

    def at(t):
        return (t.data_ptr(), t.stride(0))
    T, H, I = x.shape[0], x.shape[1], wg.shape[0]
    fields = [T, H, I, moeq.ACT["bf16"], *at(x), wg.data_ptr(), wu.data_ptr(), wg.stride(0), wu.stride(0),
              0 if gu is None else gu.data_ptr(), 0, 0, *at(dh), *at(outs[0]), outs[1].data_ptr(), outs[2].data_ptr(),
              outs[1].stride(0), outs[2].stride(0), 0, 0]
    n = moeq.lib().moeq_glu_workspace(moeq.GLU_ARGS.pack(*fields), 1)
    assert n >= 2 * T * I * 2
    guard = 1 << 18
    buf = torch.full((guard + n + guard,), 0xA5, dtype=torch.uint8, device="cuda")

    def untouched():
        return bool((buf[:guard] == 0xA5).all()) and bool((buf[guard + n:] == 0xA5).all())
    return buf[guard:guard + n], untouched


# T, H, I, pad, off: rows on 16 bytes and off them; the sizes lie on both sides of hidden * inter = 2^16, 2^19 and
# 2^23 and 2^24 (3 and 4 tokens) and of inter = 4 hidden and 64 hidden
LIMITS = [
    (1, 4096, 11008, 0, 0), (4, 4096, 4096, 0, 0), (1, 333, 260, 1, 0), (4, 1000, 517, 3, 0), (2, 1000, 517, 3, 1),
    (2, 256, 256, 3, 0), (2, 257, 256, 3, 0), (1, 301, 217, 0, 5), (3, 1024, 512, 0, 0), (3, 1024, 520, 0, 0),
    (4, 4096, 2048, 0, 0), (4, 4096, 2056, 0, 0), (4, 4096, 2048, 5, 0), (1, 8192, 4104, 8, 8), (3, 2056, 5504, 0, 0),
    (1, 1024, 4096, 0, 0), (1, 1024, 4104, 0, 0), (2, 128, 8192, 0, 0), (2, 120, 8192, 0, 0), (3, 64, 65536, 0, 0),
    (4, 4096, 4104, 0, 0), (2, 999, 1003, 0, 0), (5, 1000, 517, 3, 0), (5, 4096, 4096, 0, 0),
]


@pytest.mark.parametrize("T,H,I,pad,off", LIMITS)
def test_gradients_on_both_sides_of_the_limits(moeq, T, H, I, pad, off):
    torch = torch_mod()
    x = mat(T, H, "bf16", 101, pad=pad, off=off)
    wg = mat(I, H, "bf16", 102, scale=1.3 / H ** 0.5, pad=pad)
    wu = mat(I, H, "bf16", 103, scale=1.3 / H ** 0.5, pad=pad, off=off)
    dh = mat(T, I, "bf16", 104, scale=0.1, pad=pad, off=off)
    g, u, eg, eu = projections(x, wg, wu)
    gu = torch.stack([g, u]).to(torch.bfloat16)
    zero = torch.zeros_like(g)
    for kept, pr in ((gu, (gu[0].double(), gu[1].double(), zero, zero)), (None, (g, u, eg, eu))):
        outs = [framed(T, H, "bf16", pad, off), framed(I, H, "bf16", pad, off), framed(I, H, "bf16", pad)]
        ws, untouched = workspace_of(moeq, dh, x, wg, wu, kept, [o[0] for o in outs])
        got = moeq.glu_backward(dh, x, wg, wu, gu=kept, dx=outs[0][0], dw_gate=outs[1][0], dw_up=outs[2][0], workspace=ws)
        what = " (kept)" if kept is not None else ""
        assert untouched(), "bytes around the workspace" + what
        for o, (ref, bound), name, fr in zip(got, backward_refs(dh, x, wg, wu, *pr, "bf16"), ("dx", "dwg", "dwu"), outs):
            check(o, ref, bound, name + what)
            assert fr[1](), name + what
        # a gradient that is left out does not change the others
        dx, _, _ = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dw=False)
        _, d1, d2 = moeq.glu_backward(dh, x, wg, wu, gu=kept, need_dx=False)
        assert torch.equal(dx, got[0]) and torch.equal(d1, got[1]) and torch.equal(d2, got[2])


@pytest.mark.parametrize("T,H,I", [(1, 1024, 1024), (1, 4096, 11008), (2, 4096, 4096), (2, 2056, 5504), (3, 1000, 4000),
                                   (4, 4096, 2048)])
def test_kept_and_recomputed_projections_round_once(moeq, T, H, I):
    """Rows on 16 bytes, inter up to 4 hidden, 1 and 2 tokens at any size, 3 and 4 up to 2^23 weights: dg and du
    stay f32 with the projections kept as well as without them."""
    torch = torch_mod()
    x, dh = mat(T, H, "bf16", 111), mat(T, I, "bf16", 114, scale=0.1)
    wg, wu = mat(I, H, "bf16", 112, scale=1.3 / H ** 0.5), mat(I, H, "bf16", 113, scale=1.3 / H ** 0.5)
    g, u, eg, eu = projections(x, wg, wu)
    gu = torch.stack([g, u]).to(torch.bfloat16)
    zero = torch.zeros_like(g)
    for kept, pr in ((gu, (gu[0].double(), gu[1].double(), zero, zero)), (None, (g, u, eg, eu))):
        got = moeq.glu_backward(dh, x, wg, wu, gu=kept)
        refs = backward_refs(dh, x, wg, wu, *pr, "bf16", inner="f32")
        for o, (ref, bound), name in zip(got, refs, ("dx", "dwg", "dwu")):
            check(o, ref, bound, name + (" (kept)" if kept is not None else ""))
