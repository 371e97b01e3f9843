"""The gated block inside torch's autograd: by itself it is not seen; as the
torch.autograd.Function of glu's docstring it gives the gradients."""
import inspect
import re
import textwrap

import pytest

from _gpu_util import torch_mod
from test_gpu_dense import backward_refs, check, mat, moeq, projections  # noqa: F401  (moeq: the fixture)

pytestmark = pytest.mark.gpu


def documented_function(moeq):
    """The class of the docstring, as it stands there."""
    import torch
    doc = inspect.getdoc(moeq.glu)
    code = textwrap.dedent(doc[doc.index("    class Glu"):])
    scope = {"torch": torch, "moeq": moeq}
    exec(code, scope)
    return scope["Glu"]


def test_the_call_alone_is_detached_and_says_so(moeq):
    x, wg, wu = mat(8, 64, "bf16", 1).clone().requires_grad_(), mat(32, 64, "bf16", 2), mat(32, 64, "bf16", 3)
    assert not moeq.glu(x, wg, wu).requires_grad
    assert re.search(r"autograd does not see this call", inspect.getdoc(moeq.glu))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 4, 50, 400])
def test_the_documented_function_gives_the_gradients(moeq, T, dtype):
    torch = torch_mod()
    H, I = 96, 64
    leaves = [mat(T, H, dtype, 1).clone(), mat(I, H, dtype, 2, scale=0.13).clone(), mat(I, H, dtype, 3, scale=0.13).clone()]
    for t in leaves:
        t.requires_grad_()
    x, wg, wu = leaves
    Glu = documented_function(moeq)
    # the gradient of a sum arrives expanded (stride 0): the function makes it contiguous
    h = Glu.apply(x, wg, wu)
    (h.float().sum() * 0.5).backward()
    dh = torch.full((T, I), 0.5, device="cuda", dtype=h.dtype)
    g, u, eg, eu = projections(x.detach(), wg.detach(), wu.detach())
    # gu is rounded to the type before the backward pass reads it
    half = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    refs = backward_refs(dh, x.detach(), wg.detach(), wu.detach(), g, u, eg + (g.abs() + eg) * half, eu + (u.abs() + eu) * half, dtype)
    for t, (ref, bound), what in zip(leaves, refs, ("x", "w_gate", "w_up")):
        check(t.grad, ref, bound, what)
