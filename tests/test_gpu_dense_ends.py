"""The dense operators at the ends of their ranges: the largest number of rows."""
import pytest

from _gpu_util import torch_mod
from test_gpu_dense import moeq  # noqa: F401  (the fixture)

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
