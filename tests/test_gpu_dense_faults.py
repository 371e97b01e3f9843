"""The dense operators' bounded waits running out: MOEQ_TEST_WAIT_CYCLES, read at
the first call and when the status word is cleared, shortens the limit that
kernels give their waits.  A kernel that gives up returns, raises
MOEQ_ERR_TIMEOUT in the status word and leaves the device usable; the next call
under the normal limit is right."""
import pytest

from _gpu_util import torch_mod
from test_gpu_dense import mat

pytestmark = pytest.mark.gpu


def block(T, H, I, dtype, backward=False):
    def make(moeq):
        x, wg, wu, dh = mat(T, H, dtype, 1), mat(I, H, dtype, 2, scale=0.05), mat(I, H, dtype, 3, scale=0.05), mat(T, I, dtype, 4)
        if not backward:
            return lambda: (moeq.glu(x, wg, wu),)
        gu = moeq.glu(x, wg, wu, save=True)[1]
        return lambda: moeq.glu_backward(dh, x, wg, wu, gu=gu) + moeq.glu_backward(dh, x, wg, wu)
    return make


def int8(T, K, N, n_w):
    def make(moeq):
        torch = torch_mod()
        x, w = mat(T, K, "i8", 1), [mat(N, K, "i8", 2 + i) for i in range(n_w)]
        sx, sw = torch.rand(T, device="cuda") * 1e-3, torch.rand(N, device="cuda") * 1e-2
        if n_w == 1:
            return lambda: (moeq.matmul_i8(x, sx, w[0], sw),)
        return lambda: (moeq.glu_i8(x, sx, w[0], sw, w[1], sw, dtype="f32"),)
    return make


CALLS = {
    "tiles bf16": block(2048, 1024, 1024, "bf16"), "tiles bf16 backward": block(2048, 1024, 1024, "bf16", True),
    "tiles int8": int8(2048, 2048, 2048, 1), "tiles int8 block": int8(2048, 2048, 2048, 2),
    "clusters bf16": block(64, 4096, 2048, "bf16"), "clusters bf16 backward": block(300, 1024, 2048, "bf16", True),
    "clusters int8": int8(64, 4096, 1024, 1), "clusters int8, long": int8(64, 16384, 1024, 1), "clusters int8 block": int8(64, 4096, 1024, 2),
    "planes": block(64, 1024, 256, "f32"), "planes backward": block(64, 1024, 256, "f32", True),
    "planes, more tiles": block(700, 520, 1030, "f32", True),
}

# 64 x 4096 x 1024: 32 K blocks of 128 over clusters of 8 are 4 a CTA, which its ring of 4 stages holds: all are loaded
# before the first wait and may have landed by then, so that no wait is left to run out
MAY_NOT_WAIT = {"clusters int8"}


@pytest.mark.parametrize("limit", [1, 20000])
@pytest.mark.parametrize("call", sorted(CALLS))
def test_wait_runs_out_and_the_device_stays_usable(call, limit, monkeypatch):
    from bit_quantized_moe_routed_b200 import moeq
    torch = torch_mod()
    run = CALLS[call](moeq)
    want = run()
    assert moeq.dense_status(clear=True) == moeq.OK
    try:
        monkeypatch.setenv("MOEQ_TEST_WAIT_CYCLES", str(limit))
        assert moeq.dense_status(clear=True) == moeq.OK      # reads the limit
        for _ in range(3):
            got = run()                                      # returns: every wait is bounded
            st = moeq.dense_status(clear=True)
            assert st in (moeq.OK, moeq.TIMEOUT)
            if limit == 1 and call not in MAY_NOT_WAIT:
                assert st == moeq.TIMEOUT                    # a 1-cycle limit cannot be met
            if st == moeq.OK:
                assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        monkeypatch.delenv("MOEQ_TEST_WAIT_CYCLES", raising=False)
        moeq.dense_status(clear=True)                        # the normal limit again
    torch.cuda.synchronize()                                 # the context is intact
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    assert moeq.dense_status() == moeq.OK
