"""The dense operators' Python calls beside other Python code that runs for the device."""
import ctypes as C
import time

import pytest

from _gpu_util import torch_mod
from test_gpu_dense import mat, moeq  # noqa: F401  (moeq: the fixture)

pytestmark = pytest.mark.gpu


def test_calls_wait_for_a_full_queue_without_the_interpreters_lock(moeq):
    """Thousands of calls behind a host function in Python: the queue fills while the function sleeps, and it needs the
    lock again to return."""
    from cuda.bindings import runtime as cudart
    torch = torch_mod()
    x, wg, wu = mat(1, 64, "bf16", 1), mat(32, 64, "bf16", 2), mat(32, 64, "bf16", 3)
    want = moeq.glu(x, wg, wu)
    out = torch.empty_like(want)
    seen = []

    def slow(_):
        time.sleep(0.5)
        seen.append(time.monotonic())
    fn = C.CFUNCTYPE(None, C.c_void_p)(slow)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        err, = cudart.cudaLaunchHostFunc(stream.cuda_stream, cudart.cudaHostFn_t(C.cast(fn, C.c_void_p).value), 0)
        assert err == cudart.cudaError_t.cudaSuccess
        for _ in range(6000):
            moeq.glu(x, wg, wu, out=out)
        done = time.monotonic()
    stream.synchronize()
    assert len(seen) == 1 and torch.equal(out, want)
    assert done > seen[0]      # the queue was full: the last calls came after the function's end
