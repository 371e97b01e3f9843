"""The backward pass of the gated block on the host: the entry points over
launchers that only note what their kernels write and read (host/dense_plan.cpp).
Every step stays inside the workspace that the query names, no part lies on
another, and each kernel reads the gate gradients in the type they were
written in, on both sides of every limit between kernels."""
import itertools
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from bit_quantized_moe_routed_b200 import build
    build.build()
    out = str(tmp_path_factory.mktemp("plan") / "dense_plan")
    r = subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-x", "cu",
                        os.path.join(HERE, "host", "dense_plan.cpp"), "-o", out + ".o", "-c"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([build.NVCC, *build.ARCH, out + ".o", os.path.join(build.BUILD, "dense_api.o"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in cases)
        r = subprocess.run([out], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout.split("\n")[:-1]
    return run


SIZES = [(1, 1), (64, 138), (256, 256), (257, 256), (77, 301), (333, 260), (1000, 517), (1024, 512), (1024, 520),
         (1024, 1024), (4096, 1024), (4096, 2048), (4096, 2056), (4096, 4096), (4096, 8192), (4096, 8200), (4096, 11008),
         (8192, 28672)]


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 16, 17, 64, 1000])
def test_backward_stays_in_its_workspace(plan, T):
    cases = [(T, H, I, off16, dtype, gu, dx, dw, faster)
             for (H, I), off16, dtype, gu, (dx, dw), faster in itertools.product(
                 SIZES, (0, 1), (0, 1), (0, 1), ((1, 1), (1, 0), (0, 1)), (0, 1))]
    got = plan(cases)
    assert len(got) == len(cases)
    bad = [(c, g) for c, g in zip(cases, got) if g != "ok"]
    assert not bad, f"{len(bad)} of {len(cases)}, the first: {bad[:3]}"
