"""Decisions of the dense operators on the host.

The backward pass of the gated block: the entry points over launchers that only
note what their kernels write and read (host/dense_plan.cpp).
Every step stays inside the workspace that the query names, no part lies on
another, and each kernel reads the gate gradients in the type they were
written in, on both sides of every limit between kernels."""
import glob
import itertools
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def program(tmp, name, objects, flags=()):
    """A host program of one source and the library's objects of these sources (all of them for none): f(cases) -> lines, a case's numbers on a line."""
    from bit_quantized_moe_routed_b200 import build
    build.build()
    out = str(tmp / name)
    srcs = objects or [os.path.basename(f)[:-3] for f in glob.glob(os.path.join(build.CSRC, "*.cu"))]
    objs = [os.path.join(build.BUILD, f + ".o") for f in srcs]
    for cmd in ([*build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-x", "cu",
                 os.path.join(HERE, "host", name + ".cpp"), "-c", "-o", out + ".o"],
                [*build.ARCH, *flags, out + ".o", *objs, "-o", out]):
        r = subprocess.run([build.NVCC, *cmd], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr

    def run(cases):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in cases)
        r = subprocess.run([out], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout.split("\n")[:-1]
    return run


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return program(tmp_path_factory.mktemp("plan"), "dense_plan", ["dense_api"])


SIZES = [(1, 1), (64, 138), (256, 256), (257, 256), (77, 301), (333, 260), (1000, 517), (1024, 512), (1024, 520),
         (1024, 1024), (4096, 1024), (4096, 2048), (4096, 2056), (4096, 4096), (4096, 8192), (4096, 8200), (4096, 11008),
         (8192, 28672), (1024, 4104), (1024, 4096), (512, 8192), (128, 8192), (120, 8192), (64, 8192), (64, 65536), (4096, 4104)]


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 16, 17, 64, 1000])
def test_backward_stays_in_its_workspace(plan, T):
    cases = [(T, H, I, off16, dtype, gu, dx, dw, faster)
             for (H, I), off16, dtype, gu, (dx, dw), faster in itertools.product(
                 SIZES, (0, 1), (0, 1), (0, 1), ((1, 1), (1, 0), (0, 1)), (0, 1))]
    got = plan(cases)
    assert len(got) == len(cases)
    bad = [(c, g) for c, g in zip(cases, got) if g != "ok"]
    assert not bad, f"{len(bad)} of {len(cases)}, the first: {bad[:3]}"


def test_quantiser_grid_covers_its_rows(tmp_path):
    """Up to the 2^31 - 1 rows that the call takes: a thread group for each row, none lost to 32-bit sums."""
    run = program(tmp_path, "quant_grid", [], ["-Xlinker", "--wrap=cudaLaunchKernelExC"])
    cases = [(r, c) for r in (1, 7, 8, 9, 2**31 - 9, 2**31 - 8, 2**31 - 7, 2**31 - 1) for c in (1, 1024, 1025, 4096, 4097)]
    for (rows, cols), line in zip(cases, run(cases), strict=True):
        per = 8 if cols <= 1024 else (2 if cols <= 4096 else 1)
        assert line == f"{-(-rows // per)} 1 1 256", (rows, cols, line)


@pytest.mark.parametrize("T,H,I,off,dtype,kept,want", [
    # bf16 gate gradients [2][T][I padded to 64]: in f32 for few tokens
    (1, 4096, 11008, 0, 1, 0, 2 * 11008 * 4), (1, 4096, 11008, 0, 1, 1, 2 * 11008 * 4),
    (4, 4096, 2048, 0, 1, 0, 2 * 4 * 2048 * 4), (4, 4096, 2056, 0, 1, 1, 2 * 4 * 2112 * 2), (4, 4096, 4104, 0, 1, 0, 2 * 4 * 4160 * 2),
    (3, 4096, 2056, 0, 1, 1, 2 * 3 * 2112 * 2), (5, 4096, 4096, 0, 1, 0, 2 * 5 * 4096 * 2),
    (1, 1024, 4096, 0, 1, 1, 2 * 4096 * 4), (1, 1024, 4104, 0, 1, 1, 2 * 4160 * 2), (1, 128, 8200, 0, 1, 0, 2 * 8256 * 2),
    (2, 256, 256, 3, 1, 0, 2 * 2 * 256 * 4),
    # rows off 16 bytes: and x [T] and both W [I] in rows of 128 bytes' multiples (H = 257: 640 bytes)
    (2, 257, 256, 3, 1, 0, 2 * 640 + 2 * 256 * 640 + 2 * 2 * 256 * 2),
    (300, 257, 256, 3, 1, 1, 300 * 640 + 2 * 256 * 640 + 2 * 300 * 256 * 2),
    # f32: three planes each of x, both W, dg and du, rows padded to 64
    (4, 64, 32, 0, 0, 0, 3 * 4 * 64 * 2 + 2 * 3 * 32 * 64 * 2 + 2 * 3 * 4 * 64 * 2),
    (4, 64, 32, 3, 0, 1, 3 * 4 * 64 * 2 + 2 * 3 * 32 * 64 * 2 + 2 * 3 * 4 * 64 * 2),
])
def test_backward_workspace_to_the_byte(T, H, I, off, dtype, kept, want):
    from bit_quantized_moe_routed_b200 import build
    build.build()
    from bit_quantized_moe_routed_b200 import moeq
    a = [k << 40 for k in range(1, 9)]
    ldh, ldi = H + off, I + off
    args = moeq.GLU_ARGS.pack(T, H, I, dtype, a[0], ldh, a[1], a[2], ldh, ldh, a[3] if kept else 0, 0, 0, a[4], ldi, a[5], ldh,
                              a[6], a[7], ldh, ldh, 0, 0)
    assert moeq.lib().moeq_glu_workspace(args, 1) == want
