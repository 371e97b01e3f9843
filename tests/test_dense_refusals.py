"""Host-side refusals of the dense operators: every call here is answered by
the argument checks, before any CUDA call (made-up addresses, no GPU)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def moeq():
    from bit_quantized_moe_routed_b200 import build
    build.build()
    from bit_quantized_moe_routed_b200 import moeq as m
    return m


A = 1 << 32      # made-up device addresses, far apart
ADDR = {n: A * (i + 1) for i, n in enumerate(
    ("x", "w0", "w1", "gu", "h", "dh", "dx", "dw0", "dw1", "ws", "sx", "s0", "s1", "out"))}


def i8(moeq, n_w=1, **kw):
    d = dict(T=4, K=64, N=32, dt=1, x=ADDR["x"], ldx=64, sx=ADDR["sx"], w0=ADDR["w0"],
             w1=ADDR["w1"] if n_w == 2 else 0, ld0=64, ld1=64 if n_w == 2 else 0, s0=ADDR["s0"],
             s1=ADDR["s1"] if n_w == 2 else 0, out=ADDR["out"], ldo=32, ws=0, wsb=0)
    d.update(kw)
    return moeq.I8_ARGS.pack(*d.values())


def glu(moeq, **kw):
    d = dict(T=4, H=64, I=32, dt=1, x=ADDR["x"], ldx=64, w0=ADDR["w0"], w1=ADDR["w1"], ld0=64, ld1=64, gu=0,
             h=ADDR["h"], ldh=32, dh=ADDR["dh"], lddh=32, dx=ADDR["dx"], lddx=64, dw0=ADDR["dw0"], dw1=ADDR["dw1"],
             lddw0=64, lddw1=64, ws=ADDR["ws"], wsb=1 << 20)
    d.update(kw)
    return moeq.GLU_ARGS.pack(*d.values())


def test_packed_arguments_match_the_c_structs(moeq):
    class I8(C.Structure):
        _fields_ = [("n_tokens", C.c_int32), ("n_in", C.c_int32), ("n_out", C.c_int32), ("out_dtype", C.c_int32),
                    ("x", C.c_void_p), ("ldx", C.c_int64), ("x_scale", C.c_void_p), ("w", C.c_void_p * 2),
                    ("ldw", C.c_int64 * 2), ("w_scale", C.c_void_p * 2), ("out", C.c_void_p), ("ldo", C.c_int64),
                    ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]

    class Glu(C.Structure):
        _fields_ = [("n_tokens", C.c_int32), ("hidden", C.c_int32), ("inter", C.c_int32), ("dtype", C.c_int32),
                    ("x", C.c_void_p), ("ldx", C.c_int64), ("w", C.c_void_p * 2), ("ldw", C.c_int64 * 2),
                    ("gu", C.c_void_p), ("h", C.c_void_p), ("ldh", C.c_int64), ("dh", C.c_void_p),
                    ("lddh", C.c_int64), ("dx", C.c_void_p), ("lddx", C.c_int64), ("dw", C.c_void_p * 2),
                    ("lddw", C.c_int64 * 2), ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]
    assert moeq.I8_ARGS.size == C.sizeof(I8)
    assert moeq.GLU_ARGS.size == C.sizeof(Glu)
    g = Glu.from_buffer_copy(glu(moeq))
    assert (g.n_tokens, g.ldx, g.w[1], g.dw[1], g.lddw[1], g.workspace_bytes) == (4, 64, ADDR["w1"], ADDR["dw1"], 64,
                                                                                 1 << 20)
    a = I8.from_buffer_copy(i8(moeq, 2))
    assert (a.n_out, a.x_scale, a.ldw[1], a.w_scale[1], a.ldo) == (32, ADDR["sx"], 64, ADDR["s1"], 32)


QUANT = dict(x=ADDR["x"], dt=1, M=4, K=64, ldx=64, q=ADDR["out"], ldq=64, sc=ADDR["s0"])


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(q=None), dict(sc=None), dict(dt=2), dict(dt=-1), dict(M=-1), dict(K=0), dict(ldx=63),
    dict(ldq=63), dict(K=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31), dict(x=ADDR["x"] + 1), dict(dt=0, x=ADDR["x"] + 2), dict(sc=ADDR["s0"] + 2), dict(ldx=1 << 40),
    dict(q=ADDR["x"]), dict(q=ADDR["x"] + 3 * 128 + 127), dict(sc=ADDR["x"] + 64), dict(sc=ADDR["out"]),
])
def test_quant_i8_refuses(moeq, bad):
    a = dict(QUANT, **bad)
    assert moeq.lib().moeq_quant_i8(*a.values(), None) == moeq.INVALID_ARGUMENT


def test_no_tokens_is_a_no_op(moeq):
    lib = moeq.lib()
    assert lib.moeq_quant_i8(None, 1, 0, 64, 64, None, 64, None, None) == moeq.OK
    assert lib.moeq_matmul_i8(i8(moeq, T=0, x=0, sx=0, out=0), None) == moeq.OK
    assert lib.moeq_glu_i8(i8(moeq, 2, T=0, x=0, sx=0, out=0), None) == moeq.OK
    assert lib.moeq_glu(glu(moeq, T=0, x=0, h=0), None) == moeq.OK
    assert lib.moeq_glu_backward(glu(moeq, T=0, x=0, dh=0, dw0=0, dw1=0), None) == moeq.OK


I8_BAD = [
    dict(T=-1), dict(K=0), dict(K=131072, ldx=131072, ld0=131072, ld1=131072), dict(N=0), dict(N=(1 << 20) + 1),
    dict(dt=3), dict(x=0), dict(sx=0), dict(w0=0), dict(s0=0), dict(out=0), dict(ldx=63), dict(ld0=63), dict(ldo=31),
    dict(out=ADDR["out"] + 1), dict(dt=0, out=ADDR["out"] + 2), dict(sx=ADDR["sx"] + 1), dict(s0=ADDR["s0"] + 2),
    dict(out=ADDR["x"]), dict(out=ADDR["w0"] + 100), dict(out=ADDR["sx"]), dict(out=ADDR["s0"] + 64),
]


@pytest.mark.parametrize("bad", I8_BAD)
def test_int8_products_refuse(moeq, bad):
    lib = moeq.lib()
    assert lib.moeq_matmul_i8(i8(moeq, 1, **{k: v for k, v in bad.items() if k != "ld1"}), None) == \
        moeq.INVALID_ARGUMENT
    assert lib.moeq_glu_i8(i8(moeq, 2, **bad), None) == moeq.INVALID_ARGUMENT


def test_int8_products_refuse_the_wrong_number_of_weights(moeq):
    lib = moeq.lib()
    assert lib.moeq_matmul_i8(i8(moeq, 2), None) == moeq.INVALID_ARGUMENT
    assert lib.moeq_glu_i8(i8(moeq, 1), None) == moeq.INVALID_ARGUMENT
    for k in ("w1", "s1"):
        assert lib.moeq_glu_i8(i8(moeq, 2, **{k: 0}), None) == moeq.INVALID_ARGUMENT
    assert lib.moeq_glu_i8(i8(moeq, 2, ld1=63), None) == moeq.INVALID_ARGUMENT
    assert lib.moeq_i8_workspace(i8(moeq, 1), 2) == -1
    assert lib.moeq_i8_workspace(i8(moeq, 1), 3) == -1
    assert lib.moeq_i8_workspace(i8(moeq, 1), 1) >= 0
    assert lib.moeq_matmul_i8(None, None) == moeq.INVALID_ARGUMENT


GLU_BAD = [
    dict(T=-1), dict(H=0), dict(I=0), dict(H=(1 << 20) + 1, ldx=1 << 22, ld0=1 << 22, ld1=1 << 22, lddx=1 << 22), dict(dt=2),
    dict(x=0), dict(w0=0), dict(w1=0), dict(ldx=63), dict(ld0=63), dict(ld1=63), dict(x=ADDR["x"] + 1),
    dict(dt=0, w1=ADDR["w1"] + 2), dict(gu=ADDR["gu"] + 1),
]


@pytest.mark.parametrize("bad", GLU_BAD + [
    dict(h=0), dict(ldh=31), dict(h=ADDR["h"] + 1), dict(h=ADDR["x"]), dict(h=ADDR["w1"] + 2), dict(gu=ADDR["h"]),
    dict(gu=ADDR["x"] + 64),
])
def test_glu_refuses(moeq, bad):
    assert moeq.lib().moeq_glu(glu(moeq, **bad), None) == moeq.INVALID_ARGUMENT


@pytest.mark.parametrize("bad", GLU_BAD + [
    dict(dh=0), dict(lddh=31), dict(dh=ADDR["dh"] + 1), dict(dw0=0), dict(dw1=0), dict(dx=0, dw0=0, dw1=0),
    dict(lddx=63), dict(lddw0=63), dict(lddw1=63), dict(dx=ADDR["dx"] + 1), dict(dw1=ADDR["dw1"] + 1),
    dict(dx=ADDR["x"]), dict(dx=ADDR["dh"]), dict(dw0=ADDR["w0"]), dict(dw1=ADDR["dw0"]), dict(dx=ADDR["dw1"] + 128),
    dict(ws=0), dict(wsb=0), dict(wsb=-1), dict(ws=ADDR["ws"] + 128), dict(ws=ADDR["x"]), dict(ws=ADDR["dx"]),
    dict(gu=ADDR["dx"]), dict(gu=ADDR["ws"] + 256),
])
def test_glu_backward_refuses(moeq, bad):
    assert moeq.lib().moeq_glu_backward(glu(moeq, **bad), None) == moeq.INVALID_ARGUMENT


def test_workspace_queries(moeq):
    lib = moeq.lib()
    n = lib.moeq_glu_workspace(glu(moeq, ws=0, wsb=0), 1)
    assert n >= 2 * 4 * 32 * 2 and n % 256 == 0
    # one byte less than the query's answer is refused
    assert lib.moeq_glu_backward(glu(moeq, wsb=n - 1), None) == moeq.INVALID_ARGUMENT
    assert lib.moeq_glu_workspace(glu(moeq), 2) == -1
    assert lib.moeq_glu_workspace(glu(moeq, H=0), 0) == -1
    assert lib.moeq_glu_workspace(None, 0) == -1
    assert lib.moeq_i8_workspace(None, 1) == -1
    # aligned operands need none in the forward calls
    assert lib.moeq_glu_workspace(glu(moeq), 0) == 0
    assert lib.moeq_i8_workspace(i8(moeq, 2), 2) == 0


def test_the_binding_refuses_cpu_tensors(moeq):
    import torch
    x = torch.zeros(2, 4)
    w = torch.zeros(3, 4)
    for call in (lambda: moeq.quant_i8(x), lambda: moeq.glu(x, w, w), lambda: moeq.glu_backward(x, x, w, w),
                 lambda: moeq.matmul_i8(x, x, w, w), lambda: moeq.glu_i8(x, x, w, w, w, w)):
        with pytest.raises(moeq.MoeqError):
            call()
