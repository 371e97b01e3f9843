"""The dense operators beside the routed layer, as measured work: the matrix
product in 8-bit integers with a scale per token and per channel (alone and as
the gated block of two projections), and the gated feed-forward block
h = silu(x Wg^T) * (x Wu^T) in bf16 and f32 with its backward pass.

Each case is one pass through an operator.  With ``own`` false it runs in
elementary torch operations in 32 bits, with ``own`` true through the package's
entry points.  Shapes: x [T][hidden], Wg and Wu [inter][hidden], h [T][inter];
for the product, x [T][hidden], W [inter][hidden], out [T][inter].

Quantised rows: scale = max|x| / 127, q = round-half-even(127 x / max|x|).
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # int8 product.  One token through a square projection: a decode step
        # of a single request, the weights read once, latency counts.
        dict(name="i8_decode_1", op="i8", T=1, hidden=4096, inter=4096, x="bf16", out="bf16", pad=0),
        # Eight requests' tokens, already quantised, through the block's
        # second projection (inter -> hidden of the expert shape).
        dict(name="i8_decode_8", op="i8", T=8, hidden=2048, inter=4096, x="i8", out="bf16", pad=0),
        # A long prompt in one call, quantised on the way.
        dict(name="i8_prompt", op="i8", T=4096, hidden=4096, inter=4096, x="bf16", out="bf16", pad=0),
        # Odd sizes and row strides, f32 activations and results: a projection
        # whose width no tile divides, cut out of a wider buffer.
        dict(name="i8_ragged_f32", op="i8", T=777, hidden=1111, inter=1003, x="f32", out="f32", pad=5),
        # Gated block in int8, eight requests' tokens (quantised before, as
        # several projections share them).
        dict(name="glu_i8_decode_8", op="glu_i8", T=8, hidden=4096, inter=2048, x="i8", out="bf16", pad=0),
        # The same block over a prompt micro-batch of 2048.
        dict(name="glu_i8_prompt", op="glu_i8", T=2048, hidden=4096, inter=2048, x="bf16", out="bf16", pad=0),
        # Gated block in bf16: one token, the smallest call of a decode step.
        dict(name="glu_decode_1", op="glu", T=1, hidden=4096, inter=2048, x="bf16", save=False, pad=0),
        # A batch of 64 requests' decode tokens.
        dict(name="glu_batch_64", op="glu", T=64, hidden=4096, inter=2048, x="bf16", save=False, pad=0),
        # A training forward pass (or a prompt) of 2048 tokens that keeps both
        # projections for the backward pass.
        dict(name="glu_forward_2048", op="glu", T=2048, hidden=4096, inter=2048, x="bf16", save=True, pad=0),
        # A training step's backward pass over 8192 tokens with the kept
        # projections: all three gradients.
        dict(name="glu_backward_8192", op="glu_bwd", T=8192, hidden=4096, inter=2048, x="bf16", save=True, pad=0),
        # Backward pass with nothing kept (the projections are computed
        # again), at odd sizes and strides.
        dict(name="glu_backward_ragged", op="glu_bwd", T=1001, hidden=1000, inter=517, x="bf16", save=False, pad=3),
        # f32: a small model's forward and backward pass together.
        dict(name="glu_step_f32", op="glu_step", T=333, hidden=520, inter=260, x="f32", save=True, pad=0),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; every second one a multiple of 64 (where that is in range)."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5 and n >= 64:
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["i8", "i8", "glu_i8", "glu", "glu", "glu_bwd", "glu_step"])
    pad = rng.choice([0, 0, 0, 3, 8, 16])
    if op == "glu_step":     # f32: the small model's sizes
        return dict(op=op, T=_size(rng, 1, 512), hidden=_size(rng, 32, 1024), inter=_size(rng, 32, 512), x="f32",
                    save=rng.random() < 0.5, pad=pad)
    T = _size(rng, 1, 8192)
    hidden, inter = _size(rng, 64, 4096), _size(rng, 64, 4096 if op == "i8" else 2048)
    if op in ("i8", "glu_i8"):
        return dict(op=op, T=min(T, 4096), hidden=hidden, inter=inter, x=rng.choice(["bf16", "i8", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]), pad=pad)
    return dict(op=op, T=T, hidden=hidden, inter=inter, x="bf16", save=rng.random() < 0.5, pad=pad)


def _quant(x):
    """Rows to int8: exact for bf16 (15-bit products, and a quotient of them by 8 bits lies far from a half unless it
    is one); in 64 bits for f32, where a quotient may lie next to a half."""
    wide = x.float() if x.dtype == torch.bfloat16 else x.double()
    amax = wide.abs().amax(dim=1, keepdim=True)
    q = torch.round(wide * 127.0 / amax.clamp_min(1e-300 if wide.dtype == torch.float64 else 1e-45))
    return q.to(torch.int8), (amax.float() / 127.0).squeeze(1)


def _rows(n, k, pad, gen, scale, dtype):
    """A [n][k] matrix with `pad` more columns between its rows, some columns wider than the rest."""
    a = torch.randn((n, k + pad), generator=gen, device="cuda", dtype=torch.float32) * scale
    return a.to(dtype)[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, H, N, pad = case["T"], case["hidden"], case["inter"], case["pad"]
    st = {"case": case}
    x = _rows(T, H, pad, gen, 1.0, torch.float32)
    # activations have a few channels far wider than the others
    wide = torch.randperm(H, generator=gen, device="cuda")[: max(1, H // 128)]
    x[:, wide] *= 6.0
    if case["op"] in ("i8", "glu_i8"):
        for k in ("w",) if case["op"] == "i8" else ("wg", "wu"):
            q, s = _quant(_rows(N, H, 0, gen, 0.02, torch.float32))
            buf = torch.zeros((N, H + pad), dtype=torch.int8, device="cuda")
            buf[:, :H] = q
            st[k], st["s" + k] = buf[:, :H], s
        if case["x"] == "i8":
            q, s = _quant(x)
            buf = torch.zeros((T, H + pad), dtype=torch.int8, device="cuda")
            buf[:, :H] = q
            st["x"], st["sx"] = buf[:, :H], s
        else:
            buf = torch.zeros((T, H + pad), dtype=DT[case["x"]], device="cuda")
            buf[:, :H] = x
            st["x"] = buf[:, :H]
        return st
    dt = DT[case["x"]]
    buf = torch.zeros((T, H + pad), dtype=dt, device="cuda")
    buf[:, :H] = x
    st["x"] = buf[:, :H]
    # both projections in one buffer, as checkpoints often hold them
    both = _rows(2 * N, H, pad, gen, 0.02, dt)
    st["wg"], st["wu"] = both[:N], both[N:]
    if case["op"] != "glu":
        st["dh"] = _rows(T, N, pad, gen, 0.1, dt)
        if case["op"] == "glu_bwd" and case["save"]:
            xf = st["x"].float()
            st["gu"] = torch.stack([xf @ st["wg"].float().t(), xf @ st["wu"].float().t()]).to(dt)
    return st


def _int_product(q, w):
    """The product of int8 matrices, exact: stretches of 1024 products (each at most 2^14) sum exactly in f32."""
    k = q.shape[1]
    acc = torch.zeros((q.shape[0], w.shape[0]), dtype=torch.int32, device=q.device)
    for i in range(0, k, 1024):
        acc += (q[:, i:i + 1024].float() @ w[:, i:i + 1024].float().t()).to(torch.int32)
    return acc.float()


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_backward(dh, x, wg, wu, g, u, dt):
    s = 1.0 / (1.0 + torch.exp(-g))
    dhf = dh.float()
    dg, du = dhf * u * (s * (1.0 + g * (1.0 - s))), dhf * (g * s)
    xf = x.float()
    return ((dg @ wg.float() + du @ wu.float()).to(dt), (dg.t() @ xf).to(dt), (du.t() @ xf).to(dt))


def run(state):
    c = state["case"]
    op, x = c["op"], state["x"]
    if own:
        from bit_quantized_moe_routed_b200 import moeq
        if op in ("i8", "glu_i8"):
            q, sx = (x, state["sx"]) if c["x"] == "i8" else moeq.quant_i8(x)
            if op == "i8":
                return moeq.matmul_i8(q, sx, state["w"], state["sw"], dtype=c["out"])
            return moeq.glu_i8(q, sx, state["wg"], state["swg"], state["wu"], state["swu"], dtype=c["out"])
        if op == "glu":
            return moeq.glu(x, state["wg"], state["wu"], save=c["save"])
        if op == "glu_bwd":
            return moeq.glu_backward(state["dh"], x, state["wg"], state["wu"], gu=state.get("gu"))
        if c["save"]:
            h, gu = moeq.glu(x, state["wg"], state["wu"], save=True)
        else:
            h, gu = moeq.glu(x, state["wg"], state["wu"]), None
        return (h,) + tuple(moeq.glu_backward(state["dh"], x, state["wg"], state["wu"], gu=gu))
    if op in ("i8", "glu_i8"):
        q, sx = (x, state["sx"]) if c["x"] == "i8" else _quant(x)
        if op == "i8":
            return (_int_product(q, state["w"]) * sx[:, None] * state["sw"]).to(DT[c["out"]])
        g = _int_product(q, state["wg"]) * sx[:, None] * state["swg"]
        u = _int_product(q, state["wu"]) * sx[:, None] * state["swu"]
        return (_silu(g) * u).to(DT[c["out"]])
    dt, wg, wu = x.dtype, state["wg"], state["wu"]
    if "gu" in state:
        g, u = state["gu"][0].float(), state["gu"][1].float()
    else:
        xf = x.float()
        g, u = xf @ wg.float().t(), xf @ wu.float().t()
    if op == "glu_bwd":
        return _plain_backward(state["dh"], x, wg, wu, g, u, dt)
    h = (_silu(g) * u).to(dt)
    if op == "glu":
        return (h, torch.stack([g, u]).to(dt)) if c["save"] else h
    return (h,) + _plain_backward(state["dh"], x, wg, wu, g, u, dt)


def work(case):
    T, H, N = case["T"], case["hidden"], case["inter"]
    size = {"i8": 1, "bf16": 2, "f32": 4}
    xb = size[case["x"]]
    if case["op"] == "i8":
        return {"bytes": T * H * xb + N * H + 4 * N + T * N * size[case["out"]], "flops": 2 * T * H * N}
    if case["op"] == "glu_i8":
        return {"bytes": T * H * xb + 2 * N * H + 8 * N + T * N * size[case["out"]], "flops": 4 * T * H * N}
    w, x, h = 2 * N * H * xb, T * H * xb, T * N * xb
    kept = 2 * h if case["save"] else 0
    if case["op"] == "glu":
        return {"bytes": x + w + h + kept, "flops": 4 * T * H * N}
    grads = x + w     # dx and both weights' gradients
    if case["op"] == "glu_bwd":
        return {"bytes": h + x + w + kept + grads, "flops": (8 if case["save"] else 12) * T * H * N}
    return {"bytes": x + w + h + h + grads, "flops": 12 * T * H * N}


def _exact_quant(x):
    v = x.to(torch.float64)
    top = torch.max(torch.abs(v), dim=1).values
    safe = torch.where(top > 0, top, torch.ones_like(top))
    return torch.round(v * 127.0 / safe[:, None]), top / 127.0


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    op = case["op"]
    if op in ("i8", "glu_i8"):
        q, sx = (st["x"].to(d), st["sx"].to(d)) if case["x"] == "i8" else _exact_quant(st["x"])
        outs = [torch.einsum("tk,nk->tn", q, st[k].to(d)) * torch.outer(sx, st["s" + k].to(d))
                for k in (("w",) if op == "i8" else ("wg", "wu"))]
        return outs[0] if op == "i8" else outs[0] * torch.sigmoid(outs[0]) * outs[1]
    x, wg, wu = st["x"].to(d), st["wg"].to(d), st["wu"].to(d)
    if "gu" in st:
        g, u = st["gu"].to(d).unbind(0)
    else:
        g, u = torch.einsum("tk,nk->tn", x, wg), torch.einsum("tk,nk->tn", x, wu)
    sg = torch.sigmoid(g)
    h = g * sg * u
    if op == "glu":
        return (h, torch.stack([g, u])) if case["save"] else h
    dh = st["dh"].to(d)
    dg, du = dh * u * (sg + g * sg * (1 - sg)), dh * g * sg
    grads = (torch.einsum("tn,nk->tk", dg, wg) + torch.einsum("tn,nk->tk", du, wu),
             torch.einsum("tn,tk->nk", dg, x), torch.einsum("tn,tk->nk", du, x))
    return grads if op == "glu_bwd" else (h,) + grads
