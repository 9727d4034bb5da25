"""The row-norm and gradient operators as they are measured: cases, inputs, plain forms.

Four operators: the root-mean-square norm with the residual's addition (``rms_fwd``), its
backward pass (``rms_bwd``), the same norm with an output in 8 bits and scales
(``rms_q8``), and the global gradient norm with clipping (``grads``).

``run`` computes the plain form with elementary torch operations in 32 bits, or, where
``own`` is true, makes the calls a user makes of this repository's package.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
MAX_ELEMENTS = 8192 * 4096      # rows * columns of the largest row-norm case


def listed():
    return [
        # One token of a decoding step: latency alone.
        {"name": "fwd_1x4096_bf16", "op": "rms_fwd", "T": 1, "H": 4096, "x": "bf16", "res": "bf16", "w": "bf16",
         "y": "bf16"},
        # A training or prefill batch of one block.
        {"name": "fwd_8192x4096_bf16", "op": "rms_fwd", "T": 8192, "H": 4096, "x": "bf16", "res": "bf16", "w": "bf16",
         "y": "bf16"},
        # The norm over each head's query or key vector: very many short rows, no residual.
        {"name": "fwd_131072x128_bf16", "op": "rms_fwd", "T": 131072, "H": 128, "x": "bf16", "res": "none", "w": "fp32",
         "y": "bf16"},
        # An odd width and an odd batch, with the residual stream kept in fp32.
        {"name": "fwd_2047x1531_fp16", "op": "rms_fwd", "T": 2047, "H": 1531, "x": "fp16", "res": "fp32", "w": "fp32",
         "y": "fp16"},
        # The backward pass of a block's norm: the residual stream's gradient joins here.
        {"name": "bwd_8192x4096_bf16", "op": "rms_bwd", "T": 8192, "H": 4096, "x": "bf16", "res": "bf16", "w": "bf16",
         "y": "bf16"},
        # The backward pass over heads: short rows, the weight's gradient sums 131072 of them.
        {"name": "bwd_131072x128_bf16", "op": "rms_bwd", "T": 131072, "H": 128, "x": "bf16", "res": "none", "w": "fp32",
         "y": "bf16"},
        # A small, odd fp32 model in full precision.
        {"name": "bwd_509x1001_fp32", "op": "rms_bwd", "T": 509, "H": 1001, "x": "fp32", "res": "fp32", "w": "fp32",
         "y": "fp32"},
        # Serving with 8-bit products: a prefill batch, a scale for each token.
        {"name": "q8_4096x8192_int8", "op": "rms_q8", "T": 4096, "H": 8192, "x": "bf16", "res": "bf16", "w": "bf16",
         "q": "int8", "block": 0},
        # The same with e4m3 and a scale for each 128 columns, on an ordinary batch.
        {"name": "q8_1024x5120_e4m3_b128", "op": "rms_q8", "T": 1024, "H": 5120, "x": "bf16", "res": "bf16",
         "w": "bf16", "q": "e4m3", "block": 128},
        # A decoding step of 16 sequences.
        {"name": "q8_16x4096_int8", "op": "rms_q8", "T": 16, "H": 4096, "x": "fp16", "res": "fp16", "w": "fp16",
         "q": "int8", "block": 0},
        # Gradients of a 24-block model in bf16 (packed one behind the other in a bucket), clipped
        # into the fp32 copies that the optimizer reads.
        {"name": "clip_blocks_bf16_to_fp32", "op": "grads", "kind": "blocks", "width": 1024, "depth": 24, "g": "bf16",
         "out": "fp32"},
        # The gradients of a 3D UNet (convolutions and norm vectors of five levels) in full precision.
        {"name": "clip_unet_fp32", "op": "grads", "kind": "unet", "width": 32, "depth": 5, "g": "fp32", "out": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_fwd", "rms_bwd", "rms_bwd", "rms_q8", "rms_q8", "grads"])
    if op == "grads":
        kind = rng.choice(["blocks", "unet", "ragged"])
        g = rng.choice(["bf16", "fp16", "fp32"])
        out = rng.choice(["none", "fp32", g])
        if kind == "blocks":
            width, depth = _log_int(rng, 64, 1024), rng.randint(1, 24)
        elif kind == "unet":
            width, depth = rng.randint(8, 40), rng.randint(2, 5)
        else:
            width, depth = _log_int(rng, 10, 100_000), rng.randint(1, 400)
        return {"op": op, "kind": kind, "width": width, "depth": depth, "g": g, "out": out}
    H = _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        H = max(64, H // 64 * 64)   # most widths are whole multiples of a head
    T = _log_int(rng, 1, min(131072, MAX_ELEMENTS // H))
    if op == "rms_q8":
        x = rng.choice(["bf16", "fp16"])
        return {"op": op, "T": T, "H": H, "x": x, "res": rng.choice(["none", x, "fp32"]), "w": rng.choice([x, "fp32"]),
                "q": rng.choice(["int8", "e4m3"]), "block": rng.choice([0, 32, 64, 128])}
    x = rng.choice(["bf16", "fp16", "fp32"])
    return {"op": op, "T": T, "H": H, "x": x, "res": rng.choice(["none", x, "fp32"]), "w": rng.choice([x, "fp32"]),
            "y": rng.choice([x, x, "fp32"])}


def _sizes(case):
    """Elements of each gradient tensor of a grads case."""
    width, depth = case["width"], case["depth"]
    if case["kind"] == "blocks":
        block = [width, 4 * width * width, width, 4 * width * width, 4 * width * width, 4 * width * width]
        return [16 * width * width] + block * depth + [width]
    if case["kind"] == "unet":
        out, cin = [], 4
        for level in range(depth):
            c = width << level
            out += [27 * cin * c, c, c, 27 * c * c, c, c]
            cin = c
        for level in range(depth - 2, -1, -1):
            c = width << level
            out += [8 * 2 * c * c, 27 * 2 * c * c, c, c, 27 * c * c, c, c]
        return out
    return [1 + (width * (7 + (i * i * 31) % 97)) // 97 for i in range(depth)]


def _elements(case):
    return sum(_sizes(case)) if case["op"] == "grads" else case["T"] * case["H"]


def _rows(gen, T, H, dtype, offset=0.0):
    """A residual stream's values: unit spread, a few channels far larger than the rest."""
    scale = torch.exp(0.3 * torch.randn(H, generator=gen, device="cuda"))
    scale[torch.randint(0, H, (max(1, H // 256),), generator=gen, device="cuda")] *= 12.0
    v = torch.randn(T, H, generator=gen, device="cuda")
    return v.mul_(scale).add_(offset).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "grads":
        sizes = _sizes(case)
        total = sum(sizes)
        g, out = DTYPES[case["g"]], case["out"]
        spread = torch.exp(torch.randn(len(sizes), generator=gen, device="cuda") - 6.0)
        flat = torch.randn(total, generator=gen, device="cuda")
        flat.mul_(torch.repeat_interleave(spread, torch.tensor(sizes, device="cuda"), output_size=total))
        flat = flat.to(g)
        state = {"case": case, "flat": flat, "grads": list(flat.split(sizes)), "max_norm": 1e-3 * math.sqrt(total)}
        if out != "none":
            state["out_flat"] = torch.zeros(total, dtype=DTYPES[out], device="cuda")
            state["out"] = list(state["out_flat"].split(sizes))
        return state
    T, H = case["T"], case["H"]
    xdt, res = DTYPES[case["x"]], case["res"]
    w = (1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(DTYPES[case["w"]])
    state = {"case": case, "w": w}
    if case["op"] == "rms_bwd":
        hdt = xdt if res == "none" else DTYPES[res]
        state["h"] = _rows(gen, T, H, hdt, 0.02)
        state["rstd"] = (state["h"].double().square().mean(-1) + EPS).rsqrt().float()
        state["dy"] = (1e-2 * torch.randn(T, H, generator=gen, device="cuda")).to(DTYPES[case["y"]])
        if res != "none":
            state["dh"] = (1e-2 * torch.randn(T, H, generator=gen, device="cuda")).to(hdt)
        return state
    state["x"] = _rows(gen, T, H, xdt)
    if res != "none":
        state["r"] = _rows(gen, T, H, DTYPES[res], 0.02)
    return state


# ------------------------------------------------------------------ plain forms

def _plain_norm(state):
    """(h as stored, or None without a residual; h, rstd and y in 32 bits)."""
    x, r = state["x"], state.get("r")
    h = None if r is None else (x.float() + r.float()).to(r.dtype)
    hf = x.float() if h is None else h.float()
    rstd = (hf.square().mean(-1) + EPS).rsqrt()
    return h, rstd, hf * rstd[:, None] * state["w"].float()


def _plain_fwd(state):
    h, rstd, y = _plain_norm(state)
    y = y.to(DTYPES[state["case"]["y"]])
    return (y, rstd) if h is None else (y, rstd, h)


def _plain_bwd(state):
    case, rstd = state["case"], state["rstd"][:, None]
    dy = state["dy"].float()
    xhat = state["h"].float() * rstd
    g = dy * state["w"].float()
    dh = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if "dh" in state:
        dh = dh + state["dh"].float()
    dw = (dy * xhat).sum(0).to(state["w"].dtype)
    out = (dh.to(DTYPES[case["x"]]), dw)
    return out + (dh.to(state["h"].dtype),) if state["h"].dtype != DTYPES[case["x"]] else out


def _plain_q8(state):
    case = state["case"]
    h, rstd, y = _plain_norm(state)
    T, H = y.shape
    B = case["block"] or H
    qmax = 127.0 if case["q"] == "int8" else 448.0
    nb = -(-H // B)
    y = torch.nn.functional.pad(y, (0, nb * B - H)).view(T, nb, B)
    scale = (y.abs().amax(-1) / qmax).clamp(min=2.0 ** -126)
    q = y / scale[..., None]
    q = torch.round(q).clamp(-127, 127).to(torch.int8) if case["q"] == "int8" else q.to(torch.float8_e4m3fn)
    values = (q.float() * scale[..., None]).view(T, nb * B)[:, :H].contiguous().to(DTYPES[case["x"]])
    return (values, scale) if h is None else (values, scale, h)


def _plain_grads(state):
    # Over the whole bucket at once, which is what its tensors together hold.
    g = state["flat"].float()
    norm = g.square().sum(dtype=torch.float64).sqrt()
    if "out" not in state:
        return [norm.float()]
    coef = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    state["out_flat"].copy_(g * coef)
    return [norm.float(), state["out_flat"]]


# ------------------------------------------------------------------ the framework's calls

def _own(state):
    import unet_groupnorm_amd as gn
    case = state["case"]
    op = case["op"]
    if op == "rms_fwd":
        y, h, rstd = gn.gn_rms_forward(state["x"], state["w"], EPS, residual=state.get("r"),
                                       out_dtype=DTYPES[case["y"]])
        return (y, rstd, h) if "r" in state else (y, rstd)
    if op == "rms_bwd":
        dx, dw, dres = gn.gn_rms_backward(state["dy"], state["h"], state["rstd"], state["w"], dh=state.get("dh"),
                                          x_dtype=DTYPES[case["x"]])
        return (dx, dw, dres) if state["h"].dtype != DTYPES[case["x"]] else (dx, dw)
    if op == "rms_q8":
        q, scale, h, _ = gn.gn_rms_forward_q8(state["x"], state["w"], EPS, residual=state.get("r"),
                                              q_dtype=torch.int8 if case["q"] == "int8" else torch.float8_e4m3fn,
                                              block=case["block"])
        values = gn.gn_q8_dequantize(q, scale, DTYPES[case["x"]], block=case["block"])
        return (values, scale, h) if "r" in state else (values, scale)
    if "out" not in state:
        return [gn.gn_grad_norm(state["grads"])]
    return [gn.gn_grad_clip(state["grads"], state["max_norm"], out=state["out"]), state["out_flat"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rms_fwd":
        return _plain_fwd(state)
    if op == "rms_bwd":
        return _plain_bwd(state)
    return _plain_q8(state) if op == "rms_q8" else _plain_grads(state)


# ------------------------------------------------------------------ 64 bits

def _e4m3(v):
    """Nearest e4m3 value, ties to even, of |v| <= 448."""
    e = torch.frexp(v)[1].clamp(min=-5).double() - 4.0   # v = m * 2^(e + 4), |m| in [0.5, 1)
    step = torch.exp2(e)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grads":
        g = s["flat"].to(torch.float64)
        norm = torch.linalg.vector_norm(g)
        if case["out"] == "none":
            return [norm]
        return [norm, g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))]
    w = s["w"].to(torch.float64)
    H = case["H"]
    if case["op"] == "rms_bwd":
        h, dy = s["h"].to(torch.float64), s["dy"].to(torch.float64)
        rs = s["rstd"].to(torch.float64).unsqueeze(1)
        dot = torch.sum(dy * w * h, dim=1, keepdim=True)
        dh = rs * dy * w - rs ** 3 * h * dot / H
        if "dh" in s:
            dh = dh + s["dh"].to(torch.float64)
        dw = torch.sum(dy * h * rs, dim=0)
        return (dh, dw, dh) if s["h"].dtype != DTYPES[case["x"]] else (dh, dw)
    h = s["x"].to(torch.float64)
    if "r" in s:
        h = (h + s["r"].to(torch.float64)).to(s["r"].dtype).to(torch.float64)   # h is what is stored
    rs = 1.0 / torch.sqrt(torch.sum(h * h, dim=1) / H + EPS)
    y = torch.einsum("th,t,h->th", h, rs, w) if h.numel() < 1 << 16 else h * (rs.unsqueeze(1) * w)
    if case["op"] == "rms_fwd":
        return (y, rs, h) if "r" in s else (y, rs)
    B, qmax = case["block"] or H, 127.0 if case["q"] == "int8" else 448.0
    values, scales = torch.empty_like(y), []
    for c in range(0, H, B):
        part = y[:, c:c + B]
        sc = torch.clamp(part.abs().max(dim=1).values / qmax, min=2.0 ** -126)
        u = part / sc.unsqueeze(1)
        values[:, c:c + B] = (torch.round(u) if case["q"] == "int8" else _e4m3(u)) * sc.unsqueeze(1)
        scales.append(sc)
    scale = torch.stack(scales, dim=1)
    return (values, scale, h) if "r" in s else (values, scale)


def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2, "none": 0}
    n = _elements(case)
    if case["op"] == "grads":
        # Each gradient counted once, though the norm has to be known before the first is scaled.
        return {"bytes": n * (size[case["g"]] + size[case["out"]]), "flops": n * (2 if case["out"] == "none" else 3)}
    T, H, x, res = case["T"], case["H"], size[case["x"]], size[case["res"]]
    vec = H * size[case["w"]]
    if case["op"] == "rms_fwd":
        return {"bytes": n * (x + 2 * res + size[case["y"]]) + vec + 4 * T, "flops": 6 * n}
    if case["op"] == "rms_bwd":
        h = res or x
        both = res and res != x
        return {"bytes": n * (size[case["y"]] + h + res + x + (res if both else 0)) + 2 * vec + 4 * T, "flops": 12 * n}
    scales = T * (-(-H // case["block"]) if case["block"] else 1)
    return {"bytes": n * (x + 2 * res + x) + vec + 4 * scales, "flops": 9 * n}
