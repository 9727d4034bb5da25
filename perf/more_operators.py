"""The residual join and the 8-bit activation checkpoints as they are measured: cases, inputs, plain forms.

Three operators: the join of a block's output into the residual stream with the norms after
the block and before the next one, the gate and the scales (``join_fwd``; with a checkpoint
it also leaves what its backward pass reads in 8 bits), the join's backward pass
(``join_bwd``, from the saved tensors or from their checkpoints), and the checkpoint of an
activation by itself with its reading back (``q8``).

``run`` computes the plain form with elementary torch operations in 32 bits, or, where
``own`` is true, makes the calls a user makes of this repository's package.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8,
          "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}
READ_BACK = torch.bfloat16      # the type in which checkpoints are read back, whatever was kept
EPS = 1e-6
MAX_ELEMENTS = 8192 * 4096      # rows * columns of the largest join
MAX_Q8 = 4096 * 16384           # and of the largest checkpoint by itself


def _join(name, op, T, H, x, res, w, samples, post, gate, scale, rs=1.0, bs=1.0, ckpt="none", block=0):
    case = {"op": op, "T": T, "H": H, "x": x, "res": res, "w": w, "samples": samples, "post": post, "gate": gate,
            "scale": scale, "rs": rs, "bs": bs, "ckpt": ckpt, "block": block}
    return {"name": name, **case} if name else case


def listed():
    return [
        # One token of a decoding step of a model with norms on both sides of its blocks: latency alone.
        _join("fwd_1x4096_bf16", "join_fwd", 1, 4096, "bf16", "bf16", "bf16", 1, True, False, False),
        # A training or prefill batch of one block, with a learned gate for each channel.
        _join("fwd_8192x4096_bf16", "join_fwd", 8192, 4096, "bf16", "bf16", "bf16", 1, True, True, False),
        # A diffusion transformer's block on 16 images of 256 patches: gates and scales of each image.
        _join("fwd_16x256x1152_bf16_adaptive", "join_fwd", 4096, 1152, "bf16", "bf16", "bf16", 16, True, True, True),
        # An odd width and an odd batch, the stream in fp32 and scaled, no norm after the block.
        _join("fwd_2047x1531_fp16_fp32_stream", "join_fwd", 2047, 1531, "fp16", "fp32", "fp32", 1, False, True, False,
              rs=0.9375, bs=0.35),
        # The training batch again, leaving what the backward pass reads in 8 bits.
        _join("fwd_8192x4096_bf16_int8_b128", "join_fwd", 8192, 4096, "bf16", "bf16", "bf16", 1, True, True, False,
              ckpt="int8", block=128),
        # The backward passes of the same blocks: the training batch,
        _join("bwd_8192x4096_bf16", "join_bwd", 8192, 4096, "bf16", "bf16", "bf16", 1, True, True, False),
        # the 16 images, with gradients of every image's gate and scale,
        _join("bwd_16x256x1152_bf16_adaptive", "join_bwd", 4096, 1152, "bf16", "bf16", "bf16", 16, True, True, True),
        # a small, odd model in full precision with three sequences,
        _join("bwd_3x171x1001_fp32", "join_bwd", 513, 1001, "fp32", "fp32", "fp32", 3, True, True, False, bs=0.5),
        # the training batch from its 8-bit checkpoints,
        _join("bwd_8192x4096_bf16_int8_b128", "join_bwd", 8192, 4096, "bf16", "bf16", "bf16", 1, True, True, False,
              ckpt="int8", block=128),
        # and an ordinary batch from e4m3 with a scale a row, the stream in fp32.
        _join("bwd_1024x5120_fp16_fp32_stream_e4m3", "join_bwd", 1024, 5120, "fp16", "fp32", "fp16", 1, True, False,
              False, ckpt="e4m3", block=0),
        # A 128^3 activation of 32 channels of a 3D UNet (rows of one plane), kept for the backward pass and read back.
        {"name": "q8_unet_128cube_c32_int8_b128", "op": "q8", "T": 4096, "H": 16384, "x": "bf16", "q": "int8",
         "block": 128},
        # The patches of a small odd volume (37 * 41 voxels a plane).
        {"name": "q8_120x1517_fp32_e4m3_b32", "op": "q8", "T": 120, "H": 1517, "x": "fp32", "q": "e4m3", "block": 32},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["join_fwd", "join_fwd", "join_bwd", "join_bwd", "q8"])
    if op == "q8":
        H = _log_int(rng, 32, 32768)
        if rng.random() < 0.6:
            H = max(32, H // 32 * 32)
        return {"op": op, "T": _log_int(rng, 1, max(1, min(262144, MAX_Q8 // H))), "H": H,
                "x": rng.choice(["bf16", "fp16", "fp32"]), "q": rng.choice(["int8", "e4m3"]),
                "block": rng.choice([0, 32, 64, 128])}
    H = _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        H = max(64, H // 64 * 64)   # most widths are whole multiples of a head
    T = _log_int(rng, 1, min(65536, MAX_ELEMENTS // 2 // H))
    # One vector for all rows, or one for each of a few sequences.
    if rng.random() < 0.5:
        samples = _log_int(rng, 1, min(64, T))
        T = T // samples * samples
    else:
        samples = 1
    x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    gate, scale = rng.choice([(False, False), (True, False), (True, True), (False, True)])
    ckpt = rng.choice(["none", "none", "int8", "e4m3"])
    return _join("", op, T, H, x, rng.choice([x, "fp32"]), rng.choice([x, "fp32"]),
                 samples if gate or scale else 1, rng.random() < 0.7, gate, scale, rng.choice([1.0, 1.0, 0.75]),
                 rng.choice([1.0, 1.0, 0.125]), ckpt, rng.choice([0, 32, 64, 128]) if ckpt != "none" else 0)


def _rows(gen, T, H, dtype, offset=0.0):
    """A residual stream's values: unit spread, a few channels far larger than the rest."""
    spread = torch.exp(0.3 * torch.randn(H, generator=gen, device="cuda"))
    spread[torch.randint(0, H, (max(1, H // 256),), generator=gen, device="cuda")] *= 12.0
    v = torch.randn(T, H, generator=gen, device="cuda")
    return v.mul_(spread).add_(offset).to(dtype)


def _saves_x(case):
    """Whether the backward pass reads the block's output."""
    return case["post"] or case["gate"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, H, xdt = case["T"], case["H"], DTYPES[case["x"]]
    if case["op"] == "q8":
        return {"case": case, "x": _rows(gen, T, H, xdt, 0.1)}
    rdt, wdt, S = DTYPES[case["res"]], DTYPES[case["w"]], case["samples"]

    def vector(n, spread, offset):
        return (offset + spread * torch.randn(n, H, generator=gen, device="cuda")).to(wdt)

    state = {"case": case, "w": vector(1, 0.2, 1.0)[0]}
    if case["post"]:
        state["pw"] = vector(1, 0.2, 0.8)[0]
    if case["gate"]:
        state["gate"] = vector(S, 0.4, 0.1)
    if case["scale"]:
        state["scale"] = vector(S, 0.2, 0.0)
    x = _rows(gen, T, H, xdt, 0.05)
    h = _rows(gen, T, H, rdt, 0.02)     # the stream: before the join (forward), behind it (backward)
    if case["op"] == "join_fwd":
        state["x"], state["r"] = x, h
        return state
    state["rstd"] = (h.double().square().mean(-1) + EPS).rsqrt().float()
    if case["post"]:
        state["prstd"] = (x.double().square().mean(-1) + EPS).rsqrt().float()
    if case["ckpt"] == "none":
        state["h"] = h
        if _saves_x(case):
            state["x"] = x
    else:
        state["hq"] = _quantize(h.float(), case["ckpt"], case["block"])
        if _saves_x(case):
            state["xq"] = _quantize(x.float(), case["ckpt"], case["block"])
    state["dy"] = (1e-2 * torch.randn(T, H, generator=gen, device="cuda")).to(xdt)
    state["dh"] = (1e-2 * torch.randn(T, H, generator=gen, device="cuda")).to(rdt)
    return state


# ------------------------------------------------------------------ plain forms

def _quantize(v, kind, block):
    """(q, scale) of fp32 rows."""
    T, H = v.shape
    B = block or H
    nb = -(-H // B)
    v = torch.nn.functional.pad(v, (0, nb * B - H)).view(T, nb, B)
    scale = (v.abs().amax(-1) / QMAX[kind]).clamp(min=2.0 ** -126)
    q = v / scale[..., None]
    q = torch.round(q).clamp(-127, 127).to(torch.int8) if kind == "int8" else q.to(torch.float8_e4m3fn)
    return q.view(T, nb * B)[:, :H].contiguous(), scale


def _values(q, scale, block):
    """What (q, scale) stand for, in fp32."""
    T, H = q.shape
    return q.float() * (scale if not block else scale.repeat_interleave(block, dim=1)[:, :H])


def _by_sample(v, case):
    return v.float().view(case["samples"], -1, case["H"])


def _coefficient(state):
    """branch_scale * gate * post_weight for each sample (or a number)."""
    case, c = state["case"], state["case"]["bs"]
    if case["gate"]:
        c = state["gate"].float()[:, None] * c
    return c * state["pw"].float() if case["post"] else c


def _multiplier(state):
    """weight * (1 + scale) for each sample."""
    m = state["w"].float()
    return m * (1.0 + state["scale"].float()[:, None]) if state["case"]["scale"] else m


def _plain_fwd(state):
    case = state["case"]
    T, H = state["x"].shape
    u, out = state["x"].float(), []
    if case["post"]:
        prstd = (u.square().mean(-1) + EPS).rsqrt()
        u = u * prstd[:, None]
    u = (u.view(case["samples"], -1, H) * _coefficient(state)).view(T, H)
    h = (case["rs"] * state["r"].float() + u).to(state["r"].dtype)
    hf = h.float()
    rstd = (hf.square().mean(-1) + EPS).rsqrt()
    y = (_by_sample(hf * rstd[:, None], case) * _multiplier(state)).view(T, H).to(state["x"].dtype)
    out = [y, h, rstd] + ([prstd] if case["post"] else [])
    if case["ckpt"] != "none":
        for v in [h] + ([state["x"]] if _saves_x(case) else []):
            q, scale = _quantize(v.float(), case["ckpt"], case["block"])
            out += [_values(q, scale, case["block"]).to(READ_BACK), scale]
    return out


def _plain_bwd(state):
    case = state["case"]
    S, H = case["samples"], case["H"]
    ckpt = case["ckpt"] != "none"
    h = _values(*state["hq"], case["block"]) if ckpt else state["h"].float()
    xh = _by_sample(h * state["rstd"][:, None], case)
    dy = _by_sample(state["dy"], case)
    g = dy * _multiplier(state)
    d = state["rstd"].view(S, -1, 1) * (g - xh * (g * xh).mean(-1, keepdim=True)) + _by_sample(state["dh"], case)
    A = (dy * xh).sum(1)
    grads = {}
    if case["scale"]:
        grads["dscale"] = A * state["w"].float()
        grads["dw"] = (A * (1.0 + state["scale"].float())).sum(0)
    else:
        grads["dw"] = A.sum(0)
    c = _coefficient(state)
    dx = d * c
    if _saves_x(case):
        x = _by_sample(_values(*state["xq"], case["block"]) if ckpt else state["x"].float(), case)
        if case["post"]:
            pr = state["prstd"].view(S, -1, 1)
            x = x * pr
            dx = pr * (dx - x * (dx * x).mean(-1, keepdim=True))
        C = case["bs"] * (d * x).sum(1)
        if case["gate"]:
            grads["dgate"] = C * state["pw"].float() if case["post"] else C
        if case["post"]:
            grads["dpw"] = (C * state["gate"].float() if case["gate"] else C).sum(0)
    out = [dx.reshape(-1, H).to(state["dy"].dtype), (case["rs"] * d).view(-1, H).to(state["dh"].dtype)]
    return out + [grads[k].to(state["w"].dtype) for k in ("dw", "dpw", "dgate", "dscale") if k in grads]


def _plain_q8(state):
    case = state["case"]
    q, scale = _quantize(state["x"].float(), case["q"], case["block"])
    return [_values(q, scale, case["block"]).to(READ_BACK), scale]


# ------------------------------------------------------------------ the framework's calls

def _own(state):
    import unet_groupnorm_amd as gn
    case = state["case"]
    if case["op"] == "q8":
        q, scale = gn.gn_q8_quantize(state["x"], DTYPES[case["q"]], block=case["block"])
        return [gn.gn_q8_dequantize(q, scale, READ_BACK, block=case["block"]), scale]
    how = {"post_weight": state.get("pw"), "gate": state.get("gate"), "scale": state.get("scale"),
           "residual_scale": case["rs"], "branch_scale": case["bs"]}
    ckpt = None if case["ckpt"] == "none" else DTYPES[case["ckpt"]]
    if case["op"] == "join_fwd":
        f = gn.gn_join_forward(state["x"], state["r"], state["w"], EPS, checkpoint=ckpt, block=case["block"], **how)
        out = [f.y, f.h, f.rstd] + ([f.post_rstd] if case["post"] else [])
        if ckpt is not None:
            for saved in [f.saved_h] + ([f.saved_x] if _saves_x(case) else []):
                out += [gn.gn_q8_dequantize(*saved, READ_BACK, block=case["block"]), saved[1]]
        return out
    saved = ("h", "x") if ckpt is None else ("hq", "xq")
    b = gn.gn_join_backward(state["dy"], state[saved[0]], state["rstd"], state["w"], x=state.get(saved[1]),
                            post_rstd=state.get("prstd"), dh=state["dh"], block=case["block"], **how)
    return [b.dx, b.dres] + [g for g in (b.dweight, b.dpost_weight, b.dgate, b.dscale) if g is not None]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_fwd(state) if op == "join_fwd" else _plain_bwd(state) if op == "join_bwd" else _plain_q8(state)


# ------------------------------------------------------------------ 64 bits

def _e4m3(v):
    """Nearest e4m3 value, ties to even, of |v| <= 448."""
    e = torch.frexp(v)[1].clamp(min=-5).double() - 4.0   # v = m * 2^(e + 4), |m| in [0.5, 1)
    step = torch.exp2(e)
    return torch.round(v / step) * step


def _exact_q8(v, kind, block):
    H = v.shape[1]
    B = block or H
    values, scales = torch.empty_like(v), []
    for c in range(0, H, B):
        part = v[:, c:c + B]
        # the scale is an fp32 number, and the values go by it
        sc = torch.clamp(part.abs().max(dim=1).values / QMAX[kind], min=2.0 ** -126).float().double()
        u = part / sc.unsqueeze(1)
        values[:, c:c + B] = (torch.round(u).clamp(-127, 127) if kind == "int8" else _e4m3(u.clamp(-448, 448))) * sc.unsqueeze(1)
        scales.append(sc)
    return [values, torch.stack(scales, dim=1)]


def _decode(saved, block):
    q, scale = saved[0].float().double(), saved[1].double()
    if not block:
        return q * scale
    out = torch.empty_like(q)
    for k in range(scale.shape[1]):
        out[:, k * block:(k + 1) * block] = q[:, k * block:(k + 1) * block] * scale[:, k:k + 1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    T, H = case["T"], case["H"]
    if case["op"] == "q8":
        return _exact_q8(s["x"].double(), case["q"], case["block"])
    row = torch.arange(T, device="cuda") // (T // case["samples"])     # each row's sample
    w = s["w"].double()
    mult = w * (1.0 + s["scale"].double()[row]) if case["scale"] else w.expand(T, H)
    coef = torch.full((T, H), case["bs"], dtype=torch.float64, device="cuda")
    if case["gate"]:
        coef = coef * s["gate"].double()[row]
    if case["post"]:
        coef = coef * s["pw"].double()
    if case["op"] == "join_fwd":
        x = s["x"].double()
        pr = 1.0 / torch.sqrt(torch.sum(x * x, dim=1) / H + EPS) if case["post"] else None
        h = case["rs"] * s["r"].double() + coef * (x if pr is None else x * pr.unsqueeze(1))
        h = h.to(s["r"].dtype).double()                                # h is what is stored
        rs = 1.0 / torch.sqrt(torch.sum(h * h, dim=1) / H + EPS)
        out = [h * mult * rs.unsqueeze(1), h, rs] + ([] if pr is None else [pr])
        if case["ckpt"] != "none":
            out += _exact_q8(h, case["ckpt"], case["block"])
            if _saves_x(case):
                out += _exact_q8(x, case["ckpt"], case["block"])
        return out
    rs = s["rstd"].double().unsqueeze(1)
    h = s["h"].double() if "h" in s else _decode(s["hq"], case["block"])
    dy = s["dy"].double()
    dot = torch.sum(dy * mult * h, dim=1, keepdim=True)
    d = rs * dy * mult - rs ** 3 * h * dot / H + s["dh"].double()

    def per_sample(v):
        return torch.zeros(case["samples"], H, dtype=torch.float64, device="cuda").index_add_(0, row, v)

    grads = {"dw": torch.sum(dy * h * rs * (1.0 + s["scale"].double()[row] if case["scale"] else 1.0), dim=0)}
    if case["scale"]:
        grads["dscale"] = per_sample(dy * h * rs * w)
    dx = d * coef
    if _saves_x(case):
        x = s["x"].double() if "x" in s else _decode(s["xq"], case["block"])
        norm = x
        if case["post"]:
            pr = s["prstd"].double().unsqueeze(1)
            norm = x * pr
            dx = pr * dx - pr ** 3 * x * torch.sum(d * coef * x, dim=1, keepdim=True) / H
            grads["dpw"] = torch.sum(d * norm * case["bs"] * (s["gate"].double()[row] if case["gate"] else 1.0), dim=0)
        if case["gate"]:
            grads["dgate"] = per_sample(d * norm * case["bs"] * (s["pw"].double() if case["post"] else 1.0))
    return [dx, case["rs"] * d] + [grads[k] for k in ("dw", "dpw", "dgate", "dscale") if k in grads]


def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}
    T, H, x = case["T"], case["H"], size[case["x"]]
    n = T * H
    scales = 4 * T * (-(-H // case["block"]) if case["block"] else 1)
    if case["op"] == "q8":
        return {"bytes": n * (x + 2) + scales, "flops": 4 * n}
    res, w, S = size[case["res"]], size[case["w"]], case["samples"]
    vectors = (1 + case["post"] + S * (case["gate"] + case["scale"])) * H * w
    stats = 4 * T * (1 + case["post"])
    saved = 1 + _saves_x(case)
    if case["op"] == "join_fwd":
        # A checkpoint is counted as the values it stands for, which are what a pass returns.
        ckpt = saved * (n * 2 + scales) if case["ckpt"] != "none" else 0
        return {"bytes": n * (2 * x + 2 * res) + vectors + stats + ckpt, "flops": 12 * n}
    kept = (res + (x if _saves_x(case) else 0)) * n if case["ckpt"] == "none" else saved * (n + scales)
    return {"bytes": n * (2 * x + 2 * res) + kept + 2 * vectors + stats, "flops": 26 * n}
