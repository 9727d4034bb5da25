"""The row norm on the GPU against its definition in 64 bits (tests/ops_reference.py): forward,
8-bit output, backward and autograd, over widths from one column to the widest, odd and
unaligned ones among them, every combination of types, and special values."""
import itertools
import random

import pytest
import torch

import unet_groupnorm_amd as gn
from tests import ops_reference as R
from unet_groupnorm_amd._lib import GnGradTensor, lib
from unet_groupnorm_amd.gn import GnError

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6
INF = float("inf")


def say(msg):
    print(f"[gpu-rms] {msg}", flush=True)


def rand(shape, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + offset).to(dtype)


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def guarded(shape, dtype, shift=0):
    """An output tensor of `shape`, `shift` elements off its buffer's alignment, inside a buffer
    of sevens; check() fails if anything around it has been written."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128 + shift,), 7, device="cuda").to(dtype)
    t = buf[64 + shift:64 + shift + n].view(shape)

    def check(name):
        assert bool((buf[:64 + shift].float() == 7).all()) and bool((buf[64 + shift + n:].float() == 7).all()), \
            f"{name}: written outside"
    return t, check


WIDTHS = [1, 2, 7, 8, 9, 31, 64, 96, 100, 128, 192, 255, 256, 500, 511, 512, 513, 520, 1001, 1024, 1531, 2048, 2056, 4096,
          5120, 8192, 8200, 10007, 16384, 32761, 32768]
# x, residual, weight, y
TYPES = [(x, r, w, y) for x in (BF, F16, F32) for r, w, y in itertools.product({None, x, F32}, {None, x, F32}, {x, F32})]


def check_forward(x, w, res, out_dtype, shift=0):
    T, H = x.numel() // x.shape[-1], x.shape[-1]
    y, ok_y = guarded(x.shape, out_dtype, shift)
    rstd, ok_r = guarded(x.shape[:-1], F32)
    h, ok_h = (None, None) if res is None else guarded(x.shape, res.dtype, shift)
    got = gn.gn_rms_forward(x, w, EPS, residual=res, out_dtype=out_dtype, out=y, rstd=rstd, h=h)
    torch.cuda.synchronize()
    assert got[0] is y and got[2] is rstd
    ry, rh, rr = R.rms_forward(x, w, EPS, res)
    R.close("rstd", rstd, rr, rr * R.RSTD)
    R.close("y", y, ry, ry.abs() * R.Y + R.half_step(ry, out_dtype) * (1 + R.Y) + 1e-37)
    for name, ok in (("y", ok_y), ("rstd", ok_r)):
        ok(name)
    if res is not None:
        ok_h("h")
        R.close("h", h, rh, 0.0)
    return T, H


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(H):
    for T, x_dt, r_dt, y_dt, shift in ((1, BF, BF, BF, 0), (37, BF, None, BF, 1), (5, F16, F32, F16, 3), (6, F32, F32, F32, 1)):
        say(f"forward T={T} H={H} {x_dt} res={r_dt} shift={shift}")
        x = rand((T * H + shift,), x_dt, 1, 1.5, 0.1)[shift:].view(T, H)
        res = None if r_dt is None else rand((T * H + shift,), r_dt, 2, 3.0)[shift:].view(T, H)
        check_forward(x, rand((H,), F32, 3, 0.2, 1.0), res, y_dt, shift)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v).replace("torch.", "") for v in t))
def test_forward_types(types):
    x_dt, r_dt, w_dt, y_dt = types
    for T, H in ((3, 64), (130, 200), (9, 1024), (3, 12000)):
        say(f"forward {types} T={T} H={H}")
        res = None if r_dt is None else rand((T, H), r_dt, 5, 2.0, 0.3)
        w = None if w_dt is None else rand((H,), w_dt, 6, 0.2, 1.0)
        check_forward(rand((T, H), x_dt, 4), w, res, y_dt)


@pytest.mark.parametrize("H", [1, 3, 41, 64, 100, 1001, 1531, 4096, 8200, 32761])
def test_rstd_of_exact_sums(H):
    """Rows of small integers: the sum of squares is below 2^24, so exact in any order. What is
    left is the mean's rounding, halved by the root, and the root's own: 1.5 u."""
    for dt in (BF, F16, F32):
        say(f"rstd of integers, H={H} {dt}")
        g = torch.Generator(device="cuda")
        g.manual_seed(26)
        x = torch.randint(1, 30, (2000, H), generator=g, device="cuda").to(dt)
        rstd = gn.gn_rms_forward(x, None, 0.0)[2]
        ref = 1.0 / torch.sqrt(x.double().square().mean(-1))
        R.close("rstd", rstd, ref, ref * 1.5 * R.U * (1 + 2.0 ** -16))


def test_forward_strided_rows_and_leading_dimensions():
    wide = rand((6, 5, 300), BF, 7)
    for x in (wide[..., 100:228], wide[..., 1:300], wide[:, :1, 3:40], rand((40,), BF, 8), rand((0, 16), BF, 9)):
        say(f"forward sizes {tuple(x.shape)} strides {x.stride()}")
        w = rand((x.shape[-1],), F32, 10, 0.1, 1.0)
        y, h, rstd = gn.gn_rms_forward(x, w, EPS, residual=x.contiguous())
        ref = gn.gn_rms_forward(x.contiguous(), w, EPS, residual=x.contiguous())
        assert y.shape == h.shape == x.shape and rstd.shape == x.shape[:-1]
        for a, b in zip((y, h, rstd), ref):
            assert torch.equal(bits(a), bits(b))


def test_in_place_residual_and_output():
    x, res, w = rand((33, 1536), BF, 11), rand((33, 1536), BF, 12), rand((1536,), BF, 13)
    y, h, rstd = gn.gn_rms_forward(x, w, EPS, residual=res)
    x2, r2 = x.clone(), res.clone()
    y2, h2, rstd2 = gn.gn_rms_forward(x2, w, EPS, residual=r2, out=x2, h=r2)
    assert y2 is x2 and h2 is r2
    for a, b in ((y, x2), (h, r2), (rstd, rstd2)):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("H", [8, 100, 128, 1024, 4096, 12000])
def test_a_rows_bits_do_not_depend_on_the_batch(H):
    x, res, w = rand((300, H), BF, 14), rand((300, H), BF, 15), rand((H,), BF, 16)
    all_rows = gn.gn_rms_forward(x, w, EPS, residual=res)
    q_all = gn.gn_rms_forward_q8(x, w, EPS, residual=res)
    for a, b in ((0, 1), (7, 9), (123, 300)):
        some = gn.gn_rms_forward(x[a:b], w, EPS, residual=res[a:b])
        q_some = gn.gn_rms_forward_q8(x[a:b], w, EPS, residual=res[a:b])
        for p, s in list(zip(all_rows, some)) + list(zip(q_all[:3], q_some[:3])):
            assert torch.equal(bits(p[a:b]), bits(s))


def test_special_values():
    x = rand((8, 200), F32, 17)
    x[1, 3], x[2, 199], x[3, 0], x[4] = float("nan"), float("inf"), -float("inf"), 0.0
    x[5] *= 1e-30
    x[6] *= 1e15
    w = rand((200,), F32, 18, 0.1, 1.0)
    say("NaN, infinities, a row of zeros, rows of 1e-30 and 1e15")
    check_forward(x, w, None, F32)
    check_forward(x.to(BF), w, rand((8, 200), BF, 19) * 0, BF)
    for dt in (torch.int8, torch.float8_e4m3fn):
        q, scale, _, _ = gn.gn_rms_forward_q8(x, w, EPS, q_dtype=dt, block=32)
        v = gn.gn_q8_dequantize(q, scale, block=32)
        nan = torch.isnan(v)
        assert bool(nan[1].all())                                   # a NaN makes its row NaN
        assert bool(nan[2, 192:].all()) and not bool(nan[2, :192].any()) and float(v[2, :192].abs().max()) == 0
        assert bool(nan[3, :32].all()) and not bool(nan[3, 32:].any())
        assert not bool(nan[4:].any()) and float(v[4].abs().max()) == 0 and float(scale[4].max()) == 2.0 ** -126


# ------------------------------------------------------------------ 8 bits

def check_q8(x, w, res, q_dtype, block, shift=0):
    H = x.shape[-1]
    q, ok_q = guarded(x.shape, q_dtype, shift)
    n = -(-H // block) if block else 1
    scale, ok_s = guarded(tuple(x.shape[:-1]) + (n,), F32)
    _, _, h, rstd = gn.gn_rms_forward_q8(x, w, EPS, residual=res, q_dtype=q_dtype, block=block, out=q, scale=scale,
                                         need_rstd=True)
    v = gn.gn_q8_dequantize(q, scale, F32, block=block)
    torch.cuda.synchronize()
    ok_q("q")
    ok_s("scale")
    ry, rh, rr = R.rms_forward(x, w, EPS, res)
    R.close("rstd", rstd, rr, rr * R.RSTD)
    if res is not None:
        assert torch.equal(h.double(), rh)
    B = block or H
    qmax = 127.0 if q_dtype == torch.int8 else 448.0
    pad = torch.nn.functional.pad(ry, (0, n * B - H)).view(*x.shape[:-1], n, B)
    rs = (pad.abs().amax(-1) / qmax).clamp(min=2.0 ** -126)
    slack = R.Y + 4 * R.U
    R.close("scale", scale, rs, rs * slack)
    full = scale.double().unsqueeze(-1).expand(*scale.shape, B).reshape(*x.shape[:-1], n * B)[..., :H]
    # v is exact but for its own rounding: half a step of the format in units of the scale, plus
    # what the roundings of y and of the scale are worth at the largest quotient.
    step = full * (torch.full_like(full, 0.5) if q_dtype == torch.int8 else R.e4m3_step(ry / full))
    R.close("values", v, ry, step * (1 + slack) + full * qmax * (slack + R.U))
    # the values are q * scale, rounded once
    exact = q.to(F32).double() * full
    assert torch.equal(v.double(), exact.to(F32).double())
    for dt in (BF, F16):
        assert torch.equal(bits(gn.gn_q8_dequantize(q, scale, dt, block=block)), bits(exact.to(F32).to(dt)))


@pytest.mark.parametrize("q_dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_q8(q_dtype, block):
    for T, H, x_dt, r_dt, shift in ((1, 1, F32, None, 0), (5, 7, BF, BF, 0), (3, 24, BF, None, 1), (19, 64, BF, BF, 0),
                                    (9, 100, F16, F32, 3), (70, 128, BF, None, 0), (4, 520, BF, BF, 0),
                                    (5, 1001, F32, F32, 1), (16, 4096, F16, F16, 0), (3, 5120, BF, F32, 0),
                                    (2, 8192, BF, BF, 0), (2, 12345, BF, BF, 5), (1, 32768, BF, BF, 0)):
        say(f"q8 {q_dtype} block={block} T={T} H={H} {x_dt} res={r_dt}")
        res = None if r_dt is None else rand((T, H), r_dt, 21, 2.0)
        check_q8(rand((T, H), x_dt, 20), rand((H,), x_dt if H % 2 else F32, 22, 0.3, 1.0), res, q_dtype, block, shift)


@pytest.mark.parametrize("q_dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_q8_bits_follow_from_the_norm(q_dtype, block):
    """Given h, rstd and the weight, y is two rounded products, the scale one rounded quotient and
    q another (whose fp32 value may be another neighbour only 2^-20 ulp from halfway between two;
    none of these is): nothing is left to a tolerance, and every bit is compared. Weights down to
    subnormal numbers, where the scale meets its floor."""
    qmax = 127.0 if q_dtype == torch.int8 else 448.0
    for T, H, x_dt, r_dt, size in ((400, 4096, BF, BF, 1.0), (300, 1001, F16, F32, 1.0), (900, 100, F32, None, 1.0),
                                   (5, 3, BF, None, 1.0), (64, 8200, BF, None, 1e-28), (64, 520, F32, F32, 1e-33),
                                   (64, 1024, BF, BF, 1e-36), (64, 520, F32, F32, 2e-37), (64, 96, F32, None, 1e-39),
                                   (64, 4096, F16, F16, 1e-43), (16, 4096, F32, None, 1e30)):
        say(f"q8 bits {q_dtype} block={block} T={T} H={H} {x_dt} res={r_dt} weights of {size}")
        x, w = rand((T, H), x_dt, 23, 1.5), rand((H,), F32, 24, 0.3 * size, size)
        res = None if r_dt is None else rand((T, H), r_dt, 25, 2.0)
        q, scale, h, rstd = gn.gn_rms_forward_q8(x, w, EPS, residual=res, q_dtype=q_dtype, block=block, need_rstd=True)
        y = (h.cpu().float() * rstd.cpu().unsqueeze(-1)) * w.cpu()
        B = block or H
        n = -(-H // B)
        runs = torch.nn.functional.pad(y, (0, n * B - H)).view(T, n, B)
        want = (runs.abs().amax(-1) / qmax).clamp(min=2.0 ** -126)
        assert torch.equal(bits(scale.cpu()), bits(want)), "scale"
        v = (runs / want.unsqueeze(-1)).view(T, n * B)[:, :H]
        wq = torch.round(v).to(torch.int8) if q_dtype == torch.int8 else v.to(torch.float8_e4m3fn)
        assert torch.equal(q.cpu().float(), wq.float()), "q"


# ------------------------------------------------------------------ backward

BWD_TYPES = [(h, x, dy) for h, x, dy in itertools.product((BF, F16, F32), repeat=3)
             if (x == h or h == F32) and (dy == x or dy == F32)]


def check_backward(T, H, h_dt, x_dt, dy_dt, w_dt, with_dh, seed, shift=0):
    h = rand((T, H), h_dt, seed, 1.5, 0.2)
    rstd = (h.double().square().mean(-1) + EPS).rsqrt().float()
    dy = rand((T, H), dy_dt, seed + 1, 0.5, 0.02)
    w = None if w_dt is None else rand((H,), w_dt, seed + 2, 0.3, 1.0)
    dh = rand((T, H), h_dt, seed + 3, 0.5) if with_dh else None
    dx, ok_dx = guarded((T, H), x_dt, shift)
    dw, ok_dw = guarded((H,), F32 if w is None else w_dt)
    apart = x_dt != h_dt
    dres, ok_dres = guarded((T, H), h_dt, shift) if apart else (None, None)
    gn.gn_rms_backward(dy, h, rstd, w, dh=dh, x_dtype=x_dt, dx=dx, dweight=dw, dres=dres)
    torch.cuda.synchronize()
    d, rdw, bound, dw_bound = R.rms_backward(dy, h, rstd, w, dh)
    R.close("dx", dx, d, bound + R.half_step(d.abs() + bound, x_dt))
    R.close("dweight", dw, rdw, dw_bound + R.half_step(rdw.abs() + dw_bound, dw.dtype))
    ok_dx("dx")
    ok_dw("dweight")
    if apart:
        R.close("dres", dres, d, bound + R.half_step(d.abs() + bound, h_dt))
        ok_dres("dres")


@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H):
    for T, h_dt, with_dh in ((1, BF, True), (67, BF, False), (5, F32, True)):
        say(f"backward T={T} H={H} {h_dt} dh={with_dh}")
        check_backward(T, H, h_dt, h_dt, h_dt, F32, with_dh, 30, 1 if H % 3 == 0 else 0)


@pytest.mark.parametrize("types", BWD_TYPES, ids=lambda t: "-".join(str(v).replace("torch.", "") for v in t))
def test_backward_types(types):
    h_dt, x_dt, dy_dt = types
    for (T, H), w_dt, with_dh in itertools.product(((3, 64), (130, 200), (9, 1024), (2, 9000)), {None, x_dt, F32}, (False, True)):
        say(f"backward {types} T={T} H={H} w={w_dt} dh={with_dh}")
        check_backward(T, H, h_dt, x_dt, dy_dt, w_dt, with_dh, 40)


@pytest.mark.parametrize("T,H", [(100000, 64), (40000, 128), (5000, 100), (3001, 1024), (2050, 4096), (1500, 10000)])
def test_backward_many_rows(T, H):
    say(f"backward T={T} H={H}")
    check_backward(T, H, BF, BF, BF, BF, True, 50)
    check_backward(T, H, F32, F16, F16, F32, False, 51)


def test_backward_parts_in_place_and_bits():
    T, H = 700, 1536
    h, dy, dh = rand((T, H), BF, 60), rand((T, H), BF, 61), rand((T, H), BF, 62)
    w = rand((H,), BF, 63, 0.2, 1.0)
    rstd = gn.gn_rms_forward(h, w, EPS)[2]
    ws = torch.full((gn.gn_rms_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN if read unwritten
    dx, dw, dres = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, workspace=ws)
    assert dres is None
    again = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, need_dres=True)
    assert again[2] is again[0]
    only_dx = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, need_dweight=False)
    only_dw = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, need_dx=False)
    only_res = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, need_dx=False, need_dweight=False, need_dres=True)
    assert only_dx[1] is None and only_dw[0] is None and only_res[:2] == (None, None)
    for a, b in ((dx, again[0]), (dw, again[1]), (dx, only_dx[0]), (dw, only_dw[1]), (dx, only_res[2])):
        assert torch.equal(bits(a), bits(b))
    for place in ("dy", "h", "dh"):
        t = {"dy": dy.clone(), "h": h.clone(), "dh": dh.clone()}
        gn.gn_rms_backward(t["dy"], t["h"], rstd, w, dh=t["dh"], dx=t[place], need_dweight=True)
        assert torch.equal(bits(dx), bits(t[place])), place


def test_backward_into_a_given_residual_gradient():
    h, dy, rstd = rand((9, 200), BF, 140), rand((9, 200), BF, 141), rand((9,), F32, 142).abs()
    want = gn.gn_rms_backward(dy, h, rstd, None)[0]
    dres = torch.full_like(h, 7)
    dx, _, got = gn.gn_rms_backward(dy, h, rstd, None, dres=dres)
    assert got is dres and torch.equal(bits(dres), bits(want)) and torch.equal(bits(dx), bits(want))


def test_backward_of_no_rows_and_of_special_values():
    w = rand((64,), BF, 64)
    dx, dw, _ = gn.gn_rms_backward(rand((0, 64), BF, 65), rand((0, 64), BF, 66), rand((0,), F32, 67), w)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    h = rand((6, 96), F32, 68)
    dy = rand((6, 96), F32, 69)
    dy[1, 5], dy[2, 95] = float("nan"), float("inf")
    h[3] = 0.0
    rstd = (h.double().square().mean(-1) + EPS).rsqrt().float()
    dx, dw, _ = gn.gn_rms_backward(dy, h, rstd, None)
    d, rdw, bound, dw_bound = R.rms_backward(dy, h, rstd, None)
    fine = [0, 3, 4, 5]
    R.close("dx", dx[fine], d[fine], bound[fine])
    assert bool(torch.isnan(dx[1]).all()) and not bool(torch.isfinite(dx[2]).any())
    cols = [c for c in range(96) if c not in (5, 95)]
    assert bool(torch.isnan(dw[5])) and bool(torch.isinf(dw[95]))
    R.close("dweight", dw[cols], rdw[cols], dw_bound[cols])


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes_and_types(seed):
    rng = random.Random(seed)
    H = rng.choice([rng.randint(1, 70), rng.randint(1, 600), rng.randint(500, 5000), rng.randint(4000, 32768)])
    T = max(1, min(rng.randint(1, 3000), 2_000_000 // H))
    x_dt, shift = rng.choice([BF, F16, F32]), rng.randint(0, 7)
    r_dt, w_dt, y_dt, h_dt = (rng.choice(c) for c in ((None, x_dt, F32), (None, x_dt, F32), (x_dt, F32), (x_dt, F32)))
    dy_dt, with_dh = rng.choice([x_dt, F32]), rng.random() < 0.5
    q_dt, block = rng.choice([torch.int8, torch.float8_e4m3fn]), rng.choice([0, 32, 64, 128])
    say(f"seed {seed}: T={T} H={H} x={x_dt} res={r_dt} w={w_dt} y={y_dt} h={h_dt} dy={dy_dt} {q_dt} {block} shift={shift}")
    x = rand((T * H + shift,), x_dt, seed)[shift:].view(T, H)
    res = None if r_dt is None else rand((T * H + shift,), r_dt, seed + 1, 2.0)[shift:].view(T, H)
    w = None if w_dt is None else rand((H,), w_dt, seed + 2, 0.3, 1.0)
    check_forward(x, w, res, y_dt, shift)
    check_q8(x, w, res, q_dt, block, shift)
    check_backward(T, H, h_dt, x_dt, dy_dt, w_dt, with_dh, seed, shift)


def test_offsets_past_32_bits():
    T, H = 70001, 32760                      # 2.3e9 elements, 4.6 GB a tensor
    say(f"{T} x {H} bf16")
    x = torch.empty(T, H, dtype=BF, device="cuda")
    part = rand((1000, H), BF, 91)
    for k in range(0, T, 1000):
        x[k:k + 1000] = part[:min(1000, T - k)]
    w = rand((H,), BF, 92, 0.2, 1.0)
    want, _, want_rstd = gn.gn_rms_forward(part, w)
    y, _, rstd = gn.gn_rms_forward(x, w)
    for k in (0, 65000, 66000, 70000):       # rows before and behind 2^31 elements (row 65552)
        n = min(1000, T - k)
        assert torch.equal(bits(y[k:k + n]), bits(want[:n])) and torch.equal(rstd[k:k + n], want_rstd[:n])
    y.fill_(7)
    gn.gn_rms_backward(x, x, rstd, w, dx=y, need_dweight=False)
    ref = gn.gn_rms_backward(part, part, want_rstd, w, need_dweight=False)[0]
    for k in (0, 65000, 66000, 70000):
        n = min(1000, T - k)
        assert torch.equal(bits(y[k:k + n]), bits(ref[:n]))
    del y
    q, scale, _, _ = gn.gn_rms_forward_q8(x, w, block=128)
    qr, sr, _, _ = gn.gn_rms_forward_q8(part, w, block=128)
    v = gn.gn_q8_dequantize(q, scale, BF, block=128)
    vr = gn.gn_q8_dequantize(qr, sr, BF, block=128)
    for k in (0, 65000, 66000, 70000):
        n = min(1000, T - k)
        assert torch.equal(q[k:k + n], qr[:n]) and torch.equal(bits(v[k:k + n]), bits(vr[:n]))


# ------------------------------------------------------------------ calls past the last-level cache
#
# Calls that move over 200 MiB load their rows with another cache policy, in the backward by
# kernels of their own for rows of whole pieces: one width for each number of pieces a lane.

BIG = [(8800, 4096, BF), (18000, 2048, F16), (400000, 128, BF), (100000, 512, BF), (2200, 16384, BF), (2200, 16384, F16),
       (65536, 512, F32), (400000, 128, F32), (4500, 4096, F32), (2200, 8192, F32), (1100, 16384, F32)]


@pytest.mark.parametrize("T,H,dt", BIG, ids=lambda v: str(v).replace("torch.", ""))
def test_backward_past_the_cache(T, H, dt):
    assert T * H * dt.itemsize * 3 > 200 << 20
    say(f"backward T={T} H={H} {dt} with and without dh")
    check_backward(T, H, dt, dt, dt, dt, True, 100)
    check_backward(T, H, dt, dt, dt, None, False, 104)
    if dt != F32:
        say(f"backward T={T} H={H} {dt} of an fp32 stream")
        check_backward(T, H, F32, dt, dt, F32, True, 108)
        check_backward(T, H, dt, dt, F32, F32, True, 112)


@pytest.mark.parametrize("T,H", [(8192, 4096), (400000, 128), (2200, 16384), (40000, 1001)])
def test_backward_past_the_cache_in_place(T, H):
    say(f"backward in place T={T} H={H}")
    dy, h, dh = rand((T, H), BF, 120), rand((T, H), BF, 121), rand((T, H), BF, 122)
    w = rand((H,), BF, 123, 0.2, 1.0)
    rstd = gn.gn_rms_forward(h, w, EPS)[2]
    dx, dw, _ = gn.gn_rms_backward(dy, h, rstd, w, dh=dh)
    for place in ("dy", "h", "dh"):
        t = {"dy": dy.clone(), "h": h.clone(), "dh": dh.clone()}
        dw2 = gn.gn_rms_backward(t["dy"], t["h"], rstd, w, dh=t["dh"], dx=t[place])[1]
        assert torch.equal(bits(dx), bits(t[place])) and torch.equal(bits(dw), bits(dw2)), place


@pytest.mark.parametrize("T,H,x_dt,r_dt", [(16384, 2048, BF, BF), (400000, 128, F16, F16), (400000, 128, BF, F32),
                                           (3000, 16384, BF, BF), (40000, 1001, BF, BF), (9000, 4096, F32, F32),
                                           (10000, 4096, F16, F32), (400000, 192, BF, None)])
def test_forward_and_q8_past_the_cache(T, H, x_dt, r_dt):
    say(f"forward and q8 T={T} H={H} {x_dt} res={r_dt}")
    x, w = rand((T, H), x_dt, 130, 1.5), rand((H,), F32, 131, 0.2, 1.0)
    res = None if r_dt is None else rand((T, H), r_dt, 132, 2.0)
    check_forward(x, w, res, x_dt)
    check_q8(x, w, res, torch.int8, 0)
    check_q8(x, w, res, torch.float8_e4m3fn, 32)
    y, h, rstd = gn.gn_rms_forward(x, w, EPS, residual=res)
    h = h.clone()
    gn.gn_rms_forward(x, w, EPS, residual=res, out=x, h=res)
    assert torch.equal(bits(x), bits(y)) and (res is None or torch.equal(bits(res), bits(h)))


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("x_dt,r_dt", [(F32, F32), (F32, None), (BF, BF), (F16, F32)])
def test_autograd_against_the_formula_and_differences(x_dt, r_dt):
    T, H = 6, 40
    x = rand((2, 3, H), x_dt, 70).requires_grad_()
    res = None if r_dt is None else rand((2, 3, H), r_dt, 71).requires_grad_()
    w = rand((H,), F32, 72, 0.2, 1.0).requires_grad_()
    a, b = rand((2, 3, H), F32, 73), rand((2, 3, H), F32, 74)
    y, h = (gn.rms_norm(x, w, EPS), None) if res is None else gn.rms_norm(x, w, EPS, residual=res)
    loss = (y.float() * a).sum() + (0 if h is None else (h.float() * b).sum())
    leaves = [x, w] + ([] if res is None else [res])
    grads = torch.autograd.grad(loss, leaves)

    def f(vals):   # the loss in fp64, without roundings
        hh = vals[0] if res is None else vals[0] + vals[2]
        yy = hh * (hh.square().mean(-1, keepdim=True) + EPS).rsqrt() * vals[1]
        return (yy * a.double()).sum() + (0 if res is None else (hh * b.double()).sum())

    base = [t.detach().double() for t in leaves]
    exact = [t.clone().requires_grad_() for t in base]
    f(exact).backward()
    # Inputs in 16 bits: h is rounded in the kernel and the gradient of y arrives rounded, an
    # eps of each; the fp32 case has its own roundings alone.
    tol = 1e-5 if x_dt == F32 else 4 * torch.finfo(x_dt).eps
    for name, g, e, t in zip(("x", "weight", "residual"), grads, exact, leaves):
        assert g.dtype == t.dtype and g.shape == t.shape
        rel = float((g.double() - e.grad).norm() / e.grad.norm())
        say(f"d{name}: {rel:.2e} from the formula's gradient")
        assert rel < tol, name
    step = 1e-5
    for k, t in enumerate(base):
        d = torch.randn(t.shape, generator=torch.Generator().manual_seed(k), dtype=torch.float64).cuda()
        lo, hi = [v.clone() for v in base], [v.clone() for v in base]
        lo[k] -= step * d
        hi[k] += step * d
        diff = float((f(hi) - f(lo)) / (2 * step))
        got = float((grads[k].double() * d).sum())
        size = float((grads[k].double() * d).norm()) * d.numel() ** 0.5
        assert abs(got - diff) <= max(tol, 1e-7) * max(size, 1.0), (k, got, diff)


def test_autograd_partial_uses():
    x, res = rand((4, 5, 64), BF, 80).requires_grad_(), rand((4, 5, 64), F32, 81).requires_grad_()
    w = rand((64,), BF, 82).requires_grad_()
    y, h = gn.rms_norm(x, w, residual=res)
    h.sum().backward()                                    # the stream alone: the norm's part is zero
    assert torch.equal(res.grad, torch.ones_like(res)) and torch.equal(x.grad, torch.ones_like(x))
    assert float(w.grad.abs().max()) == 0
    x.grad = res.grad = w.grad = None
    y, h = gn.rms_norm(x, w, residual=res)
    y.sum().backward()
    want = gn.gn_rms_backward(torch.ones_like(y), h.detach(), gn.gn_rms_forward(x, w, residual=res)[2], w.detach(), x_dtype=BF)
    for a, b in ((x.grad, want[0]), (w.grad, want[1]), (res.grad, want[2])):
        assert torch.equal(bits(a), bits(b))
    # rows that are not evenly spaced, a broadcast input and a transposed gradient
    z = rand((5, 4, 64), BF, 83).transpose(0, 1).requires_grad_()
    y = gn.rms_norm(z, w)
    assert torch.equal(bits(y), bits(gn.gn_rms_forward(z.detach().contiguous(), w)[0]))
    y.transpose(0, 1).sum().backward()
    v = rand((64,), BF, 84).requires_grad_()
    gn.rms_norm(v.expand(6, 64), None).float().sum().backward()
    assert z.grad.shape == z.shape and v.grad.shape == v.shape
    with torch.no_grad():
        assert not gn.rms_norm(x, w).requires_grad
    with pytest.raises(RuntimeError):                     # no second derivative
        y = gn.rms_norm(x, w)
        (g,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
        g.float().sum().backward()


def test_autograd_of_the_stream_alone_beside_special_values():
    """Where only h is used its gradient is x's and the residual's, whatever the rows hold."""
    for x_dt, r_dt in ((BF, BF), (F16, F32), (F32, F32)):
        x, res = rand((5, 64), x_dt, 150), rand((5, 64), r_dt, 151)
        x[1, 3], x[2, 5], x[3] = float("nan"), INF, 0.0
        res[3] = 0.0
        x.requires_grad_(), res.requires_grad_()
        w = rand((64,), F32, 152).requires_grad_()
        dh = rand((5, 64), r_dt, 153)
        _, h = gn.rms_norm(x, w, 0.0, residual=res)
        h.backward(dh)
        assert torch.equal(bits(res.grad), bits(dh)) and torch.equal(bits(x.grad), bits(dh.to(x_dt)))
        assert float(w.grad.abs().max()) == 0
        _, h = gn.rms_norm(x, None, 0.0, residual=res.detach())
        (g,) = torch.autograd.grad(h, x, dh)
        assert torch.equal(bits(g), bits(dh.to(x_dt)))


@pytest.mark.parametrize("shape", [(1, 64), (1, 1, 64), (64, 1)], ids=str)
def test_autograd_of_a_weight_that_is_not_a_vector(shape):
    x = rand((4, 5, 64), BF, 88)
    flat = rand((64,), BF, 89).requires_grad_()
    w = flat.detach().reshape(shape).requires_grad_()
    for weight in (flat, w):
        gn.rms_norm(x, weight).float().square().sum().backward()
    assert w.grad.shape == shape and torch.equal(bits(w.grad.reshape(64)), bits(flat.grad))


def test_saved_tensors_that_a_later_call_overwrites():
    def graph():
        x, res, w = rand((6, 96), BF, 85).requires_grad_(), rand((6, 96), F32, 86), rand((96,), BF, 87)
        return gn.rms_norm(x, w, residual=res), x.detach(), w

    (y, h), x, w = graph()
    gn.gn_rms_forward(x, w, residual=h.detach(), h=h.detach())            # the stream in place
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    (y, h), x, w = graph()
    gn.gn_rms_forward_q8(x, w, residual=h.detach(), h=h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    (y, h), x, w = graph()
    gn.gn_rms_forward(x, w, residual=h.detach())                          # read, not written
    y.float().sum().backward()


def test_c_abi_refuses_memory_of_the_host():
    T, H = 4, 64
    x, res, y, h = (rand((T, H), BF, 93 + i) for i in range(4))
    w, rstd, dw = rand((H,), F32, 97), rand((T,), F32, 98).abs(), rand((H,), F32, 99)
    ws = torch.empty(lib.gn_rms_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    pinned = torch.zeros(1 << 14, pin_memory=True)
    host = torch.zeros(1 << 14)

    def fwd(**kw):
        a = dict(x=x, res=res, w=w, y=y, h=h, rstd=rstd)
        a.update(kw)
        a = {k: v.data_ptr() for k, v in a.items()}
        return lib.gn_rms_forward(a["x"], 1, H, a["res"], 1, a["w"], 0, T, H, 1e-6, a["y"], 1, a["h"], a["rstd"], None)

    def bwd(**kw):
        a = dict(dy=x, h=res, rstd=rstd, w=w, dh=y, dx=h, dw=dw, ws=ws)
        a.update(kw)
        a = {k: v.data_ptr() for k, v in a.items()}
        return lib.gn_rms_backward(a["dy"], 1, a["h"], 1, H, a["rstd"], a["w"], 0, a["dh"], T, H, a["dx"], 1, None, a["dw"],
                                   a["ws"], ws.numel(), None)

    def norm(data, out):
        t = (GnGradTensor * 1)()
        t[0].data, t[0].out, t[0].numel, t[0].dtype, t[0].out_dtype = data.data_ptr(), out.data_ptr(), 64, 0, 0
        return lib.gn_grad_clip(t, 1, 0, 1.0, rstd.data_ptr(), ws.data_ptr(), ws.numel(), None)

    for call, names in ((fwd, ("x", "res", "w", "y", "h", "rstd")), (bwd, ("dy", "h", "rstd", "w", "dh", "dx", "dw", "ws"))):
        assert call() == 0
        for name in names:
            for bad in (pinned, host):
                assert call(**{name: bad}) == 8, name
    assert norm(w, dw) == 0 and norm(pinned, dw) == 8 and norm(w, host) == 8
    torch.cuda.synchronize()


def test_refusals_on_the_device():
    x = rand((4, 64), BF, 90)
    for call in (lambda: gn.gn_rms_forward(x, torch.ones(64)), lambda: gn.gn_rms_forward(x, None, residual=x.cpu()),
                 lambda: gn.gn_rms_backward(x, x, torch.ones(4), None)):
        with pytest.raises((ValueError, GnError)):
            call()
    with pytest.raises(GnError):
        gn.gn_rms_forward(x, None, out=x.view(-1)[0:256].view(4, 64), residual=x)     # y over the residual
