"""The residual join and the 8-bit checkpoints on the GPU against their definition in 64 bits
(tests/join_reference.py): forward, checkpoints, backward from both, autograd, over widths from
one column to the widest, sequences of one row and more, every combination of types, and special
values."""
import itertools
import random

import pytest
import torch

import unet_groupnorm_amd as gn
from tests import join_reference as J
from unet_groupnorm_amd._lib import lib
from unet_groupnorm_amd.gn import GnError

pytestmark = pytest.mark.gpu
BF, F16, F32, I8, E4 = torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.float8_e4m3fn
EPS = 1e-6


def say(msg):
    print(f"[gpu-join] {msg}", flush=True)


def rand(shape, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + offset).to(dtype)


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def same(a, b):
    return a.shape == b.shape and torch.equal(bits(a), bits(b))


def guarded(shape, dtype, shift=0):
    """A tensor of `shape`, `shift` elements off its buffer's alignment, inside a buffer of sevens;
    check() fails if anything around it has been written."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128 + shift,), 7, device="cuda").to(dtype)
    t = buf[64 + shift:64 + shift + n].view(shape)

    def check(name):
        assert bool((buf[:64 + shift].float() == 7).all()) and bool((buf[64 + shift + n:].float() == 7).all()), \
            f"{name}: written outside"
    return t, check


class Guards:
    def __init__(self):
        self.checks = []

    def new(self, name, shape, dtype, shift=0):
        t, check = guarded(shape, dtype, shift)
        self.checks.append((name, check))
        return t

    def check(self):
        torch.cuda.synchronize()
        for name, check in self.checks:
            check(name)


def vectors(H, S, x_dt, seed, which, dts):
    """weight, post_weight, gate and scale as `which` (a subset of "wpgs") says, of the types dts."""
    make = {"w": ("weight", (H,), 1.0, 0.2), "p": ("post_weight", (H,), 0.8, 0.2), "g": ("gate", (S, H), 0.1, 0.4),
            "s": ("scale", (S, H), 0.0, 0.2)}
    out = {}
    for k, (c, dt) in enumerate(zip("wpgs", dts)):
        name, shape, mean, spread = make[c]
        out[name] = rand(shape, dt, seed + k, spread, mean) if c in which else None
    return out


def off(shape, dtype, seed, shift, scale=1.0, offset=0.0):
    n = 1
    for s in shape:
        n *= s
    return rand((n + shift,), dtype, seed, scale, offset)[shift:].view(shape)


def run_forward(T, H, x_dt, r_dt, S=1, which="wpg", post=True, dts=None, rs=1.0, bs=1.0, q_dtype=None, block=128, shift=0,
                seed=1):
    v = vectors(H, S, x_dt, seed + 10, which, dts or (F32, x_dt, F32, x_dt))
    x, r = off((T, H), x_dt, seed, shift, 1.5, 0.1), off((T, H), r_dt, seed + 1, shift, 3.0)
    g = Guards()
    n = -(-H // block) if block else 1
    how = dict(post_norm=post, residual_scale=rs, branch_scale=bs)
    out = dict(out=g.new("y", (T, H), x_dt, shift), h=g.new("h", (T, H), r_dt, shift), rstd=g.new("rstd", (T,), F32))
    if post:
        out["post_rstd"] = g.new("post_rstd", (T,), F32)
    reads_x = post or v["gate"] is not None
    if q_dtype is not None:
        for name in ["saved_h"] + (["saved_x"] if reads_x else []):
            out[name] = (g.new(name, (T, H), q_dtype, shift), g.new(name + "'s scale", (T, n), F32))
    weight = v.pop("weight")
    f = gn.gn_join_forward(x, r, weight, EPS, checkpoint=q_dtype, block=block, **v, **how, **out)
    g.check()
    J.check_forward(f, x, r, weight, EPS, **v, **how)
    if q_dtype is not None:
        J.check_checkpoint("saved_h", f.saved_h, f.h, q_dtype, block)
        if reads_x:
            J.check_checkpoint("saved_x", f.saved_x, x, q_dtype, block)
        else:
            assert f.saved_x is None
    return x, r, weight, v, how, f


def run_backward(T, H, x_dt, r_dt, S=1, which="wpg", post=True, dts=None, rs=1.0, bs=1.0, q_dtype=None, block=128, shift=0,
                 seed=1, with_dy=True, with_dh=True):
    """The backward pass against the formula, on tensors as a forward pass leaves them."""
    S = S if set(which) & set("gs") else 1
    v = vectors(H, S, x_dt, seed + 10, which, dts or (F32, x_dt, F32, x_dt))
    x, h = off((T, H), x_dt, seed, shift, 1.5, 0.1), off((T, H), r_dt, seed + 1, shift, 2.0, 0.2)
    rstd = J.inverse_rms(h.double(), EPS).float()
    post_rstd = J.inverse_rms(x.double(), EPS).float() if post else None
    dy = off((T, H), x_dt, seed + 2, shift, 0.5, 0.02) if with_dy else None
    dh = off((T, H), r_dt, seed + 3, shift, 0.5) if with_dh else None
    how = dict(post_norm=post, residual_scale=rs, branch_scale=bs)
    reads_x = post or v["gate"] is not None
    hs, xs = h, x
    h64, x64 = h.double(), x.double() if reads_x else None
    if q_dtype is not None:
        hs, xs = gn.gn_q8_quantize(h, q_dtype, block=block), gn.gn_q8_quantize(x, q_dtype, block=block)
        h64, x64 = J.decode(hs, block), J.decode(xs, block) if reads_x else None
    g = Guards()
    out = dict(dx=g.new("dx", (T, H), x_dt, shift), dres=g.new("dres", (T, H), r_dt, shift))
    weight = v.pop("weight")
    for name, t in (("dweight", weight), ("dpost_weight", v["post_weight"]), ("dgate", v["gate"]), ("dscale", v["scale"])):
        if t is not None:
            out[name] = g.new(name, t.shape, t.dtype)
    ws = torch.full((gn.gn_join_workspace_bytes(T, H, S),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN if read unwritten
    b = gn.gn_join_backward(dy, hs, rstd, weight, x=xs if reads_x else None, post_rstd=post_rstd, dh=dh, block=block,
                            x_dtype=x_dt, residual_dtype=r_dt, workspace=ws, **v, **how, **out)
    g.check()
    J.check_backward(b, J.backward(dy, dh, h64, x64, rstd, post_rstd, weight, **v, **how))
    return b


WIDTHS = [1, 2, 7, 8, 9, 31, 64, 100, 128, 255, 256, 511, 512, 520, 1001, 1152, 1531, 2048, 2056, 4096, 5120, 8192, 8200,
          10007, 16384, 32761, 32768]
PAIRS = [(BF, BF), (BF, F32), (F16, F16), (F16, F32), (F32, F32)]
NAMES = lambda v: str(v).replace("torch.", "")  # noqa: E731


# ------------------------------------------------------------------ forward

@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(H):
    for T, x_dt, r_dt, S, which, post, shift in ((1, BF, BF, 1, "wp", True, 0), (36, BF, BF, 4, "wpgs", True, 1),
                                                 (5, F16, F32, 5, "gs", False, 3), (6, F32, F32, 1, "", True, 1)):
        say(f"forward T={T} H={H} {x_dt} stream={r_dt} S={S} {which} post={post} shift={shift}")
        run_forward(T, H, x_dt, r_dt, S, which, post, shift=shift, rs=0.75 if H % 2 else 1.0)


@pytest.mark.parametrize("x_dt,r_dt", PAIRS, ids=NAMES)
@pytest.mark.parametrize("which", ["", "w", "wp", "wpg", "wgs", "wpgs", "s", "g"])
def test_forward_types(x_dt, r_dt, which):
    for (T, H), other in itertools.product(((6, 64), (132, 200), (9, 1024), (3, 12000)), (x_dt, F32)):
        say(f"forward {x_dt} {r_dt} {which} T={T} H={H} vectors {other}")
        run_forward(T, H, x_dt, r_dt, 3, which, "p" in which or H == 200, (other, x_dt, F32, other), 0.5, -1.5)


@pytest.mark.parametrize("q_dtype", [I8, E4], ids=NAMES)
@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_forward_checkpoints(q_dtype, block):
    for T, H, x_dt, r_dt, which, post, shift in (
            (1, 1, F32, F32, "wp", True, 0), (5, 7, BF, BF, "wg", False, 0), (18, 24, BF, BF, "w", True, 1),
            (20, 64, BF, F32, "wpgs", True, 0), (9, 100, F16, F32, "g", False, 3), (70, 128, BF, BF, "w", False, 0),
            (4, 520, BF, BF, "wpg", True, 0), (5, 1001, F32, F32, "wpg", True, 1), (16, 4096, F16, F16, "wpg", True, 0),
            (3, 5120, BF, F32, "wg", True, 0), (2, 8192, BF, BF, "wpg", True, 0), (2, 12345, BF, BF, "p", True, 5),
            (1, 32768, BF, BF, "wp", True, 0), (1, 32765, F32, F32, "wp", True, 0)):
        say(f"forward {q_dtype} block={block} T={T} H={H} {x_dt} stream={r_dt} {which} post={post}")
        run_forward(T, H, x_dt, r_dt, 1, which, post, q_dtype=q_dtype, block=block, shift=shift)


@pytest.mark.parametrize("x_dt,r_dt", PAIRS, ids=NAMES)
def test_a_plain_join_is_the_row_norm(x_dt, r_dt):
    for T, H in ((5, 64), (33, 1000), (7, 4096), (3, 20000)):
        x, r, w = rand((T, H), x_dt, 20), rand((T, H), r_dt, 21, 2.0), rand((H,), F32, 22, 0.2, 1.0)
        f = gn.gn_join_forward(x, r, w, EPS)
        y, h, rstd = gn.gn_rms_forward(x, w, EPS, residual=r)
        assert same(f.y, y) and same(f.h, h) and same(f.rstd, rstd) and f.post_rstd is None
        assert f.saved_h is None and f.saved_x is None


def test_in_place_and_parts():
    for T, H in ((33, 1536), (12, 100), (4, 20000)):
        x, r, w = rand((T, H), BF, 30), rand((T, H), BF, 31), rand((H,), BF, 32)
        how = dict(post_weight=rand((H,), F32, 33), gate=rand((3 if T % 3 == 0 else 1, H), BF, 34), residual_scale=0.5)
        f = gn.gn_join_forward(x, r, w, EPS, checkpoint=I8, **how)
        x2, r2 = x.clone(), r.clone()
        f2 = gn.gn_join_forward(x2, r2, w, EPS, out=x2, h=r2, checkpoint=I8, **how)
        assert f2.y is x2 and f2.h is r2
        for a, b in zip(f[:4] + f.saved_h + f.saved_x, f2[:4] + f2.saved_h + f2.saved_x):
            assert same(a, b)
        r3 = r.clone()
        f3 = gn.gn_join_forward(x, r3, None, EPS, h=r3, need_y=False, checkpoint=I8, **how)     # the stream alone
        assert f3.y is None and f3.rstd is None and f3.saved_h is None
        for a, b in ((f3.h, f.h), (f3.post_rstd, f.post_rstd), (f3.saved_x[0], f.saved_x[0])):
            assert same(a, b)
        f4 = gn.gn_join_forward(x, r, w, EPS, need_rstd=False, **how)
        assert f4.rstd is None and f4.post_rstd is None and same(f4.y, f.y)


def test_strided_rows_gates_and_scales():
    """Views as a program has them: x a slice of a wider projection, gate and scale slices of one
    modulation projection, by image."""
    B, L, H = 5, 7, 96
    wide, mod = rand((B, L, 3 * H + 4), BF, 40), rand((B, 1, 6 * H), BF, 41, 0.3)
    x, r, w = wide[..., 3:3 + H], rand((B, L, H), BF, 42), rand((H,), F32, 43)
    scale, gate = mod[..., H:2 * H], mod[..., 2 * H:3 * H]
    f = gn.gn_join_forward(x, r, w, EPS, post_norm=True, gate=gate, scale=scale)
    c = gn.gn_join_forward(x.contiguous(), r, w, EPS, post_norm=True, gate=gate.contiguous().view(B, H),
                           scale=scale.contiguous())
    assert f.y.shape == f.h.shape == x.shape and f.rstd.shape == (B, L)
    for a, b in zip(f[:4], c[:4]):
        assert same(a, b)
    J.check_forward(f, x, r, w, EPS, None, gate, scale, True)
    dy, dh = rand((B, L, H), BF, 44), rand((B, L, H), BF, 45)
    b1 = gn.gn_join_backward(dy, f.h, f.rstd, w, x=x, post_rstd=f.post_rstd, dh=dh, gate=gate, scale=scale)
    b2 = gn.gn_join_backward(dy, f.h, f.rstd, w, x=x.contiguous(), post_rstd=f.post_rstd, dh=dh, gate=gate.contiguous(),
                             scale=scale.contiguous())
    assert b1.dgate.shape == gate.shape and b1.dscale.shape == scale.shape and b1.dpost_weight.shape == (H,)
    for p, q in zip(b1, b2):
        assert same(p, q)
    J.check_backward(b1, J.backward(dy, dh, f.h.double().view(-1, H), x.double().reshape(-1, H), f.rstd, f.post_rstd, w,
                                    gate=gate, scale=scale, post_norm=True))


@pytest.mark.parametrize("H", [8, 100, 128, 1024, 4096, 12000])
def test_a_rows_bits_do_not_depend_on_the_batch(H):
    T = 300
    x, r, w, pw = rand((T, H), BF, 50), rand((T, H), BF, 51), rand((H,), BF, 52), rand((H,), BF, 53)
    gate = rand((T // 2, H), BF, 54)
    dy, dh = rand((T, H), BF, 55), rand((T, H), BF, 56)

    def go(a, b):
        how = dict(post_weight=pw, gate=gate[a // 2:b // 2])
        f = gn.gn_join_forward(x[a:b], r[a:b], w, EPS, checkpoint=I8, **how)
        g = gn.gn_join_backward(dy[a:b], f.h, f.rstd, w, x=x[a:b], post_rstd=f.post_rstd, dh=dh[a:b], **how)
        k = gn.gn_join_backward(dy[a:b], f.saved_h, f.rstd, w, x=f.saved_x, post_rstd=f.post_rstd, dh=dh[a:b], **how)
        return f[:4] + f.saved_h + f.saved_x + g[:2] + k[:2]

    every = go(0, T)
    for a, b in ((0, 2), (6, 10), (122, 300)):
        for p, q in zip(every, go(a, b)):
            assert same(p[a:b], q)


def test_special_values_stay_in_their_row():
    for H in (8, 200, 4096, 12000):
        T = 8
        x, r, w = rand((T, H), F32, 60), rand((T, H), F32, 61), rand((H,), F32, 62, 0.1, 1.0)
        x[1, 3], r[2, H - 1], x[3, 0], r[4], x[4] = float("nan"), float("inf"), -float("inf"), 0.0, 0.0
        x[5] *= 1e-30
        dy, dh = rand((T, H), F32, 63), rand((T, H), F32, 64)
        dy[6, 1], dh[7, H - 2] = float("nan"), float("inf")
        say(f"special values H={H}")
        f = gn.gn_join_forward(x, r, w, EPS, post_weight=w, checkpoint=I8, block=32)
        fine = [0, 4, 5, 6, 7]
        J.check_forward(gn.JoinForward(f.y[fine], f.h[fine], f.rstd[fine], f.post_rstd[fine], None, None), x[fine], r[fine],
                        w, EPS, w, None, None, True)
        assert bool(torch.isnan(f.h[1]).all()) and bool(torch.isnan(f.y[1]).all())
        assert float(f.rstd[2]) == 0 and bool(torch.isnan(f.y[2, H - 1])) and float(f.y[2, :H - 1].abs().max()) == 0
        assert bool(torch.isnan(f.h[3, 0])) and torch.equal(f.h[3, 1:], r[3, 1:])     # 0 * inf there, zeros beside it
        J.check_checkpoint("saved_h", f.saved_h, f.h, I8, 32)
        J.check_checkpoint("saved_x", f.saved_x, x, I8, 32)
        for saved in ((f.h, x), (f.saved_h, f.saved_x)):
            g = gn.gn_join_backward(dy, saved[0], f.rstd, w, x=saved[1], post_rstd=f.post_rstd, dh=dh, post_weight=w, block=32)
            ref = J.backward(dy, dh, *(t.double() if isinstance(t, torch.Tensor) else J.decode(t, 32) for t in saved), f.rstd,
                             f.post_rstd, w, w, post_norm=True)
            good = [0, 4, 5]
            for name in ("dx", "dres"):
                t, (v, e) = getattr(g, name), ref[name]
                J.close(name, t[good], v[good], e[good] * 1.01 + J.half_step(v[good].abs() + e[good], F32) + 1e-37)
                assert not bool(torch.isfinite(t[6]).any())
            assert bool(torch.isnan(g.dx[7]).all()) or not bool(torch.isfinite(g.dx[7]).all())
            finite = torch.isfinite(g.dres[7])
            assert not bool(finite[H - 2]) and int(finite.sum()) == H - 1


def test_gate_and_stream_that_are_shut():
    """A gate of zeros leaves the scaled stream, a residual scale of zero the branch."""
    T, H = 9, 520
    x, r, w = rand((T, H), BF, 70), rand((T, H), BF, 71), rand((H,), BF, 72)
    f = gn.gn_join_forward(x, r, w, EPS, post_norm=True, gate=torch.zeros(H, dtype=BF, device="cuda"))
    assert torch.equal(f.h, r)
    f = gn.gn_join_forward(x, r, w, EPS, branch_scale=0.0)
    assert torch.equal(f.h, r)
    f = gn.gn_join_forward(x, r, w, EPS, residual_scale=0.0)
    assert torch.equal(f.h, x)


# ------------------------------------------------------------------ checkpoints by themselves

@pytest.mark.parametrize("q_dtype", [I8, E4], ids=NAMES)
@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_quantize(q_dtype, block):
    for T, H, dt, shift, size in ((1, 1, F32, 0, 1.0), (5, 7, BF, 0, 1.0), (900, 24, BF, 1, 3.0), (333, 64, F16, 3, 1.0),
                                  (70, 100, F32, 1, 1e-20), (40, 129, BF, 0, 1.0), (64, 520, F32, 0, 1e-37),
                                  (33, 1531, BF, 1, 1.0), (16, 4096, F16, 0, 1e-4), (5, 12345, BF, 5, 1e30),
                                  (3, 32768, BF, 0, 1.0), (3, 32767, F32, 0, 1.0)):
        say(f"quantize {q_dtype} block={block} T={T} H={H} {dt}")
        x = off((T, H), dt, 80, shift, size, 0.1 * size)
        g = Guards()
        n = -(-H // block) if block else 1
        q, s = g.new("q", (T, H), q_dtype, shift), g.new("scale", (T, n), F32)
        got = gn.gn_q8_quantize(x, block=block, out=q, scale=s)
        assert got[0] is q and got[1] is s
        g.check()
        J.check_checkpoint("q", (q, s), x, q_dtype, block)
        v = gn.gn_q8_dequantize(q, s, block=block)
        assert torch.equal(v.double(), J.decode((q, s), block).float().double())


def test_quantize_layouts_and_special_values():
    wide = rand((6, 5, 300), BF, 81)
    for x in (wide[..., 100:228], wide[..., 1:300], wide[:, :1, 3:40], rand((40,), F16, 82), rand((0, 16), BF, 83)):
        q, s = gn.gn_q8_quantize(x, E4, block=32)
        assert q.shape == x.shape and s.shape == x.shape[:-1] + (-(-x.shape[-1] // 32),)
        for a, b in zip((q, s), gn.gn_q8_quantize(x.contiguous(), E4, block=32)):
            assert same(a, b)
    x = rand((6, 200), F32, 84)
    x[1, 3], x[2, 199], x[3], x[4, 64] = float("nan"), float("inf"), 0.0, -float("inf")
    for dt, block in itertools.product((I8, E4), (0, 32, 64, 128)):
        J.check_checkpoint("q", gn.gn_q8_quantize(x, dt, block=block), x, dt, block)


# ------------------------------------------------------------------ backward

@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H):
    for T, x_dt, r_dt, S, which, post, q, block in (
            (1, BF, BF, 1, "wp", True, None, 128), (66, BF, BF, 3, "wpgs", True, None, 128), (5, F32, F32, 5, "wgs", False, None, 128),
            (12, BF, BF, 1, "wpg", True, I8, 32), (6, F16, F32, 2, "wpg", True, E4, 0)):
        say(f"backward T={T} H={H} {x_dt} stream={r_dt} S={S} {which} post={post} {q} {block}")
        run_backward(T, H, x_dt, r_dt, S, which, post, q_dtype=q, block=block, shift=1 if H % 3 == 0 else 0)


@pytest.mark.parametrize("x_dt,r_dt", PAIRS, ids=NAMES)
@pytest.mark.parametrize("which", ["", "w", "wp", "wpg", "wgs", "wpgs", "s", "g"])
def test_backward_types(x_dt, r_dt, which):
    for (T, H), q, post in itertools.product(((6, 64), (132, 200), (9, 1024), (3, 9000)), (None, I8), (False, True)):
        if "p" in which and not post:
            continue
        say(f"backward {x_dt} {r_dt} {which} T={T} H={H} post={post} {q}")
        run_backward(T, H, x_dt, r_dt, 3, which, post, (x_dt, F32, x_dt, F32), 0.5, -1.5, q_dtype=q, block=64)


@pytest.mark.parametrize("with_dy,with_dh", [(True, False), (False, True)])
def test_backward_of_one_gradient_alone(with_dy, with_dh):
    for (T, H), (x_dt, r_dt), post, which, q in itertools.product(((9, 64), (30, 1000), (4, 9000)), ((BF, BF), (F16, F32)),
                                                                  (False, True), ("w", "wgs"), (None, E4)):
        say(f"backward dy={with_dy} dh={with_dh} T={T} H={H} {x_dt} {r_dt} post={post} {which} {q}")
        run_backward(T, H, x_dt, r_dt, 1, which, post, q_dtype=q, with_dy=with_dy, with_dh=with_dh)


@pytest.mark.parametrize("T,H,S", [(100000, 64, 1), (40000, 128, 400), (5000, 100, 2500), (3000, 1024, 3000), (2050, 4096, 2),
                                   (1500, 10000, 15), (1001, 520, 7), (900, 256, 300)])
def test_backward_many_rows(T, H, S):
    say(f"backward T={T} H={H} S={S}")
    run_backward(T, H, BF, BF, S, "wpgs", True, seed=50)
    run_backward(T, H, F16, F32, S, "wgs", False, seed=51)
    run_backward(T, H, BF, BF, S, "wpg", True, q_dtype=I8, block=64, seed=52)


def test_a_gate_for_all_beside_scales_for_each():
    T, H, S = 60, 200, 5
    x, h, dy, dh = (rand((T, H), BF, 90 + i) for i in range(4))
    w, gate, scale = rand((H,), F32, 94), rand((H,), BF, 95), rand((S, H), BF, 96)
    rstd = J.inverse_rms(h.double(), EPS).float()
    for g, s in ((gate, scale), (scale, gate)):
        b = gn.gn_join_backward(dy, h, rstd, w, x=x, dh=dh, gate=g, scale=s)
        assert b.dgate.shape == g.shape and b.dscale.shape == s.shape
        J.check_backward(b, J.backward(dy, dh, h.double(), x.double(), rstd, None, w, gate=g, scale=s))
        f = gn.gn_join_forward(x, h, w, EPS, gate=g, scale=s)
        J.check_forward(f, x, h, w, EPS, None, g, s)


def test_backward_parts_in_place_and_bits():
    for T, H in ((700, 1536), (90, 100), (40, 12000)):
        x, h, dy, dh = (rand((T, H), BF, 100 + i) for i in range(4))
        w, pw, gate = rand((H,), BF, 104, 0.2, 1.0), rand((H,), F32, 105), rand((2, H), BF, 106)
        f = gn.gn_join_forward(x, h, w, EPS, post_weight=pw, gate=gate)
        how = dict(post_rstd=f.post_rstd, post_weight=pw, gate=gate)
        b = gn.gn_join_backward(dy, h, f.rstd, w, x=x, dh=dh, **how)
        again = gn.gn_join_backward(dy, h, f.rstd, w, x=x, dh=dh, **how)
        for p, q in zip(b[:5], again[:5]):
            assert same(p, q)
        assert b.dscale is None
        none = dict(need_dx=False, need_dres=False, need_dweight=False, need_dpost_weight=False, need_dgate=False)
        for name in ("dx", "dres", "dweight", "dpost_weight", "dgate"):
            one = gn.gn_join_backward(dy, h, f.rstd, w, x=x, dh=dh, **how, **{**none, "need_" + name: True})
            assert same(getattr(one, name), getattr(b, name)) and sum(t is not None for t in one) == 1, name
        for place, target in (("dy", "dx"), ("x", "dx"), ("dh", "dres"), ("h", "dres")):
            t = dict(dy=dy.clone(), x=x.clone(), dh=dh.clone(), h=h.clone())
            g = gn.gn_join_backward(t["dy"], t["h"], f.rstd, w, x=t["x"], dh=t["dh"], **how, **{target: t[place]})
            for p, q in zip(b[:5], g[:5]):
                assert same(p, q), (place, target)


def test_backward_of_no_rows():
    w, gate = rand((64,), BF, 110), rand((3, 64), BF, 111)
    e = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    b = gn.gn_join_backward(e(BF, 0, 64), e(BF, 0, 64), e(F32, 0), w, x=e(BF, 0, 64), dh=e(BF, 0, 64), gate=gate)
    assert b.dx.shape == (0, 64) and torch.equal(b.dweight, torch.zeros_like(w)) and torch.equal(b.dgate, torch.zeros_like(gate))
    f = gn.gn_join_forward(e(BF, 0, 64), e(BF, 0, 64), w, checkpoint=I8, gate=gate)
    assert f.y.shape == (0, 64) and f.saved_h[0].shape == (0, 64)


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes_and_types(seed):
    rng = random.Random(seed)
    H = rng.choice([rng.randint(1, 70), rng.randint(1, 600), rng.randint(500, 5000), rng.randint(4000, 32768)])
    T = max(1, min(rng.randint(1, 2000), 1_500_000 // H))
    S = rng.choice([1, 1, rng.randint(1, T)])
    T = T // S * S
    x_dt, r_dt = rng.choice(PAIRS)
    which, post = "".join(c for c in "wpgs" if rng.random() < 0.6), rng.random() < 0.6
    post = post or "p" in which
    dts = [rng.choice([x_dt, F32]) for _ in range(4)]
    rs, bs, shift = rng.choice([1.0, 0.7]), rng.choice([1.0, -0.3]), rng.randint(0, 7)
    q, block = rng.choice([None, I8, E4]), rng.choice([0, 32, 64, 128])
    say(f"seed {seed}: T={T} H={H} S={S} {x_dt} {r_dt} {which} post={post} {dts} {q} {block} shift={shift}")
    run_forward(T, H, x_dt, r_dt, S, which, post, dts, rs, bs, q, block, shift, seed)
    run_backward(T, H, x_dt, r_dt, S, which, post, dts, rs, bs, q, block, shift, seed)


def test_offsets_past_32_bits():
    T, H = 70001, 32760                      # 2.3e9 elements, 4.6 GB a tensor
    say(f"{T} x {H} bf16")
    x = torch.empty(T, H, dtype=BF, device="cuda")
    part = rand((1000, H), BF, 191)
    for k in range(0, T, 1000):
        x[k:k + 1000] = part[:min(1000, T - k)]
    w, pw = rand((H,), BF, 192, 0.2, 1.0), rand((H,), BF, 193, 0.2, 1.0)
    want = gn.gn_join_forward(part, part, w, EPS, post_weight=pw, checkpoint=I8)
    f = gn.gn_join_forward(x, x, w, EPS, post_weight=pw, checkpoint=I8)
    rows = [(k, min(1000, T - k)) for k in (0, 65000, 66000, 70000)]    # before and behind 2^31 elements (row 65552)
    for k, n in rows:
        for a, b in zip(f[:4] + f.saved_h + f.saved_x, want[:4] + want.saved_h + want.saved_x):
            assert same(a[k:k + n], b[:n])
    q, s = gn.gn_q8_quantize(x, I8)
    for k, n in rows:
        assert same(q[k:k + n], want.saved_x[0][:n]) and same(s[k:k + n], want.saved_x[1][:n])
    del q
    for saved, saved_part in (((f.h, x), (want.h, part)), ((f.saved_h, f.saved_x), (want.saved_h, want.saved_x))):
        how = dict(post_weight=pw, need_dweight=False, need_dpost_weight=False)
        b = gn.gn_join_backward(x, saved[0], f.rstd, w, x=saved[1], post_rstd=f.post_rstd, dh=x, dx=f.y.fill_(7), **how)
        ref = gn.gn_join_backward(part, saved_part[0], want.rstd, w, x=saved_part[1], post_rstd=want.post_rstd, dh=part, **how)
        for k, n in rows:
            assert same(b.dx[k:k + n], ref.dx[:n]) and same(b.dres[k:k + n], ref.dres[:n])
        del b


# Calls past the last-level cache load their rows with another policy.
@pytest.mark.parametrize("T,H,x_dt,r_dt", [(9000, 4096, BF, BF), (40000, 1001, F16, F16), (300000, 128, BF, F32),
                                           (3000, 16384, BF, BF), (5000, 4096, F32, F32), (9000, 4096, F16, F32)], ids=NAMES)
def test_past_the_cache(T, H, x_dt, r_dt):
    say(f"past the cache T={T} H={H} {x_dt} {r_dt}")
    run_forward(T, H, x_dt, r_dt, 1, "wpg", True)
    run_backward(T, H, x_dt, r_dt, 1, "wpg", True)
    run_backward(T, H, x_dt, r_dt, T // 1000, "wgs", False, q_dtype=I8, block=0)


# ------------------------------------------------------------------ autograd, streams, graphs

@pytest.mark.parametrize("x_dt,r_dt", [(F32, F32), (BF, BF), (F16, F32)], ids=NAMES)
@pytest.mark.parametrize("post,which", [(True, "wpgs"), (False, "wg"), (True, "w"), (False, "")])
def test_autograd_against_the_formula_and_differences(x_dt, r_dt, post, which):
    B, L, H = 2, 3, 40
    v = vectors(H, B, x_dt, 200, which, (F32, F32, F32, F32))
    leaves = [rand((B, L, H), x_dt, 210), rand((B, L, H), r_dt, 211)] + [v[k] for k in ("weight", "post_weight", "gate", "scale")]
    leaves = [t if t is None else t.requires_grad_() for t in leaves]
    x, r, w, pw, gate, scale = leaves
    a, b = rand((B, L, H), F32, 212), rand((B, L, H), F32, 213)
    y, h = gn.join_norm(x, r, w, EPS, post_weight=pw, gate=gate, scale=scale, post_norm=post, residual_scale=0.75, branch_scale=1.25)
    given = [k for k, t in enumerate(leaves) if t is not None]
    grads = torch.autograd.grad((y.float() * a).sum() + (h.float() * b).sum(), [leaves[k] for k in given])

    def f(vals):   # the loss in fp64, without roundings
        x, r, w, pw, gate, scale = (vals.get(k) for k in range(6))
        u = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() if post else x
        u = u if pw is None else u * pw
        u = u if gate is None else u * gate[:, None]
        hh = 0.75 * r + 1.25 * u
        yy = hh * (hh.square().mean(-1, keepdim=True) + EPS).rsqrt()
        yy = yy if w is None else yy * w
        yy = yy if scale is None else yy * (1 + scale[:, None])
        return (yy * a.double()).sum() + (hh * b.double()).sum()

    base = {k: leaves[k].detach().double() for k in given}
    exact = {k: t.clone().requires_grad_() for k, t in base.items()}
    f(exact).backward()
    # Inputs in 16 bits: h is rounded in the kernel and the gradient of y arrives rounded, an
    # eps of each; the fp32 case has its own roundings alone.
    tol = 1e-5 if x_dt == F32 else 4 * torch.finfo(x_dt).eps
    step = 1e-5
    for g, k in zip(grads, given):
        assert g.dtype == leaves[k].dtype and g.shape == leaves[k].shape
        rel = float((g.double() - exact[k].grad).norm() / exact[k].grad.norm())
        say(f"gradient {k}: {rel:.2e} from the formula's")
        assert rel < tol, k
        d = torch.randn(base[k].shape, generator=torch.Generator().manual_seed(k), dtype=torch.float64).cuda()
        lo, hi = dict(base), dict(base)
        lo[k], hi[k] = base[k] - step * d, base[k] + step * d
        diff = float((f(hi) - f(lo)) / (2 * step))
        got = float((g.double() * d).sum())
        size = float((g.double() * d).norm()) * d.numel() ** 0.5
        assert abs(got - diff) <= max(tol, 1e-7) * max(size, 1.0), (k, got, diff)


@pytest.mark.parametrize("q_dtype", [I8, E4], ids=NAMES)
def test_autograd_from_checkpoints(q_dtype):
    """The graph's gradients are those of the checkpoints' values, and close to the graph's without."""
    B, L, H = 3, 50, 520
    t = [rand((B, L, H), BF, 220), rand((B, L, H), F32, 221), rand((H,), F32, 222, 0.2, 1.0), rand((H,), BF, 223, 0.2, 1.0),
         rand((B, 1, H), BF, 224), rand((B, 1, H), BF, 225, 0.2)]
    dy, dh = rand((B, L, H), BF, 226), rand((B, L, H), F32, 227)

    def grads(**kw):
        x, r, w, pw, g, s = leaves = [v.clone().requires_grad_() for v in t]
        y, h = gn.join_norm(x, r, w, post_weight=pw, gate=g, scale=s, **kw)
        return torch.autograd.grad([y, h], leaves, [dy, dh])

    x, r, w, pw, g, s = t
    f = gn.gn_join_forward(x, r, w, post_weight=pw, gate=g, scale=s, checkpoint=q_dtype, block=64)
    want = gn.gn_join_backward(dy, f.saved_h, f.rstd, w, x=f.saved_x, post_rstd=f.post_rstd, dh=dh, post_weight=pw, gate=g,
                               scale=s, block=64)
    got, plain = grads(checkpoint=q_dtype, block=64), grads()
    # a value is off by half a quantum of its run's largest, and a gradient is made of sums of such products
    far = 0.5 / 127 * 4 if q_dtype == I8 else 2.0 ** -4
    for p, q, e in zip(got, want, plain):
        assert same(p, q)
        assert float((p.double() - e.double()).norm() / e.double().norm()) < far


def test_autograd_partial_uses():
    x, r = rand((4, 5, 64), BF, 230).requires_grad_(), rand((4, 5, 64), F32, 231).requires_grad_()
    w, pw = rand((64,), BF, 232).requires_grad_(), rand((64,), BF, 233).requires_grad_()
    for ckpt in (None, I8):
        y, h = gn.join_norm(x, r, w, post_weight=pw, checkpoint=ckpt)
        gx, gr, gw, gp = torch.autograd.grad(h.sum(), [x, r, w, pw], retain_graph=True)
        assert torch.equal(gr, torch.ones_like(r)) and float(gw.abs().max()) == 0 and float(gx.abs().max()) > 0
        gx, gr, gw, gp = torch.autograd.grad(y.float().sum(), [x, r, w, pw])
        assert all(bool(torch.isfinite(g).all()) for g in (gx, gr, gw, gp))
    # only some leaves; rows that are not evenly spaced; a transposed gradient; broadcast inputs
    z = rand((5, 4, 64), BF, 234).transpose(0, 1).requires_grad_()
    y, h = gn.join_norm(z, r.detach().transpose(0, 1).contiguous().transpose(0, 1))
    assert same(y, gn.gn_join_forward(z.detach().contiguous(), r.detach(), None)[0])
    (y.float().transpose(0, 1) * rand((5, 4, 64), F32, 235)).sum().backward()
    v, s = rand((64,), BF, 236).requires_grad_(), rand((1, 64), BF, 237).requires_grad_()
    y, h = gn.join_norm(v.expand(6, 64), r.detach().view(-1, 64)[:6], gate=s.expand(3, 64))
    (y.float().sum() + h.sum()).backward()
    assert z.grad.shape == z.shape and v.grad.shape == v.shape and s.grad.shape == s.shape
    with torch.no_grad():
        assert not gn.join_norm(x, r, w)[0].requires_grad
    with pytest.raises(RuntimeError):                     # no second derivative
        y, _ = gn.join_norm(x, r, w)
        (g,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
        g.float().sum().backward()


def test_the_stream_alone_beside_special_values():
    """Where only h is used, the norm before the next block has no part, whatever the rows hold."""
    for x_dt, r_dt in ((BF, BF), (F16, F32), (F32, F32)):
        x, r = rand((5, 64), x_dt, 240), rand((5, 64), r_dt, 241)
        r[1, 3], r[2, 5], r[3] = float("nan"), float("inf"), 0.0
        x[3] = 0.0
        x.requires_grad_(), r.requires_grad_()
        dh = rand((5, 64), r_dt, 242)
        _, h = gn.join_norm(x, r, None, 0.0)
        gx, gr = torch.autograd.grad(h, [x, r], dh)
        assert same(gr, dh) and same(gx, dh.to(x_dt))


def test_saved_tensors_that_a_later_call_overwrites():
    def graph(ckpt=None):
        x, r, w = rand((6, 96), BF, 250).requires_grad_(), rand((6, 96), F32, 251), rand((96,), BF, 252)
        return gn.join_norm(x, r, w, checkpoint=ckpt), x.detach(), w

    (y, h), x, w = graph()
    gn.gn_join_forward(x, h.detach(), w, h=h.detach())                    # the stream in place
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    (y, h), x, w = graph(I8)
    gn.gn_join_forward(x, h.detach(), w, h=h.detach())                    # kept in 8 bits: the stream may go on in place
    y.float().sum().backward()


def blocks(n, B, L, H, dt, seed):
    """Two blocks' worth of joins one behind the other, as a model runs them: leaves, and the step."""
    mod = rand((B, 1, 2 * n * H), dt, seed, 0.3)
    w = [rand((H,), F32, seed + 1 + k, 0.1, 1.0) for k in range(2 * n)]
    mix = [rand((H, H), dt, seed + 40 + k, H ** -0.5) for k in range(n)]
    return [mod] + w + mix


def chain(leaves, stream, n, ckpt):
    mod, w, mix = leaves[0], leaves[1:1 + 2 * n], leaves[1 + 2 * n:]
    H = stream.shape[-1]
    y, h = gn.rms_norm(stream, w[0]), stream
    for k in range(n):
        x = torch.nn.functional.silu(y @ mix[k])                          # the block
        gate, scale = mod[..., 2 * k * H:(2 * k + 1) * H], mod[..., (2 * k + 1) * H:(2 * k + 2) * H]
        y, h = gn.join_norm(x, h, w[2 * k + 1], post_weight=w[(2 * k + 2) % (2 * n)], gate=gate, scale=scale,
                            checkpoint=ckpt)
    return (y.float().square().mean() + h.float().mean())


@pytest.mark.parametrize("ckpt", [None, I8, E4], ids=NAMES)
def test_a_chain_of_blocks_trains(ckpt):
    """Norm, block, join, block, join, backward through all of it and clipping: against the same in
    fp64 with torch's own operations."""
    n, B, L, H = 2, 3, 17, 64
    for dt in (F32, BF):
        stream = rand((B, L, H), F32 if dt == F32 else BF, 300).requires_grad_()
        leaves = [t.requires_grad_() for t in blocks(n, B, L, H, dt, 301)]
        loss = chain(leaves, stream, n, ckpt)
        grads = torch.autograd.grad(loss, leaves + [stream])

        def norm(v, w):
            return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w

        ref = [t.detach().double().requires_grad_() for t in leaves + [stream]]
        mod, w, mix, h = ref[0], ref[1:1 + 2 * n], ref[1 + 2 * n:-1], ref[-1]
        y = norm(h, w[0])
        for k in range(n):
            x = torch.nn.functional.silu(y @ mix[k])
            gate, scale = mod[..., 2 * k * H:(2 * k + 1) * H], mod[..., (2 * k + 1) * H:(2 * k + 2) * H]
            h = h + gate * norm(x, w[(2 * k + 2) % (2 * n)])
            y = norm(h, w[2 * k + 1]) * (1 + scale)
        exact = torch.autograd.grad(y.square().mean() + h.mean(), ref)
        # fp32: the products' and norms' roundings; bf16: a dozen roundings of 2^-8 along the chain; 8 bits: half
        # a quantum of the run's largest value (int8: 1/254 of up to 4 times the rest), e4m3's 2^-4 of the value
        tol = {None: 1e-5, I8: 0.05, E4: 0.15}[ckpt] + (0.08 if dt == BF else 0.0)
        for k, (g, e) in enumerate(zip(grads, exact)):
            rel = float((g.double() - e).norm() / e.norm())
            say(f"{ckpt} {dt} leaf {k}: {rel:.2e}")
            assert rel < tol, k
        params = [torch.nn.Parameter(t.detach().clone()) for t in leaves]
        for p, g in zip(params, grads):
            p.grad = g.clone()
        total = gn.clip_gradients(params, 1e-3)
        assert abs(float(total) - float(torch.stack([g.double().norm() for g in grads[:-1]]).norm())) < 1e-5 * float(total)


def test_on_another_stream_and_queued():
    x, r, w, pw = (rand((2048, 2048), BF, 260 + i) for i in range(2)) and [rand((2048, 2048), BF, 260), rand((2048, 2048), BF, 261),
                                                                           rand((2048,), BF, 262), rand((2048,), BF, 263)]
    want = gn.gn_join_forward(x, r, w, post_weight=pw, checkpoint=I8)
    side = torch.cuda.Stream()
    src = torch.ones(1 << 27, dtype=torch.int32, device="cuda")           # 512 MiB
    dst = torch.empty_like(src)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(side):
        for _ in range(32):                                               # about 5 ms of copies in front
            dst.copy_(src)
        f = gn.gn_join_forward(x, r, w, post_weight=pw, checkpoint=I8)
        b = gn.gn_join_backward(x, f.saved_h, f.rstd, w, x=f.saved_x, post_rstd=f.post_rstd, dh=r, post_weight=pw)
        done.record()
    assert not done.query(), "the calls returned only after the queued work had run"
    torch.cuda.synchronize()
    for p, q in zip(f[:4] + f.saved_h + f.saved_x, want[:4] + want.saved_h + want.saved_x):
        assert same(p, q)
    for p, q in zip(b[:4], gn.gn_join_backward(x, f.saved_h, f.rstd, w, x=f.saved_x, post_rstd=f.post_rstd, dh=r, post_weight=pw)[:4]):
        assert same(p, q)


def test_captured_and_replayed():
    """Two captured graphs with a workspace each, replayed in turn with new inputs and eager work
    between, against eager calls."""
    T, H, S = 96, 1152, 3

    class Graph:
        def __init__(self, seed, ckpt):
            self.ckpt = ckpt
            self.t = [rand((T, H), BF, seed + i) for i in range(4)]
            self.v = dict(post_weight=rand((H,), BF, seed + 5), gate=rand((S, H), BF, seed + 6), scale=rand((S, H), BF, seed + 7))
            self.w = rand((H,), F32, seed + 8)
            self.ws = torch.empty(gn.gn_join_workspace_bytes(T, H, S), dtype=torch.uint8, device="cuda")
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step()
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self.step()

        def step(self):
            x, r, dy, dh = self.t
            f = gn.gn_join_forward(x, r, self.w, checkpoint=self.ckpt, **self.v)
            saved = (f.h, x) if self.ckpt is None else (f.saved_h, f.saved_x)
            b = gn.gn_join_backward(dy, saved[0], f.rstd, self.w, x=saved[1], post_rstd=f.post_rstd, dh=dh, workspace=self.ws, **self.v)
            return f[:4] + b

    graphs = [Graph(400, None), Graph(420, I8)]
    for turn in range(3):
        for k, g in enumerate(graphs):
            for i, t in enumerate(g.t):
                t.copy_(rand((T, H), BF, 440 + 10 * turn + 5 * k + i))
            for t in g.out:
                t.fill_(float("nan"))
            g.ws.fill_(0xFF)
        for g in graphs:
            g.graph.replay()
        torch.cuda.synchronize()
        for g in graphs:
            for a, b in zip(g.out, g.step()):
                assert same(a, b), turn


def test_an_eager_graph_of_the_same_leaf_while_capturing():
    x, r = rand((8, 64), BF, 270).requires_grad_(), rand((8, 64), BF, 271)
    y, h = gn.join_norm(x, r)                             # alive, on the default stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="eager graph of the same leaf"):
        with torch.cuda.graph(graph):
            gn.join_norm(x, r)
    del y, h
    torch.cuda.synchronize()


# ------------------------------------------------------------------ refusals

def test_c_abi_refuses_memory_of_the_host():
    from unet_groupnorm_amd._lib import GnJoin
    T, H = 4, 64
    j = GnJoin(T=T, H=H, samples=1, x_stride=H, x_dtype=1, r_dtype=1, w_dtype=0, post_dtype=0, gate_dtype=0, scale_dtype=0,
               post_norm=1, q_dtype=0, eps=1e-6, residual_scale=1.0, branch_scale=1.0)
    m = {k: rand((T, H), BF, 280 + i) for i, k in enumerate(("x", "res", "y", "h", "dy", "dh", "dx", "dres"))}
    m.update({k: rand((H,), F32, 290 + i) for i, k in enumerate(("w", "post", "gate", "scale", "dw", "dpost", "dgate", "dscale"))})
    m.update({k: rand((T,), F32, 300 + i).abs() for i, k in enumerate(("rstd", "prstd", "hs", "xs"))})
    m.update({k: torch.zeros(T, H, dtype=I8, device="cuda") for k in ("hq", "xq")})
    m["ws"] = torch.empty(lib.gn_join_workspace_bytes(T, H, 1), dtype=torch.uint8, device="cuda")
    pinned, host = torch.zeros(1 << 16, pin_memory=True), torch.zeros(1 << 16)
    fwd = ("x", "res", "w", "post", "gate", "scale", "y", "h", "rstd", "prstd", "hq", "hs", "xq", "xs")
    bwd = ("dy", "dh", "hq", "hs", "xq", "xs", "rstd", "prstd", "w", "post", "gate", "scale", "dx", "dres", "dw", "dpost",
           "dgate", "dscale", "ws")

    def call(names, **kw):
        p = [kw.get(k, m[k]).data_ptr() for k in names]
        if names is fwd:
            return lib.gn_join_forward(j, *p, None)
        return lib.gn_join_backward(j, *p, m["ws"].numel(), None)

    for names in (fwd, bwd):
        assert call(names) == 0
        for name in names:
            for bad in (pinned, host):
                assert call(names, **{name: bad}) == 8, name
    for k, bad in itertools.product(range(3), (pinned, host)):
        p = [m["x"], m["xq"], m["xs"]]
        p[k] = bad
        assert lib.gn_q8_quantize(p[0].data_ptr(), 1, H, T, H, 0, p[1].data_ptr(), 0, p[2].data_ptr(), None) == 8
    torch.cuda.synchronize()


def test_refusals_on_the_device():
    x, r = rand((4, 64), BF, 310), rand((4, 64), BF, 311)
    for call in (lambda: gn.gn_join_forward(x, r.cpu(), None), lambda: gn.gn_join_forward(x, r, torch.ones(64)),
                 lambda: gn.gn_join_forward(x, r, None, gate=torch.ones(64)),
                 lambda: gn.gn_join_backward(x, r, torch.ones(4), None), lambda: gn.gn_join_backward(x, r, rand((4,), F32, 1), None, dh=x.cpu()),
                 lambda: gn.gn_q8_quantize(x, out=torch.zeros(4, 64, dtype=I8)),
                 lambda: gn.gn_join_forward(x, r, None, out=r), lambda: gn.gn_join_forward(x, r, None, h=x)):
        with pytest.raises((ValueError, GnError)):
            call()
