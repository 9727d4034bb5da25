"""The residual join's and the checkpoints' entry points on a host without a GPU: every declared
symbol is exported, the struct is the header's, invalid arguments are refused with the documented
status before anything touches the device, and the binding refuses tensors of the wrong sizes,
dtypes or layouts."""
import ctypes
import os
import random
import re

import pytest
import torch

import unet_groupnorm_amd as gn
from unet_groupnorm_amd._lib import GN_BF16, GN_F16, GN_F32, JOIN_STATUS_NAMES, GnJoin, lib
from unet_groupnorm_amd.gn import GnError

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gn_join.h")
BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
NAN = float("nan")


def at(k, off=0):
    """A fake aligned address; the checks below never look behind it. 1 MiB apart."""
    return ctypes.c_void_p(0x10000000 + (k << 20) + off)


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(gn_[a-z_0-9]+)\s*\(", text, flags=re.M))
    assert names == {"gn_q8_quantize", "gn_join_forward", "gn_join_workspace_bytes", "gn_join_backward"}
    for name in names:
        assert hasattr(lib, name), name


def test_status_names_match_the_header():
    text = open(HEADER).read()
    for code, name in JOIN_STATUS_NAMES.items():
        assert re.search(rf"\b{name}\s*=\s*{code}\b", text), name
        assert lib.gn_ops_status_string(code) != b"unknown status"


def test_the_struct_matches_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct gn_join \{(.*?)\} gn_join;", text, re.S).group(1)
    width = {"int64_t": 8, "int32_t": 4, "float": 4}
    fields = []
    for decl in body.split(";"):
        if decl.strip():
            ctype, names = decl.strip().split(None, 1)
            fields += [(n.strip(), width[ctype]) for n in names.split(",")]
    assert fields == [(n, ctypes.sizeof(t)) for n, t in GnJoin._fields_]


def desc(**kw):
    a = dict(T=4, H=64, samples=1, x_stride=64, gate_stride=0, scale_stride=0, block=0, x_dtype=GN_BF16, r_dtype=GN_BF16,
             w_dtype=GN_BF16, post_dtype=GN_BF16, gate_dtype=GN_BF16, scale_dtype=GN_BF16, post_norm=1, q_dtype=0, eps=1e-6,
             residual_scale=1.0, branch_scale=1.0)
    a.update(kw)
    return GnJoin(**a)


FWD = dict(x=at(0), res=at(1), w=at(2), post=at(3), gate=at(4), scale=at(5), y=at(6), h=at(7), rstd=at(8), prstd=at(9), hq=at(10),
           hs=at(11), xq=at(12), xs=at(13))
BWD = dict(dy=at(0), dh=at(1), h=at(2), hs=None, x=at(3), xs=None, rstd=at(4), prstd=at(5), w=at(6), post=at(7), gate=at(8),
           scale=at(9), dx=at(10), dres=at(11), dw=at(12), dpost=at(13), dgate=at(14), dscale=at(15), ws=at(20))


def split(kw, names):
    return {k: v for k, v in kw.items() if k in names}, {k: v for k, v in kw.items() if k not in names}


def fwd(**kw):
    p, d = split(kw, FWD)
    return lib.gn_join_forward(desc(**d), *{**FWD, **p}.values(), None)


def bwd(wsb=1 << 24, **kw):
    p, d = split(kw, BWD)
    return lib.gn_join_backward(desc(**d), *{**BWD, **p}.values(), wsb, None)


SHAPE = [(dict(T=-1), 32), (dict(H=0), 32), (dict(H=32769, x_stride=32769), 32), (dict(x_stride=63), 32), (dict(T=1 << 45), 32),
         (dict(samples=0), 48), (dict(samples=3), 48), (dict(samples=-1), 48), (dict(gate_stride=63), 48), (dict(scale_stride=-64), 48),
         (dict(samples=2, gate_stride=1 << 58), 48),
         (dict(x_dtype=3), 4), (dict(r_dtype=GN_F16), 4), (dict(w_dtype=GN_F16), 4), (dict(post_dtype=-1), 4), (dict(gate_dtype=9), 4),
         (dict(scale_dtype=GN_F16), 4), (dict(x_dtype=GN_F32), 4),
         (dict(eps=-1e-6), 5), (dict(eps=NAN), 5), (dict(residual_scale=NAN), 49), (dict(branch_scale=float("inf")), 49),
         (dict(post_norm=0), 50)]


@pytest.mark.parametrize("kw,status", SHAPE, ids=str)
def test_shapes_and_types(kw, status):
    assert fwd(**kw) == status and bwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(res=None), 1), (dict(h=None), 1), (dict(hs=None), 1), (dict(xq=None), 1),
    (dict(q_dtype=2), 4), (dict(block=16), 34), (dict(post_norm=0, post=None), 50), (dict(post_norm=0, prstd=None), 50),
    (dict(x=at(0, 1)), 7), (dict(h=at(7, 1)), 7), (dict(rstd=at(8, 2)), 7), (dict(gate=at(4, 1)), 7), (dict(hs=at(11, 2)), 7),
    (dict(y=at(0, 2)), 33), (dict(y=at(0), x_stride=128), 33), (dict(y=at(1)), 33), (dict(h=at(0)), 33), (dict(h=at(1, 2)), 33),
    (dict(y=at(2)), 33), (dict(h=at(4)), 33), (dict(rstd=at(0)), 33), (dict(prstd=at(8)), 33), (dict(hq=at(6)), 33),
    (dict(xq=at(0)), 33), (dict(xs=at(11)), 33), (dict(hs=at(10)), 33), (dict(y=at(7)), 33),
    (dict(samples=2, gate_stride=1 << 19, y=at(5)), 33),                                    # the second sequence's gate
    (dict(), 8), (dict(y=at(0)), 8), (dict(h=at(1)), 8), (dict(y=None, rstd=at(0)), 8), (dict(hq=None, hs=None), 8),
    (dict(w=None, post=None, gate=None, scale=None), 8), (dict(samples=4, gate_stride=64, scale_stride=100), 8),
    (dict(y=None, w=at(7), scale=at(7)), 8), (dict(T=0, x=None, res=None, h=None), 0), (dict(T=0, samples=0), 0),
    (dict(r_dtype=GN_F32, w_dtype=GN_F32), 8), (dict(hq=at(10, 1), xq=at(12, 3)), 8),
], ids=str)
def test_forward(kw, status):
    assert fwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dx=None, dres=None, dw=None, dpost=None, dgate=None, dscale=None), 1), (dict(h=None), 1), (dict(x=None), 1),
    (dict(rstd=None), 1), (dict(prstd=None), 1), (dict(ws=None), 1), (dict(xs=at(16)), 1), (dict(hs=at(16)), 1),
    (dict(post_norm=0, post=None, prstd=None), 50), (dict(wsb=64), 6), (dict(ws=at(20, 4)), 7), (dict(dx=at(10, 1)), 7),
    (dict(dgate=at(14, 1)), 7), (dict(hs=at(16), xs=at(17), q_dtype=3), 4), (dict(hs=at(16), xs=at(17), block=8), 34),
    (dict(dx=at(0, 2)), 33), (dict(dx=at(1)), 33), (dict(dx=at(2)), 33), (dict(dres=at(0)), 33), (dict(dres=at(3)), 33),
    (dict(dx=at(3), x_stride=128), 33), (dict(dx=at(6)), 33), (dict(dres=at(10)), 33), (dict(dw=at(4)), 33), (dict(dpost=at(12)), 33),
    (dict(dgate=at(9)), 33), (dict(dw=at(20)), 33), (dict(ws=at(0)), 33), (dict(dscale=at(5)), 33),
    (dict(hs=at(16), xs=at(17), dx=at(3)), 33), (dict(hs=at(16), xs=at(17), dx=at(16)), 33),
    (dict(), 8), (dict(dx=at(0)), 8), (dict(dx=at(3)), 8), (dict(dres=at(1)), 8), (dict(dres=at(2)), 8),
    (dict(hs=at(16), xs=at(17)), 8), (dict(hs=at(16), xs=at(17), h=at(2, 1), x=at(3, 3)), 8), (dict(dy=None, h=None, rstd=None), 8),
    (dict(dh=None), 8), (dict(post_norm=0, post=None, prstd=None, dpost=None, dgate=None, x=None), 8), (dict(dx=None, dres=None), 8),
    (dict(samples=4, gate_stride=64, scale_stride=64), 8), (dict(T=0), 8),
    (dict(T=0, dw=None, dpost=None, dgate=None, dscale=None, ws=None), 0),
], ids=str)
def test_backward(kw, status):
    assert bwd(**kw) == status


def test_quantize():
    def call(x=at(0), dt=GN_BF16, xs=64, T=4, H=64, block=0, q=at(1), qdt=0, s=at(2)):
        return lib.gn_q8_quantize(x, dt, xs, T, H, block, q, qdt, s, None)
    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1 and call(dt=3) == 4 and call(qdt=2) == 4
    assert call(block=16) == 34 and call(H=0) == 32 and call(xs=63) == 32 and call(T=-1) == 32 and call(H=32769, xs=32769) == 32
    assert call(x=at(0, 1)) == 7 and call(s=at(2, 1)) == 7 and call(q=at(0)) == 33 and call(s=at(1)) == 33 and call(s=at(0)) == 33
    assert call() == 8 and call(q=at(1, 3)) == 8 and call(T=0, x=None) == 0


def test_null_descriptor():
    assert lib.gn_join_forward(None, *FWD.values(), None) == 1
    assert lib.gn_join_backward(None, *BWD.values(), 0, None) == 1


def test_workspace_queries():
    ws = lib.gn_join_workspace_bytes
    assert ws(-1, 64, 1) == 0 and ws(4, 32769, 1) == 0 and ws(4, 64, 3) == 0 and ws(4, 64, 0) == 0
    assert ws(0, 64, 1) > 0 and ws(0, 64, 0) > 0 and ws(1, 1, 1) > 0
    rng = random.Random(1)
    for _ in range(3000):
        S = rng.choice([1, rng.randint(1, 20), rng.randint(1, 5000)])
        T, H = S * rng.choice([1, 2, rng.randint(1, 300), rng.randint(1, 20000)]), rng.randint(1, 32768)
        n = ws(T, H, S)
        means = (T * 8 + 15) // 16 * 16 if H > 8192 else 0              # of rows too wide for one kernel
        chunks, rest = divmod(n - means, H * 8)
        if chunks:
            assert rest == 0 and S <= chunks <= max(8 * 256, S) and chunks % S == 0 and chunks // S <= T // S, (T, H, S, n)
        if H > 4096 and T // S >= 4 and S < 2048:                       # groups of one row: whole turns of 256 workgroups
            used = chunks / (-(-chunks // 256) * 256)
            assert used > 0.74 or chunks // S == T // S, (T, S, chunks)


# ------------------------------------------------------------------ the binding

def _x(dtype=BF, shape=(3, 4, 64)):
    return torch.ones(shape, dtype=dtype)


def test_calls_reach_the_library_when_every_tensor_is_right():
    x, w, rs = _x(), torch.ones(64), torch.ones(3, 4)
    mod = _x(shape=(3, 1, 200))
    for call in (lambda: gn.gn_join_forward(x, x, w), lambda: gn.gn_join_forward(x, _x(F32), w, post_weight=w, checkpoint=E4, block=32),
                 lambda: gn.gn_join_forward(x, x, None, gate=mod[..., 1:65], scale=mod[..., 65:129]),
                 lambda: gn.gn_join_forward(x, x, None, gate=_x(shape=(12, 64)), scale=w),
                 lambda: gn.gn_join_forward(x, x, None, need_y=False, post_norm=True),
                 lambda: gn.gn_join_backward(x, x, rs, w, x=x, post_rstd=rs, dh=x, gate=mod[..., :64]),
                 lambda: gn.gn_join_backward(x, (_x(I8), rs), rs, w, x=(_x(I8), rs), post_rstd=rs, block=0),
                 lambda: gn.gn_join_backward(None, None, None, None, dh=x), lambda: gn.gn_q8_quantize(x, E4),
                 lambda: gn.join_norm(x, x, w, post_norm=True, checkpoint=I8)):
        with pytest.raises(GnError) as e:
            call()
        assert e.value.status == 8 and "GN_ERR_DEVICE" in str(e.value)


@pytest.mark.parametrize("kw,err", [
    (dict(gate=_x(shape=(5, 64))), ValueError), (dict(gate=_x(shape=(3, 63))), ValueError), (dict(gate=_x(torch.float64, (64,))), TypeError),
    (dict(gate=_x(shape=(3, 64)), scale=_x(shape=(4, 64))), ValueError), (dict(scale=_x(shape=(1, 64)).expand(3, 64)), ValueError),
    (dict(gate=_x(shape=(3, 128))[:, ::2]), ValueError), (dict(gate=_x(shape=(0, 64))), ValueError),
    (dict(gate=_x(torch.float16, (64,))), GnError), (dict(post_weight=torch.ones(63)), ValueError),
    (dict(post_weight=torch.ones(64), post_norm=False), ValueError), (dict(post_rstd=torch.ones(12)), ValueError),
    (dict(out=_x(F32)), TypeError), (dict(out=_x(shape=(12, 64))), ValueError), (dict(h=_x(F32)), TypeError),
    (dict(out=_x(), need_y=False), ValueError), (dict(rstd=torch.ones(12), need_y=False), ValueError),
    (dict(rstd=torch.ones(11)), ValueError), (dict(checkpoint=torch.uint8), TypeError), (dict(checkpoint=I8, block=48), GnError),
    (dict(saved_h=(_x(I8), torch.ones(3, 4, 1))), ValueError), (dict(checkpoint=I8, saved_x=(_x(I8), torch.ones(3, 4, 1))), ValueError),
    (dict(checkpoint=E4, saved_h=(_x(I8), torch.ones(3, 4, 1))), TypeError),
    (dict(checkpoint=I8, saved_h=(_x(I8), torch.ones(3, 4, 2))), ValueError), (dict(residual_scale=NAN), GnError),
], ids=lambda v: "-".join(v) if isinstance(v, dict) else v.__name__)
def test_forward_binding_refusals(kw, err):
    with pytest.raises(err) as e:
        gn.gn_join_forward(_x(), _x(), torch.ones(64), **kw)
    assert getattr(e.value, "status", 0) != 8


def test_residual_refusals():
    for r, err in ((_x(shape=(12, 64)), ValueError), (_x(torch.float16), GnError), (_x(torch.int32), TypeError),
                   (_x().transpose(0, 1).contiguous().transpose(0, 1), ValueError)):
        with pytest.raises(err):
            gn.gn_join_forward(_x(), r, None)


@pytest.mark.parametrize("kw,err", [
    (dict(dh=_x(F32), h=_x()), TypeError), (dict(dh=_x(shape=(12, 64))), ValueError), (dict(x=_x(F32), gate=torch.ones(64)), TypeError),
    (dict(x=_x(shape=(3, 64)), gate=torch.ones(64)), ValueError), (dict(h=(_x(I8), torch.ones(13))), ValueError),
    (dict(h=(_x(I8), torch.ones(12)), x=_x(), block=0), ValueError), (dict(x=(_x(I8), torch.ones(12)), block=0), ValueError),
    (dict(h=(_x(I8), torch.ones(12)), x=(_x(E4), torch.ones(12)), block=0), TypeError),
    (dict(h=(_x(), torch.ones(12)), block=0), TypeError), (dict(post_rstd=torch.ones(12), post_norm=False), ValueError),
    (dict(dx=_x(F32)), TypeError), (dict(dx=_x(), need_dx=False), ValueError), (dict(dres=_x(F32)), TypeError),
    (dict(dweight=torch.ones(63)), ValueError), (dict(dweight=torch.ones(64, dtype=BF)), TypeError),
    (dict(dgate=torch.ones(64), gate=None), ValueError), (dict(dscale=torch.ones(64), scale=_x(F32, (3, 64))), ValueError),
    (dict(workspace=torch.ones(64, dtype=torch.uint8)), GnError), (dict(workspace=torch.ones(1 << 20, dtype=torch.uint8)[::2]), ValueError),
    (dict(x_dtype=F32), TypeError), (dict(dh=_x(), residual_dtype=F32), TypeError), (dict(post_norm=True), GnError),
    (dict(gate=torch.ones(64)), GnError), (dict(rstd=torch.ones(11)), ValueError),
    (dict(h=_x().transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
], ids=lambda v: "-".join(v) if isinstance(v, dict) else v.__name__)
def test_backward_binding_refusals(kw, err):
    a = dict(h=_x(), rstd=torch.ones(3, 4))
    a.update(kw)
    with pytest.raises(err) as e:
        gn.gn_join_backward(_x(), weight=torch.ones(64), **a)
    assert getattr(e.value, "status", 0) != 8


def test_neither_gradient():
    with pytest.raises(ValueError):
        gn.gn_join_backward(None, _x(), torch.ones(3, 4), None)


def test_no_rows_and_marked_outputs():
    """Calls of no rows succeed without a GPU, and tell autograd of their outputs like any other."""
    def e(dt, *shape):
        return torch.empty(*shape, dtype=dt)

    x, r, w = e(BF, 0, 64), e(F32, 0, 64), torch.ones(64)
    given = dict(out=e(BF, 0, 64), h=e(F32, 0, 64), rstd=e(F32, 0), post_rstd=e(F32, 0))
    saved = dict(saved_h=(e(I8, 0, 64), e(F32, 0, 1)), saved_x=(e(I8, 0, 64), e(F32, 0, 1)))
    f = gn.gn_join_forward(x, r, w, post_norm=True, checkpoint=I8, block=64, **given, **saved)
    assert f.y is given["out"] and f.saved_h[0] is saved["saved_h"][0] and f.saved_x[1] is saved["saved_x"][1]
    assert [t._version for t in (*given.values(), *saved["saved_h"], *saved["saved_x"])] == [1] * 8
    dx, dres = e(BF, 0, 64), e(F32, 0, 64)
    b = gn.gn_join_backward(x, f.saved_h, f.rstd, w, x=f.saved_x, post_rstd=f.post_rstd, dh=r, block=64, dx=dx, dres=dres,
                            need_dweight=False, need_dpost_weight=False)
    assert b.dx is dx and b.dres is dres and (dx._version, dres._version) == (1, 1) and b.dweight is None
    q, s = e(I8, 0, 64), e(F32, 0, 1)
    gn.gn_q8_quantize(x, out=q, scale=s, block=0)
    assert (q._version, s._version) == (1, 1) and (x._version, r._version, w._version) == (0, 0, 0)
    y, h = gn.join_norm(e(BF, 2, 0, 64).requires_grad_(), e(BF, 2, 0, 64))
    y.float().sum().backward()


def test_quantize_binding_refusals():
    x = _x()
    for kw, err in ((dict(q_dtype=torch.uint8), TypeError), (dict(out=_x()), TypeError), (dict(out=_x(I8, (12, 64))), ValueError),
                    (dict(scale=torch.ones(3, 4, 2)), ValueError), (dict(block=7), GnError), (dict(q_dtype=E4, out=_x(I8)), TypeError)):
        with pytest.raises(err):
            gn.gn_q8_quantize(x, **kw)
    with pytest.raises(ValueError):
        gn.gn_q8_quantize(x[..., ::2])
    with pytest.raises(TypeError):
        gn.gn_q8_quantize(_x(torch.float64))
    assert gn.gn_q8_quantize(torch.empty(0, 64), out=torch.empty(0, 64, dtype=E4))[0].dtype == E4
