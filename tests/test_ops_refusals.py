"""The row norm's and the gradient list's entry points on a host without a GPU: every declared
symbol is exported, invalid arguments are refused with the documented status before anything
touches the device, and the binding refuses tensors of the wrong sizes, dtypes or layouts."""
import ctypes
import os
import random
import re

import pytest
import torch

import unet_groupnorm_amd as gn
from unet_groupnorm_amd import _gnbind
from unet_groupnorm_amd._lib import GN_BF16, GN_F16, GN_F32, OPS_STATUS_NAMES, GnGradTensor, lib
from unet_groupnorm_amd.gn import GnError

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gn_ops.h")
BF, F32 = torch.bfloat16, torch.float32


def at(k):
    """A fake aligned address; the checks below never look behind it. 1 MiB apart."""
    return ctypes.c_void_p(0x10000000 + (k << 20))


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(gn_[a-z_0-9]+)\s*\(", text, flags=re.M))
    assert len(names) == 9, names
    for name in names:
        assert hasattr(lib, name), name


def test_status_names_match_the_header():
    text = open(HEADER).read()
    for code, name in OPS_STATUS_NAMES.items():
        assert re.search(rf"\b{name}\s*=\s*{code}\b", text), name
        assert lib.gn_ops_status_string(code) != b"unknown status"
    assert lib.gn_ops_status_string(0) == b"ok" and lib.gn_ops_status_string(999) == b"unknown status"


def test_gradient_record_matches_the_header():
    text = open(HEADER).read()
    body = re.search(r"typedef struct gn_grad_tensor \{(.*?)\} gn_grad_tensor;", text, re.S).group(1)
    names = [d.split()[-1].lstrip("*") for d in body.split(";") if d.strip()]
    assert names == [n for n, _ in GnGradTensor._fields_] and ctypes.sizeof(GnGradTensor) == 32


def fwd(**kw):
    a = dict(x=at(0), xdt=GN_BF16, xs=64, res=None, rdt=GN_BF16, w=at(1), wdt=GN_BF16, T=4, H=64, eps=1e-6, y=at(2),
             ydt=GN_BF16, h=None, rstd=at(3), stream=None)
    a.update(kw)
    return lib.gn_rms_forward(*a.values())


RES = dict(res=at(4), h=at(5))
FWD_BAD = [
    (dict(x=None), 1), (dict(y=None), 1), (dict(res=at(4)), 1), (dict(h=at(4)), 1),
    (dict(T=-1), 32), (dict(H=0), 32), (dict(H=32769, xs=32769), 32), (dict(xs=63), 32), (dict(T=1 << 45), 32),
    (dict(xdt=3), 4), (dict(wdt=GN_F16), 4), (dict(ydt=GN_F16), 4), (dict(**RES, rdt=GN_F16), 4),
    (dict(xdt=GN_F32, wdt=GN_F32, ydt=GN_BF16), 4),
    (dict(eps=-1e-6), 5), (dict(eps=float("nan")), 5), (dict(eps=float("inf")), 5),
    (dict(x=ctypes.c_void_p(0x10000001)), 7), (dict(rstd=ctypes.c_void_p(0x10300002)), 7),
    (dict(w=at(1), wdt=GN_F32, y=ctypes.c_void_p(0x10200001)), 7),
    (dict(y=ctypes.c_void_p(0x10000002)), 33),            # y shifted into x
    (dict(y=at(0), xs=128), 33),                          # in place over strided rows
    (dict(y=at(0), ydt=GN_F32), 33),                      # in place in a wider type
    (dict(y=at(1)), 33), (dict(rstd=at(0)), 33), (dict(rstd=at(1)), 33),
    (dict(res=at(4), h=ctypes.c_void_p(0x10400002)), 33), (dict(res=at(4), h=at(0)), 33), (dict(res=at(4), h=at(2)), 33),
]


@pytest.mark.parametrize("kw,status", FWD_BAD, ids=str)
def test_forward_refusals(kw, status):
    assert fwd(**kw) == status


@pytest.mark.parametrize("kw", [dict(), dict(y=at(0)), dict(**RES), dict(res=at(4), h=at(4)), dict(w=None),
                                dict(xs=1000), dict(rstd=None)], ids=str)
def test_forward_good_arguments_reach_the_device_check(kw):
    assert fwd(**kw) == 8


def test_no_rows_is_a_call_that_does_nothing():
    assert fwd(T=0, x=None, y=None) == 0
    assert lib.gn_q8_dequantize(None, 0, None, 0, 64, 0, None, GN_F32, None) == 0


def q8(**kw):
    a = dict(x=at(0), xdt=GN_BF16, xs=64, res=None, rdt=GN_BF16, w=at(1), wdt=GN_BF16, T=4, H=64, eps=1e-6, block=0,
             q=at(2), qdt=0, scale=at(3), h=None, rstd=None, stream=None)
    a.update(kw)
    return lib.gn_rms_forward_q8(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(scale=None), 1), (dict(qdt=2), 4), (dict(qdt=-1), 4), (dict(block=16), 34),
    (dict(block=-32), 34), (dict(q=at(0)), 33), (dict(scale=at(2)), 33), (dict(scale=at(0)), 33), (dict(xs=1), 32),
    (dict(scale=ctypes.c_void_p(0x10300001)), 7), (dict(), 8), (dict(block=128), 8),
], ids=str)
def test_q8_refusals(kw, status):
    assert q8(**kw) == status


def test_dequantize_refusals():
    def call(q=at(0), qdt=0, s=at(1), T=4, H=64, block=0, o=at(2), odt=GN_F32):
        return lib.gn_q8_dequantize(q, qdt, s, T, H, block, o, odt, None)
    assert call(q=None) == 1 and call(s=None) == 1 and call(o=None) == 1
    assert call(qdt=5) == 4 and call(odt=9) == 4 and call(block=8) == 34 and call(H=0) == 32
    assert call(o=at(0)) == 33 and call(o=at(1)) == 33 and call(s=ctypes.c_void_p(0x10100001)) == 7 and call() == 8


def bwd(**kw):
    a = dict(dy=at(0), dydt=GN_BF16, h=at(1), hdt=GN_BF16, hs=64, rstd=at(2), w=at(3), wdt=GN_BF16, dh=None, T=4, H=64,
             dx=at(4), xdt=GN_BF16, dres=None, dw=at(5), ws=at(6), wsb=1 << 20, stream=None)
    a.update(kw)
    return lib.gn_rms_backward(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(h=None), 1), (dict(rstd=None), 1), (dict(dx=None, dw=None), 1), (dict(ws=None), 1),
    (dict(H=0), 32), (dict(hs=63), 32), (dict(T=-1), 32),
    (dict(xdt=GN_F16), 4), (dict(dydt=GN_F16), 4), (dict(wdt=GN_F16), 4), (dict(hdt=7), 4), (dict(w=None, wdt=GN_F16), 4),
    (dict(wsb=16), 6), (dict(ws=ctypes.c_void_p(0x10600004)), 7), (dict(dx=ctypes.c_void_p(0x10400001)), 7),
    (dict(dx=ctypes.c_void_p(0x10000002)), 33), (dict(dx=at(1), hs=128), 33), (dict(dx=at(3)), 33),
    (dict(dres=at(4)), 33), (dict(dw=at(0)), 33), (dict(ws=at(0)), 33), (dict(dx=at(6)), 33),
    (dict(), 8), (dict(dx=at(0)), 8), (dict(dx=at(1)), 8), (dict(dh=at(7), dx=at(7)), 8), (dict(dw=None, ws=None, wsb=0), 8),
    (dict(hdt=GN_F32, dres=at(7)), 8), (dict(T=0, dw=None, ws=None), 0),
], ids=str)
def test_backward_refusals(kw, status):
    assert bwd(**kw) == status


def test_workspace_queries():
    assert lib.gn_rms_workspace_bytes(-1, 64) == 0 and lib.gn_rms_workspace_bytes(4, 32769) == 0
    assert 0 < lib.gn_rms_workspace_bytes(0, 64) <= lib.gn_rms_workspace_bytes(1 << 20, 64) <= 4096 * 64 * 4
    assert lib.gn_grad_workspace_bytes(None, 1) == 0
    assert gn.gn_grad_workspace_bytes([torch.zeros(5)]) == 16
    assert gn.gn_grad_workspace_bytes([torch.zeros(0)]) == 16
    many = [torch.zeros(1)] * 400       # three tables
    assert gn.gn_grad_workspace_bytes(many) == (100 + 1) * 8   # a partial for each step of four


def glist(*rows):
    arr = (GnGradTensor * len(rows))()
    for a, (d, o, n, dt, odt) in zip(arr, rows):
        a.data, a.out, a.numel, a.dtype, a.out_dtype = d.value if d else None, o.value if o else None, n, dt, odt
    return arr


@pytest.mark.parametrize("rows,status", [
    ([(at(0), at(1), -1, 0, 0)], 32), ([(None, at(1), 4, 0, 0)], 1), ([(at(0), None, 4, 0, 0)], 1),
    ([(at(0), at(1), 4, 5, 0)], 4), ([(at(0), at(1), 4, GN_BF16, GN_F16)], 4), ([(at(0), at(1), 4, GN_F32, GN_BF16)], 4),
    ([(ctypes.c_void_p(0x10000002), at(1), 4, 0, 0)], 7),
    ([(at(0), at(0), 4, 0, 0), (at(0), at(0), 4, 0, 0)], 33),                    # the same tensor twice
    ([(at(0), at(1), 4, 0, 0), (at(2), at(1), 4, 0, 0)], 33),                    # one output for two
    ([(at(0), at(2), 4, 0, 0), (at(2), at(3), 4, 0, 0)], 33),                    # an output over another's data
    ([(at(0), at(0), 4, GN_BF16, GN_F32)], 33),                                  # in place in a wider type
    ([(at(0), at(8), 4, 0, 0)], 33), ([(at(9), at(1), 4, 0, 0)], 33),            # over the norm, from the workspace
    ([(at(0), at(0), 4, 0, 0), (at(1), at(1), 4, 1, 1), (None, None, 0, 0, 0)], 8),
    ([(at(3), at(3), 4, 0, 0), (at(1), at(2), 4, 1, 0)], 8),
], ids=str)
def test_clip_refusals(rows, status):
    assert lib.gn_grad_clip(glist(*rows), len(rows), 0, 1.0, at(8), at(9), 1 << 16, None) == status


def test_norm_refusals():
    t = glist((at(0), None, 4, 0, 0), (at(0), None, 4, 0, 0))       # twice: counted twice, not refused
    assert lib.gn_grad_norm(t, 2, 0, at(8), at(9), 1 << 16, None) == 8
    assert lib.gn_grad_norm(t, 0, 0, at(8), at(9), 1 << 16, None) == 32
    assert lib.gn_grad_norm(None, 1, 0, at(8), at(9), 1 << 16, None) == 1
    assert lib.gn_grad_norm(t, 2, 2, at(8), at(9), 1 << 16, None) == 35
    assert lib.gn_grad_norm(t, 2, 0, None, at(9), 1 << 16, None) == 1
    assert lib.gn_grad_norm(t, 2, 0, at(8), None, 1 << 16, None) == 1
    assert lib.gn_grad_norm(t, 2, 0, at(8), at(9), 8, None) == 6
    assert lib.gn_grad_norm(t, 2, 0, at(9), at(9), 1 << 16, None) == 33
    assert lib.gn_grad_norm(t, 2, 0, at(8), ctypes.c_void_p(0x10900008), 1 << 16, None) == 7
    t = glist((at(0), at(1), 4, 0, 0))
    for bad in (-1.0, float("nan")):
        assert lib.gn_grad_clip(t, 1, 0, bad, at(8), at(9), 1 << 16, None) == 35


# ------------------------------------------------------------------ the binding

def _x(dtype=BF, shape=(3, 5, 64)):
    return torch.ones(shape, dtype=dtype)


def test_calls_reach_the_library_when_every_tensor_is_right():
    x, w = _x(), torch.ones(64)
    for call in (lambda: gn.gn_rms_forward(x, w, residual=_x(F32)),
                 lambda: gn.gn_rms_forward_q8(x, w, block=32),
                 lambda: gn.gn_q8_dequantize(_x(torch.int8), torch.ones(3, 5, 1)),
                 lambda: gn.gn_rms_backward(x, _x(F32), torch.ones(3, 5), w, x_dtype=BF),
                 lambda: gn.gn_grad_norm([x, w]), lambda: gn.gn_grad_clip([x, w], 1.0),
                 lambda: gn.rms_norm(x[..., :32], None)):
        with pytest.raises(GnError) as e:
            call()
        assert e.value.status == 8 and "GN_ERR_DEVICE" in str(e.value)


@pytest.mark.parametrize("kw,err", [
    (dict(residual=_x(shape=(3, 64))), ValueError), (dict(residual=_x(torch.float64)), TypeError),
    (dict(residual=_x().transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
    (dict(out=_x(shape=(15, 64))), ValueError), (dict(out=_x(torch.int32)), TypeError), (dict(h=_x()), ValueError),
    (dict(residual=_x(), h=_x(F32)), TypeError), (dict(rstd=torch.ones(14)), ValueError),
    (dict(rstd=torch.ones(15, dtype=torch.float64)), ValueError), (dict(out_dtype=torch.float64), TypeError),
    (dict(out_dtype=torch.float16), GnError),
], ids=str)
def test_forward_binding_refusals(kw, err):
    with pytest.raises(err):
        gn.gn_rms_forward(_x(), torch.ones(64), **kw)


def test_row_layouts():
    w = torch.ones(64)
    for bad in (_x().transpose(1, 2), _x()[..., ::2], _x(shape=(3, 5, 130)).transpose(0, 1)[..., :64],
                torch.ones(1, dtype=BF).expand(4, 64)):
        with pytest.raises(ValueError):
            gn.gn_rms_forward(bad, None)
    with pytest.raises(ValueError):
        gn.gn_rms_forward(torch.tensor(1.0), None)
    with pytest.raises(ValueError):
        gn.gn_rms_forward(torch.ones(3, 0), None)
    with pytest.raises(ValueError):
        gn.gn_rms_forward(_x(), w[:63])
    with pytest.raises(TypeError):
        gn.gn_rms_forward(_x(torch.int32), w)
    for good in (_x(shape=(3, 5, 130))[..., 1:65], _x(shape=(3, 1, 64)).expand(3, 1, 64), _x(shape=(64,))):
        with pytest.raises(GnError) as e:
            gn.gn_rms_forward(good, w)
        assert e.value.status == 8


def test_q8_and_backward_binding_refusals():
    x, w = _x(), torch.ones(64)
    with pytest.raises(TypeError):
        gn.gn_rms_forward_q8(x, w, q_dtype=torch.uint8)
    with pytest.raises(ValueError):
        gn.gn_rms_forward_q8(x, w, block=32, scale=torch.ones(15))
    with pytest.raises(TypeError):
        gn.gn_rms_forward_q8(x, w, out=_x())
    with pytest.raises(ValueError):
        gn.gn_q8_dequantize(_x(torch.int8), torch.ones(14))
    with pytest.raises(TypeError):
        gn.gn_q8_dequantize(_x(), torch.ones(15))
    rs = torch.ones(3, 5)
    for kw, err in ((dict(dh=_x(F32)), TypeError), (dict(dx=_x(F32)), TypeError), (dict(dweight=torch.ones(63)), ValueError),
                    (dict(dweight=torch.ones(64, dtype=BF)), TypeError),
                    (dict(workspace=torch.ones(1 << 16, dtype=torch.uint8)[::2]), ValueError),
                    (dict(workspace=torch.ones(64, dtype=torch.uint8)), GnError)):
        with pytest.raises(err):
            gn.gn_rms_backward(x, x, rs, w, **kw)
    with pytest.raises(ValueError):
        gn.gn_rms_backward(x[:2], x, rs, w)
    with pytest.raises(ValueError):
        gn.gn_rms_backward(x, x, rs[:2], w)


def test_gradient_binding_refusals():
    g = [torch.ones(4, 4), torch.ones(3)]
    for call, err in ((lambda: gn.gn_grad_norm([]), ValueError), (lambda: gn.gn_grad_norm([g[0][:, ::2]]), ValueError),
                      (lambda: gn.gn_grad_norm([g[0].to_sparse()]), ValueError),
                      (lambda: gn.gn_grad_norm([g[0].double()]), TypeError), (lambda: gn.gn_grad_norm(g, 1.0), ValueError),
                      (lambda: gn.gn_grad_clip(g, 1.0, out=[torch.ones(4, 4)]), ValueError),
                      (lambda: gn.gn_grad_clip(g[:1], 1.0, out=[torch.ones(4, 4).t()]), ValueError),
                      (lambda: gn.gn_grad_clip(g[:1], 1.0, out=[torch.ones(16)]), ValueError),
                      (lambda: gn.gn_grad_clip(g, -1.0), GnError), (lambda: gn.gn_grad_clip([g[0], g[0]], 1.0), GnError),
                      (lambda: gn.gn_grad_norm(g, norm=torch.ones(2)), ValueError)):
        with pytest.raises(err):
            call()
    assert float(gn.clip_gradients([torch.nn.Parameter(torch.ones(3))], 1.0)) == 0.0   # no gradient anywhere


def test_backward_of_no_rows_without_a_weight_gradient():
    """An empty tensor's address may be null; a call that has nothing to write succeeds."""
    dy, h, rstd = torch.empty(0, 64, dtype=BF), torch.empty(0, 64), torch.empty(0)
    for weight in (None, torch.ones(64)):
        dx, dw, dres = gn.gn_rms_backward(dy, h, rstd, weight, x_dtype=BF, need_dweight=False)
        assert dx.shape == dres.shape == (0, 64) and dw is None and (dx.dtype, dres.dtype) == (BF, F32)
    x = torch.empty(2, 0, 64, requires_grad=True)
    gn.rms_norm(x).sum().backward()
    assert x.grad.shape == x.shape


def test_calls_mark_the_tensors_they_were_given_to_write():
    """Calls of no rows succeed without a GPU, and tell autograd of their outputs like any other."""
    def e(dt, *shape):
        return torch.empty(*shape, dtype=dt)

    def versions(call, **given):
        call(**given)
        return {k: v._version for k, v in given.items()}

    x, w, res = e(BF, 0, 64), torch.ones(64, dtype=BF), e(F32, 0, 64)
    assert versions(lambda **k: gn.gn_rms_forward(x, w, residual=res, **k), out=e(BF, 0, 64), h=e(F32, 0, 64),
                    rstd=e(F32, 0)) == dict(out=1, h=1, rstd=1)
    assert versions(lambda **k: gn.gn_rms_forward_q8(x, w, residual=res, **k), out=e(torch.int8, 0, 64),
                    scale=e(F32, 0, 1), h=e(F32, 0, 64), rstd=e(F32, 0)) == dict(out=1, scale=1, h=1, rstd=1)
    assert versions(lambda **k: gn.gn_q8_dequantize(e(torch.int8, 0, 64), e(F32, 0, 1), **k), out=e(F32, 0, 64)) == dict(out=1)
    assert versions(lambda **k: gn.gn_rms_backward(x, res, e(F32, 0), w, x_dtype=BF, need_dweight=False, **k),
                    dx=e(BF, 0, 64), dres=e(F32, 0, 64)) == dict(dx=1, dres=1)
    gn.gn_rms_forward(x, w, residual=res)
    assert (x._version, w._version, res._version) == (0, 0, 0)
    with torch.inference_mode():                              # tensors without a version
        gn.gn_rms_forward(e(BF, 0, 64), w, out=e(BF, 0, 64))


def test_backward_writes_every_output_it_is_given():
    """A dres given beside h of x's dtype is asked for by that; one that a flag declines is refused."""
    def e(*shape, dt=BF):
        return torch.empty(*shape, dtype=dt)

    x, rstd, w = e(0, 64), e(0, dt=F32), torch.ones(64, dtype=BF)
    dres = e(0, 64)
    got = gn.gn_rms_backward(x, x, rstd, w, dres=dres, need_dweight=False)
    assert got[2] is dres and dres._version == 1 and got[0] is not dres
    dx, dres = e(0, 64), e(0, 64)
    got = gn.gn_rms_backward(x, x, rstd, w, dx=dx, dres=dres, need_dweight=False)
    assert got[0] is dx and got[2] is dres and (dx._version, dres._version) == (1, 1)
    got = gn.gn_rms_backward(x, x, rstd, w, dres=dres, need_dx=False, need_dweight=False)
    assert got[0] is None and got[2] is dres
    for name, given in (("dx", e(0, 64)), ("dres", e(0, 64)), ("dweight", e(64))):
        with pytest.raises(ValueError, match=name):
            gn.gn_rms_backward(x, x, rstd, w, **{"need_dweight": False, name: given, "need_" + name: False})
        assert given._version == 0


@pytest.mark.parametrize("shape", [(64,), (1, 64), (1, 1, 64), (64, 1), (8, 8)], ids=str)
def test_a_weights_gradient_has_the_weights_shape(shape):
    x, rstd = _x(), torch.ones(3, 5)
    for dt in (BF, F32):
        dw = _gnbind.rms_backward(x, x, rstd, torch.ones(shape, dtype=dt), None, -1, True, False, True, None, None, None, None)[1]
        assert dw.shape == shape and dw.dtype == dt
    dw = _gnbind.rms_backward(x, x, rstd, None, None, -1, True, False, True, None, None, None, None)[1]
    assert dw.shape == (64,) and dw.dtype == F32


def test_a_dtype_that_contradicts_the_given_output_is_refused():
    def e(dt, *shape):
        return torch.empty(*shape, dtype=dt)

    E4, x, w, scale = torch.float8_e4m3fn, e(BF, 0, 64), torch.ones(64), e(F32, 0, 1)
    with pytest.raises(TypeError, match="out_dtype"):
        gn.gn_rms_forward(x, w, out_dtype=F32, out=e(BF, 0, 64))
    for asked, given in ((torch.int8, E4), (E4, torch.int8)):
        with pytest.raises(TypeError, match="q_dtype"):
            gn.gn_rms_forward_q8(x, w, q_dtype=asked, out=e(given, 0, 64))
    with pytest.raises(TypeError, match="out_dtype"):
        gn.gn_q8_dequantize(e(torch.int8, 0, 64), scale, F32, out=e(BF, 0, 64))
    # without one the output decides, and without either the default does
    assert gn.gn_rms_forward(x, w, out=e(F32, 0, 64))[0].dtype == F32 and gn.gn_rms_forward(x, w)[0].dtype == BF
    assert gn.gn_rms_forward_q8(x, w, out=e(E4, 0, 64))[0].dtype == E4 and gn.gn_rms_forward_q8(x, w)[0].dtype == torch.int8
    assert gn.gn_rms_forward_q8(x, w, q_dtype=E4)[0].dtype == E4
    q = e(torch.int8, 0, 64)
    assert gn.gn_q8_dequantize(q, scale, out=e(BF, 0, 64)).dtype == BF and gn.gn_q8_dequantize(q, scale).dtype == F32
    assert gn.gn_q8_dequantize(q, scale, BF, out=e(BF, 0, 64)).dtype == BF


def test_layouts_of_clipped_outputs():
    """Dimensions of one element have no say in a layout."""
    g = torch.ones(4, 1, 3)
    same = [torch.empty_strided((4, 1, 3), st) for st in ((3, 3, 1), (3, 1, 1), (3, 77, 1))]
    t = torch.empty_strided((4, 1, 3), (1, 4, 4)), torch.empty_strided((4, 1, 3), (1, 9, 4))
    for a, b in [(g, o) for o in same] + [(o, g) for o in same] + [t, t[::-1]] + [(torch.ones(1, 1), torch.ones(1, 1).t())]:
        with pytest.raises(GnError) as e:                     # as far as the device check
            gn.gn_grad_clip([a], 1.0, out=[b])
        assert e.value.status == 8
    for a, b in ((g, t[0]), (t[1], g), (torch.ones(2, 3), torch.ones(3, 2).t())):
        with pytest.raises(ValueError):
            gn.gn_grad_clip([a], 1.0, out=[b])


# ------------------------------------------------------------------ lists against their definition

SIZE = {GN_F32: 4, GN_BF16: 2, GN_F16: 2}


def meets(a, b):
    return a[0] < b[1] and b[0] < a[1] and a[0] < a[1] and b[0] < b[1]


def overlaps(rows, norm, ws):
    """The definition, pair by pair: no output meets another output, another tensor's data, or its
    own data except in its place; the norm and the workspace meet nothing."""
    spans = [((d, d + n * SIZE[dt]), (o, o + n * SIZE[odt]), dt == odt) for d, o, n, dt, odt in rows]
    for i, (d, o, same) in enumerate(spans):
        if meets(o, d) and not (o == d and same):
            return True
        for k, (d2, o2, _) in enumerate(spans):
            if k != i and (meets(o, o2) or meets(o, d2)):
                return True
    return meets(norm, ws) or any(meets(s, b) for d, o, _ in spans for s in (d, o) for b in (norm, ws))


def partials(sizes):
    """Partial results of a list: a share of 2048 workgroups by tiles for each table of 160
    entries of up to 2^27 elements, at most one for a step of 4 tiles of 2048."""
    entries = [min(n - k, 1 << 27) for n in sizes for k in range(0, n, 1 << 27)]
    tiles = [-(-n // 2048) for n in entries]
    tables = [sum(tiles[k:k + 160]) for k in range(0, len(tiles), 160)] or [0]
    total = max(sum(tiles), 1)
    return sum(max(1, min(-(-t // 4), t * 2048 // total)) for t in tables)


@pytest.mark.parametrize("seed", range(60))
def test_random_lists_against_the_definition(seed):
    rng = random.Random(seed)
    dense = seed % 3
    for _ in range(60):
        n, room = rng.choice([1, 2, 3, rng.randint(1, 12), rng.randint(1, 400)]), rng.choice([200, 4000, 1 << 20])
        if dense == 2:
            room *= 64                                      # mostly apart
        rows, place = [], 0
        for _ in range(n):
            dt = rng.choice([GN_F32, GN_BF16, GN_F16])
            odt, m = rng.choice([dt, GN_F32]), rng.choice([0, 1, 2, rng.randint(1, 40), rng.randint(1, 300)])
            if dense == 0:                                  # one behind the other, as in a bucket
                d, o = place, place + (n << 12)
                place += m * 4
            else:
                d, o = rng.randrange(room) * 4, rng.randrange(room) * 4
            if odt == dt and rng.random() < 0.4:
                o = d
            rows.append((0x10000000 + d, 0x10000000 + o, m, dt, odt))
        if rng.random() < 0.5:
            rng.shuffle(rows)
        need = (partials([r[2] for r in rows]) + 1) * 8
        far = rng.random() < 0.7
        norm = 0x60000000 if far else 0x10000000 + rng.randrange(room) * 4
        ws = 0x70000000 if far else 0x10000000 + rng.randrange(room) * 16
        t = glist(*((ctypes.c_void_p(d), ctypes.c_void_p(o), m, dt, odt) for d, o, m, dt, odt in rows))
        assert lib.gn_grad_workspace_bytes(t, n) == need
        want = 33 if overlaps(rows, (norm, norm + 4), (ws, ws + need)) else 8      # 8: as far as the device check
        assert lib.gn_grad_clip(t, n, 0, 1.0, norm, ws, need, None) == want, (seed, rows, norm, ws)
        assert lib.gn_grad_clip(t, n, 0, 1.0, norm, ws, need - 1, None) == 6


@pytest.mark.parametrize("sizes", [[], [0], [1], [8192], [8193], [1 << 27], [(1 << 27) + 1], [1 << 33], [5] * 160, [5] * 161,
                                   [(1 << 27) + 1] * 100, [1 << 40, 3, 1 << 29], [1 << 48] + [1] * 200, [300_000_000] + [7] * 900],
                         ids=lambda s: f"{len(s)} of {s[:1]}")
def test_partials_of_long_lists(sizes):
    t = glist(*((at(0), None, n, GN_BF16, GN_BF16) for n in sizes or [0]))
    assert lib.gn_grad_workspace_bytes(t, len(sizes or [0])) == (partials(sizes) + 1) * 8
