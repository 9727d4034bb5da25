"""The gradients' norm and clipping on the GPU, and the new calls together: in a training step,
under graph capture, on other streams."""
import math

import pytest
import torch

import unet_groupnorm_amd as gn
from tests import ops_reference as R
from unet_groupnorm_amd.gn import GnError

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


def say(msg):
    print(f"[gpu-grads] {msg}", flush=True)


def rand(n, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


# Squares of fp32 values are exact in fp64 and their sum is off by 2^-53 for each addition,
# which is nothing beside the norm's one rounding to fp32.
NORM = 1.01 * R.U


def norm64(ts, kind=2.0):
    if kind == INF:
        return max([float(t.double().abs().max()) for t in ts if t.numel()], default=0.0)
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


LISTS = {
    "one element": [1],
    "empty and tiny": [0, 1, 0, 7, 8, 9, 255, 0],
    "around a tile": [8191, 8192, 8193, 16384, 3 * 8192 + 5],
    "three tables": [1 + (i * 37) % 500 for i in range(400)],
    "long": [5_000_003, 64, 20_000_000],
    "all empty": [0, 0],
}


@pytest.mark.parametrize("kind", [2.0, INF], ids=["2", "inf"])
@pytest.mark.parametrize("dtypes", [(F32,), (BF,), (F16,), (BF, F32, F16)], ids=["fp32", "bf16", "fp16", "mixed"])
@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clip(name, dtypes, kind):
    sizes = LISTS[name]
    say(f"{name}, {dtypes}, norm {kind}")
    ts = [rand(n, dtypes[i % len(dtypes)], i, 0.01 * (1 + i % 5)) for i, n in enumerate(sizes)]
    want = norm64(ts, kind)
    norm = gn.gn_grad_norm(ts, kind)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - want) <= want * NORM
    for factor in (0.37, 4.0):
        limit = want * factor
        coef = min(1.0, limit / (want + 1e-6))
        kept = [t.clone() for t in ts]
        outs = [torch.full_like(t, 7, dtype=F32 if i % 2 else t.dtype) for i, t in enumerate(ts)]
        n2 = gn.gn_grad_clip(ts, limit, kind, out=outs)
        assert torch.equal(n2, norm)
        for t, k, o in zip(ts, kept, outs):
            assert torch.equal(bits(t), bits(k)), "an input was written"
            ref = k.double() * coef
            R.close("out", o, ref, ref.abs() * 5 * R.U + R.half_step(ref, o.dtype) * (1 + 5 * R.U))
        n3 = gn.gn_grad_clip(ts, limit, kind)
        assert torch.equal(n3, norm)
        for t, k, o in zip(ts, kept, outs):
            # where o holds the fp32 products, the call in place rounds those to t's type
            assert torch.equal(bits(t), bits(o.to(t.dtype)))
            if factor > 1:
                assert torch.equal(bits(t), bits(k))
        ts = kept


# Lists of more than 12288 tiles of 2048 elements take the factor from a kernel between the two
# passes; the first of these is the longest that does not.
LONG = {
    "12288 tiles": [12288 * 2048],
    "12289 tiles": [12288 * 2048 + 1],
    "two long tensors": [30_000_003, 64, 20_000_000],
    "several tables": [60_000 + (i * 7919) % 70_001 for i in range(400)],
    "biases beside one long tensor": [26_000_000] + [1 + (i * 37) % 300 for i in range(200)],
}


@pytest.mark.parametrize("kind", [2.0, INF], ids=["2", "inf"])
@pytest.mark.parametrize("dtypes", [(F32,), (BF,), (F16,), (BF, F32, F16)], ids=["fp32", "bf16", "fp16", "mixed"])
@pytest.mark.parametrize("name", list(LONG))
def test_norm_and_clip_of_long_lists(name, dtypes, kind, monkeypatch):
    monkeypatch.setitem(LISTS, name, LONG[name])
    test_norm_and_clip(name, dtypes, kind)


def test_long_unaligned_views_and_guards():
    sizes = [3, 8193, 26_000_001, 1, 40001, 64]
    for dt, odt in ((BF, BF), (BF, F32), (F16, F16), (F32, F32)):
        flat, dst = rand(sum(sizes) + 1, dt, 5), torch.full((sum(sizes) + 3,), 7.0, device="cuda", dtype=odt)
        ts, outs = list(flat[1:].split(sizes)), list(dst[1:-2].split(sizes))
        say(f"a long list of views one element off alignment, {dt} to {odt}")
        n = gn.gn_grad_clip(ts, 1.0, out=outs)
        want = norm64(ts)
        assert abs(float(n) - want) <= want * NORM
        ref = flat[1:].double() / (want + 1e-6)
        R.close("out", dst[1:-2], ref, ref.abs() * 5 * R.U + R.half_step(ref, odt) * (1 + 5 * R.U))
        assert float(dst[0]) == 7 and bool((dst[-2:].float() == 7).all())


@pytest.mark.parametrize("kind", [2.0, INF], ids=["2", "inf"])
def test_nan_and_infinity_in_a_long_list(kind):
    for bad in (float("nan"), INF, -INF):
        for dt in (BF, F32):
            t = [rand(100, BF, 1), rand(26_000_001, dt, 2)]
            t[1][-1] = bad
            n = gn.gn_grad_clip(t, 1.0, kind)
            if math.isnan(bad):
                assert math.isnan(float(n)) and bool(torch.isnan(t[0]).all()) and bool(torch.isnan(t[1]).all())
            else:
                assert float(n) == INF and float(t[0].abs().max()) == 0
                assert bool(torch.isnan(t[1][-1])) and int(torch.isnan(t[1]).sum()) == 1


def test_unaligned_views_and_guards():
    sizes = [3, 8193, 1000, 1, 40001, 64]
    for dt, odt in ((BF, BF), (BF, F32), (F16, F32), (F32, F32)):
        flat, dst = rand(sum(sizes) + 1, dt, 5), torch.full((sum(sizes) + 3,), 7.0, device="cuda", dtype=odt)
        ts, outs = list(flat[1:].split(sizes)), list(dst[1:-2].split(sizes))
        say(f"views one element off alignment, {dt} to {odt}")
        n = gn.gn_grad_clip(ts, 1.0, out=outs)
        want = norm64(ts)
        assert abs(float(n) - want) <= want * NORM
        ref = flat[1:].double() / (want + 1e-6)
        R.close("out", dst[1:-2], ref, ref.abs() * 5 * R.U + R.half_step(ref, odt) * (1 + 5 * R.U))
        assert float(dst[0]) == 7 and bool((dst[-2:].float() == 7).all())


def test_range_of_the_norm():
    say("squares beyond and below fp32")
    for v in (1e30, 1e-30):
        t = [torch.full((1000,), v, device="cuda"), torch.full((10,), v, device="cuda", dtype=BF)]
        want = norm64(t)
        assert abs(float(gn.gn_grad_norm(t)) - want) <= want * NORM
    big = [torch.full((4,), 3e38, device="cuda")]
    n = gn.gn_grad_clip(big, 1.0)
    assert math.isinf(float(n)) and bool((big[0] > 0.49).all()) and bool((big[0] < 0.51).all())   # only fp32 norm[0] overflows


def test_a_tensor_of_several_entries():
    n = (1 << 27) + 8197                     # longer than one entry of the table
    say(f"{n} fp16 elements")
    t = torch.full((n,), 0.5, dtype=F16, device="cuda")
    t[-1], t[1 << 27] = 3.0, -2.0
    want = math.sqrt(0.25 * (n - 2) + 13.0)
    out = [torch.full((n,), 7.0, device="cuda")]
    norm = gn.gn_grad_clip([t], 1.0, out=out)
    assert abs(float(norm) - want) <= want * NORM
    R.close("out", out[0], t.double() / (want + 1e-6), (t.double() / want).abs() * 5 * R.U)
    assert float(gn.gn_grad_norm([t], INF)) == 3.0


@pytest.mark.parametrize("kind", [2.0, INF], ids=["2", "inf"])
def test_nan_and_infinity(kind):
    for bad in (float("nan"), INF, -INF):
        for place in (0, 8191, 20000):
            t = [rand(100, BF, 1), rand(30000, F32, 2)]
            t[1][place] = bad
            n = gn.gn_grad_clip(t, 1.0, kind)
            ref_nan = math.isnan(bad)
            assert math.isnan(float(n)) if ref_nan else float(n) == INF
            if ref_nan:
                assert bool(torch.isnan(t[0]).all()) and bool(torch.isnan(t[1]).all())
            else:
                assert float(t[0].abs().max()) == 0 and bool(torch.isnan(t[1][place])) and int(torch.isnan(t[1]).sum()) == 1


@pytest.mark.parametrize("n", [1000, 26_000_001])
def test_an_infinite_limit_clips_nothing(n):
    """Whatever the norm is, infinity among it; a NaN norm still makes every output NaN."""
    for bad in (1.0, INF, -INF):
        t = [rand(100, BF, 1), rand(n, F32, 2)]
        t[1][7] = bad
        kept, outs = [v.clone() for v in t], [torch.empty_like(v) for v in t]
        for kind in (2.0, INF):
            norm = gn.gn_grad_clip(t, INF, kind, out=outs)
            assert torch.equal(gn.gn_grad_clip(t, INF, kind), norm) and (math.isinf(float(norm)) == math.isinf(bad))
            for a, b, o in zip(t, kept, outs):
                assert torch.equal(bits(a), bits(b)) and torch.equal(bits(o), bits(b))
    t[1][7] = float("nan")
    assert math.isnan(float(gn.gn_grad_clip(t, INF))) and all(bool(torch.isnan(v).all()) for v in t)


def test_layouts_and_refusals():
    conv = torch.randn(8, 4, 3, 3, 3, device="cuda").contiguous(memory_format=torch.channels_last_3d)
    t = conv.clone(memory_format=torch.preserve_format)
    want = norm64([t])
    gn.gn_grad_clip([t], 1.0)
    assert t.stride() == conv.stride()
    ref = conv.double() / (want + 1e-6)
    R.close("conv", t, ref, ref.abs() * 5 * R.U + 1e-40)
    with pytest.raises(ValueError):
        gn.gn_grad_norm([conv, torch.ones(3)])                 # two devices
    with pytest.raises(GnError):
        gn.gn_grad_clip([conv, conv], 1.0)                     # one tensor twice
    with pytest.raises(GnError):
        gn.gn_grad_clip([conv.view(-1)[:100] if conv.is_contiguous() else conv.permute(0, 2, 3, 4, 1).reshape(-1)[:100],
                         conv.permute(0, 2, 3, 4, 1).reshape(-1)[50:150]], 1.0)
    v = conv._version
    gn.gn_grad_clip([conv], 1.0)
    assert conv._version > v                                   # autograd learns of the write


def _block_step(params, x, target, norm):
    """A pre-norm residual block with a GroupNorm in front: forward, backward, clipping."""
    gw, gb, w1, w2, m1, m2 = params
    z = gn.group_norm(x, 4, gw, gb)
    rows = z.flatten(2).transpose(1, 2).contiguous()           # (N, S, C)
    h1 = norm(rows, w1, None)
    a = torch.relu(h1 @ m1)
    h2, stream = norm(a, w2, rows)
    return ((h2 @ m2 + stream - target) ** 2).mean()


def _plain_norm(x, w, res):
    s = x if res is None else x + res
    y = s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    return y if res is None else (y, s)


def _own_norm(x, w, res):
    return gn.rms_norm(x, w, 1e-6, residual=res)


def _params():
    shapes = [(16,), (16,), (16,), (16,), (16, 16), (16, 16)]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    return [torch.nn.Parameter(torch.randn(s, generator=g, device="cuda") * 0.3 + (1.0 if len(s) == 1 and i != 1 else 0.0))
            for i, s in enumerate(shapes)]


def test_a_training_step():
    x, target = rand((2, 16, 4, 5, 6), F32, 10), rand((2, 120, 16), F32, 11)
    own, ref = _params(), _params()
    for params, norm in ((own, _own_norm), (ref, _plain_norm)):
        _block_step(params, x, target, norm).backward()
    for i, (a, b) in enumerate(zip(own, ref)):
        rel = float((a.grad - b.grad).norm() / b.grad.norm())
        say(f"parameter {i}: gradient {rel:.1e} from the plain block's")
        assert rel < 1e-4
    want = norm64([p.grad for p in own])
    before = [p.grad.clone() for p in own]
    n = gn.clip_gradients(iter(own + own[:1] + [torch.nn.Parameter(torch.ones(2, device="cuda"))]), want / 2)
    assert abs(float(n) - want) <= want * NORM
    c = want / 2 / (want + 1e-6)
    for p, b in zip(own, before):
        R.close("clipped", p.grad, b.double() * c, b.double().abs() * 5 * R.U + 1e-44)
    assert abs(norm64([p.grad for p in own]) - want / 2) <= want * 1e-5


def test_graph_capture_replays():
    T, H = 300, 520
    x, res, w = rand((T, H), BF, 20), rand((T, H), BF, 21), rand(H, BF, 22)
    dy, dh = rand((T, H), BF, 23), rand((T, H), BF, 24)
    gbuf = [rand(70000, BF, 25), rand(33, F32, 26)]
    ws = torch.empty(gn.gn_rms_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")

    def step():
        y, h, rstd = gn.gn_rms_forward(x, w, residual=res)
        q, s, _, _ = gn.gn_rms_forward_q8(x, w, residual=res, block=64)
        v = gn.gn_q8_dequantize(q, s, BF, block=64)
        dx, dw, _ = gn.gn_rms_backward(dy, h, rstd, w, dh=dh, workspace=ws)
        outs = [torch.empty_like(t) for t in gbuf] + [torch.empty_like(dw)]
        n = gn.gn_grad_clip(gbuf + [dw], 1.0, out=outs)
        return [y, h, rstd, q.view(torch.int8).to(F32), s, v, dx, dw, n] + outs

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out1 = step()
    with torch.cuda.graph(g2):
        out2 = step()
    for r in range(3):
        for g, out in ((g1, out1), (g2, out2)):
            ws.fill_(0xFF)
            for t in out:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for k, (a, b) in enumerate(zip(want, out)):
                assert torch.equal(bits(a), bits(b)), f"replay {r}: output {k}"
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(want, eager):
            assert torch.equal(bits(a), bits(b))
    # new inputs in the captured buffers
    x.copy_(rand((T, H), BF, 30))
    gbuf[0].mul_(3)
    want = [t.clone() for t in step()]
    g1.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, out1):
        assert torch.equal(bits(a), bits(b))


def test_captured_backward_pass():
    params, x, target = _params(), rand((2, 16, 4, 5, 6), F32, 10), rand((2, 120, 16), F32, 11)

    def step():
        for p in params:
            p.grad = None
        loss = _block_step(params, x, target, _own_norm)
        loss.backward()
        return gn.clip_gradients(params, 0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = step().clone()
    grads = [p.grad.clone() for p in params]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = step()
    for r in range(3):
        for p in params:
            p.grad.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, want)
        for p, g in zip(params, grads):
            assert torch.equal(bits(p.grad), bits(g)), f"replay {r}"


def test_capture_beside_a_live_eager_graph_is_refused():
    x, w = rand((8, 64), F32, 50), torch.nn.Parameter(torch.ones(64, device="cuda"))
    alive = gn.rms_norm(x, w)                      # holds w's gradient accumulation on the eager stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
        try:
            with pytest.raises(RuntimeError, match="eager graph"):
                gn.rms_norm(x, w)
            y = x + 1
        finally:
            graph.capture_end()
    torch.cuda.synchronize()
    alive.sum().backward()
    assert w.grad is not None and y.shape == x.shape


def test_other_streams():
    x, w = rand((2000, 1024), BF, 40), rand(1024, BF, 41)
    ref = gn.gn_rms_forward(x, w)
    rdx = gn.gn_rms_backward(x, x, ref[2], w)
    rn = gn.gn_grad_norm([x, w])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            y, h, rstd = gn.gn_rms_forward(x, w)
            outs.append((y, rstd) + gn.gn_rms_backward(x, h, rstd, w)[:2] + (gn.gn_grad_norm([x, w]),))
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, (ref[0], ref[2], rdx[0], rdx[1], rn)):
            assert torch.equal(bits(a), bits(b))
