"""The residual join and the 8-bit checkpoints written out in 64 bits with torch, and the bounds
their kernels are held to.

u = 2^-24, first order. A row's sum is a tree of depth at most DJ = 56 (3 levels inside a piece, up
to 32 additions over a lane's pieces, 6 over a wave, 4 over waves, and room). As in
ops_reference.py a root-mean-square's inverse is off by RSTD = 26 u of itself (its sums are those of
the row norm's kernel, of depth 40 at most).

Forward, given x, r and the vectors:
- c = branch_scale * gate * post_weight: 2 u. The branch x * post_rstd * c: RSTD + 1 u for the first
  product and 2 u for c, together 29 u of it; residual_scale * r: 1 u of it; their fused
  multiply-add: 1 u of h. Then h's rounding to its type.
- rstd of the stored h: RSTD. m = weight * (1 + scale): 2 u. y = h * rstd * m: RSTD + 4 u.
Backward, given everything the kernel reads (checkpoints as q * scale, whose product rounds: 1 u):
- g = dy * m: 3 u. xh = h * rstd: 2 u. c1 = mean(g * xh): 6 u a term, the tree, the mean and its
  product with rstd: (DJ + 9) u of mean|g * xh|.
- d = (rstd * g + dh) - xh * rstd * c1: 3 + 2 u of rstd * |g|, 1 u of |dh|, 5 u of the last part,
  2 u of results no larger than the parts: 8 u of the parts together, and what c1 is off by.
- xp = x * post_rstd: 2 u; c * xp: 5 u. P = mean((rstd * g + dh) * c * xp): 5 + 5 + 1 u a term, the
  tree and the mean: (DJ + 13) u of the mean of (rstd |g| + |dh|) |c xp|. Q = mean(xh * c * xp): 2 + 5
  + 1 u, so (DJ + 10) u of the mean of |xh c xp|. c2 = P - rstd c1 Q: those, what c1 is off by times
  mean|xh c xp|, and 4 u of both parts.
- dx = post_rstd * (d * c - xp * c2): 3 u of |d c| and 2 u of |xp c2| and 3 for the rest: 8 u of the
  parts, and what d and c2 are off by.
- A sum over rows: its terms' errors, and one u of the sum of the magnitudes for each addition
  behind one another: a chunk's rows (T / 128 + 1 at most), up to 512 rows of a workgroup, the
  chunks (their number or 1024, by 128), 128 slices and 24 for products and exchanges.
"""
import torch

from tests.ops_reference import RSTD, TINY, U, close, half_step  # noqa: F401

DJ = 56


def _vec(v, T, H, none):
    """One row of v for each of T rows, in fp64."""
    if v is None:
        return torch.full((1, H), none, dtype=torch.float64, device="cuda")
    v = v.double().reshape(-1, H)
    return v.repeat_interleave(T // v.shape[0], 0) if v.shape[0] > 1 and T else v


def coefficients(T, H, weight, post_weight, gate, scale, branch_scale):
    """(c, m) in fp64, a row for each of T rows or one for all."""
    bs = torch.tensor(branch_scale, dtype=torch.float32).double().item()
    return (bs * _vec(gate, T, H, 1.0) * _vec(post_weight, T, H, 1.0), _vec(weight, T, H, 1.0) * (1 + _vec(scale, T, H, 0.0)))


def f32(v):
    return torch.tensor(v, dtype=torch.float32).double().item()


def inverse_rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(-1) + f32(eps))


def check_forward(got, x, residual, weight, eps, post_weight=None, gate=None, scale=None, post_norm=False,
                  residual_scale=1.0, branch_scale=1.0):
    """Holds a JoinForward to the definition: h to x and residual, rstd and y to h as stored."""
    H = x.shape[-1]
    T = x.numel() // H
    c, m = coefficients(T, H, weight, post_weight, gate, scale, branch_scale)
    xd, r = x.double().reshape(T, H), f32(residual_scale) * residual.double().reshape(T, H)
    branch = xd * c
    if post_norm:
        pr = inverse_rms(xd, eps)
        if got.post_rstd is not None:
            close("post_rstd", got.post_rstd.reshape(T), pr, pr * RSTD)
        branch = branch * pr.unsqueeze(1)
    h = r + branch
    bound = 29 * U * branch.abs() + U * r.abs() + U * h.abs() + 2.0 ** -148
    close("h", got.h.reshape(T, H), h, bound + half_step(h.abs() + bound, got.h.dtype))
    if got.y is None:
        return
    hs = got.h.double().reshape(T, H)
    rstd = inverse_rms(hs, eps)
    if got.rstd is not None:
        close("rstd", got.rstd.reshape(T), rstd, rstd * RSTD)
    y = hs * rstd.unsqueeze(1) * m
    close("y", got.y.reshape(T, H), y, y.abs() * (RSTD + 4 * U) * 1.01 + half_step(y.abs() * 1.0001, got.y.dtype) + 1e-37)


def decode(saved, block):
    q, scale = saved
    H = q.shape[-1]
    v = q.float().double()
    return v * (scale.double() if not block else scale.double().repeat_interleave(block, -1)[..., :H])


def check_checkpoint(name, saved, v, q_dtype, block):
    """Every bit of a checkpoint of v: a rounded quotient for the scale and another for q (whose fp32
    value may be another neighbour only 2^-20 ulp from halfway between two)."""
    q, scale = (t.cpu() for t in saved)
    v = v.cpu().float()
    H = v.shape[-1]
    B = block or H
    n = -(-H // B)
    qmax = 127.0 if q_dtype == torch.int8 else 448.0
    runs = torch.nn.functional.pad(v, (0, n * B - H)).reshape(-1, n, B)
    want = (runs.abs().amax(-1) / qmax).clamp(min=2.0 ** -126)
    bad = ~torch.isfinite(runs).all(-1)
    want[bad] = float("nan")
    assert torch.equal(torch.isnan(scale.reshape(-1, n)), bad), f"{name}: NaN scales"
    assert torch.equal(scale.reshape(-1, n)[~bad], want[~bad]), f"{name}: scale"
    e = runs / torch.where(bad, 1.0, want).unsqueeze(-1)
    e = torch.where(bad.unsqueeze(-1), 0.0, e)
    wq = torch.round(e) if q_dtype == torch.int8 else e.to(torch.float8_e4m3fn).float()
    wq = wq.reshape(-1, n * B)[:, :H].reshape(q.shape)
    assert torch.equal(q.float(), wq), f"{name}: q"


def backward(dy, dh, h, x, rstd, post_rstd, weight, post_weight=None, gate=None, scale=None, post_norm=False,
             residual_scale=1.0, branch_scale=1.0):
    """{name: (gradient, bound before its rounding)} in fp64 from fp64 h and x of shape [T, H] (values
    of checkpoints among them); x None where it is not read."""
    like = dy if dy is not None else dh
    H = like.shape[-1]
    T = like.numel() // H
    c, m = coefficients(T, H, weight, post_weight, gate, scale, branch_scale)
    rs, bs = f32(residual_scale), f32(branch_scale)
    zero = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dhd = zero if dh is None else dh.double().reshape(T, H)
    if dy is None:
        g = xh = dyd = zero
        rstd = torch.zeros(T, 1, dtype=torch.float64, device="cuda")
    else:
        rstd, dyd = rstd.double().reshape(T, 1), dy.double().reshape(T, H)
        g, xh = dyd * m, h * rstd
    c1 = (g * xh).mean(1, keepdim=True)
    e1 = (DJ + 9) * U * (g * xh).abs().mean(1, keepdim=True) * rstd       # of c1 * rstd
    c1 = c1 * rstd
    d = rstd * g + dhd - xh * c1
    parts = rstd * g.abs() + dhd.abs() + (xh * c1).abs()
    ed = 8 * U * parts + xh.abs() * e1
    out = {"dres": (rs * d, abs(rs) * (ed + U * d.abs()))}
    xp = zero
    if x is not None:
        pr = post_rstd.double().reshape(T, 1) if post_norm else torch.ones(T, 1, dtype=torch.float64, device="cuda")
        xp = x * pr
    dx, ex = d * c, c.abs() * ed + 4 * U * (d * c).abs()
    if post_norm:
        cx = (c * xp).abs()
        c2 = (d * c * xp).mean(1, keepdim=True)
        qm = (xh.abs() * cx).mean(1, keepdim=True)
        pm = ((rstd * g.abs() + dhd.abs()) * cx).mean(1, keepdim=True)
        e2 = (DJ + 13) * U * pm + c1.abs() * (DJ + 10) * U * qm + e1 * qm + 4 * U * (pm + c1.abs() * qm)
        dx = pr * (dx - xp * c2)
        ex = pr * (c.abs() * ed + xp.abs() * e2 + 8 * U * ((d * c).abs() + (xp * c2).abs()))
    out["dx"] = dx, ex
    S = max(v.numel() // H if v is not None else 1 for v in (gate, scale))
    N = min(T, T // 128 + max(1024, S) // 128 + 512 + 128) + 24

    def sums(t, e):
        """Per sequence: the sum and its bound."""
        return t.reshape(S, -1, H).sum(1), e.reshape(S, -1, H).sum(1) + N * U * t.abs().reshape(S, -1, H).sum(1)

    A, eA = sums(dyd * xh, 4 * U * (dyd * xh).abs())
    C, eC = sums(d * xp, ed * xp.abs() + 4 * U * (d * xp).abs())
    w, pw = _vec(weight, 1, H, 1.0), _vec(post_weight, 1, H, 1.0)
    gt = _vec(gate, S, H, 1.0)
    sc = 1 + _vec(scale, S, H, 0.0)

    def put(name, t, e, one):
        if one and S > 1:
            t, e = t.sum(0, keepdim=True), e.sum(0, keepdim=True) + N * U * t.abs().sum(0, keepdim=True)
        out[name] = t, e + 4 * U * t.abs()

    put("dscale", w * A, w.abs() * eA, scale is None or scale.numel() == H)
    put("dgate", bs * pw * C, (bs * pw).abs() * eC, gate is None or gate.numel() == H)
    put("dweight", sc * A, sc.abs() * (eA + 2 * U * A.abs()), True)
    put("dpost_weight", bs * gt * C, (bs * gt).abs() * (eC + 2 * U * C.abs()), True)
    return out


def check_backward(got, want):
    for name, t in got._asdict().items():
        if t is not None:
            ref, bound = want[name]
            ref, bound = ref.reshape(t.shape), bound.reshape(t.shape)
            close(name, t, ref, bound * 1.01 + half_step(ref.abs() + bound, t.dtype) + 1e-37)
