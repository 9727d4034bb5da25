"""The row norm and the gradient norm written out in 64 bits with torch, and the bounds their
kernels are held to.

u = 2^-24 is the unit roundoff of fp32. The bounds are first-order rounding analysis:

- rstd: the squares of a row are added in a tree of depth at most D = 40 (3 levels inside a
  piece of 8 columns, up to 8 additions over a lane's pieces, 6 over a wave, 4 over waves; 40
  leaves room for other shapes of the tree); all terms are positive, so the sum is off by at
  most (D + 1) u of itself and the root halves that; the mean (a product with the rounded 1 / H)
  and the addition of eps, halved, the root and the reciprocal add 4 u at most: RSTD = 26 u.
- y: two more products: Y = RSTD + 2 u of |y|, then the rounding to the output type, half its
  eps of |y| (and half its smallest subnormal).
- c = mean(g * xhat): terms with 3 roundings each, the tree, the mean: (D + 6) u of
  mean|g * xhat|. d = rstd * (g - xhat * c) + dh: 6 u of each part's magnitude.
- dweight: terms with 2 roundings, added one after the other: a lane's rows (every 256th group
  of rows), up to 512 rows of a workgroup, then 2 partial sums, 3 lane exchanges and 16 waves: at
  most (min(T, T / 256 + 514) + 24) u of the sum of the magnitudes.
"""
import torch

U = 2.0 ** -24
D = 40
RSTD = 26 * U
Y = RSTD + 2 * U
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def half_step(t, dtype):
    """What rounding to dtype may move values t by."""
    return t.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype] / 2


def rms_forward(x, weight, eps, residual=None):
    """(y, h, rstd) in fp64, h rounded to the residual's dtype as the operator defines it."""
    h = x.double()
    if residual is not None:
        h = (h + residual.double()).to(residual.dtype).double()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + torch.tensor(eps, dtype=torch.float32).double())
    y = h * rstd.unsqueeze(-1)
    return (y if weight is None else y * weight.double()), h, rstd


def rms_backward(dy, h, rstd, weight, dh=None):
    """(d, dweight, bound of d in fp32, bound of dweight in fp32) in fp64."""
    T = rstd.numel()
    dy, h, rs = dy.double(), h.double(), rstd.double().unsqueeze(-1)
    g = dy if weight is None else dy * weight.double()
    xhat = h * rs
    c = (g * xhat).mean(-1, keepdim=True)
    c_mag = (g * xhat).abs().mean(-1, keepdim=True)
    d = rs * (g - xhat * c)
    bound = rs * (6 * U * (g.abs() + (xhat * c).abs()) + xhat.abs() * (D + 6) * U * c_mag)
    if dh is not None:
        d = d + dh.double()
        bound = bound + 2 * U * (d.abs() + dh.double().abs())
    lead = tuple(range(dy.dim() - 1))
    dw, mag = (dy * xhat).sum(lead), (dy * xhat).abs().sum(lead)
    return d, dw, bound, (min(T, T // 256 + 514) + 24) * U * mag


def e4m3_step(v):
    """Half the distance between e4m3 values at v: 2^-4 of |v|, and 2^-10 among subnormals."""
    return torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)


def close(name, got, ref, bound):
    """got within bound of ref wherever ref is finite; NaN and infinities in the same places."""
    got, ref = got.double(), ref.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), f"{name}: infinities differ"
    over = ((got - ref).abs() - bound)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{name}: beyond its bound by {float(over.max()):.3g}"
