"""Plain 64-bit forms of the row-wise training operators (layer norm, dropout,
their fusion, SwiGLU backward) and, beside each value, how far a binary32
computation rounded once to the output's type may be from it.

u = 2^-24 is binary32's unit roundoff; a stored value adds half a step of its
type, eps/2 of the value (and half the smallest subnormal).  A binary32 sum of
n terms whose longest chain of additions is k is off by at most k u sum|term|
to first order.  The kernels' chains: at most 32 terms in a thread of the
kernels that keep a row on the chip, N / 512 in one of those that do not, then
at most 10 halving steps; k = 48 + N / 256 covers both.  Sums over the T rows
for the weight's gradient are bounded by k = T + 40 whatever their order.
Every bound is doubled, which covers the second-order terms left out."""
import numpy as np
import torch

import oracle as O

U = 2.0 ** -24
DROP_TAG = 0x44524F50


def half_step(v, dtype):
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def chain(N):
    return 48 + N / 256


def norm_fwd(x, w, b, eps, center):
    """(y, mean, rstd) in binary64 and their error bounds, y's without the
    last rounding."""
    x, w = x.double(), w.double()
    N = x.shape[1]
    k = chain(N)
    mean = x.mean(1, keepdim=True) if center else torch.zeros(len(x), 1, dtype=torch.float64)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    y = d * rstd * w + (b.double() if b is not None else 0.0)
    e_mean = k * U * x.abs().mean(1, keepdim=True) if center else 0.0 * mean
    # sum of (d + e)^2: the first-order term 2 e sum(d) vanishes about the
    # mean; each square and the chain cost relative roundings
    rel_rstd = 0.5 * ((k + 4) * U + (e_mean ** 2 + 2 * U * e_mean * d.abs().mean(1, keepdim=True))
                      * rstd ** 2) + 2 * U
    e_y = w.abs() * rstd * (e_mean + U * d.abs()) + (d * rstd * w).abs() * (rel_rstd + 3 * U) \
        + U * y.abs()
    return (y, mean[:, 0], rstd[:, 0]), (2 * e_y, 2 * e_mean[:, 0] + U * mean[:, 0].abs(),
                                         2 * (rel_rstd * rstd)[:, 0])


def norm_bwd(dy, x, w, mean, rstd, center, dres=None):
    """(dx + dres, dw, db) in binary64 and their bounds; mean and rstd are the
    binary32 inputs of the call, taken as exact."""
    dy, x, w, rstd = dy.double(), x.double(), w.double(), rstd.double()[:, None]
    T, N = x.shape
    k = chain(N)
    xh = (x - (mean.double()[:, None] if center else 0.0)) * rstd
    g = dy * w
    c1 = g.mean(1, keepdim=True) if center else torch.zeros(T, 1, dtype=torch.float64)
    c2 = (g * xh).mean(1, keepdim=True)
    res = dres.double() if dres is not None else torch.zeros_like(x)
    dx = rstd * (g - c1 - xh * c2) + res
    e_c1 = (k + 2) * U * g.abs().mean(1, keepdim=True) if center else 0.0
    e_c2 = (k + 6) * U * (g * xh).abs().mean(1, keepdim=True)
    e_dx = rstd * (e_c1 + xh.abs() * e_c2 + 6 * U * (g.abs() + c1.abs() + (xh * c2).abs())) \
        + 2 * U * (res.abs() + dx.abs())
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (T + 40) * U * (dy * xh).abs().sum(0)
    e_db = (T + 40) * U * dy.abs().sum(0)
    return (dx, dw, db), (2 * e_dx, 2 * e_dw, 2 * e_db)


def kept(T, N, p, seed, step=0):
    """The kept elements of dropout, from the oracle's Philox, and the scale."""
    key = (seed + step) & ((1 << 64) - 1)
    k = [key & 0xFFFFFFFF, key >> 32]
    groups = -(-N // 8)
    words = np.empty((T, groups, 4), np.uint32)
    for r in range(T):
        for j in range(groups):
            words[r, j] = O.philox4x32([j, r, 0, DROP_TAG], k, 7)
    u = words.view(np.uint16).reshape(T, groups * 8)[:, :N]  # little endian: low half first
    t = min(int(np.rint(p * 65536.0)), 65535)
    return torch.from_numpy(u.astype(np.int64) >= t), 65536.0 / (65536 - t)


def drop(x, mask, scale):
    """dropout(x) in binary64 and its bound (the scale and the product rounded)."""
    y = torch.where(mask, x.double() * scale, 0.0)
    return y, 3 * U * torch.where(mask, y.abs(), 0.0)


def swiglu_bwd(z, dh):
    """dz in binary64 and its bound.  exp is within 2 units in the last place
    (4 u), so sg and 1 - sg are within 8 u of their largest value 1, sg within
    8 u of itself."""
    F = dh.shape[1]
    g, up, dh = z[:, :F].double(), z[:, F:].double(), dh.double()
    sg = torch.sigmoid(g)
    t = 1.0 + g * (1.0 - sg)
    dg, du = dh * up * sg * t, dh * g * sg
    e_dg = (dh * up * sg).abs() * (16 * U * (1.0 + g.abs()) + 4 * U * t.abs())
    e_du = 16 * U * du.abs()
    # where exp overflows binary32 (g < -88.7) sg is flushed to zero
    tiny = (dh * up).abs().clamp(min=0) * 2.0 ** -126 * (1 + g.abs()), dh.abs() * g.abs() * 2.0 ** -126
    return torch.cat([dg, du], 1), 2 * torch.cat([e_dg + tiny[0], e_du + tiny[1]], 1)


def check(name, got, want, bound, dtype=None):
    """|got - want| <= bound (+ half a step of the stored type at the value
    furthest from zero that the bound allows), element by element."""
    got, want = got.detach().double().cpu(), want.cpu()
    bound = bound.cpu() if isinstance(bound, torch.Tensor) else torch.full_like(want, float(bound))
    if dtype is not None:
        bound = bound + half_step(want.abs() + bound, dtype)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values out of bounds; first at {i}: "
                             f"got {got[i]:.9g} want {want[i]:.9g} off {off[i]:.3g} > {bound[i]:.3g}")
