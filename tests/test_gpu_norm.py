"""Layer norm and its fusion with dropout and the residual addition, forward
and backward, against 64-bit plain forms (rows_ref.py) within bounds derived
there: every type, row lengths that end inside a chunk, a warp or a CTA's
columns, leading dimensions and offsets that are not aligned, one row and many,
extreme rows, in-place outputs, other streams, captured graphs."""
import pytest
import torch

import fp4_quantization_block_b200 as fa
import rows_ref as R
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
SEED = 0xFEDCBA9876543210


def held(x, dtype, pad=0, offset=0, fill=None):
    """x on the GPU in `dtype`, its rows x.shape[1] + pad apart, starting
    `offset` elements into a 16-byte aligned buffer."""
    T, N = x.shape
    buf = torch.full((T * (N + pad) + offset + 64,), 0.0 if fill is None else fill, dtype=dtype,
                     device="cuda")
    v = buf[offset:offset + T * (N + pad)].view(T, N + pad)[:, :N]
    v.copy_(x)
    return v


def inputs(T, N, dtype, seed, wtype=None, bias=True, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, N, generator=g) + 0.5 * torch.randn(1, N, generator=g) + 0.3
    x[:, :: 97] *= 20.0
    r = torch.randn(T, N, generator=g)
    dy = torch.randn(T, N, generator=g) * torch.randn(T, 1, generator=g).exp() * 1e-2
    ds = torch.randn(T, N, generator=g) * 1e-2
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(wtype or dtype)
    b = (0.2 * torch.randn(N, generator=g)).to(wtype or dtype) if bias else None
    mats = [held(m, dtype, pad, offset) for m in (x, r, dy, ds)]
    return mats, w.cuda(), b.cuda() if bias else None


def cpu(*ts):
    return [None if t is None else t.cpu() for t in ts]


def check_fwd(x, w, b, center, y, mean, rstd):
    xc, wc, bc = cpu(x, w, b)
    (ye, me, re), (by, bm, br) = R.norm_fwd(xc, wc, bc, EPS, center)
    R.check("y", y, ye, by, y.dtype)
    R.check("rstd", rstd, re, br)
    if center:
        R.check("mean", mean, me, bm)
    else:
        assert mean is None


def check_bwd(dy, x, w, mean, rstd, center, dres, dx, dw, db):
    c = cpu(dy, x, w, mean, rstd, dres)
    (dxe, dwe, dbe), (bx, bw, bb) = R.norm_bwd(c[0], c[1], c[2], c[3], c[4], center, c[5])
    R.check("dx", dx, dxe, bx, dx.dtype)
    R.check("dweight", dw, dwe, bw)
    if db is not None:
        R.check("dbias", db, dbe, bb)


# row lengths: one value, less than a chunk, chunks that end inside a warp,
# the borders of each layout, odd ones, and rows too long for the chip's ring
SHAPES = [(1, 1), (3, 5), (5, 8), (37, 64), (64, 200), (9, 256), (130, 264), (33, 512), (17, 520),
          (40, 1000), (1, 1024), (300, 1032), (67, 2048), (1, 4096), (150, 4096), (21, 4099),
          (700, 768), (5, 8192), (12, 8200), (7, 14336), (4, 16384), (3, 16392), (2, 28672),
          (2, 40001)]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("T,N", SHAPES, ids=[f"{t}x{n}" for t, n in SHAPES])
def test_norm_fwd_and_bwd(T, N, dtype):
    need_gpu()
    (x, _, dy, ds), w, b = inputs(T, N, dtype, seed=T * 100003 + N)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    check_fwd(x, w, b, True, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, True, None, dx, dw, db)
    dx, dw2, db2 = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    check_bwd(dy, x, w, mean, rstd, True, ds, dx, dw2, db2)
    assert torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("T,N", [(19, 72), (33, 1000), (50, 4096), (6, 14336), (2, 20000)],
                         ids=lambda v: str(v))
def test_rms_form_and_binary32_weights(T, N, dtype):
    need_gpu()
    (x, _, dy, ds), w, _ = inputs(T, N, dtype, seed=N, wtype=torch.float32, bias=False)
    y, mean, rstd = fa.layer_norm_fwd(x, w, None, EPS, center=False)
    check_fwd(x, w, None, False, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, None, rstd, center=False, bias_grad=False, dres=ds)
    assert db is None
    check_bwd(dy, x, w, None, rstd, False, ds, dx, dw, None)


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (2, 2)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("N", [1, 2, 40, 255, 256, 257, 300, 511, 512, 513, 768, 771, 1279, 1280, 4096, 4098,
                               4351, 18433])
def test_leading_dimensions_and_offsets(N, pad, offset, dtype):
    """Strided and offset matrices; what lies between the rows stays as it was."""
    need_gpu()
    T = 5
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=N + pad, pad=pad, offset=offset)
    outs = [held(torch.zeros(T, N), dtype, pad, offset, fill=7.0) for _ in range(4)]
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS, out=outs[0])
    check_fwd(x, w, b, True, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds, dx=outs[1])
    check_bwd(dy, x, w, mean, rstd, True, ds, dx, dw, db)
    y2, s, m2, r2 = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.25, SEED, out=outs[2], s=outs[3])
    assert torch.equal(s, fa.dropout_fwd(x, 0.25, SEED, residual=r))
    check_fwd(s, w, b, True, y2, m2, r2)
    for o in outs:
        whole = torch.as_strided(o, (T * (N + pad),), (1,), o.storage_offset())
        between = whole.view(T, N + pad)[:, N:]
        assert torch.all(between == 7.0)
        base = torch.as_strided(o, (offset,), (1,), 0)
        end = torch.as_strided(o, (64,), (1,), o.storage_offset() + T * (N + pad))
        assert torch.all(base == 7.0) and torch.all(end == 7.0)


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("center", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("T,N,p", [(1, 1, 0.5), (3, 13, 0.1), (40, 512, 0.1), (17, 1001, 0.0),
                                   (21, 4096, 0.1), (3, 14336, 0.5), (2, 17000, 0.25)],
                         ids=lambda v: str(v))
def test_fused_with_dropout_and_residual(T, N, p, center, dtype):
    need_gpu()
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=T + N)
    step = torch.tensor([41], dtype=torch.int64, device="cuda")
    y, s, mean, rstd = fa.dropout_add_layer_norm_fwd(x, r, w, b, p, SEED, step=step, center=center)
    mask, scale = R.kept(T, N, p, SEED, 41)
    xc, rc = cpu(x, r)
    de, db_ = R.drop(xc, mask, scale)
    se = rc.double() + de
    R.check("s", s, se, db_ + R.U * se.abs(), dtype)
    assert torch.equal(s, fa.dropout_fwd(x, p, SEED, step=step, residual=r))
    check_fwd(s, w, b, center, y, mean, rstd)

    for d in (ds, None):
        dx, dres, dw, db = fa.dropout_add_layer_norm_bwd(dy, d, s, w, mean, rstd, p, SEED, step=step,
                                                         center=center)
        check_bwd(dy, s, w, mean, rstd, center, d, dres, dw, db)
        c = cpu(dy, s, w, mean, rstd, d)
        (full, _, _), (bound, _, _) = R.norm_bwd(*c[:5], center, c[5])
        want, b3 = R.drop(full, mask, scale)
        R.check("dx", dx, want, torch.where(mask, bound * scale, 0.0) + b3, dtype)
        assert torch.all(dx.cpu()[~mask] == 0)


def test_against_differences():
    """dx, dweight and dbias against central differences of the 64-bit forward
    pass along random directions (binary32 inputs; the differences' own error
    at h = 1e-4 is below 1e-7 of the sums compared)."""
    need_gpu()
    T, N = 6, 96
    (x, _, dy, _), w, b = inputs(T, N, torch.float32, seed=5)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd)
    xc, wc, bc, dyc = (t.double().cpu() for t in (x, w, b, dy))
    g = torch.Generator().manual_seed(1)

    def loss(xv, wv, bv):
        d = xv - xv.mean(1, keepdim=True)
        return float(((d * (d.square().mean(1, keepdim=True) + EPS).rsqrt() * wv + bv) * dyc).sum())

    h = 1e-4
    for k in range(8):
        vx, vw, vb = (torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (xc, wc, bc))
        for v, grad, f in ((vx, dx, lambda e: loss(xc + e * vx, wc, bc)),
                           (vw, dw, lambda e: loss(xc, wc + e * vw, bc)),
                           (vb, db, lambda e: loss(xc, wc, bc + e * vb))):
            want = (f(h) - f(-h)) / (2 * h)
            terms = grad.double().cpu() * v
            # 64 u on each term covers the gradients' bounds at N = 96
            tol = 64 * R.U * float(terms.abs().sum()) + 1e-6 * float(terms.abs().sum())
            assert abs(float(terms.sum()) - want) <= tol, (k, float(terms.sum()), want)


@pytest.mark.parametrize("N", [512, 4096, 17000])
def test_extreme_rows(N):
    """A constant row, a row of zeros, a huge mean, tiny values; infinities and
    NaN stay in their rows."""
    need_gpu()
    (x, _, dy, _), w, b = inputs(8, N, torch.float32, seed=3)
    x[0] = 3.0
    x[1] = 0.0
    x[2] += 1.0e4
    x[3] *= 1e-30
    ref = x.clone()
    x[5, N // 2] = float("inf")
    x[6, 1] = float("nan")
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    fine = [0, 1, 2, 3, 4, 7]
    check_fwd(ref[fine], w, b, True, y[fine], mean[fine], rstd[fine])
    assert torch.isnan(y[5, N // 2]) and torch.isnan(y[6]).all()
    dx, _, _ = fa.layer_norm_bwd(dy, x, w, mean, rstd)
    dx2, _, _ = fa.layer_norm_bwd(dy[fine].contiguous(), ref[fine].contiguous(), w,
                                  mean[fine].contiguous(), rstd[fine].contiguous())
    assert torch.equal(dx[fine], dx2)


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("N", [5, 100, 264, 301, 520, 4099, 4104, 8705, 9001])
def test_rows_of_nan_leave_the_other_rows_alone(N, dtype):
    """Every fourth row of many is NaN or infinite; the others, which follow
    them through the same threads and the same memory, come out as if they were
    not there."""
    need_gpu()
    T = 1900
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=N)
    bad = torch.arange(T, device="cuda") % 4 == 1
    nan = torch.where(torch.arange(T, device="cuda")[:, None] % 8 == 1, float("nan"), float("inf")).to(dtype)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    dx, _, _ = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
    g = fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED)
    xb, dyb = torch.where(bad[:, None], nan, x), torch.where(bad[:, None], nan, dy)
    y2, mean2, rstd2 = fa.layer_norm_fwd(xb, w, b, EPS)
    dx2, _, _ = fa.layer_norm_bwd(dyb, xb, w, mean2, rstd2, dres=ds)
    f2 = fa.dropout_add_layer_norm_fwd(xb, r, w, b, 0.1, SEED)
    g2 = fa.dropout_add_layer_norm_bwd(dyb, ds, f2[1], w, f2[2], f2[3], 0.1, SEED)
    for a, c in ((y, y2), (mean, mean2), (rstd, rstd2), (dx, dx2), (f[0], f2[0]), (f[1], f2[1]),
                 (g[0], g2[0]), (g[1], g2[1])):
        assert torch.equal(a[~bad], c[~bad])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [96, 4096, 4099, 17000])
def test_in_place(N, dtype):
    need_gpu()
    T = 9
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=N)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    xi = x.clone()
    fa.layer_norm_fwd(xi, w, b, EPS, out=xi)
    assert torch.equal(xi, y)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    for k in range(3):
        a = [dy.clone(), x.clone(), ds.clone()]
        _, dw2, db2 = fa.layer_norm_bwd(a[0], a[1], w, mean, rstd, dres=a[2], dx=a[k])
        assert torch.equal(a[k], dx) and torch.equal(dw, dw2) and torch.equal(db, db2)
    y, s, mean, rstd = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
    xi, ri = x.clone(), r.clone()
    fa.dropout_add_layer_norm_fwd(xi, ri, w, b, 0.1, SEED, out=xi, s=ri)
    assert torch.equal(xi, y) and torch.equal(ri, s)
    want = fa.dropout_add_layer_norm_bwd(dy, ds, s, w, mean, rstd, 0.1, SEED)
    di, si = dy.clone(), ds.clone()
    got = fa.dropout_add_layer_norm_bwd(di, si, s, w, mean, rstd, 0.1, SEED, dx=di, dres=si)
    assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("T,N,pad,offset", [(3, 32768, 0, 0), (2, 65536, 8, 0), (3, 65537, 0, 1),
                                            (9, 70000, 0, 0), (2, 131080, 0, 0)], ids=lambda v: str(v))
def test_rows_too_long_for_the_chip(T, N, pad, offset, dtype):
    """Row lengths about the borders of the layouts for long rows, up to those
    that are read again for each pass."""
    need_gpu()
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=N, pad=pad, offset=offset)
    y, s, mean, rstd = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
    assert torch.equal(s, fa.dropout_fwd(x, 0.1, SEED, residual=r))
    check_fwd(s, w, b, True, y, mean, rstd)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    check_fwd(x, w, b, True, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    check_bwd(dy, x, w, mean, rstd, True, ds, dx, dw, db)
    dx2, dres, dw2, db2 = fa.dropout_add_layer_norm_bwd(dy, ds, x, w, mean, rstd, 0.1, SEED)
    assert torch.equal(dres, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)
    mask = (fa.dropout_fwd(torch.ones_like(dx), 0.1, SEED) != 0).cpu()
    (full, _, _), (bound, _, _) = R.norm_bwd(*cpu(dy, x, w, mean, rstd), True, ds.cpu())
    scale = 65536 / (65536 - round(0.1 * 65536))
    want, b3 = R.drop(full, mask, scale)
    R.check("dx", dx2, want, torch.where(mask, bound * scale, 0.0) + b3, dtype)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 147, 149, 297, 1185, 3553])
@pytest.mark.parametrize("N", [24, 264, 1024, 8200])
def test_row_counts_about_the_layouts_borders(T, N):
    need_gpu()
    (x, _, dy, ds), w, b = inputs(T, N, torch.bfloat16, seed=T)
    y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    check_fwd(x, w, b, True, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    check_bwd(dy, x, w, mean, rstd, True, ds, dx, dw, db)


def test_a_workspace_of_exactly_the_size_asked_for():
    """The bytes behind it stay as they were, for row counts and lengths of
    every layout."""
    need_gpu()
    for T, N in [(1, 8), (5, 4096), (40, 4096), (500, 4096), (300, 8200), (60, 20000), (40, 40001),
                 (100, 70000)]:
        (x, _, dy, _), w, b = inputs(T, N, torch.bfloat16, seed=1)
        _, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
        n = fa.layer_norm_ws_bytes(T, N)
        buf = torch.full((n + 4096,), 85, dtype=torch.uint8, device="cuda")
        got = fa.layer_norm_bwd(dy, x, w, mean, rstd, ws=buf[:n])
        want = fa.layer_norm_bwd(dy, x, w, mean, rstd)
        assert torch.all(buf[n:] == 85), (T, N)
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_two_streams_at_once_and_two_graphs_with_a_workspace_each():
    need_gpu()
    sets = [inputs(400, 4096, torch.bfloat16, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in sets]
    want = []
    for (x, r, dy, ds), w, b in sets:
        f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
        want.append(f + fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [None, None]
        for k, ((x, r, dy, ds), w, b) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
                got[k] = f + fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED)
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, c))
    graphs, outs = [], []
    for k, ((x, r, dy, ds), w, b) in enumerate(sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[k]):
            f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
            outs.append(f + fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED))
        graphs.append(g)
    for _ in range(5):
        for k, g in enumerate(graphs):
            with torch.cuda.stream(streams[k]):
                g.replay()
    torch.cuda.synchronize()
    for a, c in zip(outs, want):
        assert all(torch.equal(u, v) for u, v in zip(a, c))


def test_repeats_bit_for_bit_with_a_dirty_workspace():
    need_gpu()
    T, N = 1000, 4096
    (x, _, dy, ds), w, b = inputs(T, N, torch.bfloat16, seed=8)
    _, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    first = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
    ws = torch.full((fa.layer_norm_ws_bytes(T, N),), 255, dtype=torch.uint8, device="cuda")
    again = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds, ws=ws)
    assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_many_rows_and_offsets_past_32_bits():
    """2^31 elements and more: rows beyond the 32-bit range of an element
    offset, sampled."""
    need_gpu()
    T, N = 70000, 32768
    x = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.linspace(0.5, 1.5, N, device="cuda").bfloat16()
    y, mean, rstd = fa.layer_norm_fwd(x, w, None, EPS, out=x.clone())
    rows = [0, 65535, 65536, T - 1]
    check_fwd(x[rows], w, None, True, y[rows], mean[rows], rstd[rows])
    dx, _, _ = fa.layer_norm_bwd(y, x, w, mean, rstd, dx=y.clone())
    c = cpu(y[rows], x[rows], w, mean[rows], rstd[rows])
    (dxe, _, _), (bx, _, _) = R.norm_bwd(*c, True)
    R.check("dx", dx[rows], dxe, bx, dx.dtype)


@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float16, torch.float16), (torch.float32, torch.float32)],
                         ids=["bf16", "bf16-w32", "fp16", "fp32"])
@pytest.mark.parametrize("N", [7, 512, 1032, 4096, 4099, 9000, 70000])
def test_weights_off_16_byte_boundaries_and_gradients_in_the_callers_tensors(N, dtype, wtype):
    need_gpu()
    T = 40
    (x, r, dy, ds), w, b = inputs(T, N, dtype, seed=N, wtype=wtype)
    wide = torch.zeros(2 * N + 16, dtype=wtype, device="cuda")
    w1, b1 = wide[1:N + 1], wide[N + 4:2 * N + 4]
    w1.copy_(w)
    b1.copy_(b)
    y, mean, rstd = fa.layer_norm_fwd(x, w1, b1, EPS)
    check_fwd(x, w, b, True, y, mean, rstd)
    grads = torch.full((2 * N + 9,), 7.0, device="cuda")
    dw, db = grads[1:N + 1], grads[N + 5:2 * N + 5]
    dx, gw, gb = fa.layer_norm_bwd(dy, x, w1, mean, rstd, dres=ds, dweight=dw, dbias=db)
    assert gw is dw and gb is db
    check_bwd(dy, x, w, mean, rstd, True, ds, dx, dw, db)
    assert grads[0] == 7.0 and torch.all(grads[N + 1:N + 5] == 7.0) and torch.all(grads[2 * N + 5:] == 7.0)
    assert torch.equal(wide[N + 1:N + 4], torch.zeros_like(wide[N + 1:N + 4]))


def test_single_rows_and_columns_of_any_stride():
    """One row's stride means nothing, one column's either."""
    need_gpu()
    big = torch.randn(64, 4096, device="cuda")
    w, b = torch.rand(64, device="cuda") + 0.5, torch.rand(64, device="cuda")
    row = big.t()[5:6, :]  # strides (1, 4096): no unit column stride
    with pytest.raises(ValueError):
        fa.layer_norm_fwd(row, w, b)
    one = torch.as_strided(big, (1, 64), (3, 1), 7)
    y, mean, rstd = fa.layer_norm_fwd(one, w, b)
    check_fwd(one, w, b, True, y, mean, rstd)
    col = big[:, 9:10]
    y, mean, rstd = fa.layer_norm_fwd(col, w[:1], b[:1], center=False)
    check_fwd(col, w[:1], b[:1], False, y, mean, rstd)
    dx, dw, db = fa.layer_norm_bwd(col, col, w[:1], None, rstd, center=False)
    check_bwd(col, col, w[:1], None, rstd, False, None, dx, dw, db)
    thin = big[0:1, :].t()  # [4096, 1], strides (1, 4096)
    assert torch.equal(fa.dropout_fwd(thin, 0.5, 3), fa.dropout_fwd(thin.contiguous(), 0.5, 3))


def test_wide_rows_captured_and_replayed():
    """Rows shared by clusters, and few rows in one cluster, in a graph."""
    need_gpu()
    for T, N in ((50, 12296), (6, 4096), (70, 20001)):
        (x, r, dy, ds), w, b = inputs(T, N, torch.bfloat16, seed=T)
        f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
        want = fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_device_status_of_a_zeroed_workspace_is_clean():
    need_gpu()
    (x, _, dy, ds), w, b = inputs(100, 20000, torch.bfloat16, seed=4)
    _, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    ws = fa.workspace(fa.layer_norm_ws_bytes(100, 20000))
    fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds, ws=ws)
    assert fa.check_device_status(ws) == 0


def test_another_stream():
    need_gpu()
    (x, r, dy, ds), w, b = inputs(500, 4096, torch.bfloat16, seed=2)
    want = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
    wantb = fa.dropout_add_layer_norm_bwd(dy, ds, want[1], w, want[2], want[3], 0.1, SEED)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED)
        gotb = fa.dropout_add_layer_norm_bwd(dy, ds, got[1], w, got[2], got[3], 0.1, SEED)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got + gotb, want + wantb))


def test_captured_graph_draws_a_new_mask_at_each_replay():
    need_gpu()
    (x, r, dy, ds), w, b = inputs(64, 4096, torch.bfloat16, seed=2)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        f = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED, step=step)
        g = fa.dropout_add_layer_norm_bwd(dy, ds, f[1], w, f[2], f[3], 0.1, SEED, step=step)
    seen = []
    for k in (0, 1, 2 ** 40):
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        want = fa.dropout_add_layer_norm_fwd(x, r, w, b, 0.1, SEED + k)
        wantb = fa.dropout_add_layer_norm_bwd(dy, ds, want[1], w, want[2], want[3], 0.1, SEED + k)
        assert all(torch.equal(a, c) for a, c in zip(f + g, want + wantb))
        seen.append(f[1].clone())
    assert not torch.equal(seen[0], seen[1])
