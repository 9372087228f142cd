"""Dropout from the counter-based generator against the oracle's Philox (the
kept elements exactly, the values within one rounding), and the SwiGLU
producer's backward pass, against 64-bit plain forms (rows_ref.py)."""
import pytest
import torch

import fp4_quantization_block_b200 as fa
import rows_ref as R
from gpu_util import need_gpu
from test_gpu_norm import SEED, TYPES, held

pytestmark = pytest.mark.gpu


def rand(T, N, seed):
    return torch.randn(T, N, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("T,N,pad,offset", [(1, 1, 0, 0), (1, 4096, 0, 0), (33, 4096, 8, 0),
                                            (7, 1001, 0, 0), (40, 72, 3, 1), (300, 24, 0, 0),
                                            (5, 2056, 0, 4)], ids=lambda v: str(v))
@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
def test_dropout(T, N, pad, offset, residual, dtype):
    need_gpu()
    p = 0.1
    x, r = held(rand(T, N, 1) + 3.0, dtype, pad, offset), held(rand(T, N, 2), dtype, pad, offset)
    step = torch.tensor([12345678901], dtype=torch.int64, device="cuda")
    out = held(torch.zeros(T, N), dtype, pad, offset, fill=7.0)
    y = fa.dropout_fwd(x, p, SEED, step=step, residual=r if residual else None, out=out)
    mask, scale = R.kept(T, N, p, SEED, 12345678901)
    want, bound = R.drop(x.cpu(), mask, scale)
    if residual:
        want = want + r.cpu().double()
        bound = bound + R.U * want.abs()
        assert torch.equal(y.cpu()[~mask], r.cpu()[~mask])
    else:
        assert torch.equal(y.cpu() != 0, mask)  # no element of x is zero
        assert torch.equal(y, fa.dropout_bwd(x, p, SEED, step=step))
    R.check("y", y, want, bound, dtype)
    whole = torch.as_strided(out, (T, N + pad), (N + pad, 1), out.storage_offset())
    assert torch.all(whole[:, N:] == 7.0)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 0.5, 0.9999, 1 - 2.0 ** -40])
def test_probabilities(p):
    """p in steps of 2^-16: none dropped, one step, nearly all; the rate is
    within six standard deviations of the exact one."""
    need_gpu()
    T, N = 512, 4096
    x = torch.full((T, N), 1.0, device="cuda")
    y = fa.dropout_fwd(x, p, 77)
    t = min(round(p * 65536), 65535)
    q = t / 65536
    dropped = float((y == 0).double().mean())
    assert abs(dropped - q) <= 6 * (q * (1 - q) / (T * N)) ** 0.5 + 1e-12
    vals = y[y != 0].unique()
    if vals.numel():
        assert vals.numel() == 1
        scale = 65536 / (65536 - t)
        assert abs(float(vals[0]) - scale) <= R.U * scale
    if t == 0:
        assert torch.equal(x, y)


def test_rows_keys_and_steps_are_independent():
    """Correlation between the masks of neighbouring rows, column blocks, seeds
    and steps stays within six standard deviations of zero."""
    need_gpu()
    T, N = 512, 4096
    x = torch.full((T, N), 1.0, device="cuda")
    m = [(fa.dropout_fwd(x, 0.5, s) != 0).double() - 0.5 for s in (1, 2, 1 << 32)]
    lim = 6 * 0.25 / (T * N) ** 0.5
    pairs = [(m[0], m[1]), (m[0], m[2]), (m[0][1:], m[0][:-1]), (m[0][:, 8:], m[0][:, :-8]),
             (m[0][:, 1:], m[0][:, :-1])]
    for a, b in pairs:
        assert abs(float((a * b).mean())) <= lim * 1.01


def test_dropped_infinities_and_nan_leave_no_trace():
    need_gpu()
    T, N = 16, 256
    x = rand(T, N, 4).cuda()
    mask, _ = R.kept(T, N, 0.5, 9)
    clean = fa.dropout_fwd(x, 0.5, 9)
    bad = x.clone()
    bad[~mask.cuda()] = float("nan")
    bad[0][~mask.cuda()[0]] = float("inf")
    assert torch.equal(fa.dropout_fwd(bad, 0.5, 9), clean)


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("T,N,pad,offset", [(1501, 4099, 0, 0), (1502, 4096, 3, 1), (40003, 257, 0, 0),
                                            (1500, 4090, 2, 2), (4001, 1000, 0, 3)], ids=lambda v: str(v))
def test_many_unaligned_rows_are_those_of_an_aligned_matrix(T, N, pad, offset, dtype):
    """The mask depends on the row and the column alone: the first N columns of
    a wider, aligned matrix come out the same bits, alone, with a residual and
    in place, and nothing around the rows changes."""
    need_gpu()
    M = -(-N // 8) * 8 + 8
    g = torch.Generator(device="cuda").manual_seed(N)
    wide = [torch.randn(T, M, generator=g, device="cuda").to(dtype) for _ in range(2)]
    x, r = (held(m[:, :N], dtype, pad, offset) for m in wide)
    out = held(torch.zeros(1, 1).expand(T, N), dtype, pad, offset, fill=7.0)
    want = fa.dropout_fwd(wide[0], 0.1, SEED)[:, :N]
    assert torch.equal(fa.dropout_fwd(x, 0.1, SEED, out=out), want)
    want = fa.dropout_fwd(wide[0], 0.1, SEED, residual=wide[1])[:, :N]
    assert torch.equal(fa.dropout_fwd(x, 0.1, SEED, residual=r, out=out), want)
    whole = torch.as_strided(out, (T, N + pad), (N + pad, 1), out.storage_offset())
    assert torch.all(whole[:, N:] == 7.0)
    assert torch.all(torch.as_strided(out, (64,), (1,), out.storage_offset() + T * (N + pad)) == 7.0)
    a, c = x.clone(), r.clone()
    assert torch.equal(fa.dropout_fwd(x, 0.1, SEED, residual=c, out=c), want)
    assert torch.equal(fa.dropout_fwd(a, 0.1, SEED, residual=r, out=a), want)


@pytest.mark.parametrize("N", [64, 1001])
def test_dropout_in_place(N):
    need_gpu()
    x, r = rand(50, N, 1).cuda(), rand(50, N, 2).cuda()
    want = fa.dropout_fwd(x, 0.3, 5, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(fa.dropout_fwd(a, 0.3, 5, residual=r, out=a), want)
    assert torch.equal(fa.dropout_fwd(x, 0.3, 5, residual=b, out=b), want)


def test_dropout_past_32_bit_offsets():
    need_gpu()
    T, N = 70000, 32768
    x = torch.full((1, 1), 1.0, dtype=torch.bfloat16, device="cuda").expand(T, N).contiguous()
    y = fa.dropout_fwd(x, 0.5, 3, out=x)
    for r in (0, 65537, T - 1):
        mask, _ = R.kept(1, 8, 0.5, 3) if r == 0 else (None, None)
        if mask is not None:
            assert torch.equal(y[0, :8].cpu() != 0, mask[0])
        assert abs(float((y[r] != 0).float().mean()) - 0.5) < 6 * 0.5 / N ** 0.5


def test_gradient_against_differences():
    """Dropout is linear in x: <dx, v> is the change of <y, dy> along v."""
    need_gpu()
    x, dy, v = (rand(20, 333, k).cuda() for k in (1, 2, 3))
    dx = fa.dropout_bwd(dy, 0.2, 11).double()
    y0 = fa.dropout_fwd(x, 0.2, 11).double()
    y1 = fa.dropout_fwd(x + v, 0.2, 11).double()
    want = ((y1 - y0) * dy.double()).sum()
    terms = dx * ((x + v).double() - x.double())
    # the two forward passes round once each (u), dx once, the scale once
    tol = 4 * R.U * ((y1.abs() + y0.abs()) * dy.double().abs()).sum() + 4 * R.U * terms.abs().sum()
    assert abs(float(terms.sum() - want)) <= float(tol)


# ------------------------------------------------------- SwiGLU backward ---

def swiglu_inputs(T, F, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    gate = torch.randn(T, F, generator=g) * 3
    gate.view(-1)[::53] *= 15.0
    up = torch.randn(T, F, generator=g)
    dh = torch.randn(T, F, generator=g) * torch.randn(T, 1, generator=g).exp() * 1e-2
    z = held(torch.cat([gate, up], 1), torch.bfloat16, pad)
    return z, held(dh, torch.bfloat16, pad)


@pytest.mark.parametrize("T,F,pad", [(1, 8, 0), (3, 32, 8), (200, 160, 0), (31, 2056, 16),
                                     (96, 14336, 0), (513, 1024, 0)], ids=lambda v: str(v))
def test_swiglu_bwd(T, F, pad):
    need_gpu()
    z, dh = swiglu_inputs(T, F, seed=T + F, pad=pad)
    out = held(torch.zeros(T, 2 * F), torch.bfloat16, pad, fill=7.0)
    dz = fa.swiglu_bwd(z, dh, out=out)
    want, bound = R.swiglu_bwd(z.cpu(), dh.cpu())
    R.check("dz", dz, want, bound, torch.bfloat16)
    whole = torch.as_strided(out, (T, 2 * F + pad), (2 * F + pad, 1))
    assert torch.all(whole[:, 2 * F:] == 7.0)
    zi = z.clone() if pad == 0 else z
    assert torch.equal(fa.swiglu_bwd(zi, dh, out=zi), dz)


def test_swiglu_bwd_every_finite_gate():
    need_gpu()
    bits = torch.arange(1 << 16, dtype=torch.int32)
    g = bits[((bits >> 7) & 0xFF) != 0xFF].to(torch.int16).view(torch.bfloat16)
    g = torch.cat([g, g.new_zeros(-len(g) % 256)]).view(-1, 256)
    z = torch.cat([g, torch.full_like(g, 1.5)], 1).cuda()
    dh = torch.full_like(g, 0.75).cuda()
    want, bound = R.swiglu_bwd(z.cpu(), dh.cpu())
    R.check("dz", fa.swiglu_bwd(z, dh), want, bound, torch.bfloat16)


def test_swiglu_bwd_against_differences():
    """dz along a direction against central differences of the 64-bit forward
    pass: the bf16 roundings of dz (2^-9 each) and the differences' error."""
    need_gpu()
    z, dh = swiglu_inputs(9, 64, seed=3)
    dz = fa.swiglu_bwd(z, dh).double().cpu()
    zc, dc = z.double().cpu(), dh.double().cpu()
    g = torch.Generator().manual_seed(2)

    def loss(v):
        gate, up = v.chunk(2, 1)
        return float((gate * torch.sigmoid(gate) * up * dc).sum())

    for _ in range(8):
        v = torch.randn(zc.shape, generator=g, dtype=torch.float64)
        want = (loss(zc + 1e-4 * v) - loss(zc - 1e-4 * v)) / 2e-4
        terms = (dz * v)
        tol = (2.0 ** -8 + 1e-6) * float(terms.abs().sum())
        assert abs(float(terms.sum()) - want) <= tol
