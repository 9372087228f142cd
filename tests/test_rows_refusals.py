"""Refusals of the row-wise training operators, on the host before any launch:
the C calls' argument checks and the bindings' checks of shapes, types and
devices.  No GPU is needed."""
import ctypes
import math

import pytest
import torch

import fp4_quantization_block_b200 as fa

DEV = 0x7F0000000000  # never dereferenced: every call below fails validation first
BF16, FP32, FP16 = 0, 1, 2


def norm_fwd(**k):
    a = dict(x=DEV, ldx=64, T=4, N=64, dt=BF16, w=DEV, b=DEV, wd=BF16, eps=1e-5, center=1, y=DEV,
             ldy=64, mean=DEV, rstd=DEV)
    a.update(k)
    return fa.lib().fa4_layernorm_fwd(*a.values(), None)


def norm_bwd(**k):
    a = dict(dy=DEV, lddy=64, x=DEV, ldx=64, dres=None, lddres=0, T=4, N=64, dt=BF16, w=DEV, wd=BF16,
             center=1, mean=DEV, rstd=DEV, dx=DEV, lddx=64, dw=DEV, db=DEV, ws=DEV, wsb=1 << 24)
    a.update(k)
    return fa.lib().fa4_layernorm_bwd(*a.values(), None)


def drop_fwd(**k):
    a = dict(x=DEV, ldx=64, res=None, ldres=0, T=4, N=64, dt=BF16, p=0.1, seed=1, step=None, y=DEV,
             ldy=64)
    a.update(k)
    return fa.lib().fa4_dropout_fwd(*a.values(), None)


def drop_bwd(**k):
    a = dict(x=DEV, ldx=64, T=4, N=64, dt=BF16, p=0.1, seed=1, step=None, y=DEV, ldy=64)
    a.update(k)
    return fa.lib().fa4_dropout_bwd(*a.values(), None)


def fused_fwd(**k):
    a = dict(x=DEV, ldx=64, res=DEV, ldres=64, T=4, N=64, dt=BF16, p=0.1, seed=1, step=None, w=DEV,
             b=DEV, wd=BF16, eps=1e-5, center=1, s=DEV, lds=64, y=DEV, ldy=64, mean=DEV, rstd=DEV)
    a.update(k)
    return fa.lib().fa4_dropout_add_layernorm_fwd(*a.values(), None)


def fused_bwd(**k):
    a = dict(dy=DEV, lddy=64, ds=DEV, ldds=64, s=DEV, lds=64, T=4, N=64, dt=BF16, p=0.1, seed=1,
             step=None, w=DEV, wd=BF16, center=1, mean=DEV, rstd=DEV, dx=DEV, lddx=64, dres=DEV,
             lddres=64, dw=DEV, db=DEV, ws=DEV, wsb=1 << 24)
    a.update(k)
    return fa.lib().fa4_dropout_add_layernorm_bwd(*a.values(), None)


def swiglu_bwd(**k):
    a = dict(z=DEV, ldz=128, dh=DEV, lddh=64, T=4, F=64, dz=DEV, lddz=128)
    a.update(k)
    return fa.lib().fa4_swiglu_bwd(*a.values(), None)


SHAPE = [(dict(T=0), 2), (dict(T=-1), 2), (dict(N=0), 2), (dict(T=1 << 32), 2),
         (dict(N=1 << 31, ldx=1 << 32), 2), (dict(dt=3), 1), (dict(dt=-1), 1)]
WEIGHT = [(dict(w=None), 1), (dict(wd=5), 1), (dict(wd=FP16), 4), (dict(dt=FP32, wd=BF16), 4),
          (dict(w=DEV + 1), 3), (dict(wd=FP32, w=DEV + 2), 3)]
STATS = [(dict(rstd=None), 1), (dict(mean=None), 1), (dict(center=2), 1), (dict(rstd=DEV + 2), 3)]
DROP = [(dict(p=1.0), 1), (dict(p=-0.1), 1), (dict(p=math.nan), 1), (dict(p=math.inf), 1),
        (dict(step=DEV + 4), 3)]
WS = [(dict(ws=None), 5), (dict(wsb=300), 5), (dict(ws=DEV + 8), 3), (dict(dw=None), 1),
      (dict(dw=DEV + 2), 3), (dict(db=DEV + 1), 3)]


@pytest.mark.parametrize("call,cases", [
    (norm_fwd, SHAPE + WEIGHT + STATS + [
        (dict(x=None), 1), (dict(y=None), 1), (dict(ldx=63), 2), (dict(ldy=63), 2), (dict(x=DEV + 1), 3),
        (dict(y=DEV + 1), 3), (dict(b=DEV + 1), 3), (dict(eps=-1e-9), 1), (dict(eps=math.nan), 1),
        (dict(eps=math.inf), 1)]),
    (norm_bwd, SHAPE + WEIGHT + STATS + WS + [
        (dict(dy=None), 1), (dict(x=None), 1), (dict(dx=None), 1), (dict(lddy=63), 2),
        (dict(ldx=63), 2), (dict(lddx=63), 2), (dict(dres=DEV, lddres=63), 2),
        (dict(dres=DEV + 1, lddres=64), 3), (dict(dt=FP32, wd=FP32, dy=DEV + 2), 3)]),
    (drop_fwd, SHAPE + DROP + [
        (dict(x=None), 1), (dict(y=None), 1), (dict(ldx=63), 2), (dict(ldy=63), 2),
        (dict(res=DEV, ldres=63), 2), (dict(res=DEV + 1, ldres=64), 3), (dict(x=DEV + 1), 3)]),
    (drop_bwd, SHAPE + DROP + [(dict(x=None), 1), (dict(y=None), 1), (dict(ldx=63), 2),
                               (dict(ldy=63), 2), (dict(y=DEV + 1), 3)]),
    (fused_fwd, SHAPE + WEIGHT + STATS + DROP + [
        (dict(x=None), 1), (dict(res=None), 1), (dict(s=None), 1), (dict(y=None), 1),
        (dict(ldres=63), 2), (dict(lds=63), 2), (dict(eps=-1.0), 1)]),
    (fused_bwd, SHAPE + WEIGHT + STATS + DROP + WS + [
        (dict(dy=None), 1), (dict(s=None), 1), (dict(dx=None), 1), (dict(dres=None), 1),
        (dict(ldds=63), 2), (dict(lds=63), 2), (dict(lddres=63), 2), (dict(lddx=63), 2)]),
    (swiglu_bwd, [
        (dict(z=None), 1), (dict(dh=None), 1), (dict(dz=None), 1), (dict(T=0), 2), (dict(F=0), 2),
        (dict(F=60), 2), (dict(ldz=120), 2), (dict(ldz=132), 2), (dict(lddh=56), 2), (dict(lddh=68), 2),
        (dict(lddz=120), 2), (dict(z=DEV + 8), 3), (dict(dh=DEV + 8), 3), (dict(dz=DEV + 8), 3)]),
], ids=["norm_fwd", "norm_bwd", "drop_fwd", "drop_bwd", "fused_fwd", "fused_bwd", "swiglu_bwd"])
def test_c_calls_reject_bad_arguments(call, cases):
    for case, expect in cases:
        assert call(**case) == expect, case


OUT = DEV + (1 << 20)


@pytest.mark.parametrize("call,cases", [
    (norm_fwd, [dict(ldy=72), dict(ldx=72)]),
    (norm_bwd, [dict(dy=OUT, lddx=72), dict(x=OUT, lddx=72),
                dict(dy=OUT, x=OUT, dres=DEV, lddres=72)]),
    (drop_fwd, [dict(ldy=72), dict(x=OUT, res=DEV, ldres=72)]),
    (drop_bwd, [dict(ldy=72)]),
    (fused_fwd, [dict(), dict(s=OUT, ldy=72), dict(y=OUT, lds=72), dict(s=OUT, res=OUT, lds=72)]),
    (fused_bwd, [dict(), dict(dres=OUT, lddx=72), dict(dx=OUT, lddres=72),
                 dict(dx=OUT, dy=OUT, s=OUT, lddres=72)]),
    (swiglu_bwd, [dict(z=OUT), dict(dh=OUT, lddz=136)]),
], ids=["norm_fwd", "norm_bwd", "drop_fwd", "drop_bwd", "fused_fwd", "fused_bwd", "swiglu_bwd"])
def test_outputs_in_place_keep_their_inputs_rows(call, cases):
    """The same address under another leading dimension, and one matrix for
    two outputs."""
    for case in cases:
        assert call(**case) == 1, case


def test_workspace_sizes():
    n = ctypes.c_size_t()
    L = fa.lib()
    assert L.fa4_layernorm_ws_bytes(1, 1, ctypes.byref(n)) == 0 and n.value > 256
    assert L.fa4_layernorm_ws_bytes(1 << 20, 4096, ctypes.byref(n)) == 0
    assert 256 < n.value < 1184 * 2 * 4096 * 4 + 4096
    assert L.fa4_layernorm_ws_bytes(0, 64, ctypes.byref(n)) == 2
    assert L.fa4_layernorm_ws_bytes(64, 0, ctypes.byref(n)) == 2
    assert L.fa4_layernorm_ws_bytes(64, 64, None) == 1


def test_bindings_refuse_before_any_call():
    """Host tensors, wrong types and ranks never reach the library."""
    x = torch.zeros(4, 64)
    w = torch.ones(64)
    v = torch.zeros(4)
    for call in (lambda: fa.layer_norm_fwd(x, w), lambda: fa.layer_norm_bwd(x, x, w, v, v),
                 lambda: fa.dropout_fwd(x, 0.1, 1), lambda: fa.dropout_bwd(x, 0.1, 1),
                 lambda: fa.dropout_add_layer_norm_fwd(x, x, w, w, 0.1, 1),
                 lambda: fa.dropout_add_layer_norm_bwd(x, x, x, w, v, v, 0.1, 1),
                 lambda: fa.swiglu_bwd(x, x), lambda: fa.dropout_fwd(x.double(), 0.1, 1),
                 lambda: fa.dropout_fwd(x[0], 0.1, 1), lambda: fa.dropout_fwd(None, 0.1, 1)):
        with pytest.raises(ValueError):
            call()


def test_vector_and_step_checks():
    dev = torch.device("cpu")
    fa._vector(torch.ones(8), 8, (torch.float32,), dev, "v")
    for v in (torch.ones(9), torch.ones(8, dtype=torch.float64), torch.ones(16)[::2],
              torch.ones(8, 1), None):
        with pytest.raises(ValueError):
            fa._vector(v, 8, (torch.float32,), dev, "v")
    x = torch.zeros(2, 2)
    assert fa._step(None, x) is None
    for s in (3, torch.zeros(1), torch.zeros(2, dtype=torch.int64)):
        with pytest.raises(ValueError):
            fa._step(s, x)


@pytest.mark.gpu
def test_bindings_refuse_mismatched_operands():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w, v = torch.ones(64, device="cuda"), torch.zeros(4, device="cuda")
    for call in (lambda: fa.layer_norm_fwd(x, w[:32]), lambda: fa.layer_norm_fwd(x, w.half()),
                 lambda: fa.layer_norm_fwd(x, w, w.bfloat16()), lambda: fa.layer_norm_fwd(x, w.cpu()),
                 lambda: fa.layer_norm_fwd(x.t(), w[:4]),
                 lambda: fa.layer_norm_fwd(x, w, out=torch.zeros_like(x, dtype=torch.float32)),
                 lambda: fa.layer_norm_fwd(x[:1].expand(4, 64), w),
                 lambda: fa.layer_norm_bwd(x[:3], x, w, v, v),
                 lambda: fa.layer_norm_bwd(x, x, w, v[:3], v),
                 lambda: fa.layer_norm_bwd(x, x, w, None, v),
                 lambda: fa.layer_norm_bwd(x, x, w, v, v, dweight=w.bfloat16()),
                 lambda: fa.layer_norm_bwd(x, x, w, v, v, ws=w),
                 lambda: fa.dropout_fwd(x, 0.1, 1, residual=x.float()),
                 lambda: fa.dropout_fwd(x, 0.1, 1, step=torch.zeros(1, dtype=torch.int64)),
                 lambda: fa.swiglu_bwd(x, x), lambda: fa.swiglu_bwd(x, x[:, :32].float())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fa.dropout_fwd(x, 1.0, 1), lambda: fa.dropout_fwd(x, -0.5, 1),
                 lambda: fa.layer_norm_fwd(x, w, eps=-1.0),
                 lambda: fa.layer_norm_bwd(x, x, w, v, v,
                                           ws=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                 lambda: fa.dropout_fwd(x[:0], 0.1, 1)):
        with pytest.raises(fa.FA4Error):
            call()


def test_the_diagnostic_of_the_cluster_waits_refuses_bad_limits_and_rows():
    def call(**k):
        a = dict(dy=DEV, x=DEV, T=4, N=64, w=DEV, mean=DEV, rstd=DEV, dx=DEV, dw=DEV, db=DEV, row=-1, ns=1000,
                 ws=DEV, wsb=1 << 24)
        a.update(k)
        return fa.lib().fa4_debug_layernorm_bwd_timeout(*a.values(), None)

    for case, expect in [(dict(ns=0), 1), (dict(ns=2_000_000_001), 1), (dict(row=4), 1), (dict(row=-2), 1),
                         (dict(x=None), 1), (dict(mean=None), 1), (dict(T=0), 2), (dict(ws=None), 5),
                         (dict(wsb=300), 5), (dict(dx=DEV + 1), 3)]:
        assert call(**case) == expect, case


@pytest.mark.parametrize("call,case", [
    (norm_fwd, dict(mean=OUT, rstd=OUT)), (fused_fwd, dict(s=OUT, mean=OUT + 64, rstd=OUT + 64)),
    (norm_bwd, dict(dw=OUT, db=OUT)), (fused_bwd, dict(dres=OUT, dw=OUT + 64, db=OUT + 64)),
], ids=["norm_fwd", "fused_fwd", "norm_bwd", "fused_bwd"])
def test_one_vector_for_two_outputs_is_refused(call, case):
    """Statistics, or sums, that would overwrite one another."""
    if torch.cuda.is_available():
        pytest.skip("validation is tested without a GPU")
    assert call(**case) == 1


def test_the_diagnostics_binding_refuses_host_tensors():
    x, w, v = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16), torch.zeros(4)
    with pytest.raises(ValueError):
        fa.debug_layer_norm_bwd_timeout(x, x, w, v, v, 0, 1000, torch.zeros(1 << 16, dtype=torch.uint8))
