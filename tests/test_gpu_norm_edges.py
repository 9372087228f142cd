"""Layer norm where its launch has borders of its own: rows for which one stage
of the ring is all that fits, calls from several host threads at once, waits
between CTAs that run out, sums over the rows that are exact, rows past 2^31
elements.  Bounds as in rows_ref.py."""
import threading

import numpy as np
import pytest
import torch

import fp4_quantization_block_b200 as fa
import oracle as O
import rows_ref as R
from gpu_util import need_gpu
from test_gpu_norm import EPS, SEED, TYPES, check_bwd, cpu, held, inputs

pytestmark = pytest.mark.gpu


def one_stage_inputs(T, N, pad):
    g = torch.Generator().manual_seed(T * 7 + N)
    mats = [held(torch.randn(T, N, generator=g) + m, torch.float32, pad) for m in (0.5, 0.0, 0.0)]
    # a weight that is nowhere what it is 4, 128 or 256 columns away
    w = (torch.randn(N, generator=g) * torch.logspace(-1, 1, N)).cuda()
    return mats, w


def cold_l2():
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(1)


@pytest.mark.parametrize("T,N,pad", [(40, 7681, 0), (40, 8191, 0), (40, 8192, 4), (17, 8192, 3),
                                     (1000, 8191, 0), (20, 15361, 0), (20, 16383, 0), (9, 30721, 0),
                                     (9, 32767, 0), (3, 61441, 0), (3, 65535, 0)], ids=lambda v: str(v))
@pytest.mark.parametrize("center", [True, False], ids=["layer", "rms"])
def test_backward_with_a_ring_of_one_stage(T, N, pad, center):
    """binary32 rows off 16-byte boundaries with a residual gradient fill the
    shared memory with one row's columns: the staged weight must have arrived
    all the same, in the plain and in the fused call."""
    need_gpu()
    (x, dy, ds), w = one_stage_inputs(T, N, pad)
    _, mean, rstd = fa.layer_norm_fwd(x, w, None, EPS, center=center)
    cold_l2()
    dx, dw, db = fa.layer_norm_bwd(dy, x, w, mean, rstd, center=center, dres=ds)
    check_bwd(dy, x, w, mean, rstd, center, ds, dx, dw, db)
    cold_l2()
    dx2, dres, dw2, db2 = fa.dropout_add_layer_norm_bwd(dy, ds, x, w, mean, rstd, 0.25, SEED, center=center)
    check_bwd(dy, x, w, mean, rstd, center, ds, dres, dw2, db2)
    mask = (fa.dropout_fwd(torch.ones_like(dx), 0.25, SEED) != 0).cpu()
    (full, _, _), (bound, _, _) = R.norm_bwd(*cpu(dy, x, w, mean, rstd), center, ds.cpu())
    want, b3 = R.drop(full, mask, 1 / 0.75)
    R.check("dx", dx2, want, torch.where(mask, bound / 0.75, 0.0) + b3, torch.float32)


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_host_threads_with_rows_of_different_lengths(backward):
    """C calls of one kernel that need different amounts of shared memory, from
    four threads at once, each on a stream of its own: none is refused, and
    each gives what it gives alone."""
    need_gpu()
    L, T = fa.lib(), 40
    sets = []
    for N in (4096, 8192, 6144, 2048):
        (x, _, dy, ds), w, b = inputs(T, N, torch.bfloat16, seed=N)
        y, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
        want = (y,) if not backward else fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)
        got = [torch.zeros_like(t) for t in want]
        ws = fa.workspace(fa.layer_norm_ws_bytes(T, N))
        st = torch.cuda.Stream()
        p = [t.data_ptr() for t in (x, dy, ds, w, b, mean, rstd, *got)]
        if backward:
            args = (p[1], N, p[0], N, p[2], N, T, N, 0, p[3], 0, 1, p[5], p[6], p[7], N, p[8], p[9],
                    ws.data_ptr(), ws.numel(), st.cuda_stream)
        else:
            args = (p[0], N, T, N, 0, p[3], p[4], 0, EPS, 1, p[7], N, p[5], p[6], st.cuda_stream)
        sets.append((args, got, want, (x, dy, ds, w, b, mean, rstd, ws, st)))
    torch.cuda.synchronize()
    call = L.fa4_layernorm_bwd if backward else L.fa4_layernorm_fwd
    start, refused = threading.Barrier(len(sets)), [0] * len(sets)

    def work(k):
        args = sets[k][0]
        start.wait()
        for _ in range(10000):
            refused[k] += call(*args) != 0

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(sets)
    for _, got, want, _ in sets:
        assert all(torch.equal(u, v) for u, v in zip(got, want))


# (T, N, a row, the rows that its team takes from it on): clusters of four, of
# two and of eight, one team each, and one cluster of eight for a few rows
LEFT = [(100, 20000, 5, [5, 38, 71]), (100, 20000, 99, [99]), (200, 12288, 73, [73, 147]),
        (40, 65536, 17, [17, 32]), (6, 4096, 2, [2])]


@pytest.mark.parametrize("T,N,row,left", LEFT, ids=[f"{c[0]}x{c[1]}-{c[2]}" for c in LEFT])
def test_a_wait_that_runs_out_is_seen_in_the_outputs_and_in_the_status(T, N, row, left):
    """One CTA keeps its sums of one row to itself: the waits of its cluster end
    after 20 ms, dx of the rows left undone and the sums over the rows are NaN,
    the other rows are as they always are, the status says so, and the next call
    on the same workspace is right."""
    need_gpu()
    (x, _, dy, _), w, b = inputs(T, N, torch.bfloat16, seed=T)
    _, mean, rstd = fa.layer_norm_fwd(x, w, b, EPS)
    want = fa.layer_norm_bwd(dy, x, w, mean, rstd)
    ws = fa.workspace(fa.layer_norm_ws_bytes(T, N))
    same = fa.debug_layer_norm_bwd_timeout(dy, x, w, mean, rstd, -1, 1_000_000_000, ws)
    assert fa.check_device_status(ws) == 0
    assert all(torch.equal(a, c) for a, c in zip(same, want))
    dx, dw, db = fa.debug_layer_norm_bwd_timeout(dy, x, w, mean, rstd, row, 20_000_000, ws)
    assert fa.check_device_status(ws) == 7
    assert fa.check_device_status(ws) == 0  # read clears it
    undone = torch.zeros(T, dtype=torch.bool, device="cuda")
    undone[left] = True
    assert torch.isnan(dx[undone]).all()
    assert torch.equal(dx[~undone], want[0][~undone])
    assert torch.isnan(dw).all() and torch.isnan(db).all()
    again = fa.layer_norm_bwd(dy, x, w, mean, rstd, ws=ws)
    assert fa.check_device_status(ws) == 0
    assert all(torch.equal(a, c) for a, c in zip(again, want))


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("N", [24, 256, 300, 1024, 4096, 4099, 8200, 12288, 40001, 70000])
def test_sums_over_the_rows_take_every_row_once(N, dtype):
    """dy, x and the statistics given to the call are whole numbers, so that
    every term and every sum of dweight and dbias is exact in binary32 in any
    order (below 2^24), at row counts on both sides of each layout's borders."""
    need_gpu()
    counts = [1, 2, 15, 16, 17, 31, 32, 33, 34, 74, 75, 147, 148, 149, 295, 297, 1185, 3553]
    g = torch.Generator(device="cuda").manual_seed(N)
    w = torch.ones(N, dtype=dtype, device="cuda")
    for T in [t for t in counts if t * N <= 16_000_000]:
        x, dy, ds = (torch.randint(-8, 9, (T, N), generator=g, device="cuda").to(dtype) for _ in range(3))
        mean = torch.randint(-2, 3, (T,), generator=g, device="cuda").float()
        rstd = torch.randint(1, 3, (T,), generator=g, device="cuda").float()
        xh = (x.double() - mean[:, None]) * rstd[:, None]
        dw, db = (dy.double() * xh).sum(0), dy.double().sum(0)
        got = fa.layer_norm_bwd(dy, x, w, mean, rstd, dres=ds)[1:] + \
            fa.dropout_add_layer_norm_bwd(dy, None, x, w, mean, rstd, 0.1, SEED)[2:]
        for a, b in zip(got, (dw, db, dw, db)):
            assert torch.equal(a.double(), b), T


def kept_in_row(r, N, p, seed):
    words = [O.philox4x32([j, r, 0, R.DROP_TAG], [seed & 0xFFFFFFFF, seed >> 32], 7) for j in range(-(-N // 8))]
    u = np.asarray(words, dtype=np.uint32).reshape(-1).view(np.uint16)[:N]  # little endian: low half first
    return torch.from_numpy(u.astype(np.int64) >= round(p * 65536)).cuda()


@pytest.mark.parametrize("dtype,N", [(torch.bfloat16, 32768), (torch.bfloat16, 32765), (torch.float32, 32768),
                                     (torch.float32, 32765)], ids=["bf16", "bf16-odd", "fp32", "fp32-odd"])
def test_masks_of_rows_past_2_to_the_31_elements(dtype, N):
    """Whole rows on both sides of that border, the last one too, against the
    oracle's generator: dropout alone, and the sum that the fused call stores."""
    need_gpu()
    T, p = 70000, 0.25
    one = torch.ones(1, 1, dtype=dtype, device="cuda").expand(T, N)
    x = one.contiguous()
    y = fa.dropout_fwd(x, p, SEED)
    rows = [0, 1, 2 ** 31 // N, 2 ** 31 // N + 1, T - 1]
    masks = [kept_in_row(r, N, p, SEED) for r in rows]
    scale = torch.tensor(1 / 0.75).to(dtype).item()
    for r, m in zip(rows, masks):
        assert torch.equal(y[r], torch.where(m, scale, 0.0).to(dtype)), r
    if dtype == torch.bfloat16:
        w = torch.ones(N, dtype=dtype, device="cuda")
        _, s, _, _ = fa.dropout_add_layer_norm_fwd(x, x, w, None, p, SEED, out=y)
        kept = torch.tensor(1 + 1 / 0.75).to(dtype).item()
        for r, m in zip(rows, masks):
            assert torch.equal(s[r], torch.where(m, kept, 1.0).to(dtype)), r
