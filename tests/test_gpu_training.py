"""The training loss with its gradient, gradient clipping, and a whole teacher-forced step, on B200, each against a
plain 64-bit form and the error bounds of oracle.around."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import around
from rank_markov_draft_vanillamarkov_b200 import (DSparkError, GradientClipper, TokenConstraints, VanillaMarkov,
                                                  block_cross_entropy, clip_grad_norm, device_status, set_algo,
                                                  set_debug)
from rank_markov_draft_vanillamarkov_b200 import _native as N
from rank_markov_draft_vanillamarkov_b200.build import build

from _helpers import dtype_name, f64

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    N.load()
    device_status()
    yield
    set_algo(N.DSPARK_ALGO_AUTO)


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _within(got, want, err):
    got, want, err = (np.asarray(a, dtype=np.float64) for a in (got, want, err))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fin = np.isfinite(want)
    bad = ~(np.abs(got[fin] - want[fin]) <= err[fin])
    assert not bad.any(), (bad.sum(), np.flatnonzero(fin)[bad][:5], got[fin][bad][:5], want[fin][bad][:5],
                           err[fin][bad][:5])


# ------------------------------------------------------------------- loss --

def _rows(rows, vocab, dtype, seed, pad=0.3, weights=True, std=3.0):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.normal(0, std, (rows, vocab))).to(dtype)
    t = g.integers(0, vocab, rows)
    x[np.arange(rows), t] += torch.from_numpy(g.uniform(0, 8, rows)).to(dtype)
    t = np.where(g.random(rows) < pad, -100, t)
    w = None
    if weights:
        w = g.uniform(0.1, 2.0, rows).astype(np.float32)
        w[g.random(rows) < 0.1] = 0.0
    return x, torch.from_numpy(t), None if w is None else torch.from_numpy(w)


def _check_loss(got, x, t, w, mean=True, ignore=-100):
    loss, rows, grad = got
    exact = around.cross_entropy(f64(x).reshape(-1, x.shape[-1]), t.reshape(-1).numpy(),
                                 None if w is None else w.reshape(-1).numpy(), ignore, mean, dtype_name(x.dtype))
    assert loss.shape == () and loss.dtype == torch.float32 and rows.shape == t.shape
    _within(f64(loss), *exact[0])
    _within(f64(rows).reshape(-1), *exact[1])
    if grad is not None:
        assert grad.shape == x.shape and grad.dtype == x.dtype
        _within(f64(grad).reshape(-1, x.shape[-1]), *exact[2])


LOSS_SHAPES = [(1, 1), (3, 2), (10, 1024), (5, 7), (2, 4095), (4, 4096), (3, 4097), (7, 32003), (1, 40001), (2, 65536),
               (3, 70001), (3, 129280), (2, 151936), (1, 262147), (1, 600001), (2, 1300001), (150, 100003), (700, 33), (2100, 5)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", LOSS_SHAPES)
def test_loss_against_the_plain_form(rows, vocab, dtype):
    x, t, w = _rows(rows, vocab, dtype, seed=rows * 7 + vocab)
    if rows == 1:
        t[:] = vocab // 2
        w[:] = 0.7
    xd, td, wd = x.cuda(), t.cuda(), w.cuda()
    got = block_cross_entropy(xd, td, weights=wd)
    torch.cuda.synchronize()
    assert torch.equal(_bits(xd.cpu()), _bits(x))
    _check_loss(got, x, t, w)
    # Without the gradient, and in place: the same bits.
    loss, row, none = block_cross_entropy(xd, td, weights=wd, want_grad=False)
    assert none is None and torch.equal(loss, got[0]) and torch.equal(row, got[1])
    loss, row, grad = block_cross_entropy(xd, td, weights=wd, out_grad=xd)
    assert grad is xd and torch.equal(_bits(grad), _bits(got[2])) and torch.equal(loss, got[0])
    assert device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_loss_reductions_shapes_and_defaults(reduction, dtype):
    x, t, _ = _rows(60, 771, dtype, seed=4, weights=False)
    x, t = x.view(3, 4, 5, 771), t.view(3, 4, 5)
    got = block_cross_entropy(x.cuda(), t.cuda(), reduction=reduction)
    _check_loss(got, x, t, None, mean=reduction == "mean")
    got = block_cross_entropy(x.cuda(), t.int().cuda(), reduction=reduction, ignore_index=-100)
    _check_loss(got, x, t, None, mean=reduction == "mean")
    one = block_cross_entropy(x[0, 0, 0].cuda(), torch.tensor(7).cuda(), reduction=reduction)
    _check_loss(one, x[0, 0, 0], torch.tensor(7), None, mean=reduction == "mean")
    # Another ignored id, one of the vocabulary.
    t = t.clamp(min=0)
    t[0] = 5
    _check_loss(block_cross_entropy(x.cuda(), t.cuda(), ignore_index=5, reduction=reduction), x, t, None,
                mean=reduction == "mean", ignore=5)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("offset", [1, 3, 5])
def test_loss_alignments(offset, dtype):
    """Logits and gradient that start at different odd elements; what surrounds the gradient stays."""
    for vocab in (1000, 1003):
        x, t, w = _rows(6, vocab, dtype, seed=offset)
        hold = torch.zeros(6 * vocab + 16, dtype=dtype, device="cuda")
        out = torch.full((6 * vocab + 16,), 9.0, dtype=dtype, device="cuda")
        xd = hold[offset: offset + 6 * vocab].view(6, vocab)
        xd.copy_(x)
        for shift in (offset, offset + 2):
            out.fill_(9.0)
            g = out[shift: shift + 6 * vocab].view(6, vocab)
            _check_loss(block_cross_entropy(xd, t.cuda(), weights=w.cuda(), out_grad=g), x, t, w)
            assert (out[:shift] == 9).all() and (out[shift + 6 * vocab:] == 9).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_loss_extremes(dtype):
    """Infinities, NaN and the lowest value in live and in ignored rows; spans of exponents."""
    for vocab in (300, 20001):
        x, t, w = _rows(12, vocab, dtype, seed=vocab, pad=0.0)
        w[:] = 1.0
        inf, low = float("inf"), torch.finfo(dtype).min
        x[0, 3] = float("nan")
        x[1, 5] = inf
        x[2, :] = -inf
        x[3, :] = -inf
        x[3, t[3]] = 2.0
        x[4, t[4]] = -inf
        x[5, 1::2] = -inf
        x[6, :] = low
        x[7, 0::3] = low
        x[8, :] = float("nan")
        t[8] = -100
        x[9, :] = inf
        w[9] = 0.0
        x[10] *= 30
        x[11, :] = 0.0
        keep = [i for i in range(12) if i not in (0, 1, 2, 4)]
        got = block_cross_entropy(x.cuda(), t.cuda(), weights=w.cuda(), reduction="sum")
        _check_loss(got, x, t, w, mean=False)
        got = block_cross_entropy(x[keep].cuda(), t[keep].cuda(), weights=w[keep].cuda())
        _check_loss(got, x[keep], t[keep], w[keep])


def test_loss_without_live_rows():
    x = torch.full((4, 100), float("nan"), device="cuda")
    t = torch.full((4,), -100, device="cuda")
    for reduction in ("mean", "sum"):
        loss, rows, grad = block_cross_entropy(x, t, reduction=reduction)
        assert loss.item() == 0 and not rows.any() and not grad.any()
    loss, rows, grad = block_cross_entropy(x, torch.zeros_like(t), weights=torch.zeros(4, device="cuda"))
    assert loss.item() == 0 and not rows.any() and not grad.any()
    loss, rows, grad = block_cross_entropy(x[:0], t[:0])
    assert loss.item() == 0 and rows.shape == (0,) and grad.shape == (0, 100)


def test_loss_reports_targets_outside_the_vocabulary():
    x, t, w = _rows(6, 500, torch.float32, seed=1, pad=0.0)
    for bad in (500, -1, 1 << 40):
        t[2] = bad
        got = block_cross_entropy(x.cuda(), t.cuda(), weights=w.cuda())
        assert device_status() == N.DSPARK_STATUS_TOKEN_RANGE
        _check_loss(got, x, t, w)


def test_loss_gradient_against_differences():
    """Central differences of the 64-bit loss, whose own error is h^2 / 6 times a third derivative below 1 plus the
    cancellation of two losses near 5 (2^-52 * 5 / h)."""
    x, t, w = _rows(5, 40, torch.float32, seed=9, pad=0.2)
    _, _, grad = block_cross_entropy(x.cuda(), t.cuda(), weights=w.cuda())
    h = 1e-4
    base = f64(x)
    for i in range(5):
        for v in range(40):
            pair = []
            for s in (h, -h):
                y = base.copy()
                y[i, v] += s
                pair.append(around.cross_entropy(y, t.numpy(), w.numpy(), -100, True, "fp32")[0][0])
            assert abs((pair[0] - pair[1]) / (2 * h) - grad[i, v].item()) <= h * h + 5 * 2.0 ** -52 / h + 1e-6


def test_loss_repeats_streams_and_graphs():
    x, t, w = _rows(90, 33001, torch.bfloat16, seed=2)
    xd, td, wd = x.cuda(), t.cuda(), w.cuda()
    want = block_cross_entropy(xd, td, weights=wd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            got.append(block_cross_entropy(xd, td, weights=wd))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block_cross_entropy(xd, td, weights=wd))
        graphs.append(g)
    x2, t2, w2 = _rows(90, 33001, torch.bfloat16, seed=3)
    xd.copy_(x2), td.copy_(t2), wd.copy_(w2)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for r in outs:
        _check_loss(r, x2, t2, w2)


def test_loss_long_offsets():
    """Rows past 2^31 elements."""
    vocab = 129280
    rows = (1 << 31) // vocab + 3
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    t = torch.full((rows,), -100, device="cuda")
    pick, tp, _ = _rows(3, vocab, torch.bfloat16, seed=6, pad=0.0)
    at = torch.tensor([0, rows - 2, rows - 1])
    x[at] = pick.cuda()
    t[at] = tp.cuda()
    loss, row, grad = block_cross_entropy(x, t, out_grad=x)
    _check_loss((loss, row[at], grad[at.cuda()]), pick, tp, None)
    assert not grad[1: rows - 2].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", [(40, 1024), (64, 20001), (4, 600001)])
def test_losses_of_certain_rows_are_not_negative(rows, vocab, dtype):
    """Rows whose target stands alone at the top, at references that round either way: a loss is never below zero."""
    g = np.random.default_rng(rows)
    for top in (1.0, 7.0, 25.0, 300.0, 3e4):
        x = torch.from_numpy(g.normal(0, 0.1, (rows, vocab)) - 40.0).to(dtype)
        t = torch.from_numpy(g.integers(0, vocab, rows))
        x[torch.arange(rows), t] = torch.from_numpy(top * g.uniform(0.5, 1.0, rows)).to(dtype)
        got = block_cross_entropy(x.cuda(), t.cuda())
        assert not (got[1] < 0).any() and not got[0] < 0 and not torch.signbit(got[1]).any()
        _check_loss(got, x, t, None)



@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", [(10, 1024), (300, 8000), (700, 33), (90, 33001), (2000, 151936), (64, 300000)])
def test_loss_waits_that_expire(rows, vocab, dtype):
    """With a limit that any wait may pass, a row either has its loss and gradient or a NaN loss that the status word
    reports, and the call after it is right. Nothing is withheld: every wait would be met a little later."""
    g = torch.Generator("cuda").manual_seed(rows)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    t[::7] = -100
    want = block_cross_entropy(x, t)
    assert device_status() == 0
    set_debug(0, 1)
    try:
        for place in ("out", "in place") * 3:
            logits = x.clone()
            loss, row, grad = block_cross_entropy(logits, t, out_grad=logits if place == "in place" else None)
            status = device_status()
            lost = row.isnan()
            assert status == (N.DSPARK_STATUS_TIMEOUT if lost.any() else 0)
            assert bool(loss.isnan()) == bool(lost.any()) and not lost[t == -100].any()
            assert torch.equal(row[~lost], want[1][~lost])
            kept = ~lost & (t != -100)
            assert torch.equal(_bits(grad[kept]), _bits(want[2][kept]))
    finally:
        set_debug(0, 0)
    again = block_cross_entropy(x, t)
    assert all(torch.equal(a, b) for a, b in zip(again, want)) and device_status() == 0


def test_loss_refusals():
    x, t = torch.zeros(4, 10, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for f in (lambda: block_cross_entropy(x.double(), t), lambda: block_cross_entropy(x, t[:3]),
              lambda: block_cross_entropy(x, t, reduction="none"), lambda: block_cross_entropy(x.cpu(), t),
              lambda: block_cross_entropy(x.t().contiguous().t(), t), lambda: block_cross_entropy(x, t.cpu()),
              lambda: block_cross_entropy(x, t, weights=torch.zeros(4, device="cuda").double()),
              lambda: block_cross_entropy(x, t, weights=torch.zeros(5, device="cuda")),
              lambda: block_cross_entropy(x, t, out_grad=x.bfloat16()), lambda: block_cross_entropy(x[:, :0], t)):
        with pytest.raises(ValueError):
            f()
    flat = torch.zeros(60, device="cuda")
    with pytest.raises(DSparkError):
        block_cross_entropy(flat[:40].view(4, 10), t, out_grad=flat[10:50].view(4, 10))


# --------------------------------------------------------------- clipping --

def _grads(sizes, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(d) for n, d in sizes]


def _check_clip(norm, outs, grads, max_norm):
    want, factor = around.clip([f64(g) for g in grads], max_norm)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(norm.item() - want) <= around.CLIP_NORM_REL * want
    for o, g in zip(outs, grads):
        exact = f64(g) * factor
        rel = around.CLIP_NORM_REL + 3 * around.U32 + around.HALF_STEP[dtype_name(g.dtype)]
        assert o.dtype == g.dtype and o.shape == g.shape
        _within(f64(o), exact, rel * np.abs(exact) + 2.0 ** -133)


F, B = torch.float32, torch.bfloat16
CLIP_SETS = [
    [(1, F)], [(1, B)], [(0, F), (3, B), (0, B)], [(16384, F)], [(16385, F), (32769, B)], [(5, F)] * 40,
    [(1000003, B), (777, F), (40000, F)], [(i, B if i % 2 else F) for i in range(1, 90)], [(3000000, F), (3000001, B)],
]


@pytest.mark.parametrize("sizes", CLIP_SETS, ids=range(len(CLIP_SETS)))
@pytest.mark.parametrize("share", [0.37, 4.0])
def test_clip_against_the_plain_form(sizes, share):
    grads = _grads(sizes, seed=len(sizes))
    max_norm = share * around.clip([f64(g) for g in grads], 1.0)[0]
    dev = [g.cuda() for g in grads]
    outs = [torch.full_like(g, 5.0) for g in dev]
    clipper = GradientClipper(dev, out=outs)
    _check_clip(clipper.clip(max_norm), outs, grads, max_norm)
    assert all(torch.equal(_bits(d.cpu()), _bits(g)) for d, g in zip(dev, grads))
    norm = clip_grad_norm(dev, max_norm)
    _check_clip(norm, dev, grads, max_norm)
    assert all(torch.equal(_bits(d), _bits(o)) for d, o in zip(dev, outs))
    assert device_status() == 0


def test_clip_packed_tensors_of_any_alignment():
    """Views of flat buffers, gradients and outputs at different offsets, guard cells between them left alone."""
    sizes = [(1, B), (2, B), (100, B), (5, B), (9001, B), (33, B), (70001, B)]
    grads = _grads(sizes, seed=3)
    for shift in (0, 1, 2, 3, 7):
        flat = torch.full((90000,), 3.0, dtype=B, device="cuda")
        out = torch.full((90000,), 3.0, dtype=B, device="cuda")
        views, outs, cells, at = [], [], [], 0
        for g in grads:
            views.append(flat[at: at + g.numel()])
            outs.append(out[at + shift: at + shift + g.numel()])
            views[-1].copy_(g)
            at += g.numel() + 1 + shift % 3
            cells.append(at)
        keep = flat.clone()
        norm = GradientClipper(views, out=outs).clip(1.5)
        _check_clip(norm, outs, grads, 1.5)
        assert torch.equal(_bits(flat), _bits(keep))
        mask = torch.ones_like(out, dtype=torch.bool)
        for o in outs:
            a = (o.data_ptr() - out.data_ptr()) // 2
            mask[a: a + o.numel()] = False
        assert (out[mask] == 3).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-19, 1e18, 1e21, 1e30])
def test_clip_values_whose_squares_leave_the_range(scale, dtype):
    grads = _grads([(5000, dtype), (333, F)], seed=2, std=scale)
    dev = [g.cuda() for g in grads]
    want = around.clip([f64(g) for g in grads], 1.0)[0]
    outs = [torch.empty_like(g) for g in dev]
    norm = GradientClipper(dev, out=outs).clip(want / 3)
    assert abs(norm.item() - want) <= around.CLIP_NORM_REL * want
    _check_clip(norm, outs, grads, want / 3)


def test_clip_mixed_magnitudes_and_zeros():
    g = torch.zeros(50000)
    g[7], g[12345], g[49999] = 1e25, 1e-30, -3e24
    dev = g.cuda()
    out = torch.empty_like(dev)
    _check_clip(GradientClipper([dev], out=[out]).clip(2.0), [out], [g], 2.0)
    zero = torch.zeros(1000, device="cuda")
    assert clip_grad_norm([zero], 1.0).item() == 0 and not zero.any()
    assert clip_grad_norm([], 1.0).item() == 0
    assert clip_grad_norm([zero[:0]], 1.0).item() == 0


def test_clip_limits_and_non_finite_norms():
    g = torch.randn(3000, generator=torch.Generator().manual_seed(1))
    dev = g.cuda()
    norm = clip_grad_norm([dev], math.inf)
    assert torch.equal(dev.cpu(), g) and abs(norm.item() - g.double().norm().item()) <= 1e-6 * norm.item()
    assert clip_grad_norm([dev], 0.0).item() > 0 and not dev.any()
    for bad in (math.inf, math.nan):  # measured only, and copied, whatever the norm
        for n in (3000, 700000):
            dev = torch.ones(n, device="cuda")
            dev[n // 2] = bad
            out = torch.empty_like(dev)
            norm = GradientClipper([dev], out=[out]).clip(math.inf)
            assert not math.isfinite(norm.item())
            # x * 1 is x; of a NaN the payload is free (a product's is CUDA's own NaN).
            assert torch.allclose(out, dev, rtol=0.0, atol=0.0, equal_nan=True)
    for bad, after in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        dev = g.cuda()
        dev[2999] = bad
        out = torch.empty_like(dev)
        norm = GradientClipper([dev], out=[out]).clip(1.0)
        assert (math.isinf(norm.item()) and norm.item() > 0) if bad == math.inf else math.isnan(norm.item())
        rest = out[:2999]
        assert bool((rest == 0).all()) if after == 0.0 else bool(rest.isnan().all())
        assert math.isnan(out[2999].item())


@pytest.mark.parametrize("n", [3000, 700000])
def test_clip_limits_outside_fp32(n):
    """A limit is a 64-bit number: a finite one above fp32's range still clips."""
    g = torch.full((n,), 3e38)
    g[::3] *= -0.5
    for max_norm in (1e39, 5e40, 1e300):
        dev = g.cuda()
        out = torch.empty_like(dev)
        norm = GradientClipper([dev], out=[out]).clip(max_norm)
        assert norm.item() == math.inf  # as fp32
        exact = f64(g) * around.clip([f64(g)], max_norm)[1]
        _within(f64(out), exact, (around.CLIP_NORM_REL + 4 * around.U32) * np.abs(exact))
    dev = g.cuda()
    dev[1] = math.inf
    assert clip_grad_norm([dev], 1e39).item() == math.inf
    assert bool((dev[2:] == 0).all()) and math.isnan(dev[1].item())  # an infinite norm scales by zero


def test_clip_repeats_streams_and_graphs():
    grads = _grads([(300001, F), (70000, B), (11, F)], seed=8)
    dev = [g.cuda() for g in grads]
    outs = [[torch.empty_like(g) for g in dev] for _ in range(2)]
    clippers = [GradientClipper(dev, out=o) for o in outs]
    want = clippers[0].clip(2.0)
    keep = [o.clone() for o in outs[0]]
    graphs, norms = [], []
    torch.cuda.synchronize()
    for c in clippers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(c.clip(2.0))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, n in zip(outs, norms):
        assert torch.equal(n, want) and all(torch.equal(_bits(a), _bits(b)) for a, b in zip(o, keep))
    fresh = _grads([(300001, F), (70000, B), (11, F)], seed=9)
    for d, g in zip(dev, fresh):
        d.copy_(g)
    graphs[1].replay()
    torch.cuda.synchronize()
    _check_clip(norms[1], outs[1], fresh, 2.0)


def test_clippers_are_not_made_during_a_capture():
    """Refused before anything that would spoil the capture, which ends well; a clipper made before it is captured."""
    g = torch.randn(5000, device="cuda")
    want = g * 2
    clipper = GradientClipper([g])
    clipper.clip(math.inf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in (lambda: GradientClipper([g]), lambda: clip_grad_norm([g], 1.0), lambda: clip_grad_norm([], 1.0)):
            with pytest.raises(RuntimeError):
                f()
        g.mul_(2)
        norm = clipper.clip(math.inf)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, want) and abs(norm.item() - want.double().norm().item()) <= 1e-6 * norm.item()


def test_clip_refusals():
    g = torch.zeros(100, device="cuda")
    for f in (lambda: GradientClipper([g.double()]), lambda: GradientClipper([g.cpu()]),
              lambda: GradientClipper([g, g]), lambda: GradientClipper([g[:60], g[50:]]),
              lambda: GradientClipper([g[::2]]), lambda: GradientClipper([g], out=[]),
              lambda: GradientClipper([g], out=[g.bfloat16()]), lambda: GradientClipper([g[:50]], out=[g[20:70]]),
              lambda: GradientClipper([g[:50], g[50:]], out=[g[50:], g[:50]]),
              lambda: clip_grad_norm([g], -1.0), lambda: clip_grad_norm([g], float("nan"))):
        with pytest.raises(ValueError):
            f()


# ----------------------------------------------------- a whole step, a run --

@pytest.mark.parametrize("batch,blocks,vocab,rank,ldt,wdt", [
    (2, 3, 2056, 64, torch.bfloat16, torch.bfloat16), (2, 2, 1001, 24, torch.float32, torch.float32)])
def test_teacher_forced_step(batch, blocks, vocab, rank, ldt, wdt):
    """apply -> loss -> backward -> clip in one call: each stage against the oracle on the stage before it."""
    g = torch.Generator().manual_seed(vocab)
    w1, w2 = ((torch.randn(vocab, rank, generator=g) * 0.3).to(wdt) for _ in range(2))
    head = VanillaMarkov(w1.cuda(), w2.cuda())
    base = torch.randn(batch, blocks, 5, vocab, generator=g).to(ldt).cuda()
    prev = torch.randint(0, vocab, (batch, blocks, 5), generator=g).cuda()
    targets = torch.randint(0, vocab, (batch, blocks, 5), generator=g)
    targets[0, 0] = -100
    weights = (0.8 ** torch.arange(5.0)).expand(batch, blocks, 5).contiguous()
    keep = base.clone()
    corrected = head.apply_block_logits(base, token_ids=prev)
    loss, rows, grad = block_cross_entropy(corrected, targets.cuda(), weights=weights.cuda())
    _check_loss((loss, rows, grad), corrected.cpu(), targets, weights)
    e1, e2 = oracle.apply_block_logits_backward(f64(grad), f64(w1), f64(w2), prev.cpu().numpy())
    plain = head.teacher_forced_gradients(base, token_ids=prev, targets=targets.cuda(), weights=weights.cuda())
    assert torch.equal(_bits(base), _bits(keep)) and plain["norm"] is None
    assert torch.equal(plain["loss"], loss) and torch.equal(_bits(plain["grad_logits"]), _bits(grad))
    total = math.sqrt((e1 ** 2).sum() + (e2 ** 2).sum())
    bufs = [torch.empty(vocab, rank, device="cuda") for _ in range(2)]
    for clipper in (None, GradientClipper(bufs)):
        more = {} if clipper is None else dict(grad_w1=bufs[0], grad_w2=bufs[1], clipper=clipper)
        step = head.teacher_forced_gradients(base, token_ids=prev, targets=targets.cuda(), weights=weights.cuda(),
                                             max_norm=total / 4, **more)
        # fp32 sums of at most rows or vocab products, in any order: n u relative to the sum of magnitudes.
        assert abs(step["norm"].item() - total) <= 1e-3 * total
        for name, exact in (("grad_w1", e1), ("grad_w2", e2)):
            got = f64(step[name]) * 4
            assert np.linalg.norm(got - exact) <= 1e-3 * np.linalg.norm(exact), name
    with pytest.raises(ValueError):
        head.teacher_forced_gradients(base, token_ids=prev, targets=targets.cuda(), clipper=GradientClipper(bufs))


def test_teacher_forced_step_returns_what_its_clipper_leaves():
    """The clipped gradients come back wherever the clipper writes them; a clipper of other buffers is refused."""
    vocab, rank = 515, 16
    g = torch.Generator().manual_seed(1)
    head = VanillaMarkov(*((torch.randn(vocab, rank, generator=g) * 0.3).cuda() for _ in range(2)))
    base = torch.randn(2, 3, vocab, generator=g).cuda()
    ids = dict(token_ids=torch.randint(0, vocab, (2, 3), generator=g).cuda(),
               targets=torch.randint(0, vocab, (2, 3), generator=g).cuda())
    raw = head.teacher_forced_gradients(base, **ids)
    n = vocab * rank
    norm = math.sqrt(sum((f64(raw[k]) ** 2).sum() for k in ("grad_w1", "grad_w2")))

    def check(step, extra=0.0):
        total = math.sqrt(norm ** 2 + extra)
        assert abs(step["norm"].item() - total) <= around.CLIP_NORM_REL * total
        for k in ("grad_w1", "grad_w2"):
            exact = f64(raw[k]) * (norm / 8 / (total + 1e-6))
            _within(f64(step[k]), exact, (around.CLIP_NORM_REL + 4 * around.U32) * np.abs(exact) + 2.0 ** -133)

    bufs, outs = ([torch.empty(vocab, rank, device="cuda") for _ in range(2)] for _ in range(2))
    flat, flat_out = (torch.zeros(2 * n + 11, device="cuda") for _ in range(2))
    flat[0] = 3.0
    parts, part_outs = ([f[11 + i * n: 11 + (i + 1) * n].view(vocab, rank) for i in range(2)] for f in (flat, flat_out))
    tail = torch.ones(7, dtype=torch.bfloat16, device="cuda")
    for given, clipper, at, extra in (
            (bufs, GradientClipper(bufs), bufs, 0.0),
            (bufs, GradientClipper(bufs, out=outs), outs, 0.0),
            (bufs, GradientClipper([tail, bufs[1], bufs[0]], out=[torch.empty_like(tail), outs[1], outs[0]]), outs, 7.0),
            (parts, GradientClipper([flat], out=[flat_out]), part_outs, 9.0),
            (parts, GradientClipper([flat]), parts, 9.0)):
        step = head.teacher_forced_gradients(base, grad_w1=given[0], grad_w2=given[1], max_norm=norm / 8,
                                             clipper=clipper, **ids)
        check(step, extra)
        for k, want in zip(("grad_w1", "grad_w2"), at):
            assert step[k].data_ptr() == want.data_ptr() and step[k].shape == want.shape
    keep = [b.clone() for b in bufs]
    for wrong in (GradientClipper(outs), GradientClipper([bufs[0], outs[1]]), GradientClipper([]),
                  GradientClipper([bufs[0], bufs[1][:-1]])):
        with pytest.raises(ValueError):
            head.teacher_forced_gradients(base, grad_w1=bufs[0], grad_w2=bufs[1], max_norm=1.0, clipper=wrong, **ids)
    assert all(torch.equal(a, b) for a, b in zip(keep, bufs))  # refused before any work


def test_training_and_constrained_serving_together():
    """A step's update changes the head; the updated head then drafts under constraints that it obeys."""
    g = torch.Generator().manual_seed(0)
    vocab, rank = 1024, 64
    w = [(torch.randn(vocab, rank, generator=g) * 0.1).bfloat16().cuda() for _ in range(2)]
    head = VanillaMarkov(*w)
    base = torch.randn(4, 2, 5, vocab, generator=g).bfloat16().cuda()
    prev = torch.randint(0, vocab, (4, 2, 5), generator=g).cuda()
    targets = torch.randint(0, vocab, (4, 2, 5), generator=g).cuda()
    before = [t.clone() for t in w]
    step = head.teacher_forced_gradients(base, token_ids=prev, targets=targets, max_norm=1.0)
    for t, name in zip(w, ("grad_w1", "grad_w2")):
        t.sub_(10.0 * step[name].to(t.dtype))
    assert all(not torch.equal(a, b) for a, b in zip(w, before))
    allowed = torch.zeros(4, 5, vocab // 32, dtype=torch.int32, device="cuda")
    allowed[:, :, 3] = -1  # ids 96 to 127
    history = torch.randint(0, vocab, (4, 12), generator=g).cuda()
    c = TokenConstraints(vocab, history=history, repetition_penalty=1.2, presence_penalty=50.0)
    tokens, logits = head.sample_block_tokens(base[:, 0].contiguous(), first_prev_token_ids=prev[:, 0, 0].contiguous(),
                                              constraints=c, allowed=allowed)
    picks = tokens.cpu().numpy()
    assert ((picks >= 96) & (picks < 128)).all()
    assert all(len(set(row)) == 5 for row in picks.tolist())  # the presence penalty forbids a repeat within a block
    assert device_status() == 0
