"""What needs no GPU of the operators around the head: the 64-bit forms against hand-worked values, the clip plan and
the refusals of the C entries (no device call is made before them)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import around
from rank_markov_draft_vanillamarkov_b200 import TokenConstraints, _native as N, block_cross_entropy, clip_grad_norm
from rank_markov_draft_vanillamarkov_b200 import build as B
from rank_markov_draft_vanillamarkov_b200 import constraints as C, training as T
from rank_markov_draft_vanillamarkov_b200.head import VanillaMarkov


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def test_constrain_row_by_hand():
    row = [2.0, -2.0, 3.0, 0.5, 1.0]
    x, err = around.constrain_row(row, [0, 1], [2, 2, 0], 2.0, 0.25, 0.5, [(3, 1.0), (-1, 9.0), (3, -0.25)],
                                  np.array([True, True, True, True, False]))
    # 0: 2/2 - 0.25 - 0.5; 1: -2*2; 2: 3/2 - 0.5 - 0.5; 3: 0.5 - 0.25; 4: masked
    assert x.tolist() == [0.25, -4.0, 0.5, 0.25, -math.inf]
    assert err[4] == 0 and err[0] > 0
    assert around.choose(x) == 2 and around.choose([1.0, float("nan"), 2.0]) == 1 and around.choose([3.0, 3.0]) == 0
    assert around.choose([-math.inf] * 3) == 0


def test_allowed_words():
    words = np.array([[5, 1]], dtype=np.int32)
    assert np.flatnonzero(around.allowed_from_words(words, 40)[0]).tolist() == [0, 2, 32]
    assert around.allowed_from_words(np.array([-(1 << 31)], dtype=np.int32), 32)[31]


def test_cross_entropy_by_hand_and_differences():
    x = np.log(np.array([[1.0, 3.0], [2.0, 2.0], [1.0, 1.0]]))
    (loss, _), (rows, _), (grad, _) = around.cross_entropy(x, [1, 0, -100], [2.0, 1.0, 5.0], -100, True, "fp32")
    assert rows == pytest.approx([math.log(4 / 3), math.log(2), 0.0])
    assert loss == pytest.approx((2 * math.log(4 / 3) + math.log(2)) / 3)
    assert grad == pytest.approx(np.array([[0.5 / 3, -0.5 / 3], [-0.5 / 3, 0.5 / 3], [0, 0]]))
    g = np.random.default_rng(0)
    x, t, h = g.normal(0, 2, (4, 9)), [3, 0, 8, 2], 1e-5
    grad = around.cross_entropy(x, t, None, -100, False, "fp32")[2][0]
    for i in range(4):
        for v in range(9):
            d = np.zeros_like(x)
            d[i, v] = h
            up, dn = (around.cross_entropy(x + s * d, t, None, -100, False, "fp32")[0][0] for s in (1, -1))
            assert abs((up - dn) / (2 * h) - grad[i, v]) <= 1e-8


def test_clip_norm_bound_tells_groups_of_four_from_longer_sums():
    """The bound holds for norms whose squares are summed by four in 32 bits, and not for 32 in a row."""
    g = np.random.default_rng(0)
    a, b, c, d = (g.uniform(1, 2, 20000).astype(np.float32) for _ in range(4))
    fma = lambda x, z: (x.astype(np.float64) ** 2 + z).astype(np.float32)  # noqa: E731  x x is exact in 64 bits
    four = (fma(a, b * b) + fma(c, d * d)).astype(np.float64)
    exact = sum(x.astype(np.float64) ** 2 for x in (a, b, c, d))
    norm = np.sqrt(four).astype(np.float32).astype(np.float64)
    assert np.abs(norm / np.sqrt(exact) - 1).max() <= around.CLIP_NORM_REL
    long = np.zeros_like(a)
    for _ in range(32):
        long = long + a * a
    norm = np.sqrt(long.astype(np.float64))
    assert np.abs(norm / np.sqrt(32 * a.astype(np.float64) ** 2) - 1).max() > around.CLIP_NORM_REL


def _plan(lib, spans, capacity=None):
    n = len(spans)
    pieces = ctypes.c_int64(-1)
    args = ((ctypes.c_void_p * n)(*[s[0] for s in spans]), (ctypes.c_void_p * n)(*[s[1] for s in spans]),
            (ctypes.c_int64 * n)(*[s[2] for s in spans]), (ctypes.c_int32 * n)(*[s[3] for s in spans]), n)
    code = lib.dspark_markov_clip_plan(*args, None, 0, ctypes.byref(pieces))
    if code != N.DSPARK_OK:
        return code, None
    plan = (N.ClipPiece * max(1, pieces.value))()
    code = lib.dspark_markov_clip_plan(*args, plan, pieces.value if capacity is None else capacity,
                                       ctypes.byref(pieces))
    return code, [(p.grad, p.out, p.count, p.dtype) for p in plan[: pieces.value]]


def test_clip_plan_covers_every_element_once(lib):
    spans = [(1 << 20, 1 << 20, 40001, 1), (1 << 24, 1 << 26, 16384, 0), (0, 0, 0, 0), (1 << 28, 1 << 28, 1, 1),
             ((1 << 30) + 4, (1 << 32) + 8, 16385, 0)]
    code, pieces = _plan(lib, spans)
    assert code == N.DSPARK_OK
    for grad, out, count, dtype in spans:
        if not count:
            continue
        size = 2 if dtype else 4
        mine = [p for p in pieces if grad <= p[0] < grad + count * size]
        assert sum(p[2] for p in mine) == count and all(p[3] == dtype and p[2] > 0 for p in mine)
        at = 0
        for p in mine:
            assert p[0] == grad + at * size and p[1] == out + at * size
            at += p[2]
    assert _plan(lib, [])[1] == []


def test_clip_plan_refusals(lib):
    ok = (1 << 20, 1 << 20, 100, 0)
    assert _plan(lib, [ok, ((1 << 20) + 396, 1 << 30, 10, 0)])[0] == N.DSPARK_ERR_INVALID_ARG  # overlap
    assert _plan(lib, [ok, ok])[0] == N.DSPARK_ERR_INVALID_ARG  # the same tensor twice
    assert _plan(lib, [ok, ((1 << 20) + 400, 1 << 30, 10, 0)])[0] == N.DSPARK_OK  # neighbours
    assert _plan(lib, [(1 << 20, (1 << 20) + 4, 100, 0)])[0] == N.DSPARK_ERR_INVALID_ARG
    assert _plan(lib, [(1 << 20, 1 << 20, -1, 0)])[0] == N.DSPARK_ERR_INVALID_ARG
    assert _plan(lib, [(1 << 20, 1 << 20, 1, 3)])[0] == N.DSPARK_ERR_INVALID_ARG
    assert _plan(lib, [(0, 0, 1, 0)])[0] == N.DSPARK_ERR_INVALID_ARG
    assert _plan(lib, [((1 << 20) + 2, (1 << 20) + 2, 1, 0)])[0] == N.DSPARK_ERR_INVALID_ARG  # misaligned
    assert _plan(lib, [ok], capacity=0)[0] == N.DSPARK_ERR_INVALID_ARG


def test_c_entry_refusals(lib):
    p, bad, ok = ctypes.c_void_p(1 << 20), N.DSPARK_ERR_INVALID_ARG, N.DSPARK_OK  # never dereferenced
    far = ctypes.c_void_p(1 << 40)
    c = N.Constraints()
    c.repetition_value = 1.0
    ref = ctypes.byref(c)
    pr = lib.dspark_markov_process_logits

    def process(x=p, out=far, b=2, m=3, v=64, ib=192, ir=64, ob=192, orow=64, con=ref, draft=None, ds=3, first=0,
                al=None, tok=None, ts=3, temp=0.0, scratch=None, dt=0):
        return pr(x, out, b, m, v, ib, ir, ob, orow, con, draft, ds, first, al, 0, 0, tok, ts, temp, 0, scratch, dt,
                  None)

    assert process(b=0) == ok and process(m=0) == ok
    assert process(b=-1) == bad and process(v=0) == bad and process(dt=2) == bad and process(con=None) == bad
    assert process(x=None) == bad and process(out=None) == bad
    assert process(temp=float("nan")) == bad and process(ib=-1) == bad and process(first=-1) == bad
    assert process(ob=100) == bad and process(orow=63) == bad and process(ob=0) == bad  # rows that overlap
    assert process(out=p, orow=64, ob=200) == bad  # in place with other strides
    assert process(out=ctypes.c_void_p((1 << 20) + 256)) == bad  # another overlap
    assert process(x=ctypes.c_void_p((1 << 20) + 2)) == bad and process(scratch=ctypes.c_void_p(8)) == bad
    assert process(tok=p, scratch=far, ts=2) == bad and process(draft=p, ds=1) == bad
    assert process(v=1 << 33, ib=0, ir=0, ob=1 << 40, orow=1 << 35) == N.DSPARK_ERR_UNSUPPORTED
    assert process(b=1 << 20, m=1 << 20) == N.DSPARK_ERR_UNSUPPORTED
    for field, value in (("history_cap", -1), ("bias_count", 2), ("bias_stride", -1), ("history_stride", -1)):
        d = N.Constraints()
        setattr(d, field, value)
        assert process(con=ctypes.byref(d)) == bad, field
    size = lib.dspark_markov_constrain_scratch_bytes
    assert size(2, 3, 64, 0, 0, 0, 1) >= 48 and size(2, 3, 64, 0, 0, 0, 0) == 0
    assert size(2, 3, 64, 100, 0, 0, 0) >= 2 * 64 * 8 and size(2, 3, 64, 100, 5, 2, 1) > size(2, 3, 64, 100, 0, 2, 1)
    for refused in ((0, 3, 64, 0, 0, 0, 1), (2, 3, 0, 0, 0, 0, 1), (1 << 20, 1 << 20, 64, 0, 0, 0, 1),
                    (2, 3, 1 << 31, 0, 0, 0, 1), (2, 3, 64, 1 << 30, 0, 0, 1), (2, 3, 64, -1, 0, 0, 1)):
        assert size(*refused) == 0
    sm = lib.dspark_markov_sample_block_constrained

    def sample(base=p, out=far, b=2, m=3, rank=16, temp=0.0, con=ref, scratch=far, ldt=0):
        return sm(base, p, b, m, 64, p, p, rank, temp, 0, con, None, 0, 0, p, out, scratch, ldt, 0, None)

    assert sample(b=0) == ok and sample(m=0) == ok
    assert sample(rank=0) == bad and sample(con=None) == bad and sample(scratch=None) == bad and sample(ldt=5) == bad
    assert sample(temp=float("nan")) == bad and sample(out=p) == bad and sample(b=-1) == bad
    ce = lib.dspark_markov_block_cross_entropy

    def entropy(x=p, t=p, rows=4, v=10, loss=p, row=p, grad=far, dt=0):
        return ce(x, t, None, rows, v, -100, 1, loss, row, grad, dt, None)

    assert entropy(x=None) == bad and entropy(t=None) == bad and entropy(loss=None) == bad and entropy(v=0) == bad
    assert entropy(rows=-1) == bad and entropy(dt=7) == bad and entropy(row=None) == bad
    assert entropy(grad=ctypes.c_void_p((1 << 20) + 16)) == bad and entropy(grad=ctypes.c_void_p((1 << 40) + 2)) == bad
    assert entropy(rows=1 << 40) == N.DSPARK_ERR_UNSUPPORTED
    # Addresses between elements.
    odd = ctypes.c_void_p((1 << 20) + 2)
    assert process(al=odd) == bad and process(draft=odd, tok=None) == bad and process(tok=odd, scratch=far) == bad
    assert entropy(t=odd) == bad and entropy(loss=odd) == bad and entropy(row=odd) == bad
    for field in ("history", "history_lens", "prompt_lens", "repetition", "frequency", "presence", "bias_ids",
                  "bias_values"):
        d = N.Constraints()
        setattr(d, field, (1 << 20) + 2)
        assert process(con=ctypes.byref(d)) == bad, field
    cl = lib.dspark_markov_clip_grad_norm
    assert cl(ctypes.c_void_p(1028), 1, 1.0, p, p, None) == bad and cl(p, 1, 1.0, odd, p, None) == bad
    assert cl(None, 1, 1.0, p, p, None) == bad and cl(p, -1, 1.0, p, p, None) == bad
    assert cl(p, 1, -1.0, p, p, None) == bad and cl(p, 1, float("nan"), p, p, None) == bad
    assert cl(p, 1, 1.0, None, p, None) == bad and cl(p, 1, 1.0, p, None, None) == bad


@pytest.mark.parametrize("source", ["constraints.cu", "loss.cu", "clip.cu"])
def test_no_read_only_loads_of_what_a_kernel_may_write(source):
    """These kernels run in place; a read-only load asks for memory that the whole launch leaves alone."""
    text = open(f"{B.CSRC}/{source}").read()
    assert not any(form in text for form in ("__ldg", "ld.global.nc", "__restrict__"))


def test_constrained_sampler_refuses_sizes_before_it_asks_for_scratch(lib):
    """Such sizes may have no scratch size, so that a caller has none to give."""
    p, c = ctypes.c_void_p(1 << 20), N.Constraints()  # never dereferenced
    for batch, m, vocab, cap in ((1 << 20, 1 << 20, 64, 0), (2, 3, 1 << 31, 0), (1, 1, 64, 1 << 30)):
        c.history_cap = cap
        assert lib.dspark_markov_sample_block_constrained(
            p, p, batch, m, vocab, p, p, 16, 0.0, 0, ctypes.byref(c), None, 0, 0, p, ctypes.c_void_p(1 << 60), None, 0,
            0, None) == N.DSPARK_ERR_UNSUPPORTED


def test_structs_match_the_header():
    # The library asserts the same sizes when it is compiled: eight 8-byte fields, three floats and their padding,
    # four 8-byte fields; two pointers and two 4-byte fields.
    assert ctypes.sizeof(N.Constraints) == 112 and ctypes.sizeof(N.ClipPiece) == 24
    text = open(B.ROOT + "/include/dspark_markov.h").read()
    for name in ("DSPARK_CLIP_MAX_PARTIALS", "DSPARK_CLIP_SCRATCH_BYTES"):
        assert f"#define {name} {getattr(N, name)}\n" in text


def test_python_refusals_without_a_gpu():
    with pytest.raises(ValueError):
        TokenConstraints(0)
    with pytest.raises(ValueError):
        TokenConstraints(10, repetition_penalty=0.0)
    with pytest.raises(ValueError):
        TokenConstraints(10, frequency_penalty=math.inf)
    with pytest.raises(ValueError):
        TokenConstraints(10, history_lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        TokenConstraints(10, history=torch.zeros(2, 3, dtype=torch.int64))  # not on a GPU
    with pytest.raises(ValueError):
        block_cross_entropy(torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        clip_grad_norm([torch.zeros(3)], 1.0)


@pytest.mark.parametrize("penalty", [dict(frequency_penalty=1e39), dict(presence_penalty=-1e39),
                                     dict(repetition_penalty=1e39), dict(repetition_penalty=1e-46)])
def test_penalties_that_fp32_does_not_hold_are_refused(penalty):
    """Finite numbers that would reach the kernel as an infinity or, for the repetition penalty, as zero."""
    with pytest.raises(ValueError):
        TokenConstraints(10, **penalty)
    TokenConstraints(10, frequency_penalty=3e38, presence_penalty=1e-46, repetition_penalty=1e-40)


@pytest.mark.parametrize("fn,name", [(C.process_logits, "process_logits"), (T.block_cross_entropy, "block_cross_entropy"),
                                     (T.GradientClipper.clip, "clip"),
                                     (VanillaMarkov.teacher_forced_gradients, "teacher_forced_gradients")])
def test_entry_points_are_ranged(fn, name):
    assert fn.__wrapped__.__name__ == name


def test_the_heads_calls_are_made_on_its_device(monkeypatch):
    """The library launches on the current device, which may be another one: every call into it, those of a
    teacher-forced step among them, stands inside the guard that makes the head's device the current one."""
    from rank_markov_draft_vanillamarkov_b200 import head as H
    inside, calls = [], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            inside.append(self.device)

        def __exit__(self, *exc):
            inside.pop()

    class Library:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, list(inside)))
                return N.DSPARK_OK
            return call

    for module in (H, T, C):
        monkeypatch.setattr(module, "_device_guard", Guard)
        monkeypatch.setattr(module, "_check_cuda", lambda *a: None)
        monkeypatch.setattr(module, "_stream_ptr", lambda device: 0)
    monkeypatch.setattr(N, "load", Library)
    w = torch.zeros(64, 16)
    head = VanillaMarkov(w, w)
    x, ids = torch.zeros(2, 3, 64), torch.zeros(2, 3, dtype=torch.int64)
    head.apply_block_logits(x, token_ids=ids)
    head.apply_block_logits_backward(x, token_ids=ids)
    head.transition_logits(ids)
    head.fused_lm_head_logits(torch.zeros(2, 3, 8), torch.zeros(64, 8), token_ids=ids)
    head.sample_block_tokens(x, first_prev_token_ids=ids[:, 0])
    head.sample_block_tokens_noalloc(x, first_prev_token_ids=ids[:, 0].contiguous(), out_tokens=ids, out_logits=x)
    head.teacher_forced_gradients(x, token_ids=ids, targets=ids)
    assert len(calls) == 9 and all(at == [head.device] for _, at in calls), calls
