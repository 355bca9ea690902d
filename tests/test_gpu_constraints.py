"""Token constraints (process_logits, sample_block_tokens with constraints) against a plain 64-bit form, on B200.

Each value is held to the error of its fp32 operations (oracle.around) and one rounding to the logits' dtype; the
tokens must equal the lowest index of the largest returned value.
"""
import numpy as np
import pytest
import torch

from oracle import around
from oracle.philox import gumbel_noise
from rank_markov_draft_vanillamarkov_b200 import (DSparkError, TokenConstraints, VanillaMarkov, device_status,
                                                  last_algo, launch_count, process_logits, set_algo)
from rank_markov_draft_vanillamarkov_b200 import _native as N
from rank_markov_draft_vanillamarkov_b200.build import build

from _helpers import dtype_name, f64

pytestmark = pytest.mark.gpu
NEG = -(2.0 ** 120)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    N.load()
    device_status()
    yield
    set_algo(N.DSPARK_ALGO_AUTO)


def _words(allowed: np.ndarray) -> torch.Tensor:
    v = allowed.shape[-1]
    w = -(-v // 32)
    bits = np.zeros(allowed.shape[:-1] + (w * 32,), dtype=np.int64)
    bits[..., :v] = allowed
    if v % 32:
        bits[..., v:] = 1  # bits past the vocabulary mean nothing
    packed = (bits.reshape(*allowed.shape[:-1], w, 32) << np.arange(32)).sum(-1)
    return torch.from_numpy(packed.astype(np.uint32).view(np.int32).copy())


class Case:
    """CPU inputs of one call and their exact answer."""

    def __init__(self, batch, block, vocab, length, biases, dtype, mask, seed, drafted=True, lens=None):
        g = np.random.default_rng(seed)
        self.batch, self.block, self.vocab = batch, block, vocab
        self.logits = torch.from_numpy(g.normal(0, 3, (batch, max(1, block), vocab))).to(dtype)
        top = max(1, min(vocab, 50))  # ids that repeat, and ids all over the vocabulary
        ids = np.where(g.random((batch, length)) < 0.5, g.integers(0, top, (batch, length)),
                       g.integers(0, vocab, (batch, length)))
        self.lens = g.integers(0, length + 1, batch) if lens is None else np.asarray(lens)
        self.prompt = (self.lens * g.random(batch)).astype(np.int64)
        self.history = ids
        for b in range(batch):  # what lies behind a sequence's end is not read as ids
            self.history[b, self.lens[b]:] = -7
        f32 = lambda x: x.astype(np.float32)  # noqa: E731
        self.rep, self.freq, self.pres = f32(g.uniform(0.7, 1.5, batch)), f32(g.uniform(-0.3, 0.5, batch)), f32(
            g.uniform(-0.5, 0.7, batch))
        self.draft = None
        if block and drafted:
            self.draft = g.integers(0, top, (batch, block))
            self.draft[g.random((batch, block)) < 0.1] = -1
        self.bias_ids = self.bias_values = None
        if biases:
            self.bias_ids = g.integers(-1, vocab, (batch, biases))
            self.bias_values = f32(g.normal(0, 4, (batch, biases)))
        self.allowed = None
        if mask == "rows":
            self.allowed = g.random((batch, max(1, block), vocab)) < g.random((batch, max(1, block), 1))
            self.allowed[0, 0] = False  # a row that allows nothing
            self.allowed[-1, -1] = True
        elif mask == "batch":
            self.allowed = g.random((batch, 1, vocab)) < 0.5

    def constraints(self, **kw):
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        args = dict(history=dev(self.history.astype(np.int64)), history_lens=dev(self.lens.astype(np.int64)),
                    prompt_lens=dev(self.prompt), repetition_penalty=dev(self.rep), frequency_penalty=dev(self.freq),
                    presence_penalty=dev(self.pres), bias_ids=dev(self.bias_ids), bias_values=dev(self.bias_values))
        args.update(kw)
        return TokenConstraints(self.vocab, **args)

    def call_args(self):
        draft = None if self.draft is None else torch.from_numpy(self.draft.astype(np.int64)).cuda()
        allowed = None
        if self.allowed is not None:
            allowed = _words(self.allowed).cuda()
            if not self.block or self.allowed.shape[1] == 1 != self.block:
                allowed = allowed[:, 0].contiguous()
        return dict(draft_tokens=draft, allowed=allowed)

    def device_logits(self):
        x = self.logits.cuda()
        return x if self.block else x[:, 0].contiguous()

    def check(self, out, tokens):
        dtype = dtype_name(out.dtype)
        got = f64(out).reshape(self.logits.shape)
        x = f64(self.logits)
        for b in range(self.batch):
            for k in range(got.shape[1]):
                n, p = int(self.lens[b]), int(self.prompt[b])
                gen = list(self.history[b, p:n])
                if self.draft is not None:
                    gen += [t for t in self.draft[b, :k] if t >= 0]
                pairs = [] if self.bias_ids is None else list(zip(self.bias_ids[b], self.bias_values[b]))
                allowed = None if self.allowed is None else self.allowed[b, k % self.allowed.shape[1]]
                want, err = around.constrain_row(x[b, k], self.history[b, :p], gen, float(self.rep[b]),
                                                 float(self.freq[b]), float(self.pres[b]), pairs, allowed)
                _close(got[b, k], want, err, dtype)
        if tokens is not None:
            assert tokens.dtype == torch.int64
            picks = tokens.cpu().numpy().reshape(got.shape[:2])
            for b in range(self.batch):
                for k in range(got.shape[1]):
                    assert picks[b, k] == around.choose(got[b, k]), (b, k)


def _close(got, want, err, dtype):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    tol = err[fin] + around.HALF_STEP[dtype] * (np.abs(want[fin]) + err[fin])
    bad = ~(np.abs(got[fin] - want[fin]) <= tol)
    assert not bad.any(), (np.flatnonzero(fin)[bad][:5], got[fin][bad][:5], want[fin][bad][:5])


SHAPES = [  # batch, block, vocab, history, biases, mask
    (1, 0, 1, 1, 0, None),
    (1, 0, 7, 3, 2, "rows"),
    (3, 0, 31, 5, 4, "rows"),
    (2, 1, 32, 40, 0, "batch"),
    (2, 4, 33, 6, 3, "rows"),
    (1, 0, 1024, 1, 1, None),
    (5, 3, 1000, 17, 40, "batch"),
    (4, 8, 4096, 300, 5, "rows"),
    (3, 5, 4097, 64, 300, "rows"),
    (2, 2, 8191, 2000, 0, None),
    (1, 3, 32003, 1000, 9, "rows"),
    (2, 0, 40961, 5000, 64, "rows"),
    (9, 2, 16385, 33, 1, None),
    (1, 0, 129280, 600, 16, None),
    (1, 2, 151936, 40000, 64, "rows"),
    (40, 0, 2056, 2, 0, "rows"),
    (3, 1, 9001, 33000, 2, None),
    (1, 2, 5000, 70000, 3, None),
    (2, 3, 3001, 4, 70000, "rows"),
    (1, 19, 2500, 9, 2, "rows"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d_m%d_v%d_l%d_k%d_%s" % s)
def test_against_the_plain_form(shape, dtype):
    batch, block, vocab, length, biases, mask = shape
    case = Case(batch, block, vocab, length, biases, dtype, mask, seed=vocab + length)
    x = case.device_logits()
    keep = x.clone()
    out, tokens = process_logits(x, case.constraints(), **case.call_args())
    torch.cuda.synchronize()
    assert torch.equal(x, keep)
    case.check(out, tokens)
    # In place, without tokens: the same bits.
    same, none = process_logits(x, case.constraints(), out=x, return_tokens=False, **case.call_args())
    assert same is x and none is None and torch.equal(_bits(x), _bits(out))
    assert device_status() == 0


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["padded", "odd_start", "odd_padding", "mbv", "last_position", "out_other"])
def test_strides_and_alignments(layout, dtype):
    """Views that serving code has in hand, out of and in place, guard cells around the rows left as they were."""
    case = Case(3, 4, 5003, 50, 6, dtype, "rows", seed=5)
    x = case.logits.cuda()
    b, m, v = x.shape
    if layout == "padded":
        pads = (0, 5)  # rows of 5008 elements
    elif layout == "odd_padding":
        pads = (1, 3)
    else:
        pads = (3, 8)
    hold = torch.full((b, m, v + sum(pads)), 77.0, dtype=dtype, device="cuda")
    view = hold[:, :, pads[0]: pads[0] + v]
    if layout == "mbv":
        hold = torch.full((m, b, v + sum(pads)), 77.0, dtype=dtype, device="cuda")
        view = hold[:, :, pads[0]: pads[0] + v].transpose(0, 1)
    elif layout == "last_position":
        hold = torch.full((b, 2, m, v), 77.0, dtype=dtype, device="cuda")
        view = hold[:, 1]
    view.copy_(x)
    args = case.call_args()
    if layout == "out_other":  # rows of the output start at other alignments than the input's
        out_hold = torch.full((b, m, v + 2), 77.0, dtype=dtype, device="cuda")
        out, tokens = process_logits(view, case.constraints(), out=out_hold[:, :, 1: 1 + v], **args)
        case.check(out, tokens)
        assert (out_hold[:, :, 0] == 77).all() and (out_hold[:, :, -1] == 77).all()
        return
    out, tokens = process_logits(view, case.constraints(), **args)
    case.check(out, tokens)
    keep = hold.clone()
    process_logits(view, case.constraints(), out=view, **args)
    case.check(view, None)
    view.copy_(x)
    assert torch.equal(_bits(hold), _bits(keep))


def test_history_lengths_at_their_ends():
    """No history, lengths 0, 1 and full, lengths out of range (clamped), a prompt as long as the history."""
    for lens, prompt in (([0, 1, 6, 6], [0, 0, 0, 6]), ([6, 6, 0, 1], [6, 3, 0, 1])):
        case = Case(4, 2, 300, 6, 0, torch.float32, None, seed=1, lens=lens)
        case.prompt = np.asarray(prompt)
        case.check(*process_logits(case.device_logits(), case.constraints(), **case.call_args()))
    case = Case(2, 2, 300, 6, 0, torch.float32, None, seed=2, lens=[6, 0])
    case.prompt = np.asarray([6, 0])
    c = case.constraints(history_lens=torch.tensor([900, -3]).cuda(), prompt_lens=torch.tensor([44, -1]).cuda())
    case.check(*process_logits(case.device_logits(), c, **case.call_args()))
    none = TokenConstraints(300, repetition_penalty=1.3)
    x = case.device_logits()
    out, _ = process_logits(x, none)
    assert torch.equal(out, x)
    empty = TokenConstraints(300, history=torch.empty(2, 0, dtype=torch.int64, device="cuda"),
                             history_lens=torch.zeros(2, dtype=torch.int64, device="cuda"), presence_penalty=2.0)
    assert torch.equal(process_logits(x, empty)[0], x)
    assert device_status() == 0


def test_default_lengths_take_the_whole_history():
    case = Case(2, 0, 500, 9, 0, torch.float32, None, seed=8, lens=[9, 9])
    case.prompt = np.zeros(2, dtype=np.int64)
    c = case.constraints(history_lens=None, prompt_lens=None)
    case.check(*process_logits(case.device_logits(), c))


def test_numbers_and_shared_biases():
    """Penalties as numbers and one bias list for all sequences equal the tensor forms bit for bit."""
    case = Case(3, 2, 700, 20, 5, torch.bfloat16, None, seed=3)
    case.rep[:], case.freq[:], case.pres[:] = 1.25, 0.25, 0.5
    case.bias_ids[:], case.bias_values[:] = case.bias_ids[0], case.bias_values[0]
    a, ta = process_logits(case.device_logits(), case.constraints(), **case.call_args())
    c = case.constraints(repetition_penalty=1.25, frequency_penalty=0.25, presence_penalty=0.5,
                         bias_ids=torch.from_numpy(case.bias_ids[0].copy()).cuda(),
                         bias_values=torch.from_numpy(case.bias_values[0].copy()).cuda())
    b, tb = process_logits(case.device_logits(), c, **case.call_args())
    assert torch.equal(_bits(a), _bits(b)) and torch.equal(ta, tb)
    case.check(a, ta)


def test_last_bias_of_an_id_counts():
    x = torch.zeros(1, 100, device="cuda")
    ids = torch.tensor([[5, 9, 5, -1, 5, 9]], device="cuda")
    values = torch.tensor([[1.0, 2.0, 3.0, 9.0, 4.0, -1.0]], device="cuda")
    out, tokens = process_logits(x, TokenConstraints(100, bias_ids=ids, bias_values=values))
    want = torch.zeros(100)
    want[5], want[9] = 4.0, -1.0
    assert torch.equal(out[0].cpu(), want) and tokens.item() == 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_infinities_nan_and_lowest_values(dtype):
    """They pass through the same arithmetic where allowed and vanish where not."""
    case = Case(4, 0, 2100, 30, 0, dtype, "rows", seed=12)
    x = case.logits
    low = torch.finfo(dtype).min
    case.allowed[1:, 0, :] = True
    x[1, 0, 100], x[1, 0, 200], x[1, 0, 300] = float("inf"), float("-inf"), low
    x[2, 0, 1700] = x[2, 0, 400] = float("nan")
    x[3, 0, 0] = float("nan")
    x[3, 0, 1] = float("inf")
    case.allowed[3, 0, 0] = case.allowed[3, 0, 1] = False
    case.history[1:, 0] = [100, 400, 1]
    case.lens[1:] = np.maximum(case.lens[1:], 1)
    case.history[case.history < 0] = 3
    case.check(*process_logits(case.device_logits(), case.constraints(), **case.call_args()))
    x[:] = float("-inf")
    out, tokens = process_logits(case.device_logits(), case.constraints(), **case.call_args())
    assert torch.equal(tokens.cpu(), torch.zeros(4, dtype=torch.int64)) and bool((out == float("-inf")).all())
    x[:] = low
    case.allowed[:] = True
    out, tokens = process_logits(case.device_logits(), TokenConstraints(2100), **case.call_args())
    assert torch.equal(out, case.device_logits()) and int(tokens.sum()) == 0


def test_ties_take_the_lowest_id():
    x = torch.zeros(2, 20000, dtype=torch.bfloat16, device="cuda")
    x[0, 19999] = x[0, 12345] = x[0, 777] = 4.0
    x[1] = -0.0
    x[1, 17] = 0.0
    _, tokens = process_logits(x, TokenConstraints(20000))
    assert tokens.tolist() == [777, 0]


@pytest.mark.parametrize("what", ["history", "history_negative", "draft", "bias"])
def test_ids_outside_the_vocabulary_are_left_out_and_reported(what):
    case = Case(2, 3, 1500, 12, 4, torch.float32, None, seed=21, lens=[12, 12])
    case.prompt[:] = 2
    bad = {"history": 1500, "history_negative": -1, "draft": 1 << 40, "bias": 1500}[what]
    history, draft, bias = case.history.copy(), case.draft.copy(), case.bias_ids.copy()
    if what.startswith("history"):
        history[1, 5] = bad
    elif what == "draft":
        draft[0, 1] = bad
        case.draft[0, 1] = -1
    else:
        bias[0, 2] = bad
        case.bias_ids[0, 2] = -1
    t = lambda a: torch.from_numpy(a.astype(np.int64)).cuda()  # noqa: E731
    c = case.constraints(history=t(history), bias_ids=t(bias))
    out, tokens = process_logits(case.device_logits(), c, draft_tokens=t(draft))
    assert device_status() == N.DSPARK_STATUS_TOKEN_RANGE
    if what.startswith("history"):  # compare against a history without the entry
        keep = [i for i in range(12) if i != 5]
        full = case.history
        case.history = np.concatenate([full[:, keep], full[:, :1]], axis=1)
        case.history[0] = full[0]
        case.lens = np.asarray([12, 11])
    case.check(out, tokens)


def test_long_offsets():
    """Rows further apart than 2^31 elements."""
    v, far = 4099, (1 << 31) + 8
    flat = torch.empty(far + v, dtype=torch.bfloat16, device="cuda")
    case = Case(2, 0, v, 10, 3, torch.bfloat16, "rows", seed=30)
    x = flat.as_strided((2, v), (far, 1))
    x.copy_(case.device_logits())
    out, tokens = process_logits(x, case.constraints(), **case.call_args())
    case.check(out, tokens)
    process_logits(x, case.constraints(), out=x, **case.call_args())
    assert torch.equal(_bits(x.contiguous()), _bits(out))


def test_repeats_are_equal_and_streams_do_not_share_state():
    case = Case(6, 4, 20011, 400, 20, torch.bfloat16, "rows", seed=40)
    c, args, x = case.constraints(), case.call_args(), case.device_logits()
    first, tok = process_logits(x, c, **args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            got.append(process_logits(x, c, **args))
    torch.cuda.synchronize()
    for out, t in got:
        assert torch.equal(_bits(out), _bits(first)) and torch.equal(t, tok)


def test_captured_calls_follow_the_buffers():
    """Two graphs over one object replayed after the history, the logits and the masks changed, also at once."""
    a, b = (Case(3, 2, 6001, 80, 4, torch.float32, "rows", seed=s, lens=[80, 3, 11]) for s in (50, 51))
    c, args, x = a.constraints(), a.call_args(), a.device_logits()
    process_logits(x, c, **args)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(process_logits(x, c, **args))
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out, tokens in outs:
        a.check(out, tokens)
    other, oargs = b.constraints(), b.call_args()
    x.copy_(b.device_logits())
    for mine, theirs in zip(c._kept, other._kept):
        mine.copy_(theirs)
    for key in args:
        args[key].copy_(oargs[key])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, tokens in outs:
        b.check(out, tokens)


def test_one_row_for_many_sequences():
    """An input row shared by all sequences (stride 0), each with its own history; written out of place."""
    case = Case(5, 0, 3001, 40, 2, torch.bfloat16, "rows", seed=60)
    case.logits[:] = case.logits[:1]
    x = case.logits[0].cuda().expand(5, 3001)
    case.check(*process_logits(x, case.constraints(), **case.call_args()))
    with pytest.raises(DSparkError):
        process_logits(x, case.constraints(), out=x, **case.call_args())


@pytest.mark.parametrize("batch,block,vocab", [(1, 40, 700), (2, 9, 5000), (70, 3, 1500), (1, 70, 20000)])
def test_long_blocks_count_every_drafted_token(batch, block, vocab):
    """Blocks past the rows that one CTA takes, with the same tokens drafted again and again."""
    case = Case(batch, block, vocab, 5, 3, torch.float32, "rows", seed=block)
    case.draft = np.random.default_rng(1).integers(0, 3, (batch, block))
    case.check(*process_logits(case.device_logits(), case.constraints(), **case.call_args()))


@pytest.mark.parametrize("temperature", [0.7, float("inf")])
@pytest.mark.parametrize("batch,block,vocab,dtype", [(3, 40, 70, torch.float32), (1, 9, 33, torch.bfloat16),
                                                     (300, 17, 600, torch.bfloat16), (2, 8, 30000, torch.float32)])
def test_draws_of_a_block(batch, block, vocab, dtype, temperature):
    """The C entry draws from the constrained logits of a block; only allowed tokens, at any temperature."""
    case = Case(batch, block, vocab, 6, 3, dtype, "rows", seed=batch)
    case.allowed[..., 5] = True
    x, args, c = case.device_logits(), case.call_args(), case.constraints()
    out, tokens = torch.empty_like(x), torch.empty(batch, block, dtype=torch.int64, device="cuda")
    scratch = c._scratch(x.device, batch, block, block - 1, True)
    words = args["allowed"].shape[-1]
    for _ in range(5):
        N.check(N.load().dspark_markov_process_logits(
            x.data_ptr(), out.data_ptr(), batch, block, vocab, block * vocab, vocab, block * vocab, vocab, c._ref,
            args["draft_tokens"].data_ptr(), block, 0, args["allowed"].data_ptr(), block * words, words,
            tokens.data_ptr(), block, temperature, 77, scratch.data_ptr(), 0 if dtype == torch.float32 else 1,
            torch.cuda.current_stream().cuda_stream), "process_logits")
        got, picks = f64(out), tokens.cpu().numpy()
        if _ == 0:
            case.check(out, None)
        for b in range(0, batch, max(1, batch // 8)):
            for k in range(block):
                assert case.allowed[b, k, picks[b, k]], (b, k)
                s = got[b, k] / min(temperature, 1e38) + gumbel_noise(77, b, k, vocab)
                assert s[picks[b, k]] >= s.max() - 1e-4, (b, k)


def _draw(c, x, out, draft, allowed, temperature, seed=77):
    """The tokens of a (B, M, V) view drawn by the C entry into the view ``out``."""
    batch, block, vocab = x.shape
    tokens = torch.full((batch, block), -5, dtype=torch.int64, device="cuda")
    scratch = c._scratch(x.device, batch, block, block - 1 if draft is not None else 0, True)
    words = allowed.shape[-1] if allowed is not None else 0
    N.check(N.load().dspark_markov_process_logits(
        x.data_ptr(), out.data_ptr(), batch, block, vocab, x.stride(0), x.stride(1), out.stride(0), out.stride(1),
        c._ref, draft.data_ptr() if draft is not None else None, block, 0,
        allowed.data_ptr() if allowed is not None else None, block * words, words, tokens.data_ptr(), block,
        temperature, seed, scratch.data_ptr(), 0 if x.dtype == torch.float32 else 1,
        torch.cuda.current_stream().cuda_stream), "process_logits")
    return tokens


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [1, 5, 13, 1001, 32003])
@pytest.mark.parametrize("listed", ["all", "first", "last", "none"])
def test_draws_of_rows_that_allow_nothing(listed, vocab, dtype):
    """Token 0, wherever rows start in and out, whatever the history lists; other rows draw what they allow."""
    ids = {"all": list(range(vocab)), "first": [0], "last": [vocab - 1], "none": []}[listed]
    history = torch.tensor([ids, ids], dtype=torch.int64, device="cuda").view(2, len(ids))
    c = TokenConstraints(vocab, history=history, repetition_penalty=1.2, presence_penalty=0.5)
    masks = np.zeros((2, 3, vocab), dtype=bool)
    masks[1, 1, vocab // 2] = True
    allowed = _words(masks).cuda()
    g = torch.Generator().manual_seed(vocab)
    for at_in, at_out in ((0, 0), (1, 1), (0, 1), (1, 3), (5, 5)):
        hold = torch.zeros(6 * vocab + 16, dtype=dtype, device="cuda")
        x = hold[at_in: at_in + 6 * vocab].view(2, 3, vocab)
        x.copy_(torch.randn(2, 3, vocab, generator=g))
        other = torch.zeros(6 * vocab + 16, dtype=dtype, device="cuda")
        out = other[at_out: at_out + 6 * vocab].view(2, 3, vocab)
        for temperature in (0.7, 1e-3, float("inf"), 0.0):
            want = [[0, 0, 0], [0, vocab // 2, 0]]
            assert _draw(c, x, out, None, allowed, temperature).tolist() == want, (at_in, at_out, temperature)
            assert bool((out[0] == float("-inf")).all())
        assert _draw(c, x, x, None, allowed, 0.7).tolist() == want
    assert device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("temperature", [1e-5, 0.1, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("listed", [False, True], ids=["copied", "listed"])
def test_draws_from_logits_whose_quotient_leaves_the_range(listed, temperature, dtype):
    """Only allowed tokens, and of those the largest where they lie further apart than any noise."""
    vocab, low = 700, torch.finfo(dtype).min
    at = [699, 400, 130, 33, 3]
    # Allowed logits of each row, by those ids; the largest, or None where several are.
    rows = [([low] * 5, None), ([low, low, -1e38, low, low], 130), ([-1e38, low, -3e38, low, -2e38], 699),
            ([1e38, 3e38, 2e38, 1.0, low], 400), ([3e38, -low, 3.2e38, 0.0, 0.0], 400), ([-2e37, -1e37, low, low, low], 400),
            ([float("-inf"), low, float("-inf"), low, low], None), ([float("inf"), -low, 0.0, 1.0, 2.0], 699)]
    x = torch.zeros(len(rows), 1, vocab)
    masks = np.zeros((len(rows), 1, vocab), dtype=bool)
    masks[:, 0, at] = True
    for i, (values, _) in enumerate(rows):
        x[i, 0, at] = torch.tensor(values)
    x = x.to(dtype).cuda()
    # Penalties that change nothing keep listed logits as they are.
    c = TokenConstraints(vocab, history=torch.tensor(at, device="cuda").expand(len(rows), 5).contiguous()) if listed \
        else TokenConstraints(vocab)
    finite = [np.isfinite(f64(x[i, 0, at])) for i in range(len(rows))]
    for seed in range(20):
        out = torch.empty_like(x)
        picks = _draw(c, x, out, None, _words(masks).cuda(), temperature, seed)[:, 0].tolist()
        assert torch.equal(_bits(out[:, :, at]), _bits(x[:, :, at]))
        for i, (_, want) in enumerate(rows):
            if want is not None:
                assert picks[i] == want, (i, seed)
            else:
                assert picks[i] in at and finite[i][at.index(picks[i])], (i, seed)
    assert device_status() == 0


def test_empty_calls():
    n = launch_count()
    c = TokenConstraints(50)
    for shape in ((0, 50), (0, 3, 50), (4, 0, 50)):
        out, tokens = process_logits(torch.empty(shape, device="cuda"), c)
        assert out.shape == shape and tokens.shape == shape[:-1]
    assert launch_count() == n


def test_refusals():
    x = torch.zeros(2, 3, 64, device="cuda")
    c = TokenConstraints(64)
    bad = [
        lambda: process_logits(x.double(), c),
        lambda: process_logits(x.cpu(), c),
        lambda: process_logits(x[0, 0], c),
        lambda: process_logits(x, TokenConstraints(65)),
        lambda: process_logits(x.transpose(1, 2).contiguous().transpose(1, 2), c),
        lambda: process_logits(x, c, out=x.bfloat16()),
        lambda: process_logits(x, c, out=x[:1]),
        lambda: process_logits(x, c, draft_tokens=torch.zeros(2, 2, dtype=torch.int64, device="cuda")),
        lambda: process_logits(x, c, draft_tokens=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: process_logits(x[:, 0], c, draft_tokens=torch.zeros(2, 1, dtype=torch.int64, device="cuda")),
        lambda: process_logits(x, c, allowed=torch.zeros(2, 3, 2, dtype=torch.int64, device="cuda")),
        lambda: process_logits(x, c, allowed=torch.zeros(2, 3, 3, dtype=torch.int32, device="cuda")),
        lambda: process_logits(x, c, allowed=torch.zeros(2, 3, 2, dtype=torch.int32)),
        lambda: process_logits(x, c, out_tokens=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: process_logits(x, TokenConstraints(64, history=torch.zeros(3, 4, dtype=torch.int64, device="cuda"))),
        lambda: TokenConstraints(64, history=torch.zeros(3, 4, dtype=torch.int32, device="cuda")),
        lambda: TokenConstraints(64, history=torch.zeros(4, 3, dtype=torch.int64, device="cuda").t()),
        lambda: TokenConstraints(64, history=torch.zeros(3, 4, dtype=torch.int64, device="cuda"),
                                 history_lens=torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: TokenConstraints(64, bias_ids=torch.zeros(3, dtype=torch.int64, device="cuda")),
        lambda: TokenConstraints(64, bias_ids=torch.zeros(3, dtype=torch.int64, device="cuda"),
                                 bias_values=torch.zeros(4, device="cuda")),
        lambda: TokenConstraints(64, frequency_penalty=torch.zeros(2, dtype=torch.float64, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    # Overlap that is not in place, and rows that overlap one another, are refused by the library.
    flat = torch.zeros(1000, device="cuda")
    with pytest.raises(DSparkError):
        process_logits(flat[:64].view(1, 64), c, out=flat[32:96].view(1, 64))
    with pytest.raises(DSparkError):
        process_logits(x, c, out=flat.as_strided((2, 3, 64), (64, 64, 1)))
    with pytest.raises(DSparkError):
        process_logits(x, c, out=x.view(6, 64).as_strided((2, 3, 64), (64, 128, 1)))


# ----------------------------------------------------------- in the sampler --

def _head(vocab, rank, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    w = [(torch.randn(vocab, rank, generator=g) * 0.3).to(dtype).cuda() for _ in range(2)]
    return VanillaMarkov(*w)


@pytest.mark.parametrize("batch,m,vocab,rank,ldt,wdt", [
    (4, 5, 2056, 64, torch.bfloat16, torch.bfloat16),
    (3, 4, 2056, 128, torch.float32, torch.bfloat16),
    (2, 3, 1001, 64, torch.bfloat16, torch.bfloat16),
    (130, 2, 1024, 64, torch.bfloat16, torch.bfloat16),
    (2, 6, 515, 16, torch.float32, torch.float32),
    (1, 1, 1024, 256, torch.bfloat16, torch.bfloat16),
])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_constrained_sampler(batch, m, vocab, rank, ldt, wdt, temperature):
    """The chain equals the teacher-forced correction of its own tokens, constrained as a block."""
    head = _head(vocab, rank, wdt, seed=vocab + rank)
    case = Case(batch, m, vocab, 30, 5, ldt, "rows", seed=batch + m)
    case.allowed[0, 0, ::3] = True
    base = case.logits.cuda()
    first = torch.arange(batch, device="cuda") * 7 % vocab
    allowed = case.call_args()["allowed"]
    tokens, logits = head.sample_block_tokens(base, first_prev_token_ids=first, temperature=temperature, seed=77,
                                              constraints=case.constraints(), allowed=allowed)
    prev = torch.cat([first[:, None], tokens[:, :-1]], dim=1)
    corrected = head.apply_block_logits(base, token_ids=prev)
    case.logits, case.draft = corrected.cpu(), tokens.cpu().numpy()
    want, greedy = process_logits(corrected, case.constraints(), draft_tokens=tokens, allowed=allowed)
    case.check(want, greedy)
    # The corrections of a block and of its positions sum the same products, perhaps in another order: their
    # roundings may differ by one step, which the repetition penalty scales by less than 2.
    a, b = f64(logits), f64(want)
    fin = np.isfinite(b)
    assert np.array_equal(fin, np.isfinite(a))
    step = 4 * around.HALF_STEP[dtype_name(ldt)]
    assert (np.abs(a[fin] - b[fin]) <= step * (np.abs(b[fin]) + np.abs(f64(corrected))[fin] + 8.0)).all()
    assert tokens.dtype == torch.int64
    picks = tokens.cpu().numpy()
    for i in range(batch):
        for k in range(m):
            if temperature == 0.0:
                assert picks[i, k] == around.choose(a[i, k])
            else:
                s = a[i, k] / temperature + gumbel_noise(77, i, k, vocab)
                assert s[picks[i, k]] >= s.max() - 1e-4, (i, k)
    assert device_status() == 0


@pytest.mark.parametrize("vocab,dtype", [(5, torch.bfloat16), (13, torch.bfloat16), (1001, torch.float32),
                                         (2056, torch.bfloat16)])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_constrained_sampler_of_rows_that_allow_nothing(vocab, dtype, temperature):
    """Such a position gives token 0, which the next position then follows like any other."""
    head = _head(vocab, 64, dtype, seed=vocab)
    base = torch.randn(3, 4, vocab, device="cuda").to(dtype)
    history = torch.arange(vocab, device="cuda").expand(3, vocab).contiguous()
    masks = np.zeros((3, 4, vocab), dtype=bool)
    masks[1, 2, vocab - 2] = True
    tokens, logits = head.sample_block_tokens(
        base, first_prev_token_ids=torch.tensor([1, 2, 3], device="cuda"), temperature=temperature, seed=5,
        constraints=TokenConstraints(vocab, history=history, frequency_penalty=0.5), allowed=_words(masks).cuda())
    want = torch.zeros(3, 4, dtype=torch.int64)
    want[1, 2] = vocab - 2
    assert torch.equal(tokens.cpu(), want)
    assert np.array_equal(f64(logits) > -np.inf, masks)
    assert device_status() == 0


@pytest.mark.parametrize("batch,m,vocab,rank,ldt", [(3, 3, 129280, 128, torch.bfloat16),
                                                    (2, 2, 129280, 64, torch.float32),
                                                    (2, 4, 151936, 64, torch.bfloat16)])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_constrained_sampler_at_full_vocabularies(batch, m, vocab, rank, ldt, temperature):
    """The strided corrections on the tensor cores, and lists in several parts of the vocabulary."""
    test_constrained_sampler(batch, m, vocab, rank, ldt, torch.bfloat16, temperature)
    assert last_algo() == 1  # process_logits came last
    head = _head(vocab, rank, torch.bfloat16, seed=1)
    head.sample_block_tokens(torch.zeros(batch, m, vocab, dtype=ldt, device="cuda"),
                             first_prev_token_ids=torch.zeros(batch, dtype=torch.int64, device="cuda"),
                             temperature=temperature, constraints=TokenConstraints(vocab))
    assert last_algo() == 2


def test_sampler_without_effective_constraints_is_the_plain_sampler():
    head = _head(2056, 64, torch.bfloat16, seed=2)
    base = torch.randn(4, 5, 2056, device="cuda").bfloat16()
    first = torch.tensor([1, 2, 3, 4], device="cuda")
    t0, c0 = head.sample_block_tokens(base, first_prev_token_ids=first)
    t1, c1 = head.sample_block_tokens(base, first_prev_token_ids=first, constraints=TokenConstraints(2056))
    assert (t0 == t1).all()
    assert (f64(c0) - f64(c1)).__abs__().max() <= 2 ** -7 * np.abs(f64(c0)).max()


def test_constrained_sampler_in_a_graph():
    head = _head(2056, 64, torch.bfloat16, seed=3)
    case = Case(3, 4, 2056, 20, 3, torch.bfloat16, "batch", seed=9)
    base, first = case.logits.cuda(), torch.tensor([5, 6, 7], device="cuda")
    c, allowed = case.constraints(), case.call_args()["allowed"]
    want = head.sample_block_tokens(base, first_prev_token_ids=first, constraints=c, allowed=allowed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = head.sample_block_tokens(base, first_prev_token_ids=first, constraints=c, allowed=allowed)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(_bits(got[1]), _bits(want[1]))


def test_constrained_sampler_refusals():
    head = _head(256, 64, torch.bfloat16, seed=4)
    base = torch.zeros(2, 3, 256, dtype=torch.bfloat16, device="cuda")
    first = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        head.sample_block_tokens(base, first_prev_token_ids=first, constraints=TokenConstraints(255))
    with pytest.raises(ValueError):
        head.sample_block_tokens(base, first_prev_token_ids=first,
                                 allowed=torch.zeros(2, 2, 8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        head.sample_block_tokens(base, first_prev_token_ids=first, constraints=TokenConstraints(256),
                                 out_tokens=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(DSparkError):
        head.sample_block_tokens(base, first_prev_token_ids=first, constraints=TokenConstraints(256), out_logits=base)


def test_histories_past_the_supported_length_are_refused():
    """By the library's error, from both callers; 8 GB that nothing touches."""
    history = torch.empty(1, 1 << 30, dtype=torch.int64, device="cuda")
    c = TokenConstraints(256, history=history, history_lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    base = torch.zeros(1, 3, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(DSparkError):
        process_logits(base, c)
    with pytest.raises(DSparkError):
        _head(256, 64, torch.bfloat16, seed=4).sample_block_tokens(
            base, first_prev_token_ids=torch.zeros(1, dtype=torch.int64, device="cuda"), constraints=c)
