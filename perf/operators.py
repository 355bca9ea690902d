"""Cases of the operators around the Markov head, in their plain form and as the library runs them.

Three operators stand next to the head's own entry points:

* ``process_logits``: penalties for repeated tokens, additive biases and grammar masks on corrected
  logits, with the greedy choice of every row, before a token is drawn or a drafted block verified;
* ``block_cross_entropy``: the teacher-forced training loss on corrected logits together with its
  gradient, which ``apply_block_logits_backward`` takes;
* ``GradientClipper``: the global norm over the head's (and any other) gradients, and clipping by it.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100

# The repository's vocabularies (129280, 151936, 1024), its 5- and 8-token blocks, its 320- and
# 2560-row training batches and its ranks; 32003 stands for a vocabulary of odd size, whose rows
# start at every alignment.
LISTED = (
    # One sequence decoding one token at a time: the smallest serving call, where latency is all.
    dict(name="step_b1_v129280", op="process", dtype="bf16", batch=1, block=0, vocab=129280, history=600, bias=16,
         mask=False),
    # A full decoding batch at fp32 logits after long contexts, each sequence with its grammar mask.
    dict(name="step_b64_v129280_long", op="process", dtype="fp32", batch=64, block=0, vocab=129280, history=32768,
         bias=0, mask=True),
    # Verification of drafted 8-token blocks: every position has its own history and mask.
    dict(name="verify_b32_m8_v151936", op="process", dtype="bf16", batch=32, block=8, vocab=151936, history=2048,
         bias=64, mask=True),
    # A small batch of 5-token blocks over an odd vocabulary.
    dict(name="verify_b7_m5_v32003", op="process", dtype="bf16", batch=7, block=5, vocab=32003, history=1000, bias=9,
         mask=True),
    # The smallest training step: ten fp32 rows.
    dict(name="loss_r10_v1024_fp32", op="loss", dtype="fp32", rows=10, vocab=1024, pad=0.0),
    # The ordinary teacher-forced batch (4 x 16 blocks of 5).
    dict(name="loss_r320_v129280", op="loss", dtype="bf16", rows=320, vocab=129280, pad=0.0),
    # The same with the fp32 logits that an fp32 LM head gives.
    dict(name="loss_r320_v129280_fp32", op="loss", dtype="fp32", rows=320, vocab=129280, pad=0.0),
    # The large batch, a fifth of its blocks padding.
    dict(name="loss_r2560_v129280_pad20", op="loss", dtype="bf16", rows=2560, vocab=129280, pad=0.2),
    # A ragged batch over an odd vocabulary.
    dict(name="loss_r135_v32003", op="loss", dtype="bf16", rows=135, vocab=32003, pad=0.2),
    # Gradients of the smallest head.
    dict(name="clip_v1024_k16", op="clip", vocab=1024, rank=16, others=0, most=1, clip=True),
    # Gradients of the head at its full vocabulary, rank 128.
    dict(name="clip_v129280_k128", op="clip", vocab=129280, rank=128, others=0, most=1, clip=True),
    # The head's gradients within those of a drafter: many ragged tensors of both types, packed in flat buffers.
    dict(name="clip_v32003_k64_many", op="clip", vocab=32003, rank=64, others=180, most=1000000, clip=True),
)


def listed():
    return [dict(c) for c in LISTED]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("process", "loss", "clip"))
    if op == "process":
        vocab = _log_int(rng, 1000, 151936)
        batch = _log_int(rng, 1, 64)
        block = rng.choice((0, 0, 1, 2, 3, 5, 8))
        return dict(op=op, dtype=rng.choice(("bf16", "fp32")), batch=batch,
                    block=min(block, max(1, 256 // batch)) if block else 0, vocab=vocab,
                    history=_log_int(rng, 1, 32768), bias=rng.choice((0, 1, 7, 64, 300)), mask=rng.random() < 0.6)
    if op == "loss":
        vocab = _log_int(rng, 1000, 151936)
        rows = min(_log_int(rng, 1, 4000), 2560 * 129280 // vocab)
        return dict(op=op, dtype=rng.choice(("bf16", "fp32")), rows=rows if rows * vocab < 1 << 27 else rows // 2,
                    vocab=vocab, pad=rng.choice((0.0, 0.2, 0.5)))
    return dict(op=op, vocab=_log_int(rng, 1000, 151936), rank=rng.choice((16, 64, 128, 200, 256)),
                others=rng.choice((0, 1, 5, 40, 180)), most=_log_int(rng, 100, 1000000), clip=rng.random() < 0.75)


# ------------------------------------------------------------------ inputs --

def _zipf(shape, vocab, gen):
    """Token ids with probabilities falling like 1 / (rank + 1), as text has them."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)) - 1).long().clamp_(0, vocab - 1)


def _pack_bits(allowed):
    """Truth values [..., V] as int32 words [..., ceil(V / 32)]: token v is bit v % 32 of word v // 32."""
    v = allowed.shape[-1]
    words = -(-v // 32)
    padded = torch.nn.functional.pad(allowed, (0, words * 32 - v)).view(*allowed.shape[:-1], words, 32)
    packed = (padded.long() << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int()


def _prepare_process(case, gen):
    b, m, v = case["batch"], max(1, case["block"]), case["vocab"]
    s = {}
    shape = (b, v) if not case["block"] else (b, m, v)
    logits = torch.randn((b, m, v), generator=gen, device="cuda") * 2.0
    # A few strong candidates in each row, as trained logits have.
    strong = torch.randint(0, v, (b, m, 4), generator=gen, device="cuda")
    logits.scatter_add_(2, strong, 4.0 + 4.0 * torch.rand((b, m, 4), generator=gen, device="cuda"))
    s["logits"] = logits.to(DTYPES[case["dtype"]]).view(shape)
    cap = case["history"]
    s["history"] = _zipf((b, cap), v, gen)
    # Sequences of different lengths in one batch; the first fills the buffer.
    s["history_lens"] = (torch.rand(b, generator=gen, device="cuda") * cap).long() + 1
    s["history_lens"][0] = cap
    s["history_lens"].clamp_(max=cap)
    s["prompt_lens"] = (s["history_lens"] * torch.rand(b, generator=gen, device="cuda")).long()
    s["repetition"] = 1.0 + 0.3 * torch.rand(b, generator=gen, device="cuda")
    s["frequency"] = 0.5 * torch.rand(b, generator=gen, device="cuda")
    s["presence"] = 0.5 * torch.rand(b, generator=gen, device="cuda")
    s["draft"] = _zipf((b, m), v, gen) if case["block"] else None
    s["bias_ids"] = s["bias_values"] = s["allowed"] = None
    if case["bias"]:
        k = min(case["bias"], v)
        s["bias_ids"] = torch.rand((b, v), generator=gen, device="cuda").topk(k, dim=1).indices
        s["bias_values"] = torch.randn((b, k), generator=gen, device="cuda") * 3.0
    if case["mask"]:
        # A grammar state allows a share of the vocabulary between next to nothing and nearly all.
        share = torch.rand((b, m, 1), generator=gen, device="cuda") ** 2
        s["allowed"] = _pack_bits(torch.rand((b, m, v), generator=gen, device="cuda") < share)
        if not case["block"]:
            s["allowed"] = s["allowed"].view(b, -1)
    s["out"] = torch.empty_like(s["logits"])
    s["tokens"] = torch.empty(shape[:-1], dtype=torch.int64, device="cuda")
    if own:
        # A serving program keeps one such object for its batch and updates the buffers behind it.
        from rank_markov_draft_vanillamarkov_b200 import TokenConstraints
        s["constraints"] = TokenConstraints(
            v, history=s["history"], history_lens=s["history_lens"], prompt_lens=s["prompt_lens"],
            repetition_penalty=s["repetition"], frequency_penalty=s["frequency"], presence_penalty=s["presence"],
            bias_ids=s["bias_ids"], bias_values=s["bias_values"])
    return s


def _prepare_loss(case, gen):
    r, v = case["rows"], case["vocab"]
    s = {"targets": _zipf((r,), v, gen)}
    logits = torch.randn((r, v), generator=gen, device="cuda") * 2.0
    # The model already leans towards the right token, more in some rows than in others.
    lean = 12.0 * torch.rand((r, 1), generator=gen, device="cuda")
    s["logits"] = logits.scatter_add_(1, s["targets"][:, None], lean).to(DTYPES[case["dtype"]])
    # Later positions of a block weigh less; padding rows carry the ignored target.
    s["weights"] = 0.8 ** (torch.arange(r, device="cuda") % 5).float()
    at = torch.randperm(r, generator=gen, device="cuda")[: int(round(case["pad"] * r))]
    s["targets"][at] = IGNORE
    s["grad"] = torch.empty_like(s["logits"])
    return s


def _clip_sizes(case):
    """The other tensors' elements, ragged between 1 and `most`: (type, elements) of each, alternating types."""
    n = case["others"]
    return [("bf16" if i % 2 else "fp32", max(1, int(round(math.exp(math.log(case["most"]) * ((i * 7919 + 13) % 1009) / 1008)))))
            for i in range(n)]


def _prepare_clip(case, gen):
    v, k = case["vocab"], case["rank"]
    sizes = [("fp32", v * k), ("fp32", v * k)] + _clip_sizes(case)
    total = {t: sum(n for u, n in sizes if u == t) for t in DTYPES}
    # Gradients packed one after another in one flat buffer for each type, as buckets for an all-reduce are.
    flat = {t: (torch.randn(total[t], generator=gen, device="cuda") * 1e-3).to(DTYPES[t]) for t in DTYPES if total[t]}
    # The embedding's gradient has rows for the tokens that occurred only.
    seen = torch.zeros(v, 1, device="cuda")
    seen[_zipf((320,), v, gen)] = 1.0
    flat["fp32"][: v * k].view(v, k).mul_(seen)
    out = {t: torch.empty_like(x) for t, x in flat.items()}
    s = {"flat": flat, "out": out}
    for name, of in (("grads", flat), ("outs", out)):
        at, views = {t: 0 for t in DTYPES}, []
        for i, (t, n) in enumerate(sizes):
            x = of[t][at[t]: at[t] + n]
            views.append(x.view(v, k) if i < 2 else x)
            at[t] += n
        s[name] = views
    elements = sum(n for _, n in sizes[1:])
    s["max_norm"] = 1e-3 * math.sqrt(elements) * (0.31 if case["clip"] else 3.1)
    if own:
        # A training program's gradient buffers stay where they are, and so does the object that knows them.
        from rank_markov_draft_vanillamarkov_b200 import GradientClipper
        s["clipper"] = GradientClipper(s["grads"], out=s["outs"])
    return s


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"process": _prepare_process, "loss": _prepare_loss, "clip": _prepare_clip}[case["op"]](case, gen)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------- plain forms --

def _plain_process(s):
    logits = s["logits"]
    x = logits.float()
    if x.dim() == 2:
        x = x[:, None, :]
    b, m, v = x.shape
    at = torch.arange(s["history"].shape[1], device="cuda")
    valid = at < s["history_lens"][:, None]
    generated = valid & (at >= s["prompt_lens"][:, None])
    zero = torch.zeros((b, v), dtype=torch.int32, device="cuda")
    count = zero.scatter_add(1, s["history"], generated.int())[:, None, :]
    seen = zero.scatter_add(1, s["history"], valid.int())[:, None, :]
    if s["draft"] is not None:
        # Position k has seen the drafted tokens before it.
        before = torch.ones((m, m), dtype=torch.int32, device="cuda").tril(-1).expand(b, m, m)
        drafted = torch.zeros((b, m, v), dtype=torch.int32, device="cuda")
        drafted = drafted.scatter_add(2, s["draft"][:, None, :].expand(b, m, m), before)
        count, seen = count + drafted, seen + drafted
    r = s["repetition"][:, None, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None, None] * count
    x = x - s["presence"][:, None, None] * (count > 0)
    if s["bias_ids"] is not None:
        bias = torch.zeros((b, v), device="cuda").scatter(1, s["bias_ids"], s["bias_values"])
        x = x + bias[:, None, :]
    if s["allowed"] is not None:
        words = s["allowed"].view(b, -1, s["allowed"].shape[-1])
        bits = (words[..., None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
        x = torch.where(bits.flatten(-2)[..., :v] != 0, x, -math.inf)
    y = x.to(logits.dtype)
    best = y.amax(-1, keepdim=True)
    tokens = torch.where(y == best, torch.arange(v, device="cuda"), v).amin(-1)
    return {"logits": y.view(logits.shape), "tokens": tokens.view(logits.shape[:-1])}


def _plain_loss(s):
    x, t = s["logits"].float(), s["targets"]
    valid = t != IGNORE
    w = torch.where(valid, s["weights"], 0.0)
    total = w.sum()
    scale = torch.where(total > 0, w / total, 0.0)
    at = torch.where(valid, t, 0)[:, None]
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    z = e.sum(-1, keepdim=True)
    rows = torch.where(valid, torch.log(z[:, 0]) - x.gather(1, at)[:, 0], 0.0)
    p = e / z
    p.scatter_add_(1, at, torch.full_like(z, -1.0))
    grad = torch.where(valid[:, None], p * scale[:, None], 0.0)
    return {"loss": (scale * rows).sum(), "rows": rows, "grad": grad.to(s["logits"].dtype)}


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["flat"].values()]).sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float(), "grads": {t: (x.float() * scale).to(x.dtype) for t, x in s["flat"].items()}}


def run(s):
    if not own:
        return {"process": _plain_process, "loss": _plain_loss, "clip": _plain_clip}[s["op"]](s)
    import rank_markov_draft_vanillamarkov_b200 as head
    if s["op"] == "process":
        out, tokens = head.process_logits(s["logits"], s["constraints"], draft_tokens=s["draft"], allowed=s["allowed"],
                                          out=s["out"], out_tokens=s["tokens"])
        return {"logits": out, "tokens": tokens}
    if s["op"] == "loss":
        loss, rows, grad = head.block_cross_entropy(s["logits"], s["targets"], weights=s["weights"],
                                                    ignore_index=IGNORE, reduction="mean", out_grad=s["grad"])
        return {"loss": loss, "rows": rows, "grad": grad}
    return {"norm": s["clipper"].clip(s["max_norm"]), "grads": s["out"]}


# -------------------------------------------------------- work and 64 bits --

def work(case):
    if case["op"] == "process":
        e = 2 if case["dtype"] == "bf16" else 4
        b, m, v = case["batch"], max(1, case["block"]), case["vocab"]
        n = b * m * v
        words = b * m * -(-v // 32) * 4 if case["mask"] else 0
        # Half of the padded history on average is a sequence's own; biases are an id and a value.
        return {"bytes": 2 * n * e + words + b * case["history"] * 4 + b * case["bias"] * 12 + b * m * 8, "flops": n}
    if case["op"] == "loss":
        e = 2 if case["dtype"] == "bf16" else 4
        r, v = case["rows"], case["vocab"]
        live = r - int(round(case["pad"] * r))
        # Ignored rows' logits need not be read; their gradient is written all the same.
        return {"bytes": (live + r) * v * e + r * 16, "flops": 5 * live * v}
    sizes = _clip_sizes(case)
    n = 2 * case["vocab"] * case["rank"] * 4 + sum(k * (2 if t == "bf16" else 4) for t, k in sizes)
    return {"bytes": 2 * n, "flops": n}


def _exact_process(s):
    b = s["logits"].shape[0]
    x = s["logits"].double().reshape(b, -1, s["logits"].shape[-1]).clone()
    v = x.shape[-1]
    for i in range(b):
        n, p = int(s["history_lens"][i]), int(s["prompt_lens"][i])
        rep, freq, pres = (float(s[k][i]) for k in ("repetition", "frequency", "presence"))
        count = torch.bincount(s["history"][i, p:n], minlength=v)
        prompt = torch.bincount(s["history"][i, :p], minlength=v) > 0
        for k in range(x.shape[1]):
            if k:
                count[s["draft"][i, k - 1]] += 1
            row = x[i, k]
            hit = prompt | (count > 0)
            row[hit] = torch.where(row[hit] > 0, row[hit] / rep, row[hit] * rep)
            row -= freq * count.double()
            row[count > 0] -= pres
            if s["bias_ids"] is not None:
                row[s["bias_ids"][i]] += s["bias_values"][i].double()
            if s["allowed"] is not None:
                words = s["allowed"].view(b, -1, s["allowed"].shape[-1])[i, k].long()
                at = torch.arange(v, device="cuda")
                row[((words[at // 32] >> (at % 32)) & 1) == 0] = -math.inf
    return {"logits": x.view(s["logits"].shape), "tokens": None}


def _exact_loss(s):
    keep = s["targets"] != IGNORE
    live = torch.nonzero(keep)[:, 0]
    rows = torch.zeros(len(keep), dtype=torch.float64, device="cuda")
    grad = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    w = s["weights"].double() * keep
    total = w.sum()
    if len(live):
        logp = torch.log_softmax(s["logits"][live].double(), dim=1)
        t = s["targets"][live]
        pick = torch.arange(len(live), device="cuda")
        rows[live] = -logp[pick, t]
        p = logp.exp_()
        p[pick, t] -= 1.0
        grad[live] = p.mul_((w[live] / total)[:, None])
    return {"loss": (w * rows).sum() / total if len(live) else w.sum(), "rows": rows, "grad": grad}


def _exact_clip(s):
    norm = math.sqrt(sum(float(torch.dot(g.double().flatten(), g.double().flatten())) for g in s["grads"]))
    scale = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": {t: x.double() * scale for t, x in s["flat"].items()}}


def exact(case, seed):
    return {"process": _exact_process, "loss": _exact_loss, "clip": _exact_clip}[case["op"]](prepare(case, seed))
