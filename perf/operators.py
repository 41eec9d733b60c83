"""Cases of the vocabulary operators: what a language model runs where its hidden states meet its vocabulary.

  head     the output projection with its softmax cross entropy, in pieces of the vocabulary, without keeping
           the logits: loss and log-sum-exp per row, and the gradients of the hidden states and of the weight
  distill  distillation from a teacher's top logits: loss per row, and the gradient of the student's logits
  embed    the embedding lookup with scaling, and the table's gradient, summed in the order of the sorted tokens

``run`` computes them in a plain form, or, where ``own`` is true, by the calls of ``ls_vocab``.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_IGNORE = -100


# --- cases --------------------------------------------------------------------
def _head(name, mode, dtype, rows, hidden, vocab, smoothing=0.0, ignored=0.0):
    return {"name": name, "op": "head", "mode": mode, "dtype": dtype, "rows": rows, "hidden": hidden,
            "vocab": vocab, "smoothing": smoothing, "ignored": ignored}


def _distill(name, mode, dtype, rows, vocab, k, temperature, tail):
    return {"name": name, "op": "distill", "mode": mode, "dtype": dtype, "rows": rows, "vocab": vocab, "k": k,
            "temperature": temperature, "tail": tail}


def _embed(name, mode, dtype, tokens, hidden, vocab, ids="zipf", padded=0.0):
    return {"name": name, "op": "embed", "mode": mode, "dtype": dtype, "tokens": tokens, "hidden": hidden,
            "vocab": vocab, "ids": ids, "padded": padded}


def listed():
    return [
        # One token's log-probability while serving a GPT-2-large head: the weight is read once, nothing else counts.
        _head("head score 1 token", "score", "bf16", 1, 1280, 50257),
        # The perplexity of one ragged batch with a Transformer-base head.
        _head("head score 333 rows", "score", "f16", 333, 512, 32000),
        # A small model's training step, where launches and latency count; no size is a multiple of a tile.
        _head("head train small", "train", "f16", 130, 264, 4099, 0.1, 0.1),
        # A BERT-base training step (8 x 512 tokens) with label smoothing and some padding.
        _head("head train BERT-base", "train", "f16", 4096, 768, 30522, 0.1, 0.1),
        # A GPT-2-large training step (4 x 1024 tokens), the vocabulary not padded.
        _head("head train GPT-2-large", "train", "bf16", 4096, 1280, 50257),
        # Watching the distillation loss of a handful of tokens, in FP32.
        _distill("distill loss 5 rows", "loss", "f32", 5, 50264, 10, 1.0, False),
        # A BERT-base student (padded vocabulary) trained on 32 stored logits for each token.
        _distill("distill train BERT-base", "train", "f16", 4096, 30528, 32, 2.0, False),
        # A large vocabulary; the teacher's stored log-sum-exp keeps the mass of its tail.
        _distill("distill train wide", "train", "bf16", 2047, 131072, 64, 1.0, True),
        # One decoding step of a batch of 32: one row for each sequence.
        _embed("embed lookup 32", "lookup", "f16", 32, 1280, 50257),
        # A Transformer-base step, 64 x 64 tokens with padding, every id about as likely.
        _embed("embed train uniform", "train", "f32", 4096, 512, 32000, "uniform", 0.1),
        # A GPT-2-large step: the dense gradient's rows that no token has are most of the work.
        _embed("embed train GPT-2-large", "train", "f16", 4096, 1280, 50257),
        # A long batch of BERT-base tokens: a few ids have thousands of them.
        _embed("embed train 128K tokens", "train", "bf16", 131072, 768, 30522, "zipf", 0.05),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["head", "head", "distill", "embed"])
    if op == "head":
        most = 4096 * 1280 * 50257
        while True:
            rows, hidden, vocab = _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 256), _log_int(rng, 200, 131072)
            if rows * hidden * vocab <= most and hidden * vocab <= 1280 * 65536:
                break
        c = _head("", rng.choice(["score", "train", "train"]), rng.choice(["f16", "bf16"]), rows, hidden, vocab,
                  rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 0.1, 0.5]))
    elif op == "distill":
        while True:
            rows, vocab = _log_int(rng, 1, 8192), 8 * _log_int(rng, 64, 16384)
            dtype = rng.choice(["f16", "bf16", "f32"])
            if rows * vocab * (2 if dtype == "f32" else 1) <= 2047 * 131072:
                break
        c = _distill("", rng.choice(["loss", "train", "train"]), dtype, rows, vocab, _log_int(rng, 1, 256),
                     rng.choice([1.0, 2.0, 4.0]), rng.random() < 0.5)
    else:
        while True:
            tokens, hidden, vocab = _log_int(rng, 1, 131072), 8 * _log_int(rng, 8, 512), _log_int(rng, 200, 131072)
            dtype = rng.choice(["f16", "bf16", "f32"])
            if tokens * hidden * (2 if dtype == "f32" else 1) <= 131072 * 768 and hidden * vocab <= 1280 * 50257:
                break
        c = _embed("", rng.choice(["lookup", "train", "train"]), dtype, tokens, hidden, vocab,
                   rng.choice(["zipf", "uniform"]), rng.choice([0.0, 0.1]))
    del c["name"]
    return c


# --- inputs -------------------------------------------------------------------
def _ids(gen, n, vocab, kind):
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    # zipf: P(id) about 1 / (id + 1), so log(id + 1) is uniform
    ids = torch.exp(u * math.log(vocab + 1.0)) - 1.0 if kind == "zipf" else u * vocab
    return ids.long().clamp_(0, vocab - 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(t)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "head":
        rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
        # normalised hidden states, and a weight that gives logits of a standard deviation of about 2.5
        s["x"] = normal(rows, hidden)
        s["weight"] = normal(vocab, hidden, std=2.5 / math.sqrt(hidden))
        target = _ids(gen, rows, vocab, "zipf")
        s["target"] = torch.where(uniform(rows) < case["ignored"], torch.full_like(target, _IGNORE), target)
        # the mean over the rows, with a loss scale where the storage type needs one
        s["dloss"] = torch.full((rows,), (4096.0 if t == torch.float16 else 1.0) / rows, device="cuda")
    elif case["op"] == "distill":
        rows, vocab, k = case["rows"], case["vocab"], case["k"]
        s["logits"] = normal(rows, vocab, std=2.0)
        index = (uniform(rows, k) * vocab).to(torch.int32).clamp_(0, vocab - 1)
        # some rows have fewer entries, some have none: their places hold -1
        width = torch.where(uniform(rows, 1) < 0.1, uniform(rows, 1) * k, torch.full((rows, 1), float(k), device="cuda"))
        there = torch.arange(k, device="cuda")[None, :] < width.long()
        s["index"] = torch.where(there, index, torch.full_like(index, -1))
        rank = torch.arange(k, device="cuda", dtype=torch.float32)
        teacher = 9.0 - 1.5 * torch.log1p(rank)[None, :] + 0.3 * torch.randn(rows, k, generator=gen, device="cuda")
        s["teacher"] = teacher.to(t)
        s["teacher_lse"] = None
        if case["tail"]:  # the top entries hold 60 to 100 % of the teacher's mass
            scaled = s["teacher"].float() / case["temperature"]
            top = torch.log(torch.exp(torch.where(there, scaled, torch.full_like(scaled, -math.inf))).sum(1))
            top = torch.where(there.any(1), top, torch.zeros_like(top))
            s["teacher_lse"] = top - torch.log(0.6 + 0.4 * uniform(rows))
        s["dloss"] = torch.full((rows,), (4096.0 if t == torch.float16 else 1.0) / rows, device="cuda")
    else:
        tokens, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
        s["table"] = normal(vocab, hidden, std=0.02)
        ids = _ids(gen, tokens, vocab, case["ids"])
        s["tokens"] = torch.where(uniform(tokens) < case["padded"], torch.zeros_like(ids), ids)  # id 0 pads
        s["scale"] = math.sqrt(hidden)
        s["dy"] = normal(tokens, hidden) if case["mode"] == "train" else None
    return s


# --- the calls of the framework -------------------------------------------------
def _new(like, *shape, dtype=None):
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def _own_head(s, c):
    from transformer_layer_non_gb300 import ls_vocab

    x, w = s["x"], s["weight"]
    if "workspace" not in s:  # what a program keeps from step to step
        s["workspace"] = ls_vocab.new_workspace(
            ls_vocab.linear_cross_entropy_workspace_bytes(c["rows"], c["hidden"], c["vocab"]))
        s["loss"], s["lse"] = (_new(x, c["rows"], dtype=torch.float32) for _ in range(2))
        if c["mode"] == "train":
            s["dx"], s["dweight"] = torch.empty_like(x), torch.empty_like(w)
    ls_vocab.ls_linear_cross_entropy_fwd(s["loss"], s["lse"], x, w, s["target"], c["smoothing"], _IGNORE,
                                         workspace=s["workspace"])
    if c["mode"] == "score":
        return {"loss": s["loss"], "lse": s["lse"]}
    ls_vocab.ls_linear_cross_entropy_bwd(s["dx"], s["dweight"], x, w, s["target"], s["lse"], s["dloss"],
                                         c["smoothing"], _IGNORE, workspace=s["workspace"])
    return {"loss": s["loss"], "lse": s["lse"], "dx": s["dx"], "dweight": s["dweight"]}


def _own_distill(s, c):
    from transformer_layer_non_gb300 import ls_vocab

    z = s["logits"]
    if "loss" not in s:
        s["loss"], s["lse"] = (_new(z, c["rows"], dtype=torch.float32) for _ in range(2))
        if c["mode"] == "train":
            s["dlogits"] = torch.empty_like(z)
    ls_vocab.ls_distill_topk_fwd(s["loss"], s["lse"], z, s["index"], s["teacher"], s["teacher_lse"],
                                 c["temperature"])
    if c["mode"] == "loss":
        return {"loss": s["loss"], "lse": s["lse"]}
    ls_vocab.ls_distill_topk_bwd(s["dlogits"], z, s["index"], s["teacher"], s["lse"], s["teacher_lse"],
                                 s["dloss"], c["temperature"])
    return {"loss": s["loss"], "lse": s["lse"], "dlogits": s["dlogits"]}


def _own_embed(s, c):
    from transformer_layer_non_gb300 import ls_vocab

    if "y" not in s:
        s["y"] = _new(s["table"], c["tokens"], c["hidden"])
        if c["mode"] == "train":
            s["dtable"] = _new(s["table"], c["vocab"], c["hidden"], dtype=torch.float32)
            s["workspace"] = ls_vocab.new_workspace(
                ls_vocab.embedding_lookup_workspace_bytes(c["tokens"], c["hidden"], c["vocab"]))
    ls_vocab.ls_embedding_lookup_fwd(s["y"], s["tokens"], s["table"], s["scale"])
    if c["mode"] == "lookup":
        return {"y": s["y"]}
    ls_vocab.ls_embedding_lookup_bwd(s["dtable"], s["dy"], s["tokens"], s["scale"], padding_id=0,
                                     accumulate=False, workspace=s["workspace"])
    return {"y": s["y"], "dtable": s["dtable"]}


# --- the plain forms ------------------------------------------------------------
def _plain_head(s, c):
    x, w, target = s["x"].float(), s["weight"].float(), s["target"].long()
    eps = c["smoothing"]
    used = target != _IGNORE
    at = torch.where(used, target, torch.zeros_like(target))[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = (1.0 - eps) * (lse - z.gather(1, at)) + eps * (lse - z.mean(1, keepdim=True))
    loss = torch.where(used, loss[:, 0], torch.zeros_like(lse[:, 0]))
    out = {"loss": loss, "lse": lse[:, 0]}
    if c["mode"] == "train":
        g = torch.exp(z - lse) - eps / c["vocab"]
        g.scatter_add_(1, at, torch.full_like(lse, eps - 1.0))
        g *= (s["dloss"] * used)[:, None]
        out["dx"] = (g @ w).to(s["x"].dtype)
        out["dweight"] = (g.t() @ x).to(s["weight"].dtype)
    return out


def _plain_distill(s, c):
    tau = c["temperature"]
    z, t, index = s["logits"].float() / tau, s["teacher"].float() / tau, s["index"].long()
    there = (index >= 0) & (index < c["vocab"])
    index = torch.where(there, index, torch.zeros_like(index))
    t = torch.where(there, t, torch.full_like(t, -math.inf))
    some = there.any(1, keepdim=True)
    if s["teacher_lse"] is None:
        top = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(t[:, :1]))
        total = torch.where(some, torch.exp(t - top).sum(1, keepdim=True), torch.ones_like(top))
        logq = t - top - torch.log(total)
    else:
        logq = t - s["teacher_lse"][:, None]
    q = torch.exp(logq)
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    each = torch.where(there, q * (logq - (z.gather(1, index) - lse)), torch.zeros_like(q))
    out = {"loss": tau * tau * each.sum(1), "lse": lse[:, 0]}
    if c["mode"] == "train":
        d = torch.exp(z - lse) * q.sum(1, keepdim=True)
        d.scatter_add_(1, index, -q)
        d *= tau * s["dloss"][:, None]
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_embed(s, c):
    tokens = s["tokens"].long()
    out = {"y": (s["table"][tokens].float() * s["scale"]).to(s["table"].dtype)}
    if c["mode"] == "train":
        g = torch.where((tokens == 0)[:, None], torch.zeros_like(s["dy"]), s["dy"]).float() * s["scale"]
        dtable = torch.zeros(c["vocab"], c["hidden"], device=g.device)
        dtable.index_add_(0, tokens, g)
        out["dtable"] = dtable
    return out


def run(state):
    c = state["case"]
    if own:
        return {"head": _own_head, "distill": _own_distill, "embed": _own_embed}[c["op"]](state, c)
    return {"head": _plain_head, "distill": _plain_distill, "embed": _plain_embed}[c["op"]](state, c)


# --- what a pass cannot do without ------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    train = case["mode"] == "train"
    if case["op"] == "head":
        rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
        data = (rows + vocab) * hidden * size
        # read x, weight and targets, write loss and lse; a step reads the rows' gradients and writes dx and dweight.
        # One product for the logits, two more for the gradients.
        return {"bytes": data * (2 if train else 1) + rows * (16 if train else 12),
                "flops": 2.0 * rows * hidden * vocab * (3 if train else 1)}
    if case["op"] == "distill":
        rows, vocab, k = case["rows"], case["vocab"], case["k"]
        logits = rows * vocab * size
        few = rows * (k * (4 + size) + 8 + (4 if case["tail"] else 0) + (4 if train else 0))
        return {"bytes": logits * (2 if train else 1) + few, "flops": 4.0 * rows * vocab * (2 if train else 1)}
    tokens, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
    # the rows of the table that are read: at most one for each token
    rows = min(tokens, vocab)
    n = tokens * 4 + rows * hidden * size + tokens * hidden * size
    if train:
        n += tokens * hidden * size + vocab * hidden * 4
    return {"bytes": n, "flops": float(tokens * hidden * (2 if train else 1))}


# --- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "head":
        rows, vocab, eps = case["rows"], case["vocab"], case["smoothing"]
        x, w = s["x"].double(), s["weight"].double()
        used = (s["target"] != _IGNORE).double()
        # the distribution that the loss compares with: the smoothed one-hot vector of each row
        wanted = torch.full((rows, vocab), eps / vocab, dtype=torch.float64, device="cuda")
        row = torch.arange(rows, device="cuda")
        wanted[row, s["target"].clamp(min=0).long()] += 1.0 - eps
        logp = torch.mm(x, w.T)
        lse = torch.logsumexp(logp, 1)
        logp -= lse[:, None]
        out = {"loss": -(wanted * logp).sum(1) * used, "lse": lse}
        if case["mode"] == "train":
            diff = logp.exp_().sub_(wanted).mul_((used * s["dloss"].double())[:, None])
            out["dx"], out["dweight"] = torch.mm(diff, w), torch.mm(diff.T, x)
        return out
    if case["op"] == "distill":
        rows, vocab, tau = case["rows"], case["vocab"], case["temperature"]
        logp = torch.log_softmax(s["logits"].double() / tau, 1)
        lse = torch.logsumexp(s["logits"].double() / tau, 1)
        valid = s["index"] >= 0
        t = (s["teacher"].double() / tau).masked_fill(~valid, -1e300)
        base = torch.logsumexp(t, 1) if s["teacher_lse"] is None else s["teacher_lse"].double()
        logq = t - base[:, None]
        q = logq.exp() * valid
        dense = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
        dense.scatter_add_(1, s["index"].clamp(min=0).long(), q)
        entropy = (q * logq.masked_fill(~valid, 0.0)).sum(1)
        out = {"loss": tau * tau * (entropy - (dense * logp).sum(1)), "lse": lse}
        if case["mode"] == "train":
            share = dense.sum(1, keepdim=True)
            out["dlogits"] = (logp.exp_() * share - dense) * (tau * s["dloss"].double())[:, None]
        return out
    out = {"y": s["table"].double()[s["tokens"].long()] * s["scale"]}
    if case["mode"] == "train":
        # the tokens in the order of their ids, and differences of running sums at the ids' borders
        order = torch.argsort(s["tokens"].long(), stable=True)
        ids = s["tokens"].long()[order]
        total = torch.zeros(case["tokens"] + 1, case["hidden"], dtype=torch.float64, device="cuda")
        total[1:] = torch.cumsum(s["dy"].double()[order] * s["scale"], 0)
        border = torch.searchsorted(ids, torch.arange(case["vocab"] + 1, device="cuda"))
        d = total[border[1:]] - total[border[:-1]]
        d[0] = 0.0
        out["dtable"] = d
    return out
