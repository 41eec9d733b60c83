"""Cases of the decoder block's operators: what a training step or a decoding step of a gated decoder runs between its
matrix products, and between its backward pass and its update.

  rotary  rotary positions of queries and keys: interleaved or half layout, part of the head, scaled for long contexts
  norm    norms of queries and keys for each head with the rotation in the same pass, and the weights' gradients
  gated   the gated feed-forward block: both projections, the activation and the product, and its gradients
  clip    the global norm of many gradients, and the clipped gradients; or the Adam update with them

``run`` computes them in a plain form, or, where ``own`` is true, by the calls of ``ls_block``.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_ADAM = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8, "weight_decay": 0.1, "step": 7}


# --- cases --------------------------------------------------------------------
def _heads(name, op, mode, dtype, batch, seq, heads, kv_heads, head_dim, rotary_dim, interleaved, packed, base=10000.0,
           scaling="none", factor=1.0, original=0, first=0, given=False):
    """given: the positions come as an array; packed: queries and keys lie in the rows of one projection, with the values
    behind them, and not head by head."""
    return {"name": name, "op": op, "mode": mode, "dtype": dtype, "batch": batch, "seq": seq, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "packed": packed, "base": base, "scaling": scaling, "factor": factor, "original": original, "first": first,
            "given": given}


def _gated(name, mode, dtype, rows, hidden, ffn, activation):
    return {"name": name, "op": "gated", "mode": mode, "dtype": dtype, "rows": rows, "hidden": hidden, "ffn": ffn,
            "activation": activation}


def _clip(name, mode, dtype, layers, hidden, vocab, aligned, max_norm=1.0, loss_scale=1.0):
    return {"name": name, "op": "clip", "mode": mode, "dtype": dtype, "layers": layers, "hidden": hidden, "vocab": vocab,
            "aligned": aligned, "max_norm": max_norm, "loss_scale": loss_scale}


def listed():
    return [
        # One decoding step of 32 sequences, each at a position of its own, queries and keys in the projection's rows.
        _heads("rotary decode 32", "rotary", "forward", "bf16", 32, 1, 20, 20, 64, 64, False, True, given=True),
        # A GPT-2-large training step (4 x 1024 tokens), head by head as the reshape of Q, K and V leaves them.
        _heads("rotary train GPT-2-large", "rotary", "train", "f16", 4, 1024, 20, 20, 64, 64, True, False),
        # The far end of a long context, its frequencies scaled by parts; half of each head is rotated, keys are shared.
        _heads("rotary long context", "rotary", "forward", "bf16", 1, 16411, 32, 8, 128, 64, False, True, 500000.0, "yarn",
               16.0, 8192, 114000),
        # A single token of one sequence: nothing but latency.
        _heads("norm decode 1", "norm", "forward", "f32", 1, 1, 16, 4, 80, 80, False, True, first=4099),
        # A BERT-base training step (8 x 512 tokens).
        _heads("norm train BERT-base", "norm", "train", "f16", 8, 512, 12, 12, 64, 64, True, False),
        # A training step with shared keys and wide heads, a ragged length.
        _heads("norm train wide", "norm", "train", "bf16", 3, 2733, 32, 8, 128, 128, False, True, 1000000.0, given=True),
        # One token through a GPT-2-large block: the weights are read once, nothing else counts.
        _gated("gated decode 1 token", "forward", "bf16", 1, 1280, 5120, "silu"),
        # A ragged batch through a Transformer-base block.
        _gated("gated 333 rows", "forward", "f16", 333, 512, 2048, "gelu_tanh"),
        # A GPT-2-large training step (4 x 1024 tokens).
        _gated("gated train GPT-2-large", "train", "bf16", 4096, 1280, 5120, "silu"),
        # A small model's gradients, FP32, the tensors one behind the other without padding.
        _clip("clip small", "clip", "f32", 2, 264, 1001, False),
        # All gradients of a GPT-2-large, clipped before an optimiser of the program's own.
        _clip("clip GPT-2-large", "clip", "bf16", 36, 1280, 50257, True),
        # A BERT-base step: unscaled, clipped and updated.
        _clip("clip update BERT-base", "update", "f16", 12, 768, 30522, True, 1.0, 1024.0),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "gated", "gated", "clip"])
    if op in ("rotary", "norm"):
        while True:
            batch, seq = _log_int(rng, 1, 64), _log_int(rng, 1, 16384)
            kv = _log_int(rng, 1, 16)
            heads, dim = kv * rng.choice([1, 1, 2, 4, 8]), 8 * _log_int(rng, 2, 32)
            dtype = rng.choice(["f16", "bf16", "f32"])
            if batch * seq * (heads + 2 * kv) * dim <= 8 << 24:
                break
        rotary = rng.choice([dim, dim, max(2, dim // 2), 2 * rng.randint(1, dim // 2)])
        scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
        c = _heads("", op, rng.choice(["forward", "train"]), dtype, batch, seq, heads, kv, dim, rotary, rng.random() < 0.5,
                   rng.random() < 0.5, rng.choice([10000.0, 500000.0]), scaling,
                   1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]), 4096 if scaling == "yarn" else 0,
                   _log_int(rng, 1, 1000000) - 1, rng.random() < 0.5)
    elif op == "gated":
        while True:
            rows, hidden, ffn = _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 512), 8 * _log_int(rng, 16, 1792)
            if rows * hidden * ffn <= 4096 * 1280 * 5120 and hidden * ffn <= 4096 * 14336 // 2:
                break
        c = _gated("", rng.choice(["forward", "train"]), rng.choice(["f16", "bf16"]), rows, hidden, ffn,
                   rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))
    else:
        mode = rng.choice(["clip", "update"])
        while True:
            layers, hidden, vocab = _log_int(rng, 1, 40), _log_int(rng, 33, 1536), _log_int(rng, 100, 65536)
            if layers * 16 * hidden * hidden + hidden * vocab <= (300 << 20 if mode == "clip" else 100 << 20):
                break
        c = _clip("", mode, rng.choice(["f16", "bf16", "f32"]), layers, hidden, vocab, rng.random() < 0.5,
                  rng.choice([0.5, 1.0, 1e9]), rng.choice([1.0, 1024.0]))
    del c["name"]
    return c


# --- inputs -------------------------------------------------------------------
def _frequencies(c):
    """Radians for each step of the position, in 64 bits, and the factor on cosines and sines."""
    rd = c["rotary_dim"]
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda") * 2.0 / rd
    if c["scaling"] == "ntk":  # the base raised so that the slowest pair is slowed by the factor
        return (c["base"] * c["factor"] ** (rd / max(rd - 2.0, 1.0))) ** -i, 1.0
    w = c["base"] ** -i
    if c["scaling"] == "linear":
        return w / c["factor"], 1.0
    if c["scaling"] == "yarn":
        # pairs that turn fewer than once in the original context are slowed by the factor, those that turn more
        # than 32 times are left, the others lie between, linearly in the pair's number
        def number(turns):
            return rd * math.log(c["original"] / (2.0 * math.pi * turns)) / (2.0 * math.log(c["base"]))

        low, high = max(math.floor(number(32.0)), 0), min(math.ceil(number(1.0)), rd - 1)
        slow = ((torch.arange(rd // 2, dtype=torch.float64, device="cuda") - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return w * (1.0 - slow) + w / c["factor"] * slow, 0.1 * math.log(c["factor"]) + 1.0
    return w, 1.0


def _tensor_sizes(c):
    """Elements of the gradients of a gated decoder: the embedding, and for each layer its products and norms."""
    h = c["hidden"]
    layer = [h, 3 * h * h, h * h, h, 4 * h * h, 4 * h * h, 4 * h * h]
    return [c["vocab"] * h] + layer * c["layers"] + [h]


def _offsets(c):
    """Where each tensor begins in the flat buffer, and the buffer's length."""
    step = 8 if c["aligned"] else 1
    at = [0]
    for n in _tensor_sizes(c):
        at.append(at[-1] + (n + step - 1) // step * step)
    return at


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(t)

    s = {"case": dict(case)}
    if case["op"] in ("rotary", "norm"):
        batch, seq, heads, kv, dim = (case[k] for k in ("batch", "seq", "heads", "kv_heads", "head_dim"))
        if case["packed"]:  # [batch, seq, heads, head_dim], as the projection of Q, K and V leaves them
            rows = normal(batch, seq, heads + 2 * kv, dim)
            s["q"], s["k"] = rows[:, :, :heads], rows[:, :, heads:heads + kv]
        else:
            s["q"], s["k"] = normal(batch, heads, seq, dim).transpose(1, 2), normal(batch, kv, seq, dim).transpose(1, 2)
        s["positions"] = None
        if case["given"]:  # sequences that begin at different places, as left-padded or continued ones do
            start = (torch.rand(batch, 1, generator=gen, device="cuda") * 5000).int() + case["first"]
            s["positions"] = (start + torch.arange(seq, device="cuda", dtype=torch.int32)).to(torch.int32)
        if case["op"] == "norm":
            s["wq"], s["wk"] = ((1.0 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(t) for _ in range(2))
        if case["mode"] == "train":  # the gradients come head by head, from the attention
            s["gq"], s["gk"] = normal(batch, heads, seq, dim), normal(batch, kv, seq, dim)
    elif case["op"] == "gated":
        rows, hidden, ffn = case["rows"], case["hidden"], case["ffn"]
        s["x"] = normal(rows, hidden)
        s["wg"], s["wu"] = (normal(ffn, hidden, std=1.0 / math.sqrt(hidden)) for _ in range(2))
        if case["mode"] == "train":
            s["dh"] = normal(rows, ffn)
    else:
        at, sizes = _offsets(case), _tensor_sizes(case)
        # gradients of a norm of about 3, times the loss scale
        std = case["loss_scale"] * 3.0 / math.sqrt(sum(sizes))
        s["flat"] = normal(at[-1], std=std)
        for begin, n, end in zip(at, sizes, at[1:]):
            s["flat"][begin + n:end] = 0
        if case["mode"] == "update":
            s["param"] = normal(at[-1], std=0.02)
            s["m"] = torch.randn(at[-1], generator=gen, device="cuda").mul_(std / case["loss_scale"])
            s["v"] = torch.rand(at[-1], generator=gen, device="cuda").mul_((std / case["loss_scale"]) ** 2)
    return s


# --- the calls of the framework -------------------------------------------------
def _by_head(like, heads):
    """Memory [batch, heads, seq, head_dim], as attention reads it."""
    batch, seq, _, dim = like.shape
    return torch.empty(batch, heads, seq, dim, dtype=like.dtype, device=like.device)


def _own_heads(s, c):
    from transformer_layer_non_gb300 import ls_block

    if "rotation" not in s:  # what a program keeps from step to step
        s["rotation"] = ls_block.Rotation(c["rotary_dim"], base=c["base"], interleaved=c["interleaved"],
                                          scaling=c["scaling"], factor=c["factor"], original_positions=c["original"])
        s["yq"], s["yk"] = _by_head(s["q"], c["heads"]), _by_head(s["k"], c["kv_heads"])
        if c["mode"] == "train":
            if c["packed"]:  # the gradient of the projection's rows
                rows = torch.empty(c["batch"], c["seq"], c["heads"] + 2 * c["kv_heads"], c["head_dim"],
                                   dtype=s["q"].dtype, device="cuda")
                s["dq"], s["dk"] = rows[:, :, :c["heads"]], rows[:, :, c["heads"]:c["heads"] + c["kv_heads"]]
            else:
                s["dq"], s["dk"] = (_by_head(s["q"], n).transpose(1, 2) for n in (c["heads"], c["kv_heads"]))
            if c["op"] == "norm":
                s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
                s["workspace"] = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(c["head_dim"]))
    yq, yk = s["yq"].transpose(1, 2), s["yk"].transpose(1, 2)
    where = {"positions": s["positions"], "first_position": c["first"]}
    if c["op"] == "rotary":
        ls_block.ls_rotary_fwd(yq, yk, s["q"], s["k"], s["rotation"], **where)
    else:
        ls_block.ls_qk_norm_rotary_fwd(yq, yk, s["q"], s["k"], s["wq"], s["wk"], s["rotation"], eps=_EPS, **where)
    out = {"q": s["yq"], "k": s["yk"]}
    if c["mode"] == "forward":
        return out
    gq, gk = s["gq"].transpose(1, 2), s["gk"].transpose(1, 2)
    if c["op"] == "rotary":
        ls_block.ls_rotary_bwd(s["dq"], s["dk"], gq, gk, s["rotation"], **where)
        return {**out, "dq": s["dq"], "dk": s["dk"]}
    ls_block.ls_qk_norm_rotary_bwd(s["dq"], s["dk"], s["dwq"], s["dwk"], gq, gk, s["q"], s["k"], s["wq"], s["wk"],
                                   s["rotation"], eps=_EPS, workspace=s["workspace"], **where)
    return {**out, "dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}


def _own_gated(s, c):
    from transformer_layer_non_gb300 import ls_block

    x, wg, wu = s["x"], s["wg"], s["wu"]
    if "h" not in s:
        s["h"] = torch.empty(c["rows"], c["ffn"], dtype=x.dtype, device="cuda")
        if c["mode"] == "train":
            s["dx"], s["dwg"], s["dwu"] = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
            s["workspace"] = ls_block.new_workspace(
                ls_block.gated_linear_workspace_bytes(c["rows"], c["hidden"], c["ffn"]))
    ls_block.ls_gated_linear_fwd(s["h"], x, wg, wu, c["activation"])
    if c["mode"] == "forward":
        return {"h": s["h"]}
    ls_block.ls_gated_linear_bwd(s["dx"], s["dwg"], s["dwu"], s["dh"], x, wg, wu, c["activation"],
                                 workspace=s["workspace"])
    return {"h": s["h"], "dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}


def _own_clip(s, c):
    from transformer_layer_non_gb300 import ls_block

    if "grads" not in s:
        at, sizes = _offsets(c), _tensor_sizes(c)
        s["grads"] = ls_block.TensorList([s["flat"][b:b + n] for b, n in zip(at, sizes)])
        s["norm"], s["factor"] = (torch.empty(1, device="cuda") for _ in range(2))
        s["workspace"] = ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
        if c["mode"] == "clip":
            s["clipped"] = torch.zeros_like(s["flat"])
            s["outs"] = ls_block.TensorList([s["clipped"][b:b + n] for b, n in zip(at, sizes)])
    ls_block.ls_grad_norm(s["norm"], s["factor"], s["grads"], c["max_norm"], 1.0 / c["loss_scale"],
                          workspace=s["workspace"])
    if c["mode"] == "clip":
        ls_block.ls_scale_gradients(s["outs"], s["grads"], s["factor"])
        return {"norm": s["norm"], "clipped": s["clipped"]}
    ls_block.ls_adam_update_scaled(s["param"], s["flat"], s["m"], s["v"], s["factor"], **_ADAM)
    return {"norm": s["norm"], "param": s["param"], "m": s["m"], "v": s["v"]}


# --- the plain forms ------------------------------------------------------------
def _turn(x, cos, sin, c):
    """x [batch, seq, heads, head_dim] in 32 bits, rotated; cos and sin [batch or 1, seq, 1, pairs]."""
    rd = c["rotary_dim"]
    rotated, rest = x[..., :rd], x[..., rd:]
    if c["interleaved"]:
        a, b = rotated[..., 0::2], rotated[..., 1::2]
        rotated = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = rotated[..., :rd // 2], rotated[..., rd // 2:]
        rotated = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((rotated, rest), -1)


def _plain_heads(s, c):
    w, scale = _frequencies(c)
    at = s["positions"]
    if at is None:
        at = torch.arange(c["first"], c["first"] + c["seq"], device="cuda")[None]
    angle = (at.double()[..., None] * w)[:, :, None]
    cos, sin = (torch.cos(angle) * scale).float(), (torch.sin(angle) * scale).float()
    t, norm = s["q"].dtype, c["op"] == "norm"
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if norm:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
            u, weight = x * r, s["w" + name].float()
            x = u * weight
        out[name] = _turn(x, cos, sin, c).transpose(1, 2).to(t).contiguous()
        if c["mode"] == "train":
            g = _turn(s["g" + name].transpose(1, 2).float(), cos, -sin, c)
            if norm:
                out["dw" + name] = (g * u).sum((0, 1, 2)).to(t)
                g = g * weight
                g = (g - u * (g * u).mean(-1, keepdim=True)) * r
            out["d" + name] = g.to(t)
    return out


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "relu":
        there = (g > 0).to(g.dtype)
        return g * there, there
    if kind == "silu":
        e = torch.sigmoid(g)
        return g * e, e * (1.0 + g * (1.0 - e))
    if kind == "gelu":
        e = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * e, e + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    e = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + e), 0.5 * (1.0 + e) + 0.5 * g * (1.0 - e * e) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain_gated(s, c):
    t, x, wg, wu = s["x"].dtype, s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, slope = _act(g, c["activation"])
    out = {"h": (a * u).to(t)}
    if c["mode"] == "train":
        dh = s["dh"].float()
        dg, du = dh * u * slope, dh * a
        out["dx"] = (dg @ wg + du @ wu).to(t)
        out["dwg"], out["dwu"] = (dg.t() @ x).to(t), (du.t() @ x).to(t)
    return out


def _plain_clip(s, c):
    t, g = s["flat"].dtype, s["flat"].float()
    norm = (torch.sqrt((g * g).sum(dtype=torch.float64)) / c["loss_scale"]).float().reshape(1)
    factor = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0) / c["loss_scale"]
    if c["mode"] == "clip":
        return {"norm": norm, "clipped": (g * factor).to(t)}
    p, b1, b2 = _ADAM, _ADAM["beta1"], _ADAM["beta2"]
    g *= factor
    s["m"].mul_(b1).add_(g * (1.0 - b1))
    s["v"].mul_(b2).add_(g * g * (1.0 - b2))
    step = s["m"] / (1.0 - b1 ** p["step"]) / (torch.sqrt(s["v"] / (1.0 - b2 ** p["step"])) + p["eps"])
    s["param"].copy_((s["param"].float() * (1.0 - p["lr"] * p["weight_decay"]) - p["lr"] * step).to(t))
    return {"norm": norm, "param": s["param"], "m": s["m"], "v": s["v"]}


def run(state):
    c = state["case"]
    if own:
        return {"rotary": _own_heads, "norm": _own_heads, "gated": _own_gated, "clip": _own_clip}[c["op"]](state, c)
    return {"rotary": _plain_heads, "norm": _plain_heads, "gated": _plain_gated, "clip": _plain_clip}[c["op"]](state, c)


# --- what a pass cannot do without ------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("rotary", "norm"):
        n = case["batch"] * case["seq"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        passes = 2  # read and written by the forward; the backward reads the gradient, with the norm x too, and writes
        if case["mode"] == "train":
            passes += 3 if case["op"] == "norm" else 2
        return {"bytes": n * size * passes + (case["batch"] * case["seq"] * 4 if case["given"] else 0),
                "flops": float(n * (4 * passes if case["op"] == "norm" else 3 * passes))}
    if case["op"] == "gated":
        rows, hidden, ffn = case["rows"], case["hidden"], case["ffn"]
        # forward: x and both weights read, h written, two products; backward: those and dh read, their gradients
        # written, four products
        data = rows * hidden + 2 * hidden * ffn + rows * ffn
        train = case["mode"] == "train"
        return {"bytes": data * size * (3 if train else 1), "flops": 4.0 * rows * hidden * ffn * (3 if train else 1)}
    n = sum(_tensor_sizes(case))
    if case["mode"] == "clip":  # read for the norm, read and written
        return {"bytes": 3 * n * size + 8, "flops": 3.0 * n}
    return {"bytes": n * (4 * size + 16) + 8, "flops": 16.0 * n}


# --- the definitions in 64 bits ----------------------------------------------------
def _exact_heads(s, c):
    rd, dim = c["rotary_dim"], c["head_dim"]
    w, scale = _frequencies(c)
    at = torch.arange(c["seq"], device="cuda", dtype=torch.float64)[None] + c["first"]
    if s["positions"] is not None:
        at = s["positions"].double()
    # the rotation as multiplication of complex numbers
    unit = torch.polar(torch.full_like(at[..., None] * w, scale), at[..., None] * w)[:, :, None]
    order = torch.arange(rd, device="cuda")
    order = order.view(-1, 2) if c["interleaved"] else order.view(2, -1).t()
    first, second = order[:, 0], order[:, 1]

    def turned(x, by):
        y, z = x.clone(), torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if c["op"] == "norm":
            length = torch.sqrt(x.square().sum(-1, keepdim=True) / dim + _EPS)
            weight = s["w" + name].double()
            out[name] = turned(x / length * weight, unit).transpose(1, 2)
        else:
            out[name] = turned(x, unit).transpose(1, 2)
        if c["mode"] == "train":
            g = turned(s["g" + name].transpose(1, 2).double(), unit.conj())
            if c["op"] == "norm":
                out["dw" + name] = (g * x / length).flatten(0, 2).sum(0)
                g = g * weight
                g = g / length - x * (g * x).sum(-1, keepdim=True) / (dim * length ** 3)
            out["d" + name] = g
    return out


def _exact_gated(s, c):
    x = s["x"].double()
    gate, up = torch.mm(x, s["wg"].double().T), torch.mm(x, s["wu"].double().T)
    gate.requires_grad_(c["mode"] == "train")
    kind = c["activation"]
    value = (torch.relu(gate) if kind == "relu" else torch.nn.functional.silu(gate) if kind == "silu"
             else torch.nn.functional.gelu(gate, approximate="tanh" if kind == "gelu_tanh" else "none"))
    out = {"h": value.detach() * up}
    if c["mode"] == "train":
        dh = s["dh"].double()
        dg, = torch.autograd.grad(value, gate, dh * up)
        du = dh * value.detach()
        out["dx"] = torch.mm(dg, s["wg"].double()).addmm_(du, s["wu"].double())
        out["dwg"], out["dwu"] = torch.mm(dg.T, x), torch.mm(du.T, x)
    return out


def _exact_clip(s, c):
    g = s["flat"].double().div_(c["loss_scale"])
    norm = torch.linalg.vector_norm(g).reshape(1)
    g *= min(1.0, c["max_norm"] / (float(norm) + 1e-6))
    if c["mode"] == "clip":
        return {"norm": norm, "clipped": g}
    p, t = _ADAM, _ADAM["step"]
    m = torch.lerp(g, s["m"].double(), p["beta1"])
    v = torch.lerp(g.square(), s["v"].double(), p["beta2"])
    mean, spread = m / (1.0 - p["beta1"] ** t), (v / (1.0 - p["beta2"] ** t)).sqrt_()
    param = s["param"].double()
    return {"norm": norm, "param": param - p["lr"] * (p["weight_decay"] * param + mean / (spread + p["eps"])),
            "m": m, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_heads, "norm": _exact_heads, "gated": _exact_gated, "clip": _exact_clip}[case["op"]](s, case)
