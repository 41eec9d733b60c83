"""Plain 64-bit implementations of the vocabulary operators and, for each
output, a bound on what FP32 arithmetic and one rounding to the storage type
may add.  Everything is torch float64 on the inputs' device.

Roundings: half a step of the storage type, u16 = eps/2 (2^-8 BF16, 2^-11
FP16, 2^-24 FP32); an FP32 sum of n terms in any order is off by at most
n * 2^-24 of the sum of their magnitudes, and tensor cores, which may drop
low bits instead of rounding, by twice that.  exp2 of the hardware is good to
2^-22, and its argument, an FP32 product of up to 2^7 in magnitude for terms
that matter, to 2^-17 of an exponent bit (ARG): terms further down than that
are below 2^-128 of the sum.
"""
import torch

U32 = 2.0 ** -24
ARG = 2.0 ** -17
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -126,
        torch.float64: 0.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        at = torch.argmax(torch.where(bad, err / bound, torch.zeros_like(err)))
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds; worst at {int(at)}: "
            f"got {got.flatten()[at]!r} ref {ref.flatten()[at]!r} "
            f"bound {(bound + 0 * err).flatten()[at]!r}")


def linear_cross_entropy(x, w, target, eps=0.0, ignore=-100, dloss=None, wtype=None):
    """(values, bounds) of loss, lse, dx, dweight."""
    t = x.dtype
    u = half_step(t)
    x, w = x.double(), w.double()
    rows, hidden = x.shape
    vocab = w.shape[0]
    y = target.long()
    used = (y != ignore) & (y >= 0) & (y < vocab)
    z = x @ w.T
    zb = (hidden * 2 * U32) * (x.abs() @ w.abs().T) + U32 * z.abs()
    lse = torch.logsumexp(z, 1)
    row = torch.arange(rows, device=x.device)
    want = torch.full_like(z, eps / vocab)
    want[row[used], y[used]] += 1 - eps
    loss = torch.where(used, lse - (want * z).sum(1), torch.zeros_like(lse))
    p = torch.exp(z - lse[:, None])
    lseb = (p * zb).sum(1) + vocab * U32 + 2.0 ** -22 + ARG + 4 * U32 * lse.abs()
    lossb = lseb + (want * zb).sum(1) + vocab * U32 * eps * z.abs().mean(1) + 8 * U32 * (
        lse.abs() + (want * z.abs()).sum(1))
    d = torch.ones(rows, dtype=torch.float64, device=x.device) if dloss is None else dloss.double()
    d = d * used
    g = d[:, None] * (p - want)
    # p's own error, then one rounding of g; FP16 keeps g down to 2^-39 of the largest dloss
    gb = d.abs()[:, None] * (p * (zb + lseb[:, None] + 2.0 ** -22 + ARG) + 4 * U32 * (p + want))
    gb = gb + u * g.abs() + (d.abs().max() * 2.0 ** -38 if t == torch.float16 else 0.0)
    dx, dw = g @ w, g.T @ x
    dxb = gb @ w.abs() + (vocab * 2 * U32) * (g.abs() @ w.abs()) + 2 * u * dx.abs() + TINY[t]
    wt = wtype or t
    dwb = gb.T @ x.abs() + (rows * 2 * U32) * (g.abs().T @ x.abs()) + 2 * half_step(wt) * dw.abs() + TINY[wt]
    return (loss, lse, dx, dw), (lossb * used, lseb, dxb, dwb)


def distill(z, index, teacher, teacher_lse=None, tau=1.0, dloss=None):
    """(values, bounds) of loss, lse, dlogits."""
    t = z.dtype
    rows, vocab = z.shape
    k = index.shape[1]
    zs, ts = z.double() / tau, teacher.double() / tau
    there = (index >= 0) & (index < vocab)
    at = torch.where(there, index, torch.zeros_like(index)).long()
    ts = torch.where(there, ts, torch.full_like(ts, -float("inf")))
    some = (ts > -float("inf")).any(1)
    if teacher_lse is None:
        base = torch.where(some, torch.logsumexp(ts, 1), torch.zeros_like(ts[:, 0]))
    else:
        base = teacher_lse.double()
    logq = ts - base[:, None]
    q = torch.exp(logq)
    lse = torch.logsumexp(zs, 1)
    logp = zs.gather(1, at) - lse[:, None]
    live = there & (q > 0)
    zero = torch.zeros_like(q)
    loss = tau * tau * torch.where(live, q * (logq - logp), zero).sum(1)
    lseb = vocab * U32 + 2.0 ** -22 + ARG + 8 * U32 * (lse.abs() + zs.amax(1).abs())
    # q: exp of an argument rounded a few times; base: a sum of k terms
    qrel = (k + 16) * U32 + 8 * U32 * torch.where(live, ts.abs() + base.abs()[:, None], zero)
    size = torch.where(live, logq.abs() + logp.abs(), zero)
    lossb = tau * tau * torch.where(live, q * (size * (qrel + (k + 16) * U32) + qrel
                                               + lseb[:, None] + 8 * U32 * zs.gather(1, at).abs()),
                                    zero).sum(1)
    d = torch.ones(rows, dtype=torch.float64, device=z.device) if dloss is None else dloss.double()
    Q = torch.where(live, q, zero).sum(1)
    p = torch.exp(zs - lse[:, None])
    dense = torch.zeros_like(p).scatter_add_(1, at, torch.where(live, q, zero))
    denseb = torch.zeros_like(p).scatter_add_(1, at, torch.where(live, q * (qrel + k * U32), zero))
    Qb = (torch.where(live, q * qrel, zero)).sum(1) + k * U32 * Q
    c = (tau * d)[:, None]
    dz = c * (Q[:, None] * p - dense)
    dzb = c.abs() * (p * (Q * (lseb + 2.0 ** -22 + ARG + 8 * U32) + Qb)[:, None] + denseb
                     + 8 * U32 * (Q[:, None] * p + dense)) + half_step(t) * dz.abs() + TINY[t]
    # the hardware's exp2 flushes results below 2^-126 to zero
    dzb = dzb + c.abs() * Q[:, None] * 2.0 ** -126
    dz, dzb = dz * (Q > 0)[:, None], torch.where((Q > 0)[:, None], dzb, torch.zeros_like(dzb))
    return (loss, lse, dz), (lossb, lseb, dzb)


def embedding_lookup(table, tokens, scale, dy=None, padding_id=-1, start=None):
    """(values, bounds) of y and, with dy, of the table's gradient."""
    vocab, hidden = table.shape
    there = (tokens >= 0) & (tokens < vocab)
    at = torch.where(there, tokens, torch.zeros_like(tokens)).long()
    y = table.double()[at] * scale * there[:, None]
    yb = (half_step(table.dtype) + 2 * U32) * y.abs() + TINY[table.dtype]
    if dy is None:
        return (y,), (yb,)
    add = there & (tokens != padding_id)
    g = dy.double() * add[:, None]
    total = torch.zeros(vocab, hidden, dtype=torch.float64, device=dy.device)
    size, count = total.clone(), total[:, 0].clone()
    total.index_add_(0, at, g)
    size.index_add_(0, at, g.abs())
    count.index_add_(0, at, add.double())
    d = total * scale
    db = abs(scale) * size * (count[:, None] + 4) * U32
    if start is not None:
        d = d + start.double()
        db = db + 2 * U32 * (start.double().abs() + d.abs())
    return (y, d), (yb, db)
