"""64-bit definitions of the decoder block's operators for the tests, with a
bound for every output, derived from the storage types' half steps and the
lengths of the FP32 sums.  Nothing here is shared with the library."""
import numpy as np
import torch

U = 2.0 ** -24  # half a step of FP32


def half_step(dtype, ref):
    """The rounding of ref to dtype: half a step, and below the normal numbers half the smallest one."""
    smallest = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return torch.finfo(dtype).eps / 2 * ref.abs() + smallest


def check(got, ref, bound, what=""):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = int(torch.where(bad, (got - ref).abs() / bound, torch.zeros_like(ref)).nan_to_num(1e300).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.numel()} values out of bounds; worst at {i}: got "
                             f"{float(got.flatten()[i])!r} ref {float(ref.flatten()[i])!r} bound "
                             f"{float(bound.flatten()[i]):.3g}")


# --- rotation --------------------------------------------------------------------
def radians(rotary_dim, base=10000.0, scaling="none", factor=1.0, original=0):
    """The frequencies by their definitions, pair by pair."""
    out = []
    for i in range(rotary_dim // 2):
        b = base * factor ** (rotary_dim / max(rotary_dim - 2, 1)) if scaling == "ntk" else base
        w = b ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            def number(turns):
                return rotary_dim * np.log(original / (2 * np.pi * turns)) / (2 * np.log(base))

            low = max(np.floor(number(32.0)), 0)
            high = min(np.ceil(number(1.0)), rotary_dim - 1)
            slow = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            w = w * (1.0 - slow) + w / factor * slow
        out.append(float(w))
    return out


def cos_sin(w, positions):
    """cos and sin of w[i] * position, [..., pairs], the angle reduced in extended precision."""
    two_pi = 8 * np.arctan(np.longdouble(1))
    angle = np.multiply.outer(np.asarray(positions, dtype=np.longdouble), np.asarray(w, dtype=np.longdouble))
    angle = angle - two_pi * np.rint(angle / two_pi)
    return (torch.from_numpy(f(angle).astype(np.float64)) for f in (np.cos, np.sin))


def pairs(rotary_dim, interleaved):
    i = torch.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotate(x, cos, sin, interleaved, scale=1.0, transpose=False):
    """x [batch, seq, heads, dim] in 64 bits; cos and sin [batch or 1, seq, pairs].  Returns the rotation and the
    size of what each element is made of."""
    a, b = pairs(2 * cos.shape[-1], interleaved)
    c, s = cos[:, :, None].to(x.device), sin[:, :, None].to(x.device)
    s = -s if transpose else s
    y, size = x.clone(), x.abs()
    y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
    y[..., b] = scale * (x[..., a] * s + x[..., b] * c)
    size[..., a] = size[..., b] = abs(scale) * (x[..., a].abs() + x[..., b].abs())
    return y, size


def rotary_bound(ref, size, dtype):
    # cos and sin are off by 3 steps at most (the angle's rounding, sincospif, the scale), products and sum by 3 more
    return half_step(dtype, ref) + 8 * U * size


def norm_forward(x, w, eps, turn):
    """y, its bound's parts, and u, r for the backward; turn(x) -> rotation, size (identity without one)."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y, size = turn(x * r * w)
    return y, size, x * r, r


def norm_bound(ref, size, dtype):
    # mean of squares: a lane's 16 terms and 5 exchanges, halved by the root; rsqrt 4, products 3, the rotation 8
    return half_step(dtype, ref) + 28 * U * size


def norm_backward(x, dy, w, eps, turn_back):
    """dx, dweight, and bounds' parts: what their terms add up to."""
    dim = x.shape[-1]
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = x * r
    g, size = turn_back(dy)
    dx = r * (w * g - u * (w * g * u).mean(-1, keepdim=True))
    parts = r * (w.abs() * size + u.abs() * (w.abs() * size * u.abs()).sum(-1, keepdim=True) / dim)
    return dx, (g * u).sum((0, 1, 2)), parts, (size * u.abs()).sum((0, 1, 2))


def norm_dx_bound(ref, parts, dtype):
    return half_step(dtype, ref) + 64 * U * parts


def norm_dw_bound(ref, parts, rows, dtype):
    # each term is off by 28 steps; a lane adds at most rows / 1000 of them (more than 1000 groups work on many rows),
    # then come up to 64 groups, 10 CTAs of a slice and 32 slices
    return half_step(dtype, ref) + (160 + rows / 1000) * U * parts


# --- the gated block ---------------------------------------------------------------
def activation(g, kind):
    """act and its slope."""
    if kind == "relu":
        return torch.relu(g), (g > 0).double()
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-g / 2 ** 0.5)
        return g * phi, phi + g * torch.exp(-g * g / 2) / (2 * np.pi) ** 0.5
    k = (2 / np.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
