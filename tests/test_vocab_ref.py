"""The 64-bit implementations of tests/vocab_ref.py against finite differences
and against torch's own losses, on the CPU."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402


def _differences(f, a, h=1e-5):
    out = torch.zeros_like(a)
    for i in range(a.numel()):
        b = a.clone().flatten()
        b[i] += h
        up = f(b.view_as(a))
        b[i] -= 2 * h
        out.view(-1)[i] = (up - f(b.view_as(a))) / (2 * h)
    return out


@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_linear_cross_entropy_reference(eps):
    torch.manual_seed(0)
    x, w = torch.randn(5, 8).double(), torch.randn(11, 8).double()
    target = torch.tensor([3, -100, 10, 0, 99], dtype=torch.int32)
    d = torch.rand(5).double()
    (loss, lse, dx, dw), _ = vocab_ref.linear_cross_entropy(x, w, target, eps, -100, d)

    def total(x, w):
        return (vocab_ref.linear_cross_entropy(x, w, target, eps)[0][0] * d).sum()

    assert torch.allclose(dx, _differences(lambda a: total(a, w), x), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda a: total(x, a), w), atol=1e-8)
    y = torch.tensor([3, -100, 10, 0, -100])
    want = torch.nn.functional.cross_entropy(x @ w.T, y, reduction="none", label_smoothing=eps)
    assert torch.allclose(loss, want, atol=1e-12)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_reference(tail):
    torch.manual_seed(1)
    z = torch.randn(4, 16).double()
    index = torch.tensor([[1, 5, 9], [2, 2, -1], [-1, -1, 77], [15, 0, 3]], dtype=torch.int32)
    teacher = torch.randn(4, 3).double()
    base = torch.logsumexp(teacher / 2, 1) + 0.3 if tail else None
    d = torch.rand(4).double()
    (loss, lse, dz), _ = vocab_ref.distill(z, index, teacher, base, 2.0, d)

    def total(z):
        return (vocab_ref.distill(z, index, teacher, base, 2.0)[0][0] * d).sum()

    assert torch.allclose(dz, _differences(total, z), atol=1e-8)
    assert loss[2] == 0 and (dz[2] == 0).all()
    if not tail:  # rows without repeats: torch's KL divergence against the dense teacher
        for r in (0, 3):
            q = torch.zeros(16).double()
            q[index[r].long()] = torch.softmax(teacher[r] / 2, 0)
            kl = torch.nn.functional.kl_div(torch.log_softmax(z[r] / 2, 0), q, reduction="sum")
            assert abs(float(loss[r] - 4 * kl)) < 1e-12


def test_embedding_lookup_reference():
    torch.manual_seed(2)
    table = torch.randn(7, 8).double()
    tokens = torch.tensor([1, 6, 1, -1, 9, 0, 1], dtype=torch.int32)
    dy = torch.randn(7, 8).double()
    (y, d), _ = vocab_ref.embedding_lookup(table.float(), tokens, 2.0, dy, padding_id=0)
    want = torch.zeros(7, 8).double()
    for i, t in enumerate(tokens.tolist()):
        if 0 < t < 7:
            want[t] += 2.0 * dy[i]
    assert torch.allclose(d, want)
    assert (y[3] == 0).all() and (y[4] == 0).all()
