"""The two ways through the block operators' binding, the compiled one and the one
that looks closer, make the same calls and refuse the same arguments."""
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block, ls_ops  # noqa: E402

pytestmark = pytest.mark.gpu


def everything(dtype=torch.float16):
    """One call of each operator, most of them with all arguments; what they wrote."""
    gen = torch.Generator(device="cuda").manual_seed(5)

    def draw(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * 0.3).to(dtype)

    rows = draw(2, 9, 7, 32)
    q, k, gq, gk = rows[:, :, :4], rows[:, :, 4:6], draw(2, 9, 4, 32), draw(2, 9, 2, 32)
    wq, wk = draw(32), draw(32)
    ws = ls_block.new_workspace(max(ls_block.qk_norm_rotary_workspace_bytes(32),
                                    ls_block.gated_linear_workspace_bytes(40, 64, 136)))
    at = torch.arange(18, device="cuda", dtype=torch.int32)
    out = []
    for rot in (ls_block.Rotation(32, interleaved=True), ls_block.Rotation(16, scaling="linear", factor=2.0)):
        for where in ({}, {"first_position": 5}, {"positions": at}, {"positions": at.view(2, 9), "stream": None}):
            y = [torch.empty_like(t) for t in (gq, gk, gq, gk, gq, gk, gq, gk)]
            ls_block.ls_rotary_fwd(y[0], y[1], q, k, rot, **where)
            ls_block.ls_rotary_bwd(y[2], y[3], gq, gk, rot, **where)
            ls_block.ls_qk_norm_rotary_fwd(y[4], y[5], q, k, wq, None, rot, 1e-5, **where)
            dw = [torch.empty_like(wq), torch.empty_like(wk)]
            ls_block.ls_qk_norm_rotary_bwd(y[6], y[7], dw[0], dw[1], gq, gk, q, k, wq, wk, rot, workspace=ws, **where)
            out += y + dw
    one = torch.empty_like(gq)
    ls_block.ls_qk_norm_rotary_fwd(one, None, q, None, None, None)
    out.append(one)
    if dtype is not torch.float32:
        x, wg, wu, dh = draw(40, 64), draw(136, 64), draw(136, 64), draw(40, 136)
        for act in ls_block.ACTIVATIONS:
            h, dx, dw = torch.empty_like(dh), torch.empty_like(x), [torch.empty_like(wg), torch.empty_like(wu)]
            ls_block.ls_gated_linear_fwd(h, x, wg, wu, act)
            ls_block.ls_gated_linear_bwd(dx, dw[0], dw[1], dh, x, wg, wu, act, workspace=ws)
            more = [torch.ones(136, 64, device="cuda") for _ in range(2)]
            ls_block.ls_gated_linear_bwd(None, more[0], more[1], dh, x, wg, wu, act, workspace=ws)
            out += [h, dx, *dw, *more]
    grads = [draw(5, 7), draw(64), draw(0), draw(3, 2, 4)]
    norm, factor = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ls_block.ls_grad_norm(norm, factor, ls_block.TensorList(grads), 0.5, 0.25, workspace=ws)
    ls_block.ls_grad_norm(norm, None, grads, workspace=ws)
    scaled = [torch.empty_like(g) for g in grads]
    ls_block.ls_scale_gradients(ls_block.TensorList(scaled), ls_block.TensorList(grads), factor)
    ls_block.ls_scale_gradients(grads, grads, factor)
    p, g = draw(100), draw(100)
    m, v = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    ls_block.ls_adam_update_scaled(p, g, m, v, factor, 1e-2, step=3, weight_decay=0.1)
    torch.cuda.synchronize()
    return [*out, norm, factor, *scaled, *grads, p, m, v]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_both_ways_write_the_same(dtype, monkeypatch):
    require_gpu()
    everything(dtype)  # the first call loads the compiled half
    made = []
    compiled = ls_block._call
    assert not isinstance(compiled, (type(None), ls_block._Closer))

    class Counted:
        def __getattr__(self, name):
            def call(*args):
                made.append((name, getattr(compiled, name)(*args)))
                return made[-1][1]
            return call

    monkeypatch.setattr(ls_block, "_call", Counted())
    a = everything(dtype)
    # all but the lists that are no TensorList went the compiled way
    assert {name for name, status in made if status == 0} >= {
        "rotary_fwd", "rotary_bwd", "norm_fwd", "norm_bwd", "grad_norm", "scale_gradients", "adam"}
    assert sorted(name for name, status in made if status != 0) == ["grad_norm", "scale_gradients"]
    monkeypatch.setattr(ls_block, "_call", ls_block._Closer())
    b = everything(dtype)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def refused():
    x = torch.zeros(2, 3, 4, 64, device="cuda").half()
    y, rot, w = torch.empty_like(x), ls_block.Rotation(64), torch.ones(64, device="cuda").half()
    f = torch.ones(1, device="cuda")
    m, g = torch.zeros(40, 64, device="cuda").half(), torch.zeros(72, 64, device="cuda").half()
    h = torch.empty(40, 72, device="cuda").half()
    p, s = torch.zeros(50, device="cuda").half(), torch.zeros(50, device="cuda")
    rotate, norm, gated = ls_block.ls_rotary_fwd, ls_block.ls_qk_norm_rotary_fwd, ls_block.ls_gated_linear_fwd
    lists = ls_block.TensorList([m])
    return [
        (TypeError, lambda: rotate(None, None, None, None, rot)), (TypeError, lambda: rotate(y, None, 3, None, rot)),
        (TypeError, lambda: rotate(y.float(), None, x, None, rot)), (ValueError, lambda: rotate(y.cpu(), None, x, None, rot)),
        (ValueError, lambda: rotate(y[:1], None, x, None, rot)), (ValueError, lambda: rotate(y[..., :32], None, x, None, rot)),
        (ValueError, lambda: rotate(y.transpose(2, 3), None, x.transpose(2, 3), None, rot)),
        (ValueError, lambda: rotate(y, None, x, None, ls_block.Rotation(64, device="cpu"))),
        (TypeError, lambda: rotate(y, None, x, None, rot, positions=torch.zeros(2, 3, device="cuda"))),
        (ValueError, lambda: rotate(y, None, x, None, rot, positions=torch.zeros(7, device="cuda", dtype=torch.int32))),
        (TypeError, lambda: rotate(y, None, x, None, rot, positions=[0, 1])),
        (ValueError, lambda: rotate(y, None, x, None, rot, first_position=2 ** 63)),
        (ls_ops.LsError, lambda: rotate(y, None, x, None, rot, first_position=2 ** 31 - 1)),
        (ls_ops.LsError, lambda: rotate(None, None, x, None, rot)), (ls_ops.LsError, lambda: rotate(y, y, x, None, rot)),
        (ls_ops.LsError, lambda: rotate(y[:, :, :3], None, x, None, rot)),
        (TypeError, lambda: rotate(y.int(), None, x.int(), None, rot)),
        (TypeError, lambda: norm(y, None, x, None, w.float(), None, rot)),
        (ValueError, lambda: norm(y, None, x, None, w[:32], None, rot)),
        (ls_ops.LsError, lambda: norm(y, None, x, None, w, w, rot)),
        (ls_ops.LsError, lambda: norm(y, None, x, None, w, None, rot, eps=-1.0)),
        (ValueError, lambda: gated(h, m, g, g, "tanh")), (TypeError, lambda: gated(h, m, g.float(), g)),
        (ValueError, lambda: gated(h.t(), m, g, g)), (ValueError, lambda: gated(h, m[:, :32], g, g)),
        (ValueError, lambda: gated(h, m, g, g[:64])), (ls_ops.LsError, lambda: gated(m[:, :64], m, g[:64], g[:64])),
        (ls_ops.LsError, lambda: ls_block.ls_gated_linear_bwd(m.clone(), None, None, h, m, g, g)),
        (ls_ops.LsError, lambda: ls_block.ls_grad_norm(f, None, lists)),
        (TypeError, lambda: ls_block.ls_grad_norm(f.half(), None, lists, workspace=s)),
        (TypeError, lambda: ls_block.ls_grad_norm(f, None, [m, 5], workspace=s)),
        (ValueError, lambda: ls_block.ls_grad_norm(f, None, [g.t()], workspace=s)),
        (ValueError, lambda: ls_block.ls_scale_gradients(lists, [m, m], f)),
        (ls_ops.LsError, lambda: ls_block.ls_scale_gradients([g], [m], f)),
        (TypeError, lambda: ls_block.ls_adam_update_scaled(p, p.float(), s, s.clone(), f, 1e-3)),
        (ValueError, lambda: ls_block.ls_adam_update_scaled(p, p.clone(), s[:9], s.clone(), f, 1e-3)),
        (ls_ops.LsError, lambda: ls_block.ls_adam_update_scaled(p, p.clone(), s, s.clone(), f, -1.0)),
        (ls_ops.LsError, lambda: ls_block.ls_adam_update_scaled(p, p.clone(), s, s, f, 1e-3)),
    ]


def test_both_ways_refuse_the_same(monkeypatch):
    require_gpu()
    everything()
    for way in (ls_block._call, ls_block._Closer()):
        monkeypatch.setattr(ls_block, "_call", way)
        for i, (error, call) in enumerate(refused()):
            with pytest.raises(error) as e:
                call()
            assert str(e.value), i
            if error is ls_ops.LsError:
                assert e.value.status != 0 and ls_block.last_error()
