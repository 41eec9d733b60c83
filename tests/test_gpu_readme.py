"""README's example of the decoder block's operators runs as it is written, given
the tensors that it names."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("batch,seq,hidden,ffn", [(2, 9, 128, 264), (1, 1, 1280, 5120)])
def test_the_decoder_blocks_example(batch, seq, hidden, ffn):
    require_gpu()
    text = open(os.path.join(ROOT, "README.md")).read()
    section = text[text.index("### The decoder block's operators"):]
    code = re.search(r"```python\n(.*?)```", section, flags=re.S).group(1)
    heads, kv, head_dim = 4, 2, 128

    def t(*shape):
        return torch.randn(*shape, device="cuda").bfloat16()

    model = torch.nn.Linear(8, 8).cuda()
    for p in model.parameters():
        p.grad = torch.full_like(p, 4.0)
    names = dict(
        batch=batch, seq=seq, hidden=hidden, ffn=ffn, heads=heads, kv=kv, head_dim=head_dim, loss_scale=2.0, model=model,
        qkv=t(batch * seq, (heads + 2 * kv) * head_dim), q_weight=t(head_dim), k_weight=t(head_dim),
        positions=torch.arange(batch * seq, device="cuda", dtype=torch.int32).view(batch, seq),
        yq=t(batch, heads, seq, head_dim), yk=t(batch, kv, seq, head_dim), dyq=t(batch, heads, seq, head_dim),
        dyk=t(batch, kv, seq, head_dim), dq=t(batch, seq, heads, head_dim), dk=t(batch, seq, kv, head_dim),
        dqw=t(head_dim), dkw=t(head_dim), h=t(batch * seq, ffn), dh=t(batch * seq, ffn), x=t(batch * seq, hidden),
        dx=t(batch * seq, hidden), gate_weight=t(ffn, hidden), up_weight=t(ffn, hidden), dgate=t(ffn, hidden),
        dup=t(ffn, hidden), norm=torch.zeros(1, device="cuda"), factor=torch.zeros(1, device="cuda"))
    exec(compile(code, "README.md", "exec"), names)
    torch.cuda.synchronize()
    assert ls_block.check_device_errors() == 0
    # 72 gradients of 4, half of which is their unscaled value
    assert abs(float(names["norm"]) - 2.0 * 72 ** 0.5) < 1e-5
    for p in model.parameters():
        assert torch.allclose(p.grad, torch.full_like(p, 72 ** -0.5), rtol=1e-5)
