"""Rotation and norm where rows meet the lanes in other ways: halves that are no
multiple of a vector, heads of one and two lanes, tokens that follow one another
in a group, sequences that end inside it, and the most tokens there can be."""
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_heads as heads  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu

CASES = [  # dtype, batch, seq, heads, kv, dim, rotary, interleaved, memory, given, scaling
    ("f16", 3, 41, 5, 2, 40, 40, False, "rows", True, "none"),        # halves of 20
    ("bf16", 2, 300, 2, 1, 24, 24, False, "by head", False, "none"),  # of 12, few heads
    ("f32", 2, 50, 3, 1, 56, 52, False, "wide", True, "linear"),      # of 26
    ("f16", 2, 33, 4, 2, 88, 38, False, "turned", False, "none"),     # of 19
    ("f32", 1, 77, 6, 3, 32, 26, False, "rows", True, "none"),        # of 13
    ("bf16", 1, 19, 3, 3, 184, 14, False, "by head", True, "none"),   # of 7, a wide head
    ("f16", 1, 11, 2, 2, 480, 470, False, "rows", False, "none"),     # of 235
    ("f32", 1, 11, 2, 2, 496, 494, False, "rows", False, "none"),
    ("bf16", 7, 65, 3, 1, 16, 16, False, "rows", True, "none"),       # one lane
    ("f32", 7, 65, 3, 1, 16, 10, False, "turned", False, "none"),
    ("f16", 4, 129, 1, 1, 8, 6, True, "wide", True, "none"),
    ("f32", 4, 129, 1, 1, 8, 8, False, "wide", False, "none"),
    ("bf16", 900, 7, 2, 1, 32, 32, True, "rows", True, "none"),       # sequences shorter than a warp's tokens
    ("f16", 3000, 3, 2, 2, 24, 24, False, "by head", False, "none"),
    ("f32", 3000, 3, 1, 1, 40, 22, True, "rows", True, "yarn"),
    ("bf16", 1, 9001, 2, 2, 96, 62, True, "rows", True, "linear"),    # tokens one after the other
    ("f16", 2, 5003, 1, 1, 64, 64, False, "by head", False, "none"),
    ("bf16", 3, 7, 65, 13, 24, 18, True, "rows", False, "none"),      # many heads
]


@pytest.mark.parametrize("case", CASES, ids=heads.name)
def test_rotary(case):
    heads.test_rotary(case)


@pytest.mark.parametrize("case", CASES, ids=heads.name)
def test_in_place(case):
    heads.test_rotary_in_place_gives_the_same_bits(case)


@pytest.mark.parametrize("case", CASES, ids=heads.name)
def test_norm(case):
    heads.test_norm(case, True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter,rd", [(False, 16), (False, 24), (False, 20), (False, 22), (True, 24), (True, 22), (True, 2)])
def test_any_bits_behind_the_rotation_stay(dtype, inter, rd):
    """NaNs of every kind too; in place nothing behind it is written."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    word = torch.int32 if dtype is torch.float32 else torch.int16
    x = torch.ones(2, 9, 3, 40, device="cuda").to(dtype)
    bits = torch.randint(-2 ** 15, 2 ** 15, x.shape, generator=gen, device="cuda")
    x.view(word)[..., rd:] = ((bits << 16) + 12345 if dtype is torch.float32 else bits)[..., rd:].to(word)
    rot, y, z = ls_block.Rotation(rd, interleaved=inter), torch.empty_like(x), x.clone()
    ls_block.ls_rotary_fwd(y, None, x, None, rot, first_position=3)
    ls_block.ls_rotary_fwd(z, None, z, None, rot, first_position=3)
    assert torch.equal(y[..., rd:].view(word), x[..., rd:].view(word))
    assert torch.equal(z.view(word), y.view(word)) and torch.isfinite(y[..., :rd]).all()


@pytest.mark.parametrize("rd", [2, 8])
def test_the_most_tokens(rd):
    """batch * seq = 2^30, the inputs' rows all one."""
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 16 GB")
    batch, seq, dim = 64, 1 << 24, 8
    rot, one = ls_block.Rotation(rd), torch.ones(1, 1, 1, dim, device="cuda").half()
    y = torch.zeros(batch, seq, 1, dim, dtype=torch.float16, device="cuda")
    ls_block.ls_rotary_fwd(y, None, one.expand(batch, seq, 1, dim), None, rot)
    few = torch.empty(1, 4096, 1, dim, dtype=torch.float16, device="cuda")
    for first in (0, 12345678, seq - 4096):
        ls_block.ls_rotary_fwd(few, None, one.expand(1, 4096, 1, dim), None, rot, first_position=first)
        for b in (0, 31, batch - 1):
            assert torch.equal(y[b, first:first + 4096], few[0])


def test_states_that_take_turns():
    """Calls on several streams, each with its own buffers and workspace, give the bits of calls one by one."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(7)
    rot = ls_block.Rotation(64)
    sets, want = [], []
    for n in (700, 1300):
        x, g = (torch.randn(1, n, 8, 64, generator=gen, device="cuda").half() for _ in range(2))
        w, dw = torch.ones(64, device="cuda").half(), torch.empty(64, device="cuda").half()
        ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(64))
        sets.append((torch.empty_like(x), dw, g, x, w, ws))
    def call(s, stream=None):
        ls_block.ls_qk_norm_rotary_bwd(s[0], None, s[1], None, s[2], None, s[3], None, s[4], None, rot, workspace=s[5],
                                       stream=stream)
    for s in sets:
        call(s)
        want.append((s[0].clone(), s[1].clone()))
        s[0].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for s, stream in zip(sets, streams):
            call(s, stream)
    torch.cuda.synchronize()
    for s, (dx, dw) in zip(sets, want):
        assert torch.equal(s[0], dx) and torch.equal(s[1], dw)
