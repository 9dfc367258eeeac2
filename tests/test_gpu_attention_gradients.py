"""Gradients of packed attention and rotary positions as a model's graph asks for them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402
from attention_reference import assert_within, attention  # noqa: E402


def _rand(shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("before", [1, 3, 8])
def test_incoming_gradient_off_a_16_byte_boundary(before, dtype):
    """What torch.cat hands back is a contiguous piece of a larger gradient."""
    sizes = [150, 20]
    qo = torch.tensor([0, 150, 170], device="cuda")
    q, k, v = (_rand((170, h, 64), 10 + i, dtype).requires_grad_() for i, h in enumerate((4, 2, 2)))
    g = _rand((before + q.numel(),), 13, dtype)
    y = torch.cat([torch.zeros(before, dtype=dtype, device="cuda"), fps.packed_attention(q, k, v, qo).flatten()])
    y.backward(g)
    dout = g[before:].view_as(q).clone()
    want = attention(q.detach(), k.detach(), v.detach(), qo, qo, dout=dout)
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        assert_within(t.grad, want[name], name)
    table = fps.RotaryTable((16, 16))
    pos = _rand((170, 2), 14, torch.float32)
    x = _rand((170, 4, 64), 15, dtype).requires_grad_()
    torch.cat([torch.zeros(before, dtype=dtype, device="cuda"), fps.apply_rotary(x, pos, table).flatten()]).backward(g)
    assert torch.equal(x.grad, fps.rotary_embed(dout, pos, table, inverse=True))
