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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [[128, 77, 300], [100, 60]])
def test_training_step_in_a_graph(sizes, dtype):
    """The public call and its gradients captured, and replayed on other values: as the same step outside."""
    n = sum(sizes)
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), device="cuda")
    q, k, v = (_rand((n, h, 64), 20 + i, dtype).requires_grad_() for i, h in enumerate((4, 2, 2)))
    dout = _rand((n, 4, 64), 23, dtype)

    def step():
        out = fps.packed_attention(q, k, v, off, max_tokens=max(sizes))
        return [out.detach(), *torch.autograd.grad(out, (q, k, v), dout)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed, size in ((30, 1.0), (40, 100.0), (50, 1e-3)):
        with torch.no_grad():
            for i, t in enumerate((q, k, v, dout)):
                t.copy_(_rand(t.shape, seed + i, torch.float32) * (size if t is dout else 1.0))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_workspaces_of_calls_on_two_streams():
    """Each stream with a workspace of its own, many calls in flight; a workspace is one call's at a time."""
    sizes = [500, 40, 128]
    n = sum(sizes)
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), device="cuda")
    q, k, v = (_rand((n, h, 128), 60 + i, torch.float16) for i, h in enumerate((4, 2, 2)))
    dout = _rand((n, 4, 128), 63, torch.float16)
    out, lse = fps.attention_forward(q, k, v, off)
    want = (out, *fps.attention_backward(dout, q, k, v, out, lse, off))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    ws = [torch.empty(1 << 24, dtype=torch.uint8, device="cuda") for _ in streams]
    for _ in range(8):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                o, l2 = fps.attention_forward(q, k, v, off, workspace=w)
                got.append((o, *fps.attention_backward(dout, q, k, v, o, l2, off, workspace=w)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
