"""Rows whose place passes 2^31 elements: the same bits as in a tensor of their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

FAR = (1 << 24) + 4096  # rows of 128 values: 2^31 elements and more


def _off(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int64, device="cuda")


def _far(rows, dtype):
    """[FAR, 1, 128] of zeros but for its last rows."""
    t = torch.zeros((FAR, 1, 128), dtype=dtype, device="cuda")
    t[FAR - len(rows):] = rows
    return t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [[300, 100], [64]])
def test_last_events_of_a_long_batch(sizes, dtype):
    """Before them events of one key in sight of each query, as many rows as it takes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n = sum(sizes)
    q, k, v, dout = (torch.randn((n, 1, 128), generator=g, device="cuda").to(dtype) for _ in range(4))
    kw = dict(causal=True, window=20, sinks=2)
    want = fps.attention_forward(q, k, v, _off(sizes), check_device=True, **kw)
    grads = fps.attention_backward(dout, q, k, v, *want, _off(sizes), **kw)
    before = FAR - n
    off = _off([before // 2, before - before // 2] + sizes)
    Q, K, V = (_far(t, dtype) for t in (q, k, v))
    out, lse = fps.attention_forward(Q, K, V, off, check_device=True, **kw)
    assert torch.equal(out[-n:], want[0]) and torch.equal(lse[:, -n:], want[1])
    assert bool((out[: FAR - n] == 0).all())
    got = fps.attention_backward(_far(dout, dtype), Q, K, V, out, lse, off, check_device=True, **kw)
    for a, b in zip(got, grads):
        assert torch.equal(a[-n:], b) and bool((a[: FAR - n] == 0).all())


def test_summary_query_over_far_keys():
    """The keys of the last event lie beyond 2^31 elements, and its rows in the workspace with them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((2, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((5000, 1, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    K, V = _far(k, torch.bfloat16), _far(v, torch.bfloat16)
    out, lse = fps.attention_forward(q, K, V, _off([1, 1]), _off([FAR - 5000, 5000]), check_device=True)
    want = torch.softmax((q[1:].double()[:, 0] @ k.double()[:, 0].T) * 128 ** -0.5, 1) @ v.double()[:, 0]
    assert float((out[1].double() - want).norm() / want.norm()) <= 2.0 ** -7
    assert bool((out[0] == 0).all())


def test_rotary_of_far_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    table = fps.RotaryTable((32, 32))
    x = torch.randn((500, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.rand((500, 2), generator=g, device="cuda") * 100
    P = torch.zeros((FAR, 2), device="cuda")
    P[-500:] = pos
    got = fps.rotary_embed(_far(x, torch.bfloat16), P, table)
    assert torch.equal(got[-500:], fps.rotary_embed(x, pos, table)) and bool((got[:-500] == 0).all())
