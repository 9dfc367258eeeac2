"""Outputs given by the caller: beside their inputs in one buffer, and over them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402


def _rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 2, 70])
def test_rotary_into_other_heads_of_the_same_rows(T, dtype):
    table = fps.RotaryTable((16, 16))
    pos = _rand((T, 2), 1, torch.float32)
    rows = _rand((T, 12, 64), 2, dtype)
    heads_first = _rand((12, T, 64), 3, dtype).transpose(0, 1)
    wide = _rand((T, 6, 128), 4, dtype)
    for base, x, out in ((rows, rows[:, :6], rows[:, 6:]), (rows, rows[:, 6:], rows[:, :6]), (rows, rows[:, ::2], rows[:, 1::2]),
                         (heads_first, heads_first[:, :6], heads_first[:, 6:]), (wide, wide[:, :, :64], wide[:, :, 64:])):
        before = x.clone()
        want = fps.rotary_embed(before, pos, table)
        assert fps.rotary_embed(x, pos, table, out=out) is out
        assert torch.equal(out, want) and torch.equal(x, before)
    # a broadcast row of x, into memory of its own
    one = _rand((1, 6, 64), 5, dtype)
    assert torch.equal(fps.rotary_embed(one.expand(T, 6, 64), pos, table), fps.rotary_embed(one.repeat(T, 1, 1), pos, table))


def test_rotary_outputs_that_overlap():
    T, table = 70, fps.RotaryTable((16, 16))
    pos = _rand((T, 2), 1, torch.float32)
    rows = _rand((T, 12, 64), 2)
    keep = rows.clone()
    flat = rows.flatten()
    for x, out in ((rows[:, :6], rows[:, 5:11]), (rows[:, 1:7], rows[:, :6]), (rows[:-1, :6], rows[1:, :6]),
                   (flat[:64 * 60].view(60, 1, 64), flat[8:64 * 60 + 8].view(60, 1, 64)),
                   (rows[:35, :6], flat[: 35 * 6 * 64].view(35, 6, 64)),
                   (_rand((T, 2, 64), 3), flat.as_strided((T, 2, 64), (64, 64, 1))), (_rand((T, 2, 64), 3), flat.as_strided((T, 2, 64), (96, 64, 1)))):
        with pytest.raises(fps.FpsError):
            fps.rotary_embed(x, pos[: len(x)], table, out=out)
    assert torch.equal(rows, keep)


def test_attention_outputs():
    off = torch.tensor([0, 40, 70], device="cuda")
    buf = _rand((4, 70, 4, 64), 6)
    q, k, v, out = buf
    want, _ = fps.attention_forward(q, k, v, off)
    fps.attention_forward(q, k, v, off, out=out)
    assert torch.equal(out, want)
    for bad in (q, k, v, buf.flatten()[64:64 + out.numel()].view_as(out)):
        with pytest.raises(fps.FpsError):
            fps.attention_forward(q, k, v, off, out=bad)
    # one query's row among the keys' rows, at heads that are not read
    kv = _rand((70, 12, 64), 7)
    keep = kv.clone()
    one = torch.tensor([0, 1], device="cuda")
    ko = torch.tensor([0, 70], device="cuda")
    q1 = _rand((1, 4, 64), 8)
    want, _ = fps.attention_forward(q1, kv[:, :4], kv[:, 4:8], one, ko)
    fps.attention_forward(q1, kv[:, :4], kv[:, 4:8], one, ko, out=kv[20:21, 8:])
    assert torch.equal(kv[20:21, 8:], want) and torch.equal(kv[:, :8], keep[:, :8])
    with pytest.raises(fps.FpsError):
        fps.attention_forward(q1, kv[:, :4], kv[:, 4:8], one, ko, out=kv[20:21, 7:11])
