"""The binding of the packed-token operators, with the launch stood in for on
the host: what it checks, and what it hands to the library and to autograd."""
import pytest

import farthest_point_sampling_b200 as fps
from farthest_point_sampling_b200 import api

torch = pytest.importorskip("torch")
BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """Host tensors pass for the device's; a call to the library is noted by name and goes no further."""
    made = []
    monkeypatch.setattr(api, "_cuda_device", lambda t: t.device)
    monkeypatch.setattr(api, "_call", lambda fn, where, device, *args: made.append((where, args)))
    return made


def _qkv(n=6, H=2, G=1, D=16, **kw):
    return [torch.zeros((n, h, D), dtype=BF16, **kw) for h in (H, G, G)], torch.tensor([0, 2, n])


def test_workspace_of_another_device_or_without_memory(calls):
    (q, k, v), off = _qkv()
    need = 1 << 20
    good = torch.empty(need, dtype=torch.uint8)
    out, lse = fps.attention_forward(q, k, v, off, workspace=good)
    fps.attention_backward(q, q, k, v, out, lse, off, workspace=good)
    assert [c[0] for c in calls] == ["fps_attention", "fps_attention_backward"]
    for bad in (torch.empty(need, dtype=torch.uint8, device="meta"), torch.empty(1, dtype=torch.uint8).expand(need),
                torch.empty(2 * need, dtype=torch.uint8)[::2], torch.empty(16, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            fps.attention_forward(q, k, v, off, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            fps.attention_backward(q, q, k, v, out, lse, off, workspace=bad)
    assert len(calls) == 2


def test_check_device_reads_the_status_after_each_pass(calls, monkeypatch):
    (q, k, v), off = _qkv(requires_grad=True)
    monkeypatch.setattr(api, "device_status", lambda ws: calls.append(("status", ws)))
    mine = torch.empty(1 << 20, dtype=torch.uint8)
    out = fps.packed_attention(q, k, v, off, workspace=mine, check_device=True)
    out.backward(torch.zeros_like(out))
    assert [c[0] for c in calls] == ["fps_attention", "status", "fps_attention_backward", "status"]
    assert calls[1][1] is mine and calls[3][1] is not mine
    del calls[:]
    with torch.no_grad():
        fps.packed_attention(q, k, v, off, workspace=mine, check_device=True)
        fps.packed_attention(q, k, v, off)
    assert [c[0] for c in calls] == ["fps_attention", "status", "fps_attention"] and calls[1][1] is mine


@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_tangents_are_refused(calls, which):
    """A dual tensor whose tangent the call would drop raises, with and without a gradient to come."""
    import torch.autograd.forward_ad as fwad

    for grad in (False, True):
        t, off = _qkv(requires_grad=grad)
        with fwad.dual_level():
            t[which] = fwad.make_dual(t[which], torch.ones_like(t[which]))
            with pytest.raises(NotImplementedError):
                fps.packed_attention(*t, off)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                fps.packed_attention(*t, off)
            plain, off = _qkv()
            assert fps.packed_attention(*plain, off).shape == plain[0].shape


def test_forward_mode_tangents_of_rotary_are_refused(calls):
    import torch.autograd.forward_ad as fwad

    table = fps.RotaryTable((4, 4))
    x, pos = torch.zeros((3, 2, 16)), torch.zeros((3, 2))
    with fwad.dual_level():
        with pytest.raises(NotImplementedError):
            fps.apply_rotary(fwad.make_dual(x, torch.ones_like(x)), pos, table)
        with pytest.raises(NotImplementedError):
            fps.apply_rotary(x, fwad.make_dual(pos, torch.ones_like(pos)), table)


def test_incoming_gradients_are_made_readable():
    base = torch.arange(1 + 4 * 2 * 16, dtype=torch.float32).to(BF16)
    aligned = base[:-1].view(4, 2, 16)
    assert aligned.data_ptr() % 16 == 0 and api._dense_heads(aligned) is aligned
    for t in (base[1:].view(4, 2, 16), torch.ones((), dtype=BF16).expand(4, 2, 16), aligned.transpose(1, 2).contiguous().transpose(1, 2),
              base[1:33].view(1, 2, 16)):
        got = api._dense_heads(t)
        assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, t)
