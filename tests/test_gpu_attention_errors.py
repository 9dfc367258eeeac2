"""What a call gives that the device finds wrong: a status, and NaN in the rows
it could not compute."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

BF16 = torch.bfloat16


def _rand(shape, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _off(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int64, device="cuda")


def _stale(*shapes):
    """Memory of the outputs' sizes that holds numbers, given back to the allocator."""
    for s in shapes:
        t = torch.full(s, 3.0, dtype=BF16, device="cuda")
        del t


@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("nq,nk,hint", [([100, 300, 0, 20], [100, 300, 0, 20], 128), ([200, 90, 257, 3], [200, 90, 257, 3], 256),
                                        ([1, 1, 1, 1], [64, 900, 128, 2], 128)])
def test_rows_of_an_event_above_the_stated_longest_are_nan(nq, nk, hint, dtype):
    """The other events' rows, and those behind the last event, are as without the hint."""
    tail = 5
    qo, ko = _off(nq), _off(nk)
    q, dout = _rand((sum(nq) + tail, 4, 64), 1, dtype), _rand((sum(nq) + tail, 4, 64), 2, dtype)
    k, v = _rand((sum(nk) + tail, 2, 64), 3, dtype), _rand((sum(nk) + tail, 2, 64), 4, dtype)
    out0, lse0 = fps.attention_forward(q, k, v, qo, ko)
    grads0 = fps.attention_backward(dout, q, k, v, out0, lse0, qo, ko)
    _stale(q.shape, k.shape, k.shape, q.shape)
    out, lse = fps.attention_forward(q, k, v, qo, ko, max_tokens=hint)
    grads = fps.attention_backward(dout, q, k, v, out0, lse0, qo, ko, max_tokens=hint)
    bad = [max(a, b) > hint for a, b in zip(nq, nk)]
    q_bad = torch.tensor([x for x, n in zip(bad, nq) for _ in range(n)] + [False] * tail, device="cuda")
    k_bad = torch.tensor([x for x, n in zip(bad, nk) for _ in range(n)] + [False] * tail, device="cuda")
    for got, want, rows in ((out, out0, q_bad), (grads[0], grads0[0], q_bad), (grads[1], grads0[1], k_bad), (grads[2], grads0[2], k_bad)):
        assert bool(got[rows].isnan().all())
        assert torch.allclose(got[~rows].float(), want[~rows].float(), rtol=2 * torch.finfo(dtype).eps, atol=1e-5)
    assert bool(lse[:, q_bad].isnan().all())
    given = torch.full_like(q, 7.0)
    fps.attention_forward(q, k, v, qo, ko, max_tokens=hint, out=given)
    assert bool(given[q_bad].isnan().all()) and bool((given[-tail:] == 7.0).all())


@pytest.mark.parametrize("queries", [0, 1])
def test_rows_after_offsets_that_do_not_rise_are_nan(queries):
    """Offsets are taken 1024 events at a time; those of an earlier thousand count."""
    B = 2100
    ko = _off([3] * B)
    ko[1500] = 0
    ko[B] = 0
    qo = _off([queries] * B) if queries else ko
    n = 3 * B
    n_q = queries * B or n
    q, k, v = _rand((n_q, 2, 64), 5), _rand((n, 2, 64), 6), _rand((n, 2, 64), 7)
    good_k = _off([3] * B)
    good_q = _off([queries] * B) if queries else good_k
    want, _ = fps.attention_forward(q, k, v, good_q, good_k)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    _stale(q.shape)
    out, lse = fps.attention_forward(q, k, v, qo, ko, workspace=ws)
    with pytest.raises(fps.FpsError) as err:
        fps.device_status(ws)
    assert err.value.detail == 1
    done = 1024 * (queries or 3)
    assert torch.equal(out[:done], want[:done])
    assert bool(out[done:].isnan().all()) and bool(lse[:, done:].isnan().all())
    dout = _rand(q.shape, 8)
    good = fps.attention_backward(dout, q, k, v, want, torch.zeros_like(lse), good_q, good_k)
    _stale(q.shape, k.shape, k.shape)
    got = fps.attention_backward(dout, q, k, v, want, torch.zeros_like(lse), qo, ko, workspace=ws)
    for g, w, at in zip(got, good, (done, 3 * 1024, 3 * 1024)):
        assert torch.equal(g[:at], w[:at]) and bool(g[at:].isnan().all())


@pytest.mark.parametrize("grad", [False, True])
def test_the_public_call_reports(grad):
    """With check_device the call raises what the device found; without it the status is in the given workspace."""
    qo = _off([100, 129])
    q, k, v = (_rand((229, 2, 64), 9 + i).requires_grad_(grad) for i in range(3))
    assert bool(fps.packed_attention(q, k, v, qo, max_tokens=129, check_device=True).isfinite().all())
    bad = _off([100, 129])
    bad[1] = 300
    for offsets, hint, reason in ((qo, 128, 4), (bad, 0, 1)):
        with pytest.raises(fps.FpsError) as err:
            fps.packed_attention(q, k, v, offsets, max_tokens=hint, check_device=True)
        assert err.value.detail == reason
        ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
        out = fps.packed_attention(q, k, v, offsets, max_tokens=hint, workspace=ws)
        with pytest.raises(fps.FpsError) as err:
            fps.device_status(ws)
        assert err.value.detail == reason
        assert bool(out[100:].isnan().all()) and bool(out[:100].isfinite().all()) == (reason == 4)


def test_the_backward_pass_reports():
    """Its own plan finds what has gone wrong with the offsets since."""
    qo = _off([100, 129])
    q, k, v = (_rand((229, 2, 64), 19 + i).requires_grad_() for i in range(3))
    for check in (True, False):
        off = qo.clone()
        out = fps.packed_attention(q, k, v, off, check_device=check)
        off.data[1] = 300  # behind autograd's back
        if check:
            with pytest.raises(fps.FpsError) as err:
                out.sum().backward()
            assert err.value.detail == 1
        else:
            out.sum().backward()
            assert all(bool(t.grad.isnan().all()) for t in (q, k, v))


@pytest.mark.parametrize("nq,nk", [([100, 30], [100, 30]), ([1, 1, 1], [40, 2000, 0]), ([], []), ([20, 1], [300, 5])])
@pytest.mark.parametrize("given", [False, True])
def test_lse_of_rows_behind_the_last_event(nq, nk, given):
    """They see no key; what the memory held before does not show."""
    tail = 7
    qo, ko = _off(nq), _off(nk)
    q = _rand((sum(nq) + tail, 4, 64), 29)
    k, v = _rand((sum(nk) + tail, 2, 64), 30), _rand((sum(nk) + tail, 2, 64), 31)
    for _ in range(3):
        t = torch.full((4, len(q)), 3.0, device="cuda")
        del t
        out, lse = fps.attention_forward(q, k, v, qo, ko, out=torch.full_like(q, 7.0) if given else None)
        assert bool(torch.isneginf(lse[:, -tail:]).all()) and not bool(lse.isnan().any())
        assert bool((out[-tail:] == (7.0 if given else 0.0)).all())
