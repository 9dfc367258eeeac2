"""Multi-axis rotary positions (C ``fps_rotary``) against the formula in float64.

An output is x1 c - x2 s from float32 sines and cosines: their error is at
most 2^-22 (angle 2^-23 turns of 2 pi and the function's own 2^-23), the two
products and the sum add 3 * 2^-24 of |x1| + |x2|, and the result is rounded
once to its type: |err| <= (2^-21) (|x1| + |x2|) + u |y| with u = eps / 2."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _rand(shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _positions(T, axes, seed, reach=5000.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand((T, axes), generator=g, device="cuda") - 0.5) * 2 * reach


def _reference(x, pos, dims, base, scale, interleaved, inverse=False):
    w, a = [], []
    for ax, d in enumerate(dims):
        n = d // 2
        w += [(scale[ax] if scale else 1.0) * base ** (-i / n) for i in range(n)]
        a += [ax] * n
    R = len(w)
    theta = pos.double()[:, a] * torch.tensor(w, dtype=torch.float64, device=x.device)
    c, s = torch.cos(theta)[:, None], torch.sin(theta)[:, None] * (-1.0 if inverse else 1.0)
    y = x.double().clone()
    i1 = torch.arange(R, device=x.device) * (2 if interleaved else 1)
    i2 = i1 + (1 if interleaved else R)
    x1, x2 = x.double()[..., i1], x.double()[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    bound = torch.zeros_like(y)
    turned = torch.cat((i1, i2))
    u = torch.finfo(x.dtype).eps / 2
    bound[..., i1] = bound[..., i2] = 2.0 ** -21 * (x1.abs() + x2.abs())
    r = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps / 2
    bound[..., turned] += (u * y[..., turned].abs()).clamp_min(r)
    return y, bound


def _check(got, want):
    y, bound = want
    err = (got.double() - y).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,dims", [
    (1, 1, 2, (2,)), (3, 5, 64, (16, 16, 16, 16)), (130, 12, 64, (16, 16, 16, 16)), (777, 7, 72, (12, 12, 12, 24)),
    (50, 3, 40, (2, 4, 6, 8)), (33, 2, 46, (6, 10, 14)), (9, 40, 128, (32, 32, 32, 32)), (5, 300, 16, (4, 4, 4, 4)),
    (21, 1, 256, (64, 64, 64, 64)), (64, 4, 30, (10, 0, 20)),
])
def test_forward(dtype, interleaved, T, H, D, dims):
    x, pos = _rand((T, H, D), 1, dtype), _positions(T, len(dims), 2)
    scale = [0.5 + 0.1 * a for a in range(len(dims))]
    table = fps.RotaryTable(dims, base=1000.0, axis_scale=scale, interleaved=interleaved)
    _check(fps.rotary_embed(x, pos, table), _reference(x, pos, dims, 1000.0, scale, interleaved))
    _check(fps.rotary_embed(x, pos, table, inverse=True), _reference(x, pos, dims, 1000.0, scale, interleaved, inverse=True))


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows_and_in_place(dtype):
    """The query and key heads of a fused row; the value heads stay as they are."""
    T, D, dims = 300, 64, (16, 16, 16, 16)
    table = fps.RotaryTable(dims)
    rows, pos = _rand((T, 9, D), 3, dtype), _positions(T, 4, 4, 300.0)
    before = rows.clone()
    want = _reference(rows[:, :6], pos, dims, 10000.0, None, False)
    _check(fps.rotary_embed(rows[:, :6], pos, table), want)
    assert torch.equal(rows, before)
    back = fps.rotary_embed(rows[:, :6], pos, table, out=rows[:, :6])
    assert back.data_ptr() == rows.data_ptr()
    _check(rows[:, :6], want)
    assert torch.equal(rows[:, 6:], before[:, 6:])
    # heads before rows, and rows that start off a 16-byte boundary
    y = _rand((4, T, D), 5, dtype).transpose(0, 1)
    _check(fps.rotary_embed(y, pos, table), _reference(y, pos, dims, 10000.0, None, False))
    z = _rand((T * 4 * D + 1,), 6, dtype)[1:].view(T, 4, D)
    _check(fps.rotary_embed(z, pos, table), _reference(z, pos, dims, 10000.0, None, False))


def test_positions_of_a_wider_row_and_far_positions():
    T, dims = 257, (8, 8)
    table = fps.RotaryTable(dims, axis_scale=(1.0, 1.0))
    wide = _positions(T, 4, 7, 3e6)
    x = _rand((T, 2, 16), 8)
    _check(fps.rotary_embed(x, wide[:, 1:3], table), _reference(x, wide[:, 1:3], dims, 10000.0, None, False))


def test_gradient():
    """The gradient against the formula's (the inverse turn), against differences, and through any layout of the incoming one."""
    T, H, D, dims = 65, 3, 40, (4, 8, 12, 16)
    table = fps.RotaryTable(dims, interleaved=True)
    pos = _positions(T, 4, 9, 100.0)
    x = _rand((T, H, D), 10).requires_grad_(True)
    dy = _rand((T, H, D), 11)
    y = fps.apply_rotary(x, pos, table)
    (dx,) = torch.autograd.grad(y, x, dy)
    _check(dx, _reference(dy, pos, dims, 10000.0, None, True, inverse=True))
    step = _rand((T, H, D), 12)
    diff = ((fps.rotary_embed((x + step).detach(), pos, table).double() * dy).sum()
            - (fps.rotary_embed(x.detach(), pos, table).double() * dy).sum())
    assert abs(float(diff - (dx.double() * step).sum())) <= 1e-4 * float((dx.double() * step).abs().sum())
    x2 = _rand((T, H, D), 10).requires_grad_(True)
    fps.apply_rotary(x2, pos, table).sum().backward()  # an expanded gradient
    _check(x2.grad, _reference(torch.ones_like(dy), pos, dims, 10000.0, None, True, inverse=True))


def test_no_rows_nonfinite_and_other_stream():
    table = fps.RotaryTable((4, 4))
    assert fps.rotary_embed(torch.empty((0, 2, 8), device="cuda"), torch.empty((0, 2), device="cuda"), table).shape == (0, 2, 8)
    x, pos = _rand((6, 2, 8), 13), _positions(6, 2, 14, 10.0)
    pos[2, 0] = float("nan")
    pos[3, 1] = float("inf")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = fps.rotary_embed(x, pos, table)
    s.synchronize()
    ok = [0, 1, 4, 5]
    _check(y[ok], _reference(x[ok], pos[ok], (4, 4), 10000.0, None, False))
    assert bool(y[2, :, [0, 1, 4, 5]].isnan().all()) and bool(y[3, :, [2, 3, 6, 7]].isnan().all())
    assert bool(y[2, :, [2, 3, 6, 7]].isfinite().all())


def test_captured_and_replayed():
    table = fps.RotaryTable((16, 16, 16, 16))
    x, pos = _rand((200, 6, 64), 15, torch.bfloat16), _positions(200, 4, 16)
    out = torch.empty_like(x)
    fps.rotary_embed(x, pos, table, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fps.rotary_embed(x, pos, table, out=out)
    x.copy_(_rand((200, 6, 64), 17, torch.bfloat16))
    graph.replay()
    _check(out, _reference(x, pos, (16, 16, 16, 16), 10000.0, None, False))
