"""Refusals of the packed-token transformer operators, found on the host before
any launch: none of these calls reaches a GPU."""
import ctypes
import math

import pytest

import farthest_point_sampling_b200 as fps
from farthest_point_sampling_b200 import _lib

torch = pytest.importorskip("torch")
X = ctypes.c_void_p(256)


def test_rotary_table():
    t = fps.RotaryTable((4, 0, 6), base=100.0, axis_scale=(2.0, 1.0, -0.5))
    assert t.axes == 3 and t.pairs == 5 and list(t.c.axis[:5]) == [0, 0, 2, 2, 2]
    want = [2.0, 2.0 * 100 ** -0.5, -0.5, -0.5 * 100 ** (-1 / 3), -0.5 * 100 ** (-2 / 3)]
    for p, w in enumerate(want):
        # a float pair holds the float64 value to 2^-48
        assert abs(t.c.turns_hi[p] + t.c.turns_lo[p] - w / (2 * math.pi)) <= 2.0 ** -47 * abs(w)
    for bad in (dict(axis_dims=(3,)), dict(axis_dims=(0, 0)), dict(axis_dims=(-2, 4)), dict(axis_dims=(4,), base=0.0),
                dict(axis_dims=(4,), base=float("nan")), dict(axis_dims=(4,), axis_scale=(float("inf"),)),
                dict(axis_dims=(258,)), dict(axis_dims=(2,) * 9), dict(axis_dims=(4,), axis_scale=(1e300,))):
        with pytest.raises(fps.FpsError):
            fps.RotaryTable(**bad)
    with pytest.raises(ValueError):
        fps.RotaryTable(())
    with pytest.raises(ValueError):
        fps.RotaryTable((4, 4), axis_scale=(1.0,))


def test_rotary_argument_errors():
    lib = fps.load_library()
    t = fps.RotaryTable((4, 4)).c

    def call(x=X, y=X, dtype=1, T=5, H=2, D=16, xs=(32, 16), ys=(32, 16), pos=X, ps=2, table=t):
        return lib.fps_rotary(x, y, dtype, T, H, D, *xs, *ys, pos, ps, ctypes.byref(table) if table is not None else None, 0, None)

    assert call(dtype=3) == _lib.FPS_ERR_ARG
    assert call(T=-1) == _lib.FPS_ERR_ARG
    assert call(H=0) == _lib.FPS_ERR_ARG
    assert call(D=6) == _lib.FPS_ERR_ARG  # fewer values than the table turns
    assert call(D=512) == _lib.FPS_ERR_TOO_LARGE
    assert call(T=1 << 29) == _lib.FPS_ERR_TOO_LARGE
    assert call(table=None) == _lib.FPS_ERR_ARG
    assert call(pos=None) == _lib.FPS_ERR_ARG
    assert call(x=None) == _lib.FPS_ERR_ARG
    assert call(x=ctypes.c_void_p(257)) == _lib.FPS_ERR_ARG
    assert call(ps=1) == _lib.FPS_ERR_ARG
    assert call(xs=(64, 16)) == _lib.FPS_ERR_ARG  # in place with other strides
    assert call(ys=(32, 8), y=ctypes.c_void_p(4096)) == _lib.FPS_ERR_ARG  # heads of y overlap
    assert call(T=0) == _lib.FPS_OK
    broken = _lib.RotaryTableStruct.from_buffer_copy(t)
    broken.axis[3] = 7
    assert call(table=broken) == _lib.FPS_ERR_ARG


def _args(**kw):
    a = _lib.AttentionArgs()
    base = dict(q=256, k=256, v=256, dtype=1, heads=4, kv_heads=2, head_dim=64, n_q=10, n_kv=10, q_token_stride=256,
                q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64, q_offsets=256,
                kv_offsets=256, events=2, scale=0.125, causal=0, window=-1, sinks=0, max_tokens=0, zero_tail=0)
    base.update(kw)
    for name, value in base.items():
        setattr(a, name, value)
    return a


def test_attention_argument_errors():
    lib = fps.load_library()
    ws = lib.fps_attention_workspace_bytes(ctypes.byref(_args()), 0)
    wsb = lib.fps_attention_workspace_bytes(ctypes.byref(_args()), 1)
    assert ws > 0 and wsb > 0

    def both(code, **kw):
        a = _args(**kw)
        assert lib.fps_attention(ctypes.byref(a), X, X, X, 1 << 40, None) == code, kw
        assert lib.fps_attention_backward(ctypes.byref(a), X, X, X, 256, 64, X, X, X, X, 1 << 40, None) == code, kw

    for kw in (dict(dtype=0), dict(heads=3), dict(heads=0), dict(kv_heads=0), dict(head_dim=12), dict(head_dim=0), dict(n_q=-1),
               dict(n_kv=-1), dict(events=-1), dict(max_tokens=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(causal=2), dict(window=-2), dict(sinks=-1), dict(q=0), dict(k=0), dict(v=0),
               dict(q=264), dict(q_offsets=0), dict(kv_offsets=0), dict(q_token_stride=0), dict(q_head_stride=0),
               dict(k_token_stride=100), dict(v_head_stride=-64)):
        both(_lib.FPS_ERR_ARG, **kw)
    for kw in (dict(head_dim=136), dict(n_q=1 << 29), dict(n_kv=1 << 31), dict(heads=1 << 17, kv_heads=1),
               dict(n_q=(1 << 29) - 1, heads=4096, kv_heads=1)):
        both(_lib.FPS_ERR_TOO_LARGE, **kw)
    a = _args()
    ref = ctypes.byref(a)
    assert lib.fps_attention(None, X, X, X, ws, None) == _lib.FPS_ERR_ARG
    assert lib.fps_attention(ref, None, X, X, ws, None) == _lib.FPS_ERR_ARG
    assert lib.fps_attention(ref, ctypes.c_void_p(264), X, X, ws, None) == _lib.FPS_ERR_ARG
    assert lib.fps_attention(ref, X, X, X, ws - 1, None) == _lib.FPS_ERR_WORKSPACE
    assert lib.fps_attention(ref, X, X, None, ws, None) == _lib.FPS_ERR_WORKSPACE
    assert lib.fps_attention(ref, X, X, ctypes.c_void_p(128), ws, None) == _lib.FPS_ERR_WORKSPACE
    bw = lib.fps_attention_backward
    assert bw(ref, X, None, X, 256, 64, X, X, X, X, wsb, None) == _lib.FPS_ERR_ARG
    assert bw(ref, X, X, X, 256, 60, X, X, X, X, wsb, None) == _lib.FPS_ERR_ARG
    assert bw(ref, X, X, X, 256, 64, X, None, X, X, wsb, None) == _lib.FPS_ERR_ARG
    assert bw(ref, X, X, X, 256, 64, X, X, X, X, wsb - 1, None) == _lib.FPS_ERR_WORKSPACE


def test_binding_refusals():
    t = fps.RotaryTable((4, 4))
    x = torch.zeros((3, 2, 16))
    with pytest.raises(ValueError, match="CUDA"):
        fps.rotary_embed(x, torch.zeros((3, 2)), t)
    with pytest.raises(ValueError, match="CUDA"):
        fps.apply_rotary(x, torch.zeros((3, 2)), t)
    with pytest.raises(ValueError, match="gradient"):
        fps.apply_rotary(x, torch.zeros((3, 2), requires_grad=True), t)
    off = torch.tensor([0, 3])
    h = x.to(torch.bfloat16)
    for call in (lambda: fps.packed_attention(h, h, h, off), lambda: fps.attention_forward(h, h, h, off),
                 lambda: fps.attention_backward(h, h, h, h, h, torch.zeros((2, 3)), off)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workspace_of_long_and_refused_calls():
    """Long events keep float32 sums of key-tile pieces; their room stays bounded."""
    lib = fps.load_library()

    def size(**kw):
        return lib.fps_attention_workspace_bytes(ctypes.byref(_args(**kw)), 1)

    for kw in (dict(causal=2), dict(window=-2), dict(sinks=-1), dict(window=5, sinks=-(1 << 40))):
        assert size(**kw) == 0 and lib.fps_attention_workspace_bytes(ctypes.byref(_args(**kw)), 0) == 0
    big = dict(heads=8, kv_heads=2, head_dim=128, n_q=1 << 20, n_kv=1 << 20)
    for events in (1, 64, 1 << 20):
        # -lse and -D; lists of n / 128 + events tiles of queries and as many of keys, and of the events
        lists = 8 * (1 << 20) * 2 * 4 + 32 * (2 * (1 << 13) + 3 * events)
        for mask in (dict(), dict(causal=1), dict(window=0, sinks=1), dict(window=511, sinks=1 << 30, causal=1), dict(window=1 << 40)):
            # at most 4 pieces for each of 148 blocks and a few more, 128 x 256 floats each
            got = size(events=events, **big, **mask)
            assert lists <= got <= lists + (4 * 148 + 8) * (128 * 256 * 4 + 64) + (1 << 16), (events, mask)


def test_recorded_traffic_is_of_these_sources():
    """The measured DRAM bytes of the sampling kernels stay those of the sources that are here."""
    import os
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, root)
    try:
        import bench
    finally:
        sys.path.remove(root)
    with open(os.path.join(root, "profiles", "traffic.md")) as fh:
        assert bench.kernel_source_hash() in fh.read()


def test_rotary_refuses_outputs_that_overlap():
    """Element sizes of 2: a row of D = 16 values takes 32 bytes."""
    lib = fps.load_library()
    t = fps.RotaryTable((4, 4)).c

    def call(y, xs, ys, T=5, H=2, x=4096):
        return lib.fps_rotary(ctypes.c_void_p(x), ctypes.c_void_p(y), 1, T, H, 16, *xs, *ys, X, 2, ctypes.byref(t), 0, None)

    far = 1 << 20
    # rows of y over one another: both strides D, a head stride that meets the next row, and no stride at all
    for ys, T, H in (((16, 16), 5, 2), ((48, 40), 5, 2), ((40, 48), 5, 3), ((16, 64), 5, 2), ((16, 32), 3, 2), ((48, 64), 5, 4), ((17, 16), 2, 2)):
        assert call(far, (32, 16), ys, T, H) == _lib.FPS_ERR_ARG, (ys, T, H)
    # y a little behind or before x: by values, by heads, by rows
    for off in (2, 16, 30, -2, 32, -32, 64, -64, 4 * 64, -4 * 64, 4 * 64 + 32 + 30):
        assert call(4096 + off, (32, 16), (32, 16)) == _lib.FPS_ERR_ARG, off
    # the heads beside x of the same rows, one too few
    assert call(4096 + 32, (96, 16), (96, 16)) == _lib.FPS_ERR_ARG
    # within each other's reach with other strides
    assert call(4096 + 32, (96, 16), (192, 16)) == _lib.FPS_ERR_ARG
    assert call(4096 + 64, (0, 0), (32, 16), x=4096 + 64 + 32) == _lib.FPS_ERR_ARG


def test_attention_refuses_outputs_over_inputs():
    lib = fps.load_library()
    # q [10, 4, 64], k and v [10, 2, 64]: 512 and 256 bytes a row
    at = dict(q=1 << 16, k=1 << 17, v=1 << 18)
    a = _args(**at)
    ref = ctypes.byref(a)
    ptr = lambda p: ctypes.c_void_p(p)  # noqa: E731
    far = [ptr((1 << 20) + (i << 16)) for i in range(6)]
    size = {"q": 5120, "k": 2560, "v": 2560}
    for name, p in at.items():
        for out in (p, p + size[name] - 16, p - 5120 + 16):
            assert lib.fps_attention(ref, ptr(out), far[0], far[1], 1 << 40, None) == _lib.FPS_ERR_ARG, (name, out - p)

    def backward(out=far[0], dout=far[1], dq=far[2], dk=far[3], dv=far[4]):
        return lib.fps_attention_backward(ref, out, far[5], dout, 256, 64, dq, dk, dv, X, 1 << 40, None)

    for p in (*(ptr(x) for x in at.values()), far[0], far[1]):
        for name in ("dq", "dk", "dv"):
            assert backward(**{name: p}) == _lib.FPS_ERR_ARG, (name, p)
    assert backward(dq=far[3]) == backward(dv=far[3]) == backward(dv=far[2]) == _lib.FPS_ERR_ARG
    # a head of the queries' own row between two that q reads
    a = _args(**{**at, "q_token_stride": 1024, "q_head_stride": 128, "n_q": 1, "heads": 2})
    assert lib.fps_attention(ctypes.byref(a), ptr(at["q"] + 16), far[0], far[1], 1 << 40, None) == _lib.FPS_ERR_ARG
