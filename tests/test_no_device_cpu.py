"""The packed-token operators on a host without a GPU: an error code, and the
process goes on.  In a child that sees no device, so that nothing is launched."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, sys
sys.path.insert(0, {root!r})
import farthest_point_sampling_b200 as fps
from farthest_point_sampling_b200 import _lib

lib, P = fps.load_library(), [ctypes.c_void_p((i + 1) << 20) for i in range(8)]
table = fps.RotaryTable((4, 4)).c
for dtype in (0, 1, 2):
    assert lib.fps_rotary(P[0], P[1], dtype, 5, 2, 16, 32, 16, 32, 16, P[2], 2, ctypes.byref(table), 0, None) == _lib.FPS_ERR_CUDA
a = _lib.AttentionArgs(P[0].value, P[1].value, P[2].value, 1, 4, 2, 64, 10, 10, 256, 64, 128, 64, 128, 64, 256, 256, 2, 0.125, 0, -1, 0, 0, 0)
ref = ctypes.byref(a)
assert lib.fps_attention(ref, P[3], P[4], P[7], 1 << 20, None) == _lib.FPS_ERR_CUDA
assert lib.fps_attention_backward(ref, P[3], P[4], P[3], 256, 64, P[5], P[6], ctypes.c_void_p(9 << 20), P[7], 1 << 20, None) == _lib.FPS_ERR_CUDA
print("done")
"""


def test_calls_without_a_device_return_an_error():
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0 and r.stdout == "done\n", (r.returncode, r.stderr[-800:])


OVERLAP = """
import ctypes, itertools, random, sys
sys.path.insert(0, {root!r})
import farthest_point_sampling_b200 as fps
from farthest_point_sampling_b200 import _lib

lib, rng = fps.load_library(), random.Random(3)
table = fps.RotaryTable((2,)).c
D, seen = 4, set()


def rows(at, T, H, token, head):
    return [range(at + t * token + h * head, at + t * token + h * head + D) for t in range(T) for h in range(H)]


def meet(a, b):
    return any(r.start < s.stop and s.start < r.stop for r in a for s in b)


for _ in range(40000):
    T, H = rng.randint(1, 5), rng.randint(1, 4)
    ys = rng.randint(4, 40), rng.randint(4, 40)
    xs = ys if rng.random() < 0.7 else (rng.randint(0, 40), rng.randint(0, 40))
    y = 4096
    x = y + rng.randint(-150, 150) if rng.random() < 0.9 else y
    X, Y = rows(x, T, H, *xs), rows(y, T, H, *ys)
    own = any(meet([a], [b]) for a, b in itertools.combinations(Y, 2))
    used = [k for k, n in enumerate((T, H)) if n > 1]
    if x == y:
        bad = xs != ys
    elif all(xs[k] == ys[k] for k in used):
        bad = meet(X, Y)
    else:
        bad = max(r.stop for r in X) > min(r.start for r in Y) and max(r.stop for r in Y) > min(r.start for r in X)
    got = lib.fps_rotary(ctypes.c_void_p(2 * x), ctypes.c_void_p(2 * y), 1, T, H, D, *xs, *ys, ctypes.c_void_p(1 << 20), 1, ctypes.byref(table), 0, None)
    want = _lib.FPS_ERR_ARG if own or bad else _lib.FPS_ERR_CUDA
    assert got == want, (T, H, x - y, xs, ys, own, bad, got)
    seen.add((own, bad, xs == ys))
assert len(seen) == 8
a = _lib.AttentionArgs()
for name, value in dict(q=1 << 30, v=1 << 31, dtype=1, kv_heads=1, head_dim=8, events=1, q_offsets=256, kv_offsets=256, scale=1.0, window=-1,
                        q_token_stride=64, q_head_stride=8, v_token_stride=64, v_head_stride=8).items():
    setattr(a, name, value)
for _ in range(20000):
    n_q, heads, n_kv = rng.randint(1, 3), rng.randint(1, 2), rng.randint(1, 6)
    a.n_q, a.heads, a.n_kv, a.kv_heads = n_q, heads, n_kv, heads
    a.k_token_stride, a.k_head_stride = 8 * rng.randint(1, 12), 8 * rng.randint(1, 12)
    a.k = 1 << 20
    out = (1 << 20) + 16 * rng.randint(-30, 120)
    starts = [(1 << 20) + 2 * (t * a.k_token_stride + h * a.k_head_stride) for t in range(n_kv) for h in range(heads)]
    K = [range(s, s + 16) for s in starts]
    bad = meet([range(out, out + n_q * heads * 16)], K)
    got = lib.fps_attention(ctypes.byref(a), ctypes.c_void_p(out), None, ctypes.c_void_p(1 << 32), 1 << 40, None)
    assert got == (_lib.FPS_ERR_ARG if bad else _lib.FPS_ERR_CUDA), (n_q, heads, n_kv, a.k_token_stride, a.k_head_stride, out - (1 << 20), bad, got)
print("done")
"""


def test_overlaps_found_are_those_of_the_rows():
    """Which outputs are refused, against each row's range of bytes."""
    r = subprocess.run([sys.executable, "-c", OVERLAP.format(root=ROOT)], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0 and r.stdout == "done\n", (r.returncode, r.stderr[-800:])
