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
