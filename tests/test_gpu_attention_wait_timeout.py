"""The attention kernels' bounded waits, made to run out.

A host-side test setting (``fps_set_attention_test``) shortens the limit and
makes the first block of a kernel leave its first load out, so that the waits
for that tile run out.  The launch must end by itself, report
FPS_DEV_WAIT_TIMEOUT through the status word, and leave the CUDA context
usable: the same call then gives the same bits as before.  Nothing faults or
hangs: every wait of the kernels has a limit, and its warps leave together.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

FPS_DEV_WAIT_TIMEOUT = 6
FORWARD, SHORT, QUERIES, KEYS = 1, 2, 4, 8
POLLS = 2000  # of up to 20 us


def _inputs(sizes, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = lambda h: torch.randn((sum(sizes), h, D), generator=g, device="cuda").to(dtype)  # noqa: E731
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), device="cuda")
    return rows(4), rows(2), rows(2), rows(4), off


@pytest.mark.parametrize("D,dtype", [(64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("skip,sizes", [(FORWARD, [300, 40, 900]), (FORWARD, [100]), (SHORT, [100, 128, 30]), (QUERIES, [300, 40, 900]),
                                        (KEYS, [300, 40, 900]), (KEYS, [200])])
def test_wait_timeout_is_reported_and_the_context_stays_usable(skip, sizes, D, dtype):
    lib = fps.load_library()
    q, k, v, dout, off = _inputs(sizes, D, dtype)
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")

    def run(only=None):
        out, lse = first if only == "backward" else fps.attention_forward(q, k, v, off, workspace=ws, check_device=True)
        if only == "forward":
            return out, lse
        return (out, lse, *fps.attention_backward(dout, q, k, v, out, lse, off, workspace=ws, check_device=True))

    first = run("forward")
    clean = run()
    try:
        lib.fps_set_attention_test(POLLS, skip)
        with pytest.raises(fps.FpsError) as err:
            run("forward" if skip == FORWARD else "backward")
        assert err.value.detail == FPS_DEV_WAIT_TIMEOUT
    finally:
        lib.fps_set_attention_test(0, 0)
    torch.cuda.synchronize()
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(run(), clean))


def test_a_short_limit_alone_reports_nothing():
    lib = fps.load_library()
    q, k, v, dout, off = _inputs([300, 40, 900], 64, torch.bfloat16)
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    try:
        lib.fps_set_attention_test(POLLS, 0)
        out, lse = fps.attention_forward(q, k, v, off, workspace=ws, check_device=True)
        fps.attention_backward(dout, q, k, v, out, lse, off, workspace=ws, check_device=True)
    finally:
        lib.fps_set_attention_test(0, 0)
