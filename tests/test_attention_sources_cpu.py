"""What can be read from the attention kernels' sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "farthest_point_sampling_b200", "csrc")


def test_waits_end_alike_for_a_whole_warp():
    """Between two waits the warps run instructions that need all their lanes
    (TMEM reads and writes, ballots): a wait that gave up for some lanes only
    would leave the others in one of them for good.  So a lane waits alone in
    one place, where the warp then agrees on the answer."""
    polls = []
    for path in glob.glob(os.path.join(CSRC, "attention*.cu*")) + [os.path.join(CSRC, "tcgen05.cuh")]:
        with open(path) as fh:
            text = re.sub(r"//[^\n]*", "", fh.read())
        polls += [(os.path.basename(path), m.group(0)) for m in re.finditer(r"[^\n]*\b(mbar_wait|mbar_wait_lane|mbar_try)\([^\n]*", text)]
    assert {p[0] for p in polls} == {"tcgen05.cuh"}
    assert [re.sub(r"\s+", " ", p[1]).strip() for p in polls] == [
        "__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {",
        "__device__ __forceinline__ bool mbar_wait_lane(uint32_t bar, uint32_t parity, volatile WaitState* state) {",
        "for (int i = 0; !mbar_try(bar, parity); ++i)",
        "return __all_sync(0xffffffffu, mbar_wait_lane(bar, parity, state));",
    ]
