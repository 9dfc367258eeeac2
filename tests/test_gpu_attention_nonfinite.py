"""Attention of packed events whose inputs are not numbers: rows that see a NaN
are NaN, in every kernel a call may take, and other events keep their bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


def _rand(shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _off(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int64, device="cuda")


# Keys of one event of 700 that hold a NaN: all of them; 16 in a row, one warp's
# of a tile in the kernel for few queries (and all of that warp's in the event of
# 64 keys); its first and its second chunk of 256 keys; the last key alone.
BAD_KEYS = {"all": slice(0, 700), "sixteen": slice(16, 32), "first chunk": slice(0, 256), "second chunk": slice(256, 512),
            "last": slice(699, 700)}


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 128), (BF16, 40)])
@pytest.mark.parametrize("nq", [1, 2, 40])
@pytest.mark.parametrize("where", ["query", *BAD_KEYS])
def test_rows_that_see_nan_are_nan(where, nq, dtype, D):
    """nq = 1 and 2: the kernel for few queries, in one chunk and in three; 40: the tile kernel."""
    nk = [300, 700, 64, 1]
    qo, ko = _off([nq] * 4), _off(nk)
    q, k, v = _rand((4 * nq, 4, D), 1, dtype), _rand((sum(nk), 2, D), 2, dtype), _rand((sum(nk), 2, D), 3, dtype)
    clean, clean_lse = fps.attention_forward(q, k, v, qo, ko)
    for event in (1, 2) if where in ("query", "all", "sixteen") else (1,):
        q2, k2 = q.clone(), k.clone()
        rows = slice(event * nq, (event + 1) * nq)
        if where == "query":
            q2[rows] = float("nan")
        else:
            at = BAD_KEYS[where]
            k2[int(ko[event]) + at.start:min(int(ko[event]) + at.stop, int(ko[event + 1]))] = float("nan")
        out, lse = fps.attention_forward(q2, k2, v, qo, ko)
        assert bool(out[rows].isnan().all()) and bool(lse[:, rows].isnan().all())
        others = [i for i in range(4 * nq) if not rows.start <= i < rows.stop]
        assert torch.equal(out[others], clean[others]) and torch.equal(lse[:, others], clean_lse[:, others])


@pytest.mark.parametrize("nq", [1, 2, 40])
def test_one_query_row_that_is_nan(nq):
    """The other rows of its event see only numbers."""
    nk = [900]
    q, k, v = _rand((nq, 4, 64), 4, BF16), _rand((900, 4, 64), 5, BF16), _rand((900, 4, 64), 6, BF16)
    clean = fps.attention_forward(q, k, v, _off([nq]), _off(nk))
    q[nq - 1, 2] = float("nan")
    out, lse = fps.attention_forward(q, k, v, _off([nq]), _off(nk))
    bad = torch.zeros((nq, 4), dtype=torch.bool, device="cuda")
    bad[nq - 1, 2] = True
    assert torch.equal(out.isnan().all(2), bad) and torch.equal(lse.isnan(), bad.T)
    assert torch.equal(out[~bad], clean[0][~bad])
