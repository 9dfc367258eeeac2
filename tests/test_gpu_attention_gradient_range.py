"""Gradients of long events and of incoming gradients far from 1 in size.

With n keys in sight a softmax weight is about 1 / n and a score gradient that
times |dO|: in float16 both leave the normal range, where a rounding no longer
follows the value.  Errors are taken in norm over a whole gradient.

Rounding a value of the normal range costs 0.432 half steps of it in the mean of
squares (sqrt(E ulp(x)^2 / 12) / (eps / 2)).  With dS rounded, dQ_id = scale
sum_j dS_ij K_jd is off by what these independent errors add up to,

    0.432^2 (eps / 2)^2 scale^2 sum_j dS_ij^2 K_jd^2   (its square),

and dK and dV alike; D from the rounded output adds an eighth of it at most (17
keys in sight or more), and the last rounding what rounding the exact gradient
costs, which is computed.  The square root of the sum may be exceeded by 0.15 of
it, for what 0.432 leaves to how the values' mantissas lie (0.29 to 0.58 for a
single one); beyond that something else is lost.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


def _rand(shape, seed, dtype, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * size).to(dtype)


def _off(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int64, device="cuda")


def _exact(q, k, v, dout, nq, nk, causal):
    """dq, dk and dv of the definition in float64, an event and a head at a
    time, and for each the sum of the squares of its products' terms."""
    group, scale = q.shape[1] // k.shape[1], q.shape[2] ** -0.5
    dq, dk, dv = (torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v))
    squares = [0.0, 0.0, 0.0]
    a = b = 0
    for n, m in zip(nq, nk):
        for h in range(q.shape[1]) if n and m else ():
            Q, dO = (t[a:a + n, h].double() for t in (q, dout))
            K, V = (t[b:b + m, h // group].double() for t in (k, v))
            S = Q @ K.T * scale
            if causal:
                p = torch.arange(n, device=q.device)[:, None] + m - n
                S.masked_fill_(torch.arange(m, device=q.device)[None] > p, float("-inf"))
            P = torch.softmax(S, 1)
            del S
            dS = P * (dO @ V.T - ((P @ V) * dO).sum(1, keepdim=True))
            dq[a:a + n, h] = scale * dS @ K
            dk[b:b + m, h // group] += scale * dS.T @ Q
            dv[b:b + m, h // group] += P.T @ dO
            P.square_()
            dS.square_()
            for i, terms in enumerate((scale ** 2 * dS @ K.square(), scale ** 2 * dS.T @ Q.square(), P.T @ dO.square())):
                squares[i] += float(terms.sum())
        a, b = a + n, b + m
    return zip((dq, dk, dv), squares)


def _check(q, k, v, dout, nq, nk, causal=False, max_tokens=0):
    qo, ko = _off(nq), _off(nk)
    got = fps.attention_backward(dout, q, k, v, *fps.attention_forward(q, k, v, qo, ko, causal=causal, max_tokens=max_tokens), qo, ko,
                                 causal=causal, max_tokens=max_tokens)
    u = torch.finfo(q.dtype).eps / 2
    for g, (w, squares), name in zip(got, _exact(q, k, v, dout, nq, nk, causal), ("dq", "dk", "dv")):
        once = float((w.to(q.dtype).double() - w).square().sum())
        limit = 1.15 * (once + 1.125 * (0.432 * u) ** 2 * squares) ** 0.5
        err = float((g.double() - w).norm())
        assert err <= limit, (name, err / limit, limit / float(w.norm()))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3])
@pytest.mark.parametrize("n,D,H,G,causal", [(9000, 64, 2, 1, False), (12000, 64, 1, 1, False), (9000, 128, 2, 2, True), (2000, 8, 2, 2, False)])
def test_long_events(n, D, H, G, causal, size, dtype):
    q, dout = _rand((n, H, D), 1, dtype), _rand((n, H, D), 2, dtype, size)
    k, v = _rand((n, G, D), 3, dtype), _rand((n, G, D), 4, dtype)
    _check(q, k, v, dout, [n], [n], causal)


def test_one_query_over_many_keys():
    """Weights of 1 / 200000, for a few rows of the queries' own."""
    nq, nk = [3, 1], [200000, 30000]
    q, dout = _rand((4, 4, 64), 5, F16), _rand((4, 4, 64), 6, F16, 1e-2)
    k, v = _rand((230000, 2, 64), 7, F16), _rand((230000, 2, 64), 8, F16)
    _check(q, k, v, dout, nq, nk)


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3])
@pytest.mark.parametrize("D,H,G", [(8, 2, 2), (64, 4, 4), (64, 6, 2), (128, 4, 2)])
@pytest.mark.parametrize("hint", [0, 128])
def test_short_events(D, H, G, size, hint):
    nq = nk = [128, 100, 128, 77, 64] * 8
    n = sum(nq)
    q, dout = _rand((n, H, D), 9, F16), _rand((n, H, D), 10, F16, size)
    k, v = _rand((n, G, D), 11, F16), _rand((n, G, D), 12, F16)
    _check(q, k, v, dout, nq, nk, max_tokens=hint)


@pytest.mark.parametrize("sizes", [[100, 128], [900, 300]])
def test_large_gradients_of_peaked_rows(sizes):
    """Score gradients beyond 65504, float16's largest, of gradients that fit: keys and queries are small where they are."""
    n = sum(sizes)
    q, k = _rand((n, 2, 64), 13, F16, 8.0), _rand((n, 2, 64), 14, F16, 0.5)
    v, dout = _rand((n, 2, 64), 15, F16, 200.0), _rand((n, 2, 64), 16, F16, 200.0)
    q *= 1e-2
    k *= 1e-2
    _check(q, k, v, dout, sizes, sizes)


def test_events_do_not_set_each_others_range():
    """An event's gradients are the same bits whatever the sizes of the others' values, not-a-numbers among them."""
    sizes = [90, 700, 128, 5]
    n, at = sum(sizes), [0, 90, 790, 918, 923]
    q, dout = _rand((n, 4, 64), 17, F16), _rand((n, 4, 64), 18, F16)
    k, v = _rand((n, 2, 64), 19, F16), _rand((n, 2, 64), 20, F16)
    off = _off(sizes)

    def run(d, w):
        return fps.attention_backward(d, q, k, w, *fps.attention_forward(q, k, w, off), off)

    first = run(dout, v)
    for event in range(4):
        rows = slice(at[event], at[event + 1])
        others = [i for i in range(n) if not rows.start <= i < rows.stop]
        for x in (1e3, 1e-4, float("inf"), float("nan")):
            d, w = dout.clone(), v.clone()
            d[rows] *= x
            w[rows] *= x
            assert all(torch.equal(a[others], b[others]) for a, b in zip(run(d, w), first))
