"""Attention of packed events (C ``fps_attention`` / ``fps_attention_backward``)
against float64, element by element within the bound that
``attention_reference`` derives."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the gpu marker is deselected on CPU hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import farthest_point_sampling_b200 as fps  # noqa: E402
from attention_reference import assert_within, attention  # noqa: E402
from farthest_point_sampling_b200 import _lib  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


def _rand(shape, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _off(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int64, device="cuda")


def _inputs(nq, nk, H, G, D, dtype, seed, tail=0):
    q, dout = _rand((sum(nq) + tail, H, D), seed, dtype), _rand((sum(nq) + tail, H, D), seed + 1, dtype)
    k, v = _rand((sum(nk) + tail, G, D), seed + 2, dtype), _rand((sum(nk) + tail, G, D), seed + 3, dtype)
    return q, k, v, dout, _off(nq), _off(nk)


def _check(q, k, v, dout, qo, ko, max_tokens=0, **mask):
    """Forward, lse and the three gradients through the raw calls."""
    out, lse = fps.attention_forward(q, k, v, qo, ko, max_tokens=max_tokens, **mask)
    want = attention(q, k, v, qo, ko, dout=dout, **mask)
    n_q, n_k = int(qo[-1]), int(ko[-1])
    assert_within(out, want["out"], "out")
    assert_within(lse[:, :n_q], tuple(x[:, :n_q] for x in want["lse"]), "lse")
    lse[:, n_q:] = float("nan")  # rows of no event are not read
    got = fps.attention_backward(dout, q, k, v, out, lse, qo, ko, max_tokens=max_tokens, **mask)
    for g, name in zip(got, ("dq", "dk", "dv")):
        assert_within(g, want[name], name)
        assert bool((g[n_q if name == "dq" else n_k:] == 0).all())
    return out, got


SIZES = [
    [1], [2, 1, 3], [128], [129, 5, 0, 64], [127, 128, 1, 0, 0, 256, 31], [300, 17, 700],
    [16, 15, 33, 8, 7, 1, 64, 65, 63, 100], [0, 0], [1000],
]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_whole_events(sizes, dtype, D):
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 3, 3, D, dtype, 10)
    _check(q, k, v, dout, qo, qo)


@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 48, 56, 72, 80, 96, 104, 120])
def test_head_sizes(D):
    sizes = [70, 200, 3]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 4, 2, D, BF16 if D % 16 else F16, 20 + D)
    _check(q, k, v, dout, qo, ko)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 0), (0, 1), (1, 2), (17, 0), (63, 5), (128, 16), (127, 130), (300, 128), (5000, 3), (-1, 9), (3, 1 << 50)])
@pytest.mark.parametrize("D", [64, 128])
def test_windows_and_sinks(causal, window, sinks, D):
    sizes = [400, 1, 130, 0, 777]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 4, 2, D, F16 if sinks % 2 else BF16, 30)
    _check(q, k, v, dout, qo, ko, causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("causal,window,sinks", [(False, -1, 0), (True, -1, 0), (True, 10, 3), (False, 40, 2)])
@pytest.mark.parametrize("nq,nk", [
    ([1, 1, 1], [5, 300, 1]), ([2, 0, 7, 1], [0, 9, 400, 129]), ([200, 5, 130], [3, 260, 129]), ([1], [2000]), ([300, 1], [1, 1]),
])
def test_queries_of_their_own(nq, nk, causal, window, sinks):
    """Query rows other than the keys' rows: more queries than keys leaves rows that see nothing."""
    q, k, v, dout, qo, ko = _inputs(nq, nk, 6, 2, 64, BF16, 40)
    _check(q, k, v, dout, qo, ko, causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("H,G", [(1, 1), (5, 5), (8, 1), (12, 4), (16, 2), (33, 3), (40, 1)])
def test_shared_heads(H, G):
    for nq, nk in (([150, 40], [150, 40]), ([1, 1], [333, 64])):
        q, k, v, dout, qo, ko = _inputs(nq, nk, H, G, 64, BF16, 50 + H)
        _check(q, k, v, dout, qo, ko, causal=True)


def test_many_events():
    """More events than one planning pass takes, empty ones among them."""
    g = torch.Generator().manual_seed(1)
    sizes = torch.randint(0, 7, (5000,), generator=g).tolist()
    sizes[2500] = 150
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 1, 1, 16, BF16, 60)
    out, lse = fps.attention_forward(q, k, v, qo)
    ev = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(sizes, device="cuda"))
    same = ev[:, None] == ev[None]
    Q, K, V, dO = (t.detach()[:, 0].double() for t in (q, k, v, dout))
    S = (Q @ K.T * 0.25).masked_fill(~same, float("-inf"))
    P = torch.softmax(S, 1)
    O = P @ V
    tol = 4 * 2.0 ** -8  # a few roundings of values near 1
    assert float((out[:, 0].double() - O).abs().max()) <= tol * float(V.abs().max())
    dq, dk, dv = fps.attention_backward(dout, q, k, v, out, lse, qo)
    dS = P * (dO @ V.T - (dO * O).sum(1, keepdim=True)) * 0.25
    for got, want in ((dq, dS @ K), (dk, dS.T @ Q), (dv, P.T @ dO)):
        assert float((got[:, 0].double() - want).norm() / want.norm()) <= 2.0 ** -7


def test_scale_and_large_scores():
    """Scores up to some hundreds: the running maximum moves between key tiles."""
    sizes = [520]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 2, 2, 64, BF16, 70)
    k *= torch.linspace(0.1, 6.0, 520, device="cuda")[:, None, None].to(BF16)
    _check(q, k, v, dout, qo, ko, scale=0.9)
    _check(q, k.flip(0).contiguous(), v, dout, qo, ko, scale=0.9)
    _check(q, k, v, dout, qo, ko, scale=1e-4)


def test_strided_inputs():
    """Heads of a fused projection, and tensors with heads before rows."""
    sizes = [140, 60, 9]
    T, D = sum(sizes), 64
    rows, qo = _rand((T, 8, D), 80), _off(sizes)
    dout = _rand((T, 4, D), 81)
    _check(rows[:, :4], rows[:, 4:6], rows[:, 6:], dout, qo, qo)
    hq, hk, hv, hd = (_rand((n, T, D), 82 + n).transpose(0, 1) for n in (4, 2, 2, 4))
    _check(hq, hk, hv, hd, qo, qo, causal=True)
    wide = _rand((T, 4, 2 * D), 83)
    _check(wide[:, :, :D], wide[:, :2, D:], wide[:, 2:, D:], dout, qo, qo)
    _check(rows[:, :1], rows[:, 4:5], rows[:, 6:7], dout[:, :1], qo, qo)


def test_rows_behind_the_last_event():
    sizes = [100, 30]
    for pad in (1, 40, 300):
        q, k, v, dout, qo, ko = _inputs(sizes, sizes, 2, 2, 64, BF16, 90, tail=pad)
        for t in (q, k, v, dout):
            t[130:] = float("nan")
        want = attention(q, k, v, qo, qo)
        _check(q, k, v, dout, qo, qo)
        assert bool((fps.packed_attention(q, k, v, qo)[130:] == 0).all())
        out = torch.full_like(q, 7.0)
        fps.attention_forward(q, k, v, qo, out=out)
        assert_within(out[:130], tuple(x[:130] for x in want["out"]), "out")
        assert bool((out[130:] == 7.0).all())


def test_nonfinite_values_stay_in_their_event():
    sizes = [50, 70, 128, 20, 129]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 2, 1, 64, BF16, 100)
    clean = fps.attention_backward(dout, q, k, v, *fps.attention_forward(q, k, v, qo), qo)
    ref = fps.attention_forward(q, k, v, qo)[0]
    for bad in (float("nan"), float("inf")):
        q2, k2, v2, d2 = (t.clone() for t in (q, k, v, dout))
        for t in (q2, k2, v2, d2):
            t[50:120] = bad
            t[248:268] = bad
        out, lse = fps.attention_forward(q2, k2, v2, qo)
        got = fps.attention_backward(d2, q2, k2, v2, out, lse, qo)
        for rows in (slice(0, 50), slice(120, 248), slice(268, 397)):
            assert torch.equal(out[rows], ref[rows])
            for a, b in zip(got, clean):
                assert torch.equal(a[rows], b[rows])


def test_same_bits_twice_and_streams():
    sizes = [900, 128, 40, 260]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 4, 2, 64, BF16, 110)
    kw = dict(window=50, sinks=200)
    first = fps.attention_forward(q, k, v, qo, **kw)
    grads = fps.attention_backward(dout, q, k, v, *first, qo, **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o = fps.attention_forward(q, k, v, qo, **kw)
            got.append((o, fps.attention_backward(dout, q, k, v, *o, qo, **kw)))
    torch.cuda.synchronize()
    for o, g in got:
        assert all(torch.equal(a, b) for a, b in zip(o, first))
        assert all(torch.equal(a, b) for a, b in zip(g, grads))


@pytest.mark.parametrize("D", [64, 128])
def test_same_bits_many_times(D):
    """Events whose last tile holds few rows, over and over: no tile is touched while another still reads it."""
    g = torch.Generator().manual_seed(3)
    sizes = [128 * int(a) + int(b) for a, b in zip(torch.randint(1, 8, (48,), generator=g), torch.randint(1, 80, (48,), generator=g))]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 8, 2, D, F16, 115)
    kw = dict(causal=True, window=300, sinks=4)
    want = attention(q, k, v, qo, qo, dout=dout, **kw)
    first = None
    for _ in range(12):
        out, lse = fps.attention_forward(q, k, v, qo, **kw)
        got = (out, lse, *fps.attention_backward(dout, q, k, v, out, lse, qo, **kw))
        if first is None:
            first = got
            for t, name in zip(got, ("out", "lse", "dq", "dk", "dv")):
                assert_within(t, want[name], name)
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_autograd_and_differences():
    sizes = [90, 33]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 4, 2, 64, F16, 120)
    want = attention(q, k, v, qo, qo, dout=dout, causal=True)
    for t in (q, k, v):
        t.requires_grad_(True)
    out = fps.packed_attention(q, k, v, qo, causal=True)
    (out * dout).sum().backward()
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        assert_within(t.grad, want[name], name)
    # differences of the float64 reference along a direction
    d = [_rand(t.shape, 130 + i, torch.float64) for i, t in enumerate((q, k, v))]
    eps = 1e-4

    def value(sign):
        t = [x.detach().double() + sign * eps * y for x, y in zip((q, k, v), d)]
        return (_dense(*t, sizes) * dout.double()).sum()

    slope = (value(1) - value(-1)) / (2 * eps)
    mine = sum((t.grad.double() * y).sum() for t, y in zip((q, k, v), d))
    size = sum((t.grad.double() * y).norm() for t, y in zip((q, k, v), d))
    assert abs(float(slope - mine)) <= 2.0 ** -8 * float(size)
    # an expanded incoming gradient
    q2 = q.detach().clone().requires_grad_(True)
    fps.packed_attention(q2, k.detach(), v.detach(), qo, causal=True).sum().backward()
    ones = attention(q.detach(), k.detach(), v.detach(), qo, qo, dout=torch.ones_like(dout), causal=True)
    assert_within(q2.grad, ones["dq"], "dq")


def _dense(q, k, v, sizes):
    outs, a = [], 0
    for n in sizes:
        Q, K, V = q[a:a + n], k[a:a + n].repeat_interleave(2, 1), v[a:a + n].repeat_interleave(2, 1)
        S = torch.einsum("ihd,jhd->hij", Q, K) / math.sqrt(q.shape[2])
        S = S.masked_fill(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(S, -1), V))
        a += n
    return torch.cat(outs)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed on other values and other offsets of the same shapes."""
    sizes = [128, 77, 300]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 2, 2, 64, BF16, 140)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def step():
        out, lse = fps.attention_forward(q, k, v, qo, workspace=ws)
        return (out, *fps.attention_backward(dout, q, k, v, out, lse, qo, workspace=ws2))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for s2 in (sizes, [5, 490, 10], [505, 0, 0], [100, 100, 100]):
        qo.copy_(_off(s2))
        q.copy_(_rand(q.shape, 150 + s2[0]))
        graph.replay()
        want = attention(q, k, v, qo, qo, dout=dout)
        for g, name in zip(got, ("out", "dq", "dk", "dv")):
            assert_within(g, want[name], name)


def test_bad_offsets_are_reported():
    sizes = [40, 60, 30]
    q, k, v, dout, qo, ko = _inputs(sizes, sizes, 2, 2, 64, BF16, 160)
    nb = 1 << 24
    for bad in ([0, 40, 30, 130], [0, 40, 100, 131], [-8, 40, 100, 130], [0, 1 << 40, 100, 130]):
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        off = torch.tensor(bad, dtype=torch.int64, device="cuda")
        out, lse = fps.attention_forward(q, k, v, off, workspace=ws)
        with pytest.raises(_lib.FpsError):
            fps.device_status(ws)
        fps.attention_backward(dout, q, k, v, out, torch.zeros_like(lse), off, workspace=ws)
        with pytest.raises(_lib.FpsError):
            fps.device_status(ws)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    fps.attention_forward(q, k, v, qo, workspace=ws)
    fps.device_status(ws)


@pytest.mark.parametrize("sizes,hint", [([128, 5, 77, 128], 128), ([256, 100, 3], 256), ([64, 1, 30], 64), ([20, 32, 7], 32), ([1, 1, 1], 1)])
def test_with_the_longest_event_known(sizes, hint):
    for D in (32, 64, 128):
        q, k, v, dout, qo, ko = _inputs(sizes, sizes, 4, 2, D, BF16, 170)
        _check(q, k, v, dout, qo, ko, max_tokens=hint)
        _check(q, k, v, dout, qo, ko, max_tokens=hint, window=9, sinks=2, causal=True)


def test_event_above_the_known_longest_is_reported():
    q, k, v, dout, qo, ko = _inputs([300, 20], [300, 20], 2, 2, 64, BF16, 180)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    out, lse = fps.attention_forward(q, k, v, qo, workspace=ws, max_tokens=128)
    with pytest.raises(_lib.FpsError):
        fps.device_status(ws)
    fps.attention_backward(dout, q, k, v, out, lse, qo, workspace=ws, max_tokens=128)
    with pytest.raises(_lib.FpsError):
        fps.device_status(ws)


def test_no_rows():
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    for n in (0, 5):
        q, k, v = (_rand((n, 2, 64), 190) for _ in range(3))
        out, lse = fps.attention_forward(q, k, v, off)
        assert bool((out == 0).all())
        assert all(bool((g == 0).all()) for g in fps.attention_backward(_rand((n, 2, 64), 191), q, k, v, out, lse, off))
    # keys without queries and queries without keys
    q, k = _rand((3, 2, 64), 192), _rand((0, 2, 64), 193)
    out, lse = fps.attention_forward(q, k, k, _off([3]), _off([0]))
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    dq, dk, dv = fps.attention_backward(q, q, k, k, out, lse, _off([3]), _off([0]))
    assert bool((dq == 0).all()) and dk.shape == k.shape
    out, lse = fps.attention_forward(k, q, q, _off([0]), _off([3]))
    dq, dk, dv = fps.attention_backward(k, k, q, q, out, lse, _off([0]), _off([3]))
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("H,G", [(2, 2), (6, 2)])
def test_runs_of_events_without_pairs(H, G):
    """Several events in a row without queries, or without keys, between others, short and long: their gradients are 0."""
    g = torch.Generator().manual_seed(2)
    nq, nk = [], []
    for _ in range(60):
        for _ in range(int(torch.randint(0, 7, (1,), generator=g))):
            n = int(torch.randint(1, 400, (1,), generator=g))
            a, b = [(0, n), (n, 0), (0, 0)][int(torch.randint(0, 3, (1,), generator=g))]
            nq.append(a)
            nk.append(b)
        n = int(torch.randint(1, 260, (1,), generator=g))
        nq.append(n)
        nk.append(n)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    for D in (64, 128):
        q, k, v, dout, qo, ko = _inputs(nq, nk, H, G, D, BF16, 210)
        _check(q, k, v, dout, qo, ko)
        out, lse = fps.attention_forward(q, k, v, qo, ko, workspace=ws)
        fps.device_status(ws)
        fps.attention_backward(dout, q, k, v, out, lse, qo, ko, workspace=ws)
        fps.device_status(ws)  # no wait ran out


def test_tokens_to_attention():
    """The run a model makes: tokenize, pack, project, turn by the centroids, attend, gradients, summary query."""
    import workloads
    b = workloads.make_workload("c0")
    dev = "cuda"
    coords, feats, offsets = (torch.from_numpy(x).to(dev) for x in (b.coords, b.feats, b.offsets))
    tok = fps.fps_tokenize(coords, feats, offsets, K=b.K)
    packed, doc, tok_off = fps.pack_tokens(tok["pooled"], offsets=offsets)
    cent, _, _ = fps.pack_tokens(tok["centroids"], offsets=offsets)
    H, D = 4, 64
    w = _rand((feats.shape[1], 3 * H * D), 200, torch.float32).requires_grad_(True)
    qkv = (packed @ w).to(BF16).view(-1, 3 * H, D)
    table = fps.RotaryTable((16, 16, 16, 16), axis_scale=(0.1, 0.1, 0.1, 0.03))
    qk = fps.apply_rotary(qkv[:, :2 * H], cent, table)
    out = fps.packed_attention(qk[:, :H], qk[:, H:], qkv[:, 2 * H:], tok_off, max_tokens=b.K)
    want = attention(qk[:, :H].detach(), qk[:, H:].detach(), qkv[:, 2 * H:].detach(), tok_off, tok_off)
    assert_within(out, want["out"], "out")
    out.float().square().sum().backward()
    assert bool(w.grad.isfinite().all()) and float(w.grad.abs().max()) > 0
    one = torch.arange(b.B + 1, dtype=torch.int64, device=dev)
    summary = _rand((b.B, H, D), 201)
    s = fps.packed_attention(summary, qk[:, H:].detach(), qkv[:, 2 * H:].detach(), one, kv_offsets=tok_off)
    want = attention(summary, qk[:, H:].detach(), qkv[:, 2 * H:].detach(), one, tok_off)
    assert_within(s, want["out"], "summary")


@pytest.mark.parametrize("causal,window,sinks", [(False, -1, 0), (True, -1, 0), (True, 50, 4), (False, 300, 130), (False, 0, 1), (True, 20, 5000)])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16), (40, F16), (88, BF16)])
def test_key_tiles_in_pieces(causal, window, sinks, D, dtype):
    """Key tiles that so many queries of so many heads see that their work is
    cut into pieces; beside them events whose tiles are whole, and none."""
    nq, nk = [1500, 3, 0, 200, 1000], [1500, 40, 0, 200, 130]
    q, k, v, dout, qo, ko = _inputs(nq, nk, 8, 2, D, dtype, 110)
    _check(q, k, v, dout, qo, ko, causal=causal, window=window, sinks=sinks)
    _check(q, k, v, dout, qo, ko, causal=causal, window=window, sinks=sinks, max_tokens=1500)


@pytest.mark.parametrize("D,dtype", [(8, BF16), (24, F16), (56, BF16), (72, F16), (104, BF16), (128, F16)])
@pytest.mark.parametrize("causal,window,sinks", [(False, -1, 0), (True, 700, 3), (False, 90, 600), (True, 0, 0)])
def test_few_queries_of_long_events(D, dtype, causal, window, sinks):
    """One to three queries of an event whose keys take several parts."""
    nq, nk = [1, 2, 3, 1, 1, 0, 1], [3000, 1300, 511, 0, 64, 7, 1]
    q, k, v, dout, qo, ko = _inputs(nq, nk, 8, 2, D, dtype, 120)
    _check(q, k, v, dout, qo, ko, causal=causal, window=window, sinks=sinks)


def test_few_queries_leave_other_rows():
    """Output rows behind the last event stay, also where no tile kernel runs."""
    q, k, v, dout, qo, ko = _inputs([1] * 5, [40, 0, 2000, 1, 300], 4, 4, 64, BF16, 130, tail=3)
    want = attention(q, k, v, qo, ko)
    out = torch.full_like(q, 7.0)
    fps.attention_forward(q, k, v, qo, ko, out=out)
    assert_within(out[:5], tuple(x[:5] for x in want["out"]), "out")
    assert bool((out[5:] == 7.0).all())


def test_gradient_of_a_broadcast():
    """An output gradient without memory of its own, as sum() makes it."""
    sizes = [150, 20]
    q, k, v, _, qo, _ = _inputs(sizes, sizes, 4, 2, 64, BF16, 140)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    fps.packed_attention(*leaves, qo).sum().backward()
    want = attention(q, k, v, qo, qo, dout=torch.ones_like(q))
    for t, name in zip(leaves, ("dq", "dk", "dv")):
        assert_within(t.grad, want[name], name)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (64, F16), (128, BF16), (40, F16)])
@pytest.mark.parametrize("sizes", [[1] * 9, [200, 1, 300], [128] * 3])
def test_queries_that_see_one_key(sizes, D, dtype):
    """A query that sees one key moves nothing: its weight is 1 whatever the score.

    dS = P (dP - D) is then what two float32 sums of D <= 128 products differ
    by, and the weight's distance from 1: below 2^-16 of sum |dO V| (256
    roundings of 2^-24) each.  dQ = scale dS K, and dK sums the group's; 2^-25
    is half of fp16's smallest step.
    """
    q, k, v, dout, qo, _ = _inputs(sizes, sizes, 4, 2, D, dtype, 150)
    out, lse = fps.attention_forward(q, k, v, qo, causal=True, window=0)
    assert_within(out, attention(q, k, v, qo, qo, causal=True, window=0)["out"], "out")
    dq, dk, dv = fps.attention_backward(dout, q, k, v, out, lse, qo, causal=True, window=0)
    K, V = (t.repeat_interleave(2, 1).double() for t in (k, v))
    dS = 2 * 2.0 ** -16 * (dout.double() * V).abs().sum(2, keepdim=True) * D ** -0.5
    assert bool((dq.double().abs() <= dS * K.abs() + 2.0 ** -25).all())
    limit = (dS * q.double().abs()).unflatten(1, (2, 2)).sum(2)
    assert bool((dk.double().abs() <= limit + 2.0 ** -25).all())


@pytest.mark.parametrize("causal,window,sinks", [(True, -1, 0), (True, 1, 0), (False, 1, 1), (True, 6, 3), (False, -1, 0)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradient_error_of_short_rows(causal, window, sinks, D, dtype):
    """Error of a whole gradient, in norms: that of rounding dS (or P) and then
    the gradient, and little more.  Rounding normal values costs 0.432 half
    steps, sqrt(E ulp(x)^2 / 12) / (eps / 2); two add in squares to 0.61, and
    D from the rounded output at 17 keys or more adds 2 / 16 of one's square:
    0.432 sqrt(2 + 1 / 8) = 0.63.  Above 0.65 something else is rounded.
    """
    sizes = [5, 2, 9, 300, 1, 40, 3] * 6 if window >= 0 or causal else [2, 3, 4, 5, 6] * 20
    q, k, v, dout, qo, _ = _inputs(sizes, sizes, 4, 2, D, dtype, 160)
    mask = dict(causal=causal, window=window, sinks=sinks)
    got = fps.attention_backward(dout, q, k, v, *fps.attention_forward(q, k, v, qo, **mask), qo, **mask)
    want = attention(q, k, v, qo, qo, dout=dout, **mask)
    for g, name in zip(got, ("dq", "dk", "dv")):
        w = want[name][0]
        assert float((g.double() - w).norm() / w.norm()) <= torch.finfo(dtype).eps / 2 * 0.65, name
