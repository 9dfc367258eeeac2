"""Measured cases of the packed-token transformer operators: multi-axis rotary
positions and block-diagonal attention (sliding window, sink tokens), each in
a plain torch form and as the framework's calls.

A case is one call as a user makes it: a batch of events in the packed token
layout (``pack_tokens``), the token rows of event b being ``tok_offsets[b] ..
tok_offsets[b + 1] - 1``.

Rotary positions: pair p of a head belongs to one coordinate axis a(p) and
has a frequency w_p; with theta = position[t, a(p)] * w_p,

    y1 = x1 cos(theta) - x2 sin(theta),   y2 = x2 cos(theta) + x1 sin(theta).

Attention, per event and head: query i of nq stands at position
p = i + nk - nq of the event's nk keys and sees key j when

    (|p - j| <= window, or window < 0, or j < sinks) and (j <= p if causal),

out_i = sum_j softmax_j(scale * q_i . k_j) v_j, and 0 for a query that sees
no key.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_ROWS = 256  # query rows of one block of the plain attention
_SCORES = 1 << 29  # scores of one chunk of the plain attention (2 GiB in 32 bits)


# ------------------------------------------------------------------ the cases


def _rotary(name, **kw):
    c = dict(name=name, op="rotary", direction="forward", dtype="bf16", kind="uniform", events=64, lo=5, hi=400, K=128,
             size_seed=0, heads=24, spare_heads=0, head_dim=64, axis_dims="16,16,16,16", interleaved=False, time_scale=0.03)
    c.update(kw)
    return c


def _attention(name, **kw):
    c = dict(name=name, op="attention", direction="forward", dtype="bf16", kind="uniform", events=64, lo=5, hi=400, K=128,
             size_seed=0, queries=0, heads=12, kv_heads=12, head_dim=64, causal=False, window=-1, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # one event at the smallest call: the queries and keys of its 128 tokens
        _rotary("rotary_event", events=1, lo=128, hi=128),
        # the small-event batch (4096 events, K = 128): query and key heads of a fused q, k, v row, so rows are strided
        _rotary("rotary_small_events", events=4096, size_seed=4, heads=24, spare_heads=12),
        # training in 32 bits, track events, a head whose rotated part is not the whole of it, times in ns unscaled
        _rotary("rotary_tracks_train", direction="train", dtype="fp32", kind="lognormal", events=256, lo=8, hi=20000, K=128,
                size_seed=2, heads=10, head_dim=72, axis_dims="12,12,12,24", interleaved=True, time_scale=1.0),
        # one summary query over one event's 128 tokens: the smallest serving call
        _attention("attention_summary_event", events=1, lo=128, hi=128, queries=1),
        # one summary query for each of 8 bright showers of 50k-200k pulses, heads sharing keys
        _attention("attention_summary_showers", events=8, lo=50000, hi=200000, K=0, size_seed=3, queries=1, heads=12, kv_heads=4),
        # 64 track events, ragged below K = 128
        _attention("attention_tracks", kind="lognormal", events=64, lo=8, hi=20000, size_seed=1),
        # the small-event batch at its full width
        _attention("attention_small_events", events=4096, size_seed=4),
        # the same in training: forward and the three gradients, K = 256 (two key tiles), half the events
        _attention("attention_small_events_train", direction="train", events=2048, size_seed=5, K=256, heads=8, kv_heads=8, lo=5, hi=800),
        # training at K = 128
        _attention("attention_events_train", direction="train", events=2048, size_seed=6, heads=12, kv_heads=12),
        # every pulse of 8 showers in time order: a window on both sides and the first pulses visible to all
        _attention("attention_window_showers", events=8, lo=50000, hi=200000, K=0, size_seed=3, heads=8, kv_heads=8, window=128, sinks=16),
        # pulses of track events, causal window with sinks, shared heads, 128-wide heads, 16-bit floats, training
        _attention("attention_window_train", direction="train", dtype="fp16", kind="lognormal", events=64, lo=8, hi=20000, K=0,
                   size_seed=7, heads=8, kv_heads=2, head_dim=128, causal=True, window=511, sinks=4),
        # whole causal attention over few long events, training
        _attention("attention_causal_train", direction="train", events=4, lo=4000, hi=9000, K=0, size_seed=8, heads=16, kv_heads=4,
                   head_dim=128, causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    seed = rng.randrange(1 << 30)

    def events(most, values):  # so many that one tensor of a case stays below `values`
        return _log_int(rng, 1, max(1, min(most, int(values))))

    if rng.random() < 0.3:
        pairs = [rng.choice((2, 4, 6, 8, 10, 12, 16, 20)) for _ in range(4)]
        heads, dim = rng.randint(1, 24), 2 * sum(pairs) + rng.choice((0, 0, 2, 8))
        hi, K = _log_int(rng, 8, 600), rng.choice((32, 64, 100, 128, 256))
        return _rotary("", direction=rng.choice(("forward", "train")), dtype=rng.choice(("bf16", "fp16", "fp32")),
                       events=events(2000, 2.2e8 / (min(hi, K) * heads * dim)), lo=rng.choice((1, 5)), hi=hi, K=K, size_seed=seed,
                       heads=heads, spare_heads=rng.choice((0, 0, 3, 12)), head_dim=dim, axis_dims=",".join(str(2 * p) for p in pairs),
                       interleaved=rng.random() < 0.5, time_scale=rng.choice((0.01, 0.1, 1.0)))
    kv_heads = rng.choice((1, 2, 3, 4, 8, 12))
    heads = kv_heads * rng.choice([g for g in (1, 1, 2, 3, 4, 8) if kv_heads * g <= 16])
    dim = rng.choice((32, 48, 64, 64, 80, 96, 128, 128))
    common = dict(dtype=rng.choice(("bf16", "fp16")), heads=heads, kv_heads=kv_heads, head_dim=dim, size_seed=seed)
    shape = rng.random()
    if shape < 0.2:  # summary queries
        hi = _log_int(rng, 64, 100000)
        return _attention("", events=events(512, 9e8 / (hi * kv_heads * dim)), lo=1, hi=hi, K=0, queries=rng.choice((1, 1, 2)), **common)
    direction = rng.choice(("forward", "train"))
    if shape < 0.6:  # tokens of many events
        hi, K = _log_int(rng, 8, 600), rng.choice((32, 64, 100, 128, 200, 256))
        n = events(1500, 2.4e8 / (min(hi, K) * heads * dim))
        return _attention("", direction=direction, events=n, lo=rng.choice((0, 1, 5)) if n >= 8 else 1, hi=hi, K=K, **common)
    hi = _log_int(rng, 100, 6000)  # longer events, windows and sinks
    return _attention("", direction=direction, events=events(64, 16000 / hi), lo=1, hi=hi, K=0, causal=rng.random() < 0.5,
                      window=rng.choice((-1, _log_int(rng, 1, 1000))), sinks=rng.choice((0, 1, 4, 16, rng.randint(1, 200))), **common)


def _sizes(case):
    """Tokens of each event, from the case alone."""
    r = random.Random(case["size_seed"])
    got = []
    for _ in range(case["events"]):
        n = round(r.lognormvariate(math.log(300.0), 1.0)) if case["kind"] == "lognormal" else r.randint(case["lo"], case["hi"])
        n = min(max(n, case["lo"]), case["hi"])
        got.append(min(n, case["K"]) if case["K"] else n)
    return got


def _axis_dims(case):
    return [int(d) for d in case["axis_dims"].split(",")]


def _axis_scale(case):
    return (0.1, 0.1, 0.1, case["time_scale"])


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(np.asarray(sizes, np.int64))]).astype(np.int64)


# ------------------------------------------------------------------ the inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, grad=False):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype).requires_grad_(grad)

    nk = _sizes(case)
    train = case["direction"] == "train"
    s = {"case": dict(case), "nk": nk}
    T, D = sum(nk), case["head_dim"]
    if case["op"] == "rotary":
        # positions as the detector gives them: metres within the array, times in ns
        p = torch.rand((T, 4), generator=g, device="cuda", dtype=torch.float32)
        lo, hi = torch.tensor([[-570.0, -520.0, -501.5, 0.0], [570.0, 520.0, 501.5, 5000.0]], device="cuda")
        s["positions"] = lo + (hi - lo) * p
        H = case["heads"]
        rows = normal(T, H + case["spare_heads"], D)
        s["x"] = rows[:, :H].requires_grad_(train)
        if train:
            s["dy"] = normal(T, H, D)
        if own:
            import farthest_point_sampling_b200 as fps
            s["table"] = fps.RotaryTable(_axis_dims(case), axis_scale=_axis_scale(case), interleaved=case["interleaved"])
        return s
    nq = [case["queries"]] * len(nk) if case["queries"] else nk
    s["nq"] = nq
    s["q"] = normal(sum(nq), case["heads"], D, grad=train)
    s["k"] = normal(T, case["kv_heads"], D, grad=train)
    s["v"] = normal(T, case["kv_heads"], D, grad=train)
    if train:
        s["dout"] = normal(sum(nq), case["heads"], D)
    s["kv_offsets"] = torch.from_numpy(_offsets(nk)).cuda()
    s["q_offsets"] = torch.from_numpy(_offsets(nq)).cuda() if case["queries"] else s["kv_offsets"]
    # what the program knows of its batch on the host: the longest event
    s["max_tokens"] = max(nk)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    train = case["direction"] == "train"
    if case["op"] == "rotary":
        if own:
            import farthest_point_sampling_b200 as fps
            if not train:
                return fps.rotary_embed(s["x"], s["positions"], s["table"])
            y = fps.apply_rotary(s["x"], s["positions"], s["table"])
            return [y, torch.autograd.grad(y, s["x"], s["dy"])[0]]
        x = s["x"].detach()
        y = _plain_rotary(case, x, s["positions"], 1.0)
        return [y, _plain_rotary(case, s["dy"], s["positions"], -1.0)] if train else y
    if own:
        import farthest_point_sampling_b200 as fps
        out = fps.packed_attention(s["q"], s["k"], s["v"], s["q_offsets"], kv_offsets=s["kv_offsets"], causal=case["causal"],
                                   window=case["window"], sinks=case["sinks"], max_tokens=s["max_tokens"])
        if not train:
            return out
        return [out, *torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["dout"])]
    return _plain_attention(case, s)


def _frequencies(case):
    """(axis, radians per unit) of every rotated pair, in 64 bits."""
    axis, freq = [], []
    for a, (d, scale) in enumerate(zip(_axis_dims(case), _axis_scale(case))):
        axis += [a] * (d // 2)
        freq += [scale * 10000.0 ** (-i / (d // 2)) for i in range(d // 2)]
    return axis, freq


def _plain_rotary(case, x, positions, sign):
    axis, freq = _frequencies(case)
    R = len(axis)
    theta = positions.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(theta).float()[:, None], (sign * torch.sin(theta)).float()[:, None]
    y = x.float()
    rot, rest = y[..., : 2 * R], y[..., 2 * R:]
    if case["interleaved"]:
        x1, x2 = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = rot[..., :R], rot[..., R:]
        rot = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((rot, rest), -1).to(x.dtype)


def _plain_attention(case, s):
    """Blocks of up to _ROWS queries of one event, each against the keys that
    some query of it sees, in chunks of many blocks at once: as many as keep
    the scores of a chunk within _SCORES."""
    q, k, v = s["q"].detach(), s["k"].detach(), s["v"].detach()
    dev = q.device
    (Tq, H, D), G = q.shape, k.shape[1]
    train = case["direction"] == "train"
    nq, nk = np.asarray(s["nq"], np.int64), np.asarray(s["nk"], np.int64)
    q_off, k_off = _offsets(nq), _offsets(nk)
    w, sinks, causal = case["window"], case["sinks"], case["causal"]
    rows = int(min(_ROWS, max(nq.max(initial=1), 1)))
    # every block: its event, its first query there, the span lo..hi of its keys and the sinks before it
    per = -(-nq // rows)
    ev = np.repeat(np.arange(len(nq)), per)
    first = (np.arange(len(ev)) - np.repeat(np.cumsum(per) - per, per)) * rows
    p0 = first + nk[ev] - nq[ev]
    p1 = np.minimum(first + rows, nq[ev]) - 1 + nk[ev] - nq[ev]
    lo = np.zeros_like(p0) if w < 0 else np.maximum(0, p0 - w)
    hi = np.minimum(nk[ev], p1 + 1 + (0 if causal else w)) if w >= 0 or causal else nk[ev]
    sink = np.minimum(sinks, nk[ev])
    joined = sink >= lo
    hi = np.where(joined, np.maximum(hi, sink), hi)
    lo, sink = np.where(joined, 0, lo), np.where(joined, 0, sink)
    span = np.maximum(hi - lo, 0) + sink
    wide = int(max(span.max(initial=1), 1))
    step = max(1, _SCORES // (rows * wide * H + 2 * wide * G * D))
    scale = D ** -0.5
    out = torch.zeros((Tq, H, D), device=dev, dtype=q.dtype)
    if train:
        dq = torch.zeros_like(out)
        dk, dv = (torch.zeros(k.shape, device=dev, dtype=torch.float32) for _ in range(2))
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    for c in range(0, len(ev), step):
        b = slice(c, c + step)
        i = on(first[b])[:, None] + torch.arange(rows, device=dev)
        c_nq, c_nk = on(nq[ev[b]])[:, None], on(nk[ev[b]])[:, None]
        real = i < c_nq
        qi = torch.where(real, i + on(q_off[ev[b]])[:, None], 0)
        n = torch.arange(int(max(span[b].max(), 1)), device=dev)
        j = torch.where(n < on(sink[b])[:, None], n, n - on(sink[b])[:, None] + on(lo[b])[:, None])
        held = n < on(span[b])[:, None]
        kj = torch.where(held, j + on(k_off[ev[b]])[:, None], 0)
        pos = (i + c_nk - c_nq)[:, :, None]
        see = torch.ones((), dtype=torch.bool, device=dev) if w < 0 else ((pos - j[:, None]).abs() <= w) | (j[:, None] < sinks)
        if causal:
            see = see & (j[:, None] <= pos)
        see = (see & held[:, None] & real[:, :, None])[:, None, None]
        Q = q[qi].float().view(len(i), rows, G, H // G, D).permute(0, 2, 3, 1, 4)  # [block, kv head, of its group, row, D]
        K, V = (x[kj].float().transpose(1, 2)[:, :, None] for x in (k, v))
        S = (Q * scale) @ K.transpose(-1, -2)
        S = torch.where(see, S, float("-inf"))
        top = S.amax(-1, keepdim=True)
        P = torch.exp(S - torch.where(top == float("-inf"), 0.0, top))
        total = P.sum(-1, keepdim=True)
        P = P / torch.where(total == 0, 1.0, total)
        O = P @ V
        put = lambda x: x.permute(0, 3, 1, 2, 4).reshape(len(i), rows, H, D)[real]  # noqa: E731
        out[qi[real]] = put(O).to(q.dtype)
        if train:
            dO = s["dout"][qi].float().view(len(i), rows, G, H // G, D).permute(0, 2, 3, 1, 4)
            dP = dO @ V.transpose(-1, -2)
            dS = P * (dP - (dO * O).sum(-1, keepdim=True))
            dq[qi[real]] = put(dS @ K * scale).to(q.dtype)
            dV = (P.transpose(-1, -2) @ dO).sum(2).transpose(1, 2)
            dK = (dS.transpose(-1, -2) @ (Q * scale)).sum(2).transpose(1, 2)
            dk.index_add_(0, kj[held], dK[held])
            dv.index_add_(0, kj[held], dV[held])
    return [out, dq, dk.to(k.dtype), dv.to(v.dtype)] if train else out


# ------------------------------------------------------------------ what a pass needs


def _pairs(case):
    """Query-key pairs that see one another, over the events, for one head."""
    total = 0
    w, sinks, causal = case["window"], case["sinks"], case["causal"]
    for nk in _sizes(case):
        nq = case["queries"] or nk
        p = np.arange(nq, dtype=np.int64) + nk - nq
        hi = np.full_like(p, nk)
        if w >= 0 or causal:
            hi = np.minimum(nk, p + 1 + (0 if causal else w))
        hi = np.maximum(hi, 0)
        lo = np.minimum(np.maximum(0, p - w), hi) if w >= 0 else np.zeros_like(p)
        s = np.minimum(min(sinks, nk), np.maximum(p + 1, 0) if causal else nk)
        total += int(((hi - lo) + np.minimum(s, lo) + np.maximum(0, s - hi)).sum())
    return total


def work(case):
    size, T, D = _BYTES[case["dtype"]], sum(_sizes(case)), case["head_dim"]
    train = case["direction"] == "train"
    if case["op"] == "rotary":
        values = T * case["heads"] * D
        turned = T * case["heads"] * sum(_axis_dims(case))
        passes = 2 if train else 1
        return {"bytes": passes * 2 * values * size + T * 16, "flops": passes * 3 * turned}
    Tq = case["queries"] * case["events"] if case["queries"] else T
    moved = 2 * Tq * case["heads"] * D + 2 * T * case["kv_heads"] * D  # q, out, k, v
    # two products forward; four more for the gradients
    return {"bytes": (2 if train else 1) * moved * size, "flops": (12 if train else 4) * D * case["heads"] * _pairs(case)}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    train = case["direction"] == "train"
    if case["op"] == "rotary":
        return _exact_rotary(case, s, train)
    if case["direction"] == "train" and _pairs(case) * case["heads"] * case["head_dim"] > 4e12:
        return None
    heads, group = case["heads"], case["heads"] // case["kv_heads"]
    q, k, v = (s[n].detach().double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    a = b = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        for r0 in range(0, nq if nk else 0, 512):
            r1 = min(nq, r0 + 512)
            pos = torch.arange(r0, r1, device=q.device) + (nk - nq)
            keys = torch.arange(nk, device=q.device)
            if case["window"] >= 0:
                near = (keys >= pos[0] - case["window"]) & (keys <= pos[-1] + case["window"])
                keys = keys[near | (keys < case["sinks"])]
            if not len(keys):
                continue
            t = [q[a + r0:a + r1], k[b + keys], v[b + keys]]
            t = [x.clone().requires_grad_(train) for x in t]
            kk, vv = (x.repeat_interleave(group, 1) for x in t[1:])
            logits = torch.einsum("ihd,jhd->hij", t[0], kk) * case["head_dim"] ** -0.5
            far = (pos[:, None] - keys[None]).abs()
            hidden = (far > case["window"]) & (keys[None] >= case["sinks"]) if case["window"] >= 0 else torch.zeros_like(far, dtype=torch.bool)
            if case["causal"]:
                hidden = hidden | (keys[None] > pos[:, None])
            seen = ~hidden.all(1)
            weight = torch.softmax(logits.masked_fill(hidden & seen[:, None], float("-inf")), -1)
            weight = weight * (seen[:, None] & ~hidden)
            o = torch.einsum("hij,jhd->ihd", weight, vv)
            out[a + r0:a + r1] = o.detach()
            if train:
                got = torch.autograd.grad(o, t, s["dout"][a + r0:a + r1].double())
                grads[0][a + r0:a + r1] = got[0]
                grads[1][b + keys] += got[1]
                grads[2][b + keys] += got[2]
        a, b = a + nq, b + nk
    assert out.shape[1] == heads
    return [out, *grads] if train else out


def _exact_rotary(case, s, train):
    axis, freq = _frequencies(case)
    x, R = s["x"].detach().double(), len(axis)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.stack([s["positions"][:, a].double() * f for a, f in zip(axis, freq)], 1))
    first = [2 * p if case["interleaved"] else p for p in range(R)]
    second = [2 * p + 1 if case["interleaved"] else p + R for p in range(R)]

    def turned(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    y = turned(x, turn)
    return [y, turned(s["dy"].double(), turn.conj())] if train else y
