"""Attention of packed events in float64, with a bound on how far a kernel's
results may be from it.

The kernels hold scores, sums and gradients in float32 and round the softmax
weights P and the score gradients dS once to the 16-bit type (relative error
u = eps / 2 each) for their matrix products, and each output once more.  With
f = 2^-24 and E the largest sum of |scale q_d k_d| over a visible pair, one
weight's relative error is

    e_p = 2^-20 + 4 f (D + 8) E      (score sum, exponent argument, exp2 and log),

so, per element, with A = sum_j P |v_j|, n the visible keys and s = 2^-24 for
float16 (a weight below the normal range is off by up to 2^-25 of the row's
largest, which is at least 1 / 2 of what it is measured by), 0 for bfloat16,

    |out err|  <= u |out| + (u + 2 e_p + f (n + 8)) A + s sum_j |v_j|
    |dv err|   <= u |dv| + (u + e_p + f (n + 8)) sum_i P |dO_i| + s sum_i |dO_i|
    |dS err|   <= u |dS| + e_p |dS| + P (|delta err| + f (D + 8) sum_d |dO v|)
    |delta err| <= sum_d |dO_d| |out err_d| + f (D + 8) sum_d |dO out|
    |dq err|   <= u |dq| + scale (sum_j |dS err| |k_j| + f (n + 8) sum_j |dS| |k_j| + s max|dS| sum_j |k_j|)

and dk like dq over the queries.  A rounding to float16 below its normal range
is off by up to 2^-25, half the subnormal step, whatever the value: u |x| is
taken as at least that for out, dq, dk and dv.  Second-order terms are below 2^-8 of these
and covered by the factor 1.02.
"""
import torch

F32 = 2.0 ** -24


def visible(nq, nk, causal, window, sinks, device):
    p = torch.arange(nq, device=device)[:, None] + nk - nq
    j = torch.arange(nk, device=device)[None]
    see = torch.ones((nq, nk), dtype=torch.bool, device=device)
    if window >= 0:
        see &= ((p - j).abs() <= window) | (j < sinks)
    if causal:
        see &= j <= p
    return see


def attention(q, k, v, q_off, k_off, dout=None, scale=None, causal=False, window=-1, sinks=0):
    """{"out", "lse", "dq", "dk", "dv"} as (value, bound) pairs in float64; rows of no event are 0 with bound 0."""
    u = torch.finfo(q.dtype).eps / 2
    sub = 2.0 ** -24 if q.dtype == torch.float16 else 0.0
    least = sub / 2
    half = lambda t: (u * t.abs()).clamp_min(least)  # noqa: E731 - the last rounding of an output
    scale = q.shape[2] ** -0.5 if scale is None else scale
    group = q.shape[1] // k.shape[1]
    dev, D = q.device, q.shape[2]
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=dev)  # noqa: E731
    r = {"out": (z(q), z(q)), "lse": (torch.full((q.shape[1], q.shape[0]), float("-inf"), dtype=torch.float64, device=dev),
                                     torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=dev))}
    if dout is not None:
        r.update(dq=(z(q), z(q)), dk=(z(k), z(k)), dv=(z(v), z(v)))
    qo, ko = [int(x) for x in q_off], [int(x) for x in k_off]
    for b in range(len(qo) - 1):
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if nq == 0 or nk == 0:
            continue
        see = visible(nq, nk, causal, window, sinks, dev)
        n_row, n_col = see.sum(1).double()[:, None], see.sum(0).double()[:, None]
        seen = see.any(1)
        for h in range(q.shape[1]):
            g = h // group
            Q, K, V = (t.detach().double() for t in (q[qo[b]:qo[b + 1], h], k[ko[b]:ko[b + 1], g], v[ko[b]:ko[b + 1], g]))
            S = torch.where(see, Q @ K.T * scale, float("-inf"))
            lse = torch.logsumexp(S, 1)
            P = torch.where(see, torch.exp(S - torch.where(seen, lse, 0.0)[:, None]), 0.0)
            E = float(torch.where(see, Q.abs() @ K.abs().T * scale, 0.0).max())
            e_p = 2.0 ** -20 + 4 * F32 * (D + 8) * E
            O = P @ V
            A = P @ V.abs()
            vis = see.double()
            o_err = 1.02 * (half(O) + (u + 2 * e_p + F32 * (n_row + 8)) * A + sub * (vis @ V.abs()))
            rows = slice(qo[b], qo[b + 1])
            r["out"][0][rows, h], r["out"][1][rows, h] = O, o_err
            r["lse"][0][h, rows] = lse
            r["lse"][1][h, rows] = torch.where(seen, 2 * e_p + F32 * (n_row[:, 0] + 8 + 4 * lse.abs()), 0.0)
            if dout is None:
                continue
            dO = dout[rows, h].detach().double()
            keys = slice(ko[b], ko[b + 1])
            delta = (dO * O).sum(1, keepdim=True)
            delta_err = (dO.abs() * o_err).sum(1, keepdim=True) + F32 * (D + 8) * (dO * O).abs().sum(1, keepdim=True)
            dS = P * (dO @ V.T - delta)
            dS_err = (u + e_p) * dS.abs() + P * (delta_err + F32 * (D + 8) * (dO.abs() @ V.abs().T))
            top = float(dS.abs().max())
            dq, dk, dv = scale * dS @ K, scale * dS.T @ Q, P.T @ dO
            r["dq"][0][rows, h] = dq
            r["dq"][1][rows, h] = 1.02 * (half(dq) + scale * (dS_err @ K.abs() + F32 * (n_row + 8) * (dS.abs() @ K.abs()) +
                                                                  sub * max(top, 1.0) * (vis @ K.abs())))
            r["dk"][0][keys, g] += dk
            r["dk"][1][keys, g] += 1.02 * scale * (dS_err.T @ Q.abs() + F32 * (group * n_col + 8) * (dS.abs().T @ Q.abs()) +
                                                   sub * max(top, 1.0) * (vis.T @ Q.abs()))
            r["dv"][0][keys, g] += dv
            r["dv"][1][keys, g] += 1.02 * ((u + e_p + F32 * (group * n_col + 8)) * (P.T @ dO.abs()) + sub * (vis.T @ dO.abs()))
        if dout is not None and b >= 0:
            keys = slice(ko[b], ko[b + 1])
            for name in ("dk", "dv"):  # the one rounding of the sum over a group's heads
                r[name][1][keys] += 1.02 * half(r[name][0][keys])
    return r


def assert_within(got, want, name):
    value, bound = want
    got = got.detach().double()
    both_inf = torch.isinf(value) & (got == value)
    err = torch.where(both_inf, 0.0, (got - value).abs())
    bad = ~(err <= bound)
    if bool(bad.any()):
        at = tuple(int(x) for x in torch.nonzero(bad)[0])
        worst = float((err / bound.clamp_min(1e-300)).nan_to_num(float("inf")).max())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound (worst {worst:.3g} times), first at {at}: "
                             f"got {float(got[at])}, want {float(value[at])} within {float(bound[at])}")
