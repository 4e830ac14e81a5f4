"""The windowed prefill's plain forms in float64 on the CPU: output, row statistic and gradients, each with
the sums of magnitudes that the tests' tolerances are stated in."""

import math

import torch


def allowed(length, n, window, sinks):
    """[length, length] truth values: row i sees key j.  A candidate (i >= n) stands at position n."""
    i, j = torch.arange(length)[:, None], torch.arange(length)[None]
    pos = i.clamp(max=n)
    near = torch.ones_like(pos - j, dtype=torch.bool) if window is None else pos - j < window
    return ((j <= i) & (j < n) & (near | (j < sinks))) | (i == j)


def prefill64(q, k, v, cu, past, window, sinks):
    """out [T, H, D], mag = sum_j p_ij |v_j|, lse [T, H] (base 2); rows outside the segments are NaN."""
    T, H, D = q.shape
    G = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out = torch.full((T, H, D), float("nan"), dtype=torch.float64)
    mag, lse = out.clone(), torch.full((T, H), float("nan"), dtype=torch.float64)
    for b, n in enumerate(past):
        t0, t1 = cu[b], cu[b + 1]
        ok = allowed(t1 - t0, n, window, sinks)
        for h in range(H):
            s = (q[t0:t1, h] @ k[t0:t1, h // G].T / math.sqrt(D)).masked_fill(~ok, -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            out[t0:t1, h] = p @ v[t0:t1, h // G]
            mag[t0:t1, h] = p @ v[t0:t1, h // G].abs()
            lse[t0:t1, h] = z / math.log(2.0)
    return out, mag, lse


# Relative error of a weight before it is rounded (see the tests' notes), and of one rounding to bfloat16.
WEIGHT = 2.0 ** -11
ROUND = 2.0 ** -8


def grads64(q, k, v, dout, cu, past, window, sinks):
    """{name: (gradient, tolerance before the output's rounding)} for dq, dk, dv, float64."""
    T, H, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    scale = 1.0 / math.sqrt(D)
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    g = {"dq": torch.full((T, H, D), float("nan"), dtype=torch.float64)}
    g["dk"] = torch.full((T, Hkv, D), float("nan"), dtype=torch.float64)
    g["dv"] = g["dk"].clone()
    tol = {x: y.clone() for x, y in g.items()}
    for b, n in enumerate(past):
        t0, t1 = cu[b], cu[b + 1]
        ok = allowed(t1 - t0, n, window, sinks)
        for x in ("dk", "dv"):
            g[x][t0:t1] = 0
            tol[x][t0:t1] = 0
        for h in range(H):
            Q, K, V, dO = q[t0:t1, h], k[t0:t1, h // G], v[t0:t1, h // G], dout[t0:t1, h]
            p = torch.softmax((Q @ K.T * scale).masked_fill(~ok, -math.inf), -1)
            O = p @ V
            dS = p * (dO @ V.T - (dO * O).sum(-1, keepdim=True))
            # Dvec from the stored output: its bfloat16 rounding and the forward's own error; the float32 sums
            e_dvec = (dO.abs() * (O.abs() * ROUND + (p @ V.abs()) * (ROUND + WEIGHT))).sum(-1, keepdim=True)
            e_sum = 2.0 ** -16 * (dO.abs() @ V.abs().T)
            e_dS = dS.abs() * (ROUND + WEIGHT) + p * (e_dvec + e_sum)
            g["dv"][t0:t1, h // G] += p.T @ dO
            tol["dv"][t0:t1, h // G] += (p.T @ dO.abs()) * (ROUND + WEIGHT)
            g["dk"][t0:t1, h // G] += scale * dS.T @ Q
            tol["dk"][t0:t1, h // G] += scale * e_dS.T @ Q.abs()
            g["dq"][t0:t1, h] = scale * dS @ K
            tol["dq"][t0:t1, h] = scale * e_dS @ K.abs()
    return {x: (g[x], tol[x]) for x in g}
