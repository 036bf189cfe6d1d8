"""The operators of a W8A8 Mamba-2 layer around the scan, in float64 — TEST INFRASTRUCTURE ONLY.

* `norm_codes`: RMSNorm u = v w / sqrt(mean v² + eps) of each token with one symmetric step per
  token, s = max|u| / 127, and the real-valued positions u / s whose rounding gives the codes;
* `gate`: v = y z / (1 + exp(-z));
* `matmul`: s_t[t] s_w[n] Σ_k q[t,k] Wq[n,k] + bias[n] from the exact integer sums;
* `conv`: the causal depthwise convolution of the rows' inputs behind their state's, SiLU,
  softplus of dt, zeros behind a row's last token and the row's next state.  Written token by
  token from the definition (no window arithmetic shared with the kernels).
"""
from __future__ import annotations

import numpy as np


def gate(y, z) -> np.ndarray:
    y, z = np.asarray(y, np.float64), np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        return y * (z / (1.0 + np.exp(-z)))


def norm_codes(v, weight=None, eps: float = 1e-5) -> dict:
    """v [T, d] → {"scale" [T], "pos" [T, d] (codes before rounding), "u" [T, d]}, float64."""
    v = np.asarray(v, np.float64)
    u = v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    if weight is not None:
        u = u * np.asarray(weight, np.float64)[None, :]
    top = np.abs(u).max(axis=1)
    scale = np.where(top > 0, top / 127.0, 1.0)
    return {"scale": scale, "pos": u / scale[:, None], "u": u}


def matmul(q, s_t, Wq, s_w, bias=None) -> dict:
    """{"out", "mag"}: the product in float64 and the magnitude |product| + |bias| its roundings go by."""
    acc = np.asarray(q, np.float64) @ np.asarray(Wq, np.float64).T     # exact: the sums stay below 2^53
    prod = acc * np.asarray(s_t, np.float64)[:, None] * np.asarray(s_w, np.float64)[None, :]
    b = np.zeros(acc.shape[1]) if bias is None else np.asarray(bias, np.float64)
    return {"out": prod + b[None, :], "mag": np.abs(prod) + np.abs(b)[None, :]}


def softplus(v) -> np.ndarray:
    return np.logaddexp(0.0, np.asarray(v, np.float64))


def conv(xbc, weight, bias=None, state=None, lengths=None, dt_raw=None, dt_bias=None) -> dict:
    """xbc [b, L, C], weight [W, C], state [b, W-1, C] or None, lengths [b] or None.  Returns u (before SiLU),
    out (after), mag (Σ|w s| + |bias|), state [b, W-1, C], and dt, v (before softplus) if dt_raw is given."""
    xbc, w = np.asarray(xbc, np.float64), np.asarray(weight, np.float64)
    b, L, C = xbc.shape
    W = w.shape[0]
    bias = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    lens = np.full(b, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    u, mag = np.zeros((b, L, C)), np.zeros((b, L, C))
    final = np.zeros((b, W - 1, C))
    for r in range(b):
        past = [np.zeros(C)] * (W - 1) if state is None else list(np.asarray(state, np.float64)[r])
        for t in range(int(lens[r])):
            past.append(xbc[r, t])
            taps = np.stack(past[-W:])
            u[r, t] = bias + (w * taps).sum(axis=0)
            mag[r, t] = np.abs(bias) + np.abs(w * taps).sum(axis=0)
        final[r] = np.stack(past[len(past) - (W - 1):])
    with np.errstate(over="ignore"):
        res = {"u": u, "out": u / (1.0 + np.exp(-u)), "mag": mag, "state": final, "lens": lens}
    if dt_raw is not None:
        v = np.asarray(dt_raw, np.float64) + np.asarray(dt_bias, np.float64)
        live = np.arange(L)[None, :, None] < lens[:, None, None]
        res["v"], res["dt"] = v, np.where(live, softplus(v), 0.0)
    return res
