"""fp64 gradients of the recurrence and the gate, and the norm, in numpy.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Written from the
per-token recurrence by reversing its steps one by one; no chunks.  Checked
against differences of ``oracle.forward`` in ``tests/test_oracle_gradients.py``.
"""
from __future__ import annotations

import numpy as np


def _softplus(x):
    return np.logaddexp(x, 0.0)


def _sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def _ranges(T, B, L, cu_seqlens, seq_lens):
    if cu_seqlens is not None:
        m = np.maximum.accumulate(np.clip(np.asarray(cu_seqlens, np.int64), 0, T))
        return [(int(m[i]), int(m[i + 1])) for i in range(len(m) - 1)]
    lens = [L] * B if seq_lens is None else [int(min(max(n, 0), L)) for n in seq_lens]
    return [(b * L, b * L + lens[b]) for b in range(B)]


def backward(q, k, v, d_o, *, gate=None, beta=None, a_log=None, dt_bias=None, gate_scale=None, cu_seqlens=None,
             seq_lens=None, initial_state=None, d_final_state=None, update_rule="gated_delta",
             gate_activation="none", beta_activation="none", qk_l2_norm=0, scale=0.0, batch=None):
    """Dict of fp64 gradients in the inputs' shapes; rows of tokens outside
    every request are zero.  A final state's gradient and an initial state are
    (B, HV, dv, dk)."""
    shape_q, shape_v = q.shape, v.shape
    if q.ndim == 4:
        B, L = q.shape[:2]
    else:
        B = (len(cu_seqlens) - 1 if cu_seqlens is not None else batch if batch is not None
             else len(initial_state) if initial_state is not None else len(seq_lens) if seq_lens is not None else 1)
        L = q.shape[0] // B if B and cu_seqlens is None else 0
    H, dk, HV, dv = q.shape[-2], q.shape[-1], v.shape[-2], v.shape[-1]
    f = lambda x, *s: np.asarray(x, np.float64).reshape(*s)  # noqa: E731
    q, k, v, d_o = f(q, -1, H, dk), f(k, -1, H, dk), f(v, -1, HV, dv), f(d_o, -1, HV, dv)
    T, R = q.shape[0], HV // H
    scale = scale if scale else 1.0 / np.sqrt(dk)
    decays, rate = update_rule in ("gated", "gated_delta"), update_rule in ("delta", "gated_delta")
    nq = np.sqrt((q * q).sum(-1, keepdims=True) + 1e-12) if qk_l2_norm else np.ones((T, H, 1))
    nk = np.sqrt((k * k).sum(-1, keepdims=True) + 1e-12) if qk_l2_norm else np.ones((T, H, 1))
    qh, kh = scale * q / nq, k / nk
    g = np.zeros((T, HV))
    if decays:
        g = f(gate, T, HV)
        if gate_activation == "qwen":
            x = g + np.asarray(dt_bias, np.float64)
            coef = -np.exp(np.asarray(a_log, np.float64)) if a_log is not None else np.asarray(gate_scale, np.float64)
            g = coef * _softplus(x)
    raw = None
    b = np.ones((T, HV))
    if rate:
        raw = f(beta, T, -1)
        b = np.broadcast_to(_sigmoid(raw) if beta_activation == "sigmoid" else raw, (T, HV))
    dqh, dkh, dvv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    dg, db = np.zeros((T, HV)), np.zeros((T, HV))
    d_init = np.zeros((B, HV, dv, dk))
    for r, (s, e) in enumerate(_ranges(T, B, L, cu_seqlens, seq_lens)):
        for h in range(HV):
            S = np.zeros((dv, dk)) if initial_state is None else np.asarray(initial_state[r, h], np.float64)
            past = []
            for t in range(s, e):
                kt = kh[t, h // R]
                A = np.exp(g[t, h]) * S
                miss = v[t, h] - A @ kt if rate else v[t, h]
                d = b[t, h] * miss if rate else miss
                S = A + np.outer(d, kt)
                past.append((A, miss, d, S))
            dS = np.zeros((dv, dk)) if d_final_state is None else np.asarray(d_final_state[r, h], np.float64).copy()
            for t in range(e - 1, s - 1, -1):
                A, miss, d, S = past[t - s]
                qt, kt, do = qh[t, h // R], kh[t, h // R], d_o[t, h]
                dS = dS + np.outer(do, qt)
                dqh[t, h // R] += S.T @ do
                dd = dS @ kt
                dkh[t, h // R] += dS.T @ d
                if rate:
                    db[t, h] = dd @ miss
                    dd = b[t, h] * dd
                    dkh[t, h // R] -= A.T @ dd
                    dS = dS - np.outer(dd, kt)
                dvv[t, h] = dd
                dg[t, h] = (dS * A).sum()
                dS = np.exp(g[t, h]) * dS
            d_init[r, h] = dS

    def through_norm(d, x, n):
        return (d - x * (x * d).sum(-1, keepdims=True) / n ** 2) / n if qk_l2_norm else d

    out = {"q": (scale * through_norm(dqh, q, nq)).reshape(shape_q), "k": through_norm(dkh, k, nk).reshape(shape_q),
           "v": dvv.reshape(shape_v), "initial_state": d_init}
    if decays:
        if gate_activation == "qwen":
            da = dg * coef * _sigmoid(x)
            dc = (dg * _softplus(x)).sum(0)
            out["dt_bias"], dg = da.sum(0), da
            out["a_log" if a_log is not None else "gate_scale"] = dc * coef if a_log is not None else dc
        out["gate"] = dg.reshape(gate.shape)
    if rate:
        db = db.sum(-1, keepdims=True) if raw.shape[-1] != HV else db
        if beta_activation == "sigmoid":
            db = db * _sigmoid(raw) * _sigmoid(-raw)
        out["beta"] = db.reshape(beta.shape)
    return out


def gate_backward(a, dt_bias, decay_scale, d_decay, b=None, d_beta=None):
    """(d_a, d_b or None, d_dt_bias, d_decay_scale) of the standalone gate."""
    a, d = np.asarray(a, np.float64), np.asarray(d_decay, np.float64)
    x = a + np.asarray(dt_bias, np.float64)
    d_a = d * np.asarray(decay_scale, np.float64) * _sigmoid(x)
    axes = tuple(range(a.ndim - 1))
    d_b = None
    if b is not None:
        y = np.asarray(b, np.float64)
        d_b = np.asarray(d_beta, np.float64) * _sigmoid(y) * _sigmoid(-y)
    return d_a, d_b, d_a.sum(axes), (d * _softplus(x)).sum(axes)


def rms_norm(r, weight=None, eps=1e-6):
    """(y, inv) of rows r that already hold the residual's sum."""
    r = np.asarray(r, np.float64)
    inv = 1.0 / np.sqrt((r * r).mean(-1) + eps)
    y = r * inv[..., None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), inv


def rms_norm_backward(d_y, r, weight=None, d_residual=None, eps=1e-6):
    """(d_x, d_weight) with inv = 1 / sqrt(mean r^2 + eps)."""
    r, d_y = np.asarray(r, np.float64), np.asarray(d_y, np.float64)
    inv = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    h = r * inv
    t = d_y if weight is None else d_y * np.asarray(weight, np.float64)
    d_x = inv * (t - h * (t * h).mean(-1, keepdims=True))
    if d_residual is not None:
        d_x = d_x + np.asarray(d_residual, np.float64)
    return d_x, (d_y * h).reshape(-1, r.shape[-1]).sum(0)


def e4m3_values():
    """Every finite value of the 8-bit type (4 exponent bits, bias 7, 3
    mantissa bits; 0x7f and 0xff are NaN), by its code."""
    code = np.arange(256)
    exp, man = (code >> 3) & 15, code & 7
    mag = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    mag[(code & 0x7F) == 0x7F] = np.nan
    return np.where(code >= 128, -mag, mag)
