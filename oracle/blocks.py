"""The passes around the linear calls in fp64 (oracle): the residual sum
between two norms with its gradients, and token log probabilities with theirs.

Test infrastructure: only the tests may use this module.  Formulas as in the
library's header; every sum and product is fp64.
"""

from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def residual_norm_forward(h, y, w_post, gate, scale, w_pre, eps):
    """(v, x, rstd_post, rstd_pre); None for the parts left out."""
    h, y, w_post, gate, w_pre = map(_f64, (h, y, w_post, gate, w_pre))
    rstd_post = rstd_pre = x = None
    v = h
    if y is not None:
        p = y
        if w_post is not None:
            rstd_post = 1.0 / np.sqrt((y * y).mean(1) + eps)
            p = y * rstd_post[:, None] * w_post
        v = h + scale * (1.0 if gate is None else gate) * p
    if w_pre is not None:
        rstd_pre = 1.0 / np.sqrt((v * v).mean(1) + eps)
        x = v * rstd_pre[:, None] * w_pre
    return v, x, rstd_post, rstd_pre


def residual_norm_backward(dh_out, dx, h_out, y, w_post, gate, scale, w_pre, rstd_post, rstd_pre):
    """Gradients as a dict: dh, dy and whichever of dw_post, dgate, dw_pre exist."""
    dh_out, dx, h_out, y, w_post, gate, w_pre, rstd_post, rstd_pre = map(
        _f64, (dh_out, dx, h_out, y, w_post, gate, w_pre, rstd_post, rstd_pre))
    out = {}
    g = np.zeros_like(dx) if dh_out is None else dh_out
    if dx is not None:
        n = h_out * rstd_pre[:, None]
        dn = dx * w_pre
        g = g + rstd_pre[:, None] * (dn - n * (dn * n).mean(1, keepdims=True))
        out["dw_pre"] = (dx * n).sum(0)
    out["dh"] = g
    dp = scale * g
    m = p = y
    if w_post is not None:
        m = y * rstd_post[:, None]
        p = m * w_post
    if gate is not None:
        if y is not None:
            out["dgate"] = (dp * p).sum(0)
        dp = dp * gate
    if w_post is not None:
        out["dw_post"] = (dp * m).sum(0)
        dm = dp * w_post
        dp = rstd_post[:, None] * (dm - m * (dm * m).mean(1, keepdims=True))
    out["dy"] = dp
    return out


def token_logprobs(logits, targets, inv_temperature, k=0):
    """Dict of logprob, entropy, row_max, log_sum (and top_ids, top_logprob for k > 0).

    A negative target is not scored (log probability 0), one of V or more gives
    NaN.  A row without a finite or infinite value above -inf (every logit
    -inf) has row_max -inf, log_sum 0, log probability -inf and entropy 0.  A
    row with NaN or +inf gives NaN.
    """
    x = _f64(logits)
    M, V = x.shape
    out = {"logprob": np.zeros(M), "entropy": np.zeros(M), "row_max": np.zeros(M), "log_sum": np.zeros(M)}
    if k:
        out["top_ids"], out["top_logprob"] = np.zeros((M, k), dtype=np.int32), np.zeros((M, k))
    for i in range(M):
        row = x[i]
        bad = np.isnan(row).any() or (row == np.inf).any()
        m = np.nan if np.isnan(row).any() else row.max()
        if bad:
            d, log_sum, H = np.full(V, np.nan), np.nan, np.nan
        elif m == -np.inf:
            d, log_sum, H = np.full(V, -np.inf), 0.0, 0.0
        else:
            d = (row - m) * inv_temperature
            e = np.exp(d)
            log_sum = np.log(e.sum())
            H = log_sum - np.where(e > 0, e * np.where(e > 0, d, 0.0), 0.0).sum() / e.sum()
        t = int(targets[i])
        out["logprob"][i] = 0.0 if t < 0 else np.nan if t >= V else d[t] - log_sum
        out["entropy"][i], out["row_max"][i], out["log_sum"][i] = H, m, log_sum
        if k:
            order = np.lexsort((np.arange(V), -np.where(np.isnan(row), 0, row), ~np.isnan(row)))[:k]
            out["top_ids"][i], out["top_logprob"][i] = order, d[order] - log_sum
    return out


def token_logprobs_backward(logits, targets, inv_temperature, g_logprob, g_entropy=None):
    """dlogits: NaN for rows with NaN or +inf or a target of V or more, zero for other rows whose logits are all -inf."""
    x = _f64(logits)
    M, V = x.shape
    out = np.zeros((M, V))
    f = token_logprobs(logits, targets, inv_temperature)
    for i in range(M):
        t = int(targets[i])
        if np.isnan(f["log_sum"][i]) or t >= V:
            out[i] = np.nan
            continue
        if f["row_max"][i] == -np.inf:
            continue
        lp = (x[i] - f["row_max"][i]) * inv_temperature - f["log_sum"][i]
        p = np.exp(lp)
        g = 0.0 if t < 0 else float(g_logprob[i])
        out[i] = -g * p
        if t >= 0:
            out[i, t] += g
        if g_entropy is not None:
            out[i] -= float(g_entropy[i]) * np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + f["entropy"][i]), 0.0)
        out[i] *= inv_temperature
    return out
