"""Log probabilities of given tokens, entropy and the most likely tokens of rows of logits, and their gradient, in
float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing in the product
path may import or call this module.

Readings (the pages give no formulas):
* a given id outside the vocabulary (padding) has log probability 0 and no gradient; ids may repeat;
* equal logits rank by ascending id; a logit of -inf is no alternative, and where fewer than k are left the rest is
  id -1 with -inf;
* a row of nothing but -inf has lse -inf, log probabilities -inf, entropy 0 and gradient 0.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def _log_softmax(z):
    m = z.max(-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        lse = m + np.log(np.exp(z - m).sum(-1, keepdims=True))
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(lse), z - lse, -np.inf), lse[:, 0]


def forward(z, ids=None, k=0):
    """dict of lse [T], entropy [T], logp [T, m] (with ids), top_ids and top_logp [T, k]."""
    z = np.asarray(z, F64)
    lp, lse = _log_softmax(z)
    p = np.exp(lp)
    out = dict(lse=lse, entropy=-np.sum(p * np.where(p > 0, lp, 0.0), -1))
    if ids is not None:
        ids = np.asarray(ids, np.int64)
        ok = (ids >= 0) & (ids < z.shape[1])
        out["logp"] = np.where(ok, np.take_along_axis(lp, np.where(ok, ids, 0), 1), 0.0)
    if k:
        order = np.argsort(-z, axis=-1, kind="stable")[:, :k]
        v = np.take_along_axis(z, order, 1)
        out["top_ids"] = np.where(v > -np.inf, order, -1).astype(np.int32)
        out["top_logp"] = np.where(v > -np.inf, np.take_along_axis(lp, order, 1), -np.inf)
    return out


def backward(z, ids=None, dlogp=None, dentropy=None):
    """(d L / d z, p-term) [T, V]: L = sum dlogp logp + sum dentropy entropy.  The second is the part
    p (A + b (log p + entropy)) that every entry has, in absolute value."""
    z = np.asarray(z, F64)
    T, V = z.shape
    lp, lse = _log_softmax(z)
    p = np.exp(lp)
    a = np.zeros(T)
    g = np.zeros((T, V))
    if ids is not None:
        for t in range(T):
            if not np.isfinite(lse[t]):
                continue
            for i, d in zip(np.asarray(ids)[t], np.asarray(dlogp, F64)[t]):
                if 0 <= i < V:
                    a[t] += d
                    g[t, i] += d
    f = np.broadcast_to(a[:, None], (T, V)).copy()
    if dentropy is not None:
        h = -np.sum(p * np.where(p > 0, lp, 0.0), -1)
        f = f + np.asarray(dentropy, F64)[:, None] * (np.where(p > 0, lp, 0.0) + h[:, None])
    return g - p * f, np.abs(p * f)
