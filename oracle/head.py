"""The output layer's loss from hidden states: cross entropy and top-k
distillation, and the gradient on the hidden states, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing in the product
path may import or call this module.

Readings (the pages give no formulas; the terms are those of oracle/distill.py):
* a row counts if its label lies in the vocabulary, or always without labels;
  the loss is the sum of the rows that count over their number;
* teacher ids outside the vocabulary are absent, also from the teacher's
  softmax; a row with none left has no distillation term; ids may repeat.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def head(h, w, top_v=None, top_i=None, labels=None, lm_weight=1.0, distill_weight=1.0):
    """(loss, row losses [T], d loss / d h [T, H], size): `size` [T, H] is the sum of the absolute terms of the
    gradient over the vocabulary entries that are neither label nor teacher ids, and over all (a pair)."""
    h, w = np.asarray(h, F64), np.asarray(w, F64)
    T, V = h.shape[0], w.shape[0]
    z = h @ w.T
    m = z.max(-1, keepdims=True)
    lq = z - m - np.log(np.exp(z - m).sum(-1, keepdims=True))
    rows, g, a, special = np.zeros(T), np.zeros((T, V)), np.zeros((T, V)), np.zeros((T, V), bool)
    live = np.ones(T, bool) if labels is None else (np.asarray(labels) >= 0) & (np.asarray(labels) < V)
    n = max(int(live.sum()), 1)
    for t in np.nonzero(live)[0]:
        c = 0.0
        if labels is not None:
            rows[t] -= lm_weight * lq[t, labels[t]]
            g[t, labels[t]] -= lm_weight
            a[t, labels[t]] += abs(lm_weight)
            special[t, labels[t]] = True
            c += lm_weight
        if top_i is not None:
            ok = (top_i[t] >= 0) & (top_i[t] < V)
            ids, v = top_i[t][ok], np.asarray(top_v[t], F64)[ok]
            special[t, ids] = True
            if ids.size and v.max() > -np.inf:
                e = np.exp(v - v.max())
                p = e / e.sum()
                with np.errstate(divide="ignore", invalid="ignore"):
                    rows[t] += distill_weight * np.sum(np.where(p > 0, p * (np.log(p) - lq[t, ids]), 0.0))
                np.subtract.at(g[t], ids, distill_weight * p)
                np.add.at(a[t], ids, abs(distill_weight) * p)
                c += distill_weight
        g[t] += c * np.exp(lq[t])
        a[t] += abs(c) * np.exp(lq[t])
    aw = np.abs(w)
    return rows.sum() / n, rows, g @ w / n, (np.where(special, 0.0, a) @ aw / n, a @ aw / n)
