"""Products whose rows choose their weights (oracle; test infrastructure).

The pages speak of FP4 models with experts ("TORQ") and of W4A4 products
("Bridging the Gap Between Promise and Performance for Microscaling FP4
Quantization", 2.), but define neither routing nor adapters; these are the
published definitions, so their parity is unpinned by the pages.  All of it
is float64, token by token and group by group.
"""

import numpy as np


def route(logits, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_best=1, renormalize=True,
          scale=1.0):
    """Weights (float64), chosen experts (-1: none) and which tokens are bad."""
    x = np.asarray(logits, np.float64)
    tokens, experts = x.shape
    weights, chosen = np.zeros((tokens, top_k)), np.full((tokens, top_k), -1, np.int32)
    bad = np.zeros(tokens, bool)
    b = np.zeros(experts) if bias is None else np.asarray(bias, np.float64)
    per = experts // n_groups
    for t in range(tokens):
        row = x[t]
        if np.isnan(row).any() or (row == np.inf).any():
            bad[t] = True
            continue
        on = row > -np.inf
        s = np.zeros(experts)
        if on.any():
            if score == "softmax":
                s[on] = np.exp(row[on] - row[on].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[on] = 1.0 / (1.0 + np.exp(-row[on]))
        pick = s + b
        if np.isnan(pick[on]).any() or (pick[on] == np.inf).any():
            bad[t] = True
            continue
        on = on & (pick > -np.inf)
        if n_groups > 1:
            by = pick if bias is not None or group_best == 2 else row
            value = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                best = np.sort(by[g * per:(g + 1) * per][on[g * per:(g + 1) * per]])[::-1][:group_best]
                if len(best):
                    value[g] = best.sum()
            kept = np.argsort(-value, kind="stable")[:top_groups]
            on = on & np.isin(np.arange(experts) // per, kept)
        key = np.where(on, pick if bias is not None else row, -np.inf)
        mine = np.argsort(-key, kind="stable")[:min(top_k, int(on.sum()))]
        w = s[mine]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(len(mine))
        weights[t, :len(mine)], chosen[t, :len(mine)] = w * scale, mine
    return weights, chosen, bad


def group_rows(ids, groups):
    """offsets, rows: entries by group, ascending within one, those of none last."""
    ids = np.asarray(ids).ravel()
    key = np.where((ids >= 0) & (ids < groups), ids, groups)
    rows = np.argsort(key, kind="stable").astype(np.int32)
    counts = np.bincount(key, minlength=groups + 1)[:groups]
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), rows


def silu(z):
    return z / (1.0 + np.exp(-z))


def products(a_hat, b_hat, offsets, rows, gather=0):
    """For each position of the groups' order its row of A times its group's
    matrix [groups, N, K], and sum_k |a| |b|; zeros past the last group."""
    out = np.zeros((len(rows), b_hat.shape[1]))
    mag = np.zeros_like(out)
    for g in range(len(offsets) - 1):
        p = np.arange(offsets[g], offsets[g + 1])
        a = a_hat[rows[p] // gather] if gather else a_hat[p]
        out[p] = a @ b_hat[g].T
        mag[p] = np.abs(a) @ np.abs(b_hat[g]).T
    return out, mag


def combine(y, weights, chosen=None, add=None):
    """The weighted sum, and the sum of its terms' magnitudes."""
    on = np.ones(weights.shape, bool) if chosen is None else np.asarray(chosen) >= 0
    w = np.where(on, weights, 0.0)[..., None]
    terms = np.where(on[..., None], np.asarray(y, np.float64), 0.0) * w
    out, mag = terms.sum(1), np.abs(terms).sum(1)
    if add is not None:
        out, mag = out + add, mag + np.abs(add)
    return out, mag


def lora(y, x, a, b, offsets, rows, scales=None):
    """y + s (x A^T) B^T, and s (|x| |A|^T) |B|^T."""
    out, mag = np.array(y, np.float64), np.zeros(np.shape(y))
    for g in range(len(offsets) - 1):
        r = rows[offsets[g]:offsets[g + 1]]
        s = 1.0 if scales is None else float(scales[g])
        out[r] += s * ((x[r] @ a[g].T) @ b[g].T)
        mag[r] = abs(s) * ((np.abs(x[r]) @ np.abs(a[g]).T) @ np.abs(b[g]).T)
    return out, mag
