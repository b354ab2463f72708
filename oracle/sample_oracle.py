"""Sampling in fp64: temperature, top-k, top-p and min-p of rows of logits, and
the token of a given uniform number.

Source: [E1] "Verification Phase" (the target's distribution); the pages state no
truncation: the order of the three and their borders are fixed here.
"""
import numpy as np


def truncate(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Mask of the kept entries of one row, and the weights exp((x - max) / T)."""
    x = np.asarray(x, np.float64)
    order = np.lexsort((np.arange(len(x)), -x))  # by (logit descending, index ascending)
    order = order[x[order] > -np.inf]
    t = 1.0 if temperature == 0 else temperature
    with np.errstate(invalid="ignore", under="ignore"):
        w = np.where(x > -np.inf, np.exp((x - x.max()) / t), 0.0)
    if temperature == 0:
        order = order[:1]
    else:
        if top_k > 0:
            order = order[:top_k]
        if top_p < 1:
            run = np.cumsum(w[order])
            before = np.concatenate([[0.0], run[:-1]])
            keep = before < top_p * run[-1]
            keep[0] = True
            order = order[keep]
        order = order[w[order] >= min_p]
    kept = np.zeros(len(x), bool)
    kept[order] = True
    return kept, w


def sample(x, u, **settings):
    """(token, log-prob, entries kept) of one row."""
    kept, w = truncate(x, **settings)
    index = np.flatnonzero(kept)
    run = np.cumsum(w[index])
    at = min(int(np.searchsorted(run, u * run[-1], side="right")), len(index) - 1)
    token = int(index[at])
    t = settings.get("temperature", 1.0) or 1.0
    lp = (float(x[token]) - float(np.max(x))) / t - np.log(run[-1])
    return token, 0.0 if settings.get("temperature", 1.0) == 0 else lp, len(index)
