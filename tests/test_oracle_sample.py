"""The sampling oracle against its definition by enumeration, and the
distribution that it draws from."""
import numpy as np
import pytest

import oracle


def by_definition(x, t, k, p, m):
    """The kept set, entry by entry."""
    order = sorted((i for i in range(len(x)) if x[i] > -np.inf), key=lambda i: (-x[i], i))
    if t == 0:
        return {order[0]}
    w = {i: float(np.exp((x[i] - x[order[0]]) / t)) for i in order}
    if k > 0:
        order = order[:k]
    total, run, kept = sum(w[i] for i in order), 0.0, []
    for i in order:
        if p >= 1 or run < p * total or not kept:
            kept.append(i)
        run += w[i]
    return {i for i in kept if w[i] >= m}


@pytest.mark.parametrize("seed", range(20))
def test_truncation_is_the_definition(seed):
    r = np.random.default_rng(seed)
    x = r.normal(0, 2, 12)
    x[r.integers(0, 12, 3)] = x[0]  # ties
    if seed % 3 == 0:
        x[r.integers(1, 12, 3)] = -np.inf
    for t in (0.0, 0.5, 1.0):
        for k in (0, 1, 3, 12, 40):
            for p in (0.0, 0.37, 0.9, 1.0):
                for m in (0.0, 0.11, 1.0):
                    kept, _ = oracle.truncate(x, t, k, p, m)
                    assert set(np.flatnonzero(kept)) == by_definition(x, t, k, p, m), (t, k, p, m)


def test_tokens_follow_the_truncated_distribution():
    x = np.array([0.3, 2.0, -1.0, 2.0, 1.1])
    s = dict(temperature=0.8, top_k=4, top_p=0.95)
    kept, w = oracle.truncate(x, **s)
    p = np.where(kept, w, 0) / w[kept].sum()
    n = 20000
    got = np.bincount([oracle.sample(x, (i + 0.5) / n, **s)[0] for i in range(n)], minlength=5) / n
    assert np.abs(got - p).max() <= 1.5 / n  # a grid of uniforms: each border moves one of them at most
    tok, lp, kept_n = oracle.sample(x, 0.0, **s)
    assert tok == np.flatnonzero(kept)[0] and abs(lp - np.log(p[tok])) < 1e-12 and kept_n == kept.sum()
