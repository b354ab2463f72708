"""The oracle of shared prefixes: joined with the causal attention over the keys
behind the prefix it is the attention over all of them."""
import numpy as np

import oracle


def test_join_is_the_whole_attention():
    r = np.random.default_rng(0)
    Hq, Hkv, D, P = 4, 2, 8, 37
    new, ctx = [3, 0, 5], [4, 2, 0]
    cu = np.cumsum([0] + new)
    pre_k, pre_v = r.normal(size=(P, Hkv, D)), r.normal(size=(P, Hkv, D))
    own_k = [r.normal(size=(n + c, Hkv, D)) for n, c in zip(new, ctx)]
    own_v = [r.normal(size=(n + c, Hkv, D)) for n, c in zip(new, ctx)]
    q = r.normal(size=(sum(new), Hq, D))
    o, l, _, _ = oracle.prompt_attn(q, own_k, own_v, cu, ctx, 0.4)
    out, lse, _, _, _ = oracle.prefix_attn(q, [pre_k], [pre_v], [0, sum(new)], 0.4, o, l)
    want, wl, _, _ = oracle.prompt_attn(q, [np.concatenate([pre_k, k]) for k in own_k], [np.concatenate([pre_v, v]) for v in own_v],
                                        cu, [P + c for c in ctx], 0.4)
    assert np.abs(out - want).max() < 1e-12 and np.abs(lse - wl).max() < 1e-12


def test_nothing_of_one_side():
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(2, 1, 4)), r.normal(size=(3, 1, 4)), r.normal(size=(3, 1, 4))
    o, l = r.normal(size=(2, 1, 4)), np.array([[0.3], [-np.inf]])
    empty = np.zeros((0, 1, 4))
    out, lse, *_ = oracle.prefix_attn(q, [empty], [empty], [0, 2], 0.5, o, l)
    assert np.array_equal(out[0], o[0]) and np.array_equal(out[1], 0 * o[1]) and lse[0, 0] == 0.3 and lse[1, 0] == -np.inf
    alone, ll, *_ = oracle.prefix_attn(q, [k], [v], [0, 2], 0.5)
    joined, jl, *_ = oracle.prefix_attn(q, [k], [v], [0, 2], 0.5, np.full_like(o, np.nan), np.full((2, 1), -np.inf))
    assert np.array_equal(alone, joined) and np.array_equal(ll, jl)
