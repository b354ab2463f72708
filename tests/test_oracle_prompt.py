"""Pins of the prompt-path oracle: 4-bit grid by exhaustive search, rotation
against the layer's, causal attention against tree attention of a chain."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_bytes_match_torch():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.e4m3_value(b)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    rng = np.random.default_rng(0)
    x = np.concatenate([np.exp(rng.uniform(-9, 6.1, 4000)), oracle.e4m3_value(np.arange(127)),
                        (oracle.e4m3_value(np.arange(126)) + oracle.e4m3_value(np.arange(1, 127))) / 2]).astype(np.float32)
    x = np.minimum(x, np.float32(448))
    assert np.array_equal(oracle.e4m3_byte(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert oracle.e4m3_byte(np.float32(1e9)) == 126 and oracle.e4m3_byte(np.nan) == 127


def test_kv4_nearest_code_and_ties():
    x = np.zeros((1, 16), np.float32)
    x[0] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.2500001, 0.7499999, 5.000001, -0.0, 4.9]
    codes, s = oracle.kv4_pack(x)
    assert oracle.e4m3_value(s)[0, 0] == 1.0
    got = oracle.kv4_unpack(codes, s)[0]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, 0.5, 0.5, 6, 0, 4]


def test_kv4_zero_nan_and_saturation():
    x = np.zeros((3, 16), np.float32)
    x[1, 3] = np.nan
    x[2] = 1e5
    codes, s = oracle.kv4_pack(x)
    v = oracle.kv4_unpack(codes, s)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and (v[2] == 6 * 448).all()


def test_kv4_error_is_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    codes, s = oracle.kv4_pack(x, 0.5)
    v = oracle.kv4_unpack(codes, s, 0.5)
    step = 0.5 * oracle.e4m3_value(s).repeat(16, -1)
    # the widest gap of the grid is 2 (4 to 6), and the rounded scale may leave
    # the group's largest value up to 2^-4 of 6 past the last magnitude
    assert (np.abs(v - x) <= step * 1.0 + 1e-7).all()


@pytest.mark.parametrize("D", [64, 128])
def test_rotation_is_the_layers(D):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, D))
    pos = np.array([0, 1, 7, 1000, 100000])
    ang = pos[:, None] * 500000.0 ** (-np.arange(0, D, 2) / D)
    got = oracle.rotate(x, np.stack([np.cos(ang), np.sin(ang)], 1))
    assert np.abs(got - oracle.rope(x, pos[:, None], 500000.0)).max() < 1e-12


def test_causal_attention_is_tree_attention_of_a_chain():
    rng = np.random.default_rng(3)
    n, ctx, Hq, Hkv, D = 9, 21, 4, 2, 64
    kv = rng.standard_normal((2, 2, 16, Hkv, D))
    table = np.array([[1, 0]], np.int32)
    k, v = (c[table[0]].reshape(32, Hkv, D) for c in kv)
    q = rng.standard_normal((n, Hq, D))
    out, lse, mag, _ = oracle.prompt_attn(q, [k], [v], [0, n], [ctx], D ** -0.5)
    mask = np.array([[(1 << (i + 1)) - 1 for i in range(n)]], np.uint64)
    want, wl = oracle.tree_attn(q[None], k[None, ctx:ctx + n], v[None, ctx:ctx + n], kv[0], kv[1], table,
                                np.array([ctx]), mask)
    assert np.abs(out - want[0]).max() < 1e-12 and np.abs(lse - wl[0]).max() < 1e-12
    assert (mag >= np.abs(out) - 1e-12).all()
