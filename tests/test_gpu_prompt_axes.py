"""GPU parity of the append at positions of several axes against the fp64
oracle's rotation.

Tolerances count roundings, as for the append by slot: a rotated value is three
fp32 operations against |x1 c| + |x2 s| <= hypot(x1, x2), then one rounding to
the type; pairs that are not turned are copied.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu
from test_gpu_prompt import DT, HALF, LENS, f64, make

pytestmark = pytest.mark.gpu

MAX_POS = 512


def axes_of(kind, D):
    half = D // 2
    return {"one": (1, None), "given": (1, [0] * half), "sections": (3, [0] * (half // 4) + [1] * (half // 2 - half // 8) + [2] * (half - half // 4 - half // 2 + half // 8)),
            "turns": (3, [i % 3 for i in range(half)]), "partial": (2, [i % 2 if i % 5 else -1 for i in range(half)]),
            "none": (8, [-1] * half), "eight": (8, [(5 * i) % 8 for i in range(half)])}[kind]


def places_and_turn(s, ctx, rope, pos, axis, D):
    """Cache places of the rows, and their cos and sin [T, 2, D/2] (1, 0 where a pair is not turned)."""
    places = oracle.row_places(s["cu"].cpu().numpy(), ctx, s["table"].cpu().numpy())
    axis = np.zeros(D // 2, int) if axis is None else np.array(axis)
    r = f64(rope)[pos[np.maximum(axis, 0)].T, :, np.arange(D // 2)[None]].transpose(0, 2, 1)
    return places, np.where((axis >= 0)[None, None], r, np.array([1.0, 0.0])[None, :, None])


def pair(x):
    h = x.shape[-1] // 2
    return np.tile(np.hypot(x[..., :h], x[..., h:]), 2)


@pytest.mark.parametrize("kind", ["one", "given", "sections", "turns", "partial", "none", "eight"])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,D,dtype", [
    (*LENS[2], 4, 2, 64, "fp32"), (*LENS[3], 32, 8, 128, "bf16"), (*LENS[4], 3, 1, 128, "bf16"), (*LENS[5], 5, 5, 64, "bf16"),
    (*LENS[1], 7, 1, 128, "fp32")])
def test_append_axes(new, ctx, Hq, Hkv, D, dtype, kind):
    b = need_gpu()
    s = make(len(new) * 5 + Hq, new, ctx, Hq, Hkv, D, dtype, pad=1)
    rope = b.eagle_rope_table(MAX_POS, D, 500000.0)
    A, axis = axes_of(kind, D)
    pos = np.random.default_rng(D + A).integers(0, MAX_POS, (A, s["T"])).astype(np.int32)
    pos[0, 0], pos[-1, -1] = 0, MAX_POS - 1
    q, k, v = f64(s["q"]), f64(s["k"]), f64(s["v"])
    q_out = torch.full((s["T"], Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    b.eagle_kv_append_axes(s["q"], s["k"], s["v"], rope, torch.from_numpy(pos).cuda(), s["cu"], s["ctx"], s["table"], s["kc"],
                           s["vc"], pair_axis=None if axis is None else torch.tensor(axis, dtype=torch.int32).cuda(),
                           q_out=q_out, status=s["st"])
    places, r = places_and_turn(s, ctx, rope, pos, axis, D)
    kc, vc = s["kc_np"].copy(), s["vc_np"].copy()
    want, kr = oracle.rotate(q, r), oracle.rotate(k, r)
    still = np.zeros(D, bool) if axis is None else np.tile(np.array(axis) < 0, 2)
    slack = lambda x: np.where(still, 0.0, 2.0 ** -22 * pair(x) + HALF[dtype] * np.abs(oracle.rotate(x, r)))  # noqa: E731
    assert (np.abs(f64(q_out) - want) <= slack(q)).all()
    tol, ks = np.zeros_like(kc), slack(k)
    for t, (_, _, page, slot) in enumerate(places):
        kc[page, slot], vc[page, slot], tol[page, slot] = kr[t], v[t], ks[t]
    assert np.array_equal(f64(s["vc"]), vc)
    assert (np.abs(f64(s["kc"]) - kc) <= tol).all()  # nothing else is touched either
    assert s["st"].item() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 3, 3)])
@pytest.mark.parametrize("kv4", [False, True])
def test_slot_positions_give_the_append_by_slot(D, Hq, Hkv, kv4):
    """Positions equal to the slots, on every axis: bit for bit what the append by slot writes."""
    b = need_gpu()
    new, ctx = LENS[2]
    A, axis = axes_of("turns", D)
    got = []
    for axes in (False, True):
        s = make(31, new, ctx, Hq, Hkv, D, "bf16", kv4=kv4)
        rope = b.eagle_rope_table(MAX_POS, D, 500000.0)
        cache = [s[n] for n in (("k4", "ks", "v4", "vs") if kv4 else ("kc", "vc"))]
        q_out = torch.zeros(s["T"], Hq, D, dtype=torch.bfloat16, device="cuda")
        at = [p[1] for p in oracle.row_places(s["cu"].cpu().numpy(), ctx, s["table"].cpu().numpy())]
        if axes:
            pos = torch.tensor([at] * A, dtype=torch.int32).cuda()
            call = b.eagle_kv_append_axes_kv4 if kv4 else b.eagle_kv_append_axes
            call(s["q"], s["k"], s["v"], rope, pos, s["cu"], s["ctx"], s["table"], *cache,
                 pair_axis=torch.tensor(axis, dtype=torch.int32).cuda(), q_out=q_out, status=s["st"])
        else:
            call = b.eagle_kv_append_kv4 if kv4 else b.eagle_kv_append
            call(s["q"], s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], *cache, q_out=q_out, status=s["st"])
        assert s["st"].item() == 0
        got.append([q_out] + cache)
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_4bit_axes_match_rows_turned_before():
    """4-bit pages of rows turned by the axes: the codes of the same rows, turned
    in fp32 operations one by one and appended without rotation as fp32 values."""
    b = need_gpu()
    new, ctx, Hkv, D = [5, 0, 40], [3, 2, 14], 2, 128
    s = make(77, new, ctx, 4, Hkv, D, "bf16", kv4=True)
    A, axis = axes_of("partial", D)
    pos = np.random.default_rng(3).integers(0, MAX_POS, (A, s["T"])).astype(np.int32)
    rope = b.eagle_rope_table(MAX_POS, D, 1e4)
    b.eagle_kv_append_axes_kv4(None, s["k"], s["v"], rope, torch.from_numpy(pos).cuda(), s["cu"], s["ctx"], s["table"], s["k4"],
                               s["ks"], s["v4"], s["vs"], pair_axis=torch.tensor(axis, dtype=torch.int32).cuda(), status=s["st"])
    places, r = places_and_turn(s, ctx, rope, pos, axis, D)
    c, n = (r[:, i, None].astype(np.float32) for i in (0, 1))
    x = s["k"].float().cpu().numpy()
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    turned = np.concatenate([x1 * c - x2 * n, x2 * c + x1 * n], -1)
    codes, scales = s["pack"][0][0].copy(), s["pack"][0][1].copy()
    want_c, want_s = oracle.kv4_pack(turned)
    for t, (_, _, page, slot) in enumerate(places):
        codes[page, :, slot], scales[page, :, slot] = want_c[t], want_s[t]
    assert np.array_equal(s["ks"].cpu().numpy(), scales) and np.array_equal(s["k4"].cpu().numpy(), codes)
    assert s["st"].item() == 0


def test_pairs_that_do_not_turn_keep_anything():
    """Infinities and NaN of a pair of axis -1 come through as they are, and a
    table whose cosine is 2 (or NaN) turns by it."""
    b = need_gpu()
    s = make(5, [3], [0], 1, 1, 64, "fp32")
    s["q"][1, 0, 0], s["q"][1, 0, 32], s["q"][2, 0, 33] = float("inf"), float("-inf"), float("nan")
    rope = b.eagle_rope_table(4, 64, 1e4).clone()
    rope[1, 0, 2], rope[1, 1, 2] = 2.0, 0.0
    rope[1, 0, 3] = float("nan")
    axis = [-1, -1] + [0] * 30
    q_out = torch.zeros(3, 1, 64, device="cuda")
    b.eagle_kv_append_axes(s["q"], s["k"], s["v"], rope, torch.tensor([[1, 1, 1]], dtype=torch.int32).cuda(), s["cu"], s["ctx"],
                           s["table"], s["kc"], s["vc"], pair_axis=torch.tensor(axis, dtype=torch.int32).cuda(), q_out=q_out)
    q = s["q"]
    assert torch.equal(q_out[..., [0, 1, 32]], q[..., [0, 1, 32]])
    assert torch.equal(q_out[:2, :, 33], q[:2, :, 33]) and q_out[2, 0, 33].isnan()
    assert torch.equal(q_out[..., 2], 2 * q[..., 2]) and torch.equal(q_out[..., 34], 2 * q[..., 34])
    assert q_out[..., [3, 35]].isnan().all()


@pytest.mark.parametrize("what", ["past", "negative", "other_axis", "axis_high", "axis_low"])
def test_bad_positions_skip_their_rows(what):
    b = need_gpu()
    new, ctx, D = [4, 3], [2, 15], 64
    s = make(9, new, ctx, 2, 1, D, "bf16")
    rope = b.eagle_rope_table(MAX_POS, D, 1e4)
    pos = torch.arange(7, dtype=torch.int32).repeat(2, 1).cuda()
    axis = torch.zeros(D // 2, dtype=torch.int32).cuda()
    skipped = [5]
    if what == "past":
        pos[0, 5] = MAX_POS
    elif what == "negative":
        pos[0, 5] = -1
    elif what == "other_axis":  # one that no pair turns by
        pos[1, 5] = MAX_POS + 7
    else:
        axis[40 % (D // 2)] = 2 if what == "axis_high" else -2
        skipped = list(range(7))
    q_out = torch.full((7, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    b.eagle_kv_append_axes(s["q"], s["k"], s["v"], rope, pos, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], pair_axis=axis,
                           q_out=q_out, status=s["st"])
    assert s["st"].item() == 1  # EAGLE_ERR_INVALID_ARG
    places = oracle.row_places(s["cu"].cpu().numpy(), ctx, s["table"].cpu().numpy())
    vc = s["vc_np"].copy()
    for t, (_, _, page, slot) in enumerate(places):
        if t not in skipped:
            vc[page, slot] = f64(s["v"])[t]
        assert (q_out[t] == 7.0).all().item() == (t in skipped)
    assert np.array_equal(f64(s["vc"]), vc)


def test_slots_past_the_table_are_no_positions():
    """The slot goes by ctx_lens and may lie past the rotation table."""
    b = need_gpu()
    s = make(10, [2], [40], 2, 1, 64, "bf16")
    rope = b.eagle_rope_table(8, 64, 1e4)
    q_out = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    b.eagle_kv_append_axes(s["q"], s["k"], s["v"], rope, torch.tensor([[0, 0]], dtype=torch.int32).cuda(), s["cu"], s["ctx"],
                           s["table"], s["kc"], s["vc"], q_out=q_out, status=s["st"])
    assert s["st"].item() == 0 and torch.equal(q_out, s["q"])  # position 0 turns by nothing
