"""What eagle_draft_prompt leaves in the cache, rows past the projections' 4096,
and the hand-over to eagle_draft_layer, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu
from test_gpu_prompt import DT, f64, gathered, make

pytestmark = pytest.mark.gpu

d, HQ, HKV, D, I = 256, 4, 2, 64, 128


def layer(seed, T, dt):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *sh, k=0.05: (torch.randn(*sh, generator=g) * k).to(dt)  # noqa: E731
    W = dict(norm1=1 + rn(d), qkv=rn((HQ + 2 * HKV) * D, d), o=rn(d, HQ * D), norm2=1 + rn(d), gu=rn(2 * I, d), down=rn(d, I))
    return W, rn(T, d, k=1.0)


@pytest.mark.parametrize("kind,new,ctx", [("bf16", [37, 0, 5], [0, 20, 16]), ("fp32", [9, 4], [0, 30]), ("kv4", [37, 5], [0, 16]),
                                          ("bf16", [4100, 7, 1], [0, 0, 9]), ("kv4", [4095, 2, 6], [0, 0, 3])])
def test_draft_prompt_fills_the_cache(kind, new, ctx):
    """K and V of every row in their places, nothing else touched, and outputs of
    requests with few keys, whose attention is far above the tolerance; in the
    long cases those lie past the first 4096 rows."""
    b = need_gpu()
    dt, kv4 = DT["fp32" if kind == "fp32" else "bf16"], kind == "kv4"
    s = make(83, new, ctx, HQ, HKV, D, "fp32" if kind == "fp32" else "bf16", kv4=kv4)
    W, x = layer(5, s["T"], dt)
    rope = b.eagle_rope_table(max(n + c for n, c in zip(new, ctx)), D, 1e4)
    out = torch.empty(s["T"], d, dtype=dt, device="cuda")
    names = ("k4", "v4") if kv4 else ("kc", "vc")
    kw = dict(k_scales=s["ks"], v_scales=s["vs"]) if kv4 else {}
    b.eagle_draft_prompt(x.cuda(), {k: w.cuda() for k, w in W.items()}, rope, s["cu"], s["ctx"], s[names[0]], s[names[1]],
                         s["table"], out, status=s["st"], **kw)
    assert s["st"].item() == 0

    half = 2.0 ** -24 if kind == "fp32" else 2.0 ** -8
    st = (lambda a: torch.from_numpy(a).to(dt).double().numpy()) if kind != "fp32" else (lambda a: a.astype(np.float32).astype(np.float64))
    w = {k: v.double().numpy() for k, v in W.items()}
    cu = s["cu"].cpu().numpy()
    places = oracle.row_places(cu, ctx, s["table"].cpu().numpy())
    page, slot = np.array([p[2] for p in places]), np.array([p[3] for p in places])
    h = st(oracle.rms_norm(x.double().numpy(), w["norm1"], 1e-5))
    qkv = st(oracle.linear(h, w["qkv"])).reshape(s["T"], -1, D)
    # a stored value may fall the other side of a tie: one step (two halves) of
    # the projection, and of two elements of the row's norm; fp32 sums add
    # 2 d 2^-24 of sum |h w| <= d max |h| max |w|
    hw = np.abs(h).max(-1)[:, None, None] * np.abs(w["qkv"]).max()
    e = 2 * half * np.abs(qkv) + (4 * half + 2 * d * d * 2.0 ** -24) * hw
    r = f64(rope)[[p[1] for p in places]]
    q, k, v = oracle.rotate(qkv[:, :HQ], r), oracle.rotate(qkv[:, HQ:HQ + HKV], r), qkv[:, HQ + HKV:]
    ek = e[:, HQ:HQ + HKV]
    ek = np.tile(ek[..., :D // 2] + ek[..., D // 2:], 2) + half * np.abs(k)
    for name, value, tol in (("k", k, ek), ("v", v, e[:, HQ + HKV:])):
        if kv4:
            read = torch.empty(s["P"], 16, HKV, D, dtype=torch.float32, device="cuda")
            b.eagle_kv4_read(s[name + "4"], s[name + "s"], read)
            got = f64(read)
            codes, scales = oracle.kv4_pack(value.astype(np.float32))
            value = oracle.kv4_unpack(codes, scales)
            # the same code but where the value lies by a midpoint: then a step, of
            # the grid (2 s at most) and of the scale (2^-3 of 6 s)
            step = 3 * oracle.e4m3_value(scales).repeat(16, -1).reshape(value.shape)
            assert (np.abs(got[page, slot] - value) > 2.0 ** -20).mean() < 0.02
            tol = step
        else:
            got = f64(s[name + "c"])
        assert (np.abs(got[page, slot] - value) <= tol).all(), name
        before = s[name + "c_np"].copy()
        before[page, slot] = got[page, slot]
        assert np.array_equal(got, before), name  # no other slot is touched
        s[name + "c_np"][page, slot] = value if kv4 else st(value)

    def rest(a):
        x1 = st(oracle.linear(st(a).reshape(s["T"], -1), w["o"], residual=x.double().numpy()))
        gu = st(oracle.linear(st(oracle.rms_norm(x1, w["norm2"], 1e-5)), w["gu"]))
        return oracle.linear(st(oracle.silu(gu[:, :I]) * gu[:, I:]), w["down"], residual=x1)

    a = oracle.prompt_attn(st(q), gathered(s, s["kc_np"]), gathered(s, s["vc_np"]), cu, ctx, D ** -0.5)[0]
    want = rest(a)
    # as for the layer's outputs elsewhere: a handful of roundings of the output's size
    tol = {"fp32": 1e-5, "bf16": 4 * 2.0 ** -8, "kv4": 6 * 2.0 ** -8}[kind] * (np.abs(want) + 1)
    assert (np.abs(f64(out) - want) <= tol).all()
    few = slice(int(cu[1]), s["T"])
    assert (np.abs(rest(np.zeros_like(a))[few] - want[few]) > 2 * tol[few]).any(-1).all()  # it would show


def test_prompt_then_draft_layer_over_a_poisoned_cache():
    """The prompt's call fills K and V of a cache of NaN; the next row through
    eagle_draft_layer equals the whole prompt's."""
    b = need_gpu()
    n = 50
    s = make(89, [n + 1], [0], HQ, HKV, D, "bf16")
    W, x = layer(7, n + 1, torch.bfloat16)
    W, x, rope = {k: w.cuda() for k, w in W.items()}, x.cuda(), b.eagle_rope_table(64, D, 1e4)
    whole, part = torch.empty_like(x), torch.empty_like(x[:n])
    b.eagle_draft_prompt(x, W, rope, s["cu"], s["ctx"], s["kc"], s["vc"], s["table"], whole)
    s["kc"].fill_(float("nan"))
    s["vc"].fill_(float("nan"))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    b.eagle_draft_prompt(x[:n].contiguous(), W, rope, i32(0, n), s["ctx"], s["kc"], s["vc"], s["table"], part)
    bound = lambda y: 4 * 2.0 ** -8 * (y.float().abs() + 1)  # noqa: E731
    assert ((part.float() - whole[:n].float()).abs() <= bound(whole[:n])).all()
    for c in (s["kc"], s["vc"]):
        rows = c[s["table"][0].long()].flatten(0, 1)
        assert rows[:n].isfinite().all() and rows[n:].isnan().all()
    z = lambda *sh: torch.zeros(*sh, dtype=x.dtype, device="cuda")  # noqa: E731
    out = torch.empty(1, d, dtype=x.dtype, device="cuda")
    b.eagle_draft_layer(x[n:].contiguous(), W, i32(n).view(1, 1), s["kc"], s["vc"], s["table"], i32(n), z(1, 8, HQ, D),
                        z(1, 8, HKV, D), z(1, 8, HKV, D), (1 << torch.arange(8)).view(1, 8).cuda(), 0, out, theta=1e4)
    assert ((out[0].float() - whole[n].float()).abs() <= bound(whole[n])).all()
