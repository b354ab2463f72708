"""GPU parity of the prompt path: append with rotation, 4-bit pages, causal
attention over the paged cache, against the fp64 oracle.

Tolerances count roundings.  Append: the rotated value is three fp32
operations and one rounding to the type.  Attention, per element: the output's
rounding, the rounding of the weights to the matrix type (bf16 2^-8, fp16
2^-11 for 4-bit pages, none in fp32) against sum w|v|, and fp32 arithmetic:
a score is off by at most dz = (D + 8) 2^-24 scale sum|q k|, a weight by 2 dz
relative, a sum of L terms by (L + 16) 2^-24.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "fp16": 2.0 ** -11}


def make(seed, new, ctx, Hq, Hkv, D, dtype, kv4=False, pad=0):
    """Packed rows (slices of one wider array), pools and tables; numpy copies of everything are made by the tests."""
    g = torch.Generator().manual_seed(seed)
    T, dt = sum(new), DT[dtype]
    rows = torch.randn(T, Hq + 2 * Hkv + pad, D, generator=g).to(dt).cuda()
    n_pages = [-(-(n + c) // 16) for n, c in zip(new, ctx)]
    P, width = sum(n_pages) + 2, max(n_pages + [1])
    ids = torch.randperm(P, generator=g).int()
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = ids[at:at + n]
        at += n
    s = dict(T=T, Hq=Hq, Hkv=Hkv, D=D, q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv], v=rows[:, Hq + Hkv:Hq + 2 * Hkv],
             cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda(),
             ctx=torch.tensor(ctx, dtype=torch.int32).cuda(), table=table.cuda(), P=P,
             st=torch.zeros(1, dtype=torch.int32).cuda())
    pool = torch.randn(2, P, 16, Hkv, D, generator=g)
    if kv4:
        s["pack"] = [oracle.kv4_pack(pool[i].transpose(1, 2).numpy()) for i in (0, 1)]
        (s["k4"], s["ks"]), (s["v4"], s["vs"]) = [[torch.from_numpy(a).cuda() for a in x] for x in s["pack"]]
        s["kc_np"], s["vc_np"] = [oracle.kv4_unpack(*x).transpose(0, 2, 1, 3) for x in s["pack"]]
    else:
        s["kc"], s["vc"] = pool[0].to(dt).cuda(), pool[1].to(dt).cuda()
        s["kc_np"], s["vc_np"] = f64(s["kc"]), f64(s["vc"])
    return s


def f64(t):
    return t.double().cpu().numpy()


def gathered(s, cache):
    """Per request [n_keys, Hkv, D] of a numpy cache [P, 16, Hkv, D]."""
    table = s["table"].cpu().numpy()
    return [cache[np.maximum(t, 0)].reshape(-1, *cache.shape[2:]) for t in table]


def rope_np(pos, D, theta=500000.0):
    ang = np.asarray(pos, np.float64)[:, None] * theta ** (-np.arange(0, D, 2) / D)
    return np.stack([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("D,theta", [(64, 1e4), (128, 500000.0)])
def test_rope_table(D, theta):
    b = need_gpu()
    n = 70000
    t = f64(b.eagle_rope_table(n, D, theta))
    want = rope_np(np.arange(n), D, theta)
    # fp64 angle up to 7e4 (2^-53 * 7e4 * a few), rounded to fp32
    assert t.shape == (n, 2, D // 2) and np.abs(t - want).max() <= 2.0 ** -24 + 1e-10


LENS = [
    ([1], [0]), ([1, 1, 1], [5, 15, 16]), ([0, 7, 0, 33, 1], [3, 0, 9, 31, 100]), ([16, 17, 15], [0, 1, 47]),
    ([1] * 40, list(range(40))), ([130], [257]),
]


@pytest.mark.parametrize("new,ctx", LENS)
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 64, "fp32"), (32, 8, 128, "bf16"), (3, 1, 128, "bf16"),
                                            (5, 5, 64, "bf16"), (7, 1, 128, "fp32")])
def test_append(new, ctx, Hq, Hkv, D, dtype):
    b = need_gpu()
    s = make(len(new) * 7 + Hq, new, ctx, Hq, Hkv, D, dtype, pad=1)
    rope = b.eagle_rope_table(512, D, 500000.0)
    q, k, v = f64(s["q"]), f64(s["k"]), f64(s["v"])
    q_out = torch.full((s["T"], Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    b.eagle_kv_append(s["q"], s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], q_out=q_out,
                      status=s["st"])
    places = oracle.row_places(s["cu"].cpu().numpy(), ctx, s["table"].cpu().numpy())
    r = f64(rope)[[p[1] for p in places]]
    kc, vc = s["kc_np"].copy(), s["vc_np"].copy()
    # three fp32 roundings against |x1 c| + |x2 s| <= hypot(x1, x2), then one to the type
    pair = lambda x: np.tile(np.hypot(x[..., :D // 2], x[..., D // 2:]), 2)  # noqa: E731
    want, kr = oracle.rotate(q, r), oracle.rotate(k, r)
    assert (np.abs(f64(q_out) - want) <= HALF[dtype] * np.abs(want) + 2.0 ** -22 * pair(q)).all()
    tol = np.zeros_like(kc)
    for t, (_, _, page, slot) in enumerate(places):
        kc[page, slot], vc[page, slot] = kr[t], v[t]
        tol[page, slot] = HALF[dtype] * np.abs(kr[t]) + 2.0 ** -22 * pair(k)[t]
    assert np.array_equal(f64(s["vc"]), vc)
    assert (np.abs(f64(s["kc"]) - kc) <= tol).all()  # nothing else is touched either
    assert s["st"].item() == 0


def test_append_in_place_without_rotation_and_without_q():
    b = need_gpu()
    s = make(3, [9, 4], [2, 20], 4, 2, 128, "bf16")
    q = s["q"].contiguous()
    rope = b.eagle_rope_table(64, 128, 1e4)
    want = torch.empty_like(q)
    b.eagle_kv_append(q, s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], q_out=want)
    kc = s["kc"].clone()
    b.eagle_kv_append(q, s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], q_out=q)
    assert torch.equal(q, want) and torch.equal(s["kc"], kc)
    b.eagle_kv_append(None, s["k"], s["v"], None, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], status=s["st"])
    for t, (_, _, page, slot) in enumerate(oracle.row_places(s["cu"].cpu().numpy(), [2, 20], s["table"].cpu().numpy())):
        assert torch.equal(s["kc"][page, slot], s["k"][t]) and torch.equal(s["vc"][page, slot], s["v"][t])
    assert s["st"].item() == 0


def test_append_skips_what_it_cannot_place():
    b = need_gpu()
    s = make(4, [3, 3, 3], [0, 14, 40], 4, 2, 64, "bf16")
    rope = b.eagle_rope_table(42, 64, 1e4)  # positions 40, 41 exist, 42 does not
    s["table"][1, 1] = s["P"]               # row 2 of request 1 has no page
    q_out = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    before = s["kc"].clone()
    b.eagle_kv_append(s["q"], s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], s["kc"], s["vc"], q_out=q_out,
                      status=s["st"])
    assert s["st"].item() in (1, 6)
    assert (q_out[8] == 7.0).all() and not (q_out[:8] == 7.0).all(-1).any()
    changed = (s["kc"] != before).flatten(2).any(-1).sum().item()
    assert changed == 7


@pytest.mark.parametrize("new,ctx", LENS)
@pytest.mark.parametrize("Hq,Hkv,D,ks,vs", [(4, 2, 64, 1.0, 1.0), (32, 8, 128, 0.25, 0.37), (3, 1, 128, 1.0, 2.5)])
def test_append_kv4_bits(new, ctx, Hq, Hkv, D, ks, vs):
    """Codes and scales are those of the fp32 rotation, bit for bit."""
    b = need_gpu()
    s = make(len(new) * 5 + Hq, new, ctx, Hq, Hkv, D, "bf16", kv4=True)
    rope = b.eagle_rope_table(512, D, 500000.0)
    q_out = torch.empty(s["T"], Hq, D, dtype=torch.bfloat16, device="cuda")
    b.eagle_kv_append_kv4(s["q"], s["k"], s["v"], rope, s["cu"], s["ctx"], s["table"], s["k4"], s["ks"], s["v4"], s["vs"],
                          q_out=q_out, k_scale=ks, v_scale=vs, status=s["st"])
    places = oracle.row_places(s["cu"].cpu().numpy(), ctx, s["table"].cpu().numpy())
    r = rope.cpu().numpy()[[p[1] for p in places]]
    x = s["k"].float().cpu().numpy()
    h = D // 2
    c, n = r[:, 0, None], r[:, 1, None]
    k = np.concatenate([x[..., :h] * c - x[..., h:] * n, x[..., h:] * c + x[..., :h] * n], -1)  # fp32, op by op
    (k4, k4s), (v4, v4s) = oracle.kv4_pack(k, ks), oracle.kv4_pack(s["v"].float().cpu().numpy(), vs)
    for (codes, scales), (gc, gs), new4, news in ((s["pack"][0], ("k4", "ks"), k4, k4s), (s["pack"][1], ("v4", "vs"), v4, v4s)):
        codes, scales = codes.copy(), scales.copy()
        for t, (_, _, page, slot) in enumerate(places):
            codes[page, :, slot], scales[page, :, slot] = new4[t], news[t]
        assert np.array_equal(s[gs].cpu().numpy(), scales) and np.array_equal(s[gc].cpu().numpy(), codes)
    out = torch.empty(s["P"], 16, Hkv, D, dtype=torch.float32, device="cuda")
    b.eagle_kv4_read(s["v4"], s["vs"], out, scale=vs)
    want = oracle.kv4_unpack(s["v4"].cpu().numpy(), s["vs"].cpu().numpy(), float(np.float32(vs))).transpose(0, 2, 1, 3)
    assert np.abs(f64(out) - want).max() <= 2.0 ** -24 * np.abs(want).max()
    assert s["st"].item() == 0


def test_append_kv4_edges():
    b = need_gpu()
    s = make(6, [4], [0], 1, 1, 64, "bf16", kv4=True)
    v = torch.zeros(4, 1, 64)
    v[1, 0, 5], v[2, 0, 20], v[3] = float("nan"), float("inf"), 1e-4
    s["v"] = v.bfloat16().cuda()
    b.eagle_kv_append_kv4(None, s["k"], s["v"], None, s["cu"], s["ctx"], s["table"], s["k4"], s["ks"], s["v4"], s["vs"])
    out = torch.empty(s["P"], 16, 1, 64, device="cuda")
    b.eagle_kv4_read(s["v4"], s["vs"], out)
    got = out[s["table"][0, 0].item(), :4, 0].cpu()
    assert (got[0] == 0).all() and got[1, :16].isnan().all() and (got[1, 16:] == 0).all()
    assert got[2, 20] == 2688 and (got[2, 16:32] != 0).sum() == 1 and (got[3] == 0).all()


def run_attn(b, s, kv4=False, scale=None, ks=1.0, vs=1.0, lse=True):
    out = torch.full((s["T"], s["Hq"], s["D"]), 7.0, dtype=s["q"].dtype, device="cuda")
    l = torch.full((s["T"], s["Hq"]), 7.0, device="cuda") if lse else None
    if kv4:
        b.eagle_prompt_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["ctx"], out, lse=l,
                                scale=scale, k_scale=ks, v_scale=vs, status=s["st"])
    else:
        b.eagle_prompt_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"], out, lse=l, scale=scale, status=s["st"])
    torch.cuda.synchronize()
    return out, l


def check_attn(s, out, lse, p_half, scale=None, ks=1.0, vs=1.0):
    D, cu, ctx = s["D"], s["cu"].cpu().numpy(), s["ctx"].cpu().numpy()
    scale = D ** -0.5 if scale is None else scale
    want, wl, mag, dot = oracle.prompt_attn(f64(s["q"]), gathered(s, s["kc_np"] * ks), gathered(s, s["vc_np"] * vs), cu, ctx,
                                            scale)
    L = max(int(c + n) for c, n in zip(ctx, np.diff(cu)))
    dz = (D + 8) * 2.0 ** -24 * dot
    o_half = HALF["fp32"] if s["q"].dtype == torch.float32 else HALF["bf16"]
    arith = 2 * dz + (L + 16) * 2.0 ** -24
    err = np.abs(f64(out) - want)
    bound = o_half * np.abs(want) + (p_half + arith)[..., None] * mag + 1e-30
    print(f"worst error / bound {float((err / bound).max()):.3f}")
    assert (err <= bound).all(), float((err / bound).max())
    if lse is not None:
        assert (np.abs(f64(lse) - wl) <= dz + arith + 2.0 ** -24 * (np.abs(wl) + 1)).all()
    assert s["st"].item() == 0


ATTN_LENS = [
    ([1], [0]), ([2], [0]), ([1, 1, 1, 1], [0, 15, 127, 128]), ([0, 5, 0, 31, 64, 65, 0], [10, 0, 0, 100, 63, 64, 1]),
    ([128, 129], [0, 0]), ([33], [700]), ([1] * 9, [1000, 3, 500, 127, 128, 129, 255, 256, 900]), ([300], [0]),
    ([257, 1, 70], [1, 600, 250]),
]
HEADS = [(4, 2, 64), (8, 1, 128), (3, 3, 128), (6, 2, 64), (10, 2, 128), (7, 1, 64), (16, 1, 128), (48, 1, 64), (64, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("new,ctx", ATTN_LENS)
@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
def test_attn(new, ctx, Hq, Hkv, D, kind):
    b = need_gpu()
    s = make(sum(new) + Hq, new, ctx, Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4", pad=1)
    out, lse = run_attn(b, s, kind == "kv4")
    check_attn(s, out, lse, dict(fp32=0.0, bf16=HALF["bf16"], kv4=HALF["fp16"])[kind])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
def test_attn_scales_and_no_lse(kind):
    b = need_gpu()
    s = make(77, [50, 3], [90, 200], 8, 2, 128, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    ks, vs = (0.5, 3.0) if kind == "kv4" else (1.0, 1.0)
    out, _ = run_attn(b, s, kind == "kv4", scale=0.3, ks=ks, vs=vs, lse=False)
    check_attn(s, out, None, dict(fp32=0.0, bf16=HALF["bf16"], kv4=HALF["fp16"])[kind], scale=0.3, ks=ks, vs=vs)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_what_is_masked_never_counts(kind, bad):
    """Non-finite K and V behind the mask, past a request's end and in unused
    slots leave every row that does not see them as it was; rows that see them
    are not finite."""
    b = need_gpu()
    new, ctx = [40, 150, 1], [30, 100, 17]
    s = make(5, new, ctx, 8, 2, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    clean, clse = run_attn(b, s, kind == "kv4")
    names = ("ks", "vs") if kind == "kv4" else ("kc", "vc")
    if kind == "kv4" and bad != bad:
        def poison(page, slot):
            for n in names:
                s[n][page, :, slot] = 127
    elif kind == "kv4":
        pytest.skip("4-bit pages hold no infinities")
    else:
        def poison(page, slot):
            for n in names:
                s[n][page, slot] = bad
    hit = {0: 30 + 20, 1: 100 + 149, 2: 18}  # position poisoned; request 2's lies past its end
    for r, pos in hit.items():
        poison(s["table"][r, pos // 16].item(), pos % 16)
    for page in range(s["P"]):
        if page not in s["table"].cpu().numpy():
            for slot in range(16):
                poison(page, slot)
    out, lse = run_attn(b, s, kind == "kv4")
    sees = torch.tensor([c + i >= hit[r] for r, (n, c) in enumerate(zip(new, ctx)) for i in range(n)], device="cuda")
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clse[~sees])
    assert not out[sees].isfinite().all(-1).any()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
def test_attn_bad_pages_and_lengths(kind):
    """A page id out of range reads as zeros; a malformed request is skipped."""
    b = need_gpu()
    s = make(8, [20, 30], [60, 70], 4, 2, 128, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    clean, _ = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 0
    good = s["table"].clone()
    s["table"][0, 2] = s["P"] + 3
    out, _ = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 6
    s["st"].zero_()
    assert torch.equal(out[20:], clean[20:])
    for name in ("kc_np", "vc_np"):
        s[name][good[0, 2].item()] = 0
    s["table"] = good
    check_attn(s, out, None, dict(fp32=0.0, bf16=HALF["bf16"], kv4=HALF["fp16"])[kind])
    s["ctx"][0] = -4
    out, _ = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 1 and (out[:20] == 7.0).all() and torch.equal(out[20:], clean[20:])


def test_graph_and_side_stream():
    b = need_gpu()
    s = make(9, [3, 40, 1], [300, 0, 1500], 8, 2, 128, "bf16")
    want, wl = run_attn(b, s)
    ws = b.workspace(b.eagle_prompt_attn_workspace_size(3, s["T"], 8, 2, 128))
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = lambda: b.eagle_prompt_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"], out, lse=lse, ws=ws)  # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    for _ in range(3):
        out.zero_()
        ws.fill_(255)  # nothing is expected of the workspace's contents
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 4, 128), (16, 1, 64), (16, 1, 128), (32, 8, 128), (14, 2, 64), (9, 3, 128),
                                      (17, 1, 64)])
@pytest.mark.parametrize("new,ctx", [
    ([1], [0]), ([1], [15]), ([1], [16]), ([1], [3000]), ([1, 0, 2, 1], [5, 9, 126, 1023]), ([0, 0, 3], [1, 1, 500]),
    ([1] * 33, [7 * i * i % 911 for i in range(33)]), ([1] * 600, [i % 200 for i in range(600)]),
])
@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_attn_single_tokens(new, ctx, Hq, Hkv, D, kind):
    b = need_gpu()
    s = make(sum(ctx) + Hq, new, ctx, Hq, Hkv, D, "bf16", kv4=kind == "kv4", pad=2)
    out, lse = run_attn(b, s, kind == "kv4")
    check_attn(s, out, lse, dict(bf16=HALF["bf16"], kv4=HALF["fp16"])[kind])


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (12, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("new,ctx", [([2, 2], [700, 15]), ([4, 0], [100, 5]), ([3, 2], [127, 300]), ([1, 1, 4], [0, 2000, 31])])
@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_attn_two_tokens_on_average(new, ctx, Hq, Hkv, D, kind):
    """Around two tokens per request, where 4-bit pages change kernels."""
    b = need_gpu()
    s = make(sum(new) + 3 * Hq, new, ctx, Hq, Hkv, D, "bf16", kv4=kind == "kv4", pad=1)
    out, lse = run_attn(b, s, kind == "kv4")
    check_attn(s, out, lse, dict(bf16=HALF["bf16"], kv4=HALF["fp16"])[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp32", "kv4"])
@pytest.mark.parametrize("new,ctx", [([1, 1], [300, 17]), ([70, 3], [0, 40])])
def test_offsets_past_32_bits(kind, new, ctx):
    """The same pages far into a large pool: the same bits, appended and attended to."""
    b = need_gpu()
    far = {"bf16": 2 ** 18, "fp32": 2 ** 17, "kv4": 2 ** 19}[kind] + 5  # 2^31 elements or 2^32 code bytes
    kv4 = kind == "kv4"
    s = make(14, new, ctx, 16, 8, 128, "fp32" if kind == "fp32" else "bf16", kv4=kv4)
    names = ("k4", "ks", "v4", "vs") if kv4 else ("kc", "vc")
    big = dict(s, table=torch.where(s["table"] >= 0, s["table"] + far, s["table"]))
    for n in names:
        big[n] = torch.empty((far + s["P"],) + tuple(s[n].shape[1:]), dtype=s[n].dtype, device="cuda")
        big[n][far:] = s[n]
    rope = b.eagle_rope_table(512, 128, 500000.0)
    res = []
    for x in (s, big):
        q = torch.empty((x["T"], 16, 128), dtype=x["q"].dtype, device="cuda")
        if kv4:
            b.eagle_kv_append_kv4(x["q"], x["k"], x["v"], rope, x["cu"], x["ctx"], x["table"], x["k4"], x["ks"], x["v4"],
                                  x["vs"], q_out=q, status=x["st"])
        else:
            b.eagle_kv_append(x["q"], x["k"], x["v"], rope, x["cu"], x["ctx"], x["table"], x["kc"], x["vc"], q_out=q,
                              status=x["st"])
        res.append(run_attn(b, dict(x, q=q), kv4))
    for n in names:
        assert torch.equal(big[n][far:].view(torch.uint8), s[n].view(torch.uint8))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert s["st"].item() == 0


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("new", [[1], [40]])
def test_attn_growing_scores(new, kind):
    """Scores that rise along the keys, by more than the weights' type can hold
    against the first maximum: the reference has to move."""
    b = need_gpu()
    s = make(12, new, [2000], 8, 2, 64, "bf16", kv4=kind == "kv4")
    n = 2000 + new[0]
    k = torch.randn(n, 2, 64)
    u = torch.randn(2, 64)
    u /= u.norm(dim=-1, keepdim=True)
    k = 0.1 * k + u * torch.linspace(-12, 12, n)[:, None, None]
    s["q"] = (u.repeat_interleave(4, 0)[None] * 20 + torch.randn(new[0], 8, 64)).bfloat16().cuda()
    pages = s["table"][0].long().cpu()
    pos = torch.arange(n)
    if kind == "kv4":
        full = torch.from_numpy(s["kc_np"]).float()
        full[pages[pos // 16], pos % 16] = k
        codes, scales = oracle.kv4_pack(full.transpose(1, 2).numpy())
        s["k4"], s["ks"] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
        s["kc_np"] = oracle.kv4_unpack(codes, scales).transpose(0, 2, 1, 3)
    else:
        s["kc"][pages[pos // 16].cuda(), pos.cuda() % 16] = k.bfloat16().cuda()
        s["kc_np"] = f64(s["kc"])
    out, lse = run_attn(b, s, kind == "kv4")
    check_attn(s, out, lse, dict(bf16=HALF["bf16"], kv4=HALF["fp16"])[kind])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_attn_single_token_nan_and_bad_page(kind):
    b = need_gpu()
    s = make(13, [1, 1], [40, 60], 8, 2, 128, "bf16", kv4=kind == "kv4")
    clean, clse = run_attn(b, s, kind == "kv4")
    names = ("ks", "vs") if kind == "kv4" else ("kc", "vc")
    bad = 127 if kind == "kv4" else float("nan")
    page = s["table"][0, 41 // 16].item()
    for n in names:  # past request 0's end
        if kind == "kv4":
            s[n][page, :, 41 % 16] = bad
        else:
            s[n][page, 41 % 16] = bad
    out, lse = run_attn(b, s, kind == "kv4")
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    page = s["table"][1, 0].item()
    for n in names:
        if kind == "kv4":
            s[n][page, 0, 3] = bad
        else:
            s[n][page, 3, 0] = bad
    out, lse = run_attn(b, s, kind == "kv4")
    assert torch.equal(out[0], clean[0]) and out[1, :4].isnan().all() and torch.equal(out[1, 4:], clean[1, 4:])
    assert s["st"].item() == 0
    s["table"][1, 0] = -7
    out, _ = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 6 and out.isfinite().all() and torch.equal(out[0], clean[0])


@pytest.mark.parametrize("kind,new,ctx", [("bf16", [37, 0, 5], [0, 20, 16]), ("fp32", [9, 4], [0, 30]), ("kv4", [37, 5], [0, 16]),
                                          ("bf16", [4100], [0])])
def test_draft_prompt(kind, new, ctx):
    """The layer over the prompt against the oracle's pieces, storing where the
    call stores; the cache then holds what the oracle's append gives."""
    b = need_gpu()
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    d, Hq, Hkv, D, I = 256, 4, 2, 64, 128
    s = make(21, new, ctx, Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    g = torch.Generator().manual_seed(3)
    rn = lambda *sh, k=0.05: (torch.randn(*sh, generator=g) * k).to(dt)  # noqa: E731
    W = dict(norm1=1 + rn(d), qkv=rn((Hq + 2 * Hkv) * D, d), o=rn(d, Hq * D), norm2=1 + rn(d), gu=rn(2 * I, d), down=rn(d, I))
    x = rn(s["T"], d, k=1.0)
    rope = b.eagle_rope_table(max(n + c for n, c in zip(new, ctx)), D, 1e4)
    out = torch.empty(s["T"], d, dtype=dt, device="cuda")
    Wc = {k: v.cuda() for k, v in W.items()}
    kw = dict(k_scales=s["ks"], v_scales=s["vs"]) if kind == "kv4" else {}
    names = ("k4", "v4") if kind == "kv4" else ("kc", "vc")
    b.eagle_draft_prompt(x.cuda(), Wc, rope, s["cu"], s["ctx"], s[names[0]], s[names[1]], s["table"], out, status=s["st"], **kw)
    st = (lambda a: torch.from_numpy(a).to(dt).double().numpy()) if dt != torch.float32 else (lambda a: a.astype(np.float32).astype(np.float64))
    w = {k: v.double().numpy() for k, v in W.items()}
    cu = s["cu"].cpu().numpy()
    places = oracle.row_places(cu, ctx, s["table"].cpu().numpy())
    qkv = st(oracle.linear(st(oracle.rms_norm(x.double().numpy(), w["norm1"], 1e-5)), w["qkv"])).reshape(s["T"], -1, D)
    r = f64(rope)[[p[1] for p in places]]
    q, k, v = st(oracle.rotate(qkv[:, :Hq], r)), oracle.rotate(qkv[:, Hq:Hq + Hkv], r), qkv[:, Hq + Hkv:]
    if kind == "kv4":
        k, v = (oracle.kv4_unpack(*oracle.kv4_pack(a.astype(np.float32))) for a in (k, v))
    else:
        k = st(k)
    for t, (_, _, page, slot) in enumerate(places):
        s["kc_np"][page, slot], s["vc_np"][page, slot] = k[t], v[t]
    a = st(oracle.prompt_attn(q, gathered(s, s["kc_np"]), gathered(s, s["vc_np"]), cu, ctx, D ** -0.5)[0]).reshape(s["T"], -1)
    x1 = st(oracle.linear(a, w["o"], residual=x.double().numpy()))
    gu = st(oracle.linear(st(oracle.rms_norm(x1, w["norm2"], 1e-5)), w["gu"]))
    want = oracle.linear(st(oracle.silu(gu[:, :I]) * gu[:, I:]), w["down"], residual=x1)
    # each stored intermediate may round the other way by one step where the
    # sums differ in fp32: a handful of roundings of the output's size, and for
    # 4-bit pages a code may fall the other side of a midpoint
    tol = {"fp32": 1e-5, "bf16": 4 * 2.0 ** -8, "kv4": 6 * 2.0 ** -8}[kind]
    err = np.abs(f64(out) - want)
    print(f"{kind}: worst {float((err / (np.abs(want) + 1)).max()):.2e} of {tol:.2e}")
    assert (err <= tol * (np.abs(want) + 1)).all() and s["st"].item() == 0


def test_prompt_then_draft_layer():
    """A prompt through eagle_draft_prompt, then the next row through
    eagle_draft_layer over the cache it filled, equals the whole prompt with
    that row through eagle_draft_prompt."""
    b = need_gpu()
    d, Hq, Hkv, D, I, n = 256, 4, 2, 64, 128, 50
    s = make(22, [n + 1], [0], Hq, Hkv, D, "bf16")
    g = torch.Generator().manual_seed(4)
    rn = lambda *sh, k=0.05: (torch.randn(*sh, generator=g) * k).bfloat16().cuda()  # noqa: E731
    W = dict(norm1=1 + rn(d), qkv=rn((Hq + 2 * Hkv) * D, d), o=rn(d, Hq * D), norm2=1 + rn(d), gu=rn(2 * I, d), down=rn(d, I))
    x, rope = rn(n + 1, d, k=1.0), b.eagle_rope_table(64, D, 1e4)
    whole = torch.empty_like(x)
    b.eagle_draft_prompt(x, W, rope, s["cu"], s["ctx"], s["kc"], s["vc"], s["table"], whole)
    s["kc"].fill_(float("nan"))
    part = torch.empty(n, d, dtype=x.dtype, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    b.eagle_draft_prompt(x[:n].contiguous(), W, rope, cu, s["ctx"], s["kc"], s["vc"], s["table"], part)
    assert torch.equal(part[:32], whole[:32]) or (part - whole[:n]).abs().max() < 0.05
    z = lambda *sh: torch.zeros(*sh, dtype=x.dtype, device="cuda")  # noqa: E731
    out = torch.empty(1, d, dtype=x.dtype, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    b.eagle_draft_layer(x[n:].contiguous(), W, i32([n]).view(1, 1), s["kc"], s["vc"], s["table"], i32(n), z(1, 8, Hq, D),
                        z(1, 8, Hkv, D), z(1, 8, Hkv, D), (1 << torch.arange(8)).view(1, 8).cuda(), 0, out, theta=1e4)
    assert (out[0].float() - whole[n].float()).abs().max() <= 4 * 2.0 ** -8 * (1 + whole[n].float().abs().max())
