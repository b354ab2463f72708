"""GPU parity of the attention over shared prefixes against the fp64 oracle.

Tolerances count roundings, as for the causal attention: the output's rounding,
the rounding of the weights to the matrix type (bf16 2^-8, fp16 2^-11 for 4-bit
pages, none in fp32) against sum w|v| of the prefix, and fp32 arithmetic: a score
is off by at most dz = (D + 8) 2^-24 scale sum|q k|, a weight by 2 dz relative, a
sum of L terms by (L + 16) 2^-24; the own part's weight by 2^-21 more (its
exponential 2^-22, its argument and the quotient), against sum w|v| of both.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu
from test_gpu_prompt import HALF, f64, gathered, make

pytestmark = pytest.mark.gpu
KINDS = ["fp32", "bf16", "kv4"]
P_HALF = dict(fp32=0.0, bf16=HALF["bf16"], kv4=HALF["fp16"])


def setup(kind, rows, lens, Hq, Hkv, D, seed, own=True, pad=1):
    """q of all rows, the groups' pages, and the rows' own results."""
    s = make(seed, rows, [max(0, L - n) for n, L in zip(rows, lens)], Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16",
             kv4=kind == "kv4", pad=pad)
    g = torch.Generator().manual_seed(seed + 1)
    T = s["T"]
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["own_out"] = torch.randn(T, Hq, D, generator=g).to(s["q"].dtype).cuda() if own else None
    spread = torch.tensor([np.log(max(L, 1)) for n, L in zip(rows, lens) for _ in range(n)])[:, None]
    s["own_lse"] = (spread + 2 * torch.randn(T, Hq, generator=g)).float().cuda() if own else None
    return s


def run(b, s, kind, scale=None, ks=1.0, vs=1.0, lse=True, **kw):
    T, Hq, D = s["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=s["q"].dtype, device="cuda")
    ls = torch.full((T, Hq), 7.0, device="cuda") if lse else None
    args = dict(lse=ls, own_out=s["own_out"], own_lse=s["own_lse"], scale=scale, status=s["st"], **kw)
    if kind == "kv4":
        b.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["lens"], out, k_scale=ks,
                                v_scale=vs, **args)
    else:
        b.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], out, **args)
    return out, ls


def check(s, out, lse, kind, scale=None, ks=1.0, vs=1.0):
    T, Hq, D = s["q"].shape
    scale = D ** -0.5 if scale is None else scale
    lens = s["lens"].tolist()
    keys, values = ([x[:n] for x, n in zip(gathered(s, s[c] * f), lens)] for c, f in (("kc_np", ks), ("vc_np", vs)))
    own = (None, None) if s["own_out"] is None else (f64(s["own_out"]), f64(s["own_lse"]))
    want, wl, mag, both, dot = oracle.prefix_attn(f64(s["q"]), keys, values, s["cu"].tolist(), scale, *own)
    dz = (D + 8) * 2.0 ** -24 * dot
    if kind == "kv4":
        dz = dz + 2.0 ** -24 * dot  # a row of q in fp16: 2^-25 of its largest for what lies below 2^-14 of it
    arith = 2 * dz + (max(lens + [0]) + 16) * 2.0 ** -24 + 2.0 ** -21
    o_half = HALF["fp32" if kind == "fp32" else "bf16"]
    err = np.abs(f64(out) - want)
    bound = o_half * np.abs(want) + P_HALF[kind] * mag + arith[..., None] * both + 1e-30
    print(f"worst error / bound {float((err / bound).max()):.3f}")
    assert (err <= bound).all(), float((err / bound).max())
    if lse is not None:
        got = f64(lse)
        fine = np.isfinite(wl)
        assert np.array_equal(got[~fine], wl[~fine])
        assert (np.abs(got - wl)[fine] <= (dz + arith + 2.0 ** -23 * (np.abs(wl) + 1))[fine]).all()
    assert s["st"].item() == 0


GROUPS = [
    ([1], [1]), ([1], [16]), ([2], [17]), ([1, 1, 1, 1], [1, 127, 128, 129]), ([0, 5, 0, 31, 64, 65, 0], [10, 1, 0, 100, 63, 300, 1]),
    ([33], [700]), ([64], [2000]), ([3, 4, 2], [0, 400, 0]), ([200], [300]), ([300, 1, 70], [15, 5000, 250]), ([1] * 40, [100] * 40),
    ([5], [0]), ([130], [1040]),
]
HEADS = [(4, 2, 64), (8, 1, 128), (3, 3, 128), (10, 2, 128), (7, 1, 64), (48, 1, 64), (64, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("rows,lens", GROUPS)
@pytest.mark.parametrize("kind", KINDS)
def test_prefix(rows, lens, Hq, Hkv, D, kind):
    b = need_gpu()
    s = setup(kind, rows, lens, Hq, Hkv, D, sum(rows) + Hq)
    out, lse = run(b, s, kind)
    check(s, out, lse, kind)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (14, 2, 64)])
@pytest.mark.parametrize("rows,lens", [([64], [4000]), ([4], [20000]), ([700, 300], [900, 1500]), ([9] * 70, [130] * 69 + [2000])])
@pytest.mark.parametrize("kind", KINDS)
def test_prefix_larger(rows, lens, Hq, Hkv, D, kind):
    b = need_gpu()
    if kind == "fp32" and sum(rows) > 500:
        rows, lens = [r // 4 + 1 for r in rows], lens
    s = setup(kind, rows, lens, Hq, Hkv, D, len(rows) + Hq)
    out, lse = run(b, s, kind)
    check(s, out, lse, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", [([20, 3], [90, 700]), ([64], [0]), ([2, 2], [0, 1])])
def test_prefix_alone_and_scales(rows, lens, kind):
    """Without own results, with a scale of its own, cache scales, and no lse asked for."""
    b = need_gpu()
    ks, vs = (0.5, 3.0) if kind == "kv4" else (1.0, 1.0)
    s = setup(kind, rows, lens, 8, 2, 128, 77, own=False)
    out, lse = run(b, s, kind, scale=0.3, ks=ks, vs=vs)
    check(s, out, lse, kind, scale=0.3, ks=ks, vs=vs)
    s2 = setup(kind, rows, lens, 8, 2, 128, 77)
    out, _ = run(b, s2, kind, scale=0.3, ks=ks, vs=vs, lse=False)
    check(s2, out, None, kind, scale=0.3, ks=ks, vs=vs)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", [([70, 5], [300, 1000]), ([1, 1], [40, 0]), ([600], [200])])
def test_rows_without_own_keys(rows, lens, kind):
    """own_lse = -infinity: own_out is not read, NaN or not; own_lse far above and far below the prefix's."""
    b = need_gpu()
    s = setup(kind, rows, lens, 4, 2, 64, 5)
    s["own_lse"][::2, 1] = -torch.inf
    s["own_out"][::2, 1] = torch.nan
    s["own_lse"][::3, 2] = 300.0
    s["own_lse"][1::3, 3] = -300.0
    out, lse = run(b, s, kind)
    check(s, out, lse, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", [([64], [3000]), ([500, 40], [200, 0]), ([3], [129])])
def test_in_place(rows, lens, kind):
    """out and lse are own_out and own_lse themselves."""
    b = need_gpu()
    s = setup(kind, rows, lens, 8, 2, 128, 6)
    want, wl = run(b, s, kind)
    out, lse = s["own_out"].clone(), s["own_lse"].clone()
    s["own_out"], s["own_lse"] = out, lse
    args = dict(lse=lse, own_out=out, own_lse=lse, status=s["st"])
    if kind == "kv4":
        b.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["lens"], out, **args)
    else:
        b.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], out, **args)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", [([40, 150, 1], [130, 250, 18]), ([9, 8, 7], [129, 2500, 1])])
def test_what_lies_past_a_prefix_never_counts(rows, lens, kind):
    """NaN in unused slots, unused pages and other groups' pages leaves a group's rows as they were."""
    b = need_gpu()
    s = setup(kind, rows, lens, 8, 2, 64, 8)
    clean, clse = run(b, s, kind)
    names = ("ks", "vs") if kind == "kv4" else ("kc", "vc")
    used = {}
    for g, L in enumerate(lens):
        for pos in range(L):
            used.setdefault(s["table"][g, pos // 16].item(), set()).add(pos % 16)
    for n in names:
        for page in range(s["P"]):
            for slot in range(16):
                if slot not in used.get(page, ()):
                    if kind == "kv4":
                        s[n][page, :, slot] = 127
                    else:
                        s[n][page, slot] = torch.nan
    out, lse = run(b, s, kind)
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    # and within group 0 every row sees it
    if kind == "kv4":
        s["vs"][s["table"][0, 0].item(), :, 3] = 127
    else:
        s["vc"][s["table"][0, 0].item(), 3] = torch.nan
    out, lse = run(b, s, kind)
    n = rows[0]
    assert out[:n].isnan().all() and torch.equal(out[n:], clean[n:]) and torch.equal(lse, clse)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,lens", [([5], [300]), ([80, 3], [260, 2100])])
def test_scores_of_minus_infinity(rows, lens, kind):
    """Keys that score -infinity weigh nothing beside others; where all of them do,
    the own result is left, or zeros and -infinity."""
    b = need_gpu()
    s = setup(kind, rows, lens, 4, 2, 64, 9)
    s["q"].abs_()
    first = s["table"][0].tolist()
    for pos in range(lens[0]):
        s["kc"][first[pos // 16], pos % 16, 0] = -torch.inf  # kv head 0 of group 0: all
        if pos < 200:
            s["kc"][first[pos // 16], pos % 16, 1] = -torch.inf  # kv head 1: the first 200
    s["own_lse"][0, :2] = -torch.inf
    out, lse = run(b, s, kind)
    n = rows[0]
    assert (out[0, :2] == 0).all() and (lse[0, :2] == -torch.inf).all()
    assert torch.equal(out[1:n, :2], s["own_out"][1:n, :2]) and torch.equal(lse[1:n, :2], s["own_lse"][1:n, :2])
    # heads 2, 3 of group 0: as over the keys from 200 on
    keys, values = f64(s["kc"]), f64(s["vc"])
    k0, v0 = (gathered(s, c)[0][200:lens[0], 1:] for c in (keys, values))
    want, wl, *_ = oracle.prefix_attn(f64(s["q"][:n, 2:]), [k0], [v0], [0, n], 64 ** -0.5, f64(s["own_out"][:n, 2:]),
                                      f64(s["own_lse"][:n, 2:]))
    assert np.abs(f64(out[:n, 2:]) - want).max() <= (0.05 if kind == "bf16" else 1e-4)
    assert np.abs(f64(lse[:n, 2:]) - wl).max() <= 1e-4


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths(kind):
    """A page id out of range reads as zeros; a malformed group is skipped; the others are not affected."""
    b = need_gpu()
    rows, lens = [20, 30, 4], [160, 700, 50]
    s = setup(kind, rows, lens, 4, 2, 128, 10)
    clean, clse = run(b, s, kind)
    good, good_lens, good_cu = s["table"].clone(), s["lens"].clone(), s["cu"].clone()
    for bad_id in (s["P"], -1, 2 ** 31 - 1):
        s["table"][0, 2] = bad_id
        out, _ = run(b, s, kind)
        assert s["st"].item() == 6 and torch.equal(out[20:], clean[20:]) and not torch.equal(out[:20], clean[:20])
        s["st"].zero_()
        s["table"] = good.clone()
    width = good.shape[1]
    for value, code in ((-1, 1), (16 * width + 1, 6), (2 ** 31 - 1, 6)):
        s["lens"][1] = value
        out, lse = run(b, s, kind)
        assert s["st"].item() == code
        s["st"].zero_()
        assert (out[20:50] == 7).all() and (lse[20:50] == 7).all()
        # (the work is shared out otherwise: the same values from other partial sums)
        for part in (slice(0, 20), slice(50, 54)):
            assert (out[part].float() - clean[part].float()).abs().max() <= 2 ** -6 * clean[part].abs().max()
            assert (lse[part] - clse[part]).abs().max() <= 1e-5
        s["lens"] = good_lens.clone()
    for at, value in ((0, 3), (3, 52)):  # rows in front of the first group, behind the last
        s["cu"][at] = value
        out, _ = run(b, s, kind)
        assert s["st"].item() == 1
        s["st"].zero_()
        out_of = slice(0, 3) if at == 0 else slice(52, 54)
        keep = slice(3, 54) if at == 0 else slice(0, 52)
        assert (out[out_of] == 7).all()
        assert (out[keep].float() - clean[keep].float()).abs().max() <= 2 ** -6 * clean.abs().max()
        s["cu"] = good_cu.clone()
    for cu in ([0, 50, 20, 54], [0, 20, 50, 40], [0, 20, 60, 54], [-1, 20, 50, 54]):
        s["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        out, _ = run(b, s, kind)
        assert s["st"].item() == 1
        s["st"].zero_()
        if any(y < x for x, y in zip(cu, cu[1:])):
            assert (out == 7).all()
        s["cu"] = good_cu.clone()
    out, lse = run(b, s, kind)
    assert torch.equal(out, clean) and s["st"].item() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_two_groups_may_share_pages(kind):
    """One prefix the start of the other: the same pages in both tables."""
    b = need_gpu()
    s = setup(kind, [6, 9], [300, 300], 4, 2, 64, 11)
    s["table"][1] = s["table"][0]
    s["lens"][1] = 77
    out, lse = run(b, s, kind)
    check(s, out, lse, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 40])
def test_offsets_past_32_bits(kind, rows):
    """Pages whose byte offsets lie past 2^32 (2^33 in the larger types)."""
    b = need_gpu()
    Hq, Hkv, D, L = 4, 4, 128, 300
    per = Hkv * 16 * D
    P = (1 << 33) // per + 40
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    g = torch.Generator().manual_seed(3)
    pages = torch.cat([torch.arange(10) + P - 12, torch.arange(9) + 3]).int()[torch.randperm(19, generator=g)]
    table = pages[None].clone()
    s = dict(table=table.cuda(), cu=torch.tensor([0, rows], dtype=torch.int32).cuda(), lens=torch.tensor([L], dtype=torch.int32).cuda(),
             q=torch.randn(rows, Hq, D, generator=g).to(dt).cuda(), st=torch.zeros(1, dtype=torch.int32).cuda(), own_out=None, own_lse=None)
    pool = torch.randn(2, 19, 16, Hkv, D, generator=g)
    small = dict(s, table=torch.arange(19, dtype=torch.int32)[None].cuda())
    at = pages.long().cuda()
    if kind == "kv4":
        for n, (c, sc) in zip("kv", [oracle.kv4_pack(x.transpose(1, 2).numpy()) for x in pool]):
            small[n + "4"], small[n + "s"] = torch.from_numpy(c).cuda(), torch.from_numpy(sc).cuda()
            for name in (n + "4", n + "s"):
                s[name] = torch.zeros(P, *small[name].shape[1:], dtype=torch.uint8, device="cuda")
                s[name][at] = small[name]
    else:
        for n, x in zip(("kc", "vc"), pool):
            small[n] = x.to(dt).cuda()
            s[n] = torch.zeros(P, 16, Hkv, D, dtype=dt, device="cuda")
            s[n][at] = small[n]
    out, lse = run(b, s, kind)
    want, wl = run(b, small, kind)
    assert torch.equal(out, want) and torch.equal(lse, wl) and s["st"].item() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_graph_streams_and_one_workspace(kind):
    """Captured calls of different shapes with one workspace, replayed after their
    inputs changed; and a call on a stream of its own without a workspace."""
    b = need_gpu()
    cases = [setup(kind, r, L, 8, 2, 64, 12 + len(r)) for r, L in (([64], [900]), ([3, 1], [40, 2000]), ([300], [150]))]
    ws = b.workspace(max(b.eagle_prefix_attn_workspace_size(len(s["lens"]), s["T"], 8, 2, 64) for s in cases))
    first = [run(b, s, kind, ws=ws) for s in cases]
    torch.cuda.synchronize()
    graph, outs = torch.cuda.CUDAGraph(), None
    with torch.cuda.graph(graph):
        outs = [run(b, s, kind, ws=ws) for s in cases]
    for round_ in range(2):
        for o, l in outs:
            o.zero_()
            l.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = first if round_ == 0 else [run(b, s, kind) for s in cases]
        for (o, l), (x, y) in zip(outs, want):
            assert torch.equal(o, x) and torch.equal(l, y)
        for s in cases:
            s["lens"].sub_(7).clamp_(min=0)
            s["q"].mul_(0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in outs]
    for s, (o, l) in zip(cases, outs):
        args = dict(lse=l, own_out=s["own_out"], own_lse=s["own_lse"], status=s["st"], stream=side)
        if kind == "kv4":
            b.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["lens"], o, **args)
        else:
            b.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], o, **args)
    side.synchronize()
    for s, (o, l) in zip(cases, outs):
        check(s, o, l, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_prefix_and_own_keys_are_the_whole_attention(kind):
    """Rows of requests behind a shared prefix: own attention and the prefix's, joined,
    against the causal attention over requests that each hold all their keys."""
    b = need_gpu()
    P, new, ctx, Hq, Hkv, D = 333, [1, 4, 0, 17], [5, 0, 9, 300], 8, 2, 128
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    s = setup(kind, [sum(new)], [P], Hq, Hkv, D, 14)
    own = make(15, new, ctx, Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    q, T = s["q"], sum(new)
    out, lse = torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hq, device="cuda")
    if kind == "kv4":
        b.eagle_prompt_attn_kv4(q, own["k4"], own["ks"], own["v4"], own["vs"], own["table"], own["cu"], own["ctx"], out, lse=lse)
    else:
        b.eagle_prompt_attn(q, own["kc"], own["vc"], own["table"], own["cu"], own["ctx"], out, lse=lse)
    s["own_out"], s["own_lse"] = out, lse
    got, gl = run(b, s, kind)
    pre = [gathered(s, s[c])[0][:P] for c in ("kc_np", "vc_np")]
    keys, values = ([np.concatenate([p, x[:n + c]]) for x, n, c in zip(gathered(own, own[name]), new, ctx)]
                    for p, name in zip(pre, ("kc_np", "vc_np")))
    want, wl, mag, dot = oracle.prompt_attn(f64(q), keys, values, own["cu"].tolist(), [P + c for c in ctx], D ** -0.5)
    half = HALF["fp32" if kind == "fp32" else "bf16"]
    # the own result is rounded to the type, and then the joined one; both have rounded weights
    arith = (2 * (D + 9) * dot + 700 + 32) * 2.0 ** -24 + 2.0 ** -21
    assert (np.abs(f64(got) - want) <= half * np.abs(want) + (half + P_HALF[kind] + arith[..., None]) * mag).all()
    assert np.abs(f64(gl) - wl).max() <= 1e-4


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (32, 8, 128)])
@pytest.mark.parametrize("own", [True, False])
def test_many_rows_of_empty_prefixes(kind, Hq, Hkv, D, own):
    """Their own results to the bit, by many CTAs; rows without keys of their own zeros, whatever
    own_out holds; beside a group that has a prefix, and in place."""
    b = need_gpu()
    s = setup(kind, [0, 700, 3, 41, 0], [0, 0, 60, 0, 5], Hq, Hkv, D, 16, own=own)
    if own:
        s["own_lse"][::7] = -torch.inf
        s["own_out"][::7] = torch.nan
    out, lse = run(b, s, kind)
    assert s["st"].item() == 0
    rows = torch.cat([torch.arange(700), torch.arange(703, 744)]).cuda()
    if not own:
        assert (out[rows] == 0).all() and (lse[rows] == -torch.inf).all()
        return
    want = torch.where((s["own_lse"] == -torch.inf)[..., None], 0.0, s["own_out"])
    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], s["own_lse"][rows])
    args = dict(lse=s["own_lse"], own_out=s["own_out"], own_lse=s["own_lse"], status=s["st"])
    if kind == "kv4":
        b.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["lens"], s["own_out"], **args)
    else:
        b.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], s["own_out"], **args)
    assert torch.equal(s["own_out"], out) and torch.equal(s["own_lse"], lse)
