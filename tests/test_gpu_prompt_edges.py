"""GPU parity of the prompt path where it is easily got wrong: many pieces per
CTA, scores at the ends of their range, malformed lengths.  Helpers and
tolerances are those of test_gpu_prompt."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu
from test_gpu_prompt import HALF, check_attn, f64, make, run_attn

pytestmark = pytest.mark.gpu

WEIGHT_HALF = dict(bf16=HALF["bf16"], kv4=HALF["fp16"], fp32=0.0)


def set_keys(s, kind, values, which="k"):
    """Writes values[b] [n, Hkv, D] to the slots of request b's positions 0 .. n - 1."""
    name = which + "c_np"
    full = torch.from_numpy(s[name]).float().clone()
    table = s["table"].long().cpu()
    for b, x in enumerate(values):
        p = torch.arange(len(x))
        full[table[b, p // 16], p % 16] = x
    if kind == "kv4":
        codes, scales = oracle.kv4_pack(full.transpose(1, 2).numpy())
        s[which + "4"], s[which + "s"] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
        s[name] = oracle.kv4_unpack(codes, scales).transpose(0, 2, 1, 3)
    else:
        s[which + "c"] = full.to(s["q"].dtype).cuda()
        s[name] = f64(s[which + "c"])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("back", [1, 2])
def test_attn_many_two_tile_pieces_per_cta(kind, D, back):
    """More short units than SMs, so that every CTA takes several pieces of two
    tiles, with full, partly filled and single tiles among them.  The rows of
    the second tile meet, in their last or last but one block, keys that make
    them renew their reference while the first tile's rows do not."""
    b = need_gpu()
    Hq, Hkv, B = 32, 8, 60
    new = [(64, 64, 40, 64, 20)[i % 5] for i in range(B)]
    ctx = [130 + 61 * i % 400 for i in range(B)]
    s = make(31 + D, new, ctx, Hq, Hkv, D, "bf16", kv4=kind == "kv4")
    g = torch.Generator().manual_seed(17)
    u = torch.randn(Hkv, D, generator=g)
    u /= u.norm(dim=-1, keepdim=True)
    keys, q = [], []
    for n, c in zip(new, ctx):
        k = 0.3 * torch.randn(c + n, Hkv, D, generator=g)
        last = (c + n - 1) // 128
        k[max(0, last + 1 - back) * 128:(last + 2 - back) * 128] += 4 * u
        keys.append(k)
        x = torch.randn(n, Hq, D, generator=g)
        x[:32] -= 4 * u.repeat_interleave(4, 0)   # the first tile's rows turn away from those keys
        x[32:] += 4 * D ** 0.5 * u.repeat_interleave(4, 0)  # 16 in the exponent
        q.append(x)
    set_keys(s, kind, keys)
    s["q"] = torch.cat(q).bfloat16().cuda()
    out, lse = run_attn(b, s, kind == "kv4")
    check_attn(s, out, lse, WEIGHT_HALF[kind])
    again, lse2 = run_attn(b, s, kind == "kv4")
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("n,count,ctx", [(1, 40, 600), (1, 3, 3000), (2, 5, 700), (40, 3, 500)])
def test_attn_first_keys_of_minus_infinity(kind, n, count, ctx):
    """Scores of minus infinity over the first 128 + 64 keys, a plain softmax
    over the others: a row has no reference until it meets a finite score."""
    b = need_gpu()
    Hq, Hkv, D, low = 16, 8, 64, 192
    s = make(41 + n, [n] * count, [ctx] * count, Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    # channel 0 alone carries the scores: 2^119 * 2 * -6 overflows to minus
    # infinity, and the other keys have 0 there
    q = torch.zeros(s["T"], Hq, D)
    q[..., 0] = 2.0
    s["q"] = q.to(s["q"].dtype).cuda()
    key = torch.zeros(ctx + n, Hkv, D)
    key[:low, :, 0] = -2688.0
    set_keys(s, kind, [key] * count)
    assert (s["kc_np"][s["table"][0, 0].item(), 0, :, 0] < -2000).all()
    out, lse = run_attn(b, s, kind == "kv4", scale=2.0 ** 119)
    # the softmax over what is left, all scores 0
    v = [x[low:] for x in (s["vc_np"][t].reshape(-1, Hkv, D) for t in s["table"].cpu().numpy())]
    half = HALF["fp32"] if kind == "fp32" else HALF["bf16"]
    for r in range(s["T"]):
        seen = ctx + r % n + 1 - low
        x = np.repeat(v[r // n][:seen], Hq // Hkv, 1)
        want, mag = x.mean(0), np.abs(x).mean(0)
        err = np.abs(f64(out[r]) - want)
        assert (err <= half * np.abs(want) + (WEIGHT_HALF[kind] + (ctx + 16) * 2.0 ** -24) * mag).all()
        assert np.abs(f64(lse[r]) - np.log(seen)).max() <= 2.0 ** -20
    assert s["st"].item() == 0


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("new,ctx", [([1] * 3, [5, 300, 2500]), ([40, 3, 70], [0, 300, 260])])
def test_attn_rows_whose_scores_are_all_minus_infinity(kind, new, ctx):
    """Such a row gives zeros and an lse of minus infinity; its neighbours are as they were."""
    b = need_gpu()
    Hq, Hkv, D = 8, 4, 128
    s = make(43, new, ctx, Hq, Hkv, D, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    key = [torch.randn(c + n, Hkv, D, generator=torch.Generator().manual_seed(c)) for n, c in zip(new, ctx)]
    for k in key:
        k[..., 0] = 8.0
    set_keys(s, kind, key)
    clean, clse = run_attn(b, s, kind == "kv4")
    dead = torch.zeros(s["T"], Hq, dtype=torch.bool, device="cuda")
    dead[1::3, 2] = dead[0, 7] = dead[2, :] = True
    q = s["q"].clone()
    q[dead] = 0
    q[..., 0] = torch.where(dead, torch.full_like(q[..., 0], -float("inf")), q[..., 0])
    s["q"] = q
    # every dead row's score is -inf * 8 + 0 * k = -inf: no NaN among its products
    out, lse = run_attn(b, s, kind == "kv4")
    assert (out[dead] == 0).all() and (lse[dead] == -float("inf")).all()
    assert torch.equal(out[~dead], clean[~dead]) and torch.equal(lse[~dead], clse[~dead])


@pytest.mark.parametrize("new,ctx", [([1] * 5, [3, 40, 300, 200, 1000]), ([40, 9, 150], [100, 0, 260])])
@pytest.mark.parametrize("k_scale", [1.0, 2.0 ** -24, 2.0 ** -60])
def test_attn_kv4_rows_of_zeros(new, ctx, k_scale):
    """A query of zeros, or one whose factor leaves fp32's range, weighs every key alike."""
    b = need_gpu()
    s = make(47, new, ctx, 8, 2, 128, "bf16", kv4=True)
    q = s["q"].clone()
    q[::2, 1::2] = 0.0
    q[1::2, ::3] *= 2.0 ** -120
    q[0, 0] = 2.0 ** -130  # below bf16's normal numbers
    s["q"] = q
    out, lse = run_attn(b, s, True, ks=k_scale)
    check_attn(s, out, lse, HALF["fp16"], ks=k_scale)


@pytest.mark.parametrize("n,count,ctx", [(1, 20, 16383), (40, 8, 16300)])
@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("down", [20.3, 25.7])
def test_attn_leading_key_over_a_flat_tail(kind, n, count, ctx, down):
    """One key outweighs each of a long tail by 2^down, and its value is zero:
    the output is the tail's.  fp16 holds a weight 2^(z - m) with m 7 below the
    first maximum, so beside its 2^-11 a weight is off by at most half of
    fp16's smallest step, 2^-25, relative to a sum of at least 2^7."""
    b = need_gpu()
    Hq, Hkv, D = 16, 8, 64
    s = make(53, [n], [ctx], Hq, Hkv, D, "bf16", kv4=kind == "kv4")
    k, v = torch.zeros(ctx + n, Hkv, D), torch.randn(ctx + n, Hkv, D, generator=torch.Generator().manual_seed(3)) + 1
    k[0], v[0] = 1.0, 0.0
    set_keys(s, kind, [k])
    set_keys(s, kind, [v], "v")
    # the same pages for every request, so that the pieces are long
    T = n * count
    near = 1 + 0.002 * torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(4))
    s.update(T=T, q=(near * down * float(np.log(2)) / (D ** 0.5 * s["kc_np"][s["table"][0, 0].item(), 0, 0, 0])).bfloat16().cuda(),
             table=s["table"].repeat(count, 1).contiguous(), cu=torch.arange(count + 1, dtype=torch.int32).cuda() * n,
             ctx=s["ctx"].repeat(count))
    out, lse = run_attn(b, s, kind == "kv4")
    keys, values = (f64(torch.from_numpy(s[x]))[s["table"][0].cpu().numpy()].reshape(-1, Hkv, D) for x in ("kc_np", "vc_np"))
    want, wl, mag, dot = oracle.prompt_attn(f64(s["q"]), [keys] * count, [values] * count, s["cu"].cpu().numpy(),
                                            s["ctx"].cpu().numpy(), D ** -0.5)
    dz = (D + 8) * 2.0 ** -24 * dot
    arith = 2 * dz + (ctx + 16) * 2.0 ** -24
    small = 0.0 if kind == "bf16" else 2.0 ** -32 * np.abs(values).sum(0).max()
    err = np.abs(f64(out) - want)
    bound = HALF["bf16"] * np.abs(want) + (WEIGHT_HALF[kind] + arith)[..., None] * mag + small
    print(f"worst error / bound {float((err / bound).max()):.3f}, of the output {float((err / np.abs(want).max()).max()):.2e}")
    assert (err <= bound).all() and s["st"].item() == 0


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("lead,trail", [(2, 0), (0, 3), (1, 1)])
def test_attn_reports_rows_outside_every_request(kind, n, lead, trail):
    """cu_seqlens that starts late or ends early: reported, the requests' own rows are right, the others left alone."""
    b = need_gpu()
    Hkv = 2
    s = make(59, [n, n, n], [20, 300, 0], 8, Hkv, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    pad = lambda k: torch.zeros(k, *s["q"].shape[1:], dtype=s["q"].dtype, device="cuda")  # noqa: E731
    x = dict(s, T=3 * n + lead + trail, q=torch.cat([pad(lead), s["q"], pad(trail)]), cu=s["cu"] + lead)
    out, lse = run_attn(b, x, kind == "kv4")
    assert s["st"].item() == 1
    s["st"].zero_()
    rows = slice(lead, lead + 3 * n)
    check_attn(s, out[rows], lse[rows], WEIGHT_HALF[kind])
    outside = torch.ones(x["T"], dtype=torch.bool)
    outside[rows] = False
    assert (out[outside.cuda()] == 7.0).all() and (lse[outside.cuda()] == 7.0).all()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("cu,per", [([0, 6, 3, 8], 0), ([0, 8, 0, 8], 0), ([3, 0, 8, 8], 0), (None, 1), (None, 30)])
def test_attn_lists_nothing_where_cu_seqlens_falls(kind, cu, per):
    """A cu_seqlens that falls lets requests claim rows many times over: nothing is
    listed (the longest here would be 4096 requests of all rows), nothing written."""
    b = need_gpu()
    B = 3 if cu else 8192
    s = make(61, [3, 3, 2], [20, 300, 0], 8, 8, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    if cu is None:
        T = per * B
        cu = [T * (i % 2) for i in range(B + 1)]
        s.update(T=T, q=torch.zeros(T, 8, 64, dtype=s["q"].dtype, device="cuda"), ctx=torch.zeros(B, dtype=torch.int32).cuda(),
                 table=torch.zeros(B, -(-T // 16), dtype=torch.int32).cuda())
    s["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    out, lse = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 1 and (out == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("n,ctx", [(1, 2 ** 31 - 1), (20, 2 ** 31 - 8), (20, 2 ** 30 - 10), (1, 2 ** 30)])
def test_attn_refuses_positions_past_its_range(kind, n, ctx):
    """A block table wide enough for more positions than 32 bits count."""
    b = need_gpu()
    s = make(67, [n, 3], [0, 40], 8, 2, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    wide = torch.zeros(2, 2 ** 27 + 2, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"]
    clean, _ = run_attn(b, s, kind == "kv4")
    s["table"] = wide
    s["ctx"][0] = ctx
    out, lse = run_attn(b, s, kind == "kv4")
    assert s["st"].item() == 6 and (out[:n] == 7.0).all() and (lse[:n] == 7.0).all()
    assert torch.equal(out[n:], clean[n:])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
def test_attn_on_a_given_stream_without_a_workspace(kind):
    """The scratch is the given stream's: work of the current stream that takes
    memory as soon as the call returns does not disturb it."""
    b = need_gpu()
    s = make(71, [60, 1, 200] * 6, [700, 3000, 90] * 6, 16, 4, 128, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    want, wl = run_attn(b, s, kind == "kv4")
    side = torch.cuda.Stream()
    for _ in range(5):
        out, lse = torch.zeros_like(want), torch.zeros_like(wl)
        torch.cuda.synchronize()
        if kind == "kv4":
            b.eagle_prompt_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["ctx"], out, lse=lse, stream=side)
        else:
            b.eagle_prompt_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"], out, lse=lse, stream=side)
        torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
def test_attn_single_row_of_any_stride(kind):
    b = need_gpu()
    s = make(73, [1], [100], 8, 2, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    want, wl = run_attn(b, s, kind == "kv4")
    for row in (64, 3, 0, 8 * 64 + 1):
        q = torch.as_strided(s["q"].contiguous(), (1, 8, 64), (row, 64, 1))
        out, lse = run_attn(b, dict(s, q=q), kind == "kv4")
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind,q,scale,ks", [
    ("fp32", 1.0, 3.3e38, 1.0), ("bf16", 1.0, 3.3e38, 1.0), ("kv4", 1.0, 3.3e38, 1.0), ("kv4", 2.0 ** 100, 1.0, 2.0 ** 40),
    ("kv4", 1.0, 2.0 ** 100, 2.0 ** 100)])
@pytest.mark.parametrize("n,ctx", [(1, 300), (1, 2600), (50, 300)])
def test_attn_factors_past_the_range(kind, q, scale, ks, n, ctx):
    """Where scale, k_scale and a row's power of two leave fp32's range together,
    scores of 0 stay 0 and those below it weigh nothing."""
    b = need_gpu()
    s = make(79, [n], [ctx], 8, 2, 64, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    x = torch.zeros(n, 8, 64)
    x[..., 3] = q
    s["q"] = x.to(s["q"].dtype).cuda()
    key = torch.zeros(ctx + n, 2, 64)
    key[::3, :, 3] = -40.0
    set_keys(s, kind, [key])
    out, lse = run_attn(b, s, kind == "kv4", scale=scale, ks=ks)
    pages = s["table"][0].cpu().numpy()
    v = s["vc_np"][pages].reshape(-1, 2, 64)
    half = HALF["fp32"] if kind == "fp32" else HALF["bf16"]
    for r in range(n):
        w = np.arange(ctx + r + 1) % 3 != 0
        x = np.repeat(v[:ctx + r + 1][w], 4, 1)
        err = np.abs(f64(out[r]) - x.mean(0))
        assert (err <= half * np.abs(x.mean(0)) + (WEIGHT_HALF[kind] + (ctx + 16) * 2.0 ** -24) * np.abs(x).mean(0)).all()
        assert np.abs(f64(lse[r]) - np.log(w.sum())).max() <= 2.0 ** -20
    assert s["st"].item() == 0


@pytest.mark.parametrize("kind", ["fp32", "bf16", "kv4"])
@pytest.mark.parametrize("new,ctx", [([1] * 4, [5, 300, 2500, 130]), ([40, 3, 170], [0, 300, 260])])
def test_attn_non_finite_query_rows(kind, new, ctx):
    """A query of NaN or infinities is its own row's matter."""
    b = need_gpu()
    s = make(97, new, ctx, 8, 2, 128, "fp32" if kind == "fp32" else "bf16", kv4=kind == "kv4")
    clean, clse = run_attn(b, s, kind == "kv4")
    q = s["q"].clone()
    bad = torch.zeros(s["T"], 8, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[2, :] = bad[-1, 5] = bad[1::7, 1] = True
    q[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0], dtype=q.dtype, device="cuda").repeat(32)
    s["q"] = q
    out, lse = run_attn(b, s, kind == "kv4")
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clse[~bad])
    assert s["st"].item() == 0
