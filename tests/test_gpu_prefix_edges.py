"""Shared prefixes: calls whose units lie whole within a CTA (so that the main
kernel joins the own result itself, and not the kernel behind it), in place and
with values that a result must not take up."""
import pytest
import torch

from gpu_helpers import need_gpu
from test_gpu_prefix import KINDS, check, run, setup

pytestmark = pytest.mark.gpu

# On 152 SMs, 32 heads over 8: the units of the first three calls are whole, with two or
# three key blocks that both tiles share (228 of 320 and all 560, in the third the last 8 of
# 256); the others of the third have two tiles of rows; the fourth has all kinds, cut ones
# and single blocks among them.
WHOLE = [([1] * 40, [300] * 40), ([9] * 70, [130] * 70), ([2000], [300]), ([40, 5, 70] * 8, [300, 700, 100] * 8)]


def in_place(b, s, kind, out=True):
    """The call with lse (and out) the own results themselves, copies of them: (out, lse)."""
    o, l = s["own_out"].clone(), s["own_lse"].clone()
    args = dict(lse=l, own_out=o, own_lse=l, status=s["st"])
    to = o if out else torch.full_like(o, 7.0)
    if kind == "kv4":
        b.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["lens"], to, **args)
    else:
        b.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], to, **args)
    return to, l


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (32, 8, 64), (4, 4, 128)])
@pytest.mark.parametrize("rows,lens", WHOLE)
def test_whole_units_in_place(rows, lens, Hq, Hkv, D, kind):
    """lse (and out) are own_lse (and own_out) themselves: to the bit what separate arrays hold."""
    b = need_gpu()
    if kind == "fp32":
        rows = [r // 4 + 1 for r in rows]
    s = setup(kind, rows, lens, Hq, Hkv, D, len(rows) + D)
    want, wl = run(b, s, kind)
    check(s, want, wl, kind)
    for i in range(12):
        out, lse = in_place(b, s, kind, out=i % 3 != 2)
        assert torch.equal(out, want) and torch.equal(lse, wl)


# whole and cut units in one call; single blocks; cut alone; tiles of rows, whole
SHARED_OUT = [([1] * 40, [300] * 40), ([9, 3], [100, 60]), ([64], [3000]), ([2000], [300])]


def heads_of(kind, rows):
    return (32, 8, 128) if kind != "fp32" or sum(rows) < 500 else (4, 2, 64)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", SHARED_OUT)
def test_a_prefix_without_weight_does_not_count(rows, lens, kind):
    """Where the own log-sum-exp lies so far above a prefix that the prefix weighs nothing, the own
    result is taken over to the bit, whatever the prefix's values hold; beside it they are seen."""
    b = need_gpu()
    Hq, Hkv, D = heads_of(kind, rows)
    s = setup(kind, rows, lens, Hq, Hkv, D, 21)
    if kind == "kv4":
        s["vs"][s["table"][:, 0].long(), :, 3] = 127  # a NaN as the scale of 16 values
    else:
        s["vc"][s["table"][:, 0].long(), 3] = torch.inf
        s["vc"][s["table"][:, 0].long(), 5] = torch.nan
    s["own_lse"][:, ::2] = 300.0
    out, lse = run(b, s, kind)
    assert torch.equal(out[:, ::2], s["own_out"][:, ::2]) and torch.equal(lse[:, ::2], s["own_lse"][:, ::2])
    assert not out[:, 1::2].isfinite().any() and lse.isfinite().all() and s["st"].item() == 0


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("rows,lens", SHARED_OUT)
def test_a_prefix_whose_scores_are_all_minus_infinity_does_not_count(rows, lens, own, kind):
    """Nor does one without a score above -infinity: the own result, or zeros and -infinity."""
    b = need_gpu()
    s = setup(kind, rows, lens, *heads_of(kind, rows), 22, own=own)
    s["q"].abs_()
    s["kc"][:, :, 0] = -torch.inf
    s["vc"][s["table"][:, 0].long(), 3] = torch.inf
    out, lse = run(b, s, kind)
    g = s["q"].shape[1] // s["kc"].shape[2]
    if own:
        assert torch.equal(out[:, :g], s["own_out"][:, :g]) and torch.equal(lse[:, :g], s["own_lse"][:, :g])
    else:
        assert (out[:, :g] == 0).all() and (lse[:, :g] == -torch.inf).all()
    assert not out[:, g:, 0].isfinite().any() and lse[:, g:].isfinite().all() and s["st"].item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", SHARED_OUT + [([5, 6], [0, 40])])
def test_largest_and_lowest_own_sums(rows, lens, kind):
    """The type's lowest value as an own log-sum-exp, as masks have it, weighs nothing beside a prefix;
    its largest leaves the own result; the log-sum-exp in base 2 lies past fp32 in both."""
    b = need_gpu()
    s = setup(kind, rows, lens, *heads_of(kind, rows), 23)
    none = dict(s, own_lse=torch.full_like(s["own_lse"], -torch.inf))
    alone, al = run(b, none, kind)
    empty = torch.repeat_interleave(s["lens"] == 0, torch.tensor(rows).cuda())
    for low in (torch.finfo(torch.float32).min, -2.4e38, -2.3e38, -1e30):
        out, lse = run(b, dict(s, own_lse=torch.full_like(s["own_lse"], low)), kind)
        assert torch.equal(out[~empty], alone[~empty]) and torch.equal(lse[~empty], al[~empty])
        assert torch.equal(out[empty], s["own_out"][empty]) and (lse[empty] == torch.tensor(low)).all()
    for high in (torch.finfo(torch.float32).max, 2.4e38, 2.3e38, 1e30):
        out, lse = run(b, dict(s, own_lse=torch.full_like(s["own_lse"], high)), kind)
        assert torch.equal(out, s["own_out"]) and (lse == torch.tensor(high)).all()
