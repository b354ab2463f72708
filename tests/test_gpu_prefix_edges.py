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
