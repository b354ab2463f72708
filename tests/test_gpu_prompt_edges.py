"""GPU parity of the prompt path where it is easily got wrong: many pieces per
CTA, scores at the ends of their range, malformed lengths.  Helpers and
tolerances are those of test_gpu_prompt."""
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
