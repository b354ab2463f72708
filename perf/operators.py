"""The prompt and single-token path over a paged KV cache: what is timed, and its plain forms.

Three operators, each as a pass through the framework's public calls (`own`)
or in elementary torch operations in 32 bits:

  append   rotate the packed rows of many requests to their positions, write
           q out and k, v into the paged cache (16-bit, 32-bit or 4-bit pages)
  attn     causal grouped-head attention of the packed new rows over the
           paged cache: whole prompts, chunks of prompts, single tokens
  attn4    the same over a cache held in 4 bits

A request's rows are rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 of the packed
arrays, at positions ctx_lens[b] + 0, 1, ...; its pages are listed in
block_table[b].  The lengths are fixed by the case, all values by the seed.

4-bit pages: 16 channels of a token and head share one e4m3 scale
s = e4m3(max|x| / 6); a channel is one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} * s
(nearest, ties to the even code), two to a byte, the even channel low.
"""
import math
import random

import torch

own = False

PAGE = 16
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step of 64 requests, each a few hundred tokens in: the
        # smallest append, where latency is all there is
        dict(name="append_decode64", op="append", dtype="bf16", B=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=500,
             Hq=32, Hkv=8, D=128, lens=1),
        # ragged prompts of sixteen requests of an 8B-shaped model, packed
        dict(name="append_prompts", op="append", dtype="bf16", B=16, new_lo=1, new_hi=1023, ctx_lo=0, ctx_hi=300,
             Hq=32, Hkv=8, D=128, lens=2),
        # the same kind of prompts into 4-bit pages, and the pages read back
        dict(name="append_prompts_4bit", op="append4", dtype="bf16", B=8, new_lo=100, new_hi=1500, ctx_lo=0,
             ctx_hi=200, Hq=32, Hkv=8, D=128, lens=3),
        # small ragged prompts in 32 bits, the type of the parity checks
        dict(name="attn_small_fp32", op="attn", dtype="fp32", B=3, new_lo=1, new_hi=130, ctx_lo=0, ctx_hi=128,
             Hq=4, Hkv=2, D=64, lens=4),
        # one prompt of 2048 tokens (8B shape): time to first token
        dict(name="attn_prompt_2k", op="attn", dtype="bf16", B=1, new_lo=2048, new_hi=2048, ctx_lo=0, ctx_hi=0,
             Hq=32, Hkv=8, D=128, lens=5),
        # sixteen ragged prompts of 1 .. 2500 tokens, packed
        dict(name="attn_prompts_packed", op="attn", dtype="bf16", B=16, new_lo=1, new_hi=2500, ctx_lo=0, ctx_hi=0,
             Hq=32, Hkv=8, D=128, lens=6),
        # one long prompt of a 70B-shaped model: the largest
        dict(name="attn_prompt_8k", op="attn", dtype="bf16", B=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             Hq=64, Hkv=8, D=128, lens=7),
        # a scheduler's chunks of four prompts, far into long contexts
        dict(name="attn_chunks_32k", op="attn", dtype="bf16", B=4, new_lo=256, new_hi=512, ctx_lo=30000,
             ctx_hi=32256, Hq=32, Hkv=8, D=128, lens=8),
        # single tokens of 64 requests over 1024 .. 4096 cached tokens
        dict(name="attn_decode64", op="attn", dtype="bf16", B=64, new_lo=1, new_hi=1, ctx_lo=1023, ctx_hi=4095,
             Hq=32, Hkv=8, D=128, lens=9),
        # the same step over 4-bit pages
        dict(name="attn4_decode64", op="attn4", dtype="bf16", B=64, new_lo=1, new_hi=1, ctx_lo=1023, ctx_hi=4095,
             Hq=32, Hkv=8, D=128, lens=9),
        # single tokens of four requests over 32k cached tokens in 4 bits
        dict(name="attn4_decode_long", op="attn4", dtype="bf16", B=4, new_lo=1, new_hi=1, ctx_lo=32767, ctx_hi=32767,
             Hq=32, Hkv=8, D=128, lens=10),
        # chunks of prompts over 4-bit pages
        dict(name="attn4_chunks_8k", op="attn4", dtype="bf16", B=4, new_lo=200, new_hi=700, ctx_lo=4000, ctx_hi=8000,
             Hq=32, Hkv=8, D=128, lens=11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op, dtype = rng.choice([("append", "bf16"), ("append", "fp32"), ("append4", "bf16"), ("attn", "bf16"),
                            ("attn", "bf16"), ("attn", "fp32"), ("attn4", "bf16"), ("attn4", "bf16")])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    B = _log_int(rng, 1, 64)
    c = dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, lens=rng.randrange(1 << 30))
    if op.startswith("append"):
        hi = _log_int(rng, 1, max(1, 16384 // B))
        c.update(new_lo=rng.choice([0, 1, 1 + hi // 2, hi]), new_hi=hi, ctx_lo=0, ctx_hi=rng.choice([0, 17, 300, 1000]))
        c["new_lo"] = min(c["new_lo"], hi)
        return c
    # attention: prompts, chunks over a context, single tokens; the padded
    # score matrix B * Hq * new * keys is kept under 2^31
    top = 1 << 31 if dtype == "bf16" else 1 << 27
    kind = rng.choice(["prompt", "chunk", "token"])
    new = 1 if kind == "token" else _log_int(rng, 2, max(2, 8192 // B))
    ctx = 0 if kind == "prompt" else _log_int(rng, 1, max(1, min(32768, 262144 // B)))
    while B * Hq * new * (ctx + new) > top:
        new, ctx = max(1, new // 2), ctx if new > 1 else ctx // 2
    c.update(new_lo=rng.choice([min(1, new), (new + 1) // 2, new]), new_hi=new, ctx_lo=rng.choice([0, ctx // 2, ctx]),
             ctx_hi=ctx)
    return c


def _lengths(case):
    """New tokens and cached tokens of each request."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if sum(new) == 0:
        new[0] = 1
    return new, ctx


def work(case):
    new, ctx = _lengths(case)
    T, Hq, Hkv, D = sum(new), case["Hq"], case["Hkv"], case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    row4 = Hkv * (D // 2 + D // 16)  # bytes of one token in 4-bit pages, keys or values
    rows = T * (Hq + 2 * Hkv) * D * es
    if case["op"] == "append":
        # q, k, v read and written, the rotation's cos and sin
        return dict(bytes=2 * rows + T * D * 4, flops=3 * T * (Hq + Hkv) * D)
    if case["op"] == "append4":
        pages = sum(-(-(n + c) // PAGE) for n, c in zip(new, ctx)) + 3
        back = 2 * pages * PAGE * (row4 + Hkv * D * 2)  # the pages read back as 16-bit values
        return dict(bytes=rows + T * Hq * D * es + 2 * T * row4 + T * D * 4 + back, flops=3 * T * (Hq + Hkv) * D)
    keys = sum(c + n for n, c in zip(new, ctx) if n)
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    kv = 2 * keys * (row4 if case["op"] == "attn4" else Hkv * D * es)
    return dict(bytes=2 * T * Hq * D * es + T * Hq * 4 + kv, flops=4 * seen * Hq * D)


# ---------------------------------------------------------------- the inputs
def _pack4(x):
    """Codes and scales of x [..., D] in 4 bits (see the head of this file)."""
    g = x.float().unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = g.abs()
    code = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s).to(torch.uint8) + (a > 1.25 * s).to(torch.uint8)
            + (a >= 1.75 * s).to(torch.uint8) + (a > 2.5 * s).to(torch.uint8) + (a >= 3.5 * s).to(torch.uint8)
            + (a > 5.0 * s).to(torch.uint8))
    code = torch.where(s > 0, code, torch.zeros_like(code)) + 8 * torch.signbit(g).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], scale


def _unpack4(codes, scales, dtype=torch.float32):
    """The values [..., D] that codes [..., D/2] and scales [..., D/16] stand for."""
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (lut[both.int()].unflatten(-1, (-1, 16)) * scales.to(dtype).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, ctx = _lengths(case)
    B, T, Hq, Hkv, D = case["B"], sum(new), case["Hq"], case["Hkv"], case["D"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n_pages = [-(-(n + c) // PAGE) for n, c in zip(new, ctx)]
    P, width = sum(n_pages) + 3, max(n_pages + [1])
    ids = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, max_new=max(new), max_keys=max(n + c for n, c in zip(new, ctx)), table=table,
             cu=torch.tensor(cu, dtype=torch.int32, device=dev), ctx=torch.tensor(ctx, dtype=torch.int32, device=dev))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # keys have channels of uneven size, as trained models' do
    gain = torch.exp(0.4 * randn(Hkv, D))
    if case["op"].startswith("append"):
        # q, k, v are slices of the rows that one projection wrote
        qkv = randn(T, Hq + 2 * Hkv, D)
        qkv[:, Hq:Hq + Hkv] *= gain
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        # cos and sin of position * theta^(-2i/D), formed in 64 bits
        pos = torch.arange(s["max_keys"], dtype=torch.float64, device=dev)
        ang = pos[:, None] * 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
        s["rope"] = torch.stack((ang.cos(), ang.sin()), 1).float()
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    else:
        s["q"] = (1.3 * randn(T, Hq, D)).to(dt)
        s["out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, Hq, device=dev)
    if case["op"].endswith("4"):
        s["k4"], s["ks"] = _pack4(randn(P, Hkv, PAGE, D) * gain[:, None])
        s["v4"], s["vs"] = _pack4(randn(P, Hkv, PAGE, D))
        s["back"] = [torch.empty(P, PAGE, Hkv, D, dtype=dt, device=dev) for _ in "kv" if case["op"] == "append4"]
    else:
        s["kc"] = (randn(P, PAGE, Hkv, D) * gain).to(dt)
        s["vc"] = randn(P, PAGE, Hkv, D).to(dt)
    return s


# ---------------------------------------------------------------- the plain forms
def _rows(s):
    """For each packed row: its request, its index in it, and its position."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True)
    i = t - s["cu"].long()[b]
    return b, i, s["ctx"].long()[b] + i


def _rotate(x, rope):
    """x [T, H, D] turned by the rows' cos and sin [T, 2, D/2] (pair i, i + D/2)."""
    x1, x2 = x.float().chunk(2, -1)
    c, n = rope[:, 0, None], rope[:, 1, None]
    return torch.cat((x1 * c - x2 * n, x2 * c + x1 * n), -1)


def _append_plain(s):
    b, _, pos = _rows(s)
    page, slot = s["table"][b, pos // PAGE].long(), pos % PAGE
    rope = s["rope"][pos]
    q, k = _rotate(s["q"], rope).to(s["q"].dtype), _rotate(s["k"], rope)
    if s["case"]["op"] == "append":
        s["kc"][page, slot] = k.to(s["kc"].dtype)
        s["vc"][page, slot] = s["v"]
        return [q, s["kc"], s["vc"]]
    s["k4"][page, :, slot], ks = _pack4(k)
    s["ks"].view(torch.uint8)[page, :, slot] = ks.view(torch.uint8)
    s["v4"][page, :, slot], vs = _pack4(s["v"])
    s["vs"].view(torch.uint8)[page, :, slot] = vs.view(torch.uint8)
    return [q, _unpack4(s["k4"], s["ks"]).transpose(1, 2).to(q.dtype).contiguous(),
            _unpack4(s["v4"], s["vs"]).transpose(1, 2).to(q.dtype).contiguous()]


def _attn_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, N, L = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_new"], s["max_keys"]
    G = Hq // Hkv
    pages = s["table"].clamp(min=0).long()
    if c["op"] == "attn4":  # [B, pages, Hkv, PAGE, D] -> [B, Hkv, keys, D]
        k = _unpack4(s["k4"][pages], s["ks"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)).transpose(1, 2)
        v = _unpack4(s["v4"][pages], s["vs"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)).transpose(1, 2)
    else:
        k, v = s["kc"][pages].float().permute(0, 3, 1, 2, 4), s["vc"][pages].float().permute(0, 3, 1, 2, 4)
    k, v = k.reshape(B, Hkv, -1, D)[:, :, :L], v.reshape(B, Hkv, -1, D)[:, :, :L]
    i = torch.arange(N, device="cuda")
    row = (s["cu"].long()[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(B, N, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, N * G, D)
    z = torch.matmul(q * D ** -0.5, k.transpose(-1, -2)).view(B, Hkv, N, G, L)
    hidden = torch.arange(L, device="cuda") > (s["ctx"].long()[:, None] + i)[..., None]
    z.masked_fill_(hidden[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hkv, N * G, L), v).view(B, Hkv, N, G, D) / l
    lse = (m + l.log())[..., 0]
    b, i, _ = _rows(s)
    return [o[b, :, i].reshape(-1, Hq, D).to(s["q"].dtype), lse[b, :, i].reshape(-1, Hq)]


def _own(s):
    from eagle_speculative_decoding_gb300 import binding as eb
    op = s["case"]["op"]
    if op == "append":
        eb.eagle_kv_append(s["q"], s["k"], s["v"], s["rope"], s["cu"], s["ctx"], s["table"], s["kc"], s["vc"],
                           q_out=s["q_out"])
        return [s["q_out"], s["kc"], s["vc"]]
    if op == "append4":
        eb.eagle_kv_append_kv4(s["q"], s["k"], s["v"], s["rope"], s["cu"], s["ctx"], s["table"], s["k4"], s["ks"],
                               s["v4"], s["vs"], q_out=s["q_out"])
        eb.eagle_kv4_read(s["k4"], s["ks"], s["back"][0])
        eb.eagle_kv4_read(s["v4"], s["vs"], s["back"][1])
        return [s["q_out"]] + s["back"]
    if "ws" not in s:  # kept with the state, as a program keeps it from call to call
        c = s["case"]
        s["ws"] = eb.workspace(eb.eagle_prompt_attn_workspace_size(c["B"], s["q"].shape[0], c["Hq"], c["Hkv"], c["D"]))
    if op == "attn":
        eb.eagle_prompt_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"], s["out"], lse=s["lse"], ws=s["ws"])
    else:
        eb.eagle_prompt_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["ctx"], s["out"],
                                 lse=s["lse"], ws=s["ws"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    return _append_plain(state) if state["case"]["op"].startswith("append") else _attn_plain(state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    new, ctx = _lengths(case)
    T, Hq, Hkv, D = sum(new), case["Hq"], case["Hkv"], case["D"]
    kinds = {"append4": ("k4", "v4"), "attn4": ("k4", "v4")}.get(case["op"], ("kc", "vc"))

    def values(name):
        if name in ("kc", "vc"):
            return s[name].double()
        codes, scales = s[name].long(), s[name[0] + "s"].double()
        nibble = torch.empty(*codes.shape[:-1], D, dtype=torch.long, device="cuda")
        nibble[..., 0::2], nibble[..., 1::2] = codes % 16, codes // 16
        half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda").double() / 2
        return (half[nibble % 8] * (1 - 2 * (nibble // 8))) * scales.repeat_interleave(16, -1)

    if case["op"].startswith("append"):
        q, k, v = (s[x].double() for x in "qkv")
        where = torch.tensor([c + i for n, c in zip(new, ctx) for i in range(n)], device="cuda")
        cos, sin = s["rope"].double()[where].unbind(1)
        rot = torch.complex(cos, sin)[:, None]
        turn = lambda x: torch.cat(torch.view_as_real(torch.complex(x[..., :D // 2], x[..., D // 2:]) * rot).unbind(-1), -1)  # noqa: E731
        q, k = turn(q), turn(k)
        owner = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device="cuda")
        page, slot = s["table"][owner, where // PAGE].long(), where % PAGE
        if case["op"] == "append":
            kc, vc = values("kc"), values("vc")
        else:
            def snap(x):
                x = x.reshape(*x.shape[:-1], D // 16, 16)
                scale = (x.abs().max(-1).values / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double()[..., None]
                grid = torch.tensor(MAGNITUDES, device="cuda").double()
                near = (x.abs()[..., None] - scale[..., None] * grid).abs()
                # the even code wins a tie: odd codes are looked at last
                order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device="cuda")
                return (grid[order[near[..., order].argmin(-1)]] * scale * x.sign()).flatten(-2)

            k, v = snap(k), snap(v)
            kc, vc = values("k4").transpose(1, 2).contiguous(), values("v4").transpose(1, 2).contiguous()
        kc[page, slot], vc[page, slot] = k, v
        return [q, kc, vc]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    G, t0 = Hq // Hkv, 0
    kv = [values(x) for x in kinds] if case["op"] == "attn4" else [s[x] for x in kinds]
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        L = c + n
        pages = s["table"][b, :-(-L // PAGE)].long()
        late = torch.ones(n, L, dtype=torch.bool, device="cuda").triu(c + 1)
        for h in range(Hkv):
            k, v = ((x[pages, h] if case["op"] == "attn4" else x[pages, :, h].double()).reshape(-1, D)[:L] for x in kv)
            for j in range(h * G, h * G + G):
                z = (s["q"][t0:t0 + n, j].double() @ k.T) / math.sqrt(D)
                z = z.masked_fill(late, -math.inf)
                lse[t0:t0 + n, j] = torch.logsumexp(z, -1)
                out[t0:t0 + n, j] = torch.softmax(z, -1) @ v
        t0 += n
    return [out, lse]
