"""A step of a batch that shares a long prompt: what is timed, and its plain forms.

Three operators, each as a pass through the framework's public calls (`own`)
or in elementary torch operations in 32 bits (64 for the sampler's sums, whose
borders 32 bits would move):

  axes    rotate packed rows to explicit positions of several axes (time,
          height, width), write q out and k, v into the paged cache (16-, 32-
          or 4-bit pages)
  prefix  attention of groups of rows over a prefix that the group shares,
          joined with the rows' finished attention over their own keys
          (16-, 32- or 4-bit pages)
  sample  a token from each row of logits by temperature, top-k, top-p and
          min-p from a given uniform number; or the truncated logits

axes: pair i of a row's channels (i, i + D/2) turns by the angle of the
position on the pair's axis, positions[axis[i], t].  The row's slot in the
cache goes by its number, ctx_lens[b] + 0, 1, ...: an image of h x w tokens
fills h w slots and advances the positions by max(h, w).

prefix: rows cu_rows[g] .. cu_rows[g+1] - 1 see the prefix_lens[g] tokens of
the pages in prefix_table[g], all of them.

sample: entries are ordered by (logit descending, index ascending), their
weights are exp((x - max x) / T).  top-k keeps the first k; top-p keeps of
these an entry while the weights before it add up to less than p times their
sum; min-p keeps weights of at least min_p times the largest.  The token is
the first index, in the order of indices, at which the running sum of the kept
weights exceeds u times their sum.  T = 0: the first entry.
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
        # one decoding step of 64 requests behind images: latency is all there is
        dict(name="axes_decode64", op="axes", dtype="bf16", B=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=500, Hq=32, Hkv=8,
             D=128, sections="16,24,24", lens=1),
        # ragged prompts with images in them, packed (8B shape), axes in sections
        dict(name="axes_images", op="axes", dtype="bf16", B=12, new_lo=100, new_hi=1400, ctx_lo=0, ctx_hi=300, Hq=32, Hkv=8,
             D=128, sections="16,24,24", lens=2),
        # the same kind of prompts into 4-bit pages, axes taking turns, and the pages read back
        dict(name="axes_images_4bit", op="axes4", dtype="bf16", B=8, new_lo=100, new_hi=1500, ctx_lo=0, ctx_hi=200, Hq=32,
             Hkv=8, D=128, sections="turns", lens=3),
        # a few rows of two groups in 32 bits, the type of the parity checks
        dict(name="prefix_small_fp32", op="prefix", dtype="fp32", G=2, rows_lo=1, rows_hi=60, len_lo=100, len_hi=700, Hq=4,
             Hkv=2, D=64, lens=4),
        # single tokens of 64 requests behind a system prompt of 8000 tokens (8B shape)
        dict(name="prefix_tokens64", op="prefix", dtype="bf16", G=1, rows_lo=64, rows_hi=64, len_lo=8000, len_hi=8000, Hq=32,
             Hkv=8, D=128, lens=5),
        # single tokens of four requests about one long document
        dict(name="prefix_tokens4_32k", op="prefix", dtype="bf16", G=1, rows_lo=4, rows_hi=4, len_lo=32768, len_hi=32768,
             Hq=32, Hkv=8, D=128, lens=6),
        # verification: the tree rows of 64 requests with one of two system prompts, the largest
        dict(name="prefix_trees", op="prefix", dtype="bf16", G=2, rows_lo=700, rows_hi=1300, len_lo=3000, len_hi=5000, Hq=32,
             Hkv=8, D=128, lens=7),
        # single tokens behind a system prompt that is held in 4 bits
        dict(name="prefix_tokens64_4bit", op="prefix4", dtype="bf16", G=1, rows_lo=64, rows_hi=64, len_lo=8000, len_hi=8000,
             Hq=32, Hkv=8, D=128, lens=8),
        # the next token of one request, usual settings
        dict(name="sample_one", op="sample", dtype="bf16", M=1, V=128256, per=1, settings="usual", lens=9),
        # the next tokens of 64 requests, each with settings of its own (greedy and untruncated ones too)
        dict(name="sample_batch64", op="sample", dtype="fp32", M=64, V=128256, per=1, settings="mixed", lens=10),
        # an odd vocabulary, flat distributions: the nucleus holds thousands of entries
        dict(name="sample_nucleus_odd", op="sample", dtype="bf16", M=17, V=50257, per=1, settings="nucleus", lens=11),
        # the verify rows of eight requests (32 rows each), truncated before the verification
        dict(name="truncate_verify", op="truncate", dtype="fp32", M=256, V=128256, per=32, settings="mixed", lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op, dtype = rng.choice([("axes", "bf16"), ("axes", "fp32"), ("axes4", "bf16"), ("prefix", "bf16"), ("prefix", "bf16"),
                            ("prefix", "fp32"), ("prefix4", "bf16"), ("sample", "bf16"), ("sample", "fp32"),
                            ("truncate", "bf16"), ("truncate", "fp32")])
    c = dict(op=op, dtype=dtype, lens=rng.randrange(1 << 30))
    if op in ("sample", "truncate"):
        V = _log_int(rng, 100, 262144)
        M = _log_int(rng, 1, max(1, min(512, (1 << 23) // V if op == "sample" else (1 << 25) // V)))
        c.update(M=M, V=V, per=rng.choice([1, 1, 4, 31]), settings=rng.choice(["usual", "mixed", "mixed", "nucleus"]))
        return c
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    c.update(Hq=Hq, Hkv=Hkv, D=D)
    if op.startswith("axes"):
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 8192 // B))
        c.update(B=B, new_lo=min(hi, rng.choice([0, 1, 1 + hi // 2, hi])), new_hi=hi, ctx_lo=0,
                 ctx_hi=rng.choice([0, 17, 300, 1000]), sections=rng.choice(["one", "two", "turns", "partial"]))
        return c
    # the padded scores G * Hq * rows * keys are kept under 2^28 (32 bits: 2^25)
    top = 1 << 28 if dtype == "bf16" else 1 << 25
    G = rng.choice([1, 1, 2, 3, 5])
    rows, keys = _log_int(rng, 1, max(1, 2048 // G)), _log_int(rng, 1, 32768)
    while G * Hq * rows * keys > top:
        rows, keys = (max(1, rows // 2), keys) if rows > 64 or keys < 64 else (rows, keys // 2)
    c.update(G=G, rows_lo=rng.choice([min(1, rows), (rows + 1) // 2, rows]), rows_hi=rows,
             len_lo=rng.choice([0, keys // 2, keys]) if G > 1 else keys, len_hi=keys)
    return c


def _lengths(case):
    """axes: new and cached tokens of each request; prefix: rows and prefix tokens of each group."""
    r = random.Random(case["lens"])
    names = ("new", "ctx", "B") if case["op"].startswith("axes") else ("rows", "len", "G")
    a = [r.randint(case[names[0] + "_lo"], case[names[0] + "_hi"]) for _ in range(case[names[2]])]
    b = [r.randint(case[names[1] + "_lo"], case[names[1] + "_hi"]) for _ in range(case[names[2]])]
    if sum(a) == 0:
        a[0] = 1
    return a, b


def work(case):
    op = case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op in ("sample", "truncate"):
        M, V = case["M"], case["V"]
        rows = M * V * es
        # a difference, a product, an exponential and a sum for each entry
        return dict(bytes=(rows + M * 12 if op == "sample" else 2 * rows + M * 4) + 16 * -(-M // case["per"]), flops=4 * M * V)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    row4 = Hkv * (D // 2 + D // 16)  # bytes of one token in 4-bit pages, keys or values
    a, b = _lengths(case)
    T = sum(a)
    if op.startswith("axes"):
        A = _axes(case)[0]
        rows = T * (Hq + 2 * Hkv) * D * es
        if op == "axes":
            return dict(bytes=2 * rows + T * (D * 4 + A * 4), flops=3 * T * (Hq + Hkv) * D)
        pages = sum(-(-(n + c) // PAGE) for n, c in zip(a, b)) + 3
        back = 2 * pages * PAGE * (row4 + Hkv * D * 2)  # the pages read back as 16-bit values
        return dict(bytes=rows + T * Hq * D * es + 2 * T * row4 + T * (D * 4 + A * 4) + back, flops=3 * T * (Hq + Hkv) * D)
    kv = 2 * sum(b) * (row4 if op == "prefix4" else Hkv * D * es)
    return dict(bytes=3 * T * Hq * D * es + 2 * T * Hq * 4 + kv, flops=4 * sum(n * c for n, c in zip(a, b)) * Hq * D)


# ---------------------------------------------------------------- the inputs
def _pack4(x):
    """Codes and scales of x [..., D]: 16 channels share s = e4m3(max|x| / 6), a
    channel is one of +-MAGNITUDES * s (nearest, ties to the even code)."""
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


def _axes(case):
    """Number of axes, and the axis of each channel pair (-1: not turned)."""
    half, kind = case["D"] // 2, case["sections"]
    if kind == "one":
        return 1, None
    if kind == "two":  # height and width, half of the pairs each
        return 2, [int(i >= half // 2) for i in range(half)]
    if kind == "turns":  # time, height, width, time, ...; the slowest pairs follow time
        return 3, [i % 3 if i < half - half // 4 else 0 for i in range(half)]
    if kind == "partial":  # the last quarter of the pairs stays as it is
        return 3, [i % 3 if i < half - half // 4 else -1 for i in range(half)]
    sizes = [int(x) for x in kind.split(",")]
    return len(sizes), [a for a, n in enumerate(sizes) for _ in range(n)]


def _positions(case, new, ctx, axes):
    """Positions [axes, T] of text with images in it (lists, from the case alone)."""
    r = random.Random(case["lens"] + 1)
    out = [[], [], []]
    for n, c in zip(new, ctx):
        p, left = c // 2, n  # (a cached image advanced the positions by less than its tokens)
        while left:
            h, w = r.randint(3, 24), r.randint(3, 24)
            if left >= h * w and r.random() < 0.5:
                for y in range(h):
                    out[0] += [p] * w
                    out[1] += [p + y] * w
                    out[2] += range(p, p + w)
                p, left = p + max(h, w), left - h * w
            else:
                run = min(left, r.randint(1, 64))
                for x in out:
                    x += range(p, p + run)
                p, left = p + run, left - run
    return out[-axes:]


def _pages(n_pages, P, g):
    """A table of page ids, -1 past each row's own."""
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(n_pages), max(n_pages + [1])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def _starts(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _settings(case):
    """temperature, top_k, top_p, min_p of each request."""
    r = random.Random(case["lens"])
    rows = []
    for _ in range(-(-case["M"] // case["per"])):
        kind = case["settings"]
        if kind == "mixed":
            kind = r.choice(["usual", "usual", "nucleus", "greedy", "none", "min_p", "top_k", "wide"])
        t = r.choice([0.6, 0.7, 0.8, 1.0])
        rows.append(dict(usual=(t, r.choice([20, 40, 50]), r.choice([0.8, 0.9, 0.95]), 0.0),
                         nucleus=(r.choice([1.0, 1.3]), 0, r.choice([0.9, 0.95, 0.98]), 0.0), greedy=(0.0, 0, 1.0, 0.0),
                         none=(t, 0, 1.0, 0.0), min_p=(r.choice([1.0, 1.5]), 0, 1.0, r.choice([0.05, 0.1])),
                         top_k=(t, r.choice([1, 8, 64, 500]), 1.0, 0.0),
                         wide=(1.0, r.choice([2000, 5000]), 0.99, 0.0))[kind])
    return list(zip(*rows))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if case["op"] in ("sample", "truncate"):
        M, V = case["M"], case["V"]
        # a trained model's logits: a power law over the ranks, differing in steepness from row to row, and noise
        steep = 1.0 + 0.5 * torch.rand(M, 1, generator=g, device=dev)
        rank = torch.arange(1, V + 1, device=dev).float().log()[torch.argsort(randn(M, V), dim=1)]
        s["logits"] = (15.0 - steep * rank + 0.6 * randn(M, V)).to(dt)
        names = (("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32))
        for (name, kind), values in zip(names, _settings(case)):
            s[name] = torch.tensor(values, dtype=kind, device=dev)
        s["u"] = torch.rand(M, generator=g, device=dev)
        s["kept"] = torch.empty(M, dtype=torch.int32, device=dev)
        if case["op"] == "sample":
            s["tokens"], s["logprobs"] = torch.empty(M, dtype=torch.int32, device=dev), torch.empty(M, device=dev)
        else:
            s["out"] = torch.empty_like(s["logits"])
        return s

    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    a, b = _lengths(case)
    T = sum(a)
    # keys have channels of uneven size, as trained models' do
    gain = torch.exp(0.4 * randn(Hkv, D))
    s["cu"], s["ctx"] = _starts(a), torch.tensor(b, dtype=torch.int32, device=dev)
    s["max_rows"], s["max_keys"] = max(a), max(b) if case["op"].startswith("prefix") else max(x + y for x, y in zip(a, b))
    if case["op"].startswith("axes"):
        n_pages = [-(-(n + c) // PAGE) for n, c in zip(a, b)]
        # q, k, v are slices of the rows that one projection wrote
        qkv = randn(T, Hq + 2 * Hkv, D)
        qkv[:, Hq:Hq + Hkv] *= gain
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        axes, of_pair = _axes(case)
        s["pos"] = torch.tensor(_positions(case, a, b, axes), dtype=torch.int32, device=dev)
        s["axis"] = None if of_pair is None else torch.tensor(of_pair, dtype=torch.int32, device=dev)
        # cos and sin of position * theta^(-2i/D), formed in 64 bits
        pos = torch.arange(s["max_keys"] + 64, dtype=torch.float64, device=dev)
        ang = pos[:, None] * 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
        s["rope"] = torch.stack((ang.cos(), ang.sin()), 1).float()
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    else:
        n_pages = [-(-c // PAGE) for c in b]
        s["q"] = (1.3 * randn(T, Hq, D)).to(dt)
        # the rows' own keys are fewer than the prefix's: their sum weighs less, or as much
        s["own_out"] = (0.3 * randn(T, Hq, D)).to(dt)
        s["own_lse"] = math.log(1 + s["max_keys"]) + 0.8 - 1.5 * torch.rand(T, Hq, generator=g, device=dev)
        s["out"], s["lse"] = torch.empty(T, Hq, D, dtype=dt, device=dev), torch.empty(T, Hq, device=dev)
    P = sum(n_pages) + 3
    s["table"] = _pages(n_pages, P, g)
    if case["op"].endswith("4"):
        s["k4"], s["ks"] = _pack4(randn(P, Hkv, PAGE, D) * gain[:, None])
        s["v4"], s["vs"] = _pack4(randn(P, Hkv, PAGE, D))
        s["back"] = [torch.empty(P, PAGE, Hkv, D, dtype=dt, device=dev) for _ in "kv" if case["op"] == "axes4"]
    else:
        s["kc"] = (randn(P, PAGE, Hkv, D) * gain).to(dt)
        s["vc"] = randn(P, PAGE, Hkv, D).to(dt)
    return s


# ---------------------------------------------------------------- the plain forms
def _owner(s):
    """For each packed row: its request or group, and its index in it."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True)
    return b, t - s["cu"].long()[b]


def _turn(x, c, n):
    """x [T, H, D] turned by the rows' cos and sin [T, D/2] (pair i, i + D/2)."""
    x1, x2 = x.float().chunk(2, -1)
    c, n = c[:, None], n[:, None]
    return torch.cat((x1 * c - x2 * n, x2 * c + x1 * n), -1)


def _axes_plain(s):
    b, i = _owner(s)
    at = s["ctx"].long()[b] + i
    page, slot = s["table"][b, at // PAGE].long(), at % PAGE
    half = s["case"]["D"] // 2
    pair = torch.arange(half, device="cuda")
    axis = torch.zeros_like(pair) if s["axis"] is None else s["axis"].long()
    where = s["pos"].long()[axis.clamp(min=0)].T  # [T, D/2]
    c = torch.where(axis >= 0, s["rope"][where, 0, pair], 1.0)
    n = torch.where(axis >= 0, s["rope"][where, 1, pair], 0.0)
    q, k = _turn(s["q"], c, n).to(s["q"].dtype), _turn(s["k"], c, n)
    if s["case"]["op"] == "axes":
        s["kc"][page, slot] = k.to(s["kc"].dtype)
        s["vc"][page, slot] = s["v"]
        return [q, s["kc"], s["vc"]]
    s["k4"][page, :, slot], ks = _pack4(k)
    s["ks"].view(torch.uint8)[page, :, slot] = ks.view(torch.uint8)
    s["v4"][page, :, slot], vs = _pack4(s["v"])
    s["vs"].view(torch.uint8)[page, :, slot] = vs.view(torch.uint8)
    return [q, _unpack4(s["k4"], s["ks"]).transpose(1, 2).to(q.dtype).contiguous(),
            _unpack4(s["v4"], s["vs"]).transpose(1, 2).to(q.dtype).contiguous()]


def _prefix_plain(s):
    c = s["case"]
    G, Hq, Hkv, D, N, L = c["G"], c["Hq"], c["Hkv"], c["D"], s["max_rows"], max(1, s["max_keys"])
    E = Hq // Hkv
    pages = s["table"].clamp(min=0).long()
    if c["op"] == "prefix4":  # [G, pages, Hkv, PAGE, D] -> [G, Hkv, keys, D]
        k = _unpack4(s["k4"][pages], s["ks"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)).transpose(1, 2)
        v = _unpack4(s["v4"][pages], s["vs"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)).transpose(1, 2)
    else:
        k, v = s["kc"][pages].float().permute(0, 3, 1, 2, 4), s["vc"][pages].float().permute(0, 3, 1, 2, 4)
    k, v = k.reshape(G, Hkv, -1, D)[:, :, :L], v.reshape(G, Hkv, -1, D)[:, :, :L]
    row = (s["cu"].long()[:-1, None] + torch.arange(N, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(G, N, Hkv, E, D).transpose(1, 2).reshape(G, Hkv, N * E, D)
    z = torch.matmul(q * D ** -0.5, k.transpose(-1, -2))
    z.masked_fill_((torch.arange(L, device="cuda") >= s["ctx"].long()[:, None])[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    g, i = _owner(s)
    pick = lambda x: x.view(G, Hkv, N, E, -1)[g, :, i].reshape(-1, Hq, x.shape[-1])  # noqa: E731
    o, m, l = pick(torch.matmul(z, v)), pick(m), pick(l)
    # the row's own keys: a sum of e^own_lse around the same reference, and their mean
    w = s["own_lse"][..., None]
    top = torch.maximum(m, w)
    a, b = (m - top).exp(), (w - top).exp()
    total = a * l + b
    return [((a * o + b * s["own_out"].float()) / total).to(s["q"].dtype), (top + total.log())[..., 0]]


def _sample_plain(s):
    x = s["logits"].double()
    M, V = x.shape
    rows = torch.arange(M, device="cuda") // s["case"]["per"]
    t, k, p, low = (s[name][rows, None] for name in ("temperature", "top_k", "top_p", "min_p"))
    t, p, low = t.double(), p.double(), low.double()
    greedy = t == 0
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t))
    place = torch.arange(V, device="cuda")
    keep = (place < torch.where(k > 0, k, V)) & (place < torch.where(greedy, 1, V))
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, 1) - w
    keep &= (p >= 1) | (before < p * w.sum(1, keepdim=True)) | (place == 0)
    keep &= w >= low
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    count = keep.sum(1).int()
    if s["case"]["op"] == "truncate":
        return [torch.where(kept, s["logits"], -math.inf), count]
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    run = torch.cumsum(w, 1)
    total = run[:, -1:]
    token = (run <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    token = torch.minimum(token, torch.where(kept, place, 0).amax(1, keepdim=True))
    return [token[:, 0].int(), (w.gather(1, token) / total).log()[:, 0].float(), count]


def _own(s):
    from eagle_speculative_decoding_gb300 import binding as eb
    op = s["case"]["op"]
    if op == "axes":
        eb.eagle_kv_append_axes(s["q"], s["k"], s["v"], s["rope"], s["pos"], s["cu"], s["ctx"], s["table"], s["kc"], s["vc"],
                                pair_axis=s["axis"], q_out=s["q_out"])
        return [s["q_out"], s["kc"], s["vc"]]
    if op == "axes4":
        eb.eagle_kv_append_axes_kv4(s["q"], s["k"], s["v"], s["rope"], s["pos"], s["cu"], s["ctx"], s["table"], s["k4"],
                                    s["ks"], s["v4"], s["vs"], pair_axis=s["axis"], q_out=s["q_out"])
        eb.eagle_kv4_read(s["k4"], s["ks"], s["back"][0])
        eb.eagle_kv4_read(s["v4"], s["vs"], s["back"][1])
        return [s["q_out"]] + s["back"]
    if op in ("sample", "truncate"):
        how = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                   rows_per_request=s["case"]["per"], n_kept=s["kept"])
        if op == "truncate":
            eb.eagle_truncate_logits(s["logits"], s["out"], **how)
            return [s["out"], s["kept"]]
        eb.eagle_sample(s["logits"], s["u"], s["tokens"], logprobs=s["logprobs"], **how)
        return [s["tokens"], s["logprobs"], s["kept"]]
    if "ws" not in s:  # kept with the state, as a program keeps it from call to call
        c = s["case"]
        s["ws"] = eb.workspace(eb.eagle_prefix_attn_workspace_size(c["G"], s["q"].shape[0], c["Hq"], c["Hkv"], c["D"]))
    if op == "prefix":
        eb.eagle_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"], s["out"], lse=s["lse"],
                             own_out=s["own_out"], own_lse=s["own_lse"], ws=s["ws"])
    else:
        eb.eagle_prefix_attn_kv4(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["table"], s["cu"], s["ctx"], s["out"],
                                 lse=s["lse"], own_out=s["own_out"], own_lse=s["own_lse"], ws=s["ws"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _axes_plain(state) if op.startswith("axes") else _prefix_plain(state) if op.startswith("prefix") else _sample_plain(state)


# ---------------------------------------------------------------- 64 bits
def _values(s, name, D):
    """A cache in 64 bits, in its own layout."""
    if name in ("kc", "vc"):
        return s[name].double()
    codes, scales = s[name].long(), s[name[0] + "s"].double()
    nibble = torch.empty(*codes.shape[:-1], D, dtype=torch.long, device="cuda")
    nibble[..., 0::2], nibble[..., 1::2] = codes % 16, codes // 16
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda").double() / 2
    return (half[nibble % 8] * (1 - 2 * (nibble // 8))) * scales.repeat_interleave(16, -1)


def _exact_axes(case, s):
    new, ctx = _lengths(case)
    D = case["D"]
    _, of_pair = _axes(case)
    of_pair = of_pair or [0] * (D // 2)
    q, k, v = (s[x].double() for x in "qkv")
    unit = torch.ones(q.shape[0], D // 2, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(of_pair):
        if a >= 0:
            cs = s["rope"][s["pos"][a].long(), :, i].double()
            unit[:, i] = torch.complex(cs[:, 0].contiguous(), cs[:, 1].contiguous())

    def turn(x):
        y = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * unit[:, None]
        return torch.cat((y.real, y.imag), -1)

    q, k = turn(q), turn(k)
    if case["op"] == "axes":
        kc, vc = _values(s, "kc", D), _values(s, "vc", D)
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
        kc, vc = _values(s, "k4", D).transpose(1, 2).contiguous(), _values(s, "v4", D).transpose(1, 2).contiguous()
    place = torch.tensor([c + i for n, c in zip(new, ctx) for i in range(n)], device="cuda")
    owner = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device="cuda")
    page, slot = s["table"][owner, place // PAGE].long(), place % PAGE
    kc[page, slot], vc[page, slot] = k, v
    return [q, kc, vc]


def _exact_prefix(case, s):
    rows, lens = _lengths(case)
    T, Hq, Hkv, D = sum(rows), case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    four = case["op"] == "prefix4"
    kv = [_values(s, x, D) for x in (("k4", "v4") if four else ("kc", "vc"))]
    t0 = 0
    for g, (n, L) in enumerate(zip(rows, lens)):
        pages = s["table"][g, :-(-L // PAGE)].long()
        part = slice(t0, t0 + n)
        for h in range(Hq if n else 0):
            hk = h // (Hq // Hkv)
            k, v = ((x[pages, hk] if four else x[pages, :, hk]).reshape(-1, D)[:L] for x in kv)
            # the own keys stand for one more key, of score own_lse and value own_out
            z = torch.cat((s["q"][part, h].double() @ k.T / math.sqrt(D), s["own_lse"][part, h, None].double()), 1)
            w = torch.softmax(z, -1)
            out[part, h] = w[:, :-1] @ v + w[:, -1:] * s["own_out"][part, h].double()
            lse[part, h] = torch.logsumexp(z, -1)
        t0 += n
    return [out, lse]


def _exact_sample(case, s):
    tokens, logprobs, counts, left = [], [], [], []
    for r in range(case["M"]):
        x = s["logits"][r].double()
        t, k, p, low = (s[name][r // case["per"]].item() for name in ("temperature", "top_k", "top_p", "min_p"))
        if t == 0:
            kept = torch.zeros_like(x, dtype=torch.bool)
            kept[(x == x.max()).nonzero()[0]] = True
            t = 1.0
        else:
            kept = torch.ones_like(x, dtype=torch.bool)
            order = torch.sort(-x, stable=True).indices
            if k > 0:
                kept[order[k:]] = False
            if p < 1:
                prob = torch.softmax(torch.where(kept, x / t, -math.inf), 0)[order]
                kept[order[1:][torch.cumsum(prob, 0)[:-1] >= p]] = False
            if low > 0:
                kept &= (x - x.max()) / t >= math.log(low)
        counts.append(int(kept.sum()))
        if case["op"] == "truncate":
            left.append(torch.where(kept, x, -math.inf))
            continue
        index = kept.nonzero()[:, 0]
        logp = torch.log_softmax(x[index] / t, 0)
        at = torch.searchsorted(torch.cumsum(logp.exp(), 0), s["u"][r].double(), right=True).clamp(max=len(index) - 1)
        tokens.append(int(index[at]))
        logprobs.append(logp[at])
    counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
    if case["op"] == "truncate":
        return [torch.stack(left), counts]
    return [torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.stack(logprobs), counts]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_axes if op.startswith("axes") else _exact_prefix if op.startswith("prefix") else _exact_sample)(case, s)
