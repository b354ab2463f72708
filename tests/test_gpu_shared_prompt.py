"""The calls for requests behind shared prefixes, run together: rows appended at
their positions behind a prefix, attention over the own keys joined with the
prefix's, and tokens sampled or a tree verified against truncated logits.

Each step is held against fp64 on what the GPU's caches and rows hold.  An append
is bounded as in its own test.  The joined attention: the own result is rounded to
the type and then the joined one, both with rounded weights, and fp32 arithmetic
(2 (D + 9) |q||k| scale + twice the terms) 2^-24 + 2^-21, against sum w|v|.  A
projection: products of bf16 and of fp32 rounded to fp32 and summed in fp32,
(2 K + 2) 2^-24 sum |x w|, and the type's half step.
"""
import numpy as np
import pytest
import torch

import oracle
from eagle_speculative_decoding_gb300 import synth
from gpu_helpers import NORM_TOL, need_gpu, norm_err
from test_gpu_prefix import KINDS, P_HALF
from test_gpu_prompt import DT, HALF, f64

pytestmark = pytest.mark.gpu
Hq, Hkv, D, WIDTH, V, MAX_POS = 8, 2, 64, 256, 640, 256
PREFIX, OF_GROUP, OWN, STEPS = [70, 33], [3, 2], [5, 1, 12, 3, 16], 4
SETTINGS = [(0.8, 20, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.7, 0.05), (1.3, 0, 1.0, 0.0), (0.6, 5, 1.0, 0.1)]
MARGIN = 1e-4


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Server:
    """One attention layer and an LM head over requests behind shared prefixes."""

    def __init__(self, b, kind, seed):
        g = torch.Generator().manual_seed(seed)
        self.b, self.kind, self.kv4 = b, kind, kind == "kv4"
        self.dt = DT["fp32" if kind == "fp32" else "bf16"]
        n = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
        self.embed = n(V, WIDTH).to(self.dt).cuda()
        self.w_qkv, self.w_o, self.w_lm = [(n(a, c) * f).to(self.dt).cuda() for a, c, f in (
            ((Hq + 2 * Hkv) * D, WIDTH, 0.1), (WIDTH, Hq * D, 0.05), (V, WIDTH, 0.15))]
        self.rope = b.eagle_rope_table(MAX_POS, D, 10000.0)
        # pages: the prefixes', then the requests' own
        need = [-(-L // 16) for L in PREFIX] + [-(-(L + STEPS) // 16) for L in OWN]
        P = sum(need) + 1
        ids = torch.randperm(P, generator=g).tolist()
        tables = [[ids.pop() for _ in range(x)] for x in need]
        full = lambda t: i32([x + [-1] * (max(map(len, t)) - len(x)) for x in t])  # noqa: E731
        self.prefix_table, self.table = full(tables[:len(PREFIX)]), full(tables[len(PREFIX):])
        if self.kv4:
            self.pages = [torch.zeros(P, Hkv, 16, x, dtype=torch.uint8, device="cuda") for x in (D // 2, D // 16) * 2]
        else:
            self.pages = [torch.zeros(P, 16, Hkv, D, dtype=self.dt, device="cuda") for _ in range(2)]
        self.st = i32([0])

    def call(self, name, *args, **kw):
        return getattr(self.b, "eagle_" + name + ("_kv4" if self.kv4 else ""))(*args, status=self.st, **kw)

    def linear(self, x, w, residual=None, stream=None):
        y = torch.empty(x.shape[0], w.shape[0], dtype=self.dt, device="cuda")
        return self.b.eagle_linear(x, w, y, residual=residual, status=self.st, stream=stream)

    def append(self, tokens, positions, cu, ctx, table, stream=None):
        x = self.embed[tokens.long()]
        rows = self.linear(x, self.w_qkv, stream=stream).view(-1, Hq + 2 * Hkv, D)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        q_out = torch.empty(len(x), Hq, D, dtype=self.dt, device="cuda")
        self.call("kv_append_axes", q, k, v, self.rope, positions, cu, ctx, table, *self.pages, q_out=q_out, stream=stream)
        return x, rows, q_out

    def step(self, tokens, positions, cu, ctx, last, uniforms, settings, cu_groups, lens, stream=None):
        """Tokens of requests [T] -> one sampled token each; what the checks need beside."""
        x, rows, q = self.append(tokens, positions, cu, ctx, self.table, stream)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        self.call("prompt_attn", q, *self.pages, self.table, cu, ctx, out, lse=lse, stream=stream)
        self.call("prefix_attn", q, *self.pages, self.prefix_table, cu_groups, lens, out, lse=lse, own_out=out, own_lse=lse, stream=stream)
        y = self.linear(out.view(-1, Hq * D), self.w_o, residual=x, stream=stream)[last]
        logits = self.linear(y, self.w_lm, stream=stream)
        new = torch.empty(len(last), dtype=torch.int32, device="cuda")
        self.b.eagle_sample(logits, uniforms, new, status=self.st, stream=stream, **settings)
        return dict(rows=rows, q=q, out=out, lse=lse, y=y, logits=logits, tokens=new)

    def prefill(self, g):
        prompt = torch.randint(0, V, (sum(PREFIX),), generator=g).cuda()
        at = i32([list(range(PREFIX[0])) + list(range(PREFIX[1]))])
        return self.append(prompt, at, i32([0] + list(np.cumsum(PREFIX))), i32([0] * len(PREFIX)), self.prefix_table)

    def cache(self):
        """Keys and values in fp64, [P, 16, Hkv, D]."""
        if not self.kv4:
            return [f64(x) for x in self.pages]
        out = torch.empty(self.pages[0].shape[0], 16, Hkv, D, device="cuda")
        return [f64(self.b.eagle_kv4_read(c, s, out)) for c, s in (self.pages[:2], self.pages[2:])]


def rotated_rows(s, rows, positions):
    r = f64(s.rope)[positions]
    return oracle.rotate(f64(rows[:, :Hq]), r), oracle.rotate(f64(rows[:, Hq:Hq + Hkv]), r), f64(rows[:, Hq + Hkv:])


def check_append(s, rows, q, positions, places):
    half = HALF["fp32" if s.kind == "fp32" else "bf16"]
    pair = lambda x: np.tile(np.hypot(x[..., :D // 2], x[..., D // 2:]), 2)  # noqa: E731
    want, k, v = rotated_rows(s, rows, positions)
    assert (np.abs(f64(q) - want) <= half * np.abs(want) + 2.0 ** -22 * pair(want)).all()
    kc, vc = s.cache()
    for t, (_, _, page, slot) in enumerate(places):
        if s.kv4:  # of the codes 0 .. 6 the last step is 2, of a scale that is off by 2^-4 (or by 2^-10 near zero)
            for got, x in ((kc, k), (vc, v)):
                top = np.repeat(np.abs(x[t]).reshape(Hkv, D // 16, 16).max(-1), 16, -1)
                assert (np.abs(got[page, slot] - x[t]) <= 0.18 * top + 6 * 2.0 ** -10).all()
        else:
            assert (np.abs(kc[page, slot] - k[t]) <= half * np.abs(k[t]) + 2.0 ** -22 * pair(k[t])).all()
            assert np.array_equal(vc[page, slot], v[t])


def check_linear(x, w, y, half, residual=0.0):
    x, w, y = f64(x), f64(w), f64(y)
    want = x @ w.T + residual
    assert (np.abs(y - want) <= half * np.abs(want) + (2 * x.shape[1] + 2) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T + np.abs(residual))).all()


def inputs(settings=SETTINGS):
    t, k, p, m = zip(*settings)
    f = lambda x: torch.tensor(x, dtype=torch.float32).cuda()  # noqa: E731
    return dict(temperature=f(t), top_k=i32(k), top_p=f(p), min_p=f(m))


def plan(new, ctx):
    """Arrays of a step: positions behind the prefixes, borders, last rows."""
    group = np.repeat(range(len(PREFIX)), OF_GROUP)
    pos = [PREFIX[group[r]] + ctx[r] + i for r in range(len(new)) for i in range(new[r])]
    cu = np.concatenate([[0], np.cumsum(new)])
    return pos, cu, [int(cu[c]) for c in np.concatenate([[0], np.cumsum(OF_GROUP)])]


@pytest.mark.parametrize("kind", KINDS)
def test_generation_behind_shared_prefixes(kind):
    b = need_gpu()
    s, g = Server(b, kind, 1), torch.Generator().manual_seed(2)
    half, rng = HALF["fp32" if kind == "fp32" else "bf16"], np.random.default_rng(3)
    x, rows, q = s.prefill(g)
    places = oracle.row_places([0] + list(np.cumsum(PREFIX)), [0] * len(PREFIX), s.prefix_table.cpu().numpy())
    check_append(s, rows, q, [p[1] for p in places], places)
    tokens, new, ctx = torch.randint(0, V, (sum(OWN),), generator=g).cuda(), list(OWN), [0] * len(OWN)
    for step in range(STEPS):
        pos, cu, groups = plan(new, ctx)
        u = rng.random(len(OWN)).astype(np.float32) * np.float32(0.999)
        r = s.step(tokens, i32([pos]), i32(cu.tolist()), i32(ctx), torch.from_numpy(cu[1:] - 1).cuda(), torch.from_numpy(u).cuda(), inputs(),
                   i32(groups), i32(PREFIX))
        assert s.st.item() == 0
        table = s.table.cpu().numpy()
        check_append(s, r["rows"], r["q"], pos, oracle.row_places(cu, ctx, table))
        kc, vc = s.cache()
        pre = s.prefix_table.cpu().numpy()
        of = np.repeat(range(len(PREFIX)), OF_GROUP)
        flat = lambda c, pages, n: c[np.maximum(pages, 0)].reshape(-1, Hkv, D)[:n]  # noqa: E731
        keys, values = ([np.concatenate([flat(c, pre[of[i]], PREFIX[of[i]]), flat(c, table[i], ctx[i] + new[i])]) for i in range(len(OWN))]
                        for c in (kc, vc))
        want, wl, mag, dot = oracle.prompt_attn(f64(r["q"]), keys, values, cu, [PREFIX[of[i]] + ctx[i] for i in range(len(OWN))], D ** -0.5)
        arith = (2 * (D + 9) * dot + 2 * (max(PREFIX) + max(OWN) + STEPS) + 32) * 2.0 ** -24 + 2.0 ** -21
        assert (np.abs(f64(r["out"]) - want) <= half * np.abs(want) + (half + P_HALF[kind] + arith[..., None]) * mag).all()
        assert (np.abs(f64(r["lse"]) - wl) <= 2 * arith + 2.0 ** -22 * (np.abs(wl) + 1)).all()
        check_linear(r["y"], s.w_lm, r["logits"], half)
        z = f64(r["logits"])
        for i, (t, k, p, m) in enumerate(SETTINGS):
            how = dict(temperature=float(np.float32(t)), top_k=k, top_p=float(np.float32(p)), min_p=float(np.float32(m)))
            assert r["tokens"][i].item() == oracle.sample(z[i], float(u[i]), **how)[0], (step, i)
        tokens, ctx, new = r["tokens"], [c + n for c, n in zip(ctx, new)], [1] * len(OWN)


@pytest.mark.parametrize("kind", KINDS)
def test_step_in_a_graph_and_two_at_once(kind):
    """A captured step replayed on other inputs, and two steps of two servers at the
    same time on streams of their own, give the same bits as steps by themselves."""
    b = need_gpu()
    g = torch.Generator().manual_seed(5)
    servers = [Server(b, kind, 6), Server(b, kind, 7)]
    for s in servers:
        s.prefill(g)
    pos, cu, groups = plan([1] * len(OWN), OWN)
    ctx, last, at = i32(OWN), torch.from_numpy(cu[1:] - 1).cuda(), i32([pos])
    rest = (inputs(), i32(groups), i32(PREFIX))
    cu = i32(cu.tolist())
    tokens = [torch.randint(0, V, (len(OWN),), generator=g).int().cuda() for _ in range(2)]
    u = [torch.rand(len(OWN), generator=g).mul_(0.999).cuda() for _ in range(2)]
    blank = [[p.clone() for p in s.pages] for s in servers]

    def restore():
        for s, pages in zip(servers, blank):
            for p, x in zip(s.pages, pages):
                p.copy_(x)

    alone = [s.step(t, at, cu, ctx, last, x, *rest) for s, t, x in zip(servers, tokens, u)]
    caches = [[p.clone() for p in s.pages] for s in servers]
    # two at once
    restore()
    streams = [torch.cuda.Stream() for _ in servers]
    both = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for s, t, x, st in zip(servers, tokens, u, streams):
        with torch.cuda.stream(st):
            both.append(s.step(t, at, cu, ctx, last, x, *rest))
    torch.cuda.synchronize()
    same = lambda x, y: all(torch.equal(x[n], y[n]) for n in x)  # noqa: E731
    assert all(same(x, y) for x, y in zip(alone, both))
    assert all(torch.equal(p, x) for s, c in zip(servers, caches) for p, x in zip(s.pages, c))
    # a graph, whose inputs change
    restore()
    s, t, x = servers[0], tokens[0].clone(), u[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = s.step(t, at, cu, ctx, last, x, *rest)
    for other in (0, 1, 0):
        t.copy_(tokens[other])
        x.copy_(u[other])
        graph.replay()
        torch.cuda.synchronize()
        got = {n: r[n].clone() for n in r}
        assert same(got, s.step(t, at, cu, ctx, last, x, *rest))
    assert same(got, alone[0]) and all(v.st.item() == 0 for v in servers)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_tree_round_behind_a_shared_prefix(kind):
    """Tree rows over own pages joined with a shared prefix are tree attention over
    all of it; logits truncated in place; the tree verified against them."""
    b = need_gpu()
    B, R, L, depth, T = 6, 21, 150, 5, float(np.float32(0.9))
    gen = synth.generator(11)
    dt = DT[kind]
    own = [0, 3, 16, 40, 17, 90]
    q, kt, vt = [synth.normal((B, R, h, D), 1.0, dt, gen) for h in (Hq, Hkv, Hkv)]
    kc, vc, table = synth.paged_kv([L] + own, Hkv, D, 16, dt, gen)
    trees = [synth.random_tree(R, depth, gen)[0] for _ in range(B)]
    mask = torch.from_numpy(np.stack([oracle.ancestor_mask(t.numpy()).astype(np.int64) for t in trees]))
    parent, tok = torch.stack(trees).int(), torch.stack([synth.distinct_sibling_tokens(t, V, gen) for t in trees]).int()
    d = lambda x: x.contiguous().cuda()  # noqa: E731
    out, lse, st = torch.empty_like(q, device="cuda"), torch.empty(B, R, Hq, device="cuda"), i32([0])
    qd, kcd, vcd = d(q), d(kc), d(vc)
    b.eagle_tree_attn(qd, d(kt), d(vt), kcd, vcd, d(table[1:]), i32(own), d(mask), out, lse=lse, status=st)
    rows, row_lse = out.view(B * R, Hq, D), lse.view(B * R, Hq)
    b.eagle_prefix_attn(qd.view(B * R, Hq, D), kcd, vcd, d(table[:1]), i32([0, B * R]), i32([L]), rows, lse=row_lse, own_out=rows,
                        own_lse=row_lse, status=st)
    # the same with every request's keys in pages of its own
    flat = lambda c, r, n: f64(c)[np.maximum(table[r].numpy(), 0)].reshape(-1, Hkv, D)[:n]  # noqa: E731
    per = -(-(L + max(own)) // 16)
    whole = []
    for c in (kc, vc):
        w = np.zeros((B, per * 16, Hkv, D))
        for r in range(B):
            w[r, :L + own[r]] = np.concatenate([flat(c, 0, L), flat(c, r + 1, own[r])])
        whole.append(w.reshape(B * per, 16, Hkv, D))
    want, wl = oracle.tree_attn(f64(q), f64(kt), f64(vt), *whole, np.arange(B * per).reshape(B, per), np.array(own) + L,
                                mask.numpy().astype(np.uint64))
    assert norm_err(f64(out), want) < (1e-4 if kind == "fp32" else NORM_TOL)
    assert np.abs(f64(lse) - wl).max() < (1e-4 if kind == "fp32" else 2e-2)
    # logits near which the drafted tokens lie, truncated in place
    w_lm = synth.normal((V, Hq * D), 0.3, dt, gen)
    z = torch.empty(B * R, V, dtype=dt, device="cuda")
    b.eagle_linear(rows.view(B * R, Hq * D), d(w_lm), z, status=st)
    z = z.float().view(B, R, V)
    for r in range(B):
        for c in range(1, R):
            p = int(parent[r, c])
            z[r, p, int(tok[r, c])] = z[r, p].max() + (c % 3 - 1) * T
    whole_z = z.double().cpu().numpy()
    settings = dict(temperature=torch.full((B,), T, device="cuda"), top_k=i32([0, 12, 30, 0, 1, 8]),
                    top_p=torch.tensor([0.8, 1.0, 0.9, 0.6, 1.0, 0.95]).cuda())
    kept = torch.empty(B * R, dtype=torch.int32, device="cuda")
    b.eagle_truncate_logits(z.view(B * R, V), z.view(B * R, V), rows_per_request=R, n_kept=kept, status=st, **settings)
    got = z.double().cpu().numpy()
    for r in range(B):
        how = dict(temperature=T, top_k=int(settings["top_k"][r]), top_p=float(settings["top_p"][r]))
        for i in range(R):
            k, _ = oracle.truncate(whole_z[r, i], **how)
            assert np.array_equal(got[r, i], np.where(k, whole_z[r, i], -np.inf)) and kept[r * R + i].item() == k.sum()
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    path, new = [torch.empty(B, depth + 1, dtype=torch.int32, device="cuda") for _ in range(2)]
    b.eagle_tree_verify(d(parent), d(tok), T, depth, acc, path, new, target_logits=z, seed=77, offset=5, status=st)
    assert st.item() == 0
    ref = oracle.tree_verify(parent.numpy(), tok.numpy(), T, depth, target_logits=got, seed=77, offset=5)
    close = {r for _, r, m in ref["margins"] if m < MARGIN}
    assert not close and ref["accept_len"].max() >= 1
    assert np.array_equal(acc.cpu().numpy(), ref["accept_len"]) and np.array_equal(path.cpu().numpy(), ref["path_rows"])
    assert np.array_equal(new.cpu().numpy(), ref["out_tokens"])
    # nothing outside the truncated distribution is given out
    for r in range(B):
        for i in range(int(acc[r]) + 1):
            assert got[r, int(path[r, i]), int(new[r, i])] > -np.inf
