"""GPU parity of sampling and truncation against the fp64 oracle.

Tokens and the numbers of kept entries are equal: weights are good to 2^-36, so
that a border of 10^5 entries would have to lie closer than 10^-10 of the sum to
a uniform number or a top-p.  A log-prob is -(a + b), a = (max - x) / T in two
fp32 roundings, b = log1p of a rounded sum (4 roundings, counted as half steps),
and their sum's rounding: 6 * 2^-24 of itself, and 2^-35 of the weights' own.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
F = np.float32
SETTINGS = [  # temperature, top_k, top_p, min_p
    (1.0, 0, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (0.0, 5, 0.5, 0.0), (1.0, 1, 1.0, 0.0), (1.3, 0, 0.95, 0.0), (0.8, 0, 0.3, 0.0),
    (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 0.1), (1.0, 0, 1.0, 1.0), (0.9, 1500, 0.99, 0.001), (1.0, 1 << 30, 2.0, 0.0),
    (1.0, 700, 1.0, 0.0), (2.0, 3000, 1.0, 0.0), (1.0, 0, 0.9999, 0.0), (1e-30, 0, 1.0, 0.0), (1e30, 0, 1.0, 0.0),
    (1e30, 0, 0.5, 0.0), (0.05, 20, 0.9, 0.0), (1.0, 64, 1e-20, 0.0), (0.6, 40, 0.95, 0.05)]


def make(kind, M, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rank = torch.stack([torch.randperm(V, generator=g) for _ in range(M)]).float() + 1
    noise = torch.randn(M, V, generator=g)
    x = {"power": 14 - 1.3 * rank.log() + 0.5 * noise, "flat": 0.3 * noise, "normal": 4 * noise - 30, "equal": torch.full((M, V), -2.5),
         "few": torch.round(noise), "zeros": torch.where(noise > 0, 0.0, -0.0),
         "masked": torch.where((noise > 1.0) | (rank == 1), 3 * noise, -torch.inf),
         "lowest": torch.where((noise > 0.5) | (rank == 1), 2 * noise, torch.finfo(DT[dtype]).min),
         "spread": noise * 10.0 ** (6 * torch.rand(M, V, generator=g) - 5)}[kind]
    return x.to(DT[dtype])


def settings_of(rows):
    t, k, p, m = zip(*rows)
    as_t = lambda v, d: torch.tensor(v, dtype=d).cuda()  # noqa: E731
    return dict(temperature=as_t(t, torch.float32), top_k=as_t(k, torch.int32), top_p=as_t(p, torch.float32),
                min_p=as_t(m, torch.float32))


def uniforms(M, seed):
    u = np.random.default_rng(seed).random(M).astype(F)
    u[u == 1] = 0.5
    u[:2] = [0.0, 1 - 2.0 ** -24][:M]
    return u


def check(b, x, rows, u, per=1):
    """One call of each kind over all rows, against the oracle row by row."""
    M = x.shape[0]
    s = settings_of(rows)
    new = lambda d: torch.full((M,), -7, dtype=d, device="cuda")  # noqa: E731
    tok, lp, n, n2, st = new(torch.int32), new(torch.float32), new(torch.int32), new(torch.int32), torch.zeros(1, dtype=torch.int32).cuda()
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok, logprobs=lp, n_kept=n, rows_per_request=per, status=st, **s)
    out = torch.full(x.shape, 5.0, dtype=x.dtype, device="cuda")
    b.eagle_truncate_logits(x, out, n_kept=n2, rows_per_request=per, status=st, **s)
    assert st.item() == 0
    xs, got = x.double().cpu().numpy(), out.double().cpu().numpy()
    for r in range(M):
        t, k, p, m = rows[r // per]
        how = dict(temperature=float(F(t)), top_k=k, top_p=float(F(p)), min_p=float(F(m)))
        kept, _ = oracle.truncate(xs[r], **how)
        assert np.array_equal(got[r], np.where(kept, xs[r], -np.inf)), (r, how, int(kept.sum()), int((got[r] > -np.inf).sum()))
        want = oracle.sample(xs[r], float(u[r]), **how)
        assert (tok[r].item(), n[r].item(), n2[r].item()) == (want[0], want[2], want[2]), (r, how, want)
        assert abs(lp[r].item() - want[1]) <= 6 * 2.0 ** -24 * abs(want[1]) + 2.0 ** -35, (r, how, lp[r].item(), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["power", "flat", "normal", "few", "masked", "lowest", "spread", "equal", "zeros"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 20011, 50257])
def test_all_settings(kind, V, dtype):
    b = need_gpu()
    x = make(kind, len(SETTINGS), V, dtype, V + len(kind)).cuda()
    check(b, x, SETTINGS, uniforms(len(SETTINGS), V))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,V", [("power", 128256), ("normal", 128256), ("flat", 262144), ("equal", 262144), ("few", 151936)])
def test_large_vocabularies(kind, V, dtype):
    b = need_gpu()
    x = make(kind, len(SETTINGS), V, dtype, 3).cuda()
    check(b, x, SETTINGS, uniforms(len(SETTINGS), 4))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("start", [0, 1, 3, 5])
def test_rows_at_any_element(start, dtype):
    """Slices of wider rows, of odd strides, starting at any element; requests of several rows."""
    b = need_gpu()
    V = 5003
    wide = make("power", 7, V + 10, dtype, 8).cuda()
    x = wide[:, start:start + V]
    check(b, x, [SETTINGS[1], SETTINGS[4], SETTINGS[9]], uniforms(7, 9), per=3)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_place_and_odd_outputs(dtype):
    b = need_gpu()
    V, rows = 3001, SETTINGS[:8]
    x = make("power", 8, V, dtype, 10).cuda()
    s = settings_of(rows)
    want = b.eagle_truncate_logits(x, torch.empty_like(x), **s)
    wide = torch.full((8, V + 7), 5.0, dtype=x.dtype, device="cuda")
    b.eagle_truncate_logits(x, wide[:, 3:3 + V], **s)
    assert torch.equal(wide[:, 3:3 + V], want) and (wide[:, :3] == 5).all() and (wide[:, 3 + V:] == 5).all()
    b.eagle_truncate_logits(x, x, **s)
    assert torch.equal(x, want)


@pytest.mark.parametrize("kind", ["power", "flat", "few"])
def test_top_p_next_to_one(kind):
    """The largest fp32 number below 1, where the last entries' weights still reach it."""
    b = need_gpu()
    x = make(kind, 4, 61, "fp32", 21).cuda()
    check(b, x, [(t, 0, 1 - 2.0 ** -24, 0.0) for t in (0.3, 0.7, 1.0, 2.0)], uniforms(4, 22))


def test_uniform_temperature_picks_by_index():
    """At a temperature that levels everything, token = floor(u V)."""
    b = need_gpu()
    V = 4096
    x = make("normal", 64, V, "fp32", 1).cuda()
    u = uniforms(64, 2)
    tok = torch.zeros(64, dtype=torch.int32, device="cuda")
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok, temperature=torch.full((64,), 1e36, device="cuda"))
    assert np.array_equal(tok.cpu().numpy(), np.floor(u.astype(np.float64) * V).astype(int))


def test_settings_left_out():
    b = need_gpu()
    x = make("power", 5, 999, "fp32", 2).cuda()
    u = uniforms(5, 3)
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok)
    xs = x.double().cpu().numpy()
    assert tok.tolist() == [oracle.sample(xs[r], float(u[r]))[0] for r in range(5)]
    none = torch.zeros(0, 999, device="cuda")
    b.eagle_sample(none, u_ := torch.zeros(0, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"))
    b.eagle_truncate_logits(none, none.clone(), n_kept=u_.int())


@pytest.mark.parametrize("bad,code", [("nan", 7), ("inf", 7), ("empty", 7), ("t", 1), ("t_inf", 1), ("k", 1), ("p", 1), ("p_nan", 1),
                                      ("m", 1), ("u", 1), ("u_nan", 1)])
def test_rows_in_error_and_their_neighbours(bad, code):
    b = need_gpu()
    V = 2003
    x = make("power", 3, V, "fp32", 6).cuda()
    rows = [list(SETTINGS[1]) for _ in range(3)]
    u = uniforms(3, 5)
    if bad in ("nan", "inf"):
        x[1, V - 1] = float(bad)
    elif bad == "empty":
        x[1] = -torch.inf
    elif bad.startswith("u"):
        u[1] = 1.0 if bad == "u" else np.nan
    else:
        at, v = {"t": (0, -0.5), "t_inf": (0, np.inf), "k": (1, -1), "p": (2, -0.1), "p_nan": (2, np.nan), "m": (3, 1.5)}[bad]
        rows[1][at] = v
    s = settings_of(rows)
    st = torch.zeros(1, dtype=torch.int32).cuda()
    tok, lp, n = (torch.zeros(3, dtype=d, device="cuda") for d in (torch.int32, torch.float32, torch.int32))
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok, logprobs=lp, n_kept=n, status=st, **s)
    assert st.item() == code
    assert tok[1].item() == -1 and lp[1].item() == -np.inf and n[1].item() == 0
    xs = x.double().cpu().numpy()
    for r in (0, 2):
        t, k, p, m = rows[r]
        assert tok[r].item() == oracle.sample(xs[r], float(u[r]), temperature=float(F(t)), top_k=k, top_p=float(F(p)), min_p=m)[0]
    if not bad.startswith("u"):
        st.zero_()
        out = torch.full((3, V), 5.0, device="cuda")
        b.eagle_truncate_logits(x, out, n_kept=n, status=st, **s)
        assert st.item() == code and (out[1] == 5).all() and n[1].item() == 0 and (out[0] != 5).all()


def test_graph_and_another_stream():
    """A captured call follows its inputs, on a stream of its own; two runs agree bit for bit."""
    b = need_gpu()
    V, rows = 128256, SETTINGS
    M = len(rows)
    x, s = make("power", M, V, "bf16", 12).cuda(), settings_of(rows)
    u = torch.from_numpy(uniforms(M, 1)).cuda()
    tok, out = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.eagle_sample(x, u, tok, stream=side, **s)
    b.eagle_truncate_logits(x, out, stream=side, **s)
    side.synchronize()
    first, first_out = tok.clone(), out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.eagle_sample(x, u, tok, **s)
        b.eagle_truncate_logits(x, out, **s)
    tok.zero_()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, first) and torch.equal(out, first_out)
    x.copy_(make("flat", M, V, "bf16", 13))
    g.replay()
    torch.cuda.synchronize()
    want = torch.zeros_like(tok)
    b.eagle_sample(x, u, want, **s)
    assert torch.equal(tok, want) and not torch.equal(tok, first)


def test_many_rows():
    b = need_gpu()
    M, V = 5000, 61
    x = make("normal", M, V, "fp32", 14).cuda()
    u = uniforms(M, 15)
    tok = torch.zeros(M, dtype=torch.int32, device="cuda")
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok, top_p=torch.full((M,), 0.9, device="cuda"))
    xs = x.double().cpu().numpy()
    assert tok.tolist() == [oracle.sample(xs[r], float(u[r]), top_p=float(F(0.9)))[0] for r in range(M)]


@pytest.mark.parametrize("V,dtype", [(20011, "fp32"), (128256, "bf16"), (262144, "fp32"), (262144, "bf16")])
@pytest.mark.parametrize("kind", ["power", "equal", "few", "spread"])
def test_many_kept_with_borders_near_one_another(kind, V, dtype):
    """Top-p cuts of many entries with min-p in front of them, behind them and among them,
    behind a top-k, at the ends of temperature's range."""
    b = need_gpu()
    rows = [(1.3, 0, 0.95, 1e-3), (1.3, 0, 0.95, 1e-12), (1.0, 0, 0.99, 1e-5), (1.0, 0, 1 - 2.0 ** -15, 0.0),
            (1.0, 20000, 0.97, 0.0), (2.0, 60000, 0.999, 1e-6), (1e-30, 0, 0.9, 0.0), (1e-38, 0, 0.5, 0.0), (3e38, 0, 0.25, 0.0), (40.0, 0, 0.75, 0.0)]
    x = make(kind, len(rows), V, dtype, V + len(kind)).cuda()
    check(b, x, rows, uniforms(len(rows), V))


@pytest.mark.parametrize("V,dtype", [(20011, "fp32"), (128256, "bf16"), (262144, "fp32"), (262144, "bf16")])
@pytest.mark.parametrize("kind", ["power", "equal", "few", "spread", "flat"])
def test_top_p_next_to_one_of_many(kind, V, dtype):
    """p = 1 - 2^-24, which leaves out 2^-24 of the sum S.  A weight is off by 2^-45 (half a
    unit) and 2^-36 of itself, so S, and a sum in front of an entry, by at most e = V 2^-45
    + 2^-36 S, and the two borders, p S and that sum, by 2 e from one another.  What is kept is
    the head of the order, and its last entry the last in front of p S within 2 e."""
    b = need_gpu()
    temps = (0.3, 1.0, 2.5)
    x = make(kind, len(temps), V, dtype, V + len(kind)).cuda()
    s = settings_of([(t, 0, 1 - 2.0 ** -24, 0.0) for t in temps])
    n, st = torch.empty(len(temps), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).cuda()
    out = b.eagle_truncate_logits(x, torch.empty_like(x), n_kept=n, status=st, **s).double().cpu().numpy()
    tok, n2 = torch.empty_like(n), torch.empty_like(n)
    b.eagle_sample(x, torch.full((len(temps),), 1 - 2.0 ** -24, device="cuda"), tok, n_kept=n2, status=st, **s)
    assert st.item() == 0 and torch.equal(n, n2)
    for r, t in enumerate(temps):
        row, m = x[r].double().cpu().numpy(), n[r].item()
        order = np.lexsort((np.arange(V), -row))
        kept = np.zeros(V, bool)
        kept[order[:m]] = True
        assert np.array_equal(out[r], np.where(kept, row, -np.inf)) and kept[tok[r].item()]
        run = np.concatenate([[0.0], np.cumsum(np.exp((row[order] - row.max()) / float(F(t))))])
        e = V * 2.0 ** -45 + 2.0 ** -36 * run[-1]
        border = (1 - 2.0 ** -24) * run[-1]
        assert run[m - 1] < border + 2 * e and run[m] > border - 2 * e, (t, m, run[m - 1] - border, run[m] - border, e)


@pytest.mark.parametrize("M,V,dtype", [(200, 32000, "bf16"), (400, 32001, "bf16"), (700, 20011, "fp32"), (640, 65539, "bf16")])
def test_many_rows_in_smaller_clusters(M, V, dtype):
    """Every kind of row among many, on the rows' own settings; those checked are the first of each setting."""
    b = need_gpu()
    rows = [SETTINGS[i % len(SETTINGS)] for i in range(M)]
    first = len(SETTINGS)
    x = make("power", 2 * first, V, dtype, V)
    x[::3] = make("normal", 2 * first, V, dtype, V + 1)[::3]
    x = x.repeat(-(-M // (2 * first)), 1)[:M].contiguous().cuda()
    u = np.tile(uniforms(2 * first, M), -(-M // (2 * first)))[:M]
    s = settings_of(rows)
    tok, n, st = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).cuda()
    b.eagle_sample(x, torch.from_numpy(u).cuda(), tok, n_kept=n, status=st, **s)
    out = b.eagle_truncate_logits(x, torch.empty_like(x), status=st, **s)
    assert st.item() == 0
    per = 2 * first
    want = oracle_rows(x[:per], rows[:per], u[:per])
    tok, n = tok.cpu().numpy(), n.cpu().numpy()
    for r in range(M):
        assert (tok[r], n[r]) == want[r % per][:2], (r, rows[r])
    for r in range(0, M, per):  # the same rows again
        assert torch.equal(out[r:r + per], out[:min(per, M - r)])
    for r in range(per):
        assert np.array_equal(out[r].double().cpu().numpy(), want[r][2])


def oracle_rows(x, rows, u):
    """(token, entries kept, truncated row) of each row."""
    result = []
    for r, (t, k, p, m) in enumerate(rows):
        row = x[r].double().cpu().numpy()
        how = dict(temperature=float(F(t)), top_k=k, top_p=float(F(p)), min_p=float(F(m)))
        token, _, kept = oracle.sample(row, float(u[r]), **how)
        result.append((token, kept, np.where(oracle.truncate(row, **how)[0], row, -np.inf)))
    return result
