"""Refusals of the prompt-path calls, on the host: every case returns before
any CUDA call (no GPU needed)."""
import ctypes
import os

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
N, P, ODD = None, ctypes.c_void_p(256), ctypes.c_void_p(8)


@pytest.fixture(scope="module")
def L():
    from eagle_speculative_decoding_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def append(L, **kw):
    a = dict(q=P, k=P, v=P, qs=512, ks=256, vs=256, rope=P, max_pos=64, cu=P, ctx=P, B=2, T=4, Hq=4, Hkv=2, D=128,
             dtype=1, q_out=ctypes.c_void_p(512), kc=P, vc=P, pages=8, table=P, width=4)
    a.update(kw)
    return L.eagle_kv_append(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["rope"], a["max_pos"], a["cu"], a["ctx"],
                             a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["dtype"], a["q_out"], a["kc"], a["vc"],
                             a["pages"], a["table"], a["width"], N, N)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)),
    (INVALID, dict(k=N)), (INVALID, dict(v=N)), (INVALID, dict(kc=N)), (INVALID, dict(vc=N)), (INVALID, dict(cu=N)),
    (INVALID, dict(ctx=N)), (INVALID, dict(table=N)), (INVALID, dict(q=N)), (INVALID, dict(q_out=N)),
    (INVALID, dict(Hq=0)), (INVALID, dict(B=0)), (INVALID, dict(T=-1)), (INVALID, dict(Hkv=0)), (INVALID, dict(pages=0)),
    (INVALID, dict(width=0)), (INVALID, dict(max_pos=0)), (INVALID, dict(dtype=2)), (UNSUPPORTED, dict(D=96)),
    (UNSUPPORTED, dict(Hkv=600, ks=600 * 128, vs=600 * 128)), (INVALID, dict(qs=511)), (INVALID, dict(ks=128)),
    (INVALID, dict(vs=260)), (INVALID, dict(k=ODD)), (INVALID, dict(q_out=ODD)), (INVALID, dict(rope=ODD)),
    (INVALID, dict(q_out=P, qs=1024)), (UNSUPPORTED, dict(pages=(1 << 26) + 1)),
])
def test_append_refusals(L, want, kw):
    assert append(L, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (INVALID, dict(ks=N)), (INVALID, dict(k_scale=0.0)), (INVALID, dict(v_scale=float("inf"))),
    (INVALID, dict(k_scale=float("nan"))), (INVALID, dict(kc=ODD)), (UNSUPPORTED, dict(D=32)),
])
def test_append_kv4_refusals(L, want, kw):
    a = dict(T=4, D=128, kc=P, ks=P, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    assert L.eagle_kv_append_kv4(P, P, P, 512, 256, 256, P, 64, P, P, 2, a["T"], 4, 2, a["D"], ctypes.c_void_p(512),
                                 a["kc"], a["ks"], P, P, a["k_scale"], a["v_scale"], 8, P, 4, N, N) == want


def attn(L, **kw):
    a = dict(q=P, qs=512, kc=P, vc=P, pages=8, table=P, width=4, cu=P, ctx=P, out=P, B=2, T=4, Hq=4, Hkv=2, D=128,
             page=16, scale=0.1, dtype=1, ws=N, wsb=0)
    a.update(kw)
    return L.eagle_prompt_attn(a["q"], a["qs"], a["kc"], a["vc"], a["pages"], a["table"], a["width"], a["cu"], a["ctx"],
                               a["out"], N, a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["page"], a["scale"], a["dtype"],
                               a["ws"], a["wsb"], N, N)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (WORKSPACE, dict()), (WORKSPACE, dict(ws=P, wsb=16)),
    (INVALID, dict(q=N)), (INVALID, dict(kc=N)), (INVALID, dict(vc=N)), (INVALID, dict(table=N)), (INVALID, dict(cu=N)),
    (INVALID, dict(ctx=N)), (INVALID, dict(out=N)), (INVALID, dict(B=0)), (INVALID, dict(T=-1)), (INVALID, dict(Hq=5)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(dtype=7)), (INVALID, dict(qs=500)), (INVALID, dict(qs=516)), (INVALID, dict(q=ODD)),
    (INVALID, dict(out=ODD)), (UNSUPPORTED, dict(D=96)), (UNSUPPORTED, dict(page=32)),
    (UNSUPPORTED, dict(Hq=130, qs=130 * 128)), (UNSUPPORTED, dict(B=65536)), (UNSUPPORTED, dict(pages=(1 << 26) + 1)),
])
def test_attn_refusals(L, want, kw):
    assert attn(L, **kw) == want


@pytest.mark.parametrize("want,ks,k_scale,wsb", [
    (INVALID, N, 1.0, 0), (INVALID, P, -1.0, 0), (INVALID, P, float("nan"), 0), (WORKSPACE, P, 1.0, 0)])
def test_attn_kv4_refusals(L, want, ks, k_scale, wsb):
    assert L.eagle_prompt_attn_kv4(P, 512, P, ks, P, P, k_scale, 1.0, 8, P, 4, P, P, P, N, 2, 4, 4, 2, 128, 16, 0.1, N,
                                   wsb, N, N) == want


def test_table_and_read_refusals(L):
    assert L.eagle_rope_table(0, 128, 1e4, P, N) == INVALID
    assert L.eagle_rope_table(8, 128, 0.0, P, N) == INVALID
    assert L.eagle_rope_table(8, 128, 1e4, N, N) == INVALID
    assert L.eagle_rope_table(8, 96, 1e4, P, N) == UNSUPPORTED
    assert L.eagle_kv4_read(N, P, 1.0, 4, 2, 128, 1, P, N) == INVALID
    assert L.eagle_kv4_read(P, P, 0.0, 4, 2, 128, 1, P, N) == INVALID
    assert L.eagle_kv4_read(P, P, 1.0, 4, 2, 128, 3, P, N) == INVALID
    assert L.eagle_kv4_read(P, P, 1.0, 4, 2, 80, 1, P, N) == UNSUPPORTED
    assert L.eagle_kv4_read(P, P, 1.0, 4, 1025, 128, 1, P, N) == UNSUPPORTED


def test_workspace_query(L):
    assert L.eagle_prompt_attn_workspace_size(1, 1, 1, 1, 64) > 0
    assert L.eagle_prompt_attn_workspace_size(64, 8192, 32, 8, 128) >= L.eagle_prompt_attn_workspace_size(1, 1, 32, 8, 128)
    for bad in ((0, 4, 4, 2, 64), (1, 4, 5, 2, 64), (1, 4, 4, 2, 80), (1, -1, 4, 2, 64)):
        assert L.eagle_prompt_attn_workspace_size(*bad) == 0


def test_binding_refuses_strided_heads():
    from eagle_speculative_decoding_gb300 import binding as eb
    q = torch.zeros(4, 4, 256)[..., :128]
    with pytest.raises(ValueError):
        eb._row_stride("q", q, 128)
    assert eb._row_stride("q", torch.zeros(4, 6, 128)[:, :4], 128) == 6 * 128


def test_draft_prompt_refusals(L):
    def call(x=P, out=ctypes.c_void_p(512), rope=P, ks=N, vs=N, d=256, D=64, I=256, dtype=1, T=4, max_pos=8, eps=1e-5):
        return L.eagle_draft_prompt(x, P, P, P, P, P, P, eps, rope, max_pos, P, P, P, P, ks, vs, 1.0, 1.0, 8, P, 4, out, 2,
                                    T, d, 4, 2, D, I, dtype, N, 0, N, N)
    assert call(T=0) == OK and call() == WORKSPACE
    for kw in (dict(x=N), dict(out=P), dict(rope=N), dict(ks=P), dict(ks=P, vs=P, dtype=0), dict(dtype=5), dict(max_pos=0),
               dict(eps=-1.0), dict(T=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=100), dict(D=96), dict(I=100)):
        assert call(**kw) == UNSUPPORTED, kw
    assert L.eagle_draft_prompt_workspace_size(2, 5000, 256, 4, 2, 64, 256, 1) > 0
    assert L.eagle_draft_prompt_workspace_size(2, 4, 100, 4, 2, 64, 256, 1) == 0


def test_no_rows_need_no_addresses(L):
    assert append(L, T=0, q=N, k=N, v=N, q_out=N) == OK
    assert attn(L, T=0, q=N, out=N) == OK


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(x=ODD)), (INVALID, dict(out=ODD)), (INVALID, dict(qkv=ODD)), (INVALID, dict(o=ODD)), (INVALID, dict(gu=ODD)),
    (INVALID, dict(down=ODD)), (INVALID, dict(kc=ODD)), (UNSUPPORTED, dict(pages=(1 << 26) + 1)),
    (INVALID, dict(ks=P, vs=P, k_scale=0.0)), (INVALID, dict(ks=P, vs=P, v_scale=float("inf"))),
    (INVALID, dict(ks=P, vs=P, k_scale=float("nan"))), (INVALID, dict(ks=P)), (WORKSPACE, dict(k_scale=0.0)),
    (UNSUPPORTED, dict(I=32832)), (WORKSPACE, dict(I=32768)),
])
def test_draft_prompt_refuses_before_its_first_launch(L, want, kw):
    """What one of its steps would refuse is refused at the entry: the cache is
    not half filled.  (A refusal behind the entry's checks would come after the
    workspace's.)"""
    a = dict(x=P, qkv=P, o=P, gu=P, down=P, kc=P, I=256, ks=N, vs=N, k_scale=1.0, v_scale=1.0, pages=8, out=ctypes.c_void_p(512))
    a.update(kw)
    assert L.eagle_draft_prompt(a["x"], P, a["qkv"], a["o"], P, a["gu"], a["down"], 1e-5, P, 8, P, P, a["kc"], P, a["ks"],
                                a["vs"], a["k_scale"], a["v_scale"], a["pages"], P, 4, a["out"], 2, 4, 256, 4, 2, 64, a["I"], 1,
                                N, 0, N, N) == want


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 1, 64), (7, 7, 64), (64, 1, 128), (12, 4, 128)])
def test_workspace_serves_fewer_requests_and_rows(L, Hq, Hkv, D):
    """Grows with B and with T, and slowly: the paths that only short calls take
    count at the rows that they take."""
    size = L.eagle_prompt_attn_workspace_size
    Bs, Ts = (1, 2, 3, 16, 64, 1000, 65535), (1, 2, 3, 4, 5, 16, 33, 64, 65, 200, 4096, 65536, 1 << 20, 1 << 28)
    table = [[size(B, T, Hq, Hkv, D) for T in Ts] for B in Bs]
    for x in range(len(Bs)):
        for y in range(len(Ts)):
            assert 0 < table[x][y] and (x == 0 or table[x - 1][y] <= table[x][y]) and (y == 0 or table[x][y - 1] <= table[x][y])
    g = Hq // Hkv
    # slots of 256 rows, a cut's description beside them, and 48 bytes a piece;
    # fp32 units hold 64 rows (64 / g tokens)
    most = 12 * 160 * 256 * (4 * D + 8 + 48) + 48 * Hkv * (2 * 65535 * 3 + (1 << 28) // (64 // g) + 160 * 12 * 6) + 4096
    assert table[-1][-1] <= most


@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_cache_scales_without_a_reciprocal(L, name):
    """1 / 2^-129 is no fp32 number: 0 times it would be NaN."""
    a = dict(k_scale=1.0, v_scale=1.0)
    a[name] = 2.0 ** -129
    assert L.eagle_kv_append_kv4(P, P, P, 512, 256, 256, P, 64, P, P, 2, 0, 4, 2, 128, ctypes.c_void_p(512), P, P, P, P,
                                 a["k_scale"], a["v_scale"], 8, P, 4, N, N) == INVALID
    assert L.eagle_draft_prompt(P, P, P, P, P, P, P, 1e-5, P, 8, P, P, P, P, P, P, a["k_scale"], a["v_scale"], 8, P, 4,
                                ctypes.c_void_p(512), 2, 4, 256, 4, 2, 64, 256, 1, N, 0, N, N) == INVALID
    a[name] = 2.0 ** -127
    assert L.eagle_kv_append_kv4(P, P, P, 512, 256, 256, P, 64, P, P, 2, 0, 4, 2, 128, ctypes.c_void_p(512), P, P, P, P,
                                 a["k_scale"], a["v_scale"], 8, P, 4, N, N) == OK
