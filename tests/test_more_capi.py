"""Refusals of the calls for a batch behind a shared prompt, on the host: every
case returns before any CUDA call (no GPU needed)."""
import ctypes
import os

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
N, P, ODD = None, ctypes.c_void_p(256), ctypes.c_void_p(8)


@pytest.fixture(scope="module")
def L():
    from eagle_speculative_decoding_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def append(L, **kw):
    a = dict(q=P, k=P, v=P, qs=512, ks=256, vs=256, rope=P, max_pos=64, pos=P, axes=3, axis=P, cu=P, ctx=P, B=2, T=4, Hq=4,
             Hkv=2, D=128, dtype=1, q_out=ctypes.c_void_p(512), kc=P, vc=P, pages=8, table=P, width=4)
    a.update(kw)
    return L.eagle_kv_append_axes(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["rope"], a["max_pos"], a["pos"],
                                  a["axes"], a["axis"], a["cu"], a["ctx"], a["B"], a["T"], a["Hq"], a["Hkv"], a["D"],
                                  a["dtype"], a["q_out"], a["kc"], a["vc"], a["pages"], a["table"], a["width"], N, N)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(T=0, q=N, k=N, v=N, q_out=N, pos=N)), (OK, dict(T=0, axis=N, axes=1)),
    (INVALID, dict(rope=N)), (INVALID, dict(pos=N)), (INVALID, dict(axes=0)), (INVALID, dict(axes=-1)),
    (UNSUPPORTED, dict(axes=9)), (INVALID, dict(max_pos=0)), (INVALID, dict(k=N)), (INVALID, dict(vc=N)), (INVALID, dict(cu=N)),
    (INVALID, dict(ctx=N)), (INVALID, dict(table=N)), (INVALID, dict(q_out=N)), (INVALID, dict(dtype=2)), (INVALID, dict(T=-1)),
    (UNSUPPORTED, dict(D=96)), (INVALID, dict(qs=511)), (INVALID, dict(rope=ODD)), (INVALID, dict(kc=ODD)),
    (INVALID, dict(q_out=P, qs=1024)), (UNSUPPORTED, dict(pages=(1 << 26) + 1)),
])
def test_append_axes_refusals(L, want, kw):
    assert append(L, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (INVALID, dict(ks=N)), (INVALID, dict(k_scale=0.0)), (INVALID, dict(v_scale=2.0 ** -129)),
    (INVALID, dict(rope=N)), (INVALID, dict(pos=N)), (INVALID, dict(axes=0)), (UNSUPPORTED, dict(axes=9)),
    (UNSUPPORTED, dict(D=32)),
])
def test_append_axes_kv4_refusals(L, want, kw):
    a = dict(T=4, D=128, ks=P, rope=P, pos=P, axes=3, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    assert L.eagle_kv_append_axes_kv4(P, P, P, 512, 256, 256, a["rope"], 64, a["pos"], a["axes"], P, P, P, 2, a["T"], 4, 2,
                                      a["D"], ctypes.c_void_p(512), P, a["ks"], P, P, a["k_scale"], a["v_scale"], 8, P, 4, N,
                                      N) == want


def sample(L, **kw):
    a = dict(x=P, stride=100, M=4, V=100, dtype=1, per=1, u=P, tok=P)
    a.update(kw)
    return L.eagle_sample(a["x"], a["stride"], a["M"], a["V"], a["dtype"], N, N, N, N, a["per"], a["u"], a["tok"], N, N, N, N)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (OK, dict(M=0, x=N, u=N, tok=N)), (INVALID, dict(x=N)), (INVALID, dict(u=N)), (INVALID, dict(tok=N)),
    (INVALID, dict(M=-1)), (INVALID, dict(V=0)), (INVALID, dict(per=0)), (INVALID, dict(stride=99)), (INVALID, dict(dtype=2)),
    (INVALID, dict(x=ctypes.c_void_p(257))), (INVALID, dict(x=ctypes.c_void_p(258), dtype=0)), (UNSUPPORTED, dict(M=65536)),
    (UNSUPPORTED, dict(V=262145, stride=262145)),
])
def test_sample_refusals(L, want, kw):
    assert sample(L, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (INVALID, dict(x=N)), (INVALID, dict(out=N)), (INVALID, dict(out_stride=99)), (INVALID, dict(out=P, out_stride=120)),
    (INVALID, dict(out=ctypes.c_void_p(513))), (INVALID, dict(V=0)), (INVALID, dict(per=-1)), (UNSUPPORTED, dict(M=65536)),
])
def test_truncate_refusals(L, want, kw):
    a = dict(x=P, M=4, V=100, per=1, out=ctypes.c_void_p(512), out_stride=100)
    a.update(kw)
    assert L.eagle_truncate_logits(a["x"], 100, a["M"], a["V"], 1, N, N, N, N, a["per"], a["out"], a["out_stride"], N, N, N) == want


def prefix(L, **kw):
    a = dict(q=P, qs=512, kc=P, vc=P, pages=8, table=P, width=4, cu=P, lens=P, own=P, own_lse=P, out=P, G=2, T=4, Hq=4, Hkv=2,
             D=128, page=16, scale=0.1, dtype=1, ws=N, wsb=0)
    a.update(kw)
    return L.eagle_prefix_attn(a["q"], a["qs"], a["kc"], a["vc"], a["pages"], a["table"], a["width"], a["cu"], a["lens"],
                               a["own"], a["own_lse"], a["out"], N, a["G"], a["T"], a["Hq"], a["Hkv"], a["D"], a["page"],
                               a["scale"], a["dtype"], a["ws"], a["wsb"], N, N)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(T=0, q=N, out=N, own=N, own_lse=N)), (WORKSPACE, dict()), (WORKSPACE, dict(ws=P, wsb=16)),
    (WORKSPACE, dict(own=N, own_lse=N)), (INVALID, dict(own=N)), (INVALID, dict(own_lse=N)), (INVALID, dict(own=ODD)),
    (INVALID, dict(q=N)), (INVALID, dict(kc=N)), (INVALID, dict(vc=N)), (INVALID, dict(table=N)), (INVALID, dict(cu=N)),
    (INVALID, dict(lens=N)), (INVALID, dict(out=N)), (INVALID, dict(G=0)), (INVALID, dict(T=-1)), (INVALID, dict(Hq=5)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(dtype=7)), (INVALID, dict(qs=500)),
    (INVALID, dict(qs=516)), (INVALID, dict(q=ODD)), (INVALID, dict(out=ODD)), (UNSUPPORTED, dict(D=96)),
    (UNSUPPORTED, dict(page=32)), (UNSUPPORTED, dict(Hq=130, qs=130 * 128)), (UNSUPPORTED, dict(G=1025)),
    (UNSUPPORTED, dict(pages=(1 << 26) + 1)),
])
def test_prefix_refusals(L, want, kw):
    assert prefix(L, **kw) == want


@pytest.mark.parametrize("want,ks,k_scale,own", [
    (INVALID, N, 1.0, P), (INVALID, P, -1.0, P), (INVALID, P, float("nan"), P), (INVALID, P, 1.0, N), (WORKSPACE, P, 1.0, P)])
def test_prefix_kv4_refusals(L, want, ks, k_scale, own):
    assert L.eagle_prefix_attn_kv4(P, 512, P, ks, P, P, k_scale, 1.0, 8, P, 4, P, P, own, P, P, N, 2, 4, 4, 2, 128, 16, 0.1, N,
                                   0, N, N) == want


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 1, 64), (7, 7, 64), (64, 1, 128), (12, 4, 128)])
def test_prefix_workspace_serves_fewer_groups_and_rows(L, Hq, Hkv, D):
    size = L.eagle_prefix_attn_workspace_size
    Gs, Ts = (1, 2, 3, 64, 1024), (0, 1, 2, 5, 16, 33, 64, 200, 4096, 1 << 28)
    table = [[size(G, T, Hq, Hkv, D) for T in Ts] for G in Gs]
    for x in range(len(Gs)):
        for y in range(len(Ts)):
            assert 0 < table[x][y] and (x == 0 or table[x - 1][y] <= table[x][y]) and (y == 0 or table[x][y - 1] <= table[x][y])
    assert table[-1][-1] <= 2 * 160 * 256 * (4 * D + 8) + 4096
    for bad in ((0, 4, 4, 2, 64), (1025, 4, 4, 2, 64), (1, 4, 5, 2, 64), (1, 4, 4, 2, 80), (1, -1, 4, 2, 64)):
        assert size(*bad) == 0
