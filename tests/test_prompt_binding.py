"""What the binding of the prompt path refuses before it calls the library, on
CPU tensors (no GPU needed): a call whose arrays agree gets as far as the last
check, which asks for a GPU; one changed array does not."""
import pytest
import torch

from eagle_speculative_decoding_gb300 import binding as eb

I32, BF16, F32, U8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
B, T, HQ, HKV, D, P, W = 2, 5, 4, 2, 128, 6, 3


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def lengths():
    return dict(cu_seqlens=torch.tensor([0, 2, 5], dtype=I32), ctx_lens=z(B, dtype=I32), block_table=z(B, W, dtype=I32),
                status=z(1, dtype=I32))


def pages4():
    return dict(k_codes=z(P, HKV, 16, D // 2, dtype=U8), k_scales=z(P, HKV, 16, D // 16, dtype=U8),
                v_codes=z(P, HKV, 16, D // 2, dtype=U8), v_scales=z(P, HKV, 16, D // 16, dtype=U8))


def pages16():
    return dict(k_cache=z(P, 16, HKV, D), v_cache=z(P, 16, HKV, D))


def rows():
    qkv = z(T, HQ + 2 * HKV, D)
    return dict(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:], rope=z(64, 2, D // 2, dtype=F32), q_out=z(T, HQ, D))


def attn_rows():
    return dict(q=z(T, HQ, D), out=z(T, HQ, D), lse=z(T, HQ, dtype=F32))


def layer():
    d, I = 256, 128
    W_ = dict(norm1=z(d), qkv=z((HQ + 2 * HKV) * D, d), o=z(d, HQ * D), norm2=z(d), gu=z(2 * I, d), down=z(d, I))
    return dict(x=z(T, d), weights=W_, rope=z(64, 2, D // 2, dtype=F32), out=z(T, d))


CALLS = dict(
    append=(eb.eagle_kv_append, lambda: {**rows(), **lengths(), **pages16()}),
    append4=(eb.eagle_kv_append_kv4, lambda: {**rows(), **lengths(), **pages4()}),
    attn=(eb.eagle_prompt_attn, lambda: {**attn_rows(), **lengths(), **pages16()}),
    attn4=(eb.eagle_prompt_attn_kv4, lambda: {**attn_rows(), **lengths(), **pages4()}),
    draft=(eb.eagle_draft_prompt, lambda: {**layer(), **lengths(), **pages16()}),
    draft4=(eb.eagle_draft_prompt, lambda: {**layer(), **lengths(), **{k.replace("codes", "cache"): v for k, v in pages4().items()}}),
    read=(eb.eagle_kv4_read, lambda: dict(codes=z(P, HKV, 16, D // 2, dtype=U8), scales=z(P, HKV, 16, D // 16, dtype=U8),
                                          out=z(P, 16, HKV, D))),
)

INDEX = [dict(cu_seqlens=torch.tensor([0, 2, 5])), dict(ctx_lens=torch.zeros(B, dtype=torch.long)),
         dict(block_table=torch.zeros(B, W, dtype=torch.long)), dict(block_table=z(B, 2 * W, dtype=I32)[:, ::2]),
         dict(block_table=z(W, B, dtype=I32).t()), dict(block_table=z(B + 1, W, dtype=I32)), dict(cu_seqlens=z(B, dtype=I32)),
         dict(cu_seqlens=z(B + 2, dtype=I32)), dict(ctx_lens=z(B + 1, dtype=I32)), dict(ctx_lens=z(2 * B, dtype=I32)[::2]),
         dict(status=z(1, dtype=torch.long))]
CACHE = [dict(v_cache=z(P - 1, 16, HKV, D)), dict(k_cache=z(P, 16, HKV, D // 2), v_cache=z(P, 16, HKV, D // 2)),
         dict(k_cache=z(P, 32, HKV, D), v_cache=z(P, 32, HKV, D)), dict(v_cache=z(P, 16, HKV, D, dtype=F32)),
         dict(k_cache=z(P, 16, HKV, D, dtype=F32), v_cache=z(P, 16, HKV, D, dtype=F32)),
         dict(k_cache=z(P, 2, 16, HKV, D)[:, 0], v_cache=z(P, 2, 16, HKV, D)[:, 1]), dict(k_cache=z(P, 16, HKV, 2 * D)[..., :D]),
         dict(v_cache=z(P, HKV, 16, D).transpose(1, 2))]
OTHER_HEADS = [dict(k_cache=z(P, 16, 1, D), v_cache=z(P, 16, 1, D))]
CODES = [dict(v_codes=z(P - 1, HKV, 16, D // 2, dtype=U8)), dict(v_scales=z(P - 1, HKV, 16, D // 16, dtype=U8)),
         dict(k_scales=z(P, HKV, 16, D // 32, dtype=U8)), dict(k_scales=z(P, HKV, 16, D // 16, dtype=F32)),
         dict(k_codes=z(P, HKV, 16, D // 2, dtype=torch.int8)), dict(k_codes=z(P, 16, HKV, D // 2, dtype=U8).transpose(1, 2)),
         dict(v_codes=z(P, 2, HKV, 16, D // 2, dtype=U8)[:, 0]), dict(v_scales=z(P, HKV, 16, D // 8, dtype=U8)[..., ::2]),
         dict(v_codes=z(P, HKV, 32, D // 2, dtype=U8), v_scales=z(P, HKV, 32, D // 16, dtype=U8)),
         dict(v_codes=z(P + 1, HKV, 16, D // 2, dtype=U8), v_scales=z(P + 1, HKV, 16, D // 16, dtype=U8))]
ROPE = [dict(rope=z(64, 2, D // 4, dtype=F32)), dict(rope=z(64, 2, D // 2, dtype=torch.float64)),
        dict(rope=z(64, D // 2, 2, dtype=F32).transpose(1, 2)), dict(rope=z(128, 2, D // 2, dtype=F32)[::2])]
ROWS = [dict(v=z(T, HKV, D, dtype=F32)), dict(v=z(T, HKV, D // 2)), dict(q=z(T + 1, HQ, D)), dict(q=z(T, HQ, D // 2)),
        dict(q=z(T, HQ, D, dtype=F32)), dict(q_out=None), dict(q_out=z(T, HQ + 1, D)), dict(q_out=z(T, HQ, D, dtype=F32)),
        dict(q_out=z(T, HQ, 2 * D)[..., :D]), dict(q=None), dict(k=z(T, HKV, 2 * D)[..., ::2])]
OUT = [dict(out=z(T, HQ, D // 2)), dict(out=z(T - 1, HQ, D)), dict(out=z(T, HQ, D, dtype=F32)), dict(out=z(T, HQ, 2 * D)[..., :D]),
       dict(lse=z(T, HQ + 1, dtype=F32)), dict(lse=z(T, HQ)), dict(lse=z(HQ, T, dtype=F32).t()),
       dict(q=z(T, HQ, 2 * D)[..., ::2])]
LAYER = [dict(x=z(T, 512)[:, ::2]), dict(out=z(T - 1, 256)), dict(out=z(T, 256, dtype=F32)), dict(out=z(T, 512)[:, ::2])]
WEIGHTS = [dict(norm1=z(255)), dict(qkv=z((HQ + 2 * HKV) * D, 128)), dict(o=z(256, HQ * D, dtype=F32)), dict(norm2=z(512)[::2]),
           dict(gu=z(128, 256)), dict(down=z(128, 256).t()), dict(qkv=z((HQ + 2 * HKV) * D + 64, 256))]


def cases():
    both = {"append": INDEX + CACHE + OTHER_HEADS + ROPE + ROWS, "append4": INDEX + CODES + ROPE + ROWS,
            "attn": INDEX + CACHE + OUT, "attn4": INDEX + CODES + OUT, "draft": INDEX + CACHE + OTHER_HEADS + ROPE + LAYER,
            "draft4": INDEX + [{k.replace("codes", "cache"): v for k, v in c.items()} for c in CODES] + ROPE + LAYER
            + [dict(k_scales=None)],
            "read": [dict(out=z(P, 16, HKV, D // 2)), dict(out=z(P + 1, 16, HKV, D)), dict(out=z(P, HKV, 16, D).transpose(1, 2)),
                     dict(scales=z(P - 1, HKV, 16, D // 16, dtype=U8)), dict(scales=z(P, HKV, 16, D // 8, dtype=U8)[..., ::2])]}
    return [(name, i, change) for name, changes in both.items() for i, change in enumerate(changes)]


@pytest.mark.parametrize("name", CALLS)
def test_arrays_that_agree_pass_every_check_but_the_last(name):
    call, base = CALLS[name]
    with pytest.raises(ValueError, match="on the GPU"):
        call(**base())


@pytest.mark.parametrize("name,i,change", cases(), ids=lambda x: "-".join(x) if isinstance(x, dict) else str(x))
def test_arrays_that_do_not_are_refused(name, i, change):
    call, base = CALLS[name]
    with pytest.raises(ValueError) as e:
        call(**{**base(), **change})
    assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("name", ["draft", "draft4"])
@pytest.mark.parametrize("change", WEIGHTS, ids=lambda c: "-".join(c))
def test_weights_that_do_not_agree_are_refused(name, change):
    call, base = CALLS[name]
    kw = base()
    kw["weights"] = {**kw["weights"], **change}
    with pytest.raises(ValueError, match="weights"):
        call(**kw)


def test_optional_arrays_may_be_left_out():
    for name, gone in (("append", ("q", "q_out", "rope", "status")), ("append4", ("q", "q_out", "rope")), ("attn", ("lse", "status")),
                       ("attn4", ("lse",))):
        call, base = CALLS[name]
        kw = {k: None if k in gone else v for k, v in base().items()}
        with pytest.raises(ValueError, match="on the GPU"):
            call(**kw)


def test_scales_may_be_e4m3_tensors():
    call, base = CALLS["attn4"]
    kw = {k: v.view(torch.float8_e4m3fn) if k.endswith("scales") else v for k, v in base().items()}
    with pytest.raises(ValueError, match="on the GPU"):
        call(**kw)


def test_rope_table_given():
    with pytest.raises(ValueError, match="on the GPU"):
        eb.eagle_rope_table(8, D, 1e4, table=z(8, 2, D // 2, dtype=F32))
    for bad in (z(7, 2, D // 2, dtype=F32), z(8, 2, D, dtype=F32), z(8, 2, D // 2, dtype=torch.float64)):
        with pytest.raises(ValueError, match="max_pos"):
            eb.eagle_rope_table(8, D, 1e4, table=bad)


def test_a_single_row_may_have_any_stride():
    """A row's stride that no second row uses is not held against it."""
    one = z(HQ, 1, D).transpose(0, 1)
    assert one.stride(0) < HQ * D and eb._row_stride("q", one, D) == HQ * D
    assert eb._row_stride("q", z(1, D).expand(1, HQ, D)[:, :1], D) == D
    assert eb._row_stride("q", torch.as_strided(z(4000), (1, HQ, D), (4001, D, 1)), D) == HQ * D
    assert eb._row_stride("q", z(4, 6, D)[:, :HQ], D) == 6 * D
    assert eb._row_stride("q", z(HQ, D).expand(3, HQ, D), D) == 0  # for the library to refuse
