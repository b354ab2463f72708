"""What the binding of the calls for a batch behind a shared prompt refuses before
it calls the library, on CPU tensors (no GPU needed): a call whose arrays agree
gets as far as the check that asks for a GPU; one changed array does not."""
import pytest
import torch

from eagle_speculative_decoding_gb300 import binding as eb
from test_binding_streams import FakeStream, allocations  # noqa: F401 (a fixture)
from test_prompt_binding import (B, CACHE, CODES, D, F32, HQ, I32, INDEX, OUT, ROPE, ROWS, T, W, attn_rows, lengths, pages4,
                                 pages16, rows, z)


def axes():
    return dict(positions=z(3, T, dtype=I32), pair_axis=z(D // 2, dtype=I32))


def groups():
    return dict(cu_rows=torch.tensor([0, 2, 5], dtype=I32), prefix_lens=z(B, dtype=I32), prefix_table=z(B, W, dtype=I32),
                status=z(1, dtype=I32), own_out=z(T, HQ, D), own_lse=z(T, HQ, dtype=F32))


CALLS = dict(
    prefix=(eb.eagle_prefix_attn, lambda: {**attn_rows(), **groups(), **pages16()}),
    prefix4=(eb.eagle_prefix_attn_kv4, lambda: {**attn_rows(), **groups(), **pages4()}),
    axes=(eb.eagle_kv_append_axes, lambda: {**rows(), **lengths(), **pages16(), **axes()}),
    axes4=(eb.eagle_kv_append_axes_kv4, lambda: {**rows(), **lengths(), **pages4(), **axes()}),
)
AXES = [dict(positions=z(3, T + 1, dtype=I32)), dict(positions=z(3, T, dtype=torch.long)), dict(positions=z(T, 3, dtype=I32).t()),
        dict(positions=z(3, 2 * T, dtype=I32)[:, ::2]), dict(pair_axis=z(D, dtype=I32)), dict(pair_axis=z(D // 2, dtype=torch.long)),
        dict(pair_axis=z(D, dtype=I32)[::2])]


OWN = [dict(own_out=None), dict(own_lse=None), dict(own_out=z(T, HQ, D, dtype=F32)), dict(own_out=z(T - 1, HQ, D)),
       dict(own_out=z(T, HQ, 2 * D)[..., :D]), dict(own_lse=z(T, HQ)), dict(own_lse=z(T, HQ + 1, dtype=F32)),
       dict(own_lse=z(HQ, T, dtype=F32).t())]


def on_gpu(monkeypatch):
    """Lets CPU tensors pass for the GPU's in the checks."""
    monkeypatch.setattr(eb, "_lengths", lambda rows, cu, ctx, table, status: table.shape)


def cases():
    names = dict(cu_seqlens="cu_rows", ctx_lens="prefix_lens", block_table="prefix_table")
    group = [{names.get(k, k): v for k, v in c.items()} for c in INDEX]
    both = {"prefix": group + CACHE + OUT + OWN, "prefix4": group + CODES + OUT + OWN, "axes": INDEX + CACHE + ROPE + ROWS, "axes4": INDEX + CODES + ROPE + ROWS}
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


@pytest.mark.parametrize("name", ["axes", "axes4"])
@pytest.mark.parametrize("change", AXES, ids=lambda c: "-".join(c))
def test_positions_that_do_not_agree_are_refused(name, change, monkeypatch):
    call, base = CALLS[name]
    on_gpu(monkeypatch)
    with pytest.raises(ValueError, match="positions must|pair_axis must"):
        call(**{**base(), **change})
    with pytest.raises(ValueError, match="on the GPU"):
        call(**base())


def sampling():
    return dict(logits=z(T, 50, dtype=F32), uniforms=z(T, dtype=F32), tokens=z(T, dtype=I32), temperature=z(3, dtype=F32),
                top_k=z(3, dtype=I32), top_p=z(3, dtype=F32), min_p=z(3, dtype=F32), rows_per_request=2, logprobs=z(T, dtype=F32),
                n_kept=z(T, dtype=I32), status=z(1, dtype=I32))


def truncating():
    kw = {k: v for k, v in sampling().items() if k not in ("uniforms", "tokens", "logprobs")}
    return {**kw, "out": z(T, 50, dtype=F32)}


SETTINGS = [dict(temperature=z(2, dtype=F32)), dict(temperature=z(3)), dict(top_k=z(3, dtype=torch.long)), dict(top_k=z(4, dtype=I32)),
            dict(top_p=z(6, dtype=F32)[::2]), dict(min_p=z(3, 1, dtype=F32)), dict(n_kept=z(T, dtype=torch.long)),
            dict(n_kept=z(3, dtype=I32)), dict(rows_per_request=1), dict(rows_per_request=0), dict(status=z(1, dtype=torch.long)),
            dict(logits=z(T, 100, dtype=F32)[:, ::2]), dict(logits=z(50, T, dtype=F32).t())]
SAMPLE = [dict(uniforms=z(T - 1, dtype=F32)), dict(uniforms=z(T)), dict(uniforms=None), dict(tokens=z(T, dtype=torch.long)),
          dict(tokens=None), dict(logprobs=z(T)), dict(logprobs=z(2 * T, dtype=F32)[::2])]
TRUNCATE = [dict(out=z(T, 49, dtype=F32)), dict(out=z(T, 50)), dict(out=z(T, 100, dtype=F32)[:, ::2])]


@pytest.mark.parametrize("call,base,change", [(eb.eagle_sample, sampling, c) for c in SETTINGS + SAMPLE]
                         + [(eb.eagle_truncate_logits, truncating, c) for c in SETTINGS + TRUNCATE],
                         ids=lambda x: "-".join(x) if isinstance(x, dict) else getattr(x, "__name__", ""))
def test_settings_that_do_not_agree_are_refused(call, base, change, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    with pytest.raises(ValueError):
        call(**{**base(), **change})


@pytest.mark.parametrize("call,base", [(eb.eagle_sample, sampling), (eb.eagle_truncate_logits, truncating)])
def test_sampling_asks_for_a_gpu(call, base):
    with pytest.raises(ValueError, match="on the GPU"):
        call(**base())
    some = {k: None if k in ("temperature", "top_k", "top_p", "min_p", "logprobs", "n_kept", "status") else v for k, v in base().items()}
    with pytest.raises(ValueError, match="on the GPU"):
        call(**some)


@pytest.mark.parametrize("name", ["prefix", "prefix4"])
def test_own_results_off_the_gpu_are_refused(name, monkeypatch):
    call, base = CALLS[name]
    on_gpu(monkeypatch)
    with pytest.raises(ValueError, match="on the GPU"):
        call(**base())


@pytest.mark.parametrize("name", ["prefix", "prefix4"])
@pytest.mark.parametrize("given", [False, True])
def test_scratch_of_a_prefix_is_the_streams(allocations, name, given):  # noqa: F811
    call, base = CALLS[name]
    alone = dict(base(), own_out=None, own_lse=None)
    s = FakeStream() if given else None
    call(**alone, stream=s)
    assert allocations == [(s, torch.uint8)]
    allocations.clear()
    call(**alone, stream=s, ws=torch.zeros(16, dtype=torch.uint8))
    assert allocations == []


def every_array():
    """(call, its arguments, the name of one array): the arrays that a kernel writes, and the host's usual slips."""
    named = {**CALLS, "sample": (eb.eagle_sample, sampling), "truncate": (eb.eagle_truncate_logits, truncating)}
    for name, (call, base) in named.items():
        for array, value in base().items():
            written = array in ("out", "lse", "status", "q_out", "k_cache", "v_cache", "k_codes", "k_scales", "v_codes", "v_scales")
            if isinstance(value, torch.Tensor) and (name in ("sample", "truncate") or (written and not (
                    name.startswith("prefix") and array.startswith(("k_", "v_"))))):
                yield pytest.param(call, base, array, id=f"{name}-{array}")


@pytest.mark.parametrize("call,base,array", list(every_array()))
def test_one_array_off_the_gpu_is_refused(call, base, array, monkeypatch):
    """Before the library is called: the others pass for the GPU's."""
    args, called = base(), []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(eb, "_lib", Lib())
    monkeypatch.setattr(eb, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(eb, "workspace", lambda *a: torch.zeros(16, dtype=torch.uint8))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: t is not args[array]))
    with pytest.raises(ValueError, match="on the GPU"):
        call(**args)
    assert not called
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    call(**args)
    assert called
