"""Thin ctypes binding of libeagle_gb300.so (include/eagle.h).

Argument marshalling only: every function takes torch tensors that already
live on the current CUDA device, passes their data pointers, shapes and the
current stream to the C entry point of the same name, and raises if the call
returns an error.  No computation happens here and there is no fallback: if
the library is missing, the first call raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libeagle_gb300.so")

EAGLE_FP32, EAGLE_BF16 = 0, 1
EAGLE_PROPOSAL_DETERMINISTIC, EAGLE_PROPOSAL_SAMPLED = 0, 1
STATUS = {0: "EAGLE_OK", 1: "EAGLE_ERR_INVALID_ARG", 2: "EAGLE_ERR_UNSUPPORTED",
          3: "EAGLE_ERR_WORKSPACE", 4: "EAGLE_ERR_CUDA", 5: "EAGLE_ERR_BAD_TREE",
          6: "EAGLE_ERR_BAD_KV", 7: "EAGLE_ERR_NONFINITE", 8: "EAGLE_ERR_TIMEOUT"}

_P, _I, _F, _Z, _U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64
_L, _D = ctypes.c_longlong, ctypes.c_double

_SIGS = {
    "eagle_status_string": (ctypes.c_char_p, [_I]),
    "eagle_read_status": (_I, [_P, _P, _P]),
    "eagle_launch_count": (_U64, []),
    "eagle_selftest_wait_timeout": (_I, [ctypes.c_uint, _P, _P]),
    "eagle_fuse_proj_workspace_size": (_Z, [_I, _I, _I]),
    "eagle_fuse_proj": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _Z, _P, _P]),
    "eagle_fuse_proj_accepted_workspace_size": (_Z, [_I, _I, _I, _I]),
    "eagle_fuse_proj_accepted": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P, _P]),
    "eagle_draft_input_workspace_size": (_Z, [_I, _I, _I]),
    "eagle_linear_workspace_size": (_Z, [_I, _I, _I, _I]),
    "eagle_linear": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P, _P]),
    "eagle_draft_layer_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "eagle_draft_rows": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                              _P, _P]),
    "eagle_draft_layer": (_I, [_P, _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P,
                               _P, _I, _I, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _Z, _P, _P]),
    "eagle_draft_input": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _P, _Z, _P, _P]),
    "eagle_tree_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "eagle_tree_attn": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                             _I, _F, _I, _I, _P, _Z, _P, _P]),
    "eagle_lmhead_topk_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "eagle_lmhead_topk": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P, _I, _P, _Z, _P, _P]),
    "eagle_lmhead_topk_partial": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _Z, _P, _P]),
    "eagle_lmhead_topk_merge": (_I, [_I, _I, _I, _I, _F, _P, _P, _P, _P, _I, _P, _Z, _P, _P]),
    "eagle_tree_expand": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "eagle_tree_expand_lmhead": (_I, [_I, _I, _I, _I, _I, _P, _Z, _I, _I, _F, _I, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P, _P]),
    "eagle_tree_expand_static": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P]),
    "eagle_tree_expand_finalize": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _P, _P, _P, _P]),
    "eagle_tree_verify_workspace_size": (_Z, [_I, _I, _I]),
    "eagle_tree_verify": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _F, _I, _U64, _U64, _P, _I, _P,
                               _P, _P, _P, _Z, _P, _P]),
    "eagle_tree_verify_noalloc": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _F, _I, _U64, _U64, _P,
                                       _I, _P, _P, _P, _P, _P]),
    "eagle_lmhead_verify_stats": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _F, _U64, _U64, _I,
                                       _P, _P, _P, _P, _P, _I, _P, _Z, _P, _P]),
    "eagle_tree_commit": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P,
                               _I, _P, _P, _P]),
    "eagle_tree_verify_stats": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _I, _F, _U64, _U64,
                                     _P, _I, _P, _P, _P, _P, _P]),
    "eagle_rope_table": (_I, [_I, _I, _D, _P, _P]),
    "eagle_kv_append": (_I, [_P, _P, _P, _L, _L, _L, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I, _P,
                             _I, _P, _P]),
    "eagle_kv_append_kv4": (_I, [_P, _P, _P, _L, _L, _L, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                                 _F, _F, _I, _P, _I, _P, _P]),
    "eagle_kv4_read": (_I, [_P, _P, _F, _I, _I, _I, _I, _P, _P]),
    "eagle_prompt_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "eagle_prompt_attn": (_I, [_P, _L, _P, _P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _Z,
                               _P, _P]),
    "eagle_prompt_attn_kv4": (_I, [_P, _L, _P, _P, _P, _P, _F, _F, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                   _I, _F, _P, _Z, _P, _P]),
    "eagle_draft_prompt_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "eagle_draft_prompt": (_I, [_P, _P, _P, _P, _P, _P, _P, _F, _P, _I, _P, _P, _P, _P, _P, _P, _F, _F, _I, _P, _I, _P,
                                _I, _I, _I, _I, _I, _I, _I, _I, _P, _Z, _P, _P]),
}

_lib = None


class EagleError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


def lib():
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return EAGLE_BF16
    if t.dtype == torch.float32:
        return EAGLE_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(fn, code):
    if code != 0:
        raise EagleError(fn, code)


def workspace(nbytes, device=None, stream=None):
    """A caller-owned device buffer of at least ``nbytes`` (torch allocation).
    It belongs to ``stream`` if that is given, else to the current stream: the
    memory is another allocation's again only behind what that stream has been
    given until the buffer is released."""
    return _empty((max(int(nbytes), 256),), torch.uint8, device if device is not None else "cuda", stream)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def launch_count():
    return int(lib().eagle_launch_count())


def eagle_selftest_wait_timeout(limit_us, status, stream=None):
    """Bounded-wait self-test: expects status[0] = EAGLE_ERR_TIMEOUT and
    status[1] = 1 once the stream has run it."""
    _check("eagle_selftest_wait_timeout",
           lib().eagle_selftest_wait_timeout(int(limit_us), _ptr(status), _stream(stream)))


def read_status(status, stream=None):
    host = ctypes.c_int32(0)
    lib().eagle_read_status(_ptr(status), _stream(stream), ctypes.byref(host))
    return int(host.value)


# ------------------------------------------------------------------ a1
def eagle_fuse_proj_workspace_size(M, d, dtype):
    return int(lib().eagle_fuse_proj_workspace_size(M, d, dtype))


def eagle_fuse_proj(h_low, h_mid, h_high, w_proj, g, bias=None, ws=None, status=None, stream=None):
    M, d = h_low.shape
    dt = _dtype(h_low)
    if ws is None:
        ws = workspace(eagle_fuse_proj_workspace_size(M, d, dt), h_low.device, stream)
    _check("eagle_fuse_proj", lib().eagle_fuse_proj(
        _ptr(h_low), _ptr(h_mid), _ptr(h_high), _ptr(w_proj), _ptr(bias), _ptr(g), M, d, dt,
        _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return g


def eagle_fuse_proj_accepted_workspace_size(B, max_depth, d, dtype):
    return int(lib().eagle_fuse_proj_accepted_workspace_size(B, max_depth, d, dtype))


def eagle_fuse_proj_accepted(h_low, h_mid, h_high, w_proj, path_rows, accept_len, g, bias=None, ws=None,
                             status=None, stream=None):
    """g[b, j] = W_proj [h_low; h_mid; h_high] of row path_rows[b, j] (rows
    b*R + row of the [B*R, d] features) for j <= accept_len[b], zero past it;
    g is [B, max_depth+1, d]."""
    B, slots = path_rows.shape
    d = h_low.shape[1]
    R = h_low.shape[0] // B
    dt = _dtype(h_low)
    if ws is None:
        ws = workspace(eagle_fuse_proj_accepted_workspace_size(B, slots - 1, d, dt), h_low.device, stream)
    _check("eagle_fuse_proj_accepted", lib().eagle_fuse_proj_accepted(
        _ptr(h_low), _ptr(h_mid), _ptr(h_high), _ptr(w_proj), _ptr(bias), _ptr(path_rows), _ptr(accept_len),
        B, R, slots - 1, d, dt, _ptr(g), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return g


def eagle_draft_input_workspace_size(M, d, dtype):
    return int(lib().eagle_draft_input_workspace_size(M, d, dtype))


def eagle_draft_input(r, token_ids, embed, w_in, u, bias=None, ws=None, status=None, stream=None):
    """u = W_I [r; embed[token_ids]] (+ bias); token_ids int32 [M] on the device."""
    M, d = r.shape
    dt = _dtype(r)
    if ws is None:
        ws = workspace(eagle_draft_input_workspace_size(M, d, dt), r.device, stream)
    _check("eagle_draft_input", lib().eagle_draft_input(
        _ptr(r), _ptr(token_ids), _ptr(embed), embed.shape[0], _ptr(w_in), _ptr(bias), _ptr(u), M, d,
        dt, _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return u


def eagle_linear_workspace_size(M, n_out, k_in, dtype):
    return int(lib().eagle_linear_workspace_size(M, n_out, k_in, dtype))


def eagle_linear(x, w, y, bias=None, residual=None, ws=None, status=None, stream=None):
    """y = x w^T (+ bias) (+ residual)."""
    M, k_in = x.shape
    n_out = w.shape[0]
    dt = _dtype(x)
    if ws is None:
        ws = workspace(eagle_linear_workspace_size(M, n_out, k_in, dt), x.device, stream)
    _check("eagle_linear", lib().eagle_linear(
        _ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), M, n_out, k_in, dt, _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))
    return y


def eagle_draft_layer_workspace_size(B, W, d, Hq, Hkv, D, I, Rmax, max_pages, dtype):
    return int(lib().eagle_draft_layer_workspace_size(B, W, d, Hq, Hkv, D, I, Rmax, max_pages, dtype))


def eagle_draft_layer(x, weights, positions, k_cache, v_cache, block_table, ctx_lens, q_tree, k_tree,
                      v_tree, tree_mask, r0, out, eps=1e-5, theta=500000.0, ws=None, status=None,
                      stream=None):
    """The drafter's decoder layer over the B x W new nodes of one depth.
    weights: dict norm1, qkv, o, norm2, gu, down (see include/eagle.h)."""
    B, W = positions.shape
    d = x.shape[1]
    Rmax, Hq, D = q_tree.shape[1], q_tree.shape[2], q_tree.shape[3]
    Hkv = k_tree.shape[2]
    I = weights["down"].shape[1]
    dt = _dtype(x)
    if ws is None:
        ws = workspace(eagle_draft_layer_workspace_size(B, W, d, Hq, Hkv, D, I, Rmax, block_table.shape[1], dt),
                       x.device, stream)
    _check("eagle_draft_layer", lib().eagle_draft_layer(
        _ptr(x), _ptr(weights["norm1"]), _ptr(weights["qkv"]), _ptr(weights["o"]), _ptr(weights["norm2"]),
        _ptr(weights["gu"]), _ptr(weights["down"]), eps, theta, _ptr(positions), _ptr(k_cache),
        _ptr(v_cache), k_cache.shape[0], _ptr(block_table), block_table.shape[1], _ptr(ctx_lens),
        _ptr(q_tree), _ptr(k_tree), _ptr(v_tree), _ptr(tree_mask), r0, Rmax, _ptr(out), B, W, d, Hq, Hkv, D,
        I, dt, _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return out


def eagle_draft_rows(step, width, ctx_lens, node_row, row_mask, prev, r_in, tokens, positions, root_token=None,
                     frontier=None, n_frontier=None, node_parent=None, node_token=None, node_depth=None,
                     status=None, stream=None):
    """Bookkeeping of one drafter pass (see include/eagle.h)."""
    B, max_nodes = node_row.shape
    Rmax = row_mask.shape[1]
    d = prev.shape[-1]
    _check("eagle_draft_rows", lib().eagle_draft_rows(
        B, step, width, Rmax, max_nodes, d, _dtype(prev), _ptr(root_token), _ptr(frontier), _ptr(n_frontier),
        _ptr(node_parent), _ptr(node_token), _ptr(node_depth), _ptr(ctx_lens), _ptr(node_row), _ptr(row_mask),
        _ptr(prev), _ptr(r_in), _ptr(tokens), _ptr(positions), _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ a2
def eagle_tree_attn_workspace_size(B, R, Hq, Hkv, D, max_pages, page_size=16, num_splits=0,
                                   dtype=EAGLE_BF16):
    return int(lib().eagle_tree_attn_workspace_size(B, R, Hq, Hkv, D, max_pages, page_size,
                                                    num_splits, dtype))


def eagle_tree_attn(q, k_tree, v_tree, k_cache, v_cache, block_table, ctx_lens, tree_mask, out,
                    lse=None, scale=None, num_splits=0, ws=None, status=None, stream=None):
    B, R, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    P, page = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    dt = _dtype(q)
    if scale is None:
        scale = D ** -0.5
    if ws is None:
        ws = workspace(eagle_tree_attn_workspace_size(B, R, Hq, Hkv, D, max_pages, page, num_splits,
                                                      dt), q.device, stream)
    _check("eagle_tree_attn", lib().eagle_tree_attn(
        _ptr(q), _ptr(k_tree), _ptr(v_tree), _ptr(k_cache), _ptr(v_cache), P, _ptr(block_table),
        max_pages, _ptr(ctx_lens), _ptr(tree_mask), _ptr(out), _ptr(lse), B, R, Hq, Hkv, D, page,
        float(scale), num_splits, dt, _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return out


# ------------------------------------------------------------------ a3
def eagle_lmhead_topk_workspace_size(M, d, V, k, dtype):
    return int(lib().eagle_lmhead_topk_workspace_size(M, d, V, k, dtype))


def eagle_lmhead_topk(x, w_lm, k, topk_ids, topk_logprobs, temperature=1.0, bias=None,
                      row_max=None, row_sumexp=None, ws=None, status=None, stream=None):
    M, d = x.shape
    V = w_lm.shape[0]
    dt = _dtype(x)
    if ws is None:
        ws = workspace(eagle_lmhead_topk_workspace_size(M, d, V, k, dt), x.device, stream)
    _check("eagle_lmhead_topk", lib().eagle_lmhead_topk(
        _ptr(x), _ptr(w_lm), _ptr(bias), M, d, V, k, float(temperature), _ptr(topk_ids),
        _ptr(topk_logprobs), _ptr(row_max), _ptr(row_sumexp), dt, _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))
    return topk_ids, topk_logprobs


def eagle_lmhead_topk_partial(x, w_lm, k, ws, temperature=1.0, bias=None, status=None, stream=None):
    """First half of eagle_lmhead_topk: the GEMM, partials left in ws."""
    M, d = x.shape
    V = w_lm.shape[0]
    _check("eagle_lmhead_topk_partial", lib().eagle_lmhead_topk_partial(
        _ptr(x), _ptr(w_lm), _ptr(bias), M, d, V, k, float(temperature), _dtype(x), _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))


def eagle_lmhead_topk_merge(M, d, V, topk_ids, topk_logprobs, ws, dtype=EAGLE_BF16, temperature=1.0,
                            row_max=None, row_sumexp=None, status=None, stream=None):
    """Second half of eagle_lmhead_topk: merge the partials a partial call left in ws."""
    k = topk_ids.shape[-1]
    _check("eagle_lmhead_topk_merge", lib().eagle_lmhead_topk_merge(
        M, d, V, k, float(temperature), _ptr(topk_ids), _ptr(topk_logprobs), _ptr(row_max), _ptr(row_sumexp),
        dtype, _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ a4 / a5
def eagle_tree_expand(step, width, cand_ids, cand_logprobs, root_token, node_parent, node_token,
                      node_logv, node_depth, node_count, frontier, n_frontier, status=None,
                      stream=None):
    B, max_nodes = node_parent.shape
    k = cand_ids.shape[-1]
    _check("eagle_tree_expand", lib().eagle_tree_expand(
        B, step, width, k, max_nodes, _ptr(cand_ids), _ptr(cand_logprobs), _ptr(root_token),
        _ptr(node_parent), _ptr(node_token), _ptr(node_logv), _ptr(node_depth), _ptr(node_count),
        _ptr(frontier), _ptr(n_frontier), _ptr(status), _stream(stream)))


def eagle_tree_expand_lmhead(step, width, k, lm_ws, d, V, root_token, node_parent, node_token, node_logv,
                             node_depth, node_count, frontier, n_frontier, temperature=1.0, dtype=None,
                             status=None, stream=None):
    """One expansion step whose candidate lists are merged from the partials
    that eagle_lmhead_topk_partial left in lm_ws (B * P rows, P = 1 at step 0,
    else width)."""
    B, max_nodes = node_parent.shape
    if dtype is None:
        dtype = EAGLE_BF16
    _check("eagle_tree_expand_lmhead", lib().eagle_tree_expand_lmhead(
        B, step, width, k, max_nodes, _ptr(lm_ws), lm_ws.numel(), d, V, float(temperature), dtype,
        _ptr(root_token), _ptr(node_parent), _ptr(node_token), _ptr(node_logv), _ptr(node_depth),
        _ptr(node_count), _ptr(frontier), _ptr(n_frontier), _ptr(status), _stream(stream)))


def eagle_tree_expand_static(step, width, fanout, cand_ids, cand_logprobs, root_token, node_parent, node_token,
                             node_logv, node_depth, node_count, frontier, n_frontier, status=None, stream=None):
    """One depth of a static tree: frontier node j keeps its top-fanout[j] candidates."""
    B, max_nodes = node_parent.shape
    k = cand_ids.shape[-1]
    _check("eagle_tree_expand_static", lib().eagle_tree_expand_static(
        B, step, width, k, max_nodes, _ptr(fanout), _ptr(cand_ids), _ptr(cand_logprobs), _ptr(root_token),
        _ptr(node_parent), _ptr(node_token), _ptr(node_logv), _ptr(node_depth), _ptr(node_count),
        _ptr(frontier), _ptr(n_frontier), _ptr(status), _stream(stream)))


def eagle_tree_expand_finalize(budget, node_parent, node_token, node_logv, node_depth, node_count,
                               ctx_lens, token, parent_row, depth, mask, node_id, position, n_rows,
                               status=None, stream=None):
    B, max_nodes = node_parent.shape
    R = token.shape[1]
    _check("eagle_tree_expand_finalize", lib().eagle_tree_expand_finalize(
        B, max_nodes, budget, R, _ptr(node_parent), _ptr(node_token), _ptr(node_logv),
        _ptr(node_depth), _ptr(node_count), _ptr(ctx_lens), _ptr(token), _ptr(parent_row),
        _ptr(depth), _ptr(mask), _ptr(node_id), _ptr(position), _ptr(n_rows), _ptr(status),
        _stream(stream)))


# ------------------------------------------------------------------ a6 / a7
def eagle_tree_verify_workspace_size(B, R, V):
    return int(lib().eagle_tree_verify_workspace_size(B, R, V))


def eagle_tree_verify(parent_row, token, temperature, max_depth, accept_len, path_rows, out_tokens,
                      n_rows=None, target_logits=None, target_argmax=None, draft_logits=None,
                      proposal_mode=EAGLE_PROPOSAL_DETERMINISTIC, seed=0, offset=0,
                      uniforms_override=None, V=None, ws=None, status=None, stream=None):
    B, R = parent_row.shape
    if V is None:
        V = target_logits.shape[2]
    if ws is None:
        ws = workspace(eagle_tree_verify_workspace_size(B, R, V), parent_row.device, stream)
    _check("eagle_tree_verify", lib().eagle_tree_verify(
        B, R, V, _ptr(parent_row), _ptr(token), _ptr(n_rows), _ptr(target_logits),
        _ptr(target_argmax), _ptr(draft_logits), float(temperature), proposal_mode, int(seed),
        int(offset), _ptr(uniforms_override), max_depth, _ptr(accept_len), _ptr(path_rows),
        _ptr(out_tokens), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))


def eagle_tree_verify_noalloc(parent_row, token, temperature, max_depth, accept_len, path_rows,
                              out_tokens, n_rows=None, target_logits=None, target_argmax=None,
                              draft_logits=None, proposal_mode=EAGLE_PROPOSAL_DETERMINISTIC, seed=0,
                              offset=0, uniforms_override=None, V=None, status=None, stream=None):
    """eagle_tree_verify for callers that cannot allocate: no workspace
    argument, statistics kept in the library's fixed device buffer
    (B * R <= 65536; at T > 0 also B * ceil(V / 4096) <= 65536)."""
    B, R = parent_row.shape
    if V is None:
        V = target_logits.shape[2]
    _check("eagle_tree_verify_noalloc", lib().eagle_tree_verify_noalloc(
        B, R, V, _ptr(parent_row), _ptr(token), _ptr(n_rows), _ptr(target_logits),
        _ptr(target_argmax), _ptr(draft_logits), float(temperature), proposal_mode, int(seed), int(offset),
        _ptr(uniforms_override), max_depth, _ptr(accept_len), _ptr(path_rows), _ptr(out_tokens),
        _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ K8
def eagle_lmhead_verify_stats(x, w_lm, parent_row, token, temperature, race_k, race_ids,
                              race_keys, row_max, row_sumexp, child_logit, n_rows=None, bias=None,
                              seed=0, offset=0, ws=None, status=None, stream=None):
    """Verification statistics from the LM head (rows of x: request-major
    B*R); see include/eagle.h."""
    B, R = parent_row.shape
    M, d = x.shape
    V = w_lm.shape[0]
    dt = _dtype(x)
    if ws is None:
        ws = workspace(eagle_lmhead_topk_workspace_size(M, d, V, race_k, dt), x.device, stream)
    _check("eagle_lmhead_verify_stats", lib().eagle_lmhead_verify_stats(
        _ptr(x), _ptr(w_lm), _ptr(bias), B, R, d, V, _ptr(parent_row), _ptr(token), _ptr(n_rows),
        float(temperature), int(seed), int(offset), race_k, _ptr(race_ids), _ptr(race_keys),
        _ptr(row_max), _ptr(row_sumexp), _ptr(child_logit), dt, _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))


def eagle_tree_verify_stats(parent_row, token, temperature, max_depth, row_max, row_sumexp,
                            child_logit, race_ids, accept_len, path_rows, out_tokens, V,
                            n_rows=None, seed=0, offset=0, uniforms_override=None, status=None,
                            stream=None):
    B, R = parent_row.shape
    race_k = race_ids.shape[-1]
    _check("eagle_tree_verify_stats", lib().eagle_tree_verify_stats(
        B, R, V, _ptr(parent_row), _ptr(token), _ptr(n_rows), _ptr(row_max), _ptr(row_sumexp),
        _ptr(child_logit), _ptr(race_ids), race_k, float(temperature), int(seed), int(offset),
        _ptr(uniforms_override), max_depth, _ptr(accept_len), _ptr(path_rows), _ptr(out_tokens),
        _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ K9
def eagle_tree_commit(k_tree, v_tree, path_rows, accept_len, k_cache, v_cache, block_table,
                      ctx_lens, features=None, features_out=None, status=None, stream=None):
    """Publish the verified path into the paged cache (see include/eagle.h)."""
    B, R, Hkv, D = k_tree.shape
    max_depth = path_rows.shape[1] - 1
    F = 0 if features is None else features.shape[1]
    _check("eagle_tree_commit", lib().eagle_tree_commit(
        B, R, Hkv, D, max_depth, _dtype(k_tree), _ptr(k_tree), _ptr(v_tree), _ptr(path_rows),
        _ptr(accept_len), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_table),
        block_table.shape[1], _ptr(ctx_lens), _ptr(features), F, _ptr(features_out),
        _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ the prompt path
# These calls are made once per layer and decoding step, so the marshalling is
# kept short: plain integers for the pointers, no intermediate objects.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _row_stride(name, t, D, T=None, H=None):
    """Row stride of a [T, H, D] array whose heads and channels are contiguous."""
    if T is None:
        T, H, _ = t.shape
    rows, heads, last = t.stride()
    if last != 1 or (heads != D and H > 1):
        raise ValueError(f"{name}: heads and channels must be contiguous, strides {t.stride()}")
    return rows if T > 1 else H * D  # (a single row's stride leads nowhere and may be anything)


# The kernels check lengths and page ids, but take the arrays' own shapes, types
# and layouts from the arguments that are derived below; an array that is not as
# those say would be read, or its neighbours written, out of place.  Every
# attribute of a tensor costs some 60 ns or more, so each is taken once, and the
# conditions stand in line.
_I32, _F32 = torch.int32, torch.float32
_BYTES = (torch.uint8, torch.float8_e4m3fn)


def _lengths(rows, cu_seqlens, ctx_lens, block_table, status):
    """Last of a call's checks, those of the index arrays, and that they (the
    ones that are built on the host) and the rows are on the GPU: (B, max_pages)."""
    if not (cu_seqlens.dtype is _I32 and ctx_lens.dtype is _I32 and block_table.dtype is _I32
            and cu_seqlens.is_contiguous() and ctx_lens.is_contiguous() and block_table.is_contiguous()):
        raise ValueError("cu_seqlens, ctx_lens and block_table must be contiguous int32")
    B, pages = block_table.shape
    if ctx_lens.shape != (B,) or cu_seqlens.shape != (B + 1,):
        raise ValueError("cu_seqlens must be [B + 1], ctx_lens [B] and block_table [B, max_pages]")
    if status is not None and status.dtype is not _I32:
        raise ValueError("status must be int32")
    if not (rows.is_cuda and cu_seqlens.is_cuda and ctx_lens.is_cuda and block_table.is_cuda):
        raise ValueError("the arrays must be on the GPU")
    return B, pages


def _pages16(k_cache, v_cache, Hkv, D, dtype):
    """Checks of 16- or 32-bit pages: their number."""
    shape = k_cache.shape
    if v_cache.shape != shape or shape != (shape[0], 16, Hkv, D):
        raise ValueError("k_cache and v_cache must be [pages, 16, Hkv, D]")
    if not (k_cache.dtype is dtype and v_cache.dtype is dtype and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous, with the rows' dtype")
    return shape[0]


def _pages4(k_codes, k_scales, v_codes, v_scales, Hkv, D):
    """Checks of 4-bit pages: their number."""
    shape, scales = k_codes.shape, k_scales.shape
    P = shape[0]
    if (v_codes.shape != shape or v_scales.shape != scales or shape != (P, Hkv, 16, D // 2)
            or scales != (P, Hkv, 16, D // 16)):
        raise ValueError("codes must be [pages, Hkv, 16, D / 2], scales [pages, Hkv, 16, D / 16]")
    if not (k_codes.dtype is torch.uint8 and v_codes.dtype is torch.uint8 and k_scales.dtype in _BYTES
            and v_scales.dtype in _BYTES):
        raise ValueError("codes must be uint8, scales uint8 or float8_e4m3fn")
    if not (k_codes.is_contiguous() and k_scales.is_contiguous() and v_codes.is_contiguous()
            and v_scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    return P


def _rope_rows(rope, D):
    """Checks of a rotation table (or None): its positions."""
    if rope is None:
        return 0
    shape = rope.shape
    if shape != (shape[0], 2, D // 2) or rope.dtype is not _F32 or not rope.is_contiguous():
        raise ValueError("rope must be contiguous fp32 [max_pos, 2, D / 2]")
    return shape[0]


def _append_rows(q, k, v, q_out):
    """Checks of the row arrays and their strides: (T, Hkv, D, Hq, q stride, k stride, v stride)."""
    shape, dtype = k.shape, k.dtype
    T, Hkv, D = shape
    if v.shape != shape or v.dtype is not dtype:
        raise ValueError("k and v must have one dtype and one shape")
    (ks, kh, k1), (vs, vh, v1) = k.stride(), v.stride()
    if k1 != 1 or v1 != 1 or ((kh != D or vh != D) and Hkv > 1):
        raise ValueError(f"k, v: heads and channels must be contiguous, strides {k.stride()}, {v.stride()}")
    if T <= 1:
        ks = vs = Hkv * D  # (a single row's stride leads nowhere and may be anything)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return T, Hkv, D, 0, 0, ks, vs
    shape = q.shape
    rows, Hq, last = shape
    if rows != T or last != D or q.dtype is not dtype:
        raise ValueError("q must have k's rows, D and dtype")
    if q_out is None or q_out.shape != shape or q_out.dtype is not dtype or not q_out.is_contiguous():
        raise ValueError("q_out must be contiguous, with q's shape and dtype")
    return T, Hkv, D, Hq, _row_stride("q", q, D, T, Hq), ks, vs


def _attn_rows(q, out, lse):
    """Checks of the attention's row arrays: (T, Hq, D, q stride)."""
    shape = q.shape
    T, Hq, D = shape
    if out.shape != shape or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, with q's shape and dtype")
    if lse is not None and not (lse.shape == (T, Hq) and lse.dtype is _F32 and lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [T, Hq]")
    return T, Hq, D, _row_stride("q", q, D, T, Hq)


def eagle_rope_table(max_pos, D, theta, table=None, stream=None):
    """cos and sin of pos * theta^(-2i/D): [max_pos, 2, D/2] fp32 on the current device."""
    if table is None:
        table = _empty((max_pos, 2, D // 2), torch.float32, "cuda", stream)
    else:
        if _rope_rows(table, D) != max_pos:
            raise ValueError("table must be [max_pos, 2, D / 2]")
        if not table.is_cuda:
            raise ValueError("the table must be on the GPU")
    _check("eagle_rope_table", lib().eagle_rope_table(max_pos, D, float(theta), _addr(table),
                                                      _raw_stream(stream, table.device)))
    return table


def eagle_kv_append(q, k, v, rope, cu_seqlens, ctx_lens, block_table, k_cache, v_cache, q_out=None, status=None,
                    stream=None):
    """Rotate the packed rows to their positions, write q to q_out and k, v into
    the paged cache (see include/eagle.h).  q and q_out may be None, rope None
    for no rotation."""
    T, Hkv, D, Hq, qs, ks, vs = _append_rows(q, k, v, q_out)
    P, max_pos = _pages16(k_cache, v_cache, Hkv, D, k.dtype), _rope_rows(rope, D)
    B, pages = _lengths(k, cu_seqlens, ctx_lens, block_table, status)
    _check("eagle_kv_append", lib().eagle_kv_append(
        _addr(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, _addr(rope), max_pos, cu_seqlens.data_ptr(),
        ctx_lens.data_ptr(), B, T, Hq, Hkv, D, _dtype(k), _addr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), P,
        block_table.data_ptr(), pages, _addr(status), _raw_stream(stream, k.device)))


def eagle_kv_append_kv4(q, k, v, rope, cu_seqlens, ctx_lens, block_table, k_codes, k_scales, v_codes, v_scales,
                        q_out=None, k_scale=1.0, v_scale=1.0, status=None, stream=None):
    """eagle_kv_append into 4-bit pages (see include/eagle.h)."""
    T, Hkv, D, Hq, qs, ks, vs = _append_rows(q, k, v, q_out)
    if k.dtype != torch.bfloat16:
        raise ValueError("k and v must be bf16")
    P, max_pos = _pages4(k_codes, k_scales, v_codes, v_scales, Hkv, D), _rope_rows(rope, D)
    B, pages = _lengths(k, cu_seqlens, ctx_lens, block_table, status)
    _check("eagle_kv_append_kv4", lib().eagle_kv_append_kv4(
        _addr(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, _addr(rope), max_pos, cu_seqlens.data_ptr(),
        ctx_lens.data_ptr(), B, T, Hq, Hkv, D, _addr(q_out), k_codes.data_ptr(), k_scales.data_ptr(),
        v_codes.data_ptr(), v_scales.data_ptr(), k_scale, v_scale, P, block_table.data_ptr(), pages, _addr(status),
        _raw_stream(stream, k.device)))


def eagle_kv4_read(codes, scales, out, scale=1.0, stream=None):
    """The values of 4-bit pages as an ordinary [pages, 16, Hkv, D] cache."""
    P, Hkv, _, half = codes.shape
    _pages4(codes, scales, codes, scales, Hkv, 2 * half)
    if out.shape != (P, 16, Hkv, 2 * half) or not out.is_contiguous():
        raise ValueError("out must be contiguous [pages, 16, Hkv, D]")
    if not (codes.is_cuda and scales.is_cuda and out.is_cuda):
        raise ValueError("the arrays must be on the GPU")
    _check("eagle_kv4_read", lib().eagle_kv4_read(codes.data_ptr(), scales.data_ptr(), scale, P, Hkv, 2 * half,
                                                  _dtype(out), out.data_ptr(), _raw_stream(stream, out.device)))
    return out


def eagle_prompt_attn_workspace_size(B, T, Hq, Hkv, D):
    return int(lib().eagle_prompt_attn_workspace_size(B, T, Hq, Hkv, D))


def eagle_prompt_attn(q, k_cache, v_cache, block_table, cu_seqlens, ctx_lens, out, lse=None, scale=None, ws=None,
                      status=None, stream=None):
    """Causal attention of the packed rows over the paged cache (see include/eagle.h)."""
    T, Hq, D, qs = _attn_rows(q, out, lse)
    _, page, Hkv, _ = k_cache.shape
    P = _pages16(k_cache, v_cache, Hkv, D, q.dtype)
    B, pages = _lengths(q, cu_seqlens, ctx_lens, block_table, status)
    if ws is None:
        ws = workspace(eagle_prompt_attn_workspace_size(B, T, Hq, Hkv, D), q.device, stream)
    _check("eagle_prompt_attn", lib().eagle_prompt_attn(
        q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), P, block_table.data_ptr(), pages,
        cu_seqlens.data_ptr(), ctx_lens.data_ptr(), out.data_ptr(), _addr(lse), B, T, Hq, Hkv, D, page,
        D ** -0.5 if scale is None else scale, _dtype(q), ws.data_ptr(), ws.numel(), _addr(status),
        _raw_stream(stream, q.device)))
    return out


def eagle_prompt_attn_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, ctx_lens, out, lse=None,
                          scale=None, k_scale=1.0, v_scale=1.0, ws=None, status=None, stream=None):
    """eagle_prompt_attn over 4-bit pages (see include/eagle.h)."""
    if q.dtype != torch.bfloat16:
        raise ValueError("q and out must be bf16")
    T, Hq, D, qs = _attn_rows(q, out, lse)
    _, Hkv, page, _ = k_codes.shape
    P = _pages4(k_codes, k_scales, v_codes, v_scales, Hkv, D)
    B, pages = _lengths(q, cu_seqlens, ctx_lens, block_table, status)
    if ws is None:
        ws = workspace(eagle_prompt_attn_workspace_size(B, T, Hq, Hkv, D), q.device, stream)
    _check("eagle_prompt_attn_kv4", lib().eagle_prompt_attn_kv4(
        q.data_ptr(), qs, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), k_scale,
        v_scale, P, block_table.data_ptr(), pages, cu_seqlens.data_ptr(), ctx_lens.data_ptr(), out.data_ptr(),
        _addr(lse), B, T, Hq, Hkv, D, page, D ** -0.5 if scale is None else scale, ws.data_ptr(), ws.numel(),
        _addr(status), _raw_stream(stream, q.device)))
    return out


def eagle_draft_prompt_workspace_size(B, T, d, Hq, Hkv, D, I, dtype):
    return int(lib().eagle_draft_prompt_workspace_size(B, T, d, Hq, Hkv, D, I, dtype))


def eagle_draft_prompt(x, weights, rope, cu_seqlens, ctx_lens, k_cache, v_cache, block_table, out, eps=1e-5,
                       k_scales=None, v_scales=None, k_scale=1.0, v_scale=1.0, ws=None, status=None, stream=None):
    """The drafter's decoder layer over packed prompt rows, filling its paged
    cache (with k_scales and v_scales: 4-bit pages).  weights as eagle_draft_layer."""
    T, d = x.shape
    D = 2 * rope.shape[2]
    max_pos = _rope_rows(rope, D)
    Hq = weights["o"].shape[1] // D
    Hkv = (weights["qkv"].shape[0] // D - Hq) // 2
    I = weights["down"].shape[1]
    shapes = dict(norm1=(d,), qkv=((Hq + 2 * Hkv) * D, d), o=(d, Hq * D), norm2=(d,), gu=(2 * I, d), down=(d, I))
    for name, shape in shapes.items():
        w = weights[name]
        if w.shape != shape or w.dtype is not x.dtype or not w.is_contiguous():
            raise ValueError(f"weights[{name!r}] must be contiguous {list(shape)}, with x's dtype")
    if not (x.is_contiguous() and out.shape == x.shape and out.dtype is x.dtype and out.is_contiguous()):
        raise ValueError("x and out must be contiguous, with one shape and dtype")
    if k_scales is None and v_scales is None:
        P = _pages16(k_cache, v_cache, Hkv, D, x.dtype)
    elif k_scales is None or v_scales is None or x.dtype != torch.bfloat16:
        raise ValueError("4-bit pages need k_scales and v_scales, and bf16 rows")
    else:
        P = _pages4(k_cache, k_scales, v_cache, v_scales, Hkv, D)
    B, pages = _lengths(x, cu_seqlens, ctx_lens, block_table, status)
    dt = _dtype(x)
    if ws is None:
        ws = workspace(eagle_draft_prompt_workspace_size(B, T, d, Hq, Hkv, D, I, dt), x.device, stream)
    _check("eagle_draft_prompt", lib().eagle_draft_prompt(
        x.data_ptr(), _addr(weights["norm1"]), _addr(weights["qkv"]), _addr(weights["o"]), _addr(weights["norm2"]),
        _addr(weights["gu"]), _addr(weights["down"]), eps, rope.data_ptr(), max_pos, cu_seqlens.data_ptr(),
        ctx_lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scales), _addr(v_scales), k_scale, v_scale,
        P, block_table.data_ptr(), pages, out.data_ptr(), B, T, d, Hq, Hkv, D, I, dt,
        ws.data_ptr(), ws.numel(), _addr(status), _raw_stream(stream, x.device)))
    return out
