"""The prompt path in fp64: rotation and append, 4-bit pages, causal attention
of packed rows over a paged cache.

Sources: [M7.5] sections 0x03C and 0x05D (rows go to the cache by position);
the rotation is that of ``rope`` in eagle_oracle.  The pages print no 4-bit
format: the grid and its scale are fixed here from the definition (nearest
value, ties to the even code) and pinned by exhaustive search in the tests.
"""
import numpy as np

PAGE = 16
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte):
    """Value of an e4m3 byte (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f is NaN)."""
    b = np.asarray(byte).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


_E4M3 = e4m3_value(np.arange(127))  # the finite non-negative values, ascending


def e4m3_byte(x):
    """Nearest e4m3 byte of x >= 0, ties to the even byte, at most 448; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(_E4M3, x), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - _E4M3[lo], _E4M3[hi] - x
    byte = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    byte = np.where(x >= 448, 126, byte)
    return np.where(np.isnan(x), 127, byte).astype(np.uint8)


def kv4_pack(x, scale=1.0):
    """Codes [..., D/2] and scale bytes [..., D/16] of x [..., D] (fp32 values)."""
    x = np.asarray(x, np.float32) * (np.float32(1) / np.float32(scale))
    g = x.reshape(*x.shape[:-1], -1, 16)
    sb = e4m3_byte(np.abs(g).max(-1) / np.float32(6))
    s = e4m3_value(sb)[..., None]
    d = np.abs(np.abs(g.astype(np.float64))[..., None] - s[..., None] * MAGNITUDES)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])  # an even code wins a tie
    with np.errstate(invalid="ignore"):
        code = order[np.argmin(np.where(np.isnan(d), np.inf, d)[..., order], -1)]
    code = np.where(s > 0, code, 0) + 8 * np.signbit(g)
    code = code.reshape(*x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb


def kv4_unpack(codes, scales, scale=1.0):
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[both & 7] * np.where(both & 8, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, 16) * e4m3_value(scales)[..., None]).reshape(v.shape) * scale


def rotate(x, rope_rows):
    """x [T, H, D] by rope_rows [T, 2, D/2] (cos, sin), pair (i, i + D/2), fp64."""
    x = np.asarray(x, np.float64)
    h = x.shape[-1] // 2
    c, s = (np.asarray(rope_rows, np.float64)[:, i, None] for i in (0, 1))
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def row_places(cu, ctx, table):
    """(request, position, page, slot) of every packed row."""
    out = []
    for b in range(len(ctx)):
        for i in range(cu[b + 1] - cu[b]):
            p = int(ctx[b]) + i
            out.append((b, p, int(table[b][p // PAGE]), p % PAGE))
    return out


def prompt_attn(q, keys, values, cu, ctx, scale):
    """Causal attention of packed rows.  keys, values: per request [n_keys, Hkv, D].
    Returns out, lse and, for error bounds, sum_j w_j |v_j| and the largest
    scale * sum_c |q_c k_c| per (row, head)."""
    T, Hq, D = q.shape
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, dot = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(ctx)):
        n, c = int(cu[b + 1] - cu[b]), int(ctx[b])
        if n == 0:
            continue
        rows = slice(int(cu[b]), int(cu[b + 1]))
        late = np.arange(c + n)[None] > c + np.arange(n)[:, None]
        for h in range(Hq):
            hk = h // (Hq // keys[b].shape[1])
            qq, k, v = (np.asarray(a, np.float64) for a in (q[rows, h], keys[b][:c + n, hk], values[b][:c + n, hk]))
            z = np.where(late, -np.inf, qq @ k.T * scale)
            m = z.max(-1, keepdims=True)
            w = np.exp(z - m)
            l = w.sum(-1, keepdims=True)
            out[rows, h], mag[rows, h] = w / l @ v, w / l @ np.abs(v)
            lse[rows, h] = (m + np.log(l))[:, 0]
            dot[rows, h] = np.where(late, 0, np.abs(qq) @ np.abs(k).T * scale).max(-1)
    return out, lse, mag, dot


def prefix_attn(q, keys, values, cu, scale, own_out=None, own_lse=None):
    """Attention of groups of rows over the keys [n_keys, Hkv, D] of their group,
    all visible, joined with the rows' own result.  Returns out, lse and, for
    error bounds, sum_j w_j |v_j| of the prefix alone and with the own part, and the
    largest scale * sum_c |q_c k_c|."""
    T, Hq, D = q.shape
    out, mag, both = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, dot = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for g, (k_all, v_all) in enumerate(zip(keys, values)):
        rows = slice(int(cu[g]), int(cu[g + 1]))
        for h in range(Hq):
            hk = h // (Hq // k_all.shape[1])
            qq, k, v = (np.asarray(a, np.float64) for a in (q[rows, h], k_all[:, hk], v_all[:, hk]))
            z = qq @ k.T * scale
            own = own_lse is not None
            # the own keys are one more key, of score own_lse and value own_out
            L = np.asarray(own_lse[rows, h], np.float64)[:, None] if own else np.full((len(qq), 1), -np.inf)
            o = np.where(np.isneginf(L), 0.0, np.asarray(own_out[rows, h], np.float64)) if own else np.zeros((len(qq), D))
            m = np.maximum(z.max(-1, keepdims=True, initial=-np.inf), L)
            ref = np.where(np.isneginf(m), 0.0, m)
            w, wo = np.exp(z - ref), np.exp(L - ref)
            l = w.sum(-1, keepdims=True) + wo
            div = np.where(l == 0, 1.0, l)
            out[rows, h] = w / div @ v + wo / div * o
            mag[rows, h] = w / div @ np.abs(v)
            both[rows, h] = mag[rows, h] + wo / div * np.abs(o)
            with np.errstate(divide="ignore"):
                lse[rows, h] = (ref + np.log(l))[:, 0]
            dot[rows, h] = (np.abs(qq) @ np.abs(k).T * scale).max(-1, initial=0.0)
    return out, lse, mag, both, dot
