"""fp64 CPU oracle of the rotation by positions and of the paged e4m3 cache: its
append, its values and the causal attention over it (test infrastructure only).

Attention bounds are those of ``serve._softmax`` (fp16 weights, fp32 sums); the
output is rounded to bf16 once.  K' and V' are exact for scales that the append
writes.
"""
from __future__ import annotations

import numpy as np

from .kvf8s import e4m3_decode, e4m3_encode
from .kvi8r import as_f64, default_scale, fp16_round
from .serve import U_BF16, U_FP16, _softmax

E_MIN, E_MAX = -15, 7


def rotate_positions(x, table, positions, interleaved=False):
    """x [heads, n, 128] rotated by table[positions] (dim / 2 cosines, dim / 2
    sines); table and x as fp64."""
    x, t = as_f64(x), as_f64(table)[np.asarray(positions)]
    half = t.shape[1] // 2
    c, s = t[:, :half], t[:, half:]
    j = np.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def page_exponent(top):
    """Least e in E_MIN .. E_MAX with top <= 448 2^e (or the largest)."""
    for e in range(E_MIN, E_MAX):
        if top <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def _encode(x):
    """e4m3 codes; beyond 448, infinities among them, 448; NaN stays."""
    c = e4m3_encode(np.clip(np.where(np.isnan(x), 0.0, x), -448.0, 448.0))
    return np.where(np.isnan(x), np.uint8(0x7F), c)


def append(arrays, k, v, table, lengths, cu):
    """arrays: k_codes, v_codes (uint8 [pages, heads, page_size, 128]), k_scales,
    v_scales (fp64 [pages, heads]); k, v fp64 [heads, n, 128], rotated already.
    Returns new arrays."""
    out = {n: np.array(a) for n, a in arrays.items()}
    ps = out["k_codes"].shape[2]
    for t, x in (("k", k), ("v", v)):
        codes, scales = out[t + "_codes"], out[t + "_scales"]
        for i in range(len(cu) - 1):
            p0 = int(lengths[i]) - (cu[i + 1] - cu[i])
            lo = p0
            while lo < lengths[i]:
                begin = lo // ps * ps
                hi = min(begin + ps, int(lengths[i]))
                page = table[i][begin // ps]
                rows = x[:, cu[i] + lo - p0:cu[i] + hi - p0]
                for h in range(x.shape[0]):
                    size = np.abs(rows[h])
                    e = page_exponent(size[~np.isnan(size)].max(initial=0.0))
                    if lo > begin:
                        old = scales[page, h]
                        e = max(e, int(np.ceil(np.log2(old))))
                        if 2.0 ** e != old:
                            codes[page, h, :lo - begin] = _encode(e4m3_decode(codes[page, h, :lo - begin]) * old / 2.0 ** e)
                    codes[page, h, lo - begin:hi - begin] = _encode(rows[h] / 2.0 ** e)
                    scales[page, h] = 2.0 ** e
                lo = hi
    return out


def gather(codes, scales, table, length):
    """[heads, length, 128]: the cached values of one sequence."""
    ps = codes.shape[2]
    pos = np.arange(length)
    page = np.asarray(table)[pos // ps]
    x = e4m3_decode(codes[page, :, pos % ps]) * fp16_round(scales[page])[:, :, None]
    return np.swapaxes(fp16_round(x), 0, 1)


def attend(Q, arrays, table, lengths, cu, scale=None, split=False):
    """-> (O, lse, bound of O, bound of lse); rows of no sequence are NaN.

    split: bounds for a query row as the sum of two e4m3 parts, scaled so that its
    largest element lies in (224, 448].  A bf16 element of at least 2^-2 there has
    a last bit of 2^-9 or more, which the second part's least step reaches: exact,
    and so is one down to 2^-9 of the largest.  One below is off by at most half
    that step, 2^-10 / 224 < 2^-17 of the largest."""
    Q = as_f64(Q)
    size = np.abs(Q)
    top = size.max(axis=-1, keepdims=True, initial=0.0)
    lost = np.where((size > 0) & (size < top * 2.0 ** -9), 2.0 ** -17 * top, 0.0) if split else np.zeros(Q.shape)
    scale = default_scale() if scale is None else scale
    hk = arrays["k_codes"].shape[1]
    g = Q.shape[0] // hk
    O, lse = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    bo, bl = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    for i in range(len(cu) - 1):
        c0, c1, n = cu[i], cu[i + 1], int(lengths[i])
        m = c1 - c0
        if m == 0:
            continue
        k = gather(arrays["k_codes"], arrays["k_scales"], table[i], n)
        v = gather(arrays["v_codes"], arrays["v_scales"], table[i], n)
        see = np.arange(n)[None, :] <= np.arange(n - m, n)[:, None]
        for h in range(Q.shape[0]):
            e = scale * (lost[h, c0:c1] @ np.abs(k[h // g]).T).max(axis=1)
            o, z, off, zoff = _softmax(Q[h, c0:c1], k[h // g], v[h // g], see, scale, e, U_FP16, 2.0 ** -25)
            O[h, c0:c1], lse[h, c0:c1], bl[h, c0:c1] = o, z, zoff
            bo[h, c0:c1] = off + U_BF16 * np.abs(o) * (1 + 2.0 ** -7) + 2.0 ** -134
    return O, lse, bo, bl
