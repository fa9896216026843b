"""fp64 CPU oracle of the serving operators: attention over packed prompts,
the paged kvi8r cache and the attention of drafted trees over it (test
infrastructure only).

Beside each attention result it returns how far a kernel may be off it, from
the roundings that the operators' definitions leave to the kernel:

* P enters the second product rounded to the 16-bit type (relative half step
  u_p, plus tiny_p for fp16 subnormals);
* scores carry the fp32 accumulation of 128 exact products (136 steps, and a
  tensor core truncates: 2^-23 each), and for the cache the query elements
  whose fp16 rounding lies within the fp32 rotation's error of a tie may land
  one step away; an error e of a score moves its weight by a factor within
  exp(+-2 e);
* the output is rounded to bf16 once: half a step, 2^-8 of its size;
* 2^-20 of the absolute sums covers the fp32 rotation of the output, ex2
  (2^-22), the row sum and the divide.
"""
from __future__ import annotations

import numpy as np

from .kvi8r import as_f64, default_scale, dequant, fp16_round, hadamard, rotate, unrotate

U_BF16, U_FP16 = 2.0 ** -8, 2.0 ** -11


def _softmax(q, k, v, see, scale, e_extra, u_p, tiny_p):
    """One head: outputs, lse, sum of p|v|, score errors (rows without keys:
    0, -inf)."""
    s = (q @ k.T) * scale
    s = np.where(see, s, -np.inf)
    top = s.max(axis=1, initial=-np.inf, keepdims=True)
    any_key = np.isfinite(top)
    w = np.where(see, np.exp(s - np.where(any_key, top, 0.0)), 0.0)
    z = w.sum(axis=1, keepdims=True)
    p = w / np.where(any_key, z, 1.0)
    with np.errstate(divide="ignore"):
        lse = np.where(any_key, np.where(any_key, top, 0.0) + np.log(np.where(any_key, z, 1.0)), -np.inf)[:, 0]
    mag = (np.abs(q) @ np.abs(k).T) * scale
    e = 136 * 2.0 ** -23 * np.where(see, mag, 0.0).max(axis=1, initial=0.0) + e_extra
    av = p @ np.abs(v)
    vmax = np.abs(v).max(axis=0, initial=0.0)
    # fp16 weights below 2^-14 are subnormal: an absolute half step of 2^-25
    # against weights scaled so that their sum is at least z of the maximum
    sub = tiny_p * see.sum(axis=1)[:, None] * vmax[None, :] / np.where(any_key, z, 1.0)
    off = (u_p + 2 * e[:, None] + 2.0 ** -20) * av + sub
    lse_off = e + (see.sum(axis=1) + 16) * 2.0 ** -24 + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) \
        + 2.0 ** -21
    return p @ v, lse, off, lse_off


def attend_prompt(Q, K, V, cu_q, cu_k, causal=True, scale=None):
    """-> (O, lse, bound of |O_kernel - O|, bound of |lse_kernel - lse|); rows
    of no sequence are NaN."""
    Q, K, V = as_f64(Q), as_f64(K), as_f64(V)
    scale = default_scale() if scale is None else scale
    g = Q.shape[0] // K.shape[0]
    O, lse = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    bo, bl = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    for i in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
        nq, nk = q1 - q0, k1 - k0
        see = np.ones((nq, nk), dtype=bool)
        if causal:
            see = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq
        for h in range(Q.shape[0]):
            o, z, off, zoff = _softmax(Q[h, q0:q1], K[h // g, k0:k1], V[h // g, k0:k1], see, scale, 0.0, U_BF16, 0.0)
            O[h, q0:q1], lse[h, q0:q1], bl[h, q0:q1] = o, z, zoff
            bo[h, q0:q1] = off + U_BF16 * np.abs(o) * (1 + 2.0 ** -7) + 2.0 ** -134
    return O, lse, bo, bl


def gather(codes, scales, table, length):
    """Rows 0 .. length-1 of one sequence, dequantised to fp16 values:
    [kv_heads, length, 128]; codes [pages, kv_heads, page_size, 128]."""
    ps = codes.shape[2]
    pos = np.arange(length)
    page = np.asarray(table)[pos // ps]
    c = np.asarray(codes)[page, :, pos % ps]
    s = as_f64(scales)[page, :, pos % ps]
    return np.swapaxes(fp16_round(dequant(c, s)), 0, 1)


def paths(parents, m):
    """[m, m]: whether node i lies on node j's path to its root."""
    see = np.zeros((m, m), dtype=bool)
    for j in range(m):
        n = j
        while n >= 0:
            see[j, n] = True
            up = n - 1 if parents is None else int(parents[n])
            n = up if 0 <= up < n else -1
    return see


def attend_tree(Q, store, table, lengths, cu, parents=None, scale=None):
    """store: dict of k_codes, v_codes, k_scales, v_scales as numpy arrays in
    pages.  Returns as attend_prompt."""
    Q = as_f64(Q)
    scale = default_scale() if scale is None else scale
    hk = store["k_codes"].shape[1]
    g = Q.shape[0] // hk
    qr = rotate(Q)
    qh = fp16_round(qr)
    # a query element is ambiguous where the fp32 rotation's error reaches the
    # rounding tie next to it
    err = 2.0 ** -21 * np.abs(Q).sum(axis=-1, keepdims=True) / np.sqrt(128.0)
    step = np.where(fp16_round(qr + err) != fp16_round(qr - err), 2.0 ** -9 * np.abs(qh) + 2.0 ** -24, 0.0)
    H = np.abs(hadamard())
    O, lse = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    bo, bl = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    for i in range(len(cu) - 1):
        c0, c1, n = cu[i], cu[i + 1], int(lengths[i])
        m = c1 - c0
        if m == 0:
            continue
        k = gather(store["k_codes"], store["k_scales"], table[i], n)
        v = gather(store["v_codes"], store["v_scales"], table[i], n)
        see = np.ones((m, n), dtype=bool)
        see[:, n - m:] = paths(None if parents is None else parents[c0:c1], m)
        for h in range(Q.shape[0]):
            flip = scale * (step[h, c0:c1] @ np.abs(k[h // g]).T).max(axis=1)
            o, z, off, zoff = _softmax(qh[h, c0:c1], k[h // g], v[h // g], see, scale, flip, U_FP16, 2.0 ** -25)
            O[h, c0:c1], lse[h, c0:c1], bl[h, c0:c1] = unrotate(o), z, zoff
            bo[h, c0:c1] = off @ H + 2.0 ** -20 * np.abs(o).sum(axis=1, keepdims=True) \
                + U_BF16 * np.abs(O[h, c0:c1]) * (1 + 2.0 ** -7) + 2.0 ** -134
    return O, lse, bo, bl


def keep_rows(arrays, table, lengths, cu, keep):
    """Move the kept drafted rows of every sequence up, in order, in copies of
    the arrays [pages, kv_heads, page_size, ...]; returns (arrays, lengths)."""
    out = {k: np.array(a) for k, a in arrays.items()}
    left = []
    for i in range(len(cu) - 1):
        m, n = cu[i + 1] - cu[i], int(lengths[i])
        to = n - m
        for j in range(m):
            if keep[cu[i] + j]:
                for k, a in arrays.items():
                    ps, src = a.shape[2], n - m + j
                    out[k][table[i][to // ps], :, to % ps] = a[table[i][src // ps], :, src % ps]
                to += 1
        left.append(to)
    return out, left
