"""The attention of the serving operators at scores of any size that fp32 holds.
Every score here is one exact product (or a power of two of equal ones), so that
the weights are known: keys of the same score share a row evenly, lower ones
have no weight."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve as so
from store_h3kv_build_gb300 import binding as b
from store_h3kv_build_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def normal(seed, *shape):
    return synth.normal_f32(shape, seed).to(torch.bfloat16)


def close(got, want, off, what):
    got = got.cpu().double().numpy()
    assert np.isfinite(got).all(), f"{what}: {(~np.isfinite(got)).sum()} of {got.size} not finite"
    over = np.abs(got - want) > off
    assert not over.any(), f"{what}: {over.sum()} of {over.size} off by up to {np.abs(got - want).max()}"


def mean_of(v, see):
    """Mean of the rows of v [h, n, 128] that each row of see [rows, n] names,
    and how far a kernel may be off: weights of exactly 1, an fp32 sum of as
    many values (a tensor core truncates: 2^-23 each), one divide, one rounding
    to bf16 (half a step, 2^-8)."""
    v = oracle.as_f64(v)
    w = see / see.sum(1, keepdims=True)
    o, a = w @ v, w @ np.abs(v)
    return o, (see.sum(1) + 16)[:, None] * 2.0 ** -23 * a + 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7)


def check_lse(lse, score, count, what):
    """score: q k of each row; the kernel's scale is fp32, as is the result."""
    want = score * oracle.default_scale() + np.log(count)
    got = lse.cpu().double().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= 2.0 ** -20 * np.abs(want) + 1e-5).all(), what


# 1.7e9 is the first of about 2^28 in log2 units; beyond, a product of the scale
# and the maximum that is rounded to fp32 is off by powers of two of weight
SCORES = [(2.0 ** 13, 2.0 ** 9), (41216.0, 41216.0), (2.0 ** 20, 2.0 ** 20), (2.0 ** 52, 2.0 ** 50), (2.0 ** 53, 2.0 ** 56),
          (1e16, 1e18), (3e18, 3e18)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", range(len(SCORES)))
@pytest.mark.parametrize("hq,n,causal", [(1, 1, True), (1, 128, True), (1, 300, True), (1, 300, False), (160, 384, True),
                                         (160, 300, False)])
def test_prompt_equal_scores_of_any_size(cuda, hq, n, causal, size, sign):
    q, k, v = (torch.zeros((h, n, 128), dtype=torch.bfloat16) for h in (hq, 1, 1))
    q[:, :, 3], k[:, :, 3] = sign * SCORES[size][0], SCORES[size][1]
    v.copy_(normal(n, 1, n, 128))
    lse = torch.zeros((hq, n), device=DEV)
    out = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, n]), causal=causal, lse=lse)
    b.sync_status()
    see = np.tril(np.ones((n, n))) if causal else np.ones((n, n))
    want, off = mean_of(v, see)
    score = (q[0, 0, 3].double() * k[0, 0, 3].double()).item()
    what = f"{hq} heads, {n} rows, score {score:.2g}"
    close(out, want, off, what)
    check_lse(lse, np.full((1, n), score), see.sum(1)[None], what)


@pytest.mark.parametrize("hq", [1, 160])
@pytest.mark.parametrize("size", [(2.0 ** 20, 2.0 ** 20), (2.0 ** 54, 2.0 ** 56)])
def test_prompt_largest_of_scores_of_any_size(cuda, hq, size):
    # keys of unlike scores, the larger ones in any tile: their mean alone,
    # beside rows of ordinary scores and rows of the other sign
    n = 520
    g = np.random.default_rng(3)
    level = g.integers(1, 4, n)
    level[:130] = 1              # the larger ones come later
    q, k, v = normal(1, hq, n, 128), normal(2, 1, n, 128), normal(3, 1, n, 128)
    k[0, :, 3] = torch.from_numpy(level * size[1]).to(torch.bfloat16)
    q[:, :, 3] = 0
    kind = g.integers(0, 3, n)   # 0: ordinary, 1: positive, 2: negative
    for s, at in ((1, kind == 1), (-1, kind == 2)):
        q[:, at] = 0
        q[:, at, 3] = s * size[0]
    out = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, n]))
    b.sync_status()
    tri = np.tril(np.ones((n, n), dtype=bool))
    for s, at in ((1, kind == 1), (-1, kind == 2)):
        x = np.where(tri, s * level[None, :], -9)
        want, off = mean_of(v, (x == x.max(1, keepdims=True)).astype(float))
        close(out[:, at], want[:, at], off[:, at], f"sign {s}")
    at = kind == 0
    want, _, off, _ = so.attend_prompt(q, k, v, [0, n], [0, n])
    close(out[:, at], want[:, at], off[:, at], "ordinary rows")


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e6])
def test_prompt_equal_scores_with_any_scale(cuda, scale):
    n = 300
    q, k, v = normal(1, 2, n, 128), torch.zeros((2, n, 128), dtype=torch.bfloat16), normal(3, 2, n, 128)
    k[:] = normal(2, 1, 1, 128)
    out = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, n]), softmax_scale=scale)
    b.sync_status()
    want, off = mean_of(v, np.tril(np.ones((n, n))))
    close(out, want, off, f"scale {scale}")


def big_store(n, ps, hk, scale, seed):
    """Rows whose K' are all 127 * scale in every channel, in half of them
    negated, and ordinary V."""
    pages = -(-n // ps)
    g = np.random.default_rng(seed)
    sign = g.choice([-1, 1], (pages, 1, ps, 1))
    kc = np.broadcast_to(127 * sign, (pages, hk, ps, 128)).astype(np.int8)
    ks = np.full((pages, hk, ps), scale)
    vc, vs = oracle.encode_rows(normal(seed, pages, hk, ps, 128))
    ref = {"k_codes": kc, "v_codes": vc, "k_scales": ks, "v_scales": vs}
    st = b.PagedStore(*(torch.from_numpy(np.ascontiguousarray(ref[x])).to(DEV).to(t) for x, t in
                        (("k_codes", torch.int8), ("v_codes", torch.int8), ("k_scales", torch.float16),
                         ("v_scales", torch.float16))))
    return st, ref, sign[:, 0, :, 0].reshape(-1)[:n]


@pytest.mark.parametrize("hq,m", [(4, 1), (8, 2), (8, 4), (8, 40), (32, 64)])
@pytest.mark.parametrize("scale", [2.0 ** -6, 4.0, 256.0])
@pytest.mark.parametrize("n", [64, 300, 20000])
def test_tree_scores_of_any_size(cuda, hq, m, scale, n):
    # q' is 2^15 in every channel (or its negative), so a score is 128 * 2^15 *
    # 127 * scale: up to 1.4e11, an exact one
    ps, hk = 64, 2
    st, ref, sign = big_store(n, ps, hk, scale, n)
    q = torch.zeros((hq, m, 128), dtype=torch.bfloat16)
    q[..., 0] = 370688.0
    q[:, ::2] *= -1
    qr = oracle.fp16_round(oracle.rotate(oracle.as_f64(q)))
    assert (np.abs(qr) == 2.0 ** 15).all()
    table = [list(range(-(-n // ps)))]
    lse = torch.zeros((hq, m), device=DEV)
    out = b.attend_tree(q.to(DEV), st, i32(table), i32([n]), i32([0, m]), lse=lse)
    b.sync_status()
    see = np.arange(n)[None, :] <= n - m + np.arange(m)[:, None]
    x = np.where(see, np.sign(qr[0, :, :1]) * sign[None, :], -2)
    top = x.max(1, keepdims=True)
    see = (x == top).astype(float)
    score = top[None, :, 0] * 128 * 2.0 ** 15 * 127 * scale
    v = so.gather(ref["v_codes"], ref["v_scales"], table[0], n)
    w = see / see.sum(1, keepdims=True)
    o, a = w @ v, w @ np.abs(v)
    rot = np.abs(oracle.hadamard())
    o, a = oracle.unrotate(o), a @ rot
    # as in mean_of, through the rotation back
    off = (see.sum(1) + 16)[:, None] * 2.0 ** -23 * a + 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7) + 2.0 ** -20 * a
    for h in range(hq):
        close(out[h], o[h // (hq // hk)], off[h // (hq // hk)], f"{n} rows, head {h}")
    check_lse(lse, np.broadcast_to(score, (hq, m)), see.sum(1)[None], f"{n} rows lse")


@pytest.mark.parametrize("hq,m", [(1, 1), (8, 2), (8, 4), (8, 8)])
@pytest.mark.parametrize("x", [20.3, 24.6, 25.5, 28.0])
def test_tree_many_small_weights_beside_a_large_one(cuda, hq, m, x):
    """A million cached rows, each 2^-x of the weight of one: together as much
    as 2^20 2^-x.  fp16 holds a weight to half a step (2^-11 of it), or to 2^-32
    of the largest where it is subnormal.  As many sequences (over the same
    pages) as there are SMs, so that no split of the keys separates them."""
    seqs = torch.cuda.get_device_properties(0).multi_processor_count
    n, ps = 1 << 20, 128
    pages = n // ps
    st = b.PagedStore(*(torch.zeros((pages, 1, ps, 128), dtype=torch.int8, device=DEV) for _ in range(2)),
                      *(torch.zeros((pages, 1, ps), dtype=torch.float16, device=DEV) for _ in range(2)))
    st.k_codes[5, 0, 77, 0], st.k_scales[5, 0, 77] = 127, 1 / 64
    st.v_codes[..., 0], st.v_scales[:] = 100, 1 / 64
    st.v_codes[5, 0, 77] = 0
    q = torch.full((hq, seqs * m, 128), 3.0, dtype=torch.bfloat16)
    qr = oracle.fp16_round(oracle.rotate(oracle.as_f64(q)))[0, 0]
    score = qr[0] * 127 / 64
    assert (qr[1:] == 0).all()
    scale = float(np.float32(x * np.log(2.0) / score))
    parents = torch.full((seqs * m,), -1, dtype=torch.int32, device=DEV)  # every node beside the others
    out = b.attend_tree(q.to(DEV), st, i32([list(range(pages))] * seqs), i32([n] * seqs),
                        i32(list(range(0, seqs * m + 1, m))), parents, softmax_scale=scale)
    b.sync_status()
    rest = (n - m) * np.exp(-score * scale)  # n - m keys before, and itself
    want = rest / (1 + rest) * (100 / 64) / np.sqrt(128.0)
    w = np.exp2(-x)
    # the score's fp32 roundings move a weight by 2^-20 of it; sums as above
    off = want * (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -8) + (n - m) * min(2.0 ** -32, w) / (1 + rest) * (100 / 64) / np.sqrt(128.0)
    close(out, np.full((hq, seqs * m, 128), want), off, f"x {x}")
