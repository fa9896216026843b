"""Query rows of any size through the attention over e4m3 pages: zeros, rows far
below and far above one, rows with channels far larger than the rest; on the
kernel for few rows (items of 8, 16 and 32) and on both softmaxes of the one for
many."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve_f8 as so
from store_h3kv_build_gb300 import binding as b

from test_gpu_serve_f8 import DEV, arrays_of, cu_of, filled, i32, normal, within

pytestmark = pytest.mark.gpu

ROWS = [1, 3, 7, 20, 300]  # tokens of 4 heads: 4, 12, 28, 80 and 1200 rows
MANY = 20                  # from here on a query row is the sum of two e4m3 parts


def check(q, st, table, lens, news, scale, what, split=False):
    cu = cu_of(news)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    o = b.attend_paged_f8(q.to(DEV), st, torch.from_numpy(table).to(DEV), i32(lens), i32(cu), scale, lse=lse)
    b.sync_status()
    ref = so.attend(q, arrays_of(st), table, lens, cu, scale if scale > 0 else None, split=split)
    within(o, ref[0], ref[2], what)
    within(lse, ref[1], ref[3], what + " lse")


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("k_scale,scale", [(2.0 ** -30, 0.0), (None, 1e-18), (2.0 ** -30, 1e-12), (2.0 ** -20, 1e-30)])
def test_rows_of_zeros_and_factors_next_to_zero(cuda, m, ps, k_scale, scale):
    # every score is next to nothing, so that a row is the mean of the V that it sees
    lens = [m + 130, m + 1]
    st, table = filled(lens, 1, ps, m, bad=False)
    if k_scale is not None:
        st.k_scales.fill_(k_scale)
    q = normal(m, 4, 2 * m, 128)
    q[:, ::3] = 0
    q[1] *= 2.0 ** -100
    q[2] = 0
    check(q, st, table, lens, [m, m], scale, f"{m} {ps}")


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("size", [-50, -40, -20, 12])
def test_rows_of_any_size(cuda, m, size):
    lens = [m + 200, m]
    st, table = filled(lens, 2, 32, m, bad=False)
    q = normal(m + 1, 8, 2 * m, 128) * 2.0 ** size
    check(q, st, table, lens, [m, m], oracle.default_scale() * 2.0 ** -size, f"{m} {size}", split=m >= MANY)


@pytest.mark.parametrize("m", ROWS)
def test_rows_of_unlike_sizes(cuda, m):
    # each row has its own power of two
    lens = [m + 200, m]
    st, table = filled(lens, 2, 32, m, bad=False)
    q = normal(m + 1, 8, 2 * m, 128)
    rng = np.random.default_rng(m)
    q *= torch.from_numpy(2.0 ** -rng.integers(0, 40, (8, 2 * m, 1))).to(torch.bfloat16)
    check(q, st, table, lens, [m, m], 3.0, f"{m}", split=m >= MANY)


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("size", [9, 11, 13])
def test_rows_with_outlier_channels(cuda, m, size):
    # one channel 2^size times the others.  (A small softmax_scale: what the two
    # parts leave out of the other channels, 2^-17 of the outlier, is bounded by
    # sums of absolute values, of little use for scores of 10.)
    lens = [m + 200, m]
    st, table = filled(lens, 2, 32, m, bad=False)
    q = normal(m + 1, 8, 2 * m, 128)
    q[..., 5] *= 2.0 ** size
    check(q, st, table, lens, [m, m], 2.0 ** -(size - 2) if m < MANY else 2.0 ** -size, f"{m} {size}", split=m >= MANY)


@pytest.mark.parametrize("m", ROWS)
def test_factors_next_to_the_largest(cuda, m):
    # a row of 65280, the largest bf16 that fp16 holds, a softmax_scale next to
    # fp32's end: the keys whose least code gives a score share a row, zeros have none
    n, ps = m + 200, 32
    pages = -(-n // ps)
    st = b.PagedStoreF8.empty(pages, 1, ps)
    v = normal(m, 1, pages * ps, 128)
    table = i32(range(pages)).view(1, pages)
    b.paged_append_f8(v.to(DEV), v.to(DEV), st, table, i32([pages * ps]), i32([0, pages * ps]))
    some = np.random.default_rng(m).random(pages * ps) < 0.3
    some[0] = True
    st.k_codes.view(torch.uint8).zero_()
    st.k_codes.view(torch.uint8).view(-1, 128)[torch.from_numpy(some).to(DEV), 7] = 1  # 2^-9
    st.k_scales.fill_(2.0 ** -15)
    q = torch.zeros((4, m, 128))
    q[..., 7] = 65280.0
    q[3, :, 7] = -65280.0
    scale = 1.4e38
    lse = torch.zeros((4, m), device=DEV)
    o = b.attend_paged_f8(q.to(torch.bfloat16).to(DEV), st, table, i32([n]), i32([0, m]), scale, lse=lse)
    b.sync_status()
    vals = so.gather(st.v_codes.view(torch.uint8).cpu().numpy(), st.v_scales.double().cpu().numpy(), list(range(pages)), n)[0]
    see = np.arange(n)[None, :] <= n - m + np.arange(m)[:, None]
    score = 65280.0 * 2.0 ** -24 * scale
    for h in range(4):
        w = (see & (some[:n] if h < 3 else ~some[:n])[None, :]).astype(float)
        count = w.sum(1)
        w /= count[:, None]
        # weights of exactly one, an fp32 sum of as many values, a divide, a rounding to bf16
        off = (count + 16)[:, None] * 2.0 ** -23 * (w @ np.abs(vals)) + 2.0 ** -8 * np.abs(w @ vals) * (1 + 2.0 ** -7)
        within(o[h], w @ vals, off, f"head {h}")
        want = score if h < 3 else 0.0
        got = lse[h].cpu().double().numpy()
        assert (np.abs(got - want - np.log(count)) <= 2.0 ** -20 * want + 1e-4).all(), h
