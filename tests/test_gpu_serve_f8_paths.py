"""Paths of the appends to e4m3 pages and of the attention over them that take
many sequences, pages of 128 without a rotation, or keys rotated where they lie;
and what a call with bad indices leaves alone."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve_f8 as so
from store_h3kv_build_gb300 import binding as b

from test_gpu_serve_f8 import (DEV, angles, append_case, arrays_of, attend_case, bf16_of, cu_of, i32, normal,
                               rotated_within, table_of)

pytestmark = pytest.mark.gpu


def test_append_of_windows_of_many_sequences(cuda):
    # more sequences than a block has threads, each of several windows
    rng = np.random.default_rng(1)
    news = rng.integers(0, 401, 600)
    append_case(news.tolist(), (news + rng.integers(0, 200, 600)).tolist(), 1, 1, 64, 64, seed=1)


def test_attention_of_row_tiles_of_many_sequences(cuda):
    # more sequences than a block has threads, more than 32 rows each
    rng = np.random.default_rng(2)
    news = rng.integers(3, 9, 600)
    attend_case(news.tolist(), (news + rng.integers(0, 300, 600)).tolist(), 8, 1, 32, seed=2)
    news = rng.integers(0, 40, 1100)
    attend_case(news.tolist(), (news + rng.integers(0, 100, 1100)).tolist(), 8, 1, 64, seed=3)


@pytest.mark.parametrize("ps", [16, 64, 128])
def test_append_without_rotation_to_any_page(cuda, ps):
    append_case([700, 333], [900, 340], 4, 2, ps, seed=ps, rotate=False, pad=70, first=65)
    append_case([1, 3, 2, 5], [40, 3, 130, 37], 4, 2, ps, seed=ps, rotate=False)
    append_case([2000], [2100], 4, 3, ps, seed=ps, rotate=False, gain=20.0)


@pytest.mark.parametrize("dim,inter", [(128, False), (64, False), (48, True)])
@pytest.mark.parametrize("ps", [16, 64])
def test_few_tokens_rotated_in_place(cuda, ps, dim, inter):
    # some tokens of each sequence, over page borders: a page's rows of K are read
    # twice, and written between
    news, lens = [1, 12, 7, 3, 10, 0, 9, 5], [30, 33, 70, 66, 10, 4, 133, 17]
    cu, hq, hk = cu_of(news), 4, 2
    n = cu[-1]
    q, k, v = normal(1, hq, n, 128), normal(2, hk, n, 128, gain=20.0), normal(3, hk, n, 128)
    m = torch.cat([x.transpose(0, 1) for x in (q, k, v)], 1).contiguous().to(DEV).transpose(0, 1)
    dq, dk, dv = m[:hq], m[hq:hq + hk], m[hq + hk:]
    table, pages = table_of(lens, ps)
    st = b.PagedStoreF8.empty(pages, hk, ps)
    for t in st.tensors().values():
        t.view(torch.uint8).fill_(0x38)  # codes of 1; scales of 4e-5
    angle = angles(200, dim)
    pos = np.concatenate([np.arange(z - x, z) for x, z in zip(news, lens)])
    kr = so.rotate_positions(k, angle, pos, inter)
    want = so.append(arrays_of(st), kr, oracle.as_f64(v), table, lens, cu)
    b.paged_append_f8(dk, dv, st, torch.from_numpy(table).to(DEV), i32(lens), i32(cu), b.Rotation(angle.to(DEV), inter),
                      Q=dq, q_out=dq, k_out=dk)
    b.sync_status()
    assert torch.equal(dk.cpu(), bf16_of(kr)) and torch.equal(dv.cpu(), v)
    rotated_within(dq, q, so.rotate_positions(q, angle, pos, inter))
    got, owned = arrays_of(st), np.zeros((pages, ps), bool)
    for i, x in enumerate(lens):
        if news[i]:
            at = np.arange(x)
            owned[table[i][at[x - news[i]:] // ps], at[x - news[i]:] % ps] = True
    for x in "kv":
        assert np.array_equal(got[x + "_scales"], want[x + "_scales"])
        g, w = (a[x + "_codes"].swapaxes(1, 2)[owned] for a in (got, want))
        assert np.array_equal(g, w)


BAD = [dict(table=[[0, 4], [2, 3]]), dict(table=[[0, -1], [2, 3]]), dict(lens=[65, 3]), dict(lens=[3, 3]),
       dict(lens=[-1, 3]), dict(lens=[40, 1]), dict(lens=[40, 2 ** 31 - 1]), dict(cu=[0, 4, 7]), dict(cu=[0, 7, 6]),
       dict(cu=[-1, 4, 6]), dict(cu=[5, 4, 6]), dict(cu=[0, 4, 3])]


@pytest.mark.parametrize("bad", BAD)
def test_what_a_call_with_bad_indices_leaves_alone(cuda, bad):
    hk, hq, ps, n = 2, 4, 32, 6
    x = dict(dict(table=[[0, 1], [2, 3]], lens=[40, 3], cu=[0, 4, 6]), **bad)
    k, q = normal(1, hk, n, 128), normal(2, hq, n, 128)
    angle = angles(64, 64)
    table, lens, cu = torch.tensor(x["table"], dtype=torch.int32, device=DEV), i32(x["lens"]), i32(x["cu"])
    # the tokens, rows and pages of the sequences whose counts are in range
    tokens = [(i, t, x["lens"][i] - (x["cu"][i + 1] - x["cu"][i]) + t - x["cu"][i]) for i in range(2)
              if 0 <= x["cu"][i] <= x["cu"][i + 1] <= n and x["cu"][i + 1] - x["cu"][i] <= x["lens"][i] <= 64
              for t in range(x["cu"][i], x["cu"][i + 1])]
    rows = sorted({t for _, t, _ in tokens})
    left = [t for t in range(n) if t not in rows]
    pages = sorted({x["table"][i][p // ps] for i, _, p in tokens} & set(range(4)))
    away = [p for p in range(4) if p not in pages]

    st = b.PagedStoreF8.empty(4, hk, ps)
    for t in st.tensors().values():
        t.view(torch.uint8).fill_(0x33)
    qo, ko, out = (torch.full((h, n, 128), 7.0, dtype=torch.bfloat16, device=DEV) for h in (hq, hk, hq))
    lse = torch.full((hq, n), 7.0, device=DEV)

    def reported():
        with pytest.raises(b.H3kvError) as e:
            b.sync_status()
        assert e.value.status == b.H3KV_ERR_DEVICE_DATA
        b.sync_status()

    b.paged_append_f8(k.to(DEV), k.to(DEV), st, table, lens, cu, b.Rotation(angle.to(DEV)), None, q.to(DEV), qo, ko)
    reported()
    for t in st.tensors().values():
        assert (t.view(torch.uint8)[away] == 0x33).all()
    assert (qo[:, left] == 7.0).all() and (ko[:, left] == 7.0).all()
    got = arrays_of(st)
    for i, t, p in tokens:
        page = x["table"][i][p // ps]
        if page in pages:  # this sequence's rows are there
            kr = so.rotate_positions(k, angle, np.full(n, p))
            for h in range(hk):
                for name, want in (("k", kr[h, t]), ("v", oracle.as_f64(k[h, t]))):
                    scale = got[name + "_scales"][page, h]
                    assert np.array_equal(got[name + "_codes"][page, h, p % ps], so._encode(want / scale))
    for page in pages:  # slots behind the last token
        last = max(p % ps for i, _, p in tokens if x["table"][i][p // ps] == page)
        for name in ("k_codes", "v_codes"):
            assert (st.tensors()[name].view(torch.uint8)[page, :, last + 1:] == 0x33).all()
    before = {name: t.clone() for name, t in st.tensors().items()}
    b.attend_paged_f8(q.to(DEV), st, table, lens, cu, out=out, lse=lse)
    reported()
    assert (out[:, left] == 7.0).all() and (lse[:, left] == 7.0).all()
    for name, t in st.tensors().items():
        assert torch.equal(t.view(torch.uint8), before[name].view(torch.uint8))
