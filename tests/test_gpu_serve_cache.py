"""The paged cache where its rows are unusual: NaN, infinities, subnormal scales
and few rows at a time."""
import numpy as np
import pytest
import torch

import oracle
from store_h3kv_build_gb300 import binding as b
from store_h3kv_build_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def normal(seed, *shape):
    return synth.normal_f32(shape, seed).to(torch.bfloat16)


def empty_store(pages, heads, ps, fill=5):
    st = b.PagedStore.empty(pages, heads, ps)
    for t in st.tensors().values():
        t.fill_(fill)
    return st


@pytest.mark.parametrize("n", [1, 7, 300])
def test_rows_that_hold_a_nan_read_back_as_nan(cuda, n):
    heads, ps = 2, 32
    k, v = normal(1, heads, n, 128), normal(2, heads, n, 128)
    bad = list(range(0, n, 3))
    for j, i in enumerate(bad):
        k[j % 2, i, (37 * j) % 128] = float("nan")
        v[1 - j % 2, i] = float("nan")
    pages = -(-n // ps)
    st = empty_store(pages, heads, ps)
    b.paged_append(k.to(DEV), v.to(DEV), st, torch.arange(n, dtype=torch.int32, device=DEV))
    rk, rv = b.paged_read(st, torch.arange(n, dtype=torch.int32, device=DEV))
    b.sync_status()
    for x, back in ((k, rk.cpu()), (v, rv.cpu())):
        nan = x.isnan().any(-1)
        assert back[nan].isnan().all() and not back[~nan].isnan().any()
        # half a code of the row's scale in each of 128 rotated values, and bf16
        ref = x.float()[~nan]
        scale = torch.from_numpy(oracle.encode_rows(x.nan_to_num(0.0))[1]).float()[~nan]
        off = 0.6 * scale[:, None] * 128 ** 0.5 + 2.0 ** -8 * ref.abs() + 1e-6
        assert ((back.float()[~nan] - ref).abs() <= off).all()


@pytest.mark.parametrize("nodes,hq", [(1, 2), (8, 4), (40, 8)])
def test_attention_over_a_nan_row_is_nan(cuda, nodes, hq):
    # and another sequence's is not
    heads, ps, n = 2, 32, 200
    k, v = normal(1, heads, 2 * 224, 128), normal(2, heads, 2 * 224, 128)
    k[:, 70, 3] = float("nan")
    st = empty_store(14, heads, ps)
    b.paged_append(k.to(DEV), v.to(DEV), st, torch.arange(448, dtype=torch.int32, device=DEV))
    q = normal(3, hq, 2 * nodes, 128)
    out = b.attend_tree(q.to(DEV), st, i32([list(range(7)), list(range(7, 14))]), i32([n, n]), i32([0, nodes, 2 * nodes]))
    b.sync_status()
    assert out[:, :nodes].isnan().all() and out[:, nodes:].isfinite().all()


@pytest.mark.parametrize("pair", [(0.000469207763671875, 1.8253922462463379e-06), (0.023193359375, 0.00022983551025390625),
                                  (0.0233154296875, 0.00010776519775390625)])
def test_subnormal_scales_next_to_a_tie(cuda, pair):
    # (v1 + v2) / (sqrt(128) 127) rounds to an fp32 value halfway between two
    # subnormal fp16 ones, and lies 5e-8 or 2e-8 of itself below that: fp64
    # tells the side
    k = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    k[0, 0, 0], k[0, 0, 1] = pair
    assert tuple(k[0, 0, :2].tolist()) == pair
    st = empty_store(1, 1, 16)
    b.paged_append(k.to(DEV), -k.to(DEV), st, i32([3]))
    b.sync_status()
    want = oracle.encode_rows(k)[1].item()
    assert 0 < want < 2 ** -14
    assert st.k_scales[0, 0, 3].item() == want and st.v_scales[0, 0, 3].item() == want


@pytest.mark.parametrize("heads,n", [(1, 1), (2, 3), (8, 16)])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 3e3])
def test_append_of_few_rows_writes_the_scales(cuda, heads, n, size):
    # rows without zeros, scales to one fp16 step of the oracle's, codes to one
    # of theirs under the stored scale; every other row stays as it was
    ps = 16
    k, v = (normal(s, heads, n, 128).mul_(size) for s in (10 + n, 20 + n))
    st = empty_store(3, heads, ps)
    rows = torch.randperm(3 * ps, generator=torch.Generator().manual_seed(n))[:n]
    b.paged_append(k.to(DEV), v.to(DEV), st, rows.to(torch.int32).to(DEV))
    b.sync_status()
    for x, name in ((k, "k"), (v, "v")):
        codes, scales = getattr(st, name + "_codes").cpu(), getattr(st, name + "_scales").cpu()
        got = scales[rows // ps, :, rows % ps].T.double().numpy()
        want = oracle.encode_rows(x)[1]
        step = np.spacing(want.astype(np.float16)).astype(np.float64)
        assert (want > 0).all() and (np.abs(got - want) <= step).all()
        ref = oracle.quantize(oracle.rotate(x), got)
        assert np.abs(codes[rows // ps, :, rows % ps].transpose(0, 1).numpy().astype(int) - ref).max() <= 1
        rest = torch.ones(3 * ps, dtype=torch.bool)
        rest[rows] = False
        rest = rest.view(3, ps)
        assert (codes.transpose(1, 2)[rest] == 5).all() and (scales.transpose(1, 2)[rest] == 5).all()


@pytest.mark.parametrize("size", [1.0, 1e-4])
def test_append_beside_the_store_build(cuda, size):
    """The pages hold the format of h3kv_build_store, whose scales and codes
    may differ by a rounding: one fp16 step of a scale, one code."""
    heads, n, ps = 4, 4096, 64
    k, v = normal(1, heads, n, 128) * size, normal(2, heads, n, 128) * size
    k[..., ::32] *= 20
    whole = b.build_store(k.to(DEV), v.to(DEV))
    st = b.PagedStore.empty(n // ps, heads, ps)
    b.paged_append(k.to(DEV), v.to(DEV), st, torch.arange(n, dtype=torch.int32, device=DEV))
    b.sync_status()
    for name in ("k", "v"):
        c = getattr(st, name + "_codes").transpose(0, 1).reshape(heads, n, 128).int()
        s = getattr(st, name + "_scales").transpose(0, 1).reshape(heads, n)
        c0, s0 = getattr(whole, name + "_codes").int(), getattr(whole, name + "_scales")
        bits, bits0 = s.view(torch.int16).int(), s0.view(torch.int16).int()
        assert (bits - bits0).abs().max() <= 1 and (bits != bits0).sum() <= 1e-3 * bits.numel()
        same = bits == bits0
        d = (c - c0).abs()[same]
        assert d.max() <= 1 and (d != 0).sum() <= 1e-4 * d.numel()
