"""The serving operators on the GPU against their fp64 oracle: attention over
packed prompts, the paged kvi8r cache, the attention of drafted trees over it.
The attention bounds are element by element, counted from the roundings that
the operators leave to the kernel (oracle/serve.py)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve as so
from parity import compare_store
from store_h3kv_build_gb300 import binding as b
from store_h3kv_build_gb300 import synth
from store_h3kv_build_gb300.paging import PagePool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def cu_of(counts, first=0):
    return [first] + (first + np.cumsum(counts)).tolist()


def normal(seed, *shape, gain=None):
    x = synth.normal_f32(shape, seed)
    if gain is not None:
        x[..., ::32] *= gain
    return x.to(torch.bfloat16)


def within(got, ref, off, what):
    got = got.detach().cpu().double().numpy()
    real = ~np.isnan(ref)
    assert np.array_equal(np.isfinite(got[real]), np.isfinite(ref[real])), f"{what}: infinities differ"
    fin = real & np.isfinite(np.where(real, ref, 0.0))
    err = np.abs(got[fin] - ref[fin])
    over = err > off[fin]
    assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.max(err / off[fin]):.2f} of the bound"


# ----------------------------------------------------------- packed prompts --
def prompt_case(qn, kn, hq, hk, causal=True, seed=0, scale=0.0, layout="head", pad=0, first=0, gain=None):
    rows_q, rows_k = first + sum(qn) + pad, first + sum(kn) + pad
    q, k, v = normal(seed, hq, rows_q, 128), normal(seed + 1, hk, rows_k, 128, gain=gain), normal(seed + 2, hk, rows_k, 128)
    if layout == "token":  # a projection's output: the heads of a token side by side
        dq, dk, dv = (x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for x in (q, k, v))
    elif layout == "fused":  # one matrix [rows, hq + 2 hk, 128]
        assert rows_q == rows_k
        m = torch.cat([x.transpose(0, 1) for x in (q, k, v)], 1).contiguous().to(DEV).transpose(0, 1)
        dq, dk, dv = m[:hq], m[hq:hq + hk], m[hq + hk:]
    else:
        dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    cu_q, cu_k = cu_of(qn, first), cu_of(kn, first)
    lse = torch.full((hq, rows_q), 7.0, device=DEV)
    out = torch.full((hq, rows_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    if layout != "head":
        out = torch.full((rows_q, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    o = b.attend_prompt(dq, dk, dv, i32(cu_q), i32(cu_k), causal=causal, softmax_scale=scale, out=out, lse=lse)
    b.sync_status()
    assert o is out
    ref = so.attend_prompt(q, k, v, cu_q, cu_k, causal, scale if scale > 0 else None)
    what = f"{qn} {kn} {hq}/{hk} causal={causal} {layout}"
    within(out, ref[0], ref[2], what)
    within(lse, ref[1], ref[3], what + " lse")
    outside = np.isnan(ref[1])
    assert (out.cpu().float().numpy()[outside] == 7.0).all() and (lse.cpu().numpy()[outside] == 7.0).all(), what
    return out, lse


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 513, 700])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths(cuda, n, causal):
    prompt_case([n], [n], 2, 1, causal, seed=n)


@pytest.mark.parametrize("n", [128, 129, 255, 256, 257, 385, 513, 640])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths_with_many_heads(cuda, n, causal):
    # enough heads that a CTA owns 256 rows (two row tiles over the same keys)
    prompt_case([n], [n], 160, 4, causal, seed=n)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_packed_with_many_heads(cuda, causal):
    qn, pre = [140, 300, 256, 1, 129], [500, -200, 77, 0, 128]
    prompt_case(qn, [q + p for q, p in zip(qn, pre)], 64, 2, causal, seed=21, layout="token", pad=9)


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (8, 2), (6, 2), (32, 1), (24, 8)])
def test_prompt_head_groups(cuda, hq, hk):
    prompt_case([70, 1, 300], [70, 1, 300], hq, hk, seed=5)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_packed_lengths_behind_prefixes(cuda, causal):
    qn, pre = [1, 128, 37, 0, 260, 5, 129, 1], [500, 0, 91, 12, 256, 0, 127, 0]
    prompt_case(qn, [q + p for q, p in zip(qn, pre)], 4, 2, causal, seed=9, gain=20.0)


def test_prompt_rows_that_see_no_key(cuda):
    # more queries than keys: the first rows see none; a sequence without keys
    for causal in (True, False):
        prompt_case([200, 9, 300, 3], [60, 0, 130, 3], 2, 1, causal, seed=3)


def test_prompt_rows_of_no_sequence_stay(cuda):
    prompt_case([40, 7], [40, 7], 2, 1, seed=4, pad=90, first=3)
    prompt_case([40, 7], [40, 7], 2, 2, seed=4, pad=90, first=300, layout="token")


@pytest.mark.parametrize("layout", ["token", "fused"])
def test_prompt_layouts(cuda, layout):
    prompt_case([150, 33, 290], [150, 33, 290], 6, 2, seed=6, layout=layout)


@pytest.mark.parametrize("scale", [0.02, 0.5, 2.0])
def test_prompt_scales(cuda, scale):
    prompt_case([300, 20], [300, 20], 2, 1, seed=7, scale=scale)


def test_prompt_many_short_sequences(cuda):
    rng = np.random.default_rng(1)
    n = rng.integers(0, 40, 700).tolist()
    prompt_case(n, n, 2, 1, seed=8)


def test_prompt_long(cuda):
    prompt_case([1900], [4100], 3, 1, seed=10)
    prompt_case([1500], [1500], 52, 52, seed=11)


def test_prompt_values_of_other_sequences_do_not_reach(cuda):
    # infinities and NaN in the neighbours' keys and values, and behind the last
    n = [130, 70, 129, 300]
    q, k, v = normal(1, 2, 800, 128), normal(2, 2, 800, 128), normal(3, 2, 800, 128)
    cu = cu_of(n)
    ref = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu))
    for bad in (float("nan"), float("inf")):
        k2, v2 = k.clone(), v.clone()
        for a0, a1 in ((cu[1], cu[2]), (cu[3], 800)):
            k2[:, a0:a1], v2[:, a0:a1] = bad, bad
        out = b.attend_prompt(q.to(DEV), k2.to(DEV), v2.to(DEV), i32(cu))
        b.sync_status()
        for a0, a1 in ((cu[0], cu[1]), (cu[2], cu[3])):
            assert torch.equal(out[:, a0:a1], ref[:, a0:a1])


def shifted(shape, dtype=torch.bfloat16, fill=7.0, by=16):
    """A tensor that starts `by` bytes behind a 512-byte boundary."""
    n, off = int(np.prod(shape)), by // torch.empty((), dtype=dtype).element_size()
    return torch.full((n + off,), fill, dtype=dtype, device=DEV)[off:].view(shape)


def test_sixteen_byte_alignment_is_enough(cuda):
    # outputs and pools 16 bytes off give the bits of aligned ones (their
    # kernels write 32 bytes at a time)
    n = [130, 70, 300]
    q, k, v = (normal(s, 2, 500, 128) for s in (1, 2, 3))
    cu = i32(cu_of(n))
    ref = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), cu)
    off = [shifted(x.shape).copy_(x.to(DEV)) for x in (q, k, v)]
    assert torch.equal(b.attend_prompt(*off, cu, out=shifted(q.shape)), ref)
    tok = shifted((500, 2, 128)).transpose(0, 1)
    assert torch.equal(b.attend_prompt(*off, cu, out=tok), ref)
    st, _ = random_store(6, 2, 64)
    st2 = b.PagedStore(*(shifted(t.shape, t.dtype, 0).copy_(t) for t in st.tensors().values()))
    rows = i32(torch.randperm(384)[:140].tolist())
    for s in (st, st2):
        b.paged_append(k[:, :140].contiguous().to(DEV), v[:, :140].contiguous().to(DEV), s, rows)
    for x, y in zip(st.tensors().values(), st2.tensors().values()):
        assert torch.equal(x, y)
    a = b.paged_read(st, rows)
    c = b.paged_read(st2, rows, shifted((2, 140, 128)), shifted((140, 2, 128)).transpose(0, 1))
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    for nodes, hq in ((2, 4), (8, 4), (64, 8)):
        qq = normal(9, hq, nodes, 128).to(DEV)
        args = i32_2d([[4, 0, 5, 2, 1, 3]]), i32([380]), i32([0, nodes])
        assert torch.equal(b.attend_tree(qq, st, *args), b.attend_tree(qq, st2, *args, out=shifted(qq.shape)))
    b.paged_copy(st, i32([0, 1]), i32([3, 4]))
    b.paged_copy(st2, i32([0, 1]), i32([3, 4]))
    for x, y in zip(st.tensors().values(), st2.tensors().values()):
        assert torch.equal(x, y)
    b.sync_status()


def test_offsets_beyond_31_bits(cuda):
    # the last pages of a pool of 4.3 GB of codes for K (and for V), the last
    # rows of prompts of 4.5 GB
    pages, hk, ps = 1 << 15, 8, 128
    st = b.PagedStore.empty(pages, hk, ps)
    k, v = normal(1, hk, 300, 128), normal(2, hk, 300, 128)
    table = [pages - 1, pages - 3, 0]
    rows = [table[p // ps] * ps + p % ps for p in range(300)]
    b.paged_append(k.to(DEV), v.to(DEV), st, i32(rows))
    b.paged_copy(st, i32([0]), i32([pages - 2]))
    table[2] = pages - 2
    rk, rv = b.paged_read(st, i32([table[p // ps] * ps + p % ps for p in range(300)]))
    part = {n: t[[pages - 1, pages - 3, pages - 2]].cpu() for n, t in st.tensors().items()}
    ref = {n: t.double().numpy() if "scales" in n else t.numpy() for n, t in part.items()}
    for x, back in ((k, rk), (v, rv)):
        codes, scales = oracle.encode_rows(x)
        off = 1.1 * scales[..., None] + 2.0 ** -8 * np.abs(oracle.as_f64(back)) + 1e-6
        within(back, oracle.unrotate(oracle.dequant(codes, scales)), off, "read")
    for hq, nodes in ((8, 1), (16, 7), (32, 60)):
        q = normal(3, hq, nodes, 128)
        out = b.attend_tree(q.to(DEV), st, i32_2d([table]), i32([300]), i32([0, nodes]))
        want = so.attend_tree(q, ref, [[0, 1, 2]], [300], [0, nodes])
        within(out, want[0], want[2], f"tree {nodes}")
    cu, keep = i32([0, 60]), torch.zeros(60, dtype=torch.uint8, device=DEV)
    keep[40:] = 1
    assert b.paged_keep(st, i32_2d([table]), i32([300]), cu, keep).tolist() == [260]
    moved = st.k_codes[table[2], :, :4].cpu()
    assert torch.equal(moved, part["k_codes"][2, :, 40:44])  # tokens 256 .. 259 were nodes 56 .. 59, tokens 296 .. 299
    del st
    n = (1 << 21) + 1000
    q, k, v = (torch.zeros((8, n, 128), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    parts = [normal(s, 8, 400, 128) for s in (4, 5, 6)]
    for t, x in zip((q, k, v), parts):
        t[:, n - 400:] = x.to(DEV)
    out = b.attend_prompt(q, k, v, i32([n - 400, n - 130, n]))
    b.sync_status()
    want = so.attend_prompt(*parts, [0, 270, 400], [0, 270, 400])
    within(out[:, n - 400:], want[0], want[2], "prompt")


def test_prompt_same_bits_wherever_a_sequence_lies(cuda):
    q, k, v = (normal(s, 2, 900, 128).to(DEV) for s in (1, 2, 3))
    alone = b.attend_prompt(q[:, 137:600].contiguous(), k[:, 137:600].contiguous(), v[:, 137:600].contiguous(),
                            i32([0, 463]))
    packed = b.attend_prompt(q, k, v, i32([0, 137, 600, 900]))
    b.sync_status()
    assert torch.equal(alone, packed[:, 137:600])


def test_prompt_largest_scores_and_zero_values(cuda):
    q = torch.zeros((1, 140, 128), dtype=torch.bfloat16)
    q[:, :70] = 300.0
    k, v = normal(2, 1, 140, 128) * 100, normal(3, 1, 140, 128)
    out = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, 140]))
    b.sync_status()
    ref = so.attend_prompt(q, k, v, [0, 140], [0, 140])
    # equal scores: the running mean of v; huge ones: the largest alone
    within(out[:, 70:], ref[0][:, 70:], ref[2][:, 70:], "mean")
    within(out[:, :70], ref[0][:, :70], ref[2][:, :70], "largest")


@pytest.mark.parametrize("cu_q,cu_k", [([0, 50, 40], [0, 50, 60]), ([0, 50, 101], [0, 50, 100]), ([-5, 50], [0, 50]),
                                       ([0, 50], [0, 101]), ([0, 50], [60, 50]), ([0, 50], [-1, 50])])
def test_prompt_counts_out_of_range_are_reported(cuda, cu_q, cu_k):
    q = normal(1, 2, 100, 128).to(DEV)
    b.attend_prompt(q, q, q, i32(cu_q), i32(cu_k))
    with pytest.raises(b.H3kvError) as e:
        b.sync_status()
    assert e.value.status == b.H3KV_ERR_DEVICE_DATA
    b.sync_status()  # cleared
    prompt_case([100], [100], 2, 2)


def test_prompt_empty_calls(cuda):
    q = normal(1, 2, 100, 128).to(DEV)
    assert b.attend_prompt(q[:, :0], q, q, i32([0]), i32([0])).shape == (2, 0, 128)
    out = torch.full_like(q, 3.0)
    b.attend_prompt(q, q[:, :0], q[:, :0], i32([0, 60]), i32([0, 0]), out=out)
    b.sync_status()
    assert (out[:, :60] == 0).all() and (out[:, 60:] == 3.0).all()


# -------------------------------------------------------------- paged cache --
def random_store(pages, heads, ps, seed=0, gain=20.0):
    """Pages filled with quantised rows (oracle), on the GPU and as numpy."""
    k = normal(seed, pages, heads, ps, 128, gain=gain)
    v = normal(seed + 1, pages, heads, ps, 128)
    kc, ks = oracle.encode_rows(k)
    vc, vs = oracle.encode_rows(v)
    ref = {"k_codes": kc, "v_codes": vc, "k_scales": ks, "v_scales": vs}
    st = b.PagedStore(*(torch.from_numpy(ref[n]).to(DEV).to(t) for n, t in
                        (("k_codes", torch.int8), ("v_codes", torch.int8), ("k_scales", torch.float16),
                         ("v_scales", torch.float16))))
    return st, ref


def same_store(st, ref):
    for n, t in ref.items():
        assert np.array_equal(getattr(st, n).cpu().double().numpy(), np.asarray(t, dtype=np.float64)), n


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,n,layout", [(1, 1, "head"), (2, 3, "head"), (8, 37, "token"), (3, 130, "head"),
                                            (5, 200, "token")])
def test_append_and_read(cuda, ps, heads, n, layout):
    pages = -(-n // ps) + 3
    k, v = normal(n, heads, n, 128, gain=20.0), normal(n + 1, heads, n, 128)
    k[0, 0] = 0  # a row of zeros: scale 0, codes 0
    st = b.PagedStore.empty(pages, heads, ps)
    for t in st.tensors().values():
        t.fill_(5)
    g = torch.Generator().manual_seed(n)
    rows = torch.randperm(pages * ps, generator=g)[:n].to(torch.int32)
    if n > 20:
        rows[7] = -1
        rows[20] = -2 ** 31
    put = (lambda x: x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)) if layout == "token" else (lambda x: x.to(DEV))
    b.paged_append(put(k), put(v), st, rows.to(DEV))
    rk, rv = b.paged_read(st, rows.to(DEV))
    b.sync_status()
    live = (rows >= 0).numpy()
    at = rows.long().clamp(min=0)
    for x, name, back in ((k, "k", rk), (v, "v", rv)):
        codes, scales = getattr(st, name + "_codes").cpu(), getattr(st, name + "_scales").cpu()
        c = codes[at // ps, :, at % ps].transpose(0, 1)
        s = scales[at // ps, :, at % ps].transpose(0, 1)
        want = oracle.encode_rows(x)
        few = 1.0 / want[0].size  # a small case may hold one code at a tie
        got = compare_or_one(c[:, live], s[:, live], want[0][:, live], want[1][:, live], few)
        assert got
        touched = torch.zeros(pages * ps, dtype=torch.bool)
        touched[at[torch.from_numpy(live)]] = True
        rest = ~touched.view(pages, ps)
        assert (codes.transpose(1, 2)[rest] == 5).all() and (scales.transpose(1, 2)[rest] == 5).all()
        # reading back: bf16 of the un-rotated fp16(code * scale)
        deq = oracle.fp16_round(oracle.dequant(c.numpy(), s.double().numpy()))
        exp = np.where(live[None, :, None], oracle.unrotate(deq), 0.0)
        off = 2.0 ** -8 * np.abs(exp) * (1 + 2.0 ** -7) + 2.0 ** -20 * np.abs(deq).sum(-1, keepdims=True)
        within(back, exp, off, f"read {name}")


def compare_or_one(codes, scales, ref_codes, ref_scales, few):
    """The store builds' bar (codes off by one at 1e-4 of the entries, scales
    one ulp), or a single code where that is less than one."""
    d = np.abs(codes.numpy().astype(int) - ref_codes.astype(int))
    assert d.max(initial=0) <= 1 and (d != 0).sum() <= max(1, 1e-4 * d.size)
    if few < 1e-4:
        compare_store(codes, scales, ref_codes, ref_scales)
    return True


def test_append_special_rows(cuda):
    k = torch.zeros((1, 6, 128), dtype=torch.bfloat16)
    k[0, 1, 5] = -3.0             # one channel: all codes +-127
    k[0, 2] = 1e-30               # a scale that underflows to 0
    k[0, 3] = 3e38                # a scale that saturates
    k[0, 4, ::2] = 1e-6           # a subnormal scale
    k[0, 5, 0] = float("inf")
    st = b.PagedStore.empty(1, 1, 16)
    b.paged_append(k.to(DEV), k.to(DEV), st, i32(range(6)))
    b.sync_status()
    codes, scales = oracle.encode_rows(k[:, :5])
    # row 3, 128 equal values v: v sqrt(128) in element 0 and 0 exactly in the
    # others, where the oracle's matrix product leaves fp64 rounding residues
    # (about 1e22) that the largest scale 65504 does not bring below 1
    codes[0, 3] = [127] + [0] * 127
    compare_store(st.k_codes[0, :, :5], st.k_scales[0, :, :5], codes, scales)
    assert st.k_scales[0, 0, 5].item() == 65504 and torch.equal(st.k_codes[:, :, :6], st.v_codes[:, :, :6])


def test_append_and_read_rows_out_of_range(cuda):
    st, ref = random_store(3, 2, 16)
    k = normal(1, 2, 4, 128).to(DEV)
    for call in (lambda r: b.paged_append(k, k, st, r), lambda r: b.paged_read(st, r)):
        call(i32([-1, 48, 2 ** 31 - 1, -5]))
        with pytest.raises(b.H3kvError) as e:
            b.sync_status()
        assert e.value.status == b.H3KV_ERR_DEVICE_DATA
        same_store(st, ref)


@pytest.mark.parametrize("n", [1, 15, 17, 128, 131, 400])
def test_read_writes_its_rows_only(cuda, n):
    st, _ = random_store(9, 3, 64)
    rows = torch.randperm(9 * 64, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    rows[n // 2] = -1
    want = b.paged_read(st, rows.to(DEV))
    by_head = torch.full((5, n + 9, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    by_token = torch.full((n + 9, 5, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = by_head[1:4, 5:5 + n], by_token[5:5 + n, 1:4, 64:192].transpose(0, 1)
    got = b.paged_read(st, rows.to(DEV), k, v)
    b.sync_status()
    assert got[0] is k and got[1] is v and torch.equal(k, want[0]) and torch.equal(v, want[1])
    k.fill_(7.0)
    v.fill_(7.0)
    assert (by_head == 7).all() and (by_token == 7).all()


@pytest.mark.parametrize("heads,ps,n", [(1, 16, 1), (8, 64, 3), (3, 32, 7), (32, 128, 2)])
def test_copy_pages(cuda, heads, ps, n):
    st, ref = random_store(2 * n + 2, heads, ps, seed=n)
    order = torch.randperm(2 * n, generator=torch.Generator().manual_seed(n)).tolist()
    src, dst = order[:n], order[n:]
    b.paged_copy(st, i32(src + [-1, 0]), i32(dst + [2 * n, -7]))
    b.sync_status()
    for t in ref.values():
        t[dst] = t[src]
    same_store(st, ref)
    b.paged_copy(st, i32([0, 2 * n + 2]), i32([2 * n + 5, 1]))
    with pytest.raises(b.H3kvError) as e:
        b.sync_status()
    assert e.value.status == b.H3KV_ERR_DEVICE_DATA
    same_store(st, ref)


def tables(lens, ps, seed=0, extra=0):
    need = [-(-n // ps) for n in lens]
    order = torch.randperm(sum(need) + 1, generator=torch.Generator().manual_seed(seed)).tolist()
    t = np.full((len(lens), max(need + [1]) + extra), -1, dtype=np.int64)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + 1


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,nodes", [([1], [1]), ([64], [64]), ([100, 7, 0, 333], [33, 7, 0, 64]),
                                        ([65, 129, 4], [64, 50, 0])])
def test_keep_rows(cuda, ps, lens, nodes):
    t, pages = tables(lens, ps, seed=ps)
    cu = cu_of(nodes)
    for seed, share in ((0, 0.4), (1, 0.0), (2, 1.0), (3, 0.9)):
        st, ref = random_store(pages, 2, ps, seed=seed)
        keep = (torch.rand(sum(nodes), generator=torch.Generator().manual_seed(seed)) < share)
        want, left = so.keep_rows(ref, t, lens, cu, keep.tolist())
        got = b.paged_keep(st, i32_2d(t), i32(lens), i32(cu), (keep if seed else keep.to(torch.uint8)).to(DEV))
        b.sync_status()
        assert got.tolist() == left
        same_store(st, want)


def i32_2d(t):
    return torch.from_numpy(np.asarray(t)).to(torch.int32).to(DEV)


def test_keep_reports_what_is_out_of_range(cuda):
    for lens, nodes, bad in (([40], [65], None), ([10], [11], None), ([65], [3], None), ([-1], [0], None),
                             ([40], [20], -1), ([40], [20], 99)):
        st, ref = random_store(4, 2, 16)
        t = np.array([[0, 1, 2, 3]])
        if bad is not None:
            t[0, 1:] = bad
        nn = max(nodes[0], 1)
        got = b.paged_keep(st, i32_2d(t), i32(lens), i32([0, nodes[0]]),
                           torch.ones(nn, dtype=torch.uint8, device=DEV))
        with pytest.raises(b.H3kvError) as e:
            b.sync_status()
        assert e.value.status == b.H3KV_ERR_DEVICE_DATA
        if bad is None:
            assert got.tolist() == lens
        same_store(st, ref)


# ---------------------------------------------------------- drafted trees --
def random_parents(nodes, seed):
    g = np.random.default_rng(seed)
    out = []
    for m in nodes:
        out += [int(g.integers(-1, j)) if j else -1 for j in range(m)]
    return out


def tree_case(lens, nodes, hq, hk, ps, seed=0, parents="random", scale=0.0, layout="head", first=0, pad=0, gain=20.0):
    t, pages = tables(lens, ps, seed, extra=seed % 3)
    st, ref = random_store(pages, hk, ps, seed=seed, gain=gain)
    cu = cu_of(nodes, first)
    rows = first + sum(nodes) + pad
    q = normal(seed + 5, hq, rows, 128)
    dq = q.to(DEV) if layout == "head" else q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    par = None
    if parents == "random":
        par = [-1] * first + random_parents(nodes, seed) + [-1] * pad
    out = torch.full((hq, rows, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((hq, rows), 7.0, device=DEV)
    o = b.attend_tree(dq, st, i32_2d(t), i32(lens), i32(cu), None if par is None else i32(par), softmax_scale=scale,
                      out=out, lse=lse)
    b.sync_status()
    assert o is out
    want = so.attend_tree(q, ref, t, lens, cu, par, scale if scale > 0 else None)
    what = f"{lens} {nodes} {hq}/{hk} page {ps}"
    within(out, want[0], want[2], what)
    within(lse, want[1], want[3], what + " lse")
    outside = np.isnan(want[1])
    assert (out.cpu().float().numpy()[outside] == 7.0).all() and (lse.cpu().numpy()[outside] == 7.0).all()
    return out


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 640, 1000])
def test_tree_one_token(cuda, ps, n):
    tree_case([n], [1], 4, 2, ps, seed=n, parents=None)


@pytest.mark.parametrize("m", [1, 2, 5, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("n", [0, 1, 63, 127, 128, 300])
def test_tree_nodes_across_tiles(cuda, m, n):
    tree_case([n + m], [m], 4, 2, 32, seed=m + n)
    tree_case([n + m], [m], 2, 2, 64, seed=m + n, parents=None)


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (8, 1), (6, 2), (24, 8), (32, 8), (64, 1), (5, 5)])
def test_tree_head_groups(cuda, hq, hk):
    tree_case([200, 77, 390], [3, 64, 17], hq, hk, 64, seed=hq)


def test_tree_batches_of_unlike_lengths(cuda):
    lens = [5, 2000, 1, 130, 0, 3000, 64, 700, 128, 129, 2, 40]
    nodes = [5, 3, 1, 64, 0, 1, 10, 2, 0, 64, 2, 7]
    tree_case(lens, nodes, 8, 2, 64, seed=2)
    tree_case(lens, nodes, 8, 8, 16, seed=3, layout="token", first=2, pad=5)


def test_tree_many_sequences(cuda):
    g = np.random.default_rng(4)
    lens = g.integers(1, 90, 600).tolist()
    nodes = [int(g.integers(0, min(n, 4) + 1)) for n in lens]
    tree_case(lens, nodes, 2, 1, 16, seed=6)


def test_tree_many_sequences_of_many_rows(cuda):
    g = np.random.default_rng(5)
    lens = g.integers(10, 120, 620).tolist()
    nodes = [int(g.integers(5, min(n, 14) + 1)) for n in lens]
    tree_case(lens, nodes, 4, 1, 16, seed=6)


@pytest.mark.parametrize("hq,hk", [(4, 1), (32, 1), (19, 1), (8, 2)])
def test_tree_between_few_and_many_rows(cuda, hq, hk):
    # a mean of 17 to 32 rows a sequence and kv head: items of 32 rows, some
    # sequences with many of them
    g = np.random.default_rng(hq)
    n = 40 if hq < 16 else 12
    lens = g.integers(64, 700, n).tolist()
    nodes = [int(g.integers(1, 9)) for _ in lens] if hq < 16 else [1] * n
    nodes[3], nodes[7] = (64, 0) if hq < 16 else (1, 0)
    mean = sum(nodes) * (hq // hk) / n
    assert 16 < mean <= 32
    tree_case(lens, nodes, hq, hk, 32, seed=hq)
    tree_case([30000], [32 // (hq // hk)], hq, hk, 64, seed=9)


def test_tree_long_cache(cuda):
    tree_case([30000], [4], 4, 1, 64, seed=7)
    tree_case([9000, 11000], [1, 64], 8, 1, 128, seed=8)


@pytest.mark.parametrize("scale", [0.01, 0.3])
def test_tree_scales(cuda, scale):
    tree_case([300, 45], [20, 5], 4, 2, 32, seed=9, scale=scale, gain=None)


def test_tree_parents_that_name_no_earlier_node_are_roots(cuda):
    st, ref = random_store(4, 1, 32)
    q = normal(3, 2, 6, 128)
    par = [5, 1, 0, -9, 2 ** 31 - 1, 4]
    out = b.attend_tree(q.to(DEV), st, i32_2d([[2, 0, 1]]), i32([70]), i32([0, 6]), i32(par))
    b.sync_status()
    want = so.attend_tree(q, ref, [[2, 0, 1]], [70], [0, 6], par)
    within(out, want[0], want[2], "roots")


def test_tree_same_bits_again(cuda):
    st, _ = random_store(60, 2, 64)
    q = normal(1, 8, 70, 128).to(DEV)
    t, n, cu = i32_2d([list(range(30)), list(range(30, 60))]), i32([1900, 1700]), i32([0, 60, 70])
    a = b.attend_tree(q, st, t, n, cu)
    for _ in range(5):
        assert torch.equal(a, b.attend_tree(q, st, t, n, cu))
    b.sync_status()


def test_tree_workspace_holds_anything(cuda):
    # fewer units of work than CTAs, a workspace full of NaN
    st, ref = random_store(20, 2, 64)
    q = normal(1, 4, 1, 128)
    t = [list(range(16))]
    ws = torch.full((int(b.h3kv_attend_tree_workspace_bytes(4, 2, 1, 1)),), 255, dtype=torch.uint8, device=DEV)
    out = b.attend_tree(q.to(DEV), st, i32_2d(t), i32([1000]), i32([0, 1]), workspace=ws)
    b.sync_status()
    want = so.attend_tree(q, ref, t, [1000], [0, 1])
    within(out, want[0], want[2], "workspace")


def test_tree_rows_behind_the_length_do_not_reach(cuda):
    # what the free rows of the last page, and pages of others, hold
    st, _ = random_store(4, 2, 64)
    q = normal(1, 4, 3, 128).to(DEV)
    args = (i32_2d([[1, 3]]), i32([100]), i32([0, 3]))
    a = b.attend_tree(q, st, *args)
    st.k_scales[3, :, 36:] = float("nan")
    st.v_scales[3, :, 36:] = float("inf")
    for p in (0, 2):
        st.k_scales[p], st.v_scales[p] = float("nan"), float("nan")
    c = b.attend_tree(q, st, *args)
    b.sync_status()
    assert torch.equal(a, c)


@pytest.mark.parametrize("table,n,cu", [([[0, 9]], [20], [0, 3]), ([[0, -1]], [20], [0, 3]), ([[0, 1]], [33], [0, 3]),
                                        ([[0, 1]], [2], [0, 3]), ([[0, 1]], [-4], [0, 0]), ([[0, 1]], [20], [0, 5]),
                                        ([[0, 1]], [20], [-1, 2]), ([[0, 1]], [20], [2, 1])])
def test_tree_reports_what_is_out_of_range(cuda, table, n, cu):
    st, ref = random_store(4, 2, 16)
    q = normal(1, 4, 3, 128).to(DEV)
    b.attend_tree(q, st, i32_2d(table), i32(n), i32(cu))
    with pytest.raises(b.H3kvError) as e:
        b.sync_status()
    assert e.value.status == b.H3KV_ERR_DEVICE_DATA
    b.sync_status()
    tree_case([20], [3], 4, 2, 16)


def test_tree_more_nodes_than_allowed_is_reported(cuda):
    st, _ = random_store(4, 2, 64)
    b.attend_tree(normal(1, 4, 70, 128).to(DEV), st, i32_2d([[0, 1]]), i32([100]), i32([0, 65]))
    with pytest.raises(b.H3kvError) as e:
        b.sync_status()
    assert e.value.status == b.H3KV_ERR_DEVICE_DATA


# ---------------------------------------------------------- used together --
def test_a_prompt_then_drafts(cuda):
    """A prompt is attended and cached, drafts are appended, attended as trees
    and partly kept, a sequence is forked, and its chunked continuation reads
    the cached prefix back."""
    hq, hk, ps = 4, 2, 32
    pool = PagePool(24, ps)
    st = b.PagedStore.empty(24, hk, ps)
    a, c = pool.new(), pool.new()
    kept = {a: [], c: []}  # bf16 K, V of every token that is left, per sequence

    def put(seqs, counts, seed):
        k, v = normal(seed, hk, sum(counts), 128), normal(seed + 1, hk, sum(counts), 128)
        rows, at = [], 0
        for s, n in zip(seqs, counts):
            r, pairs = pool.extend(s, n)
            if pairs:
                b.paged_copy(st, i32(x for x, _ in pairs), i32(y for _, y in pairs))
            rows.append(r)
            kept[s] += [(k[:, at + j], v[:, at + j]) for j in range(n)]
            at += n
        b.paged_append(k.to(DEV), v.to(DEV), st, torch.cat(rows).to(DEV))
        return k, v

    prompt = [150, 41]
    k, v = put([a, c], prompt, 1)
    q = normal(9, hq, sum(prompt), 128)
    out = b.attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu_of(prompt)))
    b.sync_status()
    want = so.attend_prompt(q, k, v, cu_of(prompt), cu_of(prompt))
    within(out, want[0], want[2], "prompt")

    def as_store():
        return {n: t.cpu().double().numpy() if "scales" in n else t.cpu().numpy()
                for n, t in (("k_codes", st.k_codes), ("v_codes", st.v_codes), ("k_scales", st.k_scales),
                             ("v_scales", st.v_scales))}

    def draft(seqs, nodes, seed):
        put(seqs, nodes, seed)
        cu, par = cu_of(nodes), random_parents(nodes, seed)
        q = normal(seed + 2, hq, sum(nodes), 128)
        args = pool.table(seqs).to(DEV), pool.lengths(seqs).to(DEV), i32(cu)
        out = b.attend_tree(q.to(DEV), st, *args, i32(par))
        b.sync_status()
        want = so.attend_tree(q, as_store(), pool.table(seqs).numpy(), pool.lengths(seqs).tolist(), cu, par)
        within(out, want[0], want[2], "drafts")
        keep = torch.rand(sum(nodes), generator=torch.Generator().manual_seed(seed)) < 0.5
        left = b.paged_keep(st, *args, keep.to(DEV)).tolist()
        for i, s in enumerate(seqs):
            base = len(kept[s]) - nodes[i]
            new = [kept[s][base + j] for j in range(nodes[i]) if keep[cu[i] + j]]
            kept[s] = kept[s][:base] + new
            assert left[i] == len(kept[s])
            pool.truncate(s, left[i])

    def cache_holds():
        for s in pool.sequences():
            rk, rv = b.paged_read(st, pool.rows(s).to(DEV))
            for got, x in ((rk, 0), (rv, 1)):
                rows = torch.stack([t[x] for t in kept[s]], 1)
                codes, scales = oracle.encode_rows(rows)
                # a code of the build may be one off, and the result is bf16
                off = 1.1 * scales[..., None] + 2.0 ** -8 * np.abs(oracle.as_f64(got)) + 1e-6
                within(got, oracle.unrotate(oracle.dequant(codes, scales)), off, "cache")

    draft([a, c], [12, 3], 20)
    cache_holds()
    f = pool.fork(a)
    kept[f] = list(kept[a])
    draft([a, c, f], [30, 1, 64], 30)
    cache_holds()
    pool.free(c)
    del kept[c]
    pairs = pool.compact()
    if pairs:
        b.paged_copy(st, i32(x for x, _ in pairs), i32(y for _, y in pairs))
    draft([f, a], [5, 7], 40)
    cache_holds()
    # a chunk of the prompt behind its cached prefix, read back
    n = pool.length(f)
    pk, pv = b.paged_read(st, pool.rows(f).to(DEV))
    k, v = normal(50, hk, 70, 128).to(DEV), normal(51, hk, 70, 128).to(DEV)
    q = normal(52, hq, 70, 128)
    ck, cv = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
    out = b.attend_prompt(q.to(DEV), ck, cv, i32([0, 70]), i32([0, n + 70]))
    b.sync_status()
    want = so.attend_prompt(q, ck, cv, [0, 70], [0, n + 70])
    within(out, want[0], want[2], "chunk")


def test_serving_step_replays_from_a_graph(cuda):
    """One decoding step (append, attend, keep) captured once and replayed on
    new rows, lengths and tables, with an entry left out in one replay."""
    hq, hk, ps, nseq = 4, 2, 32, 3
    st, _ = random_store(12, hk, ps)
    st2 = b.PagedStore(*(t.clone() for t in st.tensors().values()))
    q, k, v = normal(1, hq, 6, 128).to(DEV), normal(2, hk, 6, 128).to(DEV), normal(3, hk, 6, 128).to(DEV)
    table = i32_2d([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    lens, cu, rows, keep = i32([20, 33, 70]), i32([0, 1, 3, 6]), i32([0] * 6), torch.ones(6, dtype=torch.uint8, device=DEV)
    out, left = torch.zeros_like(q), torch.zeros_like(lens)
    ws = torch.empty(int(b.h3kv_attend_tree_workspace_bytes(hq, hk, 6, nseq)), dtype=torch.uint8, device=DEV)

    def step(s):
        b.paged_append(k, v, s, rows)
        b.attend_tree(q, s, table, lens, cu, out=out, workspace=ws)
        b.paged_keep(s, table, lens, cu, keep, out=left)

    def rows_of(ls):
        t, r, c = table.cpu(), [], [0, 1, 3, 6]
        for i, n in enumerate(ls):
            r += [int(t[i, p // ps]) * ps + p % ps for p in range(n - (c[i + 1] - c[i]), n)]
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rows.copy_(i32(rows_of([20, 33, 70])))
    before = [t.clone() for t in st.tensors().values()]
    with torch.cuda.stream(side):
        step(st)
    torch.cuda.current_stream().wait_stream(side)
    b.sync_status()
    for t, o in zip(st.tensors().values(), before):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(st)
    for seed, ls in ((1, [20, 33, 70]), (2, [1, 2, 3]), (3, [96, 64, 33])):
        for t, s in ((q, seed), (k, seed + 10), (v, seed + 20)):
            t.copy_(normal(s, *t.shape))
        r = rows_of(ls)
        if seed == 2:
            r[1] = -1
        rows.copy_(i32(r))
        lens.copy_(i32(ls))
        keep.copy_(torch.tensor([1, 0, 1, 0, 1, 1], dtype=torch.uint8))
        g.replay()
        b.sync_status()
        got = out.clone(), left.clone()
        step(st2)
        b.sync_status()
        assert torch.equal(got[0], out) and torch.equal(got[1], left)
        for x, y in zip(st.tensors().values(), st2.tensors().values()):
            assert torch.equal(x, y)


def test_prompt_replays_from_a_graph(cuda):
    q, k, v = normal(1, 40, 900, 128).to(DEV), normal(2, 4, 900, 128).to(DEV), normal(3, 4, 900, 128).to(DEV)
    cu, out = i32([0, 300, 900]), torch.zeros_like(q)
    b.attend_prompt(q, k, v, cu, out=out)
    b.sync_status()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.attend_prompt(q, k, v, cu, out=out)
    for seed, c in ((4, [0, 300, 900]), (5, [0, 899, 900]), (6, [10, 11, 500])):
        q.copy_(normal(seed, 40, 900, 128))
        cu.copy_(i32(c))
        g.replay()
        b.sync_status()
        got = out.clone()
        assert torch.equal(b.attend_prompt(q, k, v, cu)[:, c[0]:c[2]], got[:, c[0]:c[2]])


def test_withheld_arrivals_run_into_the_wait_limit(cuda):
    """Each attention kernel of the serving operators with one arrival left
    out: its bounded wait runs out, the status says so, and the context and
    the next call are sound."""
    st, _ = random_store(40, 8, 128)
    t = i32_2d([list(range(40))])
    q = normal(1, 8, 1500, 128).to(DEV)
    qt = {n: normal(2, 64, n, 128).to(DEV) for n in (1, 2, 4, 40)}
    calls = [lambda: b.attend_prompt(q, q, q, i32([0, 1500])),
             lambda: b.attend_tree(qt[40], st, t, i32([5000]), i32([0, 40]))]
    # the kernels for few rows wait for a freed stage, which takes more tiles
    # than stages on a CTA: many sequences over the same pages
    many = 24
    for n in (1, 2, 4):
        qm = qt[n].repeat(1, many, 1)
        calls.append(lambda qm=qm, n=n: b.attend_tree(qm, st, t.expand(many, 40).contiguous(), i32([5000] * many),
                                                      i32(range(0, many * n + 1, n))))
    try:
        for call in calls:
            want = call()
            b.sync_status()
            assert b.h3kv_set_wait_timeout_ns(2_000_000) == b.H3KV_OK
            assert b.h3kv_debug_withhold_p(1) == b.H3KV_OK
            call()
            with pytest.raises(b.H3kvError) as e:
                b.sync_status()
            assert e.value.status == b.H3KV_ERR_DEVICE_TIMEOUT
            assert b.h3kv_debug_withhold_p(-1) == b.H3KV_OK
            assert b.h3kv_set_wait_timeout_ns(0) == b.H3KV_OK
            assert torch.equal(call(), want)
            b.sync_status()
    finally:
        b.h3kv_debug_withhold_p(-1)
        b.h3kv_set_wait_timeout_ns(0)


def test_calls_on_two_streams_at_once(cuda):
    st, _ = random_store(40, 2, 64)
    q = [normal(s, 8, 40, 128).to(DEV) for s in (1, 2)]
    p = [normal(s, 4, 1500, 128).to(DEV) for s in (3, 4)]
    t, n, cu = i32_2d([list(range(20)), list(range(20, 40))]), i32([1280, 1111]), i32([0, 20, 40])
    cp = i32([0, 700, 1500])
    want = [(b.attend_tree(q[i], st, t, n, cu), b.attend_prompt(p[i], p[i], p[i], cp)) for i in (0, 1)]
    b.sync_status()
    ss = [torch.cuda.Stream() for _ in (0, 1)]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append((b.attend_tree(q[i], st, t, n, cu, stream=ss[i]),
                           b.attend_prompt(p[i], p[i], p[i], cp, stream=ss[i])))
    for s in ss:
        b.sync_status(s)
    for i in (0, 1):
        for x, y in got[i]:
            assert torch.equal(x, want[i][0]) and torch.equal(y, want[i][1])
