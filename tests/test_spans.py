"""Which tensors of a serving call lie over one another: the host's arithmetic
(csrc/spans.h) against marked elements, and the refusals that rest on it."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from store_h3kv_build_gb300 import binding as b

HERE = os.path.dirname(os.path.abspath(__file__))
BAD = b.H3KV_ERR_INVALID_ARG
R = ctypes.byref
P = 1 << 20  # a pointer that is never followed
FAR = 1 << 30


def test_rows_meet_is_exact_for_equal_strides(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "spans_check")
    subprocess.run([cxx, "-std=c++17", "-O2", os.path.join(HERE, "spans_check.cpp"), "-o", exe], check=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "wrong 0" in p.stdout and "cases 2502000" in p.stdout


def rows(ptr, hs=128 * 64, rs=128):
    return R(b.h3kv_rows(ptr, hs, rs))


def store(ptr=FAR, pages=4, heads=2, page=64):
    codes, scales = pages * heads * page * 128, pages * heads * page * 2
    return R(b.h3kv_paged_store(ptr, ptr + codes, ptr + 2 * codes, ptr + 2 * codes + scales, pages, heads, page, 128))


STORE_BYTES = 2 * 4 * 2 * 64 * 130


# (only refusals: a call that passed its checks would go to a GPU)
def test_paged_calls_refuse_outputs_over_other_tensors():
    s = store()
    rd, ap, cp, kp = b.h3kv_paged_read, b.h3kv_paged_append, b.h3kv_paged_copy, b.h3kv_paged_keep
    k = P + (1 << 18)
    for v in (k, k + 16, k + 2 * 504, k - 2 * 128 * 3, k + 2 * (128 * 64 - 120)):
        assert rd(s, P, 4, rows(k), rows(v), None) == BAD, v
    # two that take turns, a row too far (equal strides); unlike strides in one extent
    assert rd(s, P, 4, rows(k, 256, 1024), rows(k + 2 * 256, 256, 1024), None) == BAD
    assert rd(s, P, 4, rows(k, 256, 1024), rows(k + 2 * 128, 384, 1024), None) == BAD
    for inside in (FAR, FAR + STORE_BYTES - 16):
        assert rd(s, P, 4, rows(inside), rows(k), None) == BAD and rd(s, P, 4, rows(k), rows(inside), None) == BAD
        assert ap(rows(inside), rows(k), P, 4, s, None) == BAD and ap(rows(k), rows(inside), P, 4, s, None) == BAD
        assert ap(rows(k), rows(k), inside, 4, s, None) == BAD
        assert cp(s, inside, P, 4, None) == BAD and cp(s, P, inside, 4, None) == BAD
    assert rd(s, k + 8, 4, rows(k), rows(k + (1 << 17)), None) == BAD
    good = [s, P, 4, P + 4096, P + 8192, 3, P + 16384, 4, P + 32768, None]
    for at in (P, P + 44, P + 4096, P + 8192 + 12, P + 16384, FAR, FAR + STORE_BYTES - 4):
        a = list(good)
        a[8] = at
        assert kp(*a) == BAD, at
    for i in (1, 3, 4, 6):
        a = list(good)
        a[i] = FAR + 128
        assert kp(*a) == BAD, i


def test_attention_refuses_outputs_over_other_tensors():
    ws = 1 << 24
    names = ("Q", "table", "lengths", "cu", "parents", "O", "lse", "workspace")
    at = {n: P + (i << 18) for i, n in enumerate(names)}
    at["workspace"] = ws

    def tree(**kw):
        x = dict(at, **kw)
        return b.h3kv_attend_tree(rows(x["Q"]), 4, 8, store(), x["table"], 4, x["lengths"], x["cu"], 3, x["parents"], 0.0,
                                  rows(x["O"]), x["lse"], x["workspace"], 1 << 40, None)

    for n in ("table", "lengths", "cu", "parents", "lse", "workspace"):
        assert tree(O=at[n]) == BAD, n
    for n in ("Q", "table", "lengths", "cu", "parents", "O"):
        assert tree(lse=at[n]) == BAD and tree(workspace=at[n]) == BAD, n
    for inside in (FAR, FAR + STORE_BYTES - 32):
        assert tree(O=inside) == BAD and tree(lse=inside) == BAD and tree(workspace=inside) == BAD

    def prompt(**kw):
        x = dict(at, **kw)
        return b.h3kv_attend_prompt(rows(x["Q"]), 4, 8, rows(x["table"]), rows(x["parents"]), 2, 8, x["lengths"],
                                    x["cu"], 3, 1, 0.0, rows(x["O"]), x["lse"], None)

    for n in ("lengths", "cu", "lse"):
        assert prompt(O=at[n]) == BAD, n
    for n in ("Q", "table", "parents", "lengths", "cu", "O"):
        assert prompt(lse=at[n]) == BAD, n


def test_the_binding_says_what_an_output_shares():
    x = torch.zeros((4, 6, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shares memory with K"):
        b._check_apart(BAD, "h3kv_paged_read", dict(K=x, V=x[:, 1:3]), {})
    with pytest.raises(ValueError, match="shares memory with lengths"):
        b._check_apart(BAD, "h3kv_attend_tree", dict(out=x[:1], lse=None, workspace=x[3]), dict(lengths=x[3]))
    with pytest.raises(b.H3kvError):
        b._check_apart(BAD, "h3kv_paged_read", dict(K=x[:2], V=x[2:]), {})
    with pytest.raises(b.H3kvError):
        b._check_apart(b.H3KV_ERR_CUDA, "h3kv_paged_read", dict(K=x, V=x), {})
    b._check_apart(b.H3KV_OK, "h3kv_paged_read", dict(K=x, V=x), {})


@pytest.mark.gpu
def test_read_into_tensors_that_take_turns_in_one_buffer(cuda):
    heads, ps, n = 3, 32, 50
    st = b.PagedStore.empty(4, heads, ps)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((heads, n, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    at = torch.randperm(4 * ps, generator=g, device="cuda")[:n].to(torch.int32)
    b.paged_append(k, v, st, at)
    want = b.paged_read(st, at)
    for shape, pick in (((n, 2, heads, 128), lambda t, i: t[:, i].transpose(0, 1)),
                        ((n, heads, 2, 128), lambda t, i: t[:, :, i].transpose(0, 1)),
                        ((heads, n, 2, 128), lambda t, i: t[:, :, i]), ((heads, 2, n, 128), lambda t, i: t[:, i]),
                        ((2, heads, n, 128), lambda t, i: t[i])):
        buf = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        got = b.paged_read(st, at, pick(buf, 0), pick(buf, 1))
        b.sync_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    buf = torch.zeros((heads, n + 1, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="shares memory with K"):
        b.paged_read(st, at, buf[:, :n], buf[:, 1:])


@pytest.mark.gpu
def test_attention_into_a_buffer_beside_its_inputs(cuda):
    # one matrix [rows, heads of Q, K, V, O]: through the C ABI (the binding
    # refuses O in the extent of Q)
    hq, hk, n = 4, 2, 150
    g = torch.Generator(device="cuda").manual_seed(1)
    m = torch.randn((n, hq + 2 * hk + hq, 128), generator=g, device="cuda").to(torch.bfloat16)
    t = m.transpose(0, 1)
    q, k, v, o = t[:hq], t[hq:hq + hk], t[hq + hk:hq + 2 * hk], t[hq + 2 * hk:]
    cu = torch.tensor([0, 60, n], dtype=torch.int32, device="cuda")
    want = b.attend_prompt(q, k, v, cu)
    at = [R(b.h3kv_rows(x.data_ptr(), x.stride(0), x.stride(1))) for x in (q, k, v, o)]
    b.check(b.h3kv_attend_prompt(at[0], hq, n, at[1], at[2], hk, n, cu.data_ptr(), cu.data_ptr(), 2, 1, 0.0, at[3], None,
                                 torch.cuda.current_stream().cuda_stream))
    b.sync_status()
    assert torch.equal(o, want)
