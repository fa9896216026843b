"""The serving operators' refusals, on the CPU: every declared entry point is
exported, and bad arguments are refused on the host before any launch, by the
C ABI and by the binding."""
import ctypes
import os
import re

import pytest
import torch

from store_h3kv_build_gb300 import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096  # a pointer that is never followed
BAD, OK, UNS = b.H3KV_ERR_INVALID_ARG, b.H3KV_OK, b.H3KV_ERR_UNSUPPORTED


def rows(ptr=P, hs=128 * 64, rs=128):
    return b.h3kv_rows(ptr, hs, rs)


def store(ptr=P, pages=4, heads=2, page=64, dim=128):
    return b.h3kv_paged_store(ptr, ptr, ptr, ptr, pages, heads, page, dim)


R = ctypes.byref


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "h3kv_serve.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(h3kv_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 8
    lib = ctypes.CDLL(b.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert set(names) <= set(b.EXPORTED)
    assert b.h3kv_strerror(b.H3KV_ERR_DEVICE_DATA).startswith(b"an index array")


def test_sizes():
    assert b.h3kv_paged_store_bytes(10, 8, 64, 128) == 2 * 10 * 8 * 64 * 130
    for bad in ((-1, 8, 64, 128), (10, -1, 64, 128), (10, 8, 48, 128), (10, 8, 64, 64), (1 << 25, 1, 64, 128)):
        assert b.h3kv_paged_store_bytes(*bad) == 0
    ws = b.h3kv_attend_tree_workspace_bytes
    assert ws(32, 8, 64, 4) >= 16
    assert ws(32, 0, 1, 1) == 0 and ws(33, 8, 1, 1) == 0 and ws(65, 1, 1, 1) == 0 and ws(8, 8, -1, 1) == 0


@pytest.mark.parametrize("st,want", [(store(page=48), BAD), (store(pages=-1), BAD), (store(heads=-1), BAD),
                                     (store(dim=64), UNS), (store(ptr=0), BAD), (store(ptr=P + 8), BAD),
                                     (store(pages=1 << 25), BAD), (store(heads=65536), BAD), (None, BAD)])
def test_paged_stores_that_are_refused(st, want):
    s = R(st) if st is not None else None
    assert b.h3kv_paged_append(R(rows()), R(rows()), P, 4, s, None) == want
    assert b.h3kv_paged_read(s, P, 4, R(rows()), R(rows()), None) == want
    assert b.h3kv_paged_copy(s, P, P, 4, None) == want
    assert b.h3kv_paged_keep(s, P, 4, P, P, 1, P, 4, P + 64, None) == want
    assert b.h3kv_attend_tree(R(rows()), 4, 4, s, P, 4, P, P, 1, None, 0.0, R(rows()), None, P, 1 << 40,
                              None) == want


def test_append_and_read_refusals():
    s = R(store())
    ap, rd = b.h3kv_paged_append, b.h3kv_paged_read
    for bad in (rows(0), rows(P + 8), rows(rs=64), rows(rs=132), rows(hs=0), rows(hs=129), rows(rs=0)):
        assert ap(R(bad), R(rows()), P, 4, s, None) == BAD
        assert ap(R(rows()), R(bad), P, 4, s, None) == BAD
        assert rd(s, P, 4, R(bad), R(rows()), None) == BAD
        assert rd(s, P, 4, R(rows()), R(bad), None) == BAD
    assert rd(s, P, 4, R(rows(hs=256)), R(rows()), None) == BAD       # output heads lie over each other
    assert ap(R(rows()), R(rows()), 0, 4, s, None) == BAD
    assert ap(R(rows()), R(rows()), P + 2, 4, s, None) == BAD
    assert ap(R(rows()), R(rows()), P, -1, s, None) == BAD
    assert ap(None, None, 0, 0, s, None) == OK and rd(s, 0, 0, None, None, None) == OK
    assert ap(None, None, 0, 4, R(store(heads=0, ptr=0)), None) == OK


def test_copy_and_keep_refusals():
    s = R(store())
    cp, kp = b.h3kv_paged_copy, b.h3kv_paged_keep
    assert cp(s, 0, P, 4, None) == BAD and cp(s, P, 0, 4, None) == BAD and cp(s, P, P, -1, None) == BAD
    assert cp(s, P + 1, P, 4, None) == BAD and cp(s, 0, 0, 0, None) == OK
    good = [s, P, 4, P, P, 3, P, 4, P + 64, None]
    for at, v in ((1, 0), (2, -1), (3, 0), (4, 0), (5, -1), (5, 65536), (6, 0), (7, -1), (8, 0), (8, P), (8, P + 8),
                  (8, P - 8), (3, P + 2)):
        a = list(good)
        a[at] = v
        assert kp(*a) == BAD, (at, v)
    a = list(good)
    a[5] = 0
    assert kp(*a) == OK


def test_attend_tree_refusals():
    good = [R(rows()), 4, 8, R(store()), P, 4, P, P, 3, None, 0.0, R(rows()), None, P, 1 << 40, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return b.h3kv_attend_tree(*a)

    assert call(_0=None) == BAD and call(_0=R(rows(0))) == BAD and call(_0=R(rows(rs=100))) == BAD
    assert call(_1=5) == BAD and call(_1=-4) == BAD and call(_1=65536) == BAD
    assert call(_1=130) == BAD                                    # 65 query heads for each kv head
    assert call(_2=-1) == BAD and call(_2=1 << 31) == BAD
    assert call(_3=R(store(heads=0))) == BAD and call(_3=R(store(pages=0))) == BAD
    assert call(_4=0) == BAD and call(_5=-1) == BAD and call(_5=0) == BAD
    assert call(_6=0) == BAD and call(_7=0) == BAD and call(_8=-1) == BAD and call(_8=65536) == BAD
    assert call(_9=P + 1) == BAD and call(_11=None) == BAD and call(_11=R(rows(hs=256))) == BAD
    assert call(_12=P + 1) == BAD and call(_13=0) == BAD and call(_13=P + 8) == BAD
    assert call(_14=b.h3kv_attend_tree_workspace_bytes(4, 2, 8, 3) - 1) == BAD
    assert call(_2=0) == OK and call(_8=0) == OK


def test_attend_prompt_refusals():
    good = [R(rows()), 4, 8, R(rows()), R(rows()), 2, 8, P, P, 3, 1, 0.0, R(rows()), None, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return b.h3kv_attend_prompt(*a)

    for at in ("_0", "_3", "_4", "_12"):
        for bad in (None, rows(0), rows(P + 2), rows(rs=64), rows(hs=64), rows(rs=129)):
            assert call(**{at: R(bad) if bad is not None else None}) == BAD, at
    assert call(_12=R(rows(hs=256))) == BAD
    assert call(_1=5) == BAD and call(_1=-2) == BAD and call(_1=65536) == BAD and call(_5=0) == BAD
    assert call(_2=-1) == BAD and call(_6=-1) == BAD and call(_2=1 << 30) == BAD and call(_6=1 << 31) == BAD
    assert call(_7=0) == BAD and call(_8=0) == BAD and call(_7=P + 2) == BAD
    assert call(_9=-1) == BAD and call(_9=65536) == BAD and call(_13=P + 2) == BAD
    assert call(_2=0) == OK and call(_9=0) == OK and call(_1=0) == OK


# ------------------------------------------------------------- the binding --
def _store(pages=4, heads=2, page=16):
    return b.PagedStore.empty(pages, heads, page, device="cpu")


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_paged_store_shapes():
    assert _store().nbytes() == 2 * 4 * 2 * 16 * 130
    with pytest.raises(ValueError, match="page_size"):
        _store(page=24)
    c, s = torch.zeros((4, 2, 16, 128), dtype=torch.int8), torch.zeros((4, 2, 16), dtype=torch.float16)
    with pytest.raises(ValueError, match="v_codes"):
        b.PagedStore(c, c[:3], s, s)
    with pytest.raises(TypeError, match="k_scales"):
        b.PagedStore(c, c, s.float(), s)
    with pytest.raises(ValueError, match="k_codes"):
        b.PagedStore(c[0], c, s, s)
    with pytest.raises(ValueError, match="contiguous"):
        b.PagedStore(c, c.transpose(0, 1).contiguous().transpose(0, 1), s, s)


def test_binding_refuses_strides_types_and_shapes():
    st = _store()
    k = _bf(2, 5, 128)
    with pytest.raises(TypeError, match="K: dtype"):
        b.paged_append(k.float(), k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="K: 3 heads"):
        b.paged_append(_bf(3, 5, 128), k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="V: 4 rows"):
        b.paged_append(k, _bf(2, 4, 128), st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="last dimension"):
        b.paged_append(_bf(2, 128, 128).transpose(1, 2), _bf(2, 128, 128), st, _i(*range(128)))
    with pytest.raises(ValueError, match="stride"):
        b.paged_append(_bf(1, 5, 128).expand(2, 5, 128), k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="stride"):
        b.paged_append(_bf(2, 5, 132)[..., :128], k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="aligned"):
        b.paged_append(_bf(2 * 5 * 128 + 4)[4:].view(2, 5, 128), k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(TypeError, match="rows: dtype"):
        b.paged_append(k, k, st, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="rows: shape"):
        b.paged_append(k, k, st, _i(0, 1))
    with pytest.raises(ValueError, match="one CUDA device"):
        b.paged_append(k, k, st, _i(0, 1, 2, 3, 4))
    with pytest.raises(ValueError, match="one CUDA device"):
        b.paged_read(st, _i(0, 1))
    with pytest.raises(ValueError, match="rows: shape"):
        b.paged_read(st, _i(0, 1).view(1, 2))
    with pytest.raises(ValueError, match="dst: shape"):
        b.paged_copy(st, _i(0, 1), _i(2))


def test_binding_refuses_tables_and_heads():
    st = _store()
    q, table, n, cu = _bf(4, 3, 128), torch.zeros((2, 4), dtype=torch.int32), _i(9, 8), _i(0, 1, 3)
    with pytest.raises(ValueError, match="3 heads, not a multiple"):
        b.attend_tree(_bf(3, 3, 128), st, table, n, cu)
    with pytest.raises(ValueError, match="page_table"):
        b.attend_tree(q, st, table[:1], n, cu)
    with pytest.raises(ValueError, match="lengths"):
        b.attend_tree(q, st, table, n[:1], cu)
    with pytest.raises(ValueError, match="cu_nodes"):
        b.attend_tree(q, st, table, n, cu[:0])
    with pytest.raises(ValueError, match="parents"):
        b.attend_tree(q, st, table, n, cu, _i(0, 0))
    with pytest.raises(ValueError, match="lse"):
        b.attend_tree(q, st, table, n, cu, lse=torch.zeros((4, 4)))
    with pytest.raises(ValueError, match="one CUDA device"):
        b.attend_tree(q, st, table, n, cu)
    with pytest.raises(TypeError, match="keep"):
        b.paged_keep(st, table, n, cu, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="keep"):
        b.paged_keep(st, table, n, cu, torch.zeros((3, 1), dtype=torch.uint8))
    k = _bf(2, 3, 128)
    with pytest.raises(ValueError, match="not a multiple"):
        b.attend_prompt(_bf(3, 3, 128), k, k, cu)
    with pytest.raises(ValueError, match="V: 2 rows"):
        b.attend_prompt(q, k, k[:, :2], cu)
    with pytest.raises(ValueError, match="cu_k"):
        b.attend_prompt(q, k, k, cu, _i(0, 3))
    with pytest.raises(TypeError, match="cu_q"):
        b.attend_prompt(q, k, k, cu.long())
    with pytest.raises(ValueError, match="one CUDA device"):
        b.attend_prompt(q, k, k, cu)


def test_outputs_over_inputs_are_refused():
    x = _bf(4, 6, 128)
    with pytest.raises(ValueError, match="shares memory with Q"):
        b._need_apart(x, Q=x)
    with pytest.raises(ValueError, match="shares memory with K"):
        b._need_apart(x[:, 2:4], Q=None, K=x[:, 3:5])
    b._need_apart(x[:2], Q=x[2:])
