"""The bounded waits of the serving operators: limits so small that every wait
gives up, and limits that a single tile keeps but a whole segment does not."""
import pytest
import torch

from store_h3kv_build_gb300 import binding as b
from store_h3kv_build_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def normal(seed, *shape):
    return synth.normal_f32(shape, seed).to(torch.bfloat16).to(DEV)


def status():
    try:
        b.sync_status()
    except b.H3kvError as e:
        return e.status
    return b.H3KV_OK


class limit:
    """Waits limited to `ns` nanoseconds within the block."""

    def __init__(self, ns):
        self.ns = ns

    def __enter__(self):
        assert b.h3kv_set_wait_timeout_ns(self.ns) == b.H3KV_OK

    def __exit__(self, *_):
        assert b.h3kv_set_wait_timeout_ns(0) == b.H3KV_OK


def test_calls_after_waits_that_all_gave_up(cuda):
    """A limit of one nanosecond: warps leave while copies are under way, also
    behind the last copy that was issued.  No CTA may be gone before its copies
    have landed (the next CTA's shared memory lies in the same place), so the
    context is sound and calls after it give the bits of before."""
    pages, hk, ps = 40, 2, 64
    st = b.PagedStore.empty(pages, hk, ps)
    n = pages * ps
    k, v, rows = normal(1, hk, n, 128), normal(2, hk, n, 128), torch.arange(n, dtype=torch.int32, device=DEV)
    q = normal(3, 8, 700, 128)
    cu = i32([0, 100, 356, 700])
    table, lens = i32([list(range(pages))] * 3), i32([n, 200, 64])
    calls = [lambda: b.paged_append(k, v, st, rows), lambda: b.paged_append(k[:, :100], v[:, :100], st, rows[:100]),
             lambda: b.attend_prompt(q, k[:, :700], v[:, :700], cu)]
    for m in (1, 4, 8, 40):
        qt, c = normal(4 + m, 8, 3 * m, 128), i32([0, m, 2 * m, 3 * m])
        calls.append(lambda qt=qt, c=c: b.attend_tree(qt, st, table, lens, c))
    want = [call() for call in calls]
    before = [t.clone() for t in st.tensors().values()]
    b.sync_status()
    for _ in range(3):
        for call in calls:
            with limit(1):
                call()
                assert status() in (b.H3KV_OK, b.H3KV_ERR_DEVICE_TIMEOUT)
        got = [call() for call in calls]
        b.sync_status()
        for x, y in zip(got, want):
            assert x is None or torch.equal(x, y)
        assert all(torch.equal(x, y) for x, y in zip(st.tensors().values(), before))
