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


def test_prompts_longer_than_the_limit(cuda):
    """Warps that wait for a segment's end are not held to the limit of a
    tile: 1024 key tiles of over a microsecond each, under a limit of 300."""
    n = 131072
    q, k, v = normal(1, 1, 300, 128), normal(2, 1, n, 128), normal(3, 1, n, 128)
    for causal, cu in ((False, [0, 300]), (True, [0, 256]), (False, [0, 1, 300])):
        keys = [0, n - 77] if len(cu) == 2 else [0, n // 2, n - 5]
        want = b.attend_prompt(q, k, v, i32(cu), i32(keys), causal=causal)[:, :cu[-1]]
        with limit(300_000):
            got = b.attend_prompt(q, k, v, i32(cu), i32(keys), causal=causal)[:, :cu[-1]]
            b.sync_status()
        assert torch.equal(got, want)


def test_trees_longer_than_the_limit(cuda):
    """The same for the cache: several long items on each CTA."""
    hk, ps, n = 8, 128, 65536
    st = b.PagedStore.empty(n // ps, hk, ps, device=DEV)
    b.paged_append(normal(1, hk, n, 128), normal(2, hk, n, 128), st, torch.arange(n, dtype=torch.int32, device=DEV))
    seqs = 29  # 232 items, 152 CTAs
    table, lens = i32([list(range(n // ps))] * seqs), i32([n] * seqs)
    for m, hq in ((1, 64), (2, 64), (4, 64), (8, 64)):
        q, cu = normal(3 + m, hq, seqs * m, 128), i32(list(range(0, seqs * m + 1, m)))
        want = b.attend_tree(q, st, table, lens, cu)
        with limit(100_000):
            got = b.attend_tree(q, st, table, lens, cu)
            b.sync_status()
        assert torch.equal(got, want)
