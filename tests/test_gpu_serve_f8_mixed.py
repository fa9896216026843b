"""Appends to e4m3 pages that mix single tokens with the chunk of a prompt, as a
serving step does: the oracle's codes, and a time that is not the chunk's tokens
one after the other."""
import numpy as np
import pytest
import torch

from store_h3kv_build_gb300 import binding as b

from test_gpu_serve_f8 import DEV, angles, append_case, cu_of, i32, normal, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("singles,chunk", [(15, 512), (63, 600), (200, 129), (3, 17)])
def test_single_tokens_beside_a_chunk(cuda, singles, chunk, ps):
    rng = np.random.default_rng(singles + ps)
    where = int(rng.integers(0, singles + 1))
    news = [1] * where + [chunk] + [1] * (singles - where)
    lens = [m + int(rng.integers(0, 150)) for m in news]
    append_case(news, lens, 4, 2, ps, seed=ps, gain=20.0, pad=3, first=5)


@pytest.mark.parametrize("rotate,dim,inter", [(False, 128, False), (True, 64, False), (True, 128, True)])
def test_chunks_of_unlike_sizes_beside_single_tokens(cuda, rotate, dim, inter):
    news = [1, 0, 700, 1, 1, 33, 64, 65, 0, 1, 2, 128, 1] + [1] * 70 + [300]
    lens = [m + 7 * i for i, m in enumerate(news)]
    append_case(news, lens, 5, 2, 64, dim, inter, seed=3, rotate=rotate)
    append_case(news, lens, 5, 2, 16, dim, inter, seed=4, rotate=rotate, positions=rotate)


@pytest.mark.parametrize("singles,chunk", [(63, 2048), (31, 512), (127, 8192)])
def test_a_mixed_append_takes_no_more_than_its_parts_several_times(cuda, singles, chunk):
    # one warp for all of the chunk took 0.42 us for each of its tokens, 10 to 80
    # times what the two calls take that append the single tokens and the chunk
    hq, hk, ps = 32, 8, 64
    lens = [100 + i for i in range(singles)] + [chunk + 40]
    table, pages = table_of(lens, ps)
    st = b.PagedStoreF8.empty(pages, hk, ps)
    for t in st.tensors().values():
        t.view(torch.uint8).fill_(0x38)
    n = singles + chunk
    q, k, v = (normal(i, h, n, 128).to(DEV) for i, h in enumerate((hq, hk, hk)))
    rot, dt, dl = b.Rotation(angles(chunk + 200, 128).to(DEV)), torch.from_numpy(table).to(DEV), i32(lens)
    qo, cu = torch.empty_like(q), i32(cu_of([1] * singles + [chunk]))
    only = i32([0, chunk])

    def mixed():
        b.paged_append_f8(k, v, st, dt, dl, cu, rot, None, q, qo)

    def apart():
        b.paged_append_f8(k[:, :singles], v[:, :singles], st, dt[:-1], dl[:-1], cu[:-1], rot, None, q[:, :singles], qo[:, :singles])
        b.paged_append_f8(k[:, singles:], v[:, singles:], st, dt[-1:], dl[-1:], only, rot, None, q[:, singles:], qo[:, singles:])

    def time_of(f):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                f()
        best = float("inf")
        for _ in range(5):
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            z.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(z) * 100)
        return best

    one, two = time_of(mixed), time_of(apart)
    b.sync_status()
    assert one < 5 * two, f"{one:.0f} us in one call, {two:.0f} us in two"
