"""Sizes that the e4m3 pages' calls refuse, on the CPU."""
import ctypes

import pytest

from store_h3kv_build_gb300 import binding as b

P, FAR = 1 << 20, 1 << 30  # pointers that are never followed
BAD, OK = b.H3KV_ERR_INVALID_ARG, b.H3KV_OK


def store(pages, heads, page):
    return ctypes.byref(b.h3kv_paged_store_f8(FAR, FAR, FAR, FAR, pages, heads, page, 128))


@pytest.mark.parametrize("pages,heads,page", [(1 << 20, 64, 128), (1 << 27, 1, 16), (1 << 26, 3, 16), (1, 65536, 16),
                                              (1 << 27, 1 << 30, 16), (2 ** 31 - 1, 2 ** 31 - 1, 16)])
def test_a_size_is_given_only_for_stores_that_the_calls_take(pages, heads, page):
    assert b.h3kv_paged_store_f8_bytes(pages, heads, page, 128) == 0
    assert b.h3kv_paged_read_f8(store(pages, heads, page), P, 0, None, None, None) == BAD


@pytest.mark.parametrize("pages,heads,page", [((1 << 18) - 1, 64, 128), ((1 << 27) - 16, 1, 16), (1, 65535, 16), (0, 8, 64),
                                              (5, 0, 64)])
def test_the_largest_stores(pages, heads, page):
    assert b.h3kv_paged_store_f8_bytes(pages, heads, page, 128) == 2 * pages * heads * (page * 128 + 4)
    assert b.h3kv_paged_read_f8(store(pages, heads, page), P, 0, None, None, None) == OK


@pytest.mark.parametrize("heads,page,n", [(1, 16, (1 << 27) - 15), (1024, 128, 1 << 20), (65535, 128, 1 << 15), (8, 128, 1 << 27)])
def test_more_copies_than_a_launch_has_blocks_are_a_bad_argument(heads, page, n):
    s = ctypes.byref(b.h3kv_paged_store_f8(1 << 50, 2 << 50, 3 << 50, 4 << 50, 4, heads, page, 128))
    assert b.h3kv_paged_copy_f8(s, P, P, n, None) == BAD
