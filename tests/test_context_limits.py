"""The test hook of the eviction's clusters, and limits of the forms for long and shared contexts (no GPU)."""
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build


def test_cluster_limit_values():
    build()
    try:
        for ok in (1, 2, 4, 8, 16, 0):
            assert _lib.gqa_paged_decode_test_cluster_limit(ok) == 0
        for bad in (-1, 3, 12, 17, 32, 2 ** 31 - 1):
            assert _lib.gqa_paged_decode_test_cluster_limit(bad) == _lib.GQA_ERR_INVALID_ARGUMENT
    finally:
        _lib.gqa_paged_decode_test_cluster_limit(0)


def test_bounds_of_pages_past_what_the_kernel_walks_are_refused():
    build()
    a = 1 << 20
    for page in (2 ** 30 + 1, 2 ** 31 - 1):
        assert _lib.load().gqa_block_bounds(a, a, a, a, None, 1, page, 1, 1, None) == _lib.GQA_ERR_INVALID_ARGUMENT
