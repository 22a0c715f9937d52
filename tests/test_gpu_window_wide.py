"""Long runs of queries on the kernel of whole tiles, which every case here is checked to take: one
tile and pairs of them, few and many chunks of 128 tokens, every type, tight tolerances."""

import pytest

from _window import Windowed, close
from test_gpu_window_values import expect, kernel, run

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


# queries, lengths, kv heads, heads per group, window, sinks
CASES = {
    "one_tile_two_chunks": ([9, 8, 7, 9], [200, 150, 30, 9], 4, 4, 60, 3),
    "one_tile_many_chunks": ([5, 9, 0, 8, 9, 9], [700, 900, 0, 333, 640, 650], 8, 4, 600, 20),
    "one_tile_all_tokens": ([5, 9, 4, 8, 9, 9], [600, 700, 4, 333, 640, 450], 8, 8, 0, 0),
    "pairs_and_a_single": ([90, 33, 64], [1000, 640, 64], 4, 4, 300, 70),
    "first_rows_leave_later_chunks": ([260, 200], [1500, 260], 2, 2, 100, 0),
    "wide_groups": ([40, 33, 17], [700, 500, 20], 2, 8, 129, 1),
    "one_head_a_group": ([300, 257, 1], [400, 257, 900], 4, 1, 64, 17),
    "all_tokens": ([130, 128, 66], [500, 128, 480], 8, 2, 0, 5),
}


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("d", [64, 128])
def test_whole_tiles(kv, q, d, name):
    counts, lens, hkv, g, window, sinks = CASES[name]
    c = Windowed(lens, hkv, d, kv, window, sinks, seed=len(name), q=q, g=g, counts=counts)
    c.scale *= 2
    assert kernel(c) == "mq_wide_kernel"
    want, tol = expect(c)
    close(run(c), want, tol)
