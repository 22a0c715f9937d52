"""Which kernel pkv_window_multiquery_attn takes, from the library's own planner: no GPU needed."""

import pytest

from paged_kv_decode_05_gb300 import binding as B
from paged_kv_decode_05_gb300.build import build

MOST = 2**31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def kernel(batch, hkv, g, max_q, mb, window, sinks, kv="bf16", q="bf16", d=128):
    code = {"bf16": B.PKV_BF16, "f16": B.PKV_F16, "i8": B.PKV_I8}
    desc = B.CacheDesc(batch * mb, 16, hkv, d, code[kv])
    return B.pkv_testing_window_multiquery_kernel(batch, hkv * g, max_q, desc, code[q], mb, window,
                                                  sinks)


def test_windows_and_sinks_of_any_size_count_as_the_whole_table():
    """One sequence's run of 64 rows over a table of 4096 blocks: split among all SMs, whichever
    way the call says that every token is seen."""
    for window, sinks in ((0, 0), (MOST, 0), (0, MOST), (MOST, MOST), (MOST, MOST - 15),
                          (MOST - 70, MOST - 16), (1, MOST), (1 << 16, 0)):
        assert kernel(1, 8, 4, 16, 4096, window, sinks) == ("mq_split_kernel", 64), (window, sinks)


def test_a_kernel_for_every_size():
    assert kernel(64, 8, 4, 5, 1000, 4096, 0)[0] == "mqt_split_kernel"
    assert kernel(64, 8, 4, 5, 1000, 4096, 0, "i8")[0] == "mqt_i8_split_kernel"
    assert kernel(64, 8, 4, 5, 1000, 4096, 0, "i8", d=64) == ("mq_split_kernel", 32)
    assert kernel(64, 8, 4, 8, 1000, 4096, 0) == ("mq_split_kernel", 32)
    assert kernel(8, 8, 4, 512, 512, 2048, 4) == ("mq_wide_kernel", 128)


@pytest.mark.parametrize("over", [dict(mb=0), dict(window=-1), dict(sinks=-1)])
def test_refusals(over):
    a = dict(dict(mb=8, window=4, sinks=1), **over)
    desc = B.CacheDesc(64, 16, 2, 128, B.PKV_BF16)
    with pytest.raises(B.PkvError):
        B.pkv_testing_window_multiquery_kernel(2, 8, 5, desc, B.PKV_BF16, a["mb"], a["window"],
                                               a["sinks"])
