"""Which kernel pkv_window_multiquery_attn takes, from the library's own planner: no GPU needed."""

import ctypes

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


# us of the kernel of whole tiles and of the split one, 4 heads a group:
# (window, batch, kv heads, queries) -> by (cache, q, head_dim)
MEASURED = {
    (4096, 1, 8, 16): ((68, 22), (57, 19), (80, 25), (64, 22)),
    (4096, 1, 8, 128): ((103, 74), (99, 47), (131, 100), (116, 55)),
    (4096, 2, 8, 128): ((103, 128), (100, 79), (132, 181), (116, 91)),
    (4096, 8, 8, 32): ((73, 127), (61, 77), (84, 178), (69, 90)),
    (512, 8, 8, 16): ((17, 25), (16, 18), (22, 28), (18, 22)),
    (512, 1, 8, 64): ((25, 21), (22, 17), (31, 24), (25, 20)),
    (512, 1, 1, 1200): ((25, 48), (23, 41), (32, 54), (26, 46)),
}


@pytest.mark.parametrize("at, kv, q, d", [(0, "bf16", "bf16", 128), (0, "f16", "f16", 128),
                                          (1, "bf16", "bf16", 64), (1, "f16", "f16", 64),
                                          (2, "i8", "f16", 128), (3, "i8", "f16", 64)])
def test_the_faster_kernel_by_type_and_head_dim(at, kv, q, d):
    for (window, batch, hkv, n), us in MEASURED.items():
        mb = (window + n + 37 + 15) // 16
        wide, split = us[at]
        name = kernel(batch, hkv, 4, n, mb, window, 4, kv, q, d)[0]
        assert name == ("mq_wide_kernel" if wide < split else "mq_split_kernel"), (window, hkv, n)


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


def test_tables_whose_tokens_pass_32_bits_are_refused():
    """2^27 blocks of 16 tokens: lengths are counted in 32 bits. Refused before any CUDA call."""
    fake, invalid = 0x100000, 1
    desc = B.CacheDesc(8, 16, 2, 128, B.PKV_BF16)
    for mb, want in ((1 << 27, invalid), (MOST, invalid), ((1 << 27) - 1, 3)):      # 3: workspace
        head = (fake, B.PKV_BF16, fake, 5, fake, fake, None, None, ctypes.byref(desc), fake, mb,
                fake, 4, 8, 0.125)
        tail = (fake, fake, 16, 64, None, None)
        assert B.lib().pkv_multiquery_attn(*head, *tail) == want
        assert B.lib().pkv_window_multiquery_attn(*head, 5, 1, *tail) == want
