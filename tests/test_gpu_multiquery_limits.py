"""Multi-query calls of more units than 31 bits count: refused on the device, nothing written."""

import pytest
import torch

from paged_kv_decode_05_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


@pytest.mark.parametrize("window", [None, 0])
def test_more_units_than_31_bits(window):
    """33 tiles of 64 rows x 65400 blocks or more x 1024 kv heads, every table entry the one block
    of a small pool; then an ordinary call with the same workspace."""
    hkv, d, n, length = 1024, 64, 2112, 1 << 20
    k = torch.ones((1, hkv, 16, d), dtype=torch.int8, device="cuda")
    scales = torch.full((1, hkv), 0.5, device="cuda")
    q = torch.zeros((n, hkv, d), device="cuda").half()
    out = torch.full((n * hkv * d + 2,), 7.0, device="cuda").half()[2:].view(n, hkv, d)
    tables = torch.zeros((1, length // 16), dtype=torch.int32, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = (B.pkv_multiquery_workspace_size if window is None
            else B.pkv_window_multiquery_workspace_size)(1, hkv, n, k)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call():
        if window is None:
            B.pkv_multiquery_attn(q, cu, n, k, k, tables, lens, 0.125, out, ws, k_scales=scales,
                                  v_scales=scales, dev_status=status)
        else:      # (an out that is not 16-byte aligned: split, as above)
            B.pkv_window_multiquery_attn(q, cu, n, k, k, tables, lens, 0.125, window, 0, out, ws,
                                         scales, scales, 0, status)
    call()
    assert int(status.item()) == B.DEV_BAD_LENGTH
    assert bool((out == 7).all())
    status.zero_()
    lens.fill_(n)
    call()
    assert int(status.item()) == 0
    assert bool((out == 0.5).all())
