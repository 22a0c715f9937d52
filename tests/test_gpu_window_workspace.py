"""One workspace size serves either type of q over an INT8 cache, at every size of run."""

import pytest
import torch

from paged_kv_decode_05_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_both_types_of_q(d, g):
    k = torch.ones((4, 2, 16, d), dtype=torch.int8, device="cuda")
    scales = torch.full((4, 2), 0.25, device="cuda")
    tables = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    for n in (1, 2, 3, 5, 8, 16, 24, 32, 40):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for dtype in (torch.bfloat16, torch.float16):
            q = torch.zeros((n, 2 * g, d), dtype=dtype, device="cuda")
            sizes = (B.pkv_multiquery_workspace_size(1, 2 * g, n, k),
                     B.pkv_window_multiquery_workspace_size(1, 2 * g, n, k),
                     B.pkv_window_decode_workspace_size(1, 2 * g, k))
            for i, size in enumerate(sizes):
                out = torch.zeros_like(q)
                ws = torch.empty(size, dtype=torch.uint8, device="cuda")
                if i == 0:
                    B.pkv_multiquery_attn(q, cu, n, k, k, tables, lens, 0.1, out, ws,
                                          k_scales=scales, v_scales=scales)
                elif i == 1:
                    B.pkv_window_multiquery_attn(q, cu, n, k, k, tables, lens, 0.1, 20, 1, out, ws,
                                                 scales, scales)
                else:
                    out = torch.zeros_like(q[:1])
                    B.pkv_window_decode_attn(q[:1], k, k, tables, lens, 0.1, 20, 1, out, ws, scales,
                                             scales)
                assert bool((out == 0.25).all()), (n, dtype, i)
