"""The long-context operators called by several host threads at once, each on a
stream of its own."""

import ctypes
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

CALLS = 3000


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _select(width, seed):
    """A call of the C function over two rows of `width` scores, its outputs, what they are to
    be, and its stream."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, 1, width)).astype(np.float32)
    scores = torch.from_numpy(x).cuda()
    lens = torch.full((2,), 16 * width, dtype=torch.int32, device="cuda")
    lists = torch.zeros((2, 1, 64), dtype=torch.int32, device="cuda")
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    args = (scores.data_ptr(), 2, 1, width, lens.data_ptr(), 0, 0, 64, lists.data_ptr(),
            counts.data_ptr(), None, ctypes.c_void_p(stream.cuda_stream))
    fn = B.lib().pkv_block_select
    want = [np.sort(np.argsort(-x[:, 0], 1, kind="stable")[:, :64], 1)[:, None]]
    return (lambda: fn(*args)), [lists], want, stream, (scores, lens, counts)


def _evict(width, seed):
    """The same of two rows of `width` weights, of which none fits its budget's blocks."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(seed)
    mb = width // 16
    x = rng.random((2, 1, width)).astype(np.float32)
    mass = torch.from_numpy(x).cuda()
    k = torch.zeros((2 * mb + 8, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    dev = dict(dtype=torch.int32, device="cuda")
    tables = torch.arange(2 * mb, **dev).view(2, mb)
    new = torch.arange(2 * mb, 2 * mb + 8, **dev).view(2, 4)
    lens = torch.full((2,), width, **dev)
    new_lens, kept = torch.zeros(2, **dev), torch.zeros((2, 1, 64), **dev)
    new_mass = torch.zeros((2, 1, 64), device="cuda")
    stream = torch.cuda.Stream()
    desc = B.cache_desc(k)
    args = (k.data_ptr(), v.data_ptr(), None, None, ctypes.byref(desc), tables.data_ptr(), mb,
            lens.data_ptr(), mass.data_ptr(), 2, 64, 0, 0, new.data_ptr(), 4, new_lens.data_ptr(),
            new_mass.data_ptr(), kept.data_ptr(), None, ctypes.c_void_p(stream.cuda_stream))
    fn = B.lib().pkv_evict_tokens
    pick = np.sort(np.argsort(-x[:, 0], 1, kind="stable")[:, :64], 1)
    want = [pick[:, None], np.take_along_axis(x[:, 0], pick, 1)[:, None]]
    return (lambda: fn(*args)), [kept, new_mass], want, stream, (k, v, tables, new, lens, mass,
                                                                 new_lens, desc)


@pytest.mark.parametrize("make, widths", [(_select, (32768, 12000)), (_evict, (32768, 17008))])
def test_rows_of_two_lengths(make, widths):
    """Rows of two lengths, which take different amounts of shared memory, both more than a
    kernel has without leave: no thread's call fails because of the other's."""
    import torch
    runs = [make(w, i) for i, w in enumerate(widths)]
    torch.cuda.synchronize()
    codes = [set(), set()]
    start = threading.Barrier(2)

    def loop(i):
        call = runs[i][0]
        start.wait()
        for n in range(CALLS):
            codes[i].add(call())
            if n % 200 == 199:
                runs[i][3].synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]
    for _, outs, want, _, _ in runs:
        for o, w in zip(outs, want):
            assert (o.cpu().numpy() == w).all()
