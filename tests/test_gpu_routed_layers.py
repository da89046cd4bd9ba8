"""`route_rows`' arrays, which have the size that any assignment fits in, in the grouped products of the split layers."""
import numpy as np
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,pat", [("nvfp4", "4:8pair"), ("nvfp4", "8:16"), ("mxfp4", "4:8pair"), ("mxfp4", "2:4")])
@pytest.mark.parametrize("t,top_k,experts,k", [(150, 4, 16, 512), (9, 2, 8, 256), (700, 3, 5, 768), (300, 1, 1, 512), (5, 1, 1, 8192)])
def test_routed_rows_feed_the_grouped_products(cuda_ok, fmt, pat, t, top_k, experts, k):
    """The same as with arrays cut to the rows in use; rows of y behind the last group stay as they were."""
    g = np.random.default_rng(t)
    n = 256
    x = torch.from_numpy(g.standard_normal((t, k)).astype(np.float32)).cuda().bfloat16()
    w = sharq.FP4Weight.quantize(torch.from_numpy(0.02 * g.standard_normal((experts, n, k)).astype(np.float32)).cuda().bfloat16(), fmt)
    ids = g.integers(0, experts, (t, top_k)).astype(np.int32)
    ids[g.random(ids.shape) < 0.4] = -1  # so that fewer rows are in use than the arrays hold, with one expert too
    r = sharq.route_rows(torch.from_numpy(ids).cuda(), experts)
    used, cap = int(r.offsets[-1]), r.rows.numel()
    assert used < cap or cap == 128  # one tile has nothing behind it
    p = sharq.prepare(x, fmt, pat)
    a = sharq.gather_prepared(p, r.rows)
    cut = sharq.gather_prepared(p, r.rows[:used])
    for dtype in (torch.float32, torch.bfloat16):
        want = sharq.linear_grouped(cut, w, r.offsets, out_dtype=dtype)
        y = torch.full((cap, n), 7.0, dtype=dtype, device="cuda")
        sharq.linear_grouped(a, w, r.offsets, out=y)
        sharq.sharq_sync_status()
        assert torch.equal(y[:used], want)
        assert bool((y[used:] == 7.0).all()), "rows behind the last group were written"
        if fmt == "nvfp4" and pat == "4:8pair":
            y.fill_(7.0)
            sharq.linear_grouped_gather(p, r.rows, w, r.offsets, out=y)
            sharq.sharq_sync_status()
            assert torch.equal(y[:used], want)
            assert bool((y[used:] == 7.0).all()), "rows behind the last group were written"


@pytest.mark.parametrize("experts", [1, 3])
def test_rows_in_front_of_the_first_group(cuda_ok, experts):
    """Offsets that do not begin at 0: the rows before them are in no group either."""
    k, n = 512, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((640, k), generator=g, device="cuda").bfloat16()
    w = sharq.FP4Weight.quantize(0.02 * torch.randn((experts, n, k), generator=g, device="cuda"), "nvfp4")
    p = sharq.prepare(x, "nvfp4", "4:8pair")
    every = [0, 640] if experts == 1 else [0, 256, 256, 640]
    some = [128, 512] if experts == 1 else [128, 256, 256, 512]
    want = sharq.linear_grouped(p, w, torch.tensor(every, dtype=torch.int32, device="cuda"))
    y = torch.full((640, n), 7.0, dtype=torch.bfloat16, device="cuda")
    sharq.linear_grouped(p, w, torch.tensor(some, dtype=torch.int32, device="cuda"), out=y)
    sharq.sharq_sync_status()
    assert torch.equal(y[128:512], want[128:512])
    assert bool((y[:128] == 7.0).all()) and bool((y[512:] == 7.0).all())
