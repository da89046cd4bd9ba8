"""The row layout of large assignments: clusters of 16 blocks, several batches of ids a warp."""
import numpy as np
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq

pytestmark = pytest.mark.gpu


def _laid_out(ids, experts, capacity):
    t, top_k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < experts)
    counts = np.bincount(flat[ok], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    at = np.flatnonzero(ok)
    order = at[np.argsort(flat[at], kind="stable")]
    key = flat[order]
    slot = offsets[key] + np.arange(len(order)) - (np.cumsum(counts) - counts)[key]
    rows, slots = np.full(capacity, -1, np.int64), np.full(t * top_k, -1, np.int64)
    rows[slot], slots[order] = order // top_k, slot
    return rows, offsets, slots.reshape(t, top_k)


@pytest.mark.parametrize("t,top_k", [(2047, 8), (2048, 8), (4099, 4), (16384, 8), (16411, 8), (42859, 7), (300013, 1), (11000, 32)])
@pytest.mark.parametrize("experts,kind", [(256, "even"), (512, "skew"), (128, "holes"), (3, "even"), (1, "even"), (33, "runs")])
def test_large_assignments(cuda_ok, t, top_k, experts, kind):
    """Even, nearly all to one expert, with ids that stand for none, and in long runs of one expert; lengths that are
    no multiple of 32 among them."""
    g = np.random.default_rng(t + experts)
    ids = g.integers(0, experts, (t, top_k)).astype(np.int32)
    if kind == "skew":
        ids[g.random(ids.shape) < 0.97] = 311
    elif kind == "holes":
        ids[g.random(ids.shape) < 0.3] = -1
        ids[g.random(ids.shape) < 0.1] = experts
        ids[g.random(ids.shape) < 0.1] = 2**31 - 1
        ids[g.random(ids.shape) < 0.1] = -(2**31)
    elif kind == "runs":
        ids = np.sort(ids.reshape(-1)).reshape(t, top_k)
    cap = sharq.sharq_route_rows_capacity(t, top_k, experts)
    want = _laid_out(ids, experts, cap)
    d = torch.from_numpy(ids).cuda()
    for _ in range(2):
        for name, got, w in zip(("rows", "offsets", "slots"), sharq.route_rows(d, experts), want):
            assert np.array_equal(got.cpu().numpy(), w), name
