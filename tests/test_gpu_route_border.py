"""Routing where fp32 cannot tell: groups whose best scores cancel, places next to each other at the border, scores and
biases at the ends of fp32's range, and weights that are not renormalized."""
import numpy as np
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq
from fp4_common import routed

pytestmark = pytest.mark.gpu

INF = float("inf")
LOW = torch.finfo(torch.float32).min


def _want(z, top_k, score, bias, groups=1, top_groups=1, group_top=1):
    """ids by stable sorts in 64 bits, and the scores."""
    z = z.double()
    t, experts = z.shape
    p = torch.softmax(z, 1) if score == "softmax" else 1 / (1 + torch.exp(-z))
    c = p if bias is None else p + bias.double()
    by = z if bias is None else c
    if groups > 1:
        value = c.view(t, groups, -1).sort(dim=2, descending=True)[0][:, :, :group_top].sum(2)
        kept = value.sort(dim=1, descending=True, stable=True)[1][:, :top_groups]
        member = torch.zeros((t, groups), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        by = by.masked_fill(~member.repeat_interleave(experts // groups, 1), -INF)
    return by.sort(dim=1, descending=True, stable=True)[1][:, :top_k], p


def _check(z, top_k, score, bias, **kw):
    ids, _ = sharq.route(z, top_k, score=score, bias=bias, **kw)
    want, _ = _want(z, top_k, score, bias, **kw)
    bad = (ids.long() != want).any(1)
    i = int(bad.nonzero()[0]) if bool(bad.any()) else -1
    assert i < 0, f"{int(bad.sum())} of {len(z)} tokens differ, first {i}: {ids[i].tolist()} for {want[i].tolist()}"


def test_groups_whose_best_two_cancel(cuda_ok):
    """Biases of +-100: the groups' values are of the size of the terms' rounding in fp32."""
    u = 2.0**-17
    z = torch.tensor([[1.2, 1.2, 2.8, -1.2]], device="cuda") * u
    bias = torch.tensor([100.0, -100.0, 100.0, -100.0], device="cuda")
    _check(z, 2, "sigmoid", bias, groups=2, top_groups=1, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2.0, 30.0, 1000.0])
@pytest.mark.parametrize("experts,groups,top_groups", [(64, 32, 8), (16, 8, 3), (256, 32, 5)])
def test_cancelling_pairs(cuda_ok, score, size, experts, groups, top_groups):
    g = torch.Generator(device="cuda").manual_seed(int(size) + experts)
    t, per = 4096, experts // groups
    bias = torch.full((experts,), -size, device="cuda")
    bias[::per] = size
    for spread in (2.0**-17, 2.0**-10):
        z = spread * torch.randn((t, experts), generator=g, device="cuda")
        _check(z, 2 * top_groups, score, bias, groups=groups, top_groups=top_groups, group_top=2)


def test_biases_at_the_ends_of_the_range(cuda_ok):
    """Sums of two that leave fp32 but not 64 bits; the lowest finite value as a mask."""
    big = 3e38
    cases = [
        [big, big, 3.2e38, 3.2e38, 0, 0, 0, 0],            # both sums beyond fp32: the second is larger
        [LOW, LOW, -3.0e38, -3.0e38, LOW, LOW, LOW, LOW],  # the same below
        [-INF, -INF, LOW, LOW, -INF, -INF, -INF, -INF],    # only the second has an expert at all
        [-INF, LOW, LOW, LOW, -INF, -INF, LOW, -INF],
        [LOW, 1.0, 0.5, 0.25, LOW, LOW, 1.5, LOW],
        [INF, 0, INF, 1, 0, 0, 0, 0],
    ]
    g = torch.Generator().manual_seed(1)
    z = torch.randn((5, 8), generator=g)
    for b in cases:
        bias = torch.tensor(b, dtype=torch.float32)
        for score in ("softmax", "sigmoid"):
            for top_groups, top_k in ((1, 1), (1, 2), (2, 3), (3, 6)):
                for group_top in (1, 2):
                    kw = dict(score=score, groups=4, top_groups=top_groups, group_top=group_top)
                    ids, w = sharq.route(z.cuda(), top_k, bias=bias.cuda(), **kw)
                    want, ww = routed(z.double().numpy(), top_k, bias=bias.numpy(), **kw)
                    assert np.array_equal(ids.cpu().numpy(), want), (b, kw)
                    assert np.all(np.abs(w.cpu().numpy() - ww) <= 2 * 27 * 2.0**-24 * np.abs(ww) + 1e-37)


@pytest.mark.parametrize("spread", [2.0**-24, 2.0**-22, 2.0**-21, 2.0**-20, 2.0**-18])
def test_places_next_to_each_other_at_the_border(cuda_ok, spread):
    """A bias that undoes the scores but for a little: places inside in an open order, and the border open too."""
    g = torch.Generator(device="cuda").manual_seed(5)
    t, experts = 20000, 48
    base = torch.randn((experts,), generator=g, device="cuda")
    z = base + spread * torch.randn((t, experts), generator=g, device="cuda") * 8
    bias = (0.7 - torch.sigmoid(base.double())).float()
    for top_k in (1, 2, 8, 31, 32):
        _check(z, top_k, "sigmoid", bias)
    p = torch.softmax(base.double(), 0)
    _check(z, 8, "softmax", (0.7 - p).float())


def test_weights_that_are_not_renormalized(cuda_ok):
    """All 32 weights of a softmax add up to 1: the numerators are the terms of the denominator.  One logit of 0 and 31
    of -c, E = e^-c: the lanes' tree adds equal terms without rounding and rounds 1 + E, 1 + 3E, 1 + 7E, 1 + 15E and
    1 + 31E, 2^-24 of each; the quotient and the products round by 2^-24 each.  (Numerators and denominator made by
    different exponentials differ by more.)"""
    c = torch.linspace(1.0, 8.0, 20000, device="cuda")
    z = -c[:, None].repeat(1, 32)
    z[torch.arange(len(c)), torch.arange(len(c)) % 32] = 0.0
    for bias in (None, torch.linspace(-1, 1, 32, device="cuda")):
        _, w = sharq.route(z, 32, score="softmax", bias=bias, renormalize=False)
        e = torch.exp(-c.double())
        tol = ((5 + 57 * e) / (1 + 31 * e) + 2) * 2.0**-24 * (1 + 2.0**-10)
        off = (w.double().sum(1) - 1).abs()
        assert bool((off <= tol).all()), f"{int((off > tol).sum())} tokens, worst {float((off / tol).max())} of the bound"
