"""Expert routing on the GPU against plain 64-bit forms: scores and top-k, the routed-row layout, the weighted sum."""
import numpy as np
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq
from fp4_common import laid_out, routed

pytestmark = pytest.mark.gpu


def _check_route(logits, top_k, **kw):
    """ids equal; weights to the rounding of p, of their sum and of the quotient: exp and a sum of up to 512 terms in
    fp32 by the pairwise tree of a warp (16 terms in a lane, 5 levels) are off by at most 2 + 21 steps of 2^-24 each
    for numerator and denominator, the quotients and the scale by 4 more."""
    bias = kw.get("bias")
    dev = logits.cuda()
    ids, w = sharq.route(dev, top_k, **{**kw, "bias": None if bias is None else bias.cuda()})
    want, ww = routed(logits.double().numpy(), top_k, **{**kw, "bias": None if bias is None else bias.numpy()})
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    bad = np.argwhere(ids != want)
    assert bad.size == 0, f"{len(bad)} ids differ, first at {bad[0].tolist()}: {ids[bad[0][0]]} for {want[bad[0][0]]}"
    assert np.all(np.abs(w - ww) <= 2 * 27 * 2.0**-24 * np.abs(ww) + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,experts,top_k", [(1, 1, 1), (1, 128, 8), (3, 7, 7), (5, 31, 4), (130, 33, 2), (67, 64, 6),
                                             (64, 200, 8), (33, 256, 32), (9, 300, 5), (17, 512, 10)])
def test_top_k(cuda_ok, score, dtype, t, experts, top_k):
    g = torch.Generator().manual_seed(t * 1000 + experts)
    logits = torch.randn((t, experts), generator=g).to(dtype)  # bf16: many ties among the largest
    _check_route(logits, top_k, score=score)
    _check_route(logits, top_k, score=score, renormalize=False, scale=2.5)
    _check_route(logits, top_k, score=score, bias=0.1 * torch.randn((experts,), generator=g))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,group_top,top_k", [(8, 4, 2, 1, 3), (64, 8, 3, 2, 8), (6, 6, 4, 2, 4),
                                                                      (256, 8, 4, 2, 8), (480, 32, 5, 1, 16),
                                                                      (512, 2, 1, 2, 32)])
def test_groups(cuda_ok, score, experts, groups, top_groups, group_top, top_k):
    g = torch.Generator().manual_seed(experts + groups)
    for dtype, with_bias in ((torch.bfloat16, False), (torch.float32, True), (torch.bfloat16, True)):
        logits = torch.randn((41, experts), generator=g).to(dtype)
        bias = 0.1 * torch.randn((experts,), generator=g) if with_bias else None
        _check_route(logits, top_k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)


def test_equal_and_nearly_equal_scores(cuda_ok):
    """Ties go to the lower index; values that fp32 rounds together but 64 bits tell apart are ranked apart."""
    logits = torch.zeros((4, 40))
    logits[1, 7] = logits[1, 23] = 1.0
    logits[2] = 16 + torch.arange(40) / 64  # sigmoid: 1 - e^-l, the last steps below 2^-24
    logits[3] = 16 - torch.arange(40) / 64
    for kw in ({}, {"bias": torch.zeros(40)}, {"groups": 4, "top_groups": 2, "group_top": 2},
               {"bias": torch.zeros(40), "groups": 4, "top_groups": 2, "group_top": 1}):
        for score in ("softmax", "sigmoid"):
            _check_route(logits, 6, score=score, **kw)
    # a bias that undoes the scores' order but for a little in the 25th bit and below
    z = torch.randn((300, 48), generator=torch.Generator().manual_seed(3))
    bias = (0.5 - torch.sigmoid(z[0].double())).float()
    _check_route(z[:1].expand(20, 48).contiguous(), 8, score="sigmoid", bias=bias)


def test_masked_experts(cuda_ok):
    """-inf and NaN take an expert out; a token with too few left has id -1 and weight 0; the lowest finite value is a
    value like any other; +inf wins."""
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    logits = torch.randn((8, 24), generator=torch.Generator().manual_seed(1))
    logits[0] = -inf
    logits[1] = nan
    logits[2, 3:] = -inf
    logits[3, ::2] = nan
    logits[4] = low
    logits[5, 1:] = low
    logits[6, [2, 9]] = inf
    logits[7, :20] = -inf
    for score in ("softmax", "sigmoid"):
        for kw in ({}, {"groups": 4, "top_groups": 2, "group_top": 2}, {"groups": 6, "top_groups": 6}):
            _check_route(logits, 8, score=score, **kw)
            _check_route(logits.to(torch.bfloat16), 8, score=score, **kw)
    bias = torch.zeros(24)
    bias[[0, 5]] = -inf
    bias[7] = nan
    _check_route(logits, 8, score="sigmoid", bias=bias)
    _check_route(logits, 4, score="softmax", bias=bias, groups=4, top_groups=1, group_top=2)


def test_route_strides_and_alignment(cuda_ok):
    base = torch.randn((50, 203), generator=torch.Generator().manual_seed(5), dtype=torch.float32)
    for dtype in (torch.float32, torch.bfloat16):
        b = base.to(dtype)
        for view in (lambda x: x[:, 3:131], lambda x: x[::2, :200], lambda x: x[:, 1:202:2], lambda x: x.t()[:, :37]):
            want = routed(view(b).double().numpy(), 5)[0]
            assert np.array_equal(sharq.route(view(b.cuda()), 5)[0].cpu().numpy(), want)


# ------------------------------------------------------------- row layout
@pytest.mark.parametrize("t,top_k,experts", [(1, 1, 1), (1, 8, 128), (13, 8, 128), (127, 2, 3), (129, 1, 5), (300, 4, 64),
                                             (700, 3, 512), (2100, 7, 100), (5000, 2, 31)])
def test_rows(cuda_ok, t, top_k, experts):
    g = np.random.default_rng(t + experts)
    ids = g.integers(0, experts, size=(t, top_k)).astype(np.int32)  # the same expert twice in a token, too
    if t > 100:
        ids[g.random(ids.shape) < 0.05] = -1      # no expert
        ids[g.random(ids.shape) < 0.02] = experts  # out of range
        ids[ids == experts // 2] = 0              # an expert without rows
    _check_rows(ids, experts)


def _check_rows(ids, experts):
    t, top_k = ids.shape
    got = sharq.route_rows(torch.from_numpy(ids).cuda(), experts)
    rows, offsets, slots = laid_out(ids, experts, sharq.sharq_route_rows_capacity(t, top_k, experts))
    assert np.array_equal(got.offsets.cpu().numpy(), offsets)
    assert np.array_equal(got.slots.cpu().numpy(), slots)
    assert np.array_equal(got.rows.cpu().numpy(), rows)


def test_rows_extremes(cuda_ok):
    """All to one expert, none anywhere, exactly whole tiles, and the assignment that needs the whole capacity."""
    _check_rows(np.full((640, 4), 9, np.int32), 16)
    _check_rows(np.full((640, 4), -1, np.int32), 16)
    _check_rows(np.repeat(np.arange(8, dtype=np.int32), 128)[:, None], 8)
    full = np.concatenate([np.arange(10), np.zeros(128 * 5)]).astype(np.int32)[:, None]
    _check_rows(full, 10)
    assert int(sharq.route_rows(torch.from_numpy(full).cuda(), 10).offsets[-1]) == \
        sharq.sharq_route_rows_capacity(len(full), 1, 10)


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("y_dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                               (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("t,top_k,n", [(1, 1, 8), (1, 8, 2048), (13, 3, 264), (200, 8, 1000), (77, 32, 40), (9, 17, 5120)])
def test_combine(cuda_ok, y_dtype, out_dtype, t, top_k, n):
    """top_k fused multiply-adds in fp32 (2^-24 of the partial sum each), then one rounding."""
    g = torch.Generator().manual_seed(t + n)
    y = torch.randn((t * top_k + 5, n), generator=g).to(y_dtype)
    slots = torch.randperm(t * top_k + 5, generator=g)[: t * top_k].view(t, top_k).to(torch.int32)
    w = torch.rand((t, top_k), generator=g)
    add = torch.randn((t, n), generator=g).to(y_dtype)
    if t > 10:
        slots[::3, 0] = -1
        slots[5] = -1                # nothing left
        slots[6, -1] = len(y)        # past the rows
        slots[7] = slots[8]          # the same rows for two tokens
    y[slots[0, 0]] = 0.0
    for a in (None, add):
        out = sharq.combine(y.cuda(), slots.cuda(), w.cuda(), add=None if a is None else a.cuda(), out_dtype=out_dtype)
        ok = ((slots >= 0) & (slots < len(y))).double()
        part = y.double()[slots.long().clamp(0, len(y) - 1)] * (w.double() * ok)[..., None]
        ref = part.sum(1) + (0 if a is None else a.double())
        mag = part.abs().sum(1) + (0 if a is None else a.double().abs())
        tol = top_k * 2.0**-24 * mag
        tol = tol + (2.0**-8 if out_dtype == torch.bfloat16 else 2.0**-24) * (ref.abs() + tol)
        assert out.dtype == out_dtype
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())


def test_combine_leaves_unused_rows_out(cuda_ok):
    """NaN and infinities in rows that no slot names never reach a token; out may be add."""
    y = torch.full((6, 16), float("nan"), device="cuda")
    y[2], y[4] = 3.0, 5.0
    slots = torch.tensor([[2, -1], [4, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [1.0, 2.0], [1.0, 1.0]], device="cuda")
    out = sharq.combine(y, slots, w)
    assert torch.equal(out.cpu(), torch.tensor([1.5, 11.0, 0.0])[:, None].expand(3, 16))
    add = torch.ones((3, 16), device="cuda")
    assert sharq.combine(y, slots, w, add=add, out=add) is add
    assert torch.equal(add.cpu(), torch.tensor([2.5, 12.0, 1.0])[:, None].expand(3, 16))


def test_python_refusals_on_the_gpu(cuda_ok):
    y = torch.zeros((4, 16), device="cuda")
    slots, w = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros((2, 2), device="cuda")
    for bad in (lambda: sharq.combine(y, slots.long(), w), lambda: sharq.combine(y, slots, w[:1]),
                lambda: sharq.combine(y, slots, w.double()), lambda: sharq.combine(y, slots, w, add=y),
                lambda: sharq.combine(y, slots.cpu(), w), lambda: sharq.combine(y, slots, w, out=y),
                lambda: sharq.route_rows(slots.long(), 4), lambda: sharq.route_rows(slots[0], 4),
                lambda: sharq.route(y, 2, bias=w[0]), lambda: sharq.route(y.double(), 2), lambda: sharq.route(y[0], 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sharq.combine(y[:, :12], slots, w), lambda: sharq.route(y, 17), lambda: sharq.route(y[:0], 2),
                lambda: sharq.route(y, 2, groups=3)):
        with pytest.raises(sharq.SharqError):
            bad()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_bias,groups,group_top", [(False, 1, 1), (True, 1, 1), (False, 8, 1), (False, 8, 2), (True, 8, 2)])
def test_many_tokens(cuda_ok, score, dtype, with_bias, groups, group_top):
    """Enough tokens that neighbours within fp32's error of each other, and equal ones, occur among those that decide:
    ids equal to a stable sort in 64 bits.  (The scores below are torch's in 64 bits; the kernel's differ from them by
    a few units of 2^-53, which separates no two that this many draws bring about.)"""
    t, experts, top_groups, top_k = 20000, 256, 4, 8
    g = torch.Generator(device="cuda").manual_seed(17)
    logits = torch.randn((t, experts), generator=g, device="cuda").to(dtype)
    bias = 0.1 * torch.randn((experts,), generator=g, device="cuda") if with_bias else None
    ids, w = sharq.route(logits, top_k, score=score, bias=bias, groups=groups, top_groups=top_groups if groups > 1 else 1,
                         group_top=group_top)
    z = logits.double()
    p = torch.softmax(z, 1) if score == "softmax" else 1 / (1 + torch.exp(-z))
    c = p if bias is None else p + bias.double()
    by = z if bias is None else c
    if groups > 1:
        value = c.view(t, groups, -1).sort(dim=2, descending=True)[0][:, :, :group_top].sum(2)
        kept = value.sort(dim=1, descending=True, stable=True)[1][:, :top_groups]
        member = torch.zeros((t, groups), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        by = by.masked_fill(~member.repeat_interleave(experts // groups, 1), -float("inf"))
    want = by.sort(dim=1, descending=True, stable=True)[1][:, :top_k]
    assert torch.equal(ids.long(), want)
    ww = p.gather(1, want)
    ww = ww / ww.sum(1, keepdim=True)
    assert bool(((w.double() - ww).abs() <= 2 * 27 * 2.0**-24 * ww).all())


def test_combine_beside_its_inputs(cuda_ok):
    """y, add and out next to each other in one buffer, none of them in another."""
    buf = torch.randn((30, 64), device="cuda")
    y, add, out = buf[:20], buf[20:25], buf[25:]
    slots = torch.arange(10, dtype=torch.int32, device="cuda").view(5, 2)
    w = torch.rand((5, 2), device="cuda")
    want = sharq.combine(y.clone(), slots, w, add=add.clone())
    before = buf[:25].clone()
    assert torch.equal(sharq.combine(y, slots, w, add=add, out=out), want)
    assert torch.equal(buf[:25], before)
    with pytest.raises(sharq.SharqError):
        sharq.combine(y, slots, w, out=buf[19:24])
