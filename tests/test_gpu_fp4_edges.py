"""Plain FP4 rows and products at the ends of their range: rows that do not exist, rows so small or so large that their
squares, their second-level scale or a product of factors leaves fp32's range."""
import numpy as np
import pytest
import torch

import oracle
from activation_sparsity_fp4_b200 import sharq
from fp4_common import check_product, quantized, read_matrix, values
from gpu_common import to_dev

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]


def _same(a, b, what):
    for name, g, w in zip(("scales", "codes", "row scales"), a, b):
        assert np.array_equal(g, w), f"{what}: {name} differ"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [256, 4096, 8224, 20000])
@pytest.mark.parametrize("kw", [dict(amax=5.0), dict(gamma=True, eps=0.0), dict(gamma=True, eps=0.0, amax=5.0), {}])
def test_rows_that_do_not_exist(cuda_ok, fmt, dtype, k, kw):
    """An index out of range stands for a row of zero codes and scales with the factor 1, whatever amax, gamma or eps,
    quantized as it is taken and gathered after it alike."""
    rng = np.random.default_rng(k)
    x = np.clip(rng.standard_normal((200, k)), -4, 4).astype(np.float32)
    kw = dict(kw)
    if kw.pop("gamma", False):
        kw["gamma"] = to_dev(rng.uniform(0.5, 1.5, k), dtype)
    xd = to_dev(x, dtype)
    rows = rng.integers(0, 200, 170).astype(np.int32)
    rows[[0, 5, 6, 169]] = [-1, 200, 2**31 - 1, -(2**31)]
    rd = torch.from_numpy(rows).cuda()
    taken = read_matrix(sharq.quantize_fp4(xd, fmt, rows=rd, **kw))
    for i in (0, 5, 6, 169):
        assert not taken[0][i].any() and not taken[1][i].any() and taken[2][i] == 1.0
    whole = sharq.quantize_fp4(xd, fmt, **kw)
    _same(read_matrix(sharq.gather_fp4(whole, rd)), taken, "gathered")
    more = torch.cat([rd, rd])  # more rows than x has: quantized once and gathered
    _same([a[:170] for a in read_matrix(sharq.quantize_fp4(xd, fmt, rows=more, **kw))], taken, "many rows")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [480, 4096, 8224, 20000])
@pytest.mark.parametrize("t", [9, 180])
def test_norm_of_small_and_large_rows(cuda_ok, fmt, k, t):
    """Without eps a row's normalized form does not depend on its magnitude: rows of 2^e times the first one (exact in
    fp32, squares up to 2^250 and down to 2^-250) have its bits; a row of zeros is zeros."""
    rng = np.random.default_rng(k)
    e = np.array(([0, -40, -60, -70, -90, -110, 70, 120, 0] * 20)[:t])
    x = (rng.choice([1.0, 1.25, 1.5, -1.0, -1.75], (1, k)) * 2.0 ** e[:, None].astype(np.float64)).astype(np.float32)
    x[8::9] = 0.0
    gamma = to_dev(rng.uniform(0.5, 1.5, k), "f32")
    got = read_matrix(sharq.quantize_fp4(to_dev(x, "f32"), fmt, gamma=gamma, eps=0.0))
    zero = quantized(np.zeros((1, k), np.float32), fmt)
    for i in range(t):
        _same([a[i] for a in got], [a[0] for a in (zero if i % 9 == 8 else got)], f"row {i}, 2^{e[i]}")
    assert got[1][0].any()


@pytest.mark.parametrize("k", [128, 4096, 20000])
def test_rows_of_tiny_magnitude(cuda_ok, k):
    """NVFP4 rows whose 2688 / A leaves fp32: still off by no more than half the widest E2M1 step of a block of scale S
    (E4M3: within 2^-4 of its value, or 2^-10 below 2^-6), both times the row's factor; zeros stay zeros."""
    rng = np.random.default_rng(k)
    e = np.arange(-146, -88, 2)
    x = (rng.uniform(-1, 1, (len(e), k)) * 2.0 ** e[:, None].astype(np.float64)).astype(np.float32)
    x[:, :16] *= np.float32(2.0**-8)  # a block whose scale is far below the row's largest
    x[:, ::5] = 0.0
    m = sharq.quantize_fp4(to_dev(x, "f32"), "nvfp4")
    scales, codes, rows = read_matrix(m)
    S = np.array([oracle.e4m3_decode([c])[0] for c in range(127)], np.float64)[scales]
    step = (S + 6 * 2.0**-10) * rows.astype(np.float64)[:, None]
    off = np.abs(values(m) - x.astype(np.float64))
    bad = np.argwhere(off > np.repeat(step, 16, axis=1) + 2.0**-20 * np.abs(x))
    assert bad.size == 0, f"row of 2^{e[bad[0][0]]}: off by {off[tuple(bad[0])]}, {len(bad)} values"
    assert not (codes[x == 0] & 7).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,n,k", [(1, 8, 64), (20, 264, 4096), (100, 520, 256), (600, 520, 512)])
def test_product_of_large_and_small_rows(cuda_ok, fmt, t, n, k):
    """Factors of rows far apart: every value whose terms stay in range is right."""
    rng = np.random.default_rng(t)
    w = rng.standard_normal((n, k)).astype(np.float32)
    x = rng.standard_normal((t, k)).astype(np.float32)
    for ex, ew in ((120, -10), (110, -100), (-100, 110), (-80, 80), (122, -60)):
        a = sharq.quantize_fp4(to_dev(x * np.float32(2.0**ex), "f32"), fmt)
        b = sharq.quantize_fp4(to_dev(w * np.float32(2.0**ew), "f32"), fmt)
        xv, wv = values(a), values(b)
        y = sharq.linear_fp4(a, b, out_dtype=torch.float32)
        sharq.sharq_sync_status()
        check_product(y.cpu().numpy(), xv, wv, False, f"2^{ex} x 2^{ew}")
        assert torch.equal(sharq.linear_fp4(a, b), y.to(torch.bfloat16))
        offsets = torch.tensor([0, (t + 127) // 128 * 128], dtype=torch.int32).cuda()
        g = sharq.linear_fp4_grouped(a, b, offsets, out_dtype=torch.float32)
        check_product(g.cpu().numpy(), xv, wv, False, f"grouped, 2^{ex} x 2^{ew}")
        # one large row among ordinary ones
        x1 = x.copy()
        x1[t // 2] *= np.float32(2.0**120)
        a = sharq.quantize_fp4(to_dev(x1, "f32"), fmt)
        c = sharq.quantize_fp4(to_dev(w * np.float32(2.0**-20), "f32"), fmt)
        for z in (sharq.linear_fp4(a, c, out_dtype=torch.float32), sharq.linear_fp4_grouped(a, c, offsets, out_dtype=torch.float32)):
            check_product(z.cpu().numpy(), values(a), values(c), False, "one large row")
