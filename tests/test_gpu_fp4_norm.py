"""RMSNorm and SwiGLU in front of FP4 quantization at the sizes of a prompt: bit for bit against the oracle's fixed order
of steps, and a row's FP4 form whatever batch it is quantized in."""
import numpy as np
import pytest
import torch

import oracle
from activation_sparsity_fp4_b200 import sharq, workloads
from fp4_common import quantized, read_matrix
from gpu_common import to_dev

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]


def _rows(seed, t, k, dtype):
    rng = np.random.default_rng(seed)
    x = (0.5 * rng.standard_normal((t, k), dtype=np.float32)) * np.float32(2.0) ** rng.integers(-8, 9, (t, 1)).astype(np.float32)
    x[rng.random((t, k), dtype=np.float32) < 0.01] *= np.float32(40.0)
    x[t // 2] = 0.0
    return workloads.to_bf16_values(x) if dtype == "bf16" else x


def _gamma(seed, k, dtype):
    g = np.random.default_rng(seed).uniform(0.5, 1.5, k).astype(np.float32)
    return workloads.to_bf16_values(g) if dtype == "bf16" else g


def _normed(x, gamma, eps=1e-6):
    """(x r) gamma, two products rounded once in fp32, r in the oracle's order of steps."""
    r = np.array([oracle.rms_rstd(row, eps) for row in x], np.float32)
    return (x * r[:, None]) * gamma


def _assert_rows(m, want, n=None):
    for name, g, w in zip(("scales", "codes", "row scales"), read_matrix(m), want):
        bad = np.argwhere(g[:n] != w[:n])
        assert bad.size == 0, f"{name}: {len(bad)} differ, first at {bad[0].tolist()}: {g[tuple(bad[0])]} for {w[tuple(bad[0])]}"


# one, two and four units of 16 a lane; one warp a row to 32; rows that a block takes one of, and several in turn
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(1, 32), (149, 512), (300, 544), (148, 4096), (149, 4096), (160, 1056), (200, 5120),
                                 (3, 14336), (149, 8192), (151, 8224), (149, 14336), (150, 16384)])
def test_norm_bit_for_bit(cuda_ok, fmt, dtype, t, k):
    x, gamma = _rows(t + k, t, k, dtype), _gamma(k, k, dtype)
    m = sharq.quantize_fp4(to_dev(x, dtype), fmt, gamma=to_dev(gamma, dtype))
    _assert_rows(m, quantized(_normed(x, gamma), fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [2048, 4096, 5120, 8224, 20000])
def test_form_of_a_row_does_not_depend_on_its_batch(cuda_ok, fmt, k):
    """Batches of 1, 148, 149 and 1000 rows, a gather of rows, and rows gathered while they are quantized."""
    t = 1000
    x, gamma = to_dev(_rows(k, t, k, "bf16"), "bf16"), to_dev(_gamma(k, k, "bf16"), "bf16")
    want = read_matrix(sharq.quantize_fp4(x, fmt, gamma=gamma))
    for at, n in ((0, 1), (777, 1), (0, 148), (300, 148), (300, 149), (851, 149)):
        got = read_matrix(sharq.quantize_fp4(x[at : at + n], fmt, gamma=gamma))
        for g, w in zip(got, want):
            assert np.array_equal(g, w[at : at + n]), (at, n)
    rng = np.random.default_rng(1)
    for src, n in ((1000, 500), (100, 150), (100, 1200)):  # quantized as they are taken; with more rows than x, gathered
        rows = rng.integers(0, src, n).astype(np.int32)
        got = read_matrix(sharq.quantize_fp4(x[:src], fmt, gamma=gamma, rows=torch.from_numpy(rows).cuda()))
        for g, w in zip(got, want):
            assert np.array_equal(g, w[rows]), (src, n)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("front", ["none", "norm", "swiglu"])
@pytest.mark.parametrize("dtype,t,k", [("f32", 40000, 96), ("bf16", 18000, 544), ("bf16", 2700, 5120), ("f32", 2700, 4096),
                                       ("bf16", 1500, 8224)])
def test_rows_in_turn(cuda_ok, fmt, front, dtype, t, k):
    """So many rows that every block takes three and more, the next one's loads in flight; rows and count with it."""
    x, y = _rows(t, t, k, dtype), _rows(t + 1, t, k, dtype)
    x, y = np.clip(x, -60, 60), np.clip(y, -60, 60)
    gamma = _gamma(k, k, dtype)
    xd, n = to_dev(x, dtype), t - t // 5
    count = torch.tensor([n], dtype=torch.int32).cuda()
    if front == "swiglu":
        h = oracle.swiglu(x, y)
        _assert_rows(sharq.quantize_fp4_swiglu(xd, to_dev(y, dtype), fmt), quantized(h, fmt))
        m = sharq.FP4Matrix(t, k, fmt)
        m.buffer.fill_(0x11)
        sharq.quantize_fp4_swiglu(xd, to_dev(y, dtype), fmt, count=count, out=m)
        want = quantized(h[:n], fmt)
    else:
        g = to_dev(gamma, dtype) if front == "norm" else None
        h = _normed(x, gamma) if front == "norm" else x
        _assert_rows(sharq.quantize_fp4(xd, fmt, gamma=g), quantized(h, fmt))
        rows = np.random.default_rng(3).integers(-t // 8, t + t // 8, t).astype(np.int32)
        m = sharq.FP4Matrix(t, k, fmt)
        m.buffer.fill_(0x11)
        sharq.quantize_fp4(xd, fmt, gamma=g, rows=torch.from_numpy(rows).cuda(), count=count, out=m)
        ok = (rows >= 0) & (rows < t)
        want = quantized(np.where(ok[:, None], h[np.clip(rows, 0, t - 1)], np.float32(0))[:n], fmt)
    _assert_rows(m, want, n)
    assert bool((m.codes[n * k // 2 :] == 0x11).all()), "rows from count on were written"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(300, 608), (149, 4096), (160, 8192), (149, 8224), (150, 14336), (4, 20000)])
def test_swiglu_bit_for_bit(cuda_ok, fmt, dtype, t, k):
    x, y = (np.clip(_rows(t + s, t, k, dtype), -60, 60) for s in (0, 1))
    _assert_rows(sharq.quantize_fp4_swiglu(to_dev(x, dtype), to_dev(y, dtype), fmt), quantized(oracle.swiglu(x, y), fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype,rows,k", [("bf16", 33000, 256), ("bf16", 33000, 576), ("bf16", 600, 576), ("f32", 600, 576),
                                          ("f32", 600, 800), ("bf16", 600, 5120)])
def test_swiglu_of_routed_rows(cuda_ok, fmt, dtype, rows, k):
    """Mostly padding, with a count, on every side of the rule for units a lane: the form of each row quantized alone."""
    rng = np.random.default_rng(rows + k)
    t = 40
    x, y = (np.clip(_rows(s, t, k, dtype), -60, 60) for s in (0, 1))
    want = quantized(oracle.swiglu(x, y), fmt)
    zero = [a[0] for a in quantized(np.zeros((1, k), np.float32), fmt)]
    pick = np.where(rng.random(rows) < 0.05, rng.integers(0, t, rows), -1)
    gu = torch.zeros((rows, 2 * k), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    at = torch.from_numpy(np.flatnonzero(pick >= 0)).cuda()
    src = torch.from_numpy(pick[pick >= 0]).cuda()
    gu[at, :k], gu[at, k:] = to_dev(x, dtype)[src], to_dev(y, dtype)[src]
    n = rows - 100
    m = sharq.quantize_fp4_swiglu(gu[:, :k], gu[:, k:], fmt, count=torch.tensor([n], dtype=torch.int32).cuda())
    for got, w, z in zip(read_matrix(m), want, zero):
        full = np.broadcast_to(z, (rows,) + z.shape).copy()
        full[pick >= 0] = w[pick[pick >= 0]]
        assert np.array_equal(got[:n], full[:n])
