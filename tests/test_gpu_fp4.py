"""The plain FP4 layers on the GPU: quantization bit for bit against the C oracle's blocks, products against 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from activation_sparsity_fp4_b200 import sharq, workloads
from fp4_common import check_product, padded_scales, quantized, read_matrix, values
from gpu_common import to_dev

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]


def _rows(seed, t, k, dtype="bf16"):
    rng = np.random.default_rng(seed)
    x = (0.5 * rng.standard_t(3, size=(t, k))).astype(np.float32)
    x[rng.random((t, k)) < 0.01] *= 40.0
    if t > 3:
        x[1] = 0.0                      # a row of zeros
        x[2, k // 2 :] *= np.float32(1e-6)  # blocks whose scale underflows
        x[3] *= np.float32(2.0**100)    # rows do not share a scale
    return workloads.to_bf16_values(x) if dtype == "bf16" else x


def _assert_matrix(m, want, zero_pad=True):
    got = read_matrix(m)
    for name, g, w in zip(("scales", "codes", "row scales"), got, want):
        bad = np.argwhere(g != w)
        assert bad.size == 0, f"{name}: {len(bad)} differ, first at {bad[0].tolist()}: {g[tuple(bad[0])]} for {w[tuple(bad[0])]}"
    if zero_pad:
        assert not padded_scales(m).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(1, 32), (5, 96), (130, 64), (33, 480), (7, 4096), (4, 5120), (3, 14336), (2, 20000)])
def test_quantize(cuda_ok, fmt, dtype, t, k):
    x = _rows(t + k, t, k, dtype)
    _assert_matrix(sharq.quantize_fp4(to_dev(x, dtype), fmt), quantized(x, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_one_amax_for_all_rows(cuda_ok, fmt):
    x = np.clip(_rows(3, 20, 256), -50, 50)
    _assert_matrix(sharq.quantize_fp4(to_dev(x, "bf16"), fmt, amax=50.0), quantized(x, fmt, amax=50.0))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_stacked_weight(cuda_ok, fmt):
    w = _rows(4, 3 * 200, 160).reshape(3, 200, 160)
    m = sharq.quantize_fp4(to_dev(w, "bf16"), fmt)
    assert (m.experts, m.rows, m.k) == (3, 200, 160)
    _assert_matrix(m, quantized(w.reshape(600, 160), fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_gathered_rows(cuda_ok, fmt, dtype):
    """Any order, the same row twice, zero rows for indexes out of range; rows from count on stay as they were."""
    x = _rows(5, 40, 224, dtype)
    rng = np.random.default_rng(6)
    rows = rng.integers(0, 40, 150).astype(np.int32)
    rows[[0, 7, 149]] = [-1, 40, 2**31 - 1]
    rows[20], rows[9] = -(2**31), rows[8]
    xr = np.where(((rows >= 0) & (rows < 40))[:, None], x[np.clip(rows, 0, 39)], np.float32(0))
    rd = torch.from_numpy(rows).cuda()
    _assert_matrix(sharq.quantize_fp4(to_dev(x, dtype), fmt, rows=rd), quantized(xr, fmt))
    for count in (0, 1, 100, 150, 1000):
        m = sharq.FP4Matrix(150, 224, fmt)
        for part in (m.codes, m.scales):
            part.fill_(0x22)
        m.row_scale.fill_(-1.0)
        sharq.quantize_fp4(to_dev(x, dtype), fmt, rows=rd, count=torch.tensor([count], dtype=torch.int32).cuda(), out=m)
        want = [a.copy() for a in quantized(xr, fmt)]
        for a, old in zip(want, (0x22, 2, -1.0)):
            a[count:] = old
        _assert_matrix(m, want, zero_pad=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t_dst,k", [(1, 32), (90, 224), (128, 2048), (300, 1056), (700, 8224)])
def test_gather(cuda_ok, fmt, t_dst, k):
    """FP4 rows by index are what quantizing the gathered rows gives, at fewer and at more rows than the source has."""
    x = _rows(k, 150, k)
    rng = np.random.default_rng(t_dst)
    rows = rng.integers(0, 150, t_dst).astype(np.int32)
    rows[rng.random(t_dst) < 0.2] = -1
    rows[0] = 150
    if t_dst > 5:
        rows[[2, 3, 4]] = [149, 149, 2**31 - 1]
    xr = np.where(((rows >= 0) & (rows < 150))[:, None], x[np.clip(rows, 0, 149)], np.float32(0))
    want, rd, xd = quantized(xr, fmt), torch.from_numpy(rows).cuda(), to_dev(x, "bf16")
    src = sharq.quantize_fp4(xd, fmt)
    _assert_matrix(sharq.gather_fp4(src, rd), want)
    _assert_matrix(sharq.quantize_fp4(xd, fmt, rows=rd), want)
    for count in (0, 1, t_dst // 2, t_dst, t_dst + 9):
        m = sharq.FP4Matrix(t_dst, k, fmt)
        for part in (m.codes, m.scales):
            part.fill_(0x22)
        m.row_scale.fill_(-1.0)
        sharq.gather_fp4(src, rd, count=torch.tensor([count], dtype=torch.int32).cuda(), out=m)
        part = [a.copy() for a in want]
        for a, old in zip(part, (0x22, 2, -1.0)):
            a[count:] = old
        _assert_matrix(m, part, zero_pad=False)
    with pytest.raises(ValueError):
        sharq.gather_fp4(src, torch.arange(150, dtype=torch.int32).cuda(), out=src)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_norm_with_an_exact_factor(cuda_ok, fmt, dtype):
    """Rows of one magnitude 2^a: the mean square is a power of four, the factor exact, and so is every step but gamma's."""
    rng = np.random.default_rng(7)
    t, k = 9, 1056
    x = rng.choice([-1.0, 1.0], size=(t, k)).astype(np.float32) * np.float32(2.0) ** rng.integers(-6, 7, (t, 1)).astype(np.float32)
    gamma = workloads.to_bf16_values(rng.uniform(0.01, 1.5, k).astype(np.float32))
    m = sharq.quantize_fp4(to_dev(x, dtype), fmt, gamma=to_dev(gamma, dtype), eps=0.0)
    _assert_matrix(m, quantized(np.sign(x) * gamma, fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,k", [(1, 32), (6, 4096), (40, 992), (3, 20000)])
def test_quantize_norm(cuda_ok, fmt, t, k):
    """Against RMSNorm in 64 bits.  An element is off by half the widest E2M1 step (1 of 4..6) of its block scale S:
    NVFP4's S is E4M3, within 2^-4 of its value (6 x 2^-4 < 1 beyond the grid) or, below 2^-6, within 2^-10, times the
    row's factor; MXFP4's elements reach just under 8 and are cut to 6.  h in fp32 is off by under 2^-20 of itself
    (a sum of k squares in a tree of at most 17 levels behind up to 160 in a row, halved by the root)."""
    x = _rows(t, t, k, "f32")
    gamma = np.random.default_rng(8).uniform(0.5, 1.5, k).astype(np.float32)
    m = sharq.quantize_fp4(to_dev(x, "f32"), fmt, gamma=to_dev(gamma, "f32"))
    h = x.astype(np.float64)
    h = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * gamma
    scales, _, rows = read_matrix(m)
    b = k // scales.shape[1]
    S = np.array([oracle.e8m0_decode([c])[0] if fmt == "mxfp4" else oracle.e4m3_decode([c])[0] for c in range(256 if fmt == "mxfp4" else 127)],
                 np.float64)[scales]
    step = 2.0 * S if fmt == "mxfp4" else (S + 6 * 2.0**-10) * rows.astype(np.float64)[:, None]
    assert np.all(np.abs(values(m) - h) <= np.repeat(step, b, axis=1) + 2.0**-20 * np.abs(h))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(1, 32), (21, 768), (3, 14336)])
def test_quantize_swiglu(cuda_ok, fmt, dtype, t, k):
    """Bit for bit; gate and up as the halves of one product, and apart."""
    rng = np.random.default_rng(9)
    gu = (2 * rng.standard_normal((t, 2 * k))).astype(np.float32)
    gu = workloads.to_bf16_values(gu) if dtype == "bf16" else gu
    h = oracle.swiglu(gu[:, :k], gu[:, k:])
    d = to_dev(gu, dtype)
    want = quantized(h, fmt)
    _assert_matrix(sharq.quantize_fp4_swiglu(d[:, :k], d[:, k:], fmt), want)
    _assert_matrix(sharq.quantize_fp4_swiglu(d[:, :k].contiguous(), d[:, k:], fmt), want)
    count = torch.tensor([t // 2], dtype=torch.int32).cuda()
    m = sharq.FP4Matrix(t, k, fmt)
    m.codes.fill_(0x11)
    sharq.quantize_fp4_swiglu(d[:, :k], d[:, k:], fmt, count=count, out=m)
    codes = want[1].copy()
    codes[t // 2 :] = 1
    assert np.array_equal(read_matrix(m)[1], codes)


def test_quantize_strides_and_alignment(cuda_ok):
    base = _rows(10, 30, 1000)
    for dtype in ("bf16", "f32"):
        d = to_dev(base, dtype)
        for cut in (slice(0, 96), slice(8, 104), slice(3, 99)):
            _assert_matrix(sharq.quantize_fp4(d[:, cut], "nvfp4"), quantized(base[:, cut], "nvfp4"))
        _assert_matrix(sharq.quantize_fp4(d[::3, :64], "mxfp4"), quantized(base[::3, :64], "mxfp4"))
        _assert_matrix(sharq.quantize_fp4(d[:1].expand(5, 1000)[:, :64], "mxfp4"), quantized(np.repeat(base[:1, :64], 5, 0), "mxfp4"))
        t = d[:, :64].t()  # (64, 30): not a multiple of 32
        with pytest.raises(sharq.SharqError):
            sharq.quantize_fp4(t, "nvfp4")


def test_python_refusals(cuda_ok):
    x = torch.zeros((4, 64), device="cuda")
    i32 = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, w = sharq.quantize_fp4(x, "nvfp4"), sharq.quantize_fp4(torch.zeros((16, 64), device="cuda"), "nvfp4")
    for bad in (lambda: sharq.quantize_fp4(x[0], "nvfp4"), lambda: sharq.quantize_fp4(x.half(), "nvfp4"),
                lambda: sharq.quantize_fp4(x, "nvfp4", rows=i32.long()), lambda: sharq.quantize_fp4(x, "nvfp4", rows=i32.cpu()),
                lambda: sharq.quantize_fp4(x, "nvfp4", gamma=x[0, :32]), lambda: sharq.quantize_fp4(x, "nvfp4", count=i32),
                lambda: sharq.quantize_fp4(x, "nvfp4", out=w), lambda: sharq.quantize_fp4(x, "mxfp4", out=a),
                lambda: sharq.quantize_fp4(x.view(2, 2, 64), "nvfp4", rows=i32),
                lambda: sharq.quantize_fp4_swiglu(x, x[:2], "nvfp4"), lambda: sharq.quantize_fp4_swiglu(x, x.bfloat16(), "nvfp4"),
                lambda: sharq.linear_fp4(a, w, out=x), lambda: sharq.linear_fp4_grouped(a, w, i32),
                lambda: sharq.gather_fp4(a, i32.long()), lambda: sharq.linear_fp4(a, w, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sharq.quantize_fp4(x[:0], "nvfp4"), lambda: sharq.quantize_fp4(x[:, :40], "nvfp4"),
                lambda: sharq.linear_fp4(w, sharq.quantize_fp4(x, "mxfp4")), lambda: sharq.linear_fp4(w, a),
                lambda: sharq.linear_fp4(a, sharq.quantize_fp4(torch.zeros((2, 8, 64), device="cuda"), "nvfp4"))):
        with pytest.raises(sharq.SharqError):
            bad()


def test_bad_rows_stay_by_themselves(cuda_ok):
    """A row with NaN or an infinity has no defined value; the others keep theirs."""
    x = _rows(11, 12, 128)
    y = x.copy()
    y[5, 7], y[8, 100] = np.nan, np.inf
    w = sharq.quantize_fp4(to_dev(_rows(12, 64, 128), "bf16"), "nvfp4")
    a = sharq.linear_fp4(sharq.quantize_fp4(to_dev(x, "f32"), "nvfp4"), w, out_dtype=torch.float32)
    b = sharq.linear_fp4(sharq.quantize_fp4(to_dev(y, "f32"), "nvfp4"), w, out_dtype=torch.float32)
    keep = [i for i in range(12) if i not in (5, 8)]
    assert torch.equal(a[keep], b[keep])


# ---------------------------------------------------------------- product
SHAPES = [(1, 8, 32), (1, 256, 256), (2, 40, 64), (16, 4096, 288), (31, 136, 1024), (32, 128, 96), (33, 264, 512),
          (64, 384, 4096), (65, 128, 256), (100, 1000, 640), (127, 8, 160), (128, 256, 14336), (129, 520, 352),
          (255, 256, 992), (256, 512, 256), (257, 776, 2048), (300, 2056, 224), (512, 4096, 512), (1000, 72, 4096),
          (2049, 264, 288)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_linear(cuda_ok, fmt, t, n, k):
    x, w = _rows(t, t, k), _rows(n, n, k) * np.float32(0.02)
    if t > 3:
        x[3] *= np.float32(2.0**-100)
    if n > 3:
        w[3] *= np.float32(2.0**-100)
    a, b = sharq.quantize_fp4(to_dev(x, "bf16"), fmt), sharq.quantize_fp4(to_dev(w, "f32"), fmt)
    xv, wv = values(a), values(b)
    y = sharq.linear_fp4(a, b, out_dtype=torch.float32)
    sharq.sharq_sync_status()
    check_product(y.cpu().numpy(), xv, wv, False, "fp32")
    yb = sharq.linear_fp4(a, b)
    assert torch.equal(yb, y.to(torch.bfloat16)), "bf16 output is the fp32 output rounded once"
    assert torch.equal(sharq.linear_fp4(a, b, out_dtype=torch.float32), y), "results repeat"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,n,k", [(40, 64, 4096), (200, 256, 512), (600, 520, 288), (3, 264, 14336)])
def test_linear_exact_sums(cuda_ok, fmt, t, n, k):
    """E2M1 grid values with every block's and row's largest magnitude 6: scales are powers of two (MXFP4: 2^0) or one
    constant (NVFP4: 448), every product a multiple of 1/4 and every partial sum below 2^24 quarters: no rounding."""
    rng = np.random.default_rng(13)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
    x, w = (rng.choice(grid, (r, k)) * rng.choice([-1, 1], (r, k)).astype(np.float32) for r in (t, n))
    x[:, ::16] = 6.0
    w[:, ::16] = -6.0
    a, b = sharq.quantize_fp4(to_dev(x, "bf16"), fmt), sharq.quantize_fp4(to_dev(w, "bf16"), fmt)
    y = sharq.linear_fp4(a, b, out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    ref = x.astype(np.float64) @ w.astype(np.float64).T
    if fmt == "mxfp4":
        assert np.array_equal(y, ref)
    else:  # 448 x 448 times the row factors 6 / 2688 (rounded to fp32), two products rounded
        assert np.all(np.abs(y - ref) <= 4 * 2.0**-24 * np.abs(ref))


def test_guard_rows_and_columns(cuda_ok):
    """Nothing is written outside y."""
    for t, n, k in ((5, 40, 96), (70, 264, 64), (300, 520, 128)):
        a, b = (sharq.quantize_fp4(to_dev(_rows(r, r, k), "bf16"), "nvfp4") for r in (t, n))
        for dtype in (torch.bfloat16, torch.float32):
            buf = torch.full((t + 40, n), 77.0, dtype=dtype, device="cuda")
            y = sharq.linear_fp4(a, b, out=buf[16 : 16 + t])
            assert torch.equal(y, sharq.linear_fp4(a, b, out_dtype=dtype))
            assert bool((buf[:16] == 77).all()) and bool((buf[16 + t :] == 77).all())


# ---------------------------------------------------------------- grouped
def _grouped_case(seed, counts, n, k, fmt, extra=0):
    ends = np.cumsum([(c + 127) // 128 * 128 for c in counts])
    offsets = np.concatenate([[0], ends]).astype(np.int32)
    x = _rows(seed, max(1, int(offsets[-1]) + extra), k)
    w = (_rows(seed + 1, len(counts) * n, k) * np.float32(0.02)).reshape(len(counts), n, k)
    a, b = sharq.quantize_fp4(to_dev(x, "bf16"), fmt), sharq.quantize_fp4(to_dev(w, "f32"), fmt)
    return a, b, offsets


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,n,k", [([1], 8, 32), ([5, 0, 130, 1], 264, 96), ([0, 0, 300], 40, 512),
                                        ([128] * 5, 512, 224), ([1] * 40, 136, 768), ([700, 3, 0, 260], 1000, 288),
                                        ([0, 0, 0], 64, 64)])
def test_grouped(cuda_ok, fmt, counts, n, k):
    """Empty experts, one row, several tiles; rows behind the last group stay as they were."""
    a, b, offsets = _grouped_case(len(counts) + n, counts, n, k, fmt, extra=200)
    od = torch.from_numpy(offsets).cuda()
    xv, wv = values(a), values(b).reshape(len(counts), n, k)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((a.rows, n), -9.0, dtype=dtype, device="cuda")
        sharq.linear_fp4_grouped(a, b, od, out=y)
        sharq.sharq_sync_status()
        got = y.float().cpu().numpy()
        for e in range(len(counts)):
            r = slice(int(offsets[e]), int(offsets[e + 1]))
            check_product(got[r], xv[r], wv[e], dtype == torch.bfloat16, f"expert {e}")
        assert np.all(got[offsets[-1] :] == -9.0)


def test_grouped_rows_in_front_of_the_first_group(cuda_ok):
    """Offsets need not begin at 0: the rows before them are in no group."""
    a, b, _ = _grouped_case(60, [300, 200, 100], 136, 288, "nvfp4")
    offsets = np.array([128, 128, 512, 640], np.int32)
    y = torch.full((a.rows, 136), -9.0, dtype=torch.float32, device="cuda")
    sharq.linear_fp4_grouped(a, b, torch.from_numpy(offsets).cuda(), out=y)
    sharq.sharq_sync_status()
    xv, wv, got = values(a), values(b).reshape(3, 136, 288), y.cpu().numpy()
    check_product(got[128:512], xv[128:512], wv[1], False)
    check_product(got[512:640], xv[512:640], wv[2], False)
    assert np.all(got[:128] == -9.0) and np.all(got[640:] == -9.0)


def test_grouped_many_experts(cuda_ok):
    """More experts than a block holds the offsets of; a few have rows."""
    counts = [0] * 1100
    for e, c in ((3, 130), (1023, 5), (1024, 128), (1099, 40)):
        counts[e] = c
    a, b, offsets = _grouped_case(70, counts, 8, 64, "nvfp4")
    y = sharq.linear_fp4_grouped(a, b, torch.from_numpy(offsets).cuda(), out_dtype=torch.float32)
    xv, wv, got = values(a), values(b).reshape(1100, 8, 64), y.cpu().numpy()
    for e in (3, 1023, 1024, 1099):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        check_product(got[r], xv[r], wv[e], False, f"expert {e}")


def test_grouped_clips_the_last_tile(cuda_ok):
    """x->rows need not be whole tiles: the last group ends at the rows there are."""
    a, b, offsets = _grouped_case(50, [100, 200], 72, 64, "nvfp4", extra=-90)
    assert a.rows == int(offsets[-1]) - 90
    buf = torch.full((a.rows + 64, 72), 5.0, dtype=torch.float32, device="cuda")
    y = sharq.linear_fp4_grouped(a, b, torch.from_numpy(offsets).cuda(), out=buf[: a.rows])
    xv, wv = values(a), values(b).reshape(2, 72, 64)
    check_product(y[:128].cpu().numpy(), xv[:128], wv[0], False)
    check_product(y[128:].cpu().numpy(), xv[128:], wv[1], False)
    assert bool((buf[a.rows :] == 5.0).all())
