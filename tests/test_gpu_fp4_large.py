"""The plain FP4 layers and routing where element and byte offsets pass 32 bits: the far end against the same rows alone."""
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq
from fp4_common import check_product

pytestmark = pytest.mark.gpu


def _parts(m, lo, hi):
    """Codes, scale words and factors of the rows [lo, hi) of a one-expert matrix, lo a multiple of 128."""
    per = m.k // (16 if m.fmt == 1 else 32)
    block = (per + 3) // 4 * 512
    scales = m.scales[lo // 128 * block : (hi + 127) // 128 * block].view(-1, (per + 3) // 4, 32, 4, 4)
    scales = scales.permute(0, 3, 2, 1, 4).reshape(-1, (per + 3) // 4 * 4)[: hi - lo]
    return m.codes.view(m.rows, m.k // 2)[lo:hi], scales, m.row_scale[lo:hi]


def _same(a, b):
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_and_gather(cuda_ok, fmt):
    t, k = 135000, 16384  # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((t, k), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.rand((k,), generator=g, device="cuda").bfloat16()
    lo = t // 128 * 128 - 128
    m = sharq.quantize_fp4(x, fmt, gamma=gamma)
    tail = sharq.quantize_fp4(x[lo:], fmt, gamma=gamma)
    _same(_parts(m, lo, t), _parts(tail, 0, t - lo))
    del m
    m = sharq.quantize_fp4_swiglu(x, x, fmt)
    _same(_parts(m, lo, t), _parts(sharq.quantize_fp4_swiglu(x[lo:], x[lo:], fmt), 0, t - lo))
    rows = torch.full((270000,), -1, dtype=torch.int32, device="cuda")  # 2.2e9 bytes of codes
    rows[-1000:] = torch.arange(t - 1000, t, dtype=torch.int32, device="cuda")
    big = sharq.gather_fp4(m, rows)
    lo2 = 270000 // 128 * 128 - 128
    _same(_parts(big, lo2, 270000), _parts(sharq.gather_fp4(m, rows[lo2:]), 0, 270000 - lo2))
    _same(_parts(big, lo2, 270000)[:1], (_parts(m, 0, t)[0][t - (270000 - lo2) :],))


def test_products(cuda_ok):
    """y of 2.3e9 values; stacked weights of 2.2e9 bytes."""
    g = torch.Generator(device="cuda").manual_seed(2)
    t, n, k = 140000, 16384, 64
    a = sharq.quantize_fp4(torch.randn((t, k), generator=g, device="cuda"), "nvfp4")
    w = sharq.quantize_fp4(torch.randn((n, k), generator=g, device="cuda"), "nvfp4")
    y = sharq.linear_fp4(a, w)
    grouped = sharq.linear_fp4_grouped(a, w, torch.tensor([0, (t + 127) // 128 * 128], dtype=torch.int32, device="cuda"))
    sharq.sharq_sync_status()

    def values(m, lo, hi):
        codes, scales, rows = _parts(m, lo, hi)
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
        v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(1)
        s = scales[:, : m.k // 16].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        return (v * s * rows.double()[:, None]).cpu().numpy()

    lo = t // 128 * 128 - 128
    xv, wv = values(a, lo, t), values(w, 0, n)
    for z in (y, grouped):
        check_product(z[lo:].float().cpu().numpy(), xv, wv, True, "last rows")
    del y, grouped
    experts, n, k = 66, 8192, 8192
    w = sharq.FP4Matrix(n, k, "nvfp4", experts)
    w.buffer.zero_()
    w1 = sharq.quantize_fp4(torch.randn((1, n, k), generator=g, device="cuda"), "nvfp4")
    for dst, src in ((w.codes, w1.codes), (w.scales, w1.scales), (w.row_scale, w1.row_scale)):
        dst[-src.numel() :] = src
    a = sharq.quantize_fp4(torch.randn((200, k), generator=g, device="cuda"), "nvfp4")
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    off[-1] = 256
    got = sharq.linear_fp4_grouped(a, w, off, out_dtype=torch.float32)
    want = sharq.linear_fp4_grouped(a, w1, off[-2:], out_dtype=torch.float32)
    assert torch.equal(got, want)


def test_combine(cuda_ok):
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, n, t = 270000, 8192, 270000  # 2.2e9 values in y and in out
    y = torch.randn((rows, n), generator=g, device="cuda", dtype=torch.bfloat16)
    slots = torch.randint(0, rows, (t, 2), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((t, 2), generator=g, device="cuda")
    out = sharq.combine(y, slots, w, add=y)
    pick = torch.tensor([0, 1, 131071, 131072, 262143, 262144, t - 2, t - 1], device="cuda")
    part = y[slots[pick].long()].double() * w[pick].double()[..., None]
    ref = part.sum(1) + y[pick].double()
    tol = 2 * 2.0**-24 * (part.abs().sum(1) + y[pick].double().abs())
    assert bool(((out[pick].double() - ref).abs() <= tol + 2.0**-8 * (ref.abs() + tol)).all())


def test_route_and_rows(cuda_ok):
    g = torch.Generator(device="cuda").manual_seed(4)
    t, experts = 4300000, 512  # 2.2e9 logits
    z = torch.randn((t, experts), generator=g, device="cuda", dtype=torch.bfloat16)
    ids, w = sharq.route(z, 8)
    for s in (slice(t - 3000, t), slice(2**31 // experts - 100, 2**31 // experts + 100)):
        i2, w2 = sharq.route(z[s], 8)
        assert torch.equal(ids[s], i2) and torch.equal(w[s], w2)
    del z
    r = sharq.route_rows(ids, experts)
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=experts)
    ends = ((counts + 127) // 128 * 128).cumsum(0)
    assert torch.equal(r.offsets[1:].long(), ends) and int(r.offsets[0]) == 0
    key, order = flat.sort(stable=True)
    slot = r.offsets[key].long() + torch.arange(len(flat), device="cuda") - (counts.cumsum(0) - counts)[key]
    assert torch.equal(r.slots.reshape(-1)[order].long(), slot)
    rows = torch.full_like(r.rows, -1)
    rows[slot] = (order // 8).to(torch.int32)
    assert torch.equal(r.rows, rows)
