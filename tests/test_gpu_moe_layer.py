"""The plain FP4 operators and expert routing together, as a mixture-of-experts layer runs them: in sequence, in a
captured graph, on several streams."""
import numpy as np
import pytest
import torch

import oracle
from activation_sparsity_fp4_b200 import sharq, workloads
from fp4_common import check_product, laid_out, quantized, read_matrix, routed, values
from gpu_common import to_dev

pytestmark = pytest.mark.gpu


class Layer:
    """Router and experts of one layer; nothing is read back by the host."""

    def __init__(self, seed, experts, top_k, hidden, inter, fmt):
        g = torch.Generator().manual_seed(seed)
        self.experts, self.top_k, self.inter, self.fmt = experts, top_k, inter, fmt
        self.bias = (0.05 * torch.randn((experts,), generator=g)).cuda()
        w1 = 0.05 * torch.randn((experts, 2 * inter, hidden), generator=g)
        w2 = 0.05 * torch.randn((experts, hidden, inter), generator=g)
        self.w1, self.w2 = sharq.quantize_fp4(w1.cuda(), fmt), sharq.quantize_fp4(w2.cuda(), fmt)

    def __call__(self, x, logits, stream=None):
        s = dict(stream=stream)
        ids, weights = sharq.route(logits, self.top_k, score="sigmoid", bias=self.bias, groups=4, top_groups=2,
                                   group_top=2, scale=1.5, **s)
        r = sharq.route_rows(ids, self.experts, **s)
        used = r.offsets[-1:]
        a = sharq.quantize_fp4(x, self.fmt, rows=r.rows, count=used, **s)
        gu = sharq.linear_fp4_grouped(a, self.w1, r.offsets, **s)
        b = sharq.quantize_fp4_swiglu(gu[:, : self.inter], gu[:, self.inter :], self.fmt, count=used, **s)
        y = sharq.linear_fp4_grouped(b, self.w2, r.offsets, **s)
        out = sharq.combine(y, r.slots, weights, add=x, **s)
        return dict(ids=ids, weights=weights, r=r, a=a, gu=gu, b=b, y=y, out=out)


def _tokens(seed, t, hidden, experts):
    rng = np.random.default_rng(seed)
    x = workloads.to_bf16_values((0.5 * rng.standard_t(3, size=(t, hidden))).astype(np.float32))
    return to_dev(x, "bf16"), torch.from_numpy(rng.standard_normal((t, experts)).astype(np.float32)).cuda()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("t,experts,top_k,hidden,inter", [(1, 8, 3, 256, 96), (150, 16, 4, 512, 160), (700, 8, 2, 288, 64)])
def test_layer(cuda_ok, fmt, t, experts, top_k, hidden, inter):
    """Every step against its plain form on what the step before it left."""
    m = Layer(t, experts, top_k, hidden, inter, fmt)
    x, logits = _tokens(t, t, hidden, experts)
    s = m(x, logits)
    sharq.sharq_sync_status()
    ids, w = routed(logits.cpu().numpy().astype(np.float64), top_k, "sigmoid", m.bias.cpu().numpy(), 4, 2, 2, True, 1.5)
    assert np.array_equal(s["ids"].cpu().numpy(), ids)
    assert np.all(np.abs(s["weights"].cpu().numpy() - w) <= 2 * 27 * 2.0**-24 * w)
    rows, offsets, slots = laid_out(ids, experts, sharq.sharq_route_rows_capacity(t, top_k, experts))
    n = int(offsets[-1])
    for got, want in zip(s["r"], (rows, offsets, slots)):
        assert np.array_equal(got.cpu().numpy(), want)
    xr = np.where((rows >= 0)[:, None], x.float().cpu().numpy()[np.clip(rows, 0, None)], np.float32(0))
    gu, y = s["gu"].float().cpu().numpy(), s["y"].float().cpu().numpy()
    for got, want in zip(read_matrix(s["a"]), quantized(xr, fmt)):
        assert np.array_equal(got[:n], want[:n])
    h = oracle.swiglu(gu[:n, :inter], gu[:n, inter:])
    for got, want in zip(read_matrix(s["b"]), quantized(h, fmt)):
        assert np.array_equal(got[:n], want)
    av, bv = values(s["a"]), values(s["b"])
    w1, w2 = (values(v).reshape(experts, v.rows, v.k) for v in (m.w1, m.w2))
    for e in range(experts):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        check_product(gu[at], av[at], w1[e], True, f"gate/up, expert {e}")
        check_product(y[at], bv[at], w2[e], True, f"down, expert {e}")
    part = y[:n].astype(np.float64)[slots] * s["weights"].cpu().numpy().astype(np.float64)[..., None]
    ref = part.sum(1) + x.float().cpu().numpy()
    tol = top_k * 2.0**-24 * (np.abs(part).sum(1) + np.abs(x.float().cpu().numpy()))
    tol = tol + 2.0**-8 * (np.abs(ref) + tol)
    assert np.all(np.abs(s["out"].float().cpu().numpy() - ref) <= tol)


def _same(a, b):
    n = int(a["r"].offsets[-1])
    assert torch.equal(a["ids"], b["ids"]) and torch.equal(a["weights"], b["weights"])
    assert all(torch.equal(u, v) for u, v in zip(a["r"], b["r"]))
    assert torch.equal(a["gu"][:n], b["gu"][:n]) and torch.equal(a["y"][:n], b["y"][:n])
    assert torch.equal(a["out"], b["out"])


def test_layer_in_a_graph(cuda_ok):
    """Captured once, replayed on other tokens and other assignments: the same bits as run directly.  Two graphs of
    the same layer share no state, in either order."""
    t, experts, hidden = 60, 16, 512
    m = Layer(1, experts, 4, hidden, 160, "nvfp4")
    x, logits = (v.clone() for v in _tokens(2, t, hidden, experts))
    x2, logits2 = _tokens(3, 33, hidden, experts)
    m(x, logits), m(x2, logits2)  # first calls
    torch.cuda.synchronize()
    graphs, kept = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, (a, b) in zip(graphs, ((x, logits), (x2, logits2))):
        with torch.cuda.graph(g):
            kept.append(m(a, b))
    for seed in (4, 5, 6):
        nx, nl = _tokens(seed, t, hidden, experts)
        x.copy_(nx)
        logits.copy_(nl)
        graphs[seed % 2].replay()
        graphs[1 - seed % 2].replay()
        torch.cuda.synchronize()
        _same(kept[0], m(nx, nl))
        _same(kept[1], m(x2, logits2))
    sharq.sharq_sync_status()


def test_layer_on_other_streams(cuda_ok):
    """On a stream given as an object, as a handle, as the current one; and on two streams at once."""
    experts, hidden = 16, 512
    m = Layer(7, experts, 4, hidden, 160, "mxfp4")
    calls = [_tokens(8 + i, 200 + 50 * i, hidden, experts) for i in range(2)]
    want = [m(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    _same(want[0], m(*calls[0], stream=streams[0]))
    _same(want[0], m(*calls[0], stream=streams[1].cuda_stream))
    with torch.cuda.stream(streams[1]):
        _same(want[0], m(*calls[0]))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(m(*c))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            _same(a, b)
    big = sharq.quantize_fp4(torch.randn((4096, 1024), device="cuda"), "nvfp4")
    a = [sharq.quantize_fp4(torch.randn((t, 1024), device="cuda"), "nvfp4") for t in (3, 700)]
    want = [sharq.linear_fp4(v, big) for v in a]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, v in zip(streams, a):
            with torch.cuda.stream(s):
                got.append(sharq.linear_fp4(v, big))
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, got))
    sharq.sharq_sync_status()
