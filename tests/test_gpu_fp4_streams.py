"""Calls on a stream of their own whose inputs the caller drops at once."""
import pytest
import torch

from activation_sparsity_fp4_b200 import sharq

pytestmark = pytest.mark.gpu


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    w = sharq.quantize_fp4(r(2, 256, 512), "nvfp4")
    off = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    return {
        "quantize": lambda: ((r(300, 512), i(300, 250), r(512)), lambda x, rows, gamma, **k: sharq.quantize_fp4(x, "nvfp4", rows=rows, gamma=gamma, **k).buffer),
        "quantize and gather": lambda: ((r(300, 512), i(300, 900)), lambda x, rows, **k: sharq.quantize_fp4(x, "mxfp4", rows=rows, **k).buffer),
        "swiglu": lambda: ((r(300, 512), r(300, 512)), lambda a, b, **k: sharq.quantize_fp4_swiglu(a, b, "mxfp4", **k).buffer),
        "gather": lambda: ((sharq.quantize_fp4(r(300, 512), "nvfp4"), i(300, 900)), lambda m, rows, **k: sharq.gather_fp4(m, rows, **k).buffer),
        "linear": lambda: ((sharq.quantize_fp4(r(300, 512), "nvfp4"), sharq.quantize_fp4(r(256, 512), "nvfp4")), lambda m, v, **k: sharq.linear_fp4(m, v, **k)),
        "grouped": lambda: ((sharq.quantize_fp4(r(256, 512), "nvfp4"),), lambda m, **k: sharq.linear_fp4_grouped(m, w, off, **k)),
        "route": lambda: ((r(3000, 64), r(64)), lambda z, b, **k: sharq.route(z, 6, bias=b, **k)[0]),
        "rows": lambda: ((i(16, 5000, 4),), lambda ids, **k: sharq.route_rows(ids, 16, **k).slots),
        "combine": lambda: ((r(900, 512), i(900, 300, 3), r(300, 3), r(300, 512)), lambda y, s, v, a, **k: sharq.combine(y, s, v, add=a, **k)),
    }


@pytest.mark.parametrize("name", ["quantize", "quantize and gather", "swiglu", "gather", "linear", "grouped", "route", "rows",
                                  "combine"])
def test_inputs_dropped_at_once(cuda_ok, name):
    """The stream is busy when the call is made, and the memory of what the call reads is asked for again meanwhile."""
    make = _inputs(1)[name]
    args, call = make()
    want = call(*args)
    scales = name in ("quantize", "quantize and gather", "swiglu", "gather")
    del args
    args, call = _inputs(1)[name]()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    got = call(*args, stream=side)
    sizes = [(a.buffer if isinstance(a, sharq.FP4Matrix) else a).nbytes for a in args]
    del args
    junk = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert len(junk) == 3 * len(sizes)
    if scales:  # of a matrix its codes: places of its scales past the last row are not written
        n = 256 * (900 if "gather" in name else 250)
        want, got = want[:n], got[:n]
    assert torch.equal(got, want)


def test_captured_on_a_given_stream(cuda_ok):
    """The stream of a capture given to the calls, inputs from outside the capture among what they read."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, z = torch.randn((200, 512), generator=g, device="cuda"), torch.randn((200, 16), generator=g, device="cuda")
    w = sharq.quantize_fp4(torch.randn((16, 256, 512), generator=g, device="cuda"), "nvfp4")

    def layer(s=None):
        ids, v = sharq.route(z, 4, stream=s)
        r = sharq.route_rows(ids, 16, stream=s)
        a = sharq.quantize_fp4(x, "nvfp4", rows=r.rows, count=r.offsets[-1:], stream=s)
        return sharq.combine(sharq.linear_fp4_grouped(a, w, r.offsets, stream=s), r.slots, v, stream=s)

    layer()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer(side)
    for seed in (5, 6):
        x.copy_(torch.randn((200, 512), generator=g, device="cuda"))
        z.copy_(torch.randn((200, 16), generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer())
    del graph
