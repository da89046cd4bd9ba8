"""CPU checks of the plain FP4 layers' and the routing calls' boundary: sizes, and every
refusal before anything is launched."""
import pytest
import torch

from activation_sparsity_fp4_b200 import build_ext, sharq

BF, F32 = sharq.BF16, sharq.F32


@pytest.fixture(scope="module", autouse=True)
def L():
    build_ext.build()
    return sharq.lib()


@pytest.fixture(autouse=True)
def nothing_launched():
    before = sharq.sharq_launch_count()
    yield
    assert sharq.sharq_launch_count() == before


def refused(status, fn, *args):
    with pytest.raises(sharq.SharqError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)


def mat(rows=128, k=256, experts=1, fmt=1, ptr=16):
    return sharq.sharq_fp4(ptr, ptr, ptr, rows, k, experts, fmt)


def test_sizes():
    assert sharq.sharq_fp4_sizes(4096, 4096, 1, "nvfp4") == (4096 * 2048, 4096 * 256, 4096 * 4)
    # 3 experts of 200 rows (two blocks of 128) and 96 elements: 6 scales in two groups of four; 3 scales in one
    assert sharq.sharq_fp4_sizes(200, 96, 3, "nvfp4") == (3 * 200 * 48, 3 * 2 * 2 * 512, 3 * 200 * 4)
    assert sharq.sharq_fp4_sizes(200, 96, 3, "mxfp4") == (3 * 200 * 48, 3 * 2 * 1 * 512, 3 * 200 * 4)


@pytest.mark.parametrize("rows,k,experts,fmt,status", [(0, 64, 1, 0, 1), (-1, 64, 1, 0, 1), (1, 0, 1, 0, 1),
                                                       (1, 48, 1, 0, 1), (1, 64, 0, 0, 1), (1, 64, 1, 7, 1),
                                                       (2**31, 64, 1, 0, 2), (2**20, 64, 2**12, 0, 2),
                                                       (1, 2**31, 1, 0, 2)])
def test_sizes_refuse(rows, k, experts, fmt, status):
    refused(status, sharq.sharq_fp4_sizes, rows, k, experts, fmt)


def test_quantize_refuses():
    q = sharq.sharq_quantize_fp4
    ok = [16, BF, 128, 256, None, None, None, 1e-6, 0.0, mat(), 0]
    for at, bad, status in [(0, 0, 1), (0, 24, 1), (1, 5, 1), (2, 0, 1), (2, 127, 1), (3, 255, 1), (3, 260, 1),
                            (4, 18, 1), (5, 18, 1), (6, 20, 1), (7, -1.0, 1), (7, float("nan"), 1),
                            (9, mat(ptr=None), 1), (9, mat(ptr=8), 1), (9, mat(k=40), 1), (9, mat(rows=0), 1),
                            (9, mat(fmt=3), 1)]:
        refused(status, q, *ok[:at], bad, *ok[at + 1 :])
    # a gather or a row count is for one matrix
    refused(1, q, 16, BF, 256, 256, 16, None, None, 1e-6, 0.0, mat(experts=2), 0)
    refused(1, q, 16, BF, 256, 256, None, 16, None, 1e-6, 0.0, mat(experts=2), 0)


def test_quantize_swiglu_refuses():
    q = sharq.sharq_quantize_fp4_swiglu
    ok = [16, 16, BF, 512, None, 0.0, mat(), 0]
    for at, bad in [(0, 0), (1, 0), (1, 18), (2, 9), (3, 128), (3, 257), (4, 2), (6, mat(experts=2)), (6, mat(k=33))]:
        refused(1, q, *ok[:at], bad, *ok[at + 1 :])


def test_amax_must_be_finite():
    for v in (float("inf"), -float("inf")):
        refused(1, sharq.sharq_quantize_fp4, 16, BF, 128, 256, None, None, None, 1e-6, v, mat(), 0)
        refused(1, sharq.sharq_quantize_fp4_swiglu, 16, 16, BF, 512, None, v, mat(), 0)


def test_amax_and_eps_that_are_no_numbers():
    nan, inf = float("nan"), float("inf")
    refused(1, sharq.sharq_quantize_fp4, 16, BF, 128, 256, None, None, None, 1e-6, nan, mat(), 0)
    refused(1, sharq.sharq_quantize_fp4_swiglu, 16, 16, BF, 512, None, nan, mat(), 0)
    refused(1, sharq.sharq_quantize_fp4, 16, BF, 128, 256, None, None, 16, inf, 0.0, mat(), 0)


def test_gather_in_place_refuses():
    refused(1, sharq.sharq_gather_fp4, mat(), 16, None, mat(), 0)
    a, b = mat(), mat(ptr=32)
    b.scales = 16
    refused(1, sharq.sharq_gather_fp4, a, 16, None, b, 0)


def test_combine_onto_another_dtype_refuses():
    refused(1, sharq.sharq_combine, 16, BF, 4, 64, 16, 16, 4, 2, 32, 32, F32, 0)
    refused(1, sharq.sharq_combine, 16, F32, 4, 64, 16, 16, 4, 2, 32, 32, BF, 0)


def test_combine_onto_its_inputs_refuses():
    """out may be add and nothing else of what is read: y is 256 x 64 bf16 (32768 bytes), add and out 4 x 64 (512)."""
    y, add, out = 1 << 20, 1 << 21, 1 << 22
    args = lambda o, a=None, dt=BF: (y, BF, 256, 64, 16, 16, 4, 8, a, o, dt, 0)
    for o, dt in ((y, BF), (y + 32768 - 16, BF), (y - 512 + 16, BF), (y - 1024 + 16, F32)):
        refused(1, sharq.sharq_combine, *args(o, None, dt))
    for o in (add + 16, add - 16, add + 512 - 16):
        refused(1, sharq.sharq_combine, *args(o, add))
    refused(1, sharq.sharq_combine, *args(y, y))


def test_stream_of_another_device_refuses():
    class On:  # stands in for a tensor, and for a stream
        is_cuda = True

        def __init__(self, i):
            self.device = torch.device("cuda", i)

    with pytest.raises(ValueError, match="stream of cuda:1"):
        with sharq._place(On(0), On(1)):
            pass


def test_gather_refuses():
    f = sharq.sharq_gather_fp4
    refused(1, f, mat(), 0, None, mat(rows=300), 0)
    refused(1, f, mat(), 18, None, mat(rows=300), 0)
    refused(1, f, mat(), 16, 18, mat(rows=300), 0)
    refused(1, f, mat(), 16, None, mat(k=512), 0)
    refused(1, f, mat(), 16, None, mat(fmt=0), 0)
    refused(1, f, mat(experts=2), 16, None, mat(), 0)
    refused(1, f, mat(), 16, None, mat(experts=2), 0)
    refused(1, f, mat(), 16, None, mat(rows=0), 0)


def test_linear_refuses():
    f = sharq.sharq_linear_fp4
    refused(1, f, mat(), mat(k=512), 16, BF, 0)
    refused(1, f, mat(), mat(fmt=0), 16, BF, 0)
    refused(1, f, mat(), mat(rows=100), 16, BF, 0)      # n not a multiple of 8
    refused(1, f, mat(), mat(experts=2), 16, BF, 0)     # a stack without offsets
    refused(1, f, mat(experts=2), mat(), 16, BF, 0)
    refused(1, f, mat(), mat(), 0, BF, 0)
    refused(1, f, mat(), mat(), 24, BF, 0)
    refused(1, f, mat(), mat(), 16, 4, 0)
    refused(1, f, mat(rows=0), mat(), 16, BF, 0)
    g = sharq.sharq_linear_fp4_grouped
    refused(1, g, mat(), mat(experts=2), 0, 16, BF, 0)
    refused(1, g, mat(), mat(experts=2), 18, 16, BF, 0)
    refused(1, g, mat(), mat(experts=2, k=512), 16, 16, BF, 0)


def test_route_refuses():
    # logits, dtype, t, experts, stride, bias, score, groups, top_groups, group_top, top_k, renormalize, scale, ids, weights
    ok = [16, BF, 4, 64, 64, None, 0, 1, 1, 1, 8, True, 1.0, 16, 16, 0]
    for at, bad, status in [(0, 0, 1), (0, 17, 1), (1, 2, 1), (2, 0, 1), (3, 0, 1), (3, 513, 2), (4, 63, 1), (5, 18, 1),
                            (6, 2, 1), (7, 0, 1), (7, 3, 1), (8, 0, 1), (8, 2, 1), (9, 0, 1), (9, 3, 1), (10, 0, 1),
                            (10, 33, 2), (13, 0, 1), (13, 18, 1), (14, 0, 1)]:
        refused(status, sharq.sharq_route, *ok[:at], bad, *ok[at + 1 :])
    refused(2, sharq.sharq_route, 16, BF, 4, 64, 64, None, 0, 64, 1, 1, 1, True, 1.0, 16, 16, 0)  # 64 groups
    refused(1, sharq.sharq_route, 16, BF, 4, 64, 64, None, 0, 8, 1, 1, 9, True, 1.0, 16, 16, 0)   # 9 of 8 experts


def test_route_rows_capacity():
    cap = sharq.sharq_route_rows_capacity
    assert cap(1, 8, 128) == 8 * 128            # eight experts with a row each
    assert cap(16, 8, 128) == 128 * 128         # every expert with a row
    assert cap(17, 8, 128) == 128 * 128         # ... and 8 more rows, which fill up
    assert cap(32, 8, 128) == 129 * 128         # ... and 128 more, which may need a tile
    assert cap(1000, 1, 1) == 1024
    for t, k, e, status in [(0, 1, 4, 1), (1, 0, 4, 1), (1, 33, 64, 2), (1, 1, 0, 1), (1, 1, 513, 2), (2**31, 1, 4, 2)]:
        refused(status, cap, t, k, e)


def test_route_rows_refuses():
    f = sharq.sharq_route_rows
    ok = [16, 16, 8, 128, 16, 128 * 128, 16, 16, 0]
    for at, bad, status in [(0, 0, 1), (0, 18, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1), (4, 0, 1), (5, 128 * 127, 5),
                            (6, 0, 1), (7, 0, 1)]:
        refused(status, f, *ok[:at], bad, *ok[at + 1 :])


def test_combine_refuses():
    ok = [16, BF, 256, 64, 16, 16, 4, 8, None, 16, BF, 0]
    for at, bad, status in [(0, 0, 1), (0, 24, 1), (1, 3, 1), (2, 0, 1), (3, 0, 1), (3, 12, 1), (4, 0, 1), (4, 18, 1),
                            (5, 0, 1), (6, 0, 1), (7, 0, 1), (7, 33, 2), (8, 24, 1), (9, 0, 1), (9, 8, 1), (10, 7, 1)]:
        refused(status, sharq.sharq_combine, *ok[:at], bad, *ok[at + 1 :])


def test_python_forms_refuse_host_tensors():
    x = torch.zeros(4, 64)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: sharq.quantize_fp4(x, "nvfp4"), lambda: sharq.quantize_fp4_swiglu(x, x, "nvfp4"),
                 lambda: sharq.route(x, 2), lambda: sharq.route_rows(ids, 8),
                 lambda: sharq.combine(x, ids, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="one shape"):
        sharq.quantize_fp4_swiglu(x, x[:, :32], "nvfp4")
    with pytest.raises(ValueError, match="dimensions"):
        sharq.route(x[0], 2)
