"""Layer norm at sizes around the borders between its kernels' layouts: rows
of a part of a warp, of a warp, of a block, of a cluster; few rows, whose sums
one cluster joins, and many; whole packs and ragged ones. Checks and tolerances
are those of test_gpu_layernorm."""
import pytest
import torch

from ring_allreduce_virtual_gb300 import training
from test_gpu_layernorm import EPS, check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu

COLS = [4, 9, 63, 64, 65, 128, 255, 257, 511, 512, 513, 1016, 1025, 1032, 2047, 2055, 2056, 2064,
        3000, 4088, 4095, 4103, 4104, 6001, 8184, 8191, 8199, 8208, 12288, 12289, 16376, 16391]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 15, 130, 700])
def test_layout_borders(rows, cols, dtype):
    x, w, b, dy = inputs(rows + cols, rows, cols, dtype, torch.float32)
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("cols", [256, 264, 320, 640, 760, 768, 776, 960, 968, 1024])
@pytest.mark.parametrize("rows", [1, 47, 400, 3000])
def test_rows_of_one_warp(rows, cols, dtype):
    x, w, b, dy = inputs(rows + cols, rows, cols, dtype, dtype)
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows,cols", [(1, 16385), (75, 20000), (90, 20001), (77, 24576), (40, 24584), (3, 32768),
                                       (39, 32769), (100, 49152), (37, 49160), (81, 65536), (20, 65537), (17, 90000),
                                       (40, 98304), (16, 98312), (31, 131072), (9, 131080)])
def test_rows_of_clusters(rows, cols, dtype):
    x, w, b, dy = inputs(rows + cols, rows, cols, dtype, torch.float32)
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)


@pytest.mark.parametrize("rows,cols", [(2, 40), (250, 64), (256, 1024), (257, 1024), (64, 4096), (65, 4096),
                                       (31, 8192), (33, 7000), (200, 1280), (205, 1281), (4096, 64), (4097, 64)])
def test_small_calls_write_nothing_but_their_outputs(rows, cols):
    x, w, b, dy = inputs(rows * cols, rows, cols, torch.bfloat16, torch.bfloat16)
    _, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    base = torch.full((2 * cols + 48,), 7.0, dtype=torch.bfloat16, device="cuda")
    dw, db = base[16:16 + cols], base[32 + cols:32 + 2 * cols]
    got = training.layer_norm_backward(dy, x, mean, rstd, w, True, dw, db)
    check_backward(dy, x, mean, rstd, w, *got)
    assert (base[:16] == 7).all() and (base[16 + cols:32 + cols] == 7).all()
    assert (base[32 + 2 * cols:] == 7).all()
    only = training.layer_norm_backward(dy, x, mean, rstd, w, False, True, False)[1]
    assert torch.equal(only, dw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=lambda t: str(t)[6:])
def test_parameters_that_the_call_before_wrote(dtype):
    # the kernel that reads them starts while the one that writes them runs
    g = torch.Generator("cuda").manual_seed(4)
    x, rows = (torch.randn(n, 4096, device="cuda", generator=g).to(dtype) for n in (300, 40))
    w, b = torch.zeros(4096, device="cuda", dtype=dtype), torch.zeros(4096, device="cuda", dtype=dtype)

    def chain(wait):
        out = []
        for row in torch.split(rows, 1):
            training.layer_norm_forward(row, out=w[None])
            wait()
            training.layer_norm_forward(row * 2, w, out=b[None])
            wait()
            out.append(training.layer_norm_forward(x, w, b)[0])
            wait()
            _, mean, rstd = training.layer_norm_forward(x)
            wait()
            training.layer_norm_backward(x, x, mean, rstd, None, False, w, b)
            wait()
            out.append(training.layer_norm_forward(x, w, b)[0])
            wait()
        return out

    assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), chain(torch.cuda.synchronize)))


def test_chains_of_calls_see_each_other():
    # every call starts while the last one ends; what it reads has to be there
    x = torch.randn(512, 4096, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    a, b = x.clone(), x.clone()
    for _ in range(100):
        a, m, r = training.layer_norm_forward(a)
        a = training.layer_norm_backward(a, a, m, r)[0] + x
        training.clip_grad_norm([a], 50.0)
    for _ in range(100):
        b, m, r = training.layer_norm_forward(b)
        torch.cuda.synchronize()
        b = training.layer_norm_backward(b, b, m, r)[0] + x
        torch.cuda.synchronize()
        training.clip_grad_norm([b], 50.0)
        torch.cuda.synchronize()
    assert torch.equal(a, b)
