"""Layer norm on the GPU against the formulas in 64 bits.

Tolerances (U = 2^-24, a rounding in 32 bits; uT, one rounding to the result's
type). A 32-bit sum of n terms added in at most k levels is off by at most
k U times the sum of their magnitudes. A row of n elements is spread over at
least 32 lanes, so k <= n / 32 + 48 (the lanes' own run, five shuffles, at most
32 warps, and the products' own roundings). A column's sum over R rows has at
most R + 64 levels, whatever the split."""
import pytest
import torch

from ring_allreduce_virtual_gb300 import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
EPS = 1e-5
TYPES = [(torch.float32, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32)]
SIZES = [(1, 1), (3, 1), (5, 2), (2, 7), (9, 8), (33, 31), (17, 32), (4, 33), (1, 64), (300, 127),
         (1217, 136), (64, 256), (31, 1000), (61, 1001), (7, 1024), (311, 2048), (157, 2051),
         (5, 4096), (160, 4097), (19, 5000), (40, 8192), (6, 8200), (3, 16384), (2, 16385),
         (9, 20480), (2, 40001), (1, 70000)]
GUARD = 96


def levels(n):
    return n / 32 + 48


def matrix(g, rows, cols, dtype, pad=0, shift=0, fill=None):
    """A rows x cols view with `pad` elements between rows, `shift` elements off
    an aligned base and guard elements around; returns (base, view)."""
    stride = cols + pad
    base = torch.full((GUARD + shift + max(rows, 1) * stride + GUARD,), 7.0, dtype=dtype, device="cuda")
    view = base[GUARD + shift:].as_strided((rows, cols), (stride, 1))
    if fill is not None:
        view.copy_(fill)
    return base, view


def untouched(base, view):
    """All of base outside view still holds the guard value."""
    b = base.clone()
    b.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(7.0)
    return bool((b == 7.0).all())


def inputs(seed, rows, cols, dtype, wtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, cols) * (1 + 0.2 * r(cols)) + 0.5 * r(cols)).to(dtype)
    return x, (1 + 0.1 * r(cols)).to(wtype), (0.1 * r(cols)).to(wtype), (0.1 * r(rows, cols)).to(dtype)


def stats64(x, eps=EPS):
    x = x.double()
    m = x.mean(1)
    v = (x - m[:, None]).square().mean(1)
    return m, v, (v + eps).rsqrt()


def check_forward(x, w, b, y, mean, rstd, eps=EPS):
    k = levels(x.shape[1])
    m, v, r = stats64(x, eps)
    dm = k * U * x.double().abs().mean(1)
    # v is off by the mean's error squared, by k U of itself, and each squared
    # distance by twice the rounding of the distance
    dr = r * ((k + 6) * U + dm ** 2 * r ** 2)
    if mean is not None:
        assert ((mean.double() - m).abs() <= dm + U * m.abs()).all()
        assert ((rstd.double() - r).abs() <= dr + 2 * U * r).all()
    d = x.double() - m[:, None]
    ww = w.double() if w is not None else torch.ones_like(d[0])
    bb = b.double() if b is not None else torch.zeros_like(d[0])
    want = d * r[:, None] * ww + bb
    far = ww.abs() * ((dm[:, None] + 2 * U * d.abs()) * r[:, None] + d.abs() * dr[:, None])
    far = far * 1.01 + 4 * U * (want.abs() + bb.abs())
    far = far + UT[y.dtype] * (want.abs() + far) + TINY[y.dtype]
    bad = (y.double() - want).abs() > far
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def check_backward(dy, x, mean, rstd, w, dx, dw, db):
    rows, n = x.shape
    k = levels(n)
    r = rstd.double()[:, None]
    u = (x.double() - mean.double()[:, None]) * r
    g0 = dy.double()
    g = g0 * w.double() if w is not None else g0
    if dx is not None:
        s, p = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
        want = r * (g - s - u * p)
        ds = (k + 4) * U * g.abs().mean(1, keepdim=True)
        dp = (k + 8) * U * (g * u).abs().mean(1, keepdim=True)
        far = r * (4 * U * (g.abs() + s.abs() + 2 * (u * p).abs()) + ds + u.abs() * dp) * 1.01
        far = far + UT[dx.dtype] * (want.abs() + far) + TINY[dx.dtype]
        bad = (dx.double() - want).abs() > far
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    for got, terms in ((dw, g0 * u), (db, g0)):
        if got is None:
            continue
        want = terms.sum(0)
        far = (rows + 64 + 8) * U * terms.abs().sum(0)
        far = far + UT[got.dtype] * (want.abs() + far) + TINY[got.dtype]
        bad = (got.double() - want).abs() > far
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("dtype,wtype", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype, wtype):
    x, w, b, _ = inputs(rows * 7 + cols, rows, cols, dtype, wtype)
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    # without statistics, and in place, the same bits
    z = x.clone()
    y2, m2, r2 = training.layer_norm_forward(z, w, b, EPS, stats=False, out=z)
    assert m2 is None and r2 is None and y2 is z and torch.equal(z, y)


@pytest.mark.parametrize("dtype,wtype", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, dtype, wtype):
    x, w, b, dy = inputs(rows * 5 + cols, rows, cols, dtype, wtype)
    _, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.dtype == dtype and dw.dtype == wtype and db.dtype == wtype
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    again = training.layer_norm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    # each output alone: the same bits
    for i, only in enumerate(((True, False, False), (False, True, False), (False, False, True))):
        got = training.layer_norm_backward(dy, x, mean, rstd, w, *only)
        assert torch.equal(got[i], again[i])
        assert all(got[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows,cols", [(3, 8), (37, 264), (33, 1001), (9, 4096), (5, 9000), (2, 40001)])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3), (0, 4)])
def test_strides_alignments_and_guards(rows, cols, dtype, pad, shift):
    x, w, b, dy = inputs(cols, rows, cols, dtype, dtype)
    _, xv = matrix(0, rows, cols, dtype, pad, shift, x)
    ybase, yv = matrix(0, rows, cols, dtype, pad + 8, shift)
    wbase, wv = matrix(0, 1, cols, dtype, 0, shift, w[None])
    bbase, bv = matrix(0, 1, cols, dtype, 0, 0, b[None])
    y, mean, rstd = training.layer_norm_forward(xv, wv[0], bv[0], EPS, out=yv)
    check_forward(x, w, b, y, mean, rstd)
    assert untouched(ybase, yv)
    _, dyv = matrix(0, rows, cols, dtype, pad, 8 - shift if shift else 0, dy)
    dbase, dxv = matrix(0, rows, cols, dtype, pad + 1, shift)
    dwbase, dwv = matrix(0, 1, cols, dtype, 0, shift)
    dbbase, dbv = matrix(0, 1, cols, dtype, 0, 0)
    dx, dw, db = training.layer_norm_backward(dyv, xv, mean, rstd, wv[0], dxv, dwv[0], dbv[0])
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    assert untouched(dbase, dxv) and untouched(dwbase, dwv) and untouched(dbbase, dbv)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows,cols", [(3, 8), (37, 264), (33, 1001), (700, 1001), (130, 2051), (9, 4096),
                                       (150, 9000), (75, 20001)])
@pytest.mark.parametrize("pad,shift", [(8, 0), (16, 8), (3, 0), (0, 1), (5, 3), (1, 7)])
def test_padded_and_shifted_rows_that_lie_alike(rows, cols, dtype, pad, shift):
    # dy, x and dx start alike and their strides differ by whole packs: the rows
    # stay on chip, with ends before and after the packs
    x, w, _, dy = inputs(cols + pad, rows, cols, dtype, dtype)
    _, mean, rstd = training.layer_norm_forward(x, w, None, EPS)
    ybase, yv = matrix(0, rows, cols, dtype, pad + 8, shift)
    _, xv = matrix(0, rows, cols, dtype, pad, shift, x)
    y, mean, rstd = training.layer_norm_forward(xv, w, None, EPS, out=yv)
    check_forward(x, w, None, y, mean, rstd)
    assert untouched(ybase, yv)
    _, dyv = matrix(0, rows, cols, dtype, pad + 16, shift, dy)
    dbase, dxv = matrix(0, rows, cols, dtype, pad + 8, shift)
    dwbase, dwv = matrix(0, 1, cols, dtype, 0, shift)
    dbbase, dbv = matrix(0, 1, cols, dtype, 0, 3)
    dx, dw, db = training.layer_norm_backward(dyv, xv, mean, rstd, w, dxv, dwv[0], dbv[0])
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    assert untouched(dbase, dxv) and untouched(dwbase, dwv) and untouched(dbbase, dbv)


@pytest.mark.parametrize("cols", [8, 333, 1024])
def test_matrices_side_by_side_in_one_buffer(cols):
    x, w, b, dy = inputs(cols, 31, cols, torch.float32, torch.float32)
    buf = torch.full((31, 4 * cols + 9), 7.0, device="cuda")
    xv, yv, dyv, dxv = (buf[:, i * cols:(i + 1) * cols] for i in range(4))
    xv.copy_(x)
    dyv.copy_(dy)
    _, mean, rstd = training.layer_norm_forward(xv, w, b, EPS, out=yv)
    check_forward(x, w, b, yv, mean, rstd)
    _, dw, db = training.layer_norm_backward(dyv, xv, mean, rstd, w, dxv)
    check_backward(dy, x, mean, rstd, w, dxv, dw, db)
    assert torch.equal(xv, x) and torch.equal(dyv, dy) and (buf[:, 4 * cols:] == 7.0).all()


@pytest.mark.parametrize("cols", [5, 512, 1001, 4096, 20000])
@pytest.mark.parametrize("has_w,has_b", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(cols, has_w, has_b):
    x, w, b, dy = inputs(cols, 23, cols, torch.bfloat16, torch.float32)
    w, b = w if has_w else None, b if has_b else None
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    assert dw.dtype == (torch.float32 if has_w else torch.bfloat16)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)


def test_no_rows():
    x = torch.empty(0, 40, device="cuda")
    y, mean, rstd = training.layer_norm_forward(x, torch.ones(40, device="cuda"))
    assert y.shape == (0, 40) and mean.shape == (0,)
    dw, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    training.layer_norm_backward(x, x, mean, rstd, None, True, dw, db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("cols", [64, 1001, 4096, 12288, 30000])
def test_constant_rows_and_large_offsets(cols):
    # a constant row has no variance: y is the bias where the mean is exact
    w, b = torch.full((cols,), 2.0, device="cuda"), torch.linspace(-1, 1, cols, device="cuda")
    x = torch.full((3, cols), 0.5, device="cuda")
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    assert torch.isfinite(y).all()
    x = torch.randn(5, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) + 1000.0
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)


@pytest.mark.parametrize("cols", [96, 1001, 2048, 20000])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_values_stay_in_their_row(cols, what):
    x, w, b, dy = inputs(cols, 12, cols, torch.float32, torch.float32)
    good = training.layer_norm_forward(x, w, b, EPS)
    gdx = training.layer_norm_backward(dy, x, good[1], good[2], w)[0]
    x[5, cols // 2] = what
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    assert torch.isnan(y[5]).all()
    keep = [i for i in range(12) if i != 5]
    assert torch.equal(y[keep], good[0][keep])
    dx = training.layer_norm_backward(dy, x, mean, rstd, w)[0]
    assert torch.equal(dx[keep], gdx[keep]) and torch.isnan(dx[5]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("cols", [96, 600, 1001, 4096, 10240, 20000])
@pytest.mark.parametrize("power", [-80, 60])
@pytest.mark.parametrize("pad", [0, 1])
def test_gradients_of_scaled_rows_scale(cols, power, dtype, pad):
    # x, mean and 1 / rstd times a power of two: u, dw and db are the same bits,
    # dx the same over it (without eps the formula has no scale of its own)
    x, w, _, dy = inputs(cols, 40, cols, dtype, torch.float32)
    _, mean, rstd = training.layer_norm_forward(x, w, None, EPS)

    def gradients(c):
        out = matrix(0, 40, cols, dtype, pad)[1]
        return training.layer_norm_backward(dy, x * c, mean * c, rstd / c, w, out)

    dx, dw, db = gradients(1.0)
    sx, sw, sb = gradients(2.0 ** power)
    assert torch.equal(sx * 2.0 ** power, dx) and torch.equal(sw, dw) and torch.equal(sb, db)


@pytest.mark.parametrize("cols", [24, 333, 4096])
def test_gradients_against_differences(cols):
    # d/dt of sum(dy * LN(x + t a, w + t c, b + t e)) by central differences of
    # the formula in 64 bits (error t^2 times a third derivative of order one,
    # far below the 32-bit gradients' own error)
    x, w, b, dy = inputs(cols, 6, cols, torch.float32, torch.float32)
    x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    training.layer_norm(x, w, b, EPS).backward(dy)
    g = torch.Generator("cuda").manual_seed(9)
    a, c, e = (torch.randn(t.shape, device="cuda", dtype=torch.float64, generator=g) for t in (x, w, b))

    def loss(t):
        x2, w2, b2 = (p.detach().double() + t * q for p, q in ((x, a), (w, c), (b, e)))
        m, v, r = stats64(x2)
        return (dy.double() * ((x2 - m[:, None]) * r[:, None] * w2 + b2)).sum()

    t = 1e-5
    want = (loss(t) - loss(-t)) / (2 * t)
    parts = [(p.grad.double() * q) for p, q in ((x, a), (w, c), (b, e))]
    got = sum(p.sum() for p in parts)
    scale = sum(p.abs().sum() for p in parts)
    assert (got - want).abs() <= (levels(cols) + 72) * U * scale + 1e-7 * scale


def test_autograd_takes_only_what_is_needed_and_expanded_gradients():
    x = torch.randn(2, 5, 48, device="cuda", requires_grad=True)
    b = torch.zeros(48, device="cuda", requires_grad=True)
    training.layer_norm(x, None, b).sum().backward()  # dy is an expanded scalar
    assert torch.equal(b.grad, torch.full((48,), 10.0, device="cuda"))
    assert x.grad.shape == x.shape and x.grad.abs().max() < 1e-5
    w = torch.ones(48, device="cuda", requires_grad=True)
    training.layer_norm(x.detach(), w).square().sum().backward()
    assert w.grad is not None
    with torch.no_grad():
        assert not training.layer_norm(x, w).requires_grad


def test_differentiable_call_takes_any_layout():
    x = torch.randn(3, 5, 48, device="cuda", requires_grad=True)
    for view in (x[:, 1:], x.transpose(1, 2), x[:, :, ::2], x[:1].expand(4, 5, 48), x[:, 0]):
        w = torch.rand(view.shape[-1], device="cuda", requires_grad=True)
        dy = torch.randn(view.shape, device="cuda")
        for got, want in zip(*(torch.autograd.grad(training.layer_norm(v, w), (x, w), dy)
                               for v in (view, view.contiguous()))):
            assert torch.equal(got, want)
    with pytest.raises(ValueError):
        training.layer_norm_forward(x[:, 1:])


def test_other_stream_and_graph():
    x, w, b, dy = inputs(1, 700, 4096, torch.bfloat16, torch.float32)
    want = training.layer_norm_forward(x, w, b, EPS)
    back = training.layer_norm_backward(dy, x, want[1], want[2], w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    z = torch.zeros_like(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        z.copy_(x)  # late: a kernel on another stream would see zeros
        got = training.layer_norm_forward(z, w, b, EPS)
        got2 = training.layer_norm_backward(dy, z, got[1], got[2], w)
    also = training.layer_norm_forward(z, w, b, EPS, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got + also, want + want))
    assert all(torch.equal(p, q) for p, q in zip(got2, back))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m, r = training.layer_norm_forward(z, w, b, EPS)
        dx, dw, db = training.layer_norm_backward(dy, z, m, r, w)
    z.zero_()
    graph.replay()
    z.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((y, m, r, dx, dw, db), want + back))


def test_offsets_past_32_bits():
    # three rows 2^31 + 16 elements apart
    cols, stride = 4096, 2 ** 31 + 16
    x, w, b, dy = inputs(4, 3, cols, torch.bfloat16, torch.float32)
    store = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    far = store.as_strided((3, cols), (stride, 1))
    far.copy_(x)
    want = training.layer_norm_forward(x, w, b, EPS)
    got = training.layer_norm_forward(far, w, b, EPS)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    back = training.layer_norm_backward(dy, x, want[1], want[2], w)
    for p, q in zip(training.layer_norm_backward(dy, far, want[1], want[2], w), back):
        assert torch.equal(p, q)
    training.layer_norm_forward(far, w, b, EPS, out=far)
    assert torch.equal(far, want[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("rows", [1, 130, 3001, 70001])
@pytest.mark.parametrize("cols", [3, 64, 72, 264, 640, 1001, 1024, 2051])
@pytest.mark.parametrize("dx", [False, True])
def test_column_sums_of_whole_numbers_are_exact(rows, cols, dtype, dx):
    # |dy u| <= 36 and 70001 rows: every partial sum is a whole number below 2^24, so
    # a row left out or taken twice shows
    g = torch.Generator("cuda").manual_seed(rows + cols)
    x, dy = (torch.randint(-6, 7, (rows, cols), generator=g, device="cuda").to(dtype) for _ in range(2))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.empty(2, cols, device="cuda").unbind()
    training.layer_norm_backward(dy, x, mean, rstd, None, dx, dw, db)
    assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0))
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("cols", [4096, 8192, 9000, 20000, 20001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=lambda t: str(t)[6:])
def test_column_sums_of_wide_rows_are_exact(cols, dtype):
    test_column_sums_of_whole_numbers_are_exact(3001, cols, dtype, True)


def test_many_rows():
    # more rows than any grid: every block walks over several
    x, w, b, dy = inputs(8, 70001, 72, torch.float16, torch.float16)
    y, mean, rstd = training.layer_norm_forward(x, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = training.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
