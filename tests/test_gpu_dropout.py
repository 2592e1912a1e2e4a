"""Dropout on the GPU against the generator written out in whole numbers. Results
are compared bit for bit: an element that stays is x / (1 - p), or with an addition the
sum of that product and the other, in one rounding of 32 bits (here of 64 bits and then of 32: the
same but where the first lands on the middle between two numbers of the second, once in 2^28),
and is rounded once to its type."""
import pytest
import torch

from ring_allreduce_virtual_gb300 import training

LOW = 0xFFFFFFFF
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def philox(counter, key):
    """Philox4x32-10 of four words and two, by the paper's rule (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & LOW, a >> 32 ^ c[3] ^ k[1], a & LOW]
        k = [k[0] + 0x9E3779B9 & LOW, k[1] + 0xBB67AE85 & LOW]
    return c


def test_generator_gives_the_known_answers():
    # the vectors published with the generator
    assert philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert philox([LOW] * 4, [LOW] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def blocks(m, stream, seed):
    """The words of the blocks of an int64 tensor m of numbers below 2^61."""
    c = [m & LOW, m >> 32, torch.full_like(m, stream), torch.zeros_like(m)]
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64
        c = [b >> 32 & LOW ^ c[1] ^ k0, b & LOW, a >> 32 & LOW ^ c[3] ^ k1, a & LOW]
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return torch.stack(c, 1)


def numbers(count, seed, offset, device):
    """u(n) of n = offset, ..., modulo 2^64."""
    first = offset // 8
    m = (first + torch.arange((offset + count + 7) // 8 - first, device=device)) % (1 << 61) \
        if offset < 1 << 63 else \
        (torch.arange((offset + count + 7) // 8 - first, device=device) - ((1 << 61) - first)) & (1 << 61) - 1
    upper, lower = (torch.stack((w & 0xFFFF, w >> 16), 2).flatten() for w in (blocks(m, s, seed) for s in (0, 1)))
    return (upper << 16 | lower)[offset - 8 * first:][:count]


def test_numbers_are_the_blocks_halfwords():
    seed, offset = 0x123456789ABCDEF0, (1 << 35) + 5
    got = numbers(40, seed, offset, "cpu")
    for i in range(40):
        m, h = divmod(offset + i, 8)
        halves = [philox([m & LOW, m >> 32, s, 0], [seed & LOW, seed >> 32])[h // 2] >> 16 * (h & 1) & 0xFFFF
                  for s in (0, 1)]
        assert got[i] == halves[0] << 16 | halves[1]


def want(x, p, seed, offset=0, residual=None):
    keep = numbers(x.numel(), seed, offset, x.device).view(x.shape) >= round(p * 2.0 ** 32)
    scale = torch.tensor(1 / (1 - p) if p < 1 else 0.0, dtype=torch.float32, device=x.device)
    r = torch.zeros_like(x) if residual is None else residual
    return torch.where(keep, (x.double() * scale.double() + r.double()).float(), r.float()).to(x.dtype)


def same(a, b):
    return a.shape == b.shape and torch.equal(*(t.contiguous().view(-1).view(torch.uint8) for t in (a, b)))


def rand(shape, dtype, seed=0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


SIZES = [(1, 1), (1, 2), (3, 5), (2, 7), (9, 8), (1, 13), (33, 31), (64, 512), (7, 1001), (5, 4096), (1217, 136),
         (300, 2051), (2500, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_and_backward(rows, cols, dtype):
    x, r = rand((rows, cols), dtype, rows), rand((rows, cols), dtype, cols)
    seed = 0x9E3779B97F4A7C15 ^ rows * cols
    for p, offset in ((0.1, 0), (0.25, 3), (0.5, 8 * rows + 4), (1 / 3, (1 << 45) + 1), (0.9, 6)):
        y = training.dropout_forward(x, p, seed, offset, r)
        assert same(y, want(x, p, seed, offset, r)), (p, offset)
        d = training.dropout_backward(x, p, seed, offset)
        assert same(d, want(x, p, seed, offset)), (p, offset)
        z = x.clone()
        assert training.dropout_forward(z, p, seed, offset, r, out=z) is z and same(z, y)
        z = r.clone()
        assert same(training.dropout_forward(x, p, seed, offset, z, out=z), y)


@pytest.mark.gpu
def test_probabilities_at_their_ends():
    x = rand((100, 257), torch.bfloat16)
    assert same(training.dropout_forward(x, 0.0, 5), x)
    assert same(training.dropout_forward(x, 1.0, 5), torch.zeros_like(x))
    assert same(training.dropout_forward(x, 1.0, 5, 0, x), x)
    # thresholds of one random number, and one below all of them
    n = 1 << 20
    x = torch.ones(n, device="cuda")
    u = numbers(n, 77, 0, "cuda")
    for t in (int(u[12345]), int(u[12345]) + 1, int(u.max()), int(u.min()) + 1, 1, (1 << 32) - 1):
        p = t / 2.0 ** 32
        y = training.dropout_forward(x, p, 77)
        assert torch.equal(y != 0, u >= t)


@pytest.mark.gpu
def test_upper_halves_that_tie():
    # 4 Mi elements: the upper half equals the threshold's 64 times on the average
    x = torch.ones(2, 1 << 21, device="cuda", dtype=torch.float16)
    p, seed = 0.3000001, 31
    u = numbers(x.numel(), seed, 5, "cuda")
    assert int((u >> 16 == round(p * 2 ** 32) >> 16).sum()) > 16
    assert same(training.dropout_forward(x, p, seed, 5), want(x, p, seed, 5))


@pytest.mark.gpu
def test_share_that_stays():
    n = 1 << 22
    x = torch.ones(n, device="cuda")
    for p in (0.05, 0.1, 0.5):
        share = (training.dropout_forward(x, p, 12345) != 0).double().mean().item()
        assert abs(share - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5  # six standard deviations


@pytest.mark.gpu
def test_ranks_draw_what_one_would():
    x, r = rand((40, 333), torch.bfloat16, 1), rand((40, 333), torch.bfloat16, 2)
    whole = training.dropout_forward(x, 0.2, 99, 1000, r)
    parts = [training.dropout_forward(x[i: i + 8], 0.2, 99, 1000 + i * 333, r[i: i + 8]) for i in range(0, 40, 8)]
    assert same(torch.cat(parts), whole)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 8), (1, 0), (3, 5), (0, 1)])
def test_strides_and_addresses(dtype, shift, pad):
    rows, cols = 37, 203
    def matrix(seed, shift, pad):  # noqa: E306
        base = torch.full((96 + shift + rows * (cols + pad) + 96,), 7.0, device="cuda", dtype=dtype)
        v = base[96 + shift:].as_strided((rows, cols), (cols + pad, 1))
        v.copy_(rand((rows, cols), dtype, seed))
        return base, v
    _, x = matrix(1, shift, pad)
    for rs, rp, ys, yp in ((shift, pad, shift, pad), (2, 3, shift, pad), (shift, pad, 1, 7)):
        _, r = matrix(2, rs, rp)
        base, y = matrix(3, ys, yp)
        assert training.dropout_forward(x, 0.4, 3, 11, r, out=y) is y
        assert same(y, want(x, 0.4, 3, 11, r))
        y.fill_(7.0)
        assert bool((base == 7.0).all())  # nothing around it was written


@pytest.mark.gpu
def test_numbers_wrap():
    x = torch.ones(100, device="cuda")
    y = training.dropout_forward(x, 0.5, 7, (1 << 64) - 21)
    a = training.dropout_forward(x[:21], 0.5, 7, (1 << 64) - 21)
    b = training.dropout_forward(x[21:], 0.5, 7, 0)
    assert same(y, torch.cat((a, b)))
    assert same(a, want(x[:21], 0.5, 7, (1 << 64) - 21)) and same(b, want(x[21:], 0.5, 7, 0))


@pytest.mark.gpu
def test_dropped_elements_count_for_nothing():
    x = torch.full((64, 65), float("nan"), device="cuda")
    r = rand((64, 65), torch.float32)
    keep = want(torch.ones_like(x), 0.5, 9) != 0
    for bad in (float("nan"), float("inf")):
        y = training.dropout_forward(x.fill_(bad), 0.5, 9, 0, r)
        assert same(y[~keep], r[~keep]) and not torch.isfinite(y[keep]).any()


@pytest.mark.gpu
def test_more_than_two_to_the_32_elements():
    n = (1 << 32) + 4099
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    y = training.dropout_forward(x, 0.5, 1, 3)
    for at in (0, (1 << 32) - 1000, n - 2000):
        assert same(y[at: at + 2000], want(x[at: at + 2000], 0.5, 1, 3 + at))


@pytest.mark.gpu
def test_no_elements():
    for shape in ((0, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        assert training.dropout_forward(x, 0.5, 1).shape == shape


@pytest.mark.gpu
def test_differentiable_call():
    x = rand((6, 10, 33), torch.float32, 1).requires_grad_()
    r = rand((6, 10, 33), torch.float32, 2).requires_grad_()
    y = training.dropout(x, 0.3, 17, 5, r)
    y.backward(dy := rand((6, 10, 33), torch.float32, 3))
    assert same(x.grad, want(dy, 0.3, 17, 5)) and same(r.grad, dy)
    # layouts that are copied, gradients that are expanded
    t = rand((33, 60), torch.float32, 4).requires_grad_()
    y = training.dropout(t.t(), 0.3, 17)
    y.sum().backward()
    assert same(t.grad, want(torch.ones(60, 33, device="cuda"), 0.3, 17).t().contiguous())


@pytest.mark.gpu
def test_seed_on_the_device_and_in_a_graph():
    x = rand((50, 77), torch.float16)
    seed = torch.tensor([41], device="cuda")
    assert same(training.dropout_forward(x, 0.3, seed, 2), want(x, 0.3, 41, 2))
    w = x.float().requires_grad_()
    y = training.dropout(w, 0.3, seed)
    seed += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        training.dropout_forward(x, 0.3, seed, 2, out=out)
        seed += 1
    seed.fill_(100)
    for i in range(3):
        g.replay()
        assert same(out, want(x, 0.3, 100 + i, 2))


@pytest.mark.gpu
def test_other_streams():
    x = rand((500, 1000), torch.bfloat16)
    expect = want(x, 0.3, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = training.dropout_forward(x, 0.3, 1, stream=s)
    with torch.cuda.stream(s):
        z = training.dropout_forward(x, 0.3, 1)
    s.synchronize()
    assert same(y, expect) and same(z, expect)
    v = y._version
    training.dropout_forward(x, 0.3, 1, out=y)
    assert y._version > v
