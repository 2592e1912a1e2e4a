"""The gradient norm and clipping on the GPU against the formulas in 64 bits.

Tolerances (U = 2^-24): a thread adds at most 64 squares in 32 bits before a
sum that keeps its rounding errors, all above that is in 64 bits; with the
squares' own roundings the sum of squares is within 70 U of itself, the norm
within 35 U, and U more for its rounding to 32 bits: 40 U. A clipped element is
off by the norm's 40 U, two roundings of the factor and one rounding to its
type."""
import math

import pytest
import torch

from ring_allreduce_virtual_gb300 import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UT = {torch.float64: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11,
      torch.bfloat16: 2.0 ** -8}
TINY = {torch.float64: 0.0, torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24,
        torch.bfloat16: 2.0 ** -133}
TYPES = list(UT)
RAGGED = [1, 2, 3, 7, 8, 9, 0, 31, 33, 255, 257, 1000, 4095, 4096, 4097, 8191, 8192, 8193, 0,
          16385, 50000, 100003, 262144, 1]


def tensors(seed, counts, types, std=0.01, shift=0):
    """One tensor for each count, cut out of a buffer for each type with guard
    elements between; types cycle."""
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(counts):
        t = types[i % len(types)]
        base = torch.randn(n + shift + 16, generator=g, device="cuda").mul_(std).to(t)
        out.append(base[shift + i % 3: shift + i % 3 + n] if shift else base[:n])
    return out


def norms64(ts):
    s = [t.double().square().sum().item() for t in ts]
    return math.sqrt(math.fsum(s)), [math.sqrt(v) for v in s]


def check_norm(ts, scale=1.0):
    want, each = norms64(ts)
    norm, norms = training.grad_norm(ts, scale=scale, per_tensor=True)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(norm.item() - abs(scale) * want) <= 40 * U * abs(scale) * want
    for got, w in zip(norms.tolist(), each):
        assert abs(got - abs(scale) * w) <= 40 * U * abs(scale) * w
    again, only = training.grad_norm(ts, scale=scale, per_tensor=True), training.grad_norm(ts, scale=scale)
    assert torch.equal(again[0], norm) and torch.equal(again[1], norms) and torch.equal(only, norm)
    return want


def check_clip(ts, most, scale=1.0):
    want = norms64(ts)[0] * abs(scale)
    c = most / want if want > most else 1.0
    if abs(want - most) < 80 * U * want:
        c = 1.0
    bases = [torch.full((t.numel() + 64,), 5.0, dtype=t.dtype, device="cuda") for t in ts]
    offs = [(t.data_ptr() % 16) // t.element_size() + 16 for t in ts]
    outs = [b[o:o + t.numel()] for b, o, t in zip(bases, offs, ts)]
    norm = training.clip_grad_norm(ts, most, scale=scale, outs=outs)
    assert abs(norm.item() - want) <= 40 * U * want
    for t, o, b, at in zip(ts, outs, bases, offs):
        w = t.double() * (scale * c)
        far = 44 * U * w.abs()
        far = far + UT[t.dtype] * (w.abs() + far) + TINY[t.dtype]
        assert ((o.double() - w).abs() <= far).all()
        assert (b[:at] == 5.0).all() and (b[at + t.numel():] == 5.0).all()
    # other alignments of the outputs, and in place: the same bits. (The order
    # of a sum follows the gradients' alignment: copies keep it.)
    other = [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:] for t in ts]
    assert torch.equal(training.clip_grad_norm(ts, most, scale=scale, outs=other), norm)
    copies = [torch.empty(t.numel() + 32, dtype=t.dtype, device="cuda")[o:o + t.numel()].copy_(t)
              for o, t in zip(offs, ts)]
    assert torch.equal(training.clip_grad_norm(copies, most, scale=scale), norm)
    for o, p, q in zip(outs, other, copies):
        assert torch.equal(o, p) and torch.equal(o, q)


@pytest.mark.parametrize("dtype", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("n", [1, 5, 8, 100, 4096, 8191, 20001, 1 << 20, (1 << 23) + 3])
def test_one_tensor(n, dtype):
    ts = tensors(n, [n], [dtype])
    want = check_norm(ts)
    check_clip(ts, want / 3)
    check_clip(ts, want * 3)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES], ids=lambda t: str(len(t)) + str(t[0])[6:])
def test_ragged_lists(types, shift):
    ts = tensors(3, RAGGED, types, shift=shift)
    want = check_norm(ts, 0.125)
    check_clip(ts, want / 10, 0.125)
    check_clip(ts, 1e6, -2.0)


@pytest.mark.parametrize("count", [63, 64, 65, 300, 959, 960, 961, 2500])
def test_long_lists(count):
    counts = [(i * 37) % 1009 for i in range(count)]
    counts[count // 2] = 3_000_000
    ts = tensors(count, counts, [torch.bfloat16, torch.float32])
    want = check_norm(ts)
    check_clip(ts, want / 2)


def test_nothing_but_empty_tensors():
    ts = [torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.float16, device="cuda")]
    norm, norms = training.grad_norm(ts, per_tensor=True)
    assert norm.item() == 0.0 and norms.tolist() == [0.0, 0.0]
    assert training.clip_grad_norm(ts, 1.0).item() == 0.0


@pytest.mark.parametrize("n", [40, 300])
def test_lists_in_any_order_in_one_buffer(n):
    # gradients and outputs in turn in one bucket; upwards, downwards, shuffled; some in place
    bucket = torch.empty(2 * n * 1001, device="cuda")
    parts = torch.split(bucket, 1001)
    for seed, order in enumerate((list(range(2 * n)), list(range(2 * n))[::-1], None)):
        g = torch.Generator("cuda").manual_seed(seed)
        bucket.copy_(torch.randn(bucket.shape, generator=g, device="cuda"))
        order = order or torch.randperm(2 * n, generator=torch.Generator().manual_seed(n)).tolist()
        ins, outs = ([parts[i] for i in order[k::2]] for k in (0, 1))
        outs = [i if k % 7 == 3 else o for k, (i, o) in enumerate(zip(ins, outs))]
        start = [t.clone() for t in ins]
        others = bucket.clone()
        norm = training.clip_grad_norm(ins, 1.0, outs=outs)
        assert abs(norm.item() - norms64(start)[0]) <= 40 * U * norm.item()
        for k, (i, o, s) in enumerate(zip(ins, outs, start)):
            w = s.double() / norm.item()
            assert ((o.double() - w).abs() <= 48 * U * w.abs()).all()
            assert o is i or torch.equal(i, s)
        for k in range(3, n, 7):  # outputs that were not asked for
            at = order[2 * k + 1] * 1001
            assert torch.equal(bucket[at: at + 1001], others[at: at + 1001])


def test_zero_gradients_and_zero_bound():
    ts = [torch.zeros(70000, device="cuda"), torch.zeros(33, dtype=torch.bfloat16, device="cuda")]
    check_norm(ts)
    check_clip(ts, 1.0)
    check_clip(ts, 0.0)
    check_clip(tensors(2, [5000, 3], [torch.float32]), 0.0)


@pytest.mark.parametrize("dtype,size", [(torch.float32, 1e30), (torch.float32, 1e-30),
                                        (torch.float32, 1e-42), (torch.bfloat16, 1e30),
                                        (torch.bfloat16, 1e-38), (torch.float64, 1e100),
                                        (torch.float16, 6e4), (torch.float16, 6e-8)])
def test_sizes_whose_squares_leave_32_bits(dtype, size):
    g = torch.Generator("cuda").manual_seed(1)
    ts = [((torch.rand(n, generator=g, device="cuda", dtype=torch.float64) + 0.5) * size).to(dtype)
          for n in (30000, 17, 1)]
    ts = [torch.where(torch.isfinite(t), t, torch.full_like(t, 1.0)) for t in ts]
    want, each = norms64(ts)
    if want < 3e38:  # the norm itself fits 32 bits
        low = 2.0 ** -149  # and may lie below the normal ones
        norm, norms = training.grad_norm(ts, per_tensor=True)
        assert abs(norm.item() - want) <= 40 * U * want + low
        assert all(abs(a - b) <= 40 * U * b + low for a, b in zip(norms.tolist(), each))
    outs = [torch.empty_like(t) for t in ts]
    training.clip_grad_norm(ts, want / 4 if want < 3e38 else 1.0, outs=outs)
    c = 0.25 if want < 3e38 else 1.0 / want
    for t, o in zip(ts, outs):
        w = t.double() * c
        # a bound below 2^-126 is held in 32 bits with less than 24 bits
        far = (44 * U + UT[dtype] + 2.0 ** -149 / max(want / 4, 2.0 ** -149)) * w.abs() + TINY[dtype]
        assert ((o.double() - w).abs() <= far * 1.01).all()


@pytest.mark.parametrize("dtype,size,most,scale", [
    (torch.float32, 1e30, 1e-9, 1.0),    # maxNorm / norm is below the normal floats
    (torch.float32, 3e38, 1e-3, 1.0),    # and the norm above all floats
    (torch.bfloat16, 1e38, 1e-5, 0.125),
    (torch.float32, 1.0, 1e-12, 1e30),   # the ratio alone is
    (torch.float32, 1e38, 1e-2, 1e-30),  # the factor alone is
])
@pytest.mark.parametrize("n", [100, 3_000_000])
def test_factors_below_the_normal_floats_keep_their_bits(dtype, size, most, scale, n):
    ts = [t * size for t in tensors(n, [n, 7], [dtype], std=1.0)]
    ts = [t.clamp(-3e38, 3e38) for t in ts]
    want = norms64(ts)[0] * scale
    outs = [torch.empty_like(t) for t in ts]
    training.clip_grad_norm(ts, most, scale=scale, outs=outs)
    # the factor as in check_clip; the bound itself may be rounded
    for t, o in zip(ts, outs):
        w = t.double() * (scale * (most / want))
        far = 46 * U * w.abs()
        far = far + UT[dtype] * (w.abs() + far) + TINY[dtype]
        assert ((o.double() - w).abs() <= far).all()


@pytest.mark.parametrize("dtype,size", [(torch.float32, 1e38), (torch.bfloat16, 1e38), (torch.float64, 1e150)])
@pytest.mark.parametrize("n", [100, 3_000_000])
def test_norms_past_the_largest_float_clip_and_infinities_do_not(dtype, size, n):
    # short and long lists; a scale that brings the norm back makes it finite
    ts = [torch.full((n,), size, dtype=dtype, device="cuda"), torch.full((7,), -size, dtype=dtype, device="cuda")]
    want = norms64(ts)[0]
    outs = [torch.empty_like(t) for t in ts]
    assert training.clip_grad_norm(ts, 2.0, outs=outs).item() == math.inf
    for t, o in zip(ts, outs):
        w = t.double() * (2.0 / want)
        assert ((o.double() - w).abs() <= (44 * U + UT[dtype]) * w.abs() * 1.01).all()
    if dtype != torch.float64:
        norm = training.clip_grad_norm(ts, 2.0, scale=2.0 ** -20, outs=outs).item()
        assert abs(norm - want * 2.0 ** -20) <= 40 * U * norm
    ts[1][3] = math.inf
    assert training.clip_grad_norm(ts, 2.0, scale=0.5, outs=outs).item() == math.inf
    assert all(torch.equal(o, t * 0.5) for t, o in zip(ts, outs))


def test_mixed_sizes_and_large_values_among_small_ones():
    ts = [torch.full((9000,), 1e-25, device="cuda"), torch.full((100,), 1e25, device="cuda"),
          torch.full((50000,), 1.0, device="cuda", dtype=torch.bfloat16)]
    check_norm(ts)


def test_long_runs_of_equal_values_keep_their_precision():
    # every addition of such a run rounds the same way
    check_norm([torch.full((1 << 25,), 1.0000001, device="cuda")])


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", TYPES, ids=lambda t: str(t)[6:])
def test_not_finite_gradients_are_not_clipped(what, dtype):
    ts = tensors(5, [4000, 9, 20000], [dtype])
    ts[1][4] = what
    norm, norms = training.grad_norm(ts, per_tensor=True)
    assert not math.isfinite(norm.item()) and not math.isfinite(norms[1].item())
    assert math.isfinite(norms[0].item()) and math.isfinite(norms[2].item())
    copies = [t.clone() for t in ts]
    norm = training.clip_grad_norm(copies, 1.0, scale=0.5)
    assert not math.isfinite(norm.item())
    for c, t in zip(copies, ts):
        assert torch.equal(c.nan_to_num(nan=3.0), (t * 0.5).nan_to_num(nan=3.0))


@pytest.mark.parametrize("counts", [[4000, 9, 20000], [4000, 9, 3_000_000], [700] * 70 + [3_000_000]],
                         ids=["short", "long", "many"])
@pytest.mark.parametrize("dtype", TYPES, ids=lambda t: str(t)[6:])
def test_norms_of_infinities_are_infinite_and_of_nans_nan(dtype, counts):
    last = len(counts) - 1
    for t, at in ((0, 0), (1, 4), (last, counts[-1] // 2 + 1), (last, counts[-1] - 1)):
        for what in ([math.inf], [-math.inf], [math.nan], [math.inf, math.nan]):
            ts = tensors(5, counts, [dtype])
            for i, v in enumerate(what):
                ts[t][at - i] = v
            norm, norms = training.grad_norm(ts, per_tensor=True)
            clipped = training.clip_grad_norm([x.clone() for x in ts], 1.0)
            for got in (norm.item(), norms[t].item(), clipped.item()):
                if any(map(math.isnan, what)):
                    assert math.isnan(got)
                else:
                    assert got == math.inf
            assert all(math.isfinite(v) for i, v in enumerate(norms.tolist()) if i != t)


def test_lists_are_checked():
    a, b = torch.zeros(8, device="cuda"), torch.zeros(9, device="cuda")
    for bad in ([a[::2]], [a.int()], [a, torch.zeros(8)], [torch.zeros(4, 4, device="cuda").t()[:, :2]]):
        with pytest.raises(ValueError):
            training.grad_norm(bad)
    for outs in ([b], [a, a], [a.half()], [torch.zeros(8)]):
        with pytest.raises(ValueError):
            training.clip_grad_norm([a], 1.0, outs=outs)


def test_other_stream_and_graph():
    ts = tensors(7, RAGGED, [torch.float32, torch.bfloat16])
    want = training.grad_norm(ts, per_tensor=True)
    clipped = [t.clone() for t in ts]
    training.clip_grad_norm(clipped, 0.01)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = training.TensorList([torch.zeros_like(t) for t in ts])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for z, t in zip(late.tensors, ts):
            z.copy_(t)
        got = training.grad_norm(late, per_tensor=True)
    also = training.clip_grad_norm(late, 0.01, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(also, want[0])
    assert all(torch.equal(p, q) for p, q in zip(late.tensors, clipped))
    outs = training.TensorList([torch.empty_like(t) for t in ts])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = training.clip_grad_norm(late, 0.01, outs=outs)
    for z, t in zip(late.tensors, ts):
        z.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, want[0])
    assert all(torch.equal(p, q) for p, q in zip(outs.tensors, clipped))


def test_elements_past_32_bits():
    n = 2 ** 32 + 77
    t = torch.zeros(n, dtype=torch.float16, device="cuda")
    t[5], t[2 ** 31 + 9], t[n - 1] = 3.0, 4.0, 12.0
    assert training.grad_norm([t]).item() == 13.0
    assert training.clip_grad_norm([t], 6.5).item() == 13.0
    assert [t[i].item() for i in (5, 2 ** 31 + 9, n - 1)] == [1.5, 2.0, 6.0]
    assert torch.count_nonzero(t[: 2 ** 31]).item() == 1
