"""The norm and rotation of query and key heads on the GPU against the formulas in 64 bits.

Tolerances (U = 2^-24, a rounding in 32 bits; UT, one rounding to the result's type). A
sum over a head of D elements is added in at most D / 32 + 24 levels (a lane's own
elements, at most 16 where a lane holds two packs, else D / 32; five shuffles), each
rounding once, its products twice more. The reciprocal root is within 2 of the last
place, 4 U, and takes half of its argument's error. A column's sum over N heads has at
most N + 64 levels, whatever the split."""
import pytest
import torch

from ring_allreduce_virtual_gb300 import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
EPS = 1e-6
TYPES = [(torch.float32, torch.float32), (torch.float16, torch.float16), (torch.float16, torch.float32),
         (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]
# batch, tokens, query heads, key heads, dim, rotary
SIZES = [(1, 1, 1, 1, 8, 8), (2, 3, 4, 2, 64, 64), (3, 17, 5, 1, 80, 32), (1, 33, 8, 8, 96, 96), (2, 9, 7, 3, 128, 128),
         (1, 5, 3, 2, 256, 128), (1, 4, 2, 1, 512, 512), (1, 3, 2, 2, 1024, 64), (2, 5, 3, 1, 130, 66),
         (1, 6, 2, 2, 7, 6), (1, 3, 2, 1, 1, 0), (2, 4, 3, 3, 48, 0), (1, 700, 12, 4, 128, 128), (5, 1, 32, 8, 128, 64),
         (1, 3000, 3, 1, 40, 16), (1, 2, 200, 100, 16, 16), (2, 3, 2, 2, 33, 32), (1, 4, 2, 2, 192, 192)]
LAYOUTS = ["dense", "packed", "heads", "shifted"]


def make(g, b, t, h, d, dtype, layout, std=1.0):
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    if layout == "packed":  # between other heads
        return r(b, t, h + 3, d)[:, :, 1: 1 + h]
    if layout == "heads":
        return r(b, h, t, d).transpose(1, 2)
    if layout == "shifted":  # heads that start anywhere
        return r(b, t, h, d + 3)[..., 2: 2 + d]
    return r(b, t, h, d)


def inputs(seed, b, t, hq, hk, d, rot, dtype, wtype, layout):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k = make(g, b, t, hq, d, dtype, layout), make(g, b, t, hk, d, dtype, layout, 3.0)
    dq, dk = make(g, b, t, hq, d, dtype, layout, 0.1), make(g, b, t, hk, d, dtype, layout, 0.1)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(wtype) for _ in range(2)]
    angle = torch.randn(50, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 9
    tables = (angle.cos().float(), angle.sin().float()) if rot else (None, None)
    pos = torch.randint(50, (b, t), generator=g, device="cuda")
    return q, k, dq, dk, w, tables, pos


def rotation(x, tables, pos, inter, back=False, magnitude=False):
    """R x (R^T x); magnitude: the sums of the terms' magnitudes."""
    if tables[0] is None:
        return x.abs() if magnitude else x
    c, s = (t.double()[pos][:, :, None] for t in tables)
    s = -s if back else s
    n = 2 * c.shape[-1]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if inter else (x[..., : n // 2], x[..., n // 2: n])
    if magnitude:
        a, b, c, s = a.abs(), b.abs(), c.abs(), -s.abs()
        y = a * c - b * s, b * c - a * s
    else:
        y = a * c - b * s, b * c + a * s
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    rest = x[..., n:]
    return torch.cat((y, rest.abs() if magnitude else rest), -1)


def check(got, want, far, what):
    far = far + UT[got.dtype] * (want.abs() + far) + TINY[got.dtype]
    bad = ~((got.double() - want).abs() <= far)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def check_forward(y, x, w, tables, pos, inter, eps=EPS):
    x, d = x.double(), x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    u = x * r * (w.double() if w is not None else 1)
    er = (d / 32 + 24 + 2) * U / 2 + 4 * U + U
    # u's error er and two products; the turn's two products and a sum
    check(y, rotation(u, tables, pos, inter), rotation(u, tables, pos, inter, magnitude=True) * (er + 6 * U) * 1.01, "y")


def check_backward(dx, dw, dy, x, w, tables, pos, inter, eps=EPS):
    x, dy, d = x.double(), dy.double(), x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    ww = w.double() if w is not None else torch.ones(d, dtype=torch.float64, device="cuda")
    u, g = x * r, rotation(dy, tables, pos, inter, back=True)
    G = rotation(dy, tables, pos, inter, back=True, magnitude=True)
    k, er = d / 32 + 24, (d / 32 + 26) * U / 2 + 5 * U
    mean, most = (g * ww * u).mean(-1, keepdim=True), (G * ww * u).abs().mean(-1, keepdim=True)
    if dx is not None:
        want = r * (g * ww - u * mean)
        # g is off by 3 U of G; the sum by its levels, three products and g; r comes in
        # three times in its term
        far = r * ((G * ww).abs() * (er + 7 * U) + u.abs() * most * ((k + 12) * U + 3 * er)) * 1.01
        check(dx, want, far, "dx")
    if dw is not None:
        n = dy.shape[0] * dy.shape[1] * dy.shape[2]
        check(dw, (g * u).sum((0, 1, 2)), ((n + 64 + 8) * U + er) * (G * u).abs().sum((0, 1, 2)), "dw")


def same(a, b):
    return a.shape == b.shape and torch.equal(*(t.contiguous().view(-1).view(torch.uint8) for t in (a, b)))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,wtype", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_and_backward(size, dtype, wtype, layout):
    q, k, dq, dk, w, tables, pos = inputs(sum(size), *size, dtype, wtype, layout)
    for inter in (False, True):
        args = (*w, *tables, pos, EPS, inter)
        yq, yk = training.qk_norm_rope_forward(q, k, *args)
        check_forward(yq, q, w[0], tables, pos, inter)
        check_forward(yk, k, w[1], tables, pos, inter)
        got = training.qk_norm_rope_backward(dq, dk, q, k, *args)
        assert got[2].dtype == wtype and got[3].dtype == wtype
        check_backward(got[0], got[2], dq, q, w[0], tables, pos, inter)
        check_backward(got[1], got[3], dk, k, w[1], tables, pos, inter)
        again = training.qk_norm_rope_backward(dq, dk, q, k, *args)
        assert all(same(a, b) for a, b in zip(got, again))
        only = training.qk_norm_rope_backward(dq, dk, q, k, *args, dq_weight=False, dk_weight=False)
        assert only[2] is None and only[3] is None and same(only[0], got[0]) and same(only[1], got[1])
        # in place, each for itself
        z = [t.clone() for t in (q, k, dq, dk)]
        yq, yk = training.qk_norm_rope_forward(z[0], z[1], *args)
        got = training.qk_norm_rope_backward(z[2], z[3], q, k, *args)
        training.qk_norm_rope_forward(z[0], z[1], *args, q_out=z[0], k_out=z[1])
        assert same(z[0], yq) and same(z[1], yk)
        training.qk_norm_rope_backward(z[2], z[3], q, k, *args, dq_in=z[2], dk_in=z[3])
        assert same(z[2], got[0]) and same(z[3], got[1])


def test_in_place_in_one_projection():
    # q, k and v of one buffer, of which v and what lies behind are not touched
    b, t, hq, hk, d = 2, 5, 6, 2, 64
    g = torch.Generator("cuda").manual_seed(3)
    buf = torch.randn(b, t, hq + 2 * hk, d, generator=g, device="cuda").bfloat16()
    was, tables = buf.clone(), (torch.randn(9, 32, device="cuda"), torch.randn(9, 32, device="cuda"))
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    q, k = buf[:, :, :hq], buf[:, :, hq: hq + hk]
    yq, yk = training.qk_norm_rope_forward(q, k, None, None, *tables, pos)
    training.qk_norm_rope_forward(q, k, None, None, *tables, pos, q_out=q, k_out=k)
    assert same(q, yq) and same(k, yk) and same(buf[:, :, hq + hk:], was[:, :, hq + hk:])
    # and gradients written into views of one projection's gradient
    grad = torch.full_like(buf, 7.0)
    q, k = was[:, :, :hq], was[:, :, hq: hq + hk]
    a = training.qk_norm_rope_backward(yq, yk, q, k, None, None, *tables, pos)
    training.qk_norm_rope_backward(yq, yk, q, k, None, None, *tables, pos, dq_in=grad[:, :, :hq],
                                   dk_in=grad[:, :, hq: hq + hk])
    assert same(grad[:, :, :hq], a[0]) and same(grad[:, :, hq: hq + hk], a[1])
    assert bool((grad[:, :, hq + hk:] == 7.0).all())


def test_in_place_in_one_projection_without_some_tokens():
    # q, k and v of one buffer of which the first token of each batch, or the last, is left out; of halves of heads;
    # of heads before tokens
    b, t, hq, hk, d = 3, 5, 6, 2, 64
    g = torch.Generator("cuda").manual_seed(4)
    tables, pos = (torch.randn(9, 16, device="cuda"), torch.randn(9, 16, device="cuda")), torch.arange(t - 1, device="cuda")

    def views(buf, layout):
        if layout == "first":
            return buf[:, 1:, :hq], buf[:, 1:, hq: hq + hk]
        if layout == "last":
            return buf[:, :-1, :hq], buf[:, :-1, hq: hq + hk]
        if layout == "halves":
            return buf[:, 1:, :, :32], buf[:, 1:, :, 32:]
        x = buf.view(b, hq + 2 * hk, t, d)[:, :, 1:].transpose(1, 2)
        return x[:, :, :hq], x[:, :, hq: hq + hk]
    for layout in ("first", "last", "halves", "heads"):
        was = torch.randn(b, t, hq + 2 * hk, d, generator=g, device="cuda").bfloat16()
        q, k = (v.contiguous() for v in views(was, layout))
        args = (None, None, *(c[:, :8] if layout == "halves" else c for c in tables))
        args = tuple(a.contiguous() if a is not None else None for a in args) + (pos,)
        yq, yk = training.qk_norm_rope_forward(q, k, *args)
        grads = training.qk_norm_rope_backward(yq, yk, q, k, *args)
        buf, grad = was.clone(), torch.full_like(was, 7.0)
        vq, vk = views(buf, layout)
        training.qk_norm_rope_forward(vq, vk, *args, q_out=vq, k_out=vk)
        gq, gk = views(grad, layout)
        training.qk_norm_rope_backward(vq, vk, *views(was, layout), *args, dq_in=gq, dk_in=gk)
        assert same(vq, yq) and same(vk, yk) and same(gq, grads[0]) and same(gk, grads[1]), layout
        for x, y in ((vq, vk), (gq, gk)):  # and nothing else
            x.fill_(0), y.fill_(0)
        for x in views(was, layout):
            x.fill_(0)
        assert same(buf, was) and int((grad != 0).sum()) == int((grad == 7.0).sum()) == grad.numel() - q.numel() - k.numel()


def test_positions():
    size = (3, 7, 4, 2, 32, 16)
    q, k, dq, dk, w, tables, _ = inputs(5, *size, torch.float32, torch.float32, "dense")
    pos = torch.arange(7, device="cuda")
    each = training.qk_norm_rope_forward(q, k, *w, *tables, pos.expand(3, 7).contiguous())
    for p in (pos, pos.int(), pos.expand(3, 7), pos.int().expand(3, 7)):
        assert all(same(a, b) for a, b in zip(each, training.qk_norm_rope_forward(q, k, *w, *tables, p)))
    flat = training.qk_norm_rope_forward(q[1], k[1], *w, *tables, pos)  # tokens without a batch
    assert same(flat[0], each[0][1]) and same(flat[1], each[1][1])
    with pytest.raises(ValueError):
        training.qk_norm_rope_forward(q, k, *w, *tables, pos[:6])
    with pytest.raises(ValueError):
        training.qk_norm_rope_forward(q, k, *w, *tables, pos.float())
    with pytest.raises(ValueError):
        training.qk_norm_rope_forward(q, k, *w, *tables)


@pytest.mark.parametrize("dim", [32, 33])
def test_positions_outside_the_tables_give_nan(dim):
    q, k, dq, dk, w, tables, pos = inputs(6, 2, 4, 3, 1, dim, 16, torch.bfloat16, torch.float32, "dense")
    good = training.qk_norm_rope_forward(q, k, *w, *tables, pos)
    for bad in (50, -1, 1 << 40, -(1 << 63)):
        p = pos.clone()
        p[1, 2] = bad
        for y, z in zip(training.qk_norm_rope_forward(q, k, *w, *tables, p), good):
            assert torch.isnan(y[1, 2, :, :16]).all() and same(y[1, 2, :, 16:], z[1, 2, :, 16:])
            y[1, 2] = z[1, 2]
            assert same(y, z)
        dx = training.qk_norm_rope_backward(dq, dk, q, k, *w, *tables, p)
        assert torch.isnan(dx[0][1, 2]).all() and torch.isfinite(dx[0][0]).all()


def test_rows_of_zeros_infinities_and_nan():
    q = torch.zeros(1, 4, 2, 64, device="cuda")
    q[0, 1, 0, 3], q[0, 2, 1, 5] = float("nan"), float("inf")
    y, none = training.qk_norm_rope_forward(q, None)
    assert none is None and not torch.isfinite(y[0, 1, 0]).any()
    assert torch.isnan(y[0, 2, 1, 5]) and bool((y[0, 3] == 0).all()) and bool((y[0, 1, 1] == 0).all())
    dq, dk, dw, dkw = training.qk_norm_rope_backward(torch.ones_like(q), None, torch.zeros_like(q), None)
    assert dk is None and dkw is None and bool((dw == 0).all())
    check_backward(dq, None, torch.ones_like(q), torch.zeros_like(q), None, (None, None), None, False)


def test_no_tokens():
    for shape in ((0, 5, 3, 16), (2, 0, 3, 16), (0, 3, 16)):
        q = torch.empty(shape, device="cuda")
        assert training.qk_norm_rope_forward(q, q.clone())[0].shape == shape
        got = training.qk_norm_rope_backward(q, q, q.clone(), q.clone())
        assert bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_no_keys():
    q = torch.randn(3, 4, 16, device="cuda")
    k = q[:, :0]
    yq, yk = training.qk_norm_rope_forward(q, k)
    assert yk.shape == (3, 0, 16) and same(yq, training.qk_norm_rope_forward(q, None)[0])
    got = training.qk_norm_rope_backward(yq, yk, q, k)
    assert got[1].shape == (3, 0, 16) and bool((got[3] == 0).all())
    assert same(got[0], training.qk_norm_rope_backward(yq, None, q, None)[0])


def test_no_keys_with_tensors_given():
    # the gradient of a weight of no keys is zeros in the tensor that is given for it
    q, dq = torch.randn(3, 4, 16, device="cuda"), torch.randn(3, 4, 16, device="cuda")
    want = training.qk_norm_rope_backward(dq, None, q, None)
    for t in (torch.float32, torch.bfloat16):
        x, d = q.to(t), dq.to(t)
        bucket = torch.full((48,), 7.0, device="cuda", dtype=t)
        got = training.qk_norm_rope_backward(d, None, x, None, dq_weight=bucket[:16], dk_weight=bucket[16:32])
        assert got[3].data_ptr() == bucket[16:].data_ptr() and got[1] is None
        assert bool((bucket[16:32] == 0).all()) and bool((bucket[32:] == 7.0).all())
        assert t is not torch.float32 or (same(got[0], want[0]) and same(bucket[:16], want[2]))
        bucket[16:32] = 7.0
        got = training.qk_norm_rope_backward(d, None, x, None, dq_weight=False, dk_weight=bucket[16:32])
        assert got[2] is None and bool((bucket[16:32] == 0).all())
    bucket.fill_(7.0)
    none = torch.empty(0, 4, 16, device="cuda", dtype=t)  # no tokens either
    training.qk_norm_rope_backward(none, None, none, None, dk_weight=bucket[16:32])
    assert bool((bucket[16:32] == 0).all()) and bool((bucket[:16] == 7.0).all())
    # a tensor for the keys that there are none of is not written, and not said to be
    other = torch.full_like(q, 7.0)
    v = other._version
    assert training.qk_norm_rope_forward(q, None, k_out=other)[1] is None
    assert training.qk_norm_rope_backward(dq, None, q, None, dk_in=other)[1] is None
    assert other._version == v and bool((other == 7.0).all())


def test_strides_of_axes_of_one_element_do_not_matter():
    q = torch.randn(2, 1, 3, 64, device="cuda").bfloat16()
    t = q.as_strided(q.shape, (192, 7, 64, 1))
    assert all(same(a, b) for a, b in zip(training.qk_norm_rope_forward(q, q.clone())[:2], training.qk_norm_rope_forward(t, t.clone())))
    one = torch.randn(1, 1, 1, 64, device="cuda").as_strided((1, 1, 1, 64), (3, 5, 7, 1))
    check_forward(training.qk_norm_rope_forward(one, None)[0], one, None, (None, None), None, False)


def test_gradients_against_differences():
    # the outputs' sum against dy along random directions, in steps of 2^-7: the third derivative of a head's
    # norm is below 16 / |x|^2 of its first, rounding is 2^-24 / 2^-7 of the outputs
    q, k, dq, dk, w, tables, pos = inputs(8, 1, 3, 2, 1, 16, 8, torch.float32, torch.float32, "dense")
    got = training.qk_norm_rope_backward(dq, dk, q, k, *w, *tables, pos)
    leaves, h = [q, k, *w], 2.0 ** -7
    for i, grad in enumerate(got):
        v = torch.randn(leaves[i].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i))

        def value(step):
            t = list(leaves)
            t[i] = t[i] + step * v
            yq, yk = training.qk_norm_rope_forward(t[0], t[1], t[2], t[3], *tables, pos)
            return (yq.double() * dq).sum() + (yk.double() * dk).sum()

        want = (value(h) - value(-h)) / (2 * h)
        size = float(dq.norm() + dk.norm()) * float(v.norm())
        assert abs(float(want - (grad.double() * v).sum())) <= 2e-3 * size


def test_differentiable_call():
    q, k, dq, dk, w, tables, pos = inputs(9, 2, 6, 4, 2, 64, 32, torch.float32, torch.float32, "packed")
    leaves = [t.clone().requires_grad_() for t in (q, k, *w)]
    yq, yk = training.qk_norm_rope(*leaves, *tables, pos, EPS)
    ((yq * dq).sum() + (yk * dk).sum()).backward()
    want = training.qk_norm_rope_backward(dq, dk, q, k, *w, *tables, pos, EPS)
    assert all(same(a.grad, b) for a, b in zip(leaves, want))
    # one result alone, keys shared by expansion, weights that want no gradient, a last axis that is not dense
    one = q[:, :, :1].clone().requires_grad_()
    yq, yk = training.qk_norm_rope(one.expand(-1, -1, 4, -1), k, w[0], None, *tables, pos, EPS)
    yq.sum().backward()
    full = training.qk_norm_rope_backward(torch.ones_like(q), torch.zeros_like(k), q[:, :, :1].expand(-1, -1, 4, -1),
                                          k, w[0], None, *tables, pos, EPS)[0]
    assert (one.grad - full.sum(2, keepdim=True)).abs().max() <= 1e-5 * full.abs().max()
    t = torch.randn(3, 64, 5, device="cuda").requires_grad_()
    y, none = training.qk_norm_rope(t.transpose(1, 2), None)
    y.backward(torch.ones_like(y))
    d = training.qk_norm_rope_backward(torch.ones_like(y), None, t.detach().transpose(1, 2).contiguous(), None)[0]
    assert none is None and same(t.grad, d.transpose(1, 2))


def test_graphs_and_streams():
    q, k, dq, dk, w, tables, pos = inputs(10, 1, 64, 8, 2, 128, 128, torch.bfloat16, torch.float32, "packed")
    args = (*w, *tables, pos)
    eager = training.qk_norm_rope_forward(q, k, *args) + training.qk_norm_rope_backward(dq, dk, q, k, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = training.qk_norm_rope_forward(q, k, *args, stream=s) + \
        training.qk_norm_rope_backward(dq, dk, q, k, *args, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = training.qk_norm_rope_forward(q, k, *args) + training.qk_norm_rope_backward(dq, dk, q, k, *args)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(eager, other, kept):
        assert same(a, b) and same(a, c)
    out = torch.empty_like(eager[0])
    v = out._version
    training.qk_norm_rope_forward(q, k, *args, q_out=out)
    assert out._version > v and same(out, eager[0])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 16), (torch.float16, 16), (torch.float32, 8), (torch.bfloat16, 8),
                                       (torch.float32, 4)], ids=str)
@pytest.mark.parametrize("heads", [1, 30, 64])
def test_heads_of_one_lane_without_keys(heads, dtype, dim, inter):
    # tokens of one step each, of which a warp takes many one after the other with angles of their own
    q, _, dq, _, w, tables, pos = inputs(dim + heads, 2, 20000, heads, 1, dim, dim, dtype, torch.float32, "dense")
    args = (w[0], None, *tables, pos, EPS, inter)
    y, none = training.qk_norm_rope_forward(q, None, *args)
    assert none is None
    check_forward(y, q, w[0], tables, pos, inter)
    got = training.qk_norm_rope_backward(dq, None, q, None, *args)
    check_backward(got[0], got[2], dq, q, w[0], tables, pos, inter)


def test_far_elements():
    # a token more than 2^32 elements behind the first
    n = (1 << 32) // 128 + 3
    q = torch.empty(n, 1, 128, device="cuda", dtype=torch.bfloat16)
    q[-4:] = torch.randn(4, 1, 128, device="cuda").bfloat16()
    pos = torch.zeros(n, device="cuda", dtype=torch.int32)
    tables = torch.full((1, 64), 0.6, device="cuda"), torch.full((1, 64), 0.8, device="cuda")
    y, _ = training.qk_norm_rope_forward(q, None, None, None, *tables, pos)
    z, _ = training.qk_norm_rope_forward(q[-4:].clone(), None, None, None, *tables, pos[-4:].clone())
    assert same(y[-4:], z)
    check_forward(z[None], q[-4:][None], None, tables, pos[-4:][None].long(), False)
