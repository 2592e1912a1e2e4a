"""Log probabilities, policy and preference losses on the GPU against the formulas in 64 bits.

Tolerances (U = 2^-24). An exponential of a row is exp2 of a product of two roundings: off by
2^-22 (two of the last place) and 3 U |d| of itself, d its distance from the row's largest
element; as |d| exp(d) <= 1/e, its part of the sum is off by at most 2^-22 + 3 U |d|, averaged over
the row with its own weight. A thread's sum grows by at most 8 roundings a pack, and is scaled
by 2^-22 each time its largest element rises, not more often than it has packs; the joining has 10
steps of both. Logarithm and target add 2^-24 and roundings of what they are."""
import math

import pytest
import torch

from ring_allreduce_virtual_gb300 import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E2 = 2.0 ** -22
UT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
TYPES = [torch.float32, torch.float16, torch.bfloat16]
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 33), (9, 127), (33, 1000), (7, 1001), (300, 264), (3, 4099), (2, 16384),
         (5, 32001), (61, 50001), (3, 131072), (2, 200003), (1, 700001), (2000, 640), (1, 1600002)]


def same(a, b):
    return a.shape == b.shape and torch.equal(*(t.contiguous().view(-1).view(torch.uint8) for t in (a, b)))


def make(seed, rows, cols, dtype, std=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * std).to(dtype)
    t = torch.randint(cols, (rows,), generator=g, device="cuda")
    x[torch.arange(rows, device="cuda"), t] += 4
    return x, t, g


def lse_far(x, lse):
    """How far lse may be off."""
    x = x.double()
    n = x.shape[1]
    m = x.amax(1, keepdim=True)
    p = (x - lse[:, None]).exp()
    away = torch.where(p > 0, p * (m - x), 0.0).sum(1)
    packs = n * (16 if x.dtype == torch.float32 else 8) / 16 / 32 + 1  # of a thread: at least 32 share a row
    steps = min(packs, n / 8 / 512 + 9)  # 8 packs a thread, until a row has 512 threads
    return E2 + 3 * U * away + (8 * steps + 20) * U + (steps + 12) * E2 + 4 * U


def check(got, want, far, what):
    bad = ~((got.double() - want).abs() <= far)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def check_logp(x, t, logp, lse):
    want = torch.logsumexp(x.double(), 1)
    far = lse_far(x, want)
    if lse is not None:
        check(lse, want, far + U * (want.abs() + far), "lse")
    lp = x.double().gather(1, t[:, None])[:, 0] - want
    check(logp, lp, far + U * (lp.abs() + far), "logp")
    return want, lp, far


def check_grad(dx, x, t, c, lse, far, ec=0.0):
    """dx = c ([target] - p), rows of c 0 are 0; c may itself be off by ec of its size (a number for each row)."""
    x = x.double()
    p = (x - lse[:, None]).exp()
    d = torch.where(p > 0, (x - lse[:, None]).abs(), 0.0)
    want = -c[:, None] * p
    want[torch.arange(len(t), device="cuda"), t] += c
    # the exponential, its argument's roundings, lse's error and its rounding; 1 - p at the target
    off = c.abs()[:, None] * p * (E2 + 4 * U * d + (far + ec + U * lse.abs())[:, None] + 4 * U) * 1.01
    # c's error changes c (1 - p) by ec |c| (1 - p) <= ec |c|
    at = off.gather(1, t[:, None]) + (c.abs() * (ec + 4 * U))[:, None]
    off.scatter_(1, t[:, None], at)
    off += UT[dx.dtype] * (want.abs() + off) + TINY[dx.dtype]
    zero = c == 0
    assert bool((dx[zero] == 0).all())
    check(dx, torch.where(zero[:, None], 0.0, want), off, "dlogits")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_logprobs(rows, cols, dtype):
    x, t, g = make(rows + cols, rows, cols, dtype)
    logp, lse = training.token_logprobs_forward(x, t)
    want, _, far = check_logp(x, t, logp, lse)
    c = torch.randn(rows, generator=g, device="cuda")
    dx = training.token_logprobs_backward(c, x, t, lse)
    check_grad(dx, x, t, c.double(), want, far)
    gain = torch.tensor(0.25, device="cuda")  # a power of two: exact
    assert same(training.token_logprobs_backward(c, x, t, lse, None, gain),
                training.token_logprobs_backward(c * 0.25, x, t, lse))
    z = x.clone()
    assert training.token_logprobs_backward(c, z, t, lse, out=z) is z and same(z, dx)
    again = training.token_logprobs_forward(x, t)
    assert same(again[0], logp) and same(again[1], lse)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shift,pad,dshift,dpad", [(0, 8, 0, 8), (1, 0, 1, 0), (3, 5, 3, 5), (0, 3, 0, 0), (2, 1, 5, 2)])
def test_strides_and_addresses(dtype, shift, pad, dshift, dpad):
    rows, cols = 23, 1003

    def matrix(shift, pad, fill=None):
        base = torch.full((96 + shift + rows * (cols + pad) + 96,), 7.0, device="cuda", dtype=dtype)
        v = base[96 + shift:].as_strided((rows, cols), (cols + pad, 1))
        if fill is not None:
            v.copy_(fill)
        return base, v

    x0, t, g = make(3, rows, cols, dtype)
    _, x = matrix(shift, pad, x0)
    logp, lse = training.token_logprobs_forward(x, t)
    want, _, far = check_logp(x0, t, logp, lse)
    c = torch.randn(rows, generator=g, device="cuda")
    base, d = matrix(dshift, dpad)
    assert training.token_logprobs_backward(c, x, t, lse, out=d) is d
    check_grad(d, x0, t, c.double(), want, far)
    loss, lp, again = policy_call(x, t, g, out=d)
    check_policy(x0, t, *policy_inputs(x0, t, g), None, d, loss, lp)
    d.fill_(7.0)
    assert bool((base == 7.0).all())  # nothing around it was written


def policy_inputs(x, t, g):
    """old_logp, advantages, weights and ref_logp: ratios inside, outside and far outside of the borders, none within
    1e-3 of one."""
    rows = len(t)
    lp = torch.log_softmax(x.double(), 1).gather(1, t[:, None])[:, 0]
    e = torch.tensor([-3.0, -0.5, -0.25, -0.2, -0.1, 0.0, 0.1, 0.18, 0.2, 0.3, 0.5, 2.0], device="cuda", dtype=torch.float64)
    i = torch.arange(rows, device="cuda")
    old = (lp - e[i % 12]).float()
    adv = torch.tensor([1.0, -0.7, 2.0, -1.5, 0.0], device="cuda")[i % 5]
    w = torch.tensor([0.25, 1.0, 0.0, 0.5, 2.0, 1.0, 0.125], device="cuda")[i % 7]
    ref = (lp + torch.tensor([0.3, -0.4, 0.0, 1.0], device="cuda")[i % 4].double()).float()
    return old, adv, w, ref


LOW, HIGH, KL, SCALE = 0.2, 0.28, 0.05, 0.75


def policy_call(x, t, g, out=None, f=training.policy_loss_gradient):
    args = policy_inputs(x, t, g)
    kw = {} if out is None else {"out": out}
    return f(x, t, *args, LOW, HIGH, KL, SCALE, **kw)


def check_policy(x, t, old, adv, w, ref, dlogp, dlogits, loss, logp, kl=KL):
    want, lp, far = check_logp(x, t, training.token_logprobs_forward(x, t)[0], None)
    used = (w != 0) & (t >= 0)
    check(logp, torch.where(used, lp, 0.0), far + U * (lp.abs() + far), "logp")
    p = lp.clone().requires_grad_()
    ratio, a = (p - old.double()).exp(), adv.double()
    each = -torch.minimum(ratio * a, ratio.clamp(1 - LOW, 1 + HIGH) * a)
    r = ref.double() - p
    each = each + kl * (r.exp() - r - 1)
    each = torch.where(used, each * w.double() * SCALE, 0.0)
    total = each.sum()
    total.backward()
    c = p.grad * used
    # both exponentials are off by logp's error and their own roundings; kl's is a difference of two
    with torch.no_grad():
        rel = far + E2 + 8 * U
        big = (ratio * a).abs() + kl * (r.exp() + r.abs() + 1)
        off = torch.where(used, w.double() * SCALE * big * rel * 1.01, 0.0)
    check(loss, total.detach(), off.sum() + 4 * U * each.detach().abs().sum() + U * total.detach().abs() + 1e-30, "loss")
    if dlogp is not None:
        check(dlogp, c, off + 4 * U * c.abs(), "dlogp")
    if dlogits is not None:
        lim = torch.where(c != 0, off / c.abs().clamp(min=1e-300), 0.0)
        check_grad(dlogits, x, t, c, want, far, lim + 4 * U)
    return off


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 1), (12, 7), (420, 264), (61, 1001), (84, 32001), (9, 131072), (7, 200003), (5, 700001)])
def test_policy(rows, cols, dtype):
    x, t, g = make(rows * cols, rows, cols, dtype)
    args = policy_inputs(x, t, g)
    loss, logp, dlogits = training.policy_loss_gradient(x, t, *args, LOW, HIGH, KL, SCALE)
    off = check_policy(x, t, *args, None, None, loss, logp)
    l2, lp2, lse, dlogp = training.policy_loss_forward(x, t, *args, LOW, HIGH, KL, SCALE)
    check_policy(x, t, *args, dlogp, None, l2, lp2)
    used = args[2] != 0
    assert bool((lse[~used] == 0).all()) and bool((dlogp[~used] == 0).all())
    # the gradient, from this row's derivative
    want = torch.logsumexp(x.double(), 1)
    far = lse_far(x, want)
    # both calls' derivatives are within `off` of the exact one
    check_grad(dlogits, x, t, dlogp.double(), want, far, torch.where(used, 2 * off / dlogp.double().abs().clamp(min=1e-300), 0.0) + 8 * U)
    z = x.clone()
    got = training.policy_loss_gradient(z, t, *args, LOW, HIGH, KL, SCALE, out=z)
    assert got[2] is z and same(z, dlogits) and same(got[0], loss) and same(got[1], logp)


def test_policy_without_weights_and_reference():
    x, t, g = make(1, 36, 517, torch.float32)
    old, adv, w, ref = policy_inputs(x, t, g)
    one = torch.ones_like(w)
    loss, logp, dx = training.policy_loss_gradient(x, t, old, adv, None, None, LOW, HIGH, KL, SCALE)
    check_policy(x, t, old, adv, one, ref, None, dx, loss, logp, kl=0.0)
    assert same(training.policy_loss_gradient(x, t, old, adv, one, ref, LOW, HIGH, 0.0, SCALE)[2], dx)
    # the targets of rows that count for nothing may be anything negative
    t2 = torch.where(torch.arange(36, device="cuda") % 3 == 0, -100, t)
    loss, logp, dx = training.policy_loss_gradient(x, t2, old, adv, None, ref, LOW, HIGH, KL, SCALE)
    w = (t2 >= 0).float()
    check_policy(x, t, old, adv, w, ref, None, dx, loss, logp)


def test_rows_that_count_for_nothing_may_hold_anything():
    x, t, g = make(2, 20, 300, torch.bfloat16)
    args = [a.clone() for a in policy_inputs(x, t, g)]
    clean = training.policy_loss_gradient(x, t, *args, LOW, HIGH, KL, SCALE)
    off = args[2] == 0
    x[off] = float("nan")
    x[off.nonzero()[0, 0], 5] = float("inf")
    for a in (args[0], args[1], args[3]):
        a[off] = float("nan")
    got = training.policy_loss_gradient(x, t, *args, LOW, HIGH, KL, SCALE)
    assert off.any() and all(same(a, b) for a, b in zip(got, clean))
    none = training.policy_loss_gradient(x, t, args[0], args[1], torch.zeros_like(args[2]))
    assert float(none[0]) == 0 and bool((none[1] == 0).all()) and bool((none[2] == 0).all())
    empty = training.policy_loss_gradient(x[:0], t[:0], *(a[:0] for a in args))
    assert float(empty[0]) == 0 and empty[2].shape == (0, 300)


@pytest.mark.parametrize("cols", [40, 3001, 140001])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_impossible_tokens_infinities_and_nan(dtype, cols):
    inf, nan = float("inf"), float("nan")
    x, t, g = make(cols, 8, cols, dtype)
    t[:] = 17
    lowest = torch.finfo(dtype).min
    x[0, 20:], x[1, 20:], x[1, :16] = -inf, lowest, lowest
    x[2, 3], x[3, cols - 1], x[4] = inf, nan, -inf
    x[5, 17] = -inf
    x[6] = lowest
    logp, lse = training.token_logprobs_forward(x, t)
    good = [0, 1, 7]
    want, _, far = check_logp(x[good], t[good], logp[good], lse[good])
    assert torch.isnan(logp[2:5]).all() and logp[5] == -inf and torch.isfinite(lse[5])
    assert abs(float(logp[6]) + math.log(cols)) <= 1e-5 * math.log(cols)
    c = torch.ones(8, device="cuda")
    dx = training.token_logprobs_backward(c, x, t, lse, training.token_logprobs_forward(x, t, True)[2])
    even = torch.full((cols,), -1 / cols, device="cuda")  # a row of the lowest number alone is an even one
    even[17] += 1
    assert ((dx[6].float() - even).abs() <= 1e-5 * even.abs() + UT[dtype] * even.abs() + TINY[dtype]).all()
    assert bool((dx[0, 20:] == 0).all()) and torch.isnan(dx[2:4]).any(1).all()
    check_grad(dx[good], x[good], t[good], c[good].double(), want, far)
    t[7] = cols  # no such token
    logp, lse = training.token_logprobs_forward(x, t)
    assert torch.isnan(logp[7])
    assert torch.isnan(training.token_logprobs_backward(c, x, t, lse)[7]).all()
    t[:2] = -1
    logp, lse = training.token_logprobs_forward(x, t)
    assert bool((logp[:2] == 0).all()) and bool((lse[:2] == 0).all())
    assert bool((training.token_logprobs_backward(c, x, t, lse)[:2] == 0).all())
    # the same through the policy's pass: rows with NaN stay by themselves
    t[:] = 17
    zero = torch.zeros(8, device="cuda")
    loss, lp, dx = training.policy_loss_gradient(x, t, zero, c, torch.ones_like(c))
    a6 = math.exp(float(lp[6]))  # the ratio, of an even row
    assert torch.isnan(loss) and torch.isnan(lp[2:5]).all() and torch.isfinite(dx[good].float()).all()
    assert ((dx[6].float() / -a6 - even).abs() <= 1e-5 * even.abs() + UT[dtype] * even.abs() + TINY[dtype] / a6).all()
    assert torch.isnan(dx[3]).any() and bool((dx[0, 20:] == 0).all())


@pytest.mark.parametrize("cols", [40, 3001, 450001])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_rows_of_no_number_without_advantage(dtype, cols):
    # a row of advantage 0 has neither loss nor gradient, but a NaN in it is not hidden
    inf, nan = float("inf"), float("nan")
    x, t, g = make(cols + 1, 7, cols, dtype)
    lp = training.token_logprobs_forward(x, t)[0]
    old, zero = lp + 0.1, torch.zeros(7, device="cuda")
    for f in (training.policy_loss_gradient, training.policy_loss_forward):
        got = f(x, t, old, zero)
        assert float(got[0]) == 0 and bool((got[-1] == 0).all())
    adv = torch.where(torch.arange(7, device="cuda") == 6, 1.0, 0.0)
    clean = training.policy_loss_gradient(x, t, old, adv)

    def look(y, targets, o):
        loss, logp, dx = training.policy_loss_gradient(y, targets, o, adv)
        l2, _, _, dlogp = training.policy_loss_forward(y, targets, o, adv)
        assert torch.isnan(loss) and torch.isnan(l2) and torch.isnan(dlogp[3])
        assert torch.isnan(dx[3]).any() and bool((dlogp[[0, 1, 2, 4, 5]] == 0).all())
        rest = [0, 1, 2, 4, 5, 6]
        assert same(dx[rest], clean[2][rest]) and same(logp[rest], clean[1][rest])
    for column, value in ((0, nan), (cols - 1, nan), (cols // 2, inf), (slice(None), -inf)):
        y = x.clone()
        y[3, column] = value
        look(y, t, old)
    none, o = t.clone(), old.clone()
    none[3], o[3] = cols, nan
    look(x, none, old)
    look(x, t, o)
    # of weight 0 it counts for nothing all the same
    w = torch.ones(7, device="cuda")
    w[3] = 0
    assert float(training.policy_loss_gradient(x, none, o, zero, w)[0]) == 0
    # an impossible token is a number: ratio 0
    y = x.clone()
    y[3, t[3]] = -inf
    got = training.policy_loss_gradient(y, t, old, zero)
    assert float(got[0]) == 0 and got[1][3] == -inf and bool((got[2] == 0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_impossible_tokens_far_from_the_reference(dtype):
    # exp(d) - d - 1 grows without bound on both sides
    inf = float("inf")
    x, t, g = make(31, 4, 100, dtype)
    lp = training.token_logprobs_forward(x, t)[0]
    adv, w = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    y = x.clone()
    y[2, t[2]] = -inf  # d = inf
    ref = lp.clone()
    ref[2] = -inf  # d = -inf
    for logits, r in ((y, lp), (x, ref)):
        for f in (training.policy_loss_gradient, training.policy_loss_forward):
            got = f(logits, t, lp, adv, w, r, kl_coef=0.1)
            assert float(got[0]) == inf
        assert float(got[3][2]) == (-inf if r is lp else got[3][2]) and torch.isfinite(got[3][[0, 1, 3]]).all()


def test_rows_of_large_logits():
    # an offset that is the same for all of a row's logits changes nothing, but for the logits' own rounding
    x, t, g = make(12, 40, 500, torch.float32)
    x = (x * 16).round() / 16
    for offset in (2.0 ** 14, -2.0 ** 17):
        y = x + offset  # exact
        logp, lse, rest = training.token_logprobs_forward(y, t, True)
        want, _, far = check_logp(x, t, logp, None)
        check((lse.double() + rest.double()) - offset, want, far + U * 2.0 ** -6, "lse and rest")
        c = torch.randn(40, generator=g, device="cuda")
        check_grad(training.token_logprobs_backward(c, y, t, lse, rest), x, t, c.double(), want, far)
        for part in (training.token_logprobs, lambda a, b: training.policy_loss(a, b, logp, c)[0]):
            w, v = x.clone().requires_grad_(), y.clone().requires_grad_()
            part(w, t).sum().backward()
            part(v, t).sum().backward()
            assert (w.grad - v.grad).abs().max() <= 1e-5 * w.grad.abs().max()
        a, b = (training.policy_loss_gradient(z, t, logp, c)[2] for z in (x, y))
        assert (a - b).abs().max() <= 1e-5 * a.abs().max()


def test_borders_of_the_clipping():
    # one logit of 0 in two: logp is -log 2 exactly to the last place, ratios next to the borders on either side
    x = torch.zeros(4, 2, device="cuda")
    t = torch.zeros(4, device="cuda", dtype=torch.int64)
    lp = -math.log(2.0)
    step = 1e-6
    old = torch.tensor([lp - math.log(1.28) - step, lp - math.log(1.28) + step, lp - math.log(0.8) + step,
                        lp - math.log(0.8) - step], device="cuda")
    adv = torch.tensor([1.0, 1.0, -1.0, -1.0], device="cuda")
    _, _, _, dlogp = training.policy_loss_forward(x, t, old, adv, None, None, LOW, HIGH)
    assert dlogp[0] == 0 and abs(float(dlogp[1]) + 1.28) < 1e-5
    assert dlogp[2] == 0 and abs(float(dlogp[3]) - 0.8) < 1e-5
    # no clipping
    _, _, _, free = training.policy_loss_forward(x, t, old, adv, None, None, float("inf"), float("inf"))
    assert bool((free != 0).all())


def preference(x, t, starts, refs, beta, eps, scale):
    """(loss, logps, dlogp) in 64 bits."""
    lp = torch.log_softmax(x.double(), 1).gather(1, t.clamp(min=0)[:, None])[:, 0].requires_grad_()
    used = torch.where(t >= 0, lp, 0.0)
    sums = torch.stack([used[a: max(a, b)].sum() for a, b in zip(starts[:-1], starts[1:])]).view(2, -1)
    d = sums - refs.double() if refs is not None else sums
    h = beta * (d[0] - d[1])
    loss = scale * ((1 - eps) * torch.nn.functional.softplus(-h) + eps * torch.nn.functional.softplus(h)).sum()
    loss.backward()
    return loss.detach(), sums.detach(), lp.grad if lp.grad is not None else torch.zeros_like(lp), h.detach()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("cols,lengths", [(7, [1, 1]), (40, [3, 0, 5, 2]), (1001, [9, 33, 1, 40, 64, 7]),
                                          (32001, [20, 11, 5, 17]), (131072, [6, 4]), (264, [2] * 130)])
def test_preference(cols, lengths, dtype):
    rows = sum(lengths) + 3  # the last three are of no sequence
    x, t, g = make(cols, rows, cols, dtype)
    t[::5] = -100
    pairs = len(lengths) // 2
    starts = torch.tensor([0] + lengths, device="cuda").cumsum(0)
    at = starts.tolist()
    beta, eps, scale = 0.1, 0.1, 1 / pairs
    refs = preference(x, t, at, None, beta, eps, scale)[1].float() + torch.randn(2, pairs, generator=g, device="cuda") * 5
    want, sums, c, h = preference(x, t, at, refs, beta, eps, scale)
    loss, logps, dlogits = training.preference_loss_gradient(x, t, refs, starts, beta, eps, scale)
    l2, s2, lse, dlogp = training.preference_loss_forward(x, t, refs, starts, beta, eps, scale)
    assert same(loss, l2) and same(logps, s2)
    wl = torch.logsumexp(x.double(), 1)
    far = lse_far(x, wl)
    lp = (x.double().gather(1, t.clamp(min=0)[:, None])[:, 0] - wl).abs()
    each = torch.where(t >= 0, far + U * (lp + far), 0.0)
    off = torch.stack([each[a:b].sum() for a, b in zip(at[:-1], at[1:])]).view(2, -1)
    check(logps, sums, off + U * (sums.abs() + off), "logps")
    dh = beta * (off.sum(0)) + U * h.abs()  # the loss changes by no more than h does
    check(loss, want, scale * (dh + 4 * U * (1 + h.abs())).sum() + 2 * U * want, "loss")
    check(dlogp, c, scale * beta * (dh.max() + 16 * U) * torch.ones_like(c), "dlogp")
    assert bool((dlogp[t < 0] == 0).all()) and bool((dlogp[sum(lengths):] == 0).all())
    check_grad(dlogits, x, t.clamp(min=0), dlogp.double(), wl, far)
    z = x.clone()
    assert same(training.preference_loss_gradient(z, t, refs, starts, beta, eps, scale, out=z)[2], dlogits) and same(z, dlogits)


def test_preference_of_padded_batches():
    x, t, g = make(4, 24, 200, torch.bfloat16)
    t[::4] = -1
    refs = torch.randn(2, 3, generator=g, device="cuda") - 20
    starts = torch.arange(0, 25, 4, device="cuda")
    packed = training.preference_loss_gradient(x, t, refs, starts)
    padded = training.preference_loss_gradient(x.view(6, 4, 200), t.view(6, 4), refs)
    assert same(packed[0], padded[0]) and same(packed[1], padded[1]) and same(packed[2], padded[2].view(24, 200))
    with pytest.raises(ValueError):
        training.preference_loss_gradient(x, t, refs)
    with pytest.raises(ValueError):
        training.preference_loss_gradient(x[:20].view(5, 4, 200), t[:20].view(5, 4), refs)


def test_pairs_of_no_rows():
    # both sequences empty: S = 0, the margin is the references' alone
    x, t = torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda", dtype=torch.int64)
    refs = torch.tensor([[3.0], [1.0]], device="cuda")
    for args in ((x, t, refs, torch.zeros(3, device="cuda", dtype=torch.int64)), (x.view(2, 0, 50), t.view(2, 0), refs)):
        loss, logps, dlogits = training.preference_loss_gradient(*args, beta=0.5)
        assert abs(float(loss) - math.log1p(math.exp(1.0))) <= 1e-6 and bool((logps == 0).all()) and dlogits.shape == args[0].shape


def test_one_row_without_axes():
    x, t, g = make(13, 1, 77, torch.float16)
    assert same(training.token_logprobs_forward(x[0], t[0])[0], training.token_logprobs_forward(x, t)[0][0])


def test_starts_that_are_no_ranges_stay_inside():
    # cut at the rows that there are; a sequence whose end is not behind its start is empty
    x, t, g = make(5, 10, 64, torch.float32)
    logp = training.token_logprobs_forward(x, t)[0]
    for starts in ([0, 5, 1000], [-7, 4, 10], [8, 3, 9], [10, 10, 10], [-(1 << 63), 5, (1 << 63) - 1]):
        s = torch.tensor(starts, device="cuda")
        _, sums, _, c = training.preference_loss_forward(x, t, None, s)
        cut = [min(max(v, 0), 10) for v in starts]
        for i in (0, 1):
            part = logp[cut[i]: max(cut[i], cut[i + 1])].double().sum()
            assert abs(float(sums[i, 0]) - float(part)) <= 1e-6 * (1 + abs(float(part)))
        assert torch.isfinite(c).all()


def test_extreme_margins():
    # h far beyond exp's range either way
    x = torch.zeros(2, 2, device="cuda")
    t = torch.zeros(2, device="cuda", dtype=torch.int64)
    s = torch.tensor([0, 1, 2], device="cuda")
    for ref, loss, c in ((1e4, 1e4, -1.0), (-1e4, 0.0, 0.0)):
        refs = torch.tensor([[ref], [0.0]], device="cuda")
        value, _, _, dlogp = training.preference_loss_forward(x, t, refs, s, 1.0)
        assert abs(float(value) - loss) <= 1e-3 and dlogp.tolist() == [c, -c]
    nan = training.preference_loss_forward(x, t, torch.full((2, 1), float("nan"), device="cuda"), s)
    assert torch.isnan(nan[0]) and torch.isnan(nan[3]).all()


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("beta", [0.5, -0.5])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_infinite_margins(dtype, beta, smoothing):
    # An impossible token makes its sequence's sum -inf and the pair's margin infinite: one term of the pair's loss is
    # infinite and the other 0, and a term that the smoothing leaves out counts for nothing.
    inf = float("inf")
    x, t, g = make(21, 8, 40, dtype)
    s = torch.arange(0, 9, 2, device="cuda")  # the rows of two chosen sequences, then of two rejected ones
    clean = training.preference_loss_forward(x, t, None, s, beta, smoothing)
    for row in (1, 4):  # of pair 0, the chosen and the rejected sequence
        y = x.clone()
        y[row, t[row]] = -inf
        up = (row == 4) == (beta > 0)  # the margin is +inf
        far = smoothing != 0.0 if up else smoothing != 1.0
        value, sums, lse, dlogp = training.preference_loss_forward(y, t, None, s, beta, smoothing)
        loss, logps, dlogits = training.preference_loss_gradient(y, t, None, s, beta, smoothing)
        assert same(value, loss) and same(sums, logps)
        assert sums[row // 4, 0] == -inf and same(sums[:, 1], clean[1][:, 1])
        # what is left is the other pair's loss, of sums that were rounded once each
        a, b = sums[:, 1].tolist()
        h = beta * (a - b)
        rest = (1 - smoothing) * math.log1p(math.exp(-h)) + smoothing * math.log1p(math.exp(h))
        off = abs(beta) * U * (abs(a) + abs(b)) + 6 * U * (1 + abs(h))
        assert float(value) == inf if far else abs(float(value) - rest) <= off
        c = beta * (smoothing if up else smoothing - 1)
        want = torch.tensor([c, c, -c, -c], device="cuda")
        assert ((dlogp[[0, 1, 4, 5]] - want).abs() <= 4 * U * abs(c)).all()
        assert same(dlogp[[2, 3, 6, 7]], clean[3][[2, 3, 6, 7]])
        lse = torch.logsumexp(y.double(), 1)
        check_grad(dlogits, y, t, dlogp.double(), lse, lse_far(y, lse))
    # a margin of two infinities is none
    y[1, t[1]] = y[4, t[4]] = -inf
    assert torch.isnan(training.preference_loss_forward(y, t, None, s, beta, smoothing)[0])


def test_differentiable_calls():
    x, t, g = make(6, 24, 90, torch.float32)
    args = policy_inputs(x, t, g)
    w = x.clone().requires_grad_()
    loss, logp = training.policy_loss(w, t, *args, LOW, HIGH, KL, SCALE)
    assert not logp.requires_grad
    (loss * 3).backward()
    l2, _, lse, dlogp = training.policy_loss_forward(x, t, *args, LOW, HIGH, KL, SCALE)
    assert same(loss.detach(), l2)
    rest = training.token_logprobs_forward(x, t, True)[2]
    assert same(w.grad, training.token_logprobs_backward(dlogp, x, t, lse, rest, torch.tensor(3.0, device="cuda")))
    direct = training.policy_loss_gradient(x, t, *args, LOW, HIGH, KL, SCALE)[2]
    assert (w.grad / 3 - direct).abs().max() <= 1e-6 * direct.abs().max()
    # token log probabilities under a loss of their own, through logits whose last axis is not dense
    u = x.t().contiguous().requires_grad_()
    c = torch.randn(24, generator=g, device="cuda")
    (training.token_logprobs(u.t(), t) * c).sum().backward()
    v = x.clone().requires_grad_()
    (torch.log_softmax(v.double(), 1).gather(1, t[:, None])[:, 0] * c).sum().backward()
    assert (u.grad.t() - v.grad).abs().max() <= 1e-6
    refs = torch.randn(2, 3, generator=g, device="cuda") - 10
    p = x.view(6, 4, 90).clone().requires_grad_()
    loss, logps = training.preference_loss(p, t.view(6, 4), refs)
    loss.backward()
    want = training.preference_loss_gradient(x.view(6, 4, 90), t.view(6, 4), refs)[2]
    assert (p.grad - want).abs().max() <= 1e-6 * want.abs().max()


def test_gradients_against_differences():
    x, t, g = make(7, 12, 20, torch.float32, 1.0)
    args = policy_inputs(x, t, g)
    dx = training.policy_loss_gradient(x, t, *args, LOW, HIGH, KL, SCALE)[2]
    refs = torch.randn(2, 2, generator=g, device="cuda") - 5
    starts = torch.tensor([0, 4, 5, 9, 12], device="cuda")
    dp = training.preference_loss_gradient(x, t, refs, starts, 0.5)[2]
    v, h = torch.randn(12, 20, generator=g, device="cuda"), 2.0 ** -9  # ratios stay on their side of the borders
    for f, d in ((lambda y: training.policy_loss_forward(y, t, *args, LOW, HIGH, KL, SCALE)[0], dx),
                 (lambda y: training.preference_loss_forward(y, t, refs, starts, 0.5)[0], dp)):
        want = (f(x + h * v).double() - f(x - h * v).double()) / (2 * h)
        # rounding of a loss of about 10 in 32 bits over 2 h, third derivatives times h^2
        assert abs(float(want - (d.double() * v).sum())) <= 2e-3 * float(d.norm() * v.norm())


def test_graphs_and_streams():
    x, t, g = make(8, 64, 5001, torch.bfloat16)
    args = policy_inputs(x, t, g)
    refs, starts = torch.randn(2, 4, generator=g, device="cuda"), torch.arange(0, 65, 8, device="cuda")

    def everything(**kw):
        logp, lse = training.token_logprobs_forward(x, t, **kw)
        return (logp, lse, training.token_logprobs_backward(logp, x, t, lse, **kw),
                *training.policy_loss_gradient(x, t, *args, **kw), *training.policy_loss_forward(x, t, *args, **kw),
                *training.preference_loss_gradient(x, t, refs, starts, **kw))

    eager = everything()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = everything(stream=s)
    s.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, each with workspaces of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = everything()
        graphs.append((graph, kept))
    for graph, _ in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c, d in zip(eager, other, graphs[0][1], graphs[1][1]):
        assert same(a, b) and same(a, c) and same(a, d)
    out = torch.empty_like(x)
    for f in (lambda: training.policy_loss_gradient(x, t, *args, out=out),
              lambda: training.preference_loss_gradient(x, t, refs, starts, out=out),
              lambda: training.token_logprobs_backward(eager[0], x, t, eager[1], out=out)):
        v = out._version
        f()
        assert out._version > v


def test_more_than_two_to_the_31_elements():
    rows, cols = 70001, 32000
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    last, t1, g = make(9, 3, cols, torch.bfloat16)
    x[-3:] = last
    t = torch.zeros(rows, device="cuda", dtype=torch.int64)
    t[-3:] = t1
    logp, lse = training.token_logprobs_forward(x, t)
    # few rows are summed by more threads, in another order: by lse_far's roundings apart
    assert (logp[-3:] - training.token_logprobs_forward(last, t1)[0]).abs().max() <= 1e-5
    assert (logp[:-3] + math.log(cols)).abs().max() <= 1e-5
    w = torch.zeros(rows, device="cuda")
    w[-3:] = 1.0
    loss, lp, dx = training.policy_loss_gradient(x, t, logp, torch.ones(rows, device="cuda"), w, out=x)
    alone = training.policy_loss_gradient(last, t1, logp[-3:].clone(), torch.ones(3, device="cuda"))
    near = alone[2].float()
    assert ((dx[-3:].float() - near).abs() <= 2 * UT[x.dtype] * near.abs()).all() and bool((dx[:-3] == 0).all())
    assert abs(float(loss - alone[0])) <= 1e-4
