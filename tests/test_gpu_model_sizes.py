"""The forms that dropout and the losses take for large calls, on the GPU against their definitions:
dropout of several units of 8 elements a thread (from 5 million elements on), policies of more rows
than fit the GPU at a time, gradients of logits in long parts (from 10 million packs of 16 bytes on).

Dropout is compared bit for bit. Tolerances of a row's sum of exponentials (U = 2^-24), by the kernels'
layouts: a thread has at most 32 packs, or 1/256 of the row's where that is more, and takes them four
at a time; such a group adds at most 18 roundings (16 elements' pairs and two joins) and scales the
sum at most once, by an exponential off by 2^-22; up to three groups more are parts. 9 steps join a
block's threads, 8 its cluster's blocks. The rest is as in test_gpu_losses."""
import pytest
import torch

import test_gpu_losses as losses
from ring_allreduce_virtual_gb300 import training
from test_gpu_dropout import numbers, rand, same, want

pytestmark = pytest.mark.gpu

U, E2 = losses.U, losses.E2
TYPES = losses.TYPES
MANY = 5_000_000 + 1_000_037  # elements


def far(x, lse):
    """How far lse may be off."""
    packs = x.shape[1] * x.element_size() / 16
    groups = max(32, packs / 256 + 1) / 4 + 3
    x = x.double()
    p = (x - lse[:, None]).exp()
    away = torch.where(p > 0, p * (x.amax(1, keepdim=True) - x), 0.0).sum(1)
    return E2 + 3 * U * away + groups * (18 * U + E2) + 12 * E2 + 20 * U + 4 * U


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shift", [0, 3])
def test_dropout_of_many_elements(dtype, shift):
    x, r = (rand((MANY + shift,), dtype, s)[shift:] for s in (1, 2))
    seed = 0xFEDCBA9876543210
    device = torch.tensor([seed - (1 << 64)], device="cuda")
    for p, offset in ((0.1, 0), (0.1000003, 1), (0.5, 4), (0.25, (1 << 41) + 7)):
        for residual in (None, r):
            expect = want(x, p, seed, offset, residual)
            assert same(training.dropout_forward(x, p, seed, offset, residual), expect), (p, offset)
            assert same(training.dropout_forward(x, p, device, offset, residual), expect), (p, offset)
            base = torch.full((MANY + shift + 64,), 7.0, device="cuda", dtype=dtype)
            z = base[shift: MANY + shift].copy_(x)
            assert training.dropout_forward(z, p, device if residual is None else seed, offset, residual, out=z) is z
            assert same(z, expect)
            assert bool((base[:shift] == 7.0).all()) and bool((base[MANY + shift:] == 7.0).all())
        z = r.clone() if shift == 0 else torch.empty_like(base)[shift: MANY + shift].copy_(r)
        assert same(training.dropout_forward(x, p, seed, offset, z, out=z), expect)
    assert same(training.dropout_forward(x, 0.0, seed), x) and same(training.dropout_forward(x, 1.0, seed, 1, r), r)


@pytest.mark.parametrize("offset", [0, 5])
def test_upper_halves_that_tie_among_many(offset):
    # the upper half equals the threshold's about 90 times; the lower one then decides
    x = torch.ones(MANY, device="cuda", dtype=torch.bfloat16)
    u = numbers(MANY, 77, offset, "cuda")
    tied = u[u >> 16 == 20000]
    assert len(tied) > 32
    for t in (int(tied[0]), int(tied[0]) + 1, int(tied.max()) + 1):
        p = t / 2.0 ** 32
        assert round(p * 2 ** 32) == t
        assert torch.equal(training.dropout_forward(x, p, 77, offset) != 0, u >= t)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(2400, 8000), (2100, 50001), (5000, 264)])
def test_policy_of_many_rows(rows, cols, dtype, monkeypatch):
    monkeypatch.setattr(losses, "lse_far", far)
    x, t, g = losses.make(rows + cols, rows, cols, dtype)
    args = losses.policy_inputs(x, t, g)
    loss, logp, dlogits = losses.policy_call(x, t, g)
    losses.check_policy(x, t, *args, None, dlogits, loss, logp)
    z = x.clone()
    got = losses.policy_call(z, t, g, out=z)
    assert same(z, dlogits) and same(got[0], loss) and same(got[1], logp)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("more,shift", [(0, 0), (3, 0), (3, 1)])
def test_gradients_in_long_parts(dtype, more, shift, monkeypatch):
    monkeypatch.setattr(losses, "lse_far", far)
    rows, cols = 700 if dtype != torch.float32 else 350, 131072 + more
    x, t, g = losses.make(more + shift, rows, cols, dtype)
    logp, lse, rest = training.token_logprobs_forward(x, t, True)
    c = torch.randn(rows, generator=g, device="cuda")
    c[::9] = 0
    base = torch.full((shift + rows * cols + 64,), 7.0, device="cuda", dtype=dtype)
    out = base[shift: shift + rows * cols].view(rows, cols)
    training.token_logprobs_backward(c, x, t, lse, rest, out=out)
    assert bool((base[:shift] == 7.0).all()) and bool((base[shift + rows * cols:] == 7.0).all())
    for i in range(0, rows, 100):
        part = slice(i, i + 100)
        exact, _, off = losses.check_logp(x[part], t[part], logp[part], lse[part])
        losses.check_grad(out[part], x[part], t[part], c[part].double(), exact, off)
    training.token_logprobs_backward(c, x, t, lse, rest, out=x)
    assert same(x, out)
