"""NaN and infinities in what counts: as torch has them in 64 bits, an infinite logit above all others
being inf - inf and so NaN. (Infinities that the bias takes out of the vocabulary, and what ignored
rows hold, have their tests in test_cross_entropy.py.)"""
import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def make(rows, H, V, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(rows + V + seed)
    W = (torch.randn((V, H), generator=g, device="cuda") * 0.1).to(dtype)
    hidden = torch.randn((rows, H), generator=g, device="cuda").to(dtype)
    targets = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return hidden, W, targets, torch.zeros(V, device="cuda", dtype=dtype)


def step(hidden, W, targets, bias, ignore_index=None):
    how = dict(bias=bias, reduction="none", ignore_index=ignore_index)
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, **how)
    one = torch.ones(hidden.shape[0], device="cuda")
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, one, **how)
    check_status()
    return loss, lse, grads


def logits(hidden, W, bias):
    """In 64 bits, summed from the products, so that inf * 0 and inf - inf are NaN as they are."""
    return (hidden.double()[:, None, :] * W.double()[None]).sum(2) + bias.double()


@pytest.mark.parametrize("rows", [5, 140, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_target_alone_is_infinite(rows, dtype):
    """By its bias, and by a hidden entry that makes every other logit -inf."""
    hidden, W, targets, bias = make(rows, 64, 300, dtype)
    bias[17] = INF
    targets.fill_(17)
    loss, lse, grads = step(hidden, W, targets, bias)
    assert torch.isnan(loss).all() and torch.isnan(lse).all()
    assert torch.isnan(grads[0]).all() and torch.isnan(grads[1]).all() and torch.isnan(grads[2]).all()
    hidden, W, targets, bias = make(rows, 64, 300, dtype)
    W[:, 3] = -W[:, 3].abs() - 0.01
    W[17, 3] = 0.5
    hidden[2, 3] = INF
    targets[2] = 17
    loss, lse, grads = step(hidden, W, targets, bias)
    for t in (loss, lse, grads[0].float().sum(1)):
        assert torch.isnan(t).nonzero().tolist() == [[2]]
    assert torch.isnan(grads[1]).all() and torch.isnan(grads[2]).all()


@pytest.mark.parametrize("rows", [5, 140, 300])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_in_a_hidden_row(rows, value):
    """That row is NaN (its logits are infinities of either sign), and so are d_W and d_bias."""
    hidden, W, targets, bias = make(rows, 64, 300)
    want = step(hidden, W, targets, bias)
    hidden[4, 3] = value
    z = logits(hidden[4:5], W, bias)
    assert torch.isnan(z).all() or (z == INF).any()
    loss, lse, grads = step(hidden, W, targets, bias)
    others = torch.arange(rows, device="cuda") != 4
    for got, was in ((loss, want[0]), (lse, want[1]), (grads[0], want[2][0])):
        assert torch.isnan(got[4]).all() and torch.equal(got[others], was[others])
    assert torch.isnan(grads[1]).all() and torch.isnan(grads[2]).all()


@pytest.mark.parametrize("rows", [5, 140, 300])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_in_a_row_of_the_table(rows, value):
    """Rows to whose logit it gives +inf or NaN are NaN; rows to whose logit it gives -inf are not
    touched in their loss, but their d_hidden is 0 * inf."""
    hidden, W, targets, bias = make(rows, 64, 300)
    targets[targets == 30] = 31
    hidden[0, 3], hidden[1, 3] = 1.0, -1.0
    want = step(hidden, W, targets, bias)
    W[30, 3] = value
    z = logits(hidden, W, bias)[:, 30]
    out = z == -INF
    assert value != value or (out.any() and not out.all())
    loss, lse, grads = step(hidden, W, targets, bias)
    assert torch.isnan(loss[~out]).all() and torch.isnan(lse[~out]).all()
    off = (loss[out] - want[0][out]).abs()
    # (entry 30 itself is gone from the sum: log(1 - p), p at most e^5 / 300)
    assert (off < 0.7).all() and not torch.isnan(off).any() and not torch.isnan(lse[out]).any()
    assert torch.isnan(grads[0][:, 3]).all()
    assert torch.isnan(grads[1]).all() and torch.isnan(grads[2]).all()


@pytest.mark.parametrize("rows", [5, 300])
def test_a_target_at_minus_infinity(rows):
    """Infinite loss, and a gradient that is finite: the softmax, less 1 at the target."""
    hidden, W, targets, bias = make(rows, 64, 300)
    bias[40] = -INF
    targets[3] = 40
    targets[targets == 40] = 41
    targets[3] = 40
    loss, lse, grads = step(hidden, W, targets, bias)
    assert (loss == INF).nonzero().tolist() == [[3]] and torch.isfinite(lse).all()
    for g in grads:
        assert torch.isfinite(g).all()
    z = logits(hidden, W, bias)
    p = torch.softmax(z, 1)
    assert float(grads[2][40]) == -1.0
    want = p[3] @ W.double() - W[40].double()
    # each entry of d off by half a step, the output by another, the softmax by 2^-12 of itself
    tol = (p[3] @ W.double().abs()) * (2.0 ** -8 + 2.0 ** -12) + 2.0 ** -8 * want.abs() \
        + (W[40].double().abs()) * 2.0 ** -20
    assert ((grads[0][3].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows", [5, 140, 300])
def test_a_target_near_the_largest_number(rows):
    """A logit that is finite, though its product with log2(e) is not: sure of its target."""
    hidden, W, targets, bias = make(rows, 64, 300)
    bias[17] = 3e38
    targets.fill_(17)
    loss, lse, grads = step(hidden, W, targets, bias)
    assert torch.count_nonzero(loss) == 0 and (lse == bias[17].float()).all()
    for g in grads:
        assert not g.any()
