"""The training operators as a model uses them together: token embedding, cross entropy over the tied
table, both gradients into one buffer; by the plain entries and through autograd."""
import math

import pytest
import torch

import fp32_accumulate_lm_b200 as lm
import training_reference as ref
from gpu_helpers import check_status
from training_reference import IGNORE, CrossEntropy, assert_close, half_step

pytestmark = pytest.mark.gpu


def batch(sequences=6, length=50, H=136, V=900, dtype=torch.bfloat16, seed=0):
    """A padded batch: ids (-1 behind a sequence's end), next-token targets (ignored where there is
    none) and a table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)).to(dtype)
    ids = torch.randint(0, V, (sequences, length), generator=g, device="cuda", dtype=torch.int32)
    ends = torch.randint(length // 3, length + 1, (sequences, 1), generator=g, device="cuda")
    at = torch.arange(length, device="cuda")
    ids[at >= ends] = -1
    targets = torch.full_like(ids, IGNORE)
    targets[:, :-1] = torch.where(ids[:, 1:] >= 0, ids[:, 1:], IGNORE)
    return ids, targets, W


def test_a_tied_step():
    ids, targets, W = batch()
    V, H = W.shape
    scale = math.sqrt(H)
    x = lm.embedding(ids, W, scale=scale)
    want, tol = ref.embedding(ids, W, scale)
    assert_close(x, want, tol, "embedding")
    hidden = x.view(-1, H)
    flat = targets.view(-1)
    loss, lse = lm.cross_entropy_f32(hidden, W, flat)
    one = torch.ones((), device="cuda")
    d_hidden, d_W, _ = lm.cross_entropy_grad(hidden, W, flat, lse, one)
    head = CrossEntropy(hidden, W, flat, grad_loss=one)
    assert_close(loss, head.loss, head.loss_tol, "loss")
    assert_close(d_W, head.d_W, head.d_W_tol, "d_W of the head")
    lm.embedding_grad(d_hidden.view(x.shape), ids, V, scale=scale, accumulate=True, out=d_W)
    check_status()
    # the formula of the whole step; d_hidden is off by its own bound when it is scattered
    table, table_tol = ref.embedding_grad(head.d_hidden.view(x.shape).to(W.dtype), ids, V, scale)
    want = head.d_W + ref.embedding_grad(head.d_hidden.view(x.shape), ids, V, scale)[0]
    spread = torch.zeros_like(want)
    held = (ids.view(-1) >= 0).nonzero()[:, 0]
    spread.index_add_(0, ids.view(-1)[held].long(), head.d_hidden_tol[held] * scale)
    tol = head.d_W_tol + spread + table_tol + half_step(W.dtype) * want.abs() * 2
    assert_close(d_W, want, tol, "d_W")


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd_of_a_tied_table(reduction):
    ids, targets, W = batch(seed=1)
    V, H = W.shape
    table = W.clone().requires_grad_()
    bias = (torch.randn(V, device="cuda") * 0.1).bfloat16().requires_grad_()
    x = lm.embed(ids, table, scale=3.0)
    x.retain_grad()
    loss = lm.linear_cross_entropy(x, table, targets, alpha=0.5, bias=bias, z_loss=1e-3,
                                   reduction=reduction)
    assert loss.shape == (targets.shape if reduction == "none" else ())
    up = torch.randn(targets.shape, device="cuda") if reduction == "none" else \
        torch.tensor(2.0, device="cuda")
    loss.backward(up)
    check_status()
    head = CrossEntropy(x.detach().view(-1, H), W, targets.view(-1), alpha=0.5,
                        bias=bias.detach(), z_loss=1e-3, reduction=reduction,
                        grad_loss=up.reshape(-1) if reduction == "none" else up)
    assert_close(loss.detach().reshape(head.loss.shape), head.loss, head.loss_tol, "loss")
    assert_close(x.grad.view(-1, H), head.d_hidden, head.d_hidden_tol, "d_hidden")
    assert_close(bias.grad, head.d_bias, head.d_bias_tol, "d_bias")
    # autograd adds the two gradients of the table, rounded each, in 16 bits
    part, part_tol = ref.embedding_grad(x.grad, ids, V, 3.0)
    want = head.d_W + part
    u = half_step(W.dtype)
    assert_close(table.grad, want, head.d_W_tol + part_tol + u * (want.abs() + head.d_W_tol), "W.grad")


def test_autograd_gives_only_what_is_wanted():
    ids, targets, W = batch(seed=2)
    x = lm.embedding(ids, W)
    frozen = x.clone().requires_grad_()
    lm.linear_cross_entropy(frozen, W, targets).backward()       # a frozen table
    assert frozen.grad is not None and W.grad is None
    table = W.clone().requires_grad_()
    lm.linear_cross_entropy(x, table, targets).backward()        # a frozen body
    one = torch.ones((), device="cuda")
    _, lse = lm.cross_entropy_f32(x.view(-1, W.shape[1]), W, targets.view(-1))
    d_hidden, d_W, _ = lm.cross_entropy_grad(x.view(-1, W.shape[1]), W, targets.view(-1), lse, one)
    assert torch.equal(frozen.grad.view(d_hidden.shape), d_hidden)
    assert torch.equal(table.grad, d_W)
    # a loss that several terms use, and a transposed upstream gradient
    table.grad = None
    rows = lm.linear_cross_entropy(x, table, targets, reduction="none")
    (rows.t().sum() + 2 * rows.sum()).backward()
    three = torch.full((targets.numel(),), 3.0, device="cuda")
    _, d_W3, _ = lm.cross_entropy_grad(x.view(-1, W.shape[1]), W, targets.view(-1), lse, three,
                                       reduction="none")
    assert torch.equal(table.grad, d_W3)
    with torch.no_grad():
        assert not lm.linear_cross_entropy(x, table, targets).requires_grad
    # not differentiable twice: an error, not a wrong number
    loss = lm.linear_cross_entropy(frozen, W, targets)
    (g,) = torch.autograd.grad(loss, frozen, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    check_status()


def test_autograd_on_another_stream():
    ids, targets, W = batch(seed=3)
    table = W.clone().requires_grad_()
    lm.linear_cross_entropy(lm.embed(ids, table), table, targets).backward()
    want = table.grad.clone()
    table.grad = None
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lm.linear_cross_entropy(lm.embed(ids, table), table, targets).backward()
    s.synchronize()
    check_status()
    assert torch.equal(table.grad, want)


def test_autograd_is_refused_in_a_capture():
    """The refusal comes before anything is launched; the forward pass alone and the plain entries
    are captured."""
    ids, targets, W = batch(seed=4)
    table = W.clone().requires_grad_()
    eager = lm.linear_cross_entropy(lm.embed(ids, table), table, targets)   # lives on
    flat, one = targets.view(-1), torch.ones((), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            lm.embed(ids, table)
        with pytest.raises(RuntimeError, match="captured"):
            lm.linear_cross_entropy(torch.zeros_like(W[:1]).expand(1, -1), table, flat[:1])
        x = lm.embedding(ids, W).view(flat.numel(), -1)
        loss, lse = lm.cross_entropy_f32(x, W, flat)
        d_hidden, d_W, _ = lm.cross_entropy_grad(x, W, flat, lse, one)
        lm.embedding_grad(d_hidden.view(*ids.shape, -1), ids, W.shape[0], accumulate=True, out=d_W)
        with torch.no_grad():
            again = lm.linear_cross_entropy(x, table, flat)
    graph.replay()
    check_status()
    assert torch.equal(again, loss) and torch.equal(loss, eager.detach())
    head = CrossEntropy(x, W, flat, grad_loss=one)
    part, part_tol = ref.embedding_grad(d_hidden.view(*ids.shape, -1), ids, W.shape[0])
    u = half_step(W.dtype)
    want = head.d_W + part
    tol = head.d_W_tol + part_tol + u * (want.abs() + head.d_W_tol)
    assert_close(d_W, want, tol, "d_W, captured")
    eager.backward()
    assert_close(table.grad, want, tol, "W.grad")
