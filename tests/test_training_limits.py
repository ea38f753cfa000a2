"""The training entries at the ends of their sizes: vocabularies, row counts and hidden sizes at which a
32-bit offset, a grid's dimension or a number of passes would run out."""
import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status
from training_reference import IGNORE, CrossEntropy, assert_close, embedding_grad, half_step

pytestmark = pytest.mark.gpu


def table(V, H, scale, seed=3, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.empty((V, H), device="cuda", dtype=dtype)
    step = max(1, (1 << 26) // H)
    for v in range(0, V, step):
        part = W[v:v + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return W


def test_a_vocabulary_of_2_28_entries():
    """1024 pieces, ids in four digits, row offsets past 2^31 elements."""
    V, H, rows = 2 ** 28 + 5, 8, 3
    W = table(V, H, 0.3)
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden = torch.randn((rows, H), generator=g, device="cuda").bfloat16()
    targets = torch.tensor([V - 1, 5, V - 70000], device="cuda", dtype=torch.int32)
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, reduction="none", ignore_index=None)
    one = torch.ones(rows, device="cuda")
    d_hidden, d_W, _ = lm.cross_entropy_grad(hidden, W, targets, lse, one, reduction="none",
                                             ignore_index=None)
    check_status()
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    first = torch.zeros((rows, H), dtype=torch.float64, device="cuda")
    for v in range(0, V, 1 << 24):
        w = W[v:v + (1 << 24)].double()
        e = torch.exp(hidden.double() @ w.t())
        total += e.sum(1)
        first += e @ w
    want = torch.log(total)
    # a running sum in fp32 of V / 128 terms in 128 segments, each merge two roundings and an
    # exponential: 2^-21 a merge, in a segment and then over the 128
    tol = torch.full_like(want, (V / 128 / 128 + 128) * 2.0 ** -21)
    assert_close(lse, want, tol, "lse")
    zt = (hidden.double() * W[targets.long()].double()).sum(1)
    assert_close(loss, want - zt, tol, "loss")
    u = half_step(W.dtype)
    mean = first / total[:, None]
    wt = W[targets.long()].double()
    # p's common error is that of lse; each entry of d half a step, the sum over V of sizes E|w|
    size = 0.3 * 4
    assert_close(d_hidden, mean - wt, size * (float(tol.max()) + u) + u * (mean - wt).abs(), "d_hidden")
    assert_close(d_W[targets.long()], -hidden.double(), (u + 2.0 ** -20) * hidden.double().abs() + 1e-6,
                 "d_W at the targets")
    some = torch.tensor([0, 77, 2 ** 27, 2 ** 28 - 1, V - 2], device="cuda")
    p = torch.exp(hidden.double() @ W[some].double().t() - want[:, None])
    assert_close(d_W[some], p.t() @ hidden.double(),
                 (p.t() @ hidden.double().abs()) * (2 * u + float(tol.max()) + 2.0 ** -12), "d_W")
    x = lm.embedding(targets, W, scale=2.0)
    assert torch.equal(x, W[targets.long()] * 2)
    lm.embedding_grad(x, targets, V, out=d_W)
    check_status()
    assert torch.equal(d_W[targets.long()], x)
    d_W[targets.long()] = 0
    assert not any(bool(d_W[v:v + (1 << 24)].any()) for v in range(0, V, 1 << 24))


def test_a_million_rows():
    rows, H, V = 2 ** 20 + 3, 64, 300
    g = torch.Generator(device="cuda").manual_seed(2)
    W = table(V, H, 0.1)
    hidden = table(rows, H, 1.0, seed=4)
    targets = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.rand((rows,), generator=g, device="cuda") < 0.3
    targets[out] = IGNORE
    hidden[out] = float("nan")
    one = torch.ones((), device="cuda")
    loss, lse = lm.cross_entropy_f32(hidden, W, targets)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, one)
    check_status()
    ref = CrossEntropy(hidden, W, targets, grad_loss=one)
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(loss, ref.loss, ref.loss_tol, "loss")
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")
    ids = targets.clone()
    d = table(rows, H, 1.0, seed=5)
    assert_close(lm.embedding_grad(d, ids, V), *embedding_grad(d, ids, V), "embedding_grad")
    check_status()


@pytest.mark.parametrize("rows", [4, 150])
def test_hidden_rows_of_2_19_entries(rows):
    H, V = 2 ** 19, 40
    W, hidden = table(V, H, 0.002), table(rows, H, 1.0, seed=6)
    targets = (torch.arange(rows, device="cuda") % V).to(torch.int32)
    one = torch.ones((), device="cuda")
    loss, lse = lm.cross_entropy_f32(hidden, W, targets)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, one)
    check_status()
    ref = CrossEntropy(hidden, W, targets, grad_loss=one)
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(loss, ref.loss, ref.loss_tol, "loss")
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")


@pytest.mark.parametrize("tokens", [5, 1100])
def test_embedding_rows_of_the_widest(tokens):
    """H = 2^24: 32768 slices of columns, a block a slice; more tokens than a block sums at once."""
    H, V = 2 ** 24, 3
    d = table(8, H, 1.0)
    base = torch.arange(8, device="cuda", dtype=torch.int32) % 5 - 1   # ids -1 .. 3 of a table of 3
    if tokens <= 8:
        ids, d = base[:tokens], d[:tokens]
        got = lm.embedding_grad(d, ids, V)
        want = [embedding_grad(d[:, k:k + 2 ** 20].contiguous(), ids, V) for k in range(0, H, 2 ** 20)]
        for k, (w, tol) in zip(range(0, H, 2 ** 20), want):
            assert_close(got[:, k:k + 2 ** 20], w, tol, "embedding_grad")
        out = lm.embedding(ids, got)
        held = (ids >= 0) & (ids < V)
        assert torch.equal(out[held], got[ids[held].long()]) and not out[~held].any()
    else:  # (a row of d_out is 32 MB, 37 GB in all)
        d = torch.ones((tokens, H), device="cuda", dtype=torch.bfloat16)
        ids = torch.full((tokens,), 2, device="cuda", dtype=torch.int32)
        ids[7], ids[8] = 0, -1
        got = lm.embedding_grad(d, ids, V)
        assert (got[2] == torch.tensor(tokens - 2.0).bfloat16().item()).all()
        assert (got[0] == 1).all() and not got[1].any()
    check_status()


def test_alpha_below_zero():
    g = torch.Generator(device="cuda").manual_seed(8)
    W, hidden = table(700, 64, 0.1), table(200, 64, 1.0, seed=9)
    targets = torch.randint(0, 700, (200,), generator=g, device="cuda", dtype=torch.int32)
    one = torch.ones((), device="cuda")
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, alpha=-0.5)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, one, alpha=-0.5)
    check_status()
    ref = CrossEntropy(hidden, W, targets, alpha=-0.5, grad_loss=one)
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(loss, ref.loss, ref.loss_tol, "loss")
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")
