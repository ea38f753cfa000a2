"""lmhead_cross_entropy_f32 and lmhead_cross_entropy_grad against the formulas in 64 bits
(tests/training_reference.py, which derives the tolerances), at the sizes and masks where tiles,
pieces of the vocabulary, splits and ragged ends meet."""
import math

import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status
from training_reference import IGNORE, CrossEntropy, assert_close

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(rows, H, V, dtype="bf16", bias=False, masked=0.0, seed=0, alpha=1.0, reduction="mean",
         garbage=True):
    g = torch.Generator(device="cuda").manual_seed(1000 * rows + 10 * H + V + seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dt = DTYPES[dtype]
    W = (normal(V, H) * (0.8 / (math.sqrt(H) * alpha))).to(dt)
    targets = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    hidden = (normal(rows, H) + W[targets.long()].float() * 4 / alpha).to(dt)
    if masked:
        out = torch.rand((rows,), generator=g, device="cuda") < masked
        targets[out] = IGNORE
        if garbage:  # what padding may hold
            hidden[out, ::2] = float("nan")
            hidden[out, 1::2] = float("inf")
    b = (normal(V) * 0.5).to(dt) if bias else None
    gl = normal(rows) / rows if reduction == "none" else torch.tensor(0.75, device="cuda")
    return hidden, W, targets, b, gl


def run_both(hidden, W, targets, b, gl, **how):
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, bias=b, **how)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, **how)
    check_status()
    ref = CrossEntropy(hidden, W, targets, bias=b, grad_loss=gl, **how)
    return loss, lse, grads, ref


def compare(loss, lse, grads, ref):
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(loss, ref.loss, ref.loss_tol, "loss")
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")
    if grads[2] is not None:
        assert_close(grads[2], ref.d_bias, ref.d_bias_tol, "d_bias")


# rows around the lone-CTA and pair tiles, vocabularies around the 128- and 256-wide ones, hidden
# sizes that end inside a K step and a tile
SIZES = [(1, 8, 1), (1, 64, 127), (3, 8, 5), (4, 256, 1024), (31, 72, 129), (127, 200, 255),
         (128, 64, 300), (129, 64, 300), (130, 136, 257), (255, 264, 256), (256, 64, 512),
         (257, 520, 513), (300, 512, 4097), (1000, 128, 8200)]


@pytest.mark.parametrize("rows,H,V", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sizes(rows, H, V, dtype):
    args = make(rows, H, V, dtype)
    compare(*run_both(*args, ignore_index=None))


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,H,V,masked", [(7, 64, 300, 0.5), (128, 136, 700, 0.3),
                                             (400, 72, 1000, 0.4), (513, 256, 600, 0.9)])
def test_masked_rows_bias_alpha_and_z_loss(rows, H, V, masked, dtype, reduction):
    args = make(rows, H, V, dtype, bias=True, masked=masked, alpha=0.25, reduction=reduction)
    compare(*run_both(*args, alpha=0.25, z_loss=1e-3, reduction=reduction))


def test_pieces_of_the_vocabulary():
    """Enough rows that the vocabulary is taken in several pieces (the last one ragged), with a bias,
    both d buffers and the sums of d_hidden over the pieces in use."""
    rows, H, V = 16640, 64, 10001
    hidden, W, targets, b, gl = make(rows, H, V, bias=True, masked=0.2)
    compare(*run_both(hidden, W, targets, b, gl))
    # the pieces' buffers hold the whole d nowhere
    assert lm.cross_entropy_grad_workspace_bytes(rows, H, V) < rows * V * 4


@pytest.mark.parametrize("rows,H,V", [(64, 128, 20000), (300, 72, 9000)])
def test_splits_of_the_vocabulary(rows, H, V):
    """Few output tiles of d_hidden: its sum over the vocabulary is split and added up again."""
    compare(*run_both(*make(rows, H, V, "f16"), reduction="sum"))


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("H", [8, 48, 64, 128, 200, 248, 264, 320, 328, 384, 448, 504, 640, 1032])
def test_edges_of_the_hidden_size(rows, H):
    """The last tile of the gradients is as narrow as what is left of H, in steps of 64 columns (128
    on a CTA pair), and takes its columns in boxes of their own."""
    for V, dtype, masked in ((1500, "bf16", 0.2), (5001, "f16", 0.0)):
        compare(*run_both(*make(rows, H, V, dtype, masked=masked, bias=True), reduction="sum"))


@pytest.mark.parametrize("H", [40, 192, 320, 448, 520, 712, 960])
def test_edges_of_big_tiles(H):
    """As above in tiles of 512 columns, of which the second accumulator may have none."""
    rows, V = 2048, 131072
    compare(*run_both(*make(rows, H, V, "bf16", masked=0.3)))


@pytest.mark.parametrize("rows,H,V,dtype", [(2100, 72, 130001, "bf16"), (4097, 64, 65537, "f16"),
                                            (16641, 136, 16200, "bf16"), (2048, 264, 131072, "f16")])
def test_big_tiles(rows, H, V, dtype):
    """2^28 logits and more take tiles of 256 x 512 and 512 x 256: ragged rows, vocabularies and
    hidden sizes, masked rows, pieces, K shorter than the ring of stages and longer."""
    assert rows * V >= 2 ** 28
    hidden, W, targets, b, gl = make(rows, H, V, dtype, bias=True, masked=0.1)
    loss, lse, grads, ref = run_both(hidden, W, targets, b, gl, z_loss=1e-4)
    compare(loss, lse, grads, ref)
    again = lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, z_loss=1e-4)
    for a, c in zip(grads, again):
        assert torch.equal(a, c)
    base = grads[1].clone()
    lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, z_loss=1e-4, accumulate=True,
                          out=(None, base, None))
    check_status()
    twice = ref.d_W + grads[1].double()
    assert_close(base, twice, ref.d_W_tol + 2.0 ** -7 * twice.abs(), "d_W, accumulated")


def test_big_tiles_with_few_rows_that_count():
    rows, H, V = 4096, 64, 65536
    hidden, W, targets, b, gl = make(rows, H, V, masked=0.99)
    compare(*run_both(hidden, W, targets, b, gl))
    targets.fill_(IGNORE)
    loss, lse, grads, ref = run_both(hidden, W, targets, b, gl)
    for t in (loss, lse, grads[0], grads[1]):
        assert torch.count_nonzero(t) == 0 and not torch.isnan(t).any()


@pytest.mark.parametrize("wanted", [(0,), (1,), (2,), (0, 1), (1, 2), (0, 2), (0, 1, 2)])
@pytest.mark.parametrize("rows", [60, 200])
def test_gradients_wanted_and_accumulated(rows, wanted):
    H, V = 136, 520
    hidden, W, targets, b, gl = make(rows, H, V, bias=True, masked=0.3, seed=1)
    base_W = torch.randn(V, H, device="cuda").mul_(0.01).bfloat16()
    base_b = torch.randn(V, device="cuda").mul_(0.01).bfloat16()
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, bias=b)
    for accumulate in (False, True):
        buffers = (torch.full_like(hidden, 7.0), base_W.clone(), base_b.clone())
        out = tuple(t if i in wanted else None for i, t in enumerate(buffers))
        lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, out=out, accumulate=accumulate)
        check_status()
        ref = CrossEntropy(hidden, W, targets, bias=b, grad_loss=gl,
                           base_W=base_W if accumulate else None,
                           base_bias=base_b if accumulate else None)
        for i, name in enumerate(("d_hidden", "d_W", "d_bias")):
            if i in wanted:
                assert_close(out[i], getattr(ref, name), getattr(ref, name + "_tol"), name)
        for i, t in enumerate((torch.full_like(hidden, 7.0), base_W, base_b)):
            if i not in wanted:
                assert torch.equal(buffers[i], t)


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_no_row_counts(rows, reduction):
    hidden, W, targets, b, gl = make(rows, 72, 300, bias=True, reduction=reduction)
    hidden.fill_(float("nan"))
    targets.fill_(IGNORE)
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, bias=b, reduction=reduction)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, reduction=reduction)
    check_status()
    for t in (loss, lse, *grads):
        assert torch.count_nonzero(t) == 0 and not torch.isnan(t).any()
    base = torch.randn_like(W)
    out = (None, base.clone(), None)
    lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, reduction=reduction, out=out,
                          accumulate=True)
    assert torch.equal(out[1], base)


def test_no_rows():
    W = torch.randn(300, 72, device="cuda").bfloat16()
    hidden = torch.empty(0, 72, device="cuda", dtype=torch.bfloat16)
    targets = torch.empty(0, device="cuda", dtype=torch.int32)
    for reduction in ("none", "sum", "mean"):
        loss, lse = lm.cross_entropy_f32(hidden, W, targets, reduction=reduction)
        assert loss.shape == ((0,) if reduction == "none" else ()) and lse.shape == (0,)
        assert loss.numel() == 0 or float(loss) == 0.0
    gl = torch.ones((), device="cuda")
    out = (torch.empty_like(hidden), torch.full_like(W, 3.0), None)
    lm.cross_entropy_grad(hidden, W, targets, lse, gl, out=out)
    assert torch.count_nonzero(out[1]) == 0
    out = (None, torch.full_like(W, 3.0), None)
    lm.cross_entropy_grad(hidden, W, targets, lse, gl, out=out, accumulate=True)
    assert torch.equal(out[1], torch.full_like(W, 3.0))


@pytest.mark.parametrize("ignore_index", [IGNORE, 0, 7, None, -2 ** 31, 2 ** 31 - 1])
def test_ignore_index(ignore_index):
    rows, H, V = 150, 64, 40
    hidden, W, targets, b, gl = make(rows, H, V)
    targets[::3] = 7
    targets[1::3] = 0
    if ignore_index is not None:
        targets[5] = ignore_index
    compare(*run_both(hidden, W, targets, b, gl, ignore_index=ignore_index))


@pytest.mark.parametrize("bad", [-1, 300, 2 ** 31 - 1, -2 ** 31])
def test_a_target_outside_the_vocabulary_is_nan(bad):
    hidden, W, targets, b, gl = make(200, 64, 300, masked=0.2, garbage=True)
    rows = (targets != IGNORE).nonzero()[:, 0]
    targets[rows[3]] = bad
    loss, lse, grads, ref = run_both(hidden, W, targets, b, torch.ones(200, device="cuda"),
                                     reduction="none")
    assert torch.isnan(loss[rows[3]]) and int(torch.isnan(loss).sum()) == 1
    assert torch.isnan(grads[0][rows[3]]).all() and torch.isnan(grads[1]).all()
    keep = torch.arange(200, device="cuda") != rows[3]
    assert_close(loss[keep], ref.loss[keep], ref.loss_tol[keep], "loss")
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(grads[0][keep], ref.d_hidden[keep], ref.d_hidden_tol[keep], "d_hidden")


@pytest.mark.parametrize("rows", [20, 200])
def test_entries_taken_out_by_the_bias(rows):
    """-inf takes entries out (whole tiles of them), the type's lowest value does so in effect; a row
    whose target is taken out has an infinite loss and finite gradients; one entry left is sure."""
    H, V = 64, 700
    hidden, W, targets, b, gl = make(rows, H, V, bias=True, reduction="none")
    b[130:600] = float("-inf")
    b[600:640] = torch.finfo(b.dtype).min
    targets[:] = torch.randint(0, 130, (rows,), device="cuda", dtype=torch.int32)
    targets[3] = 200
    targets[5] = 620
    loss, lse, grads, ref = run_both(hidden, W, targets, b, gl, reduction="none")
    keep = torch.arange(rows, device="cuda") != 3
    assert loss[3] == float("inf")
    # (the bound of z at the lowest value is that of its own rounding)
    ref.loss_tol[5] = 2.0 ** -22 * ref.loss[5]
    assert_close(loss[keep], ref.loss[keep], ref.loss_tol[keep], "loss")
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    for g in grads:
        assert torch.isfinite(g).all()
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")
    b.fill_(float("-inf"))
    b[17] = 0.5
    targets.fill_(17)
    loss, lse, grads, ref = run_both(hidden, W, targets, b, gl, reduction="none")
    assert torch.count_nonzero(loss) == 0
    for g in grads:
        assert torch.count_nonzero(g) == 0


def test_rows_sure_of_their_target():
    """A loss near 0 and the gradient's 1 - p keep their bits: the target's logit is an fp32 sum and
    enters by log1p and expm1. The bound is relative: the sums of H products and the logits of the
    other entries, each off by sum_bound of their sizes, are all that separates the two."""
    rows, H, V = 200, 256, 500
    hidden, W, targets, b, gl = make(rows, H, V, reduction="none")
    g = torch.Generator(device="cuda").manual_seed(3)
    hidden = (W[targets.long()].float() * torch.empty(rows, 1, device="cuda").uniform_(
        10, 25, generator=g)).bfloat16()
    loss, lse, grads, ref = run_both(hidden, W, targets, b, torch.ones(rows, device="cuda"),
                                     reduction="none")
    assert float(ref.loss.min()) < 1e-3
    size = (hidden.double().abs() @ W.double().abs().t()).amax(1)
    # nll = log1p(sum exp(z - z_t)): relative error at most twice that of a logit
    tol = ref.loss * (4 * size * H * 2.0 ** -24 + 2.0 ** -18)
    assert_close(loss, ref.loss, tol, "loss")
    # 1 - p of each row shows in the rows of d_hidden: relative to the row's own size
    off = (grads[0].double() - ref.d_hidden).norm(dim=1) / ref.d_hidden.norm(dim=1)
    eps_lse = 2.0 ** -24 * ref.lse.abs() / ref.loss.clamp(max=1)  # lse travels as fp32
    bound = 2 * 2.0 ** -8 + 8 * size * H * 2.0 ** -24 + 2 * eps_lse
    assert (off <= bound).all(), float((off / bound).max())


def test_a_table_of_more_than_2_31_elements():
    """Offsets past 32 bits in W and d_W: targets and ids at the table's end, checked there."""
    rows, H, V = 140, 16384, 140000
    assert V * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    W = torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    for v in range(0, V, 20000):
        W[v:v + 20000] = torch.randn((20000, H), generator=g, device="cuda") * 0.005
    hidden = torch.randn((rows, H), generator=g, device="cuda").bfloat16()
    targets = (V - 1 - torch.arange(rows, device="cuda") * 3).to(torch.int32)
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, reduction="none", ignore_index=None)
    up = torch.ones(rows, device="cuda")
    d_hidden, d_W, _ = lm.cross_entropy_grad(hidden, W, targets, lse, up, reduction="none",
                                             ignore_index=None)
    check_status()
    z = torch.cat([hidden.double() @ W[v:v + 20000].double().t() for v in range(0, V, 20000)], 1)
    tol = (hidden.double().abs() * 0.03).sum(1) * 1e-4 + 1e-5
    want = torch.logsumexp(z, 1)
    assert_close(lse, want, tol, "lse")
    assert_close(loss, want - z.gather(1, targets.long()[:, None])[:, 0], 2 * tol, "loss")
    p = torch.exp(z - want[:, None])
    p[torch.arange(rows, device="cuda"), targets.long()] -= 1.0
    last = V - 600  # the rows of all targets
    want = p[:, last:].t() @ hidden.double()
    size = p[:, last:].abs().t() @ hidden.double().abs()
    assert_close(d_W[last:], want, size * (2.0 ** -8 + 2 * float(tol.max())) + 2.0 ** -8 * want.abs(), "d_W")
    x = lm.embedding(targets, W)
    assert torch.equal(x, W[targets.long()])
    lm.embedding_grad(x, targets, V, out=d_W)
    check_status()
    assert torch.equal(d_W[targets.long()], x)
    seen = torch.zeros(V, dtype=torch.bool, device="cuda")
    seen[targets.long()] = True
    assert not d_W[~seen].any()


def test_nan_and_inf_in_rows_that_count():
    """They stay what they are: that row's loss and gradients, and d_W, are NaN; other rows' are not
    touched."""
    hidden, W, targets, b, gl = make(140, 64, 300, reduction="none")
    hidden[5, 3] = float("nan")
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, reduction="none")
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, gl, reduction="none")
    check_status()
    assert torch.isnan(loss).nonzero().tolist() == [[5]]
    assert torch.isnan(lse).nonzero().tolist() == [[5]]
    assert torch.isnan(grads[0]).all(1).nonzero().tolist() == [[5]]
    assert torch.isnan(grads[0]).any(1).nonzero().tolist() == [[5]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_of_any_size(dtype):
    """Upstream gradients over many binades, zeros and one row alone: the common power of two keeps
    fp16 in range."""
    hidden, W, targets, b, gl = make(260, 128, 700, dtype, reduction="none")
    for gl in (gl * 2.0 ** -20, gl * 2.0 ** 10, torch.zeros_like(gl),
               torch.where(torch.arange(260, device="cuda") == 4, 1.0, 0.0),
               gl * 2.0 ** (torch.arange(260, device="cuda") % 7).float()):
        loss, lse, grads, ref = run_both(hidden, W, targets, b, gl, reduction="none")
        compare(loss, lse, grads, ref)


def test_same_bits_every_time_and_rows_alone():
    """Two runs agree bit for bit; a row's loss and lse do not depend on the other rows, on the lone
    CTAs or CTA pairs that serve their number, or on masked rows between them."""
    hidden, W, targets, b, gl = make(600, 264, 3000, bias=True, masked=0.3, reduction="none")
    how = dict(bias=b, reduction="none")
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, **how)
    first = lm.cross_entropy_grad(hidden, W, targets, lse, gl, **how)
    for _ in range(3):
        again = lm.cross_entropy_f32(hidden, W, targets, **how)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        for a, c in zip(lm.cross_entropy_grad(hidden, W, targets, lse, gl, **how), first):
            assert torch.equal(a, c)
    # more rows than a block of the fold takes on another way
    many = torch.arange(2400, device="cuda") % 600
    big = lm.cross_entropy_f32(hidden[many], W, targets[many], **how)
    assert torch.equal(big[0], loss[many]) and torch.equal(big[1], lse[many])
    for rows in (slice(0, 1), slice(5, 60), slice(100, 300), slice(599, 600)):
        part = lm.cross_entropy_f32(hidden[rows].contiguous(), W, targets[rows].contiguous(), **how)
        assert torch.equal(part[0], loss[rows]) and torch.equal(part[1], lse[rows])
    check_status()


def test_lone_ctas_and_pairs_agree():
    """With CTA pairs off (test build) the same call gives the same loss and gradients within the
    bound, and the same loss bits."""
    hidden, W, targets, b, gl = make(300, 136, 1500, masked=0.1)
    with lm.test_hooks():
        loss, lse, grads, ref = run_both(hidden, W, targets, b, gl)
        lm.set_cta_pairs(False)
        try:
            alone = run_both(hidden, W, targets, b, gl)
        finally:
            lm.set_cta_pairs(True)
    assert torch.equal(alone[0], loss) and torch.equal(alone[1], lse)
    compare(*alone)


def test_nothing_else_is_written():
    """Outputs inside larger buffers, and a workspace of exactly the stated size."""
    rows, H, V = 130, 72, 300
    hidden, W, targets, b, gl = make(rows, H, V, bias=True, masked=0.3)
    edge = 256

    def framed(n, dtype):
        whole = torch.full((n + 2 * edge,), 77, dtype=dtype, device="cuda")
        return whole, whole[edge:edge + n]

    frames = [framed(1, torch.float32), framed(rows, torch.float32),
              framed(rows * H, W.dtype), framed(V * H, W.dtype), framed(V, W.dtype)]
    loss, lse, dh, dw, db = (f[1] for f in frames)
    lm.cross_entropy_f32(
        hidden, W, targets, bias=b, out=(loss.view(()), lse),
        workspace=(ws := framed(lm.cross_entropy_workspace_bytes(rows, H, V), torch.uint8))[1])
    frames.append(ws)
    lm.cross_entropy_grad(
        hidden, W, targets, lse, gl, bias=b, out=(dh.view(rows, H), dw.view(V, H), db),
        workspace=(ws := framed(lm.cross_entropy_grad_workspace_bytes(rows, H, V), torch.uint8))[1])
    frames.append(ws)
    check_status()
    for whole, _ in frames:
        assert (whole[:edge] == 77).all() and (whole[-edge:] == 77).all()
    ref = CrossEntropy(hidden, W, targets, bias=b, grad_loss=gl)
    compare(loss.view(()), lse, (dh.view(rows, H), dw.view(V, H), db), ref)


def test_other_streams_and_two_calls_at_once():
    a = make(300, 128, 2000, seed=1)
    c = make(90, 264, 900, seed=2, masked=0.4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        got = []
        for (hidden, W, targets, b, gl), s in zip((a, c), streams):
            loss, lse = lm.cross_entropy_f32(hidden, W, targets, stream=s)
            got.append((loss, lse, lm.cross_entropy_grad(hidden, W, targets, lse, gl, stream=s)))
    for s in streams:
        s.synchronize()
    check_status()
    for (hidden, W, targets, b, gl), (loss, lse, grads) in zip((a, c), got):
        compare(loss, lse, grads, CrossEntropy(hidden, W, targets, grad_loss=gl))
    # a raw stream handle, and the default stream by its handle
    for s in (streams[0].cuda_stream, 0):
        hidden, W, targets, b, gl = a
        loss, lse = lm.cross_entropy_f32(hidden, W, targets, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(loss, got[0][0]) and torch.equal(lse, got[0][1])


def test_captured_and_replayed():
    """A step in a CUDA graph, replayed on new inputs with another number of rows that count."""
    rows, H, V = 200, 128, 1000
    hidden, W, targets, b, gl = make(rows, H, V, bias=True, masked=0.2, seed=1)

    def step():
        loss, lse = lm.cross_entropy_f32(hidden, W, targets, bias=b)
        return loss, lse, lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse, grads = step()
    for seed, masked in ((2, 0.7), (3, 0.0), (4, 1.0)):
        new = make(rows, H, V, bias=True, masked=masked, seed=seed)
        for old, t in zip((hidden, W, targets, b), new):
            old.copy_(t)
        graph.replay()
        check_status()
        compare(loss, lse, grads, CrossEntropy(hidden, W, targets, bias=b, grad_loss=gl))


def test_the_gradient_against_differences():
    """The summed loss at h + e d and h - e d, every number of which bf16 holds, against the gradient
    along d. The difference errs by the two losses' fp32 errors over 2 e and by its own e^2 / 6
    times the third derivative along d, at most 8 max_v |d . w_v|^3 a row."""
    rows, H, V, e = 16, 64, 200, 1.0 / 16
    g = torch.Generator(device="cuda").manual_seed(11)
    hidden = torch.randint(-16, 17, (rows, H), generator=g, device="cuda").float() / 16
    W = (torch.randint(-16, 17, (V, H), generator=g, device="cuda").float() / 64).bfloat16()
    targets = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    one = torch.ones((), device="cuda")
    _, lse = lm.cross_entropy_f32(hidden.bfloat16(), W, targets, reduction="sum")
    d_hidden, d_W, _ = lm.cross_entropy_grad(hidden.bfloat16(), W, targets, lse, one,
                                             reduction="sum")
    for _ in range(4):
        d = torch.randint(-1, 2, (rows, H), generator=g, device="cuda").float()
        d *= (torch.rand((rows, H), generator=g, device="cuda") < 0.1)
        ends = [lm.cross_entropy_f32((hidden + s * e * d).bfloat16(), W, targets,
                                     reduction="sum")[0].double() for s in (1, -1)]
        difference = float((ends[0] - ends[1]) / (2 * e))
        along = float((d_hidden.double() * d).sum())
        third = float((d.double() @ W.double().t()).abs().amax(1).pow(3).sum()) * 8 / 6 * e * e
        ref = CrossEntropy((hidden + e * d).bfloat16(), W, targets, reduction="sum",
                           grad_loss=one)
        tol = float(ref.loss_tol) / e + third + float((ref.d_hidden_tol * d.abs()).sum())
        assert abs(difference - along) <= tol, (difference, along, tol)
        assert tol < 0.5 * max(1.0, float(d_hidden.double().norm() * d.norm()))


def test_starved_loads_time_out_cleanly():
    """Every wait of the products gives up after its limit, on lone CTAs and on pairs, and the next
    call is right."""
    for rows, V in ((30, 700), (300, 700), (2100, 130000)):  # lone CTAs, pairs, big tiles
        hidden, W, targets, b, gl = make(rows, 64, V)
        with lm.test_hooks():
            lm.device_status(clear=True)
            lm.set_fault_injection(True, wait_limit_ns=5_000_000)
            try:
                loss, lse = lm.cross_entropy_f32(hidden, W, targets)
                lm.cross_entropy_grad(hidden, W, targets, lse, gl)
                torch.cuda.synchronize()
            finally:
                lm.set_fault_injection(False, 0)
            assert lm.device_status(clear=True) & 0xFF == lm.LMHEAD_ERR_TIMEOUT
            lm.set_fault_injection(True, wait_limit_ns=5_000_000)
            try:
                with pytest.raises(lm.LmheadError):
                    lm.cross_entropy_f32(hidden, W, targets, check=True)
            finally:
                lm.set_fault_injection(False, 0)
            compare(*run_both(hidden, W, targets, b, gl))
